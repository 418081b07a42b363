// products.hip -- tile choice of the product kernels.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "products.hpp"

namespace ar {

TileShape product_tile(int kind, const ProductPlan& plan, int device) {
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device) != hipSuccess || cus < 1) cus = 256;
  const uint32_t half = kind == PK_GATED ? 2 : 1;
  uint64_t tiles = 0;
  for (int i = 0; i < plan.a.nprob; ++i) {
    const Problem& p = plan.a.p[i];
    tiles += (((uint64_t)p.m + 255) / 256) * (((uint64_t)p.n * half + 255) / 256);
  }
  const bool large = plan.aligned && tiles >= (uint64_t)cus;
  return large ? TileShape{256, 256 / half} : TileShape{128, 128 / half};
}

}  // namespace ar
