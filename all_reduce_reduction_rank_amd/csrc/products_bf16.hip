// products_bf16.hip -- the product kernels for bf16 payloads.
#include "product_kernels.hpp"

namespace ar {

hipError_t launch_products_bf16(int kind, ProductPlan& plan, int device, hipStream_t stream) {
  return launch_typed<DT_BF16>(kind, plan, device, stream);
}

}  // namespace ar
