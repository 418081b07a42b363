// products_f32.hip -- the product kernels for f32 payloads.
#include "product_kernels.hpp"

namespace ar {

hipError_t launch_products_f32(int kind, ProductPlan& plan, int device, hipStream_t stream) {
  return launch_typed<DT_F32>(kind, plan, device, stream);
}

}  // namespace ar
