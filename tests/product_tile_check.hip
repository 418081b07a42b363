// Prints the tile class product_tile takes for each product named on standard
// input, one per line: kind dtype head nprob, then m n k nseg fold mode of every
// problem.
#include <stdio.h>

#include "../all_reduce_reduction_rank_amd/csrc/products.hpp"

namespace ar {  // nothing is launched here
hipError_t launch_products_bf16(int, ProductPlan&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_products_f32(int, ProductPlan&, int, hipStream_t) { return hipSuccess; }
}  // namespace ar

int main() {
  int kind, dtype, head, nprob;
  while (scanf("%d %d %d %d", &kind, &dtype, &head, &nprob) == 4) {
    ar::ProductPlan plan;
    plan.head = head;
    for (int i = 0; i < nprob; ++i) {
      unsigned long long m, n, k;
      unsigned nseg, fold, mode;
      if (scanf("%llu %llu %llu %u %u %u", &m, &n, &k, &nseg, &fold, &mode) != 6) return 1;
      ar::Problem* p = plan.add(m, n, k, (k + 7) / 8 * 8, (k + 7) / 8 * 8, (n + 7) / 8 * 8);
      p->nseg = nseg;
      p->fold = fold;
      p->mode = mode;
    }
    printf("%d\n", ar::product_tile(kind, dtype, plan, 0));
  }
  return 0;
}
