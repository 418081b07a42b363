// Prints the tile class product_tile takes, and the workgroups that share a
// tile's K, for each product named on standard input, one per line: kind dtype
// head may_share k_parts nprob, then m n k nseg fold mode of every problem.
#include <stdio.h>

#include "../all_reduce_reduction_rank_amd/csrc/products.hpp"

namespace ar {  // nothing is launched here
hipError_t launch_products_bf16(int, ProductPlan&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_products_f32(int, ProductPlan&, int, hipStream_t) { return hipSuccess; }
}  // namespace ar

int main() {
  int kind, dtype, head, share, parts, nprob;
  while (scanf("%d %d %d %d %d %d", &kind, &dtype, &head, &share, &parts, &nprob) == 6) {
    ar::ProductPlan plan;
    plan.head = head;
    plan.may_share = share != 0;
    plan.k_parts = (uint32_t)parts;
    for (int i = 0; i < nprob; ++i) {
      unsigned long long m, n, k;
      unsigned nseg, fold, mode;
      if (scanf("%llu %llu %llu %u %u %u", &m, &n, &k, &nseg, &fold, &mode) != 6) return 1;
      ar::Problem* p = plan.add(m, n, k, (k + 7) / 8 * 8, (k + 7) / 8 * 8, (n + 7) / 8 * 8);
      p->nseg = nseg;
      p->fold = fold;
      p->mode = mode;
    }
    const ar::TileChoice c = ar::product_tile(kind, dtype, plan, 0);
    printf("%d %u\n", c.tile, c.shares);
  }
  return 0;
}
