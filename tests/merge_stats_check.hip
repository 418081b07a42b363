// Joins (max, sum of exponentials) pairs with the kernels' own merge_stats.
// Standard input: the number of pairs, then max and sum of each; one line of
// output with the joined pair per set.
#include <stdio.h>

#include "../all_reduce_reduction_rank_amd/csrc/products.hpp"

int main() {
  int n;
  while (scanf("%d", &n) == 1) {
    float2 x = make_float2(0.f, 0.f);
    for (int i = 0; i < n; ++i) {
      float2 y;
      if (scanf("%f %f", &y.x, &y.y) != 2) return 1;
      x = i ? ar::merge_stats(x, y) : y;
    }
    printf("%.9g %.9g\n", x.x, x.y);
  }
  return 0;
}
