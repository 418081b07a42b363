// Host check of fold_items (heads.hpp), compiled and run by tests/test_heads_limits.py.
#include <cstdio>

#include "../all_reduce_reduction_rank_amd/csrc/heads.hpp"

int main() {
  int bad = 0;
  for (uint32_t threads : {64u, 256u, 512u})
    for (int bits = 0; bits <= 32; ++bits)
      for (int64_t d = -2; d <= 2; ++d) {
        const int64_t items = ((int64_t)1 << bits) + d;
        if (items < 0) continue;
        const ar::Fold f = ar::fold_items(items, threads);
        const bool ok = (uint64_t)f.x * threads < (1ull << 32) && (uint64_t)f.x * f.folds >= (uint64_t)items &&
                        (items == 0 || (uint64_t)f.x * (f.folds - 1) < (uint64_t)items) && f.folds * 8ull <= 65535;
        if (!ok) ++bad, printf("%lld items of %u threads: %u x %u\n", (long long)items, threads, f.x, f.folds);
      }
  return bad != 0;
}
