// products.hip -- tile choice of the product kernels, and copies of matrices
// whose rows are not whole 16-byte chunks.
//
// A launch takes the tile class with the smallest estimated time.  A
// workgroup of class c takes fixed + steps x (alone | full) us, a step being
// 128 bytes of k (of each wave's part of K): `alone` while its CU runs no
// other and no round of workgroups is behind it, `full` with as many as fit.
// Measured on bf16 products of 8 ranks [m, 5120] x [1728 pairs, 5120] (80 steps)
// and [m, 1728] x [5120, 1728] (27):
//
//   us            m = 64   128   256   512  1024 |   64   128   256   512  1024
//   Large            143   150   172   171   302 |   51    55    60   111   162
//   Small             96   110   125   218   373 |   39    46    76   106   174
//   Flat              65    99   157   247   490 |   38    47    67   119   214
//   Split             73   116   185   347   687 |   42    60   108   205   377
//   Thin (m = 1)      55                         |   31
//
// One small product, [512, 4096] x [1024, 4096]: 83, 50, 31, 16 us.  Thin
// is for up to 64 rows where other tiles would be few (bf16) or mostly empty
// (fp32): logits of 27 rows, width 7424, 4 x 296 columns in fp32 137 us in Split, 35 in
// Thin.  With more tiles than run at once it reads the weights again for every
// 16 rows: [17, 7360] x [6816 pairs, 7360] x 2 and back, bf16, 125 us in Flat, 144
// in Thin; fp32 loss step [43, 3172] x 60815 over 2 ranks 1228 in Split, 1456 in
// Thin, but the loss of [30, 1408] x 101216 over 3 ranks 237 and 182.
//
// A product with few tiles and a long K (a gradient summed over the vocabulary)
// has 2 to 16 workgroups share each tile's K, where the shorter sums are worth a
// second kernel that adds them: fp32 [11, 7522] x [7522, 314], 5 tiles of 64
// columns, and its gradients 313 us unshared, 95 with 16 shares.
//
// fp32 runs 16 times as many instructions per byte, so its steps cost what
// its matrix instructions do, and the choice is which tile fills the CUs most
// evenly: two ranks of [1024, 1024] x [8000, 1024] 290 us in Small and 315 in
// Tall, but [1024, 8000] x [8000, 1024] 536, 307, Split 297 (all from a cold clock;
// after a second of such calls the first takes 265).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "products.hpp"

namespace ar {

namespace {

struct ClassCost {
  uint32_t bm, bn, parts, resident;  // parts: of K; resident: workgroups per CU
  double fixed, alone, full;         // us: of a workgroup, of a step
  double f32;                        // fp32 matrix instructions: time over Tall's
};
constexpr ClassCost COST[TILE_CLASSES] = {
    {Large::BM, Large::BN, Large::WK, 1, 9.0, 1.75, 1.75, 0.0},  // bf16 only
    {Small::BM, Small::BN, Small::WK, 2, 4.0, 1.15, 1.35, 0.96},
    {Tall::BM, Tall::BN, Tall::WK, 3, 4.0, 0.75, 1.2, 1.0},      // fp32 only
    {Flat::BM, Flat::BN, Flat::WK, 2, 4.0, 0.75, 0.95, 0.0},  // bf16 only
    {Split::BM, Split::BN, Split::WK, 1, 4.5, 0.8, 1.6, 1.22},
    {Thin::BM, Thin::BN, Thin::WK, 2, 4.5, 0.25, 0.6, 1.22},
};
// Sharing a tile's K among workgroups: a second kernel, and the sums written
// and read.
constexpr double SHARE_US = 4.0, SHARE_BYTES_PER_US = 3e6;
constexpr double F32_FLOPS_PER_CU_US = 0.55e6;  // of 0.61e6 (16x16x4 at 2.4 GHz)

constexpr int PACK_THREADS = 256, PACK_CHUNKS = 4;  // chunks per thread

typedef uint32_t v4u_any __attribute__((ext_vector_type(4), aligned(2)));

// Each thread makes 16-byte chunks of the copies: one load at any (element)
// address for a whole chunk, element by element at a row's end, so that
// nothing past the matrix is read.
__global__ __launch_bounds__(PACK_THREADS) void pack_kernel(Packer::Args a) {
  int q = 0;
  while (q + 1 < a.n && blockIdx.x >= a.e[q + 1].first) ++q;
  const Packer::Entry& e = a.e[q];
  const uint64_t total = e.rows * e.chunks;
  const uint32_t per = 16 / a.es;
  const uint64_t base = (uint64_t)(blockIdx.x - e.first) * (PACK_THREADS * PACK_CHUNKS) + threadIdx.x;
#pragma unroll
  for (int i = 0; i < PACK_CHUNKS; ++i) {
    const uint64_t t = base + (uint64_t)i * PACK_THREADS;
    if (t >= total) break;
    const uint64_t row = t / e.chunks;
    const uint32_t col = (uint32_t)(t % e.chunks) * per;
    const char* src = e.src + (row * e.cols + col) * a.es;
    v4u v = {0, 0, 0, 0};
    const int64_t target = e.live ? a.target[row] : 0;
    if (e.live && (target < 0 || (uint64_t)target >= a.vocab)) {
    } else if (col + per <= e.cols) {
      v = *(const v4u_any*)src;
    } else if (a.es == 2) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < e.cols) v[j / 2] |= (uint32_t)((const uint16_t*)src)[j] << (16 * (j % 2));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j < e.cols) v[j] = ((const uint32_t*)src)[j];
    }
    *(v4u*)(e.dst + t * 16) = v;
  }
}

}  // namespace

Packer::Rows Packer::rows(const void* src, uint64_t rows, uint64_t cols) {
  if ((cols * es_) % 16 == 0 || rows == 0) return {(const char*)src, pitch(cols, es_)};
  return copy(src, rows, cols, 0);
}

Packer::Rows Packer::live_rows(const void* src, uint64_t rows, uint64_t cols, const int64_t* target, uint64_t vocab) {
  if (rows == 0) return {(const char*)src, pitch(cols, es_)};
  a_.target = target;
  a_.vocab = vocab;
  return copy(src, rows, cols, 1);
}

Packer::Rows Packer::copy(const void* src, uint64_t rows, uint64_t cols, uint32_t live) {
  for (int i = 0; i < a_.n; ++i)  // the same matrix on several ranks
    if (a_.e[i].src == (const char*)src && a_.e[i].rows == rows && a_.e[i].cols == cols && a_.e[i].live == live)
      return {a_.e[i].dst, pitch(cols, es_)};
  Entry& e = a_.e[a_.n++];
  e.src = (const char*)src;
  e.dst = space_;
  e.rows = rows;
  e.cols = (uint32_t)cols;
  e.live = live;
  e.chunks = (uint32_t)(pitch(cols, es_) * es_ / 16);
  e.first = (uint32_t)blocks_;
  blocks_ += (rows * e.chunks + PACK_THREADS * PACK_CHUNKS - 1) / (PACK_THREADS * PACK_CHUNKS);
  space_ += copy_bytes(rows, cols, es_);
  return {e.dst, pitch(cols, es_)};
}

hipError_t Packer::launch(hipStream_t stream) const {
  if (!blocks_) return hipSuccess;
  if (blocks_ >= (1ull << 31)) return hipErrorInvalidValue;
  Args a = a_;
  a.es = (int32_t)es_;
  hipLaunchKernelGGL(pack_kernel, dim3((unsigned)blocks_), dim3(PACK_THREADS), 0, stream, a);
  return hipGetLastError();
}

TileChoice product_tile(int kind, int dtype, const ProductPlan& plan, int device) {
  int n_cu = 0;
  if (hipDeviceGetAttribute(&n_cu, hipDeviceAttributeMultiprocessorCount, device) != hipSuccess || n_cu < 1) n_cu = 256;
  const double cus = n_cu;
  const uint32_t half = kind == PK_GATED ? 2 : 1;
  const uint64_t per_step = dtype == DT_BF16 ? 64 : 32;  // k of 128 bytes
  const bool reads_terms = kind == PK_STORE_NT || kind == PK_GRADS;  // other kinds write them
  const int sharing = plan.sharing();
  uint32_t max_m = 0, fold = 0;
  double results = 0;  // values of the problems that may share
  for (int i = 0; i < plan.a.nprob; ++i) {
    const Problem& p = plan.a.p[i];
    max_m = p.m > max_m ? p.m : max_m;
    fold = p.fold > fold ? p.fold : fold;  // the same in all of a launch's problems
    if (i < sharing) results += (double)(p.m - p.fold) * p.n;
  }
  TileChoice best = {TILE_SMALL, 1};
  double best_us = 1e30;
  for (int c = 0; c < TILE_CLASSES; ++c) {
    const ClassCost& k = COST[c];
    if (c == TILE_TALL ? dtype == DT_BF16 : (c == TILE_LARGE || c == TILE_FLAT) && dtype != DT_BF16) continue;
    if (c == TILE_LARGE && fold) continue;
    if (c == TILE_THIN && max_m > THIN_MAX_ROWS) continue;
    if (fold && reads_terms && k.bm != 2 * fold) continue;
    if (plan.k_parts && k.parts != plan.k_parts) continue;
    for (uint32_t shares = 1; shares <= (sharing ? MAX_SHARES : 1); shares *= 2) {
      double tiles = 0, work = 0, longest = 0, shortest = 1e30;  // work: steps of all tiles
      for (int i = 0; i < plan.a.nprob; ++i) {
        const Problem& p = plan.a.p[i];
        const uint32_t by = i < sharing ? shares : 1;
        const double t = (double)((p.m + k.bm - 1) / k.bm) * (double)(((uint64_t)p.n * half + k.bn - 1) / k.bn) * by;
        if (t == 0) continue;
        const uint64_t steps = (uint64_t)p.nseg * ((p.k + per_step - 1) / per_step);
        const double s = (double)((steps + k.parts * by - 1) / (k.parts * by));
        tiles += t;
        work += t * s;
        longest = s > longest ? s : longest;
        shortest = s < shortest ? s : shortest;
      }
      if (tiles == 0) continue;
      const double slots = cus * k.resident;
      const double rounds = (double)(uint64_t)(tiles / slots);
      const double rest = tiles - rounds * slots;
      // every 16 rows read the weights again: from the caches, if all of them run
      // at once; fp32 gains more by half as many empty rows as by fewer reads
      if (c == TILE_THIN && rounds > 0 && max_m > (uint32_t)Thin::BM * (dtype == DT_BF16 ? 1 : 2)) continue;
      double us;
      if (dtype != DT_BF16) {
        // matrix instructions: a CU works its tiles off one after the other,
        // however many share it (`one`: a tile by itself, one wave per SIMD)
        const double mm = k.f32 * 2.0 * k.bm * k.bn * per_step * k.parts / F32_FLOPS_PER_CU_US;
        const double per = mm * k.resident > k.full ? mm : k.full / k.resident;
        const double one = 1.2 * mm > k.alone ? 1.2 * mm : k.alone;
        const double each = (double)(uint64_t)((tiles + cus - 1) / cus);
        const double turns = (double)(uint64_t)((each + k.resident - 1) / k.resident);
        const double busy = longest == shortest ? each * longest * per : (work / cus + 0.5 * shortest) * per;
        us = turns * k.fixed + (busy > longest * one ? busy : longest * one);
      } else if (rounds == 0) {
        us = k.fixed + longest * (rest <= cus ? k.alone : k.full);
      } else if (longest == shortest) {
        us = rounds * (k.fixed + longest * k.full) +
             (rest == 0 ? 0 : k.fixed + longest * (rest <= cus && k.resident > 1 ? k.alone : k.full));
      } else {  // long tiles first, and none longer than the whole
        const double all = (work / slots + 0.5 * shortest) * k.full;
        us = tiles / slots * k.fixed + (all > longest * k.full ? all : longest * k.full);
      }
      if (shares > 1) us += SHARE_US + shares * results * 8 / SHARE_BYTES_PER_US;
      if (us < best_us) {
        best_us = us;
        best = {c, shares};
      }
    }
  }
  return best;
}

hipError_t launch_grads(int dtype, ProductPlan& plan, int device, hipStream_t stream) {
  if (plan.head == 0 || plan.a.p[0].fold == 0) return launch_products(PK_GRADS, dtype, plan, device, stream);
  ProductPlan rest = plan;
  rest.may_share = false;
  rest.a.nprob = plan.a.nprob - plan.head;
  rest.head = 0;
  for (int i = 0; i < rest.a.nprob; ++i) rest.a.p[i] = plan.a.p[plan.head + i];
  plan.a.nprob = plan.head;
  const hipError_t e = launch_products(PK_GRADS, dtype, plan, device, stream);
  return e != hipSuccess ? e : launch_products(PK_GRADS, dtype, rest, device, stream);
}

}  // namespace ar
