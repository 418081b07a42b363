// products.hpp -- the product kernels (products_*.hip) by layout and
// epilogue, as the layer operators launch them.
#pragma once

#include <math.h>

#include "product.hpp"

namespace ar {

enum ProductKind : int {
  // A, B: L_K, L_K (x W^T)
  PK_GATED = 0,    // paired; c = {act(g) u, g, u} (c[1], c[2] may be null)
  PK_STORE_NT,     // c[0] = C
  PK_STATS,        // per row: c[0] = (max, sum of exponentials) of the tile, c[1] = target's logit
  PK_DLOGITS,      // a[1] = lse; c[0] = (exp(C - lse) - onehot(target)) * grad
  // A, B: L_K, L_R (dy W)
  PK_GATED_BWD,    // C = dh, a[1], b[1] = g, u; c = {dg, du, h}
  // Both products that end a backward pass, in one launch: problems by layout
  // (Problem::mode GRAD_*)
  PK_GRADS,
};

// Problem::mode of PK_GRADS
enum : uint32_t {
  GRAD_TN = 1,       // A, B: L_R, L_R (dy^T x): c[0] = C; otherwise L_K, L_R (dy W):
  GRAD_ADD = 2,      // add the fp32 sum so far (c[1])
  GRAD_PARTIAL = 4,  // write the fp32 sum (c[1]) instead of the result (c[0])
};
// ProductArgs::act
enum : uint32_t { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };

// The (max, sum of exp(v - max)) pairs of two sets of values, joined: each sum
// is scaled by exp(its max - the joint max).  An infinite joint max shifts by 0
// instead, so that +inf gives an infinite sum (not inf - inf).  An empty set, or
// one of -inf alone, is (-inf, 0); its own max in the exponent weighs it 0
// wherever the other set lies, and a sum of NaN stays NaN.
__host__ __device__ __forceinline__ float stats_shift(float top) { return fabsf(top) == INFINITY ? 0.f : top; }
__host__ __device__ __forceinline__ float2 merge_stats(float2 x, float2 y) {
  const float top = fmaxf(x.x, y.x), shift = stats_shift(top);
  return make_float2(top, x.y * expf(x.x - shift) + y.y * expf(y.x - shift));
}

// Bytes of c[2] for MAX_SHARES blocks of every rank's [rows, cols] result; 0 where
// the result has tiles enough by itself (128 of 64 x 128) and is not shared.
constexpr uint64_t share_bytes(int n, uint64_t rows, uint64_t cols) {
  return (uint64_t)n * rows * cols <= 128ull * 64 * 128 ? (MAX_SHARES * rows * cols * 4 + 255) & ~255ull : 0;
}

// Rows down to a bf16 intermediate's second terms (Problem::fold): half the rows
// of the tile that will read it, or 0 where the intermediate keeps one term.
// With up to 32 rows the second terms cost next to nothing (they fill rows of
// a tile that would be empty), and few roundings do not average out: with one
// term, results of one-token calls came out up to 1.5 times as far from the
// exact ones as the result's own rounding puts them, with two 1.00 times.
// With 33 to 64 rows they would take a tile of twice the rows (the down
// projection of 64 rows x 8 x 1728 x 5120: 38 -> 48 us) for roundings that
// average out (1.41 to 1.43 times).
constexpr uint32_t fold_of(uint64_t rows, int dtype) {
  return dtype != DT_BF16 || rows == 0 ? 0 : rows <= Thin::BM / 2 ? Thin::BM / 2 : rows <= Flat::BM / 2 ? Flat::BM / 2 : 0;
}

// Tile class that a launch of this plan takes (its problems are final).
enum TileClass : int { TILE_LARGE = 0, TILE_SMALL, TILE_TALL, TILE_FLAT, TILE_SPLIT, TILE_THIN, TILE_CLASSES };
struct TileChoice {
  int tile;
  uint32_t shares;  // workgroups per tile's K, of the problems that may share
};
TileChoice product_tile(int kind, int dtype, const ProductPlan& plan, int device);
// Columns of C a tile of a class that is not paired covers: PK_STATS writes
// one partial per row and that many columns.
constexpr uint32_t tile_cols(int tile) {
  constexpr uint32_t cols[TILE_CLASSES] = {Large::BN, Small::BN, Tall::BN, Flat::BN, Split::BN, Thin::BN};
  return cols[tile];
}
// The fewest columns a tile covers in a product of that many rows: Thin tiles are
// for few rows (product_tile), the others have 64 columns or more.
constexpr uint32_t THIN_MAX_ROWS = 4 * Thin::BM;
constexpr uint32_t min_tile_cols(uint64_t rows) { return rows <= THIN_MAX_ROWS ? Thin::BN : Split::BN; }
static_assert(Split::BN <= Tall::BN && Split::BN <= Flat::BN && Split::BN <= Small::BN && Split::BN <= Large::BN, "");
// Order in which a class adds up K (ProductPlan::k_parts).
constexpr uint32_t tile_k_parts(int tile) { return tile == TILE_SPLIT ? Split::WK : tile == TILE_THIN ? Thin::WK : 1; }

// Products read rows that start on 16-byte boundaries.  A matrix whose rows do
// not (an odd width) is copied into the workspace once per call, its rows
// padded with zeros to whole 16-byte chunks.  Measured against reading such
// rows in place through registers, element by element at their ends: the
// copies cost less than the products gain (cross entropy step of 611 rows,
// width 1003, vocabulary 10007 over 3 ranks, bf16: 288 -> 170 us).
class Packer {
 public:
  struct Rows {
    const char* p;
    uint64_t ld;
  };
  // Bytes of the copy of a [rows, cols] matrix; 0 if none is needed.
  static uint64_t bytes(uint64_t rows, uint64_t cols, uint64_t es) {
    return (cols * es) % 16 ? copy_bytes(rows, cols, es) : 0;
  }
  static uint64_t copy_bytes(uint64_t rows, uint64_t cols, uint64_t es) {
    return (rows * pitch(cols, es) * es + 255) & ~255ull;
  }
  static uint64_t pitch(uint64_t cols, uint64_t es) { return (cols * es + 15) / 16 * 16 / es; }

  Packer(char* space, uint64_t es) : space_(space), es_(es) {}
  // A row-major [rows, cols] matrix without gaps, or its copy to be.
  Rows rows(const void* src, uint64_t rows, uint64_t cols);
  // The copy of a [rows, cols] matrix with zeros in the rows whose target is
  // outside [0, vocab).
  Rows live_rows(const void* src, uint64_t rows, uint64_t cols, const int64_t* target, uint64_t vocab);
  // Make the copies (one kernel, or none).
  hipError_t launch(hipStream_t stream) const;

  static constexpr int MAX = 5 * MAX_RANKS;
  struct Entry {
    const char* src;
    char* dst;
    uint64_t rows;
    uint32_t cols, chunks;  // elements, 16-byte chunks of a row
    uint32_t first;         // first workgroup
    uint32_t live;          // only rows with a target are copied
  };
  struct Args {
    Entry e[MAX];
    const int64_t* target;
    uint64_t vocab;
    int32_t n, es;
  };

 private:
  Rows copy(const void* src, uint64_t rows, uint64_t cols, uint32_t live);

  char* space_;
  uint64_t es_;
  Args a_ = {};
  uint64_t blocks_ = 0;
};

hipError_t launch_products_bf16(int kind, ProductPlan& plan, int device, hipStream_t stream);
hipError_t launch_products_f32(int kind, ProductPlan& plan, int device, hipStream_t stream);
inline hipError_t launch_products(int kind, int dtype, ProductPlan& plan, int device, hipStream_t stream) {
  return dtype == DT_BF16 ? launch_products_bf16(kind, plan, device, stream)
                          : launch_products_f32(kind, plan, device, stream);
}

// A PK_GRADS plan: dx problems first (`head` of them), then GRAD_TN.  One launch;
// two where dx's operand has second terms, which fix dx's tile class.
hipError_t launch_grads(int dtype, ProductPlan& plan, int device, hipStream_t stream);

}  // namespace ar
