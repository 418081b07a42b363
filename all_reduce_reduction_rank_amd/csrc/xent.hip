// xent.hip -- softmax cross entropy of a linear layer whose vocabulary is
// split over the ranks (ar_linear_cross_entropy and its backward pass).
// The logits l = x W^T are never stored.
//
// Forward: each tile of logits is reduced in registers to its rows' maximum
// and sum of exponentials (and the target's logit, if it lies in the tile).
// A second kernel joins the tiles of every rank, the all-reduce of the split
// softmax: lse = log sum_v exp(l_v), loss = lse - l_target, stored to every
// rank.  It reads 8 bytes per row and tile (32 to 256 columns).
//
// Backward, one piece of each rank's vocabulary at a time: recompute the
// piece's logits, store d = (exp(l - lse) - onehot) grad for the piece only,
// then dx += d W and dW = d^T x.  dx is added up over the pieces in fp32 and
// rounded once; d is rounded to bf16 for the matrix cores, over a common scale
// (scale_kernel) or, with up to 32 rows, in two terms (fold_of).  The piece caps
// the memory d takes.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/ar.h"
#include "layer.hpp"
#include "products.hpp"

using namespace ar;

namespace {

struct CombineArgs {
  const float2* part[MAX_RANKS];  // [tiles of the rank][rows]
  float* loss[MAX_RANKS];
  float* lse[MAX_RANKS];
  uint32_t tiles[MAX_RANKS], max_tiles;
  const float* at;  // target's logit per row
  const int64_t* target;
  uint64_t vocab;
  uint32_t rows;
  int32_t nranks;
};

constexpr int COMBINE_THREADS = 1024;

// Joins the partials of R rows (a power of two up to 64) per workgroup:
// thread (slot, row) takes every (1024 / R)-th tile of its row, then the
// slots are joined in LDS.  64 rows side by side read whole lines; with
// fewer rows in the call all threads still work.
__global__ __launch_bounds__(COMBINE_THREADS) void combine_kernel(CombineArgs a, uint32_t rows_per_wg) {
  __shared__ float2 s[COMBINE_THREADS];
  const uint32_t slots = COMBINE_THREADS / rows_per_wg;
  const uint32_t r = threadIdx.x % rows_per_wg, slot = threadIdx.x / rows_per_wg;
  const uint64_t row = (uint64_t)blockIdx.x * rows_per_wg + r;
  float2 x = make_float2(-INFINITY, 0.f);
  if (row < a.rows) {
    // one tile of every rank at a time: their loads go out together
    for (uint32_t t = slot; t < a.max_tiles; t += slots) {
      float2 y[MAX_RANKS];
#pragma unroll
      for (int q = 0; q < MAX_RANKS; ++q) {
        y[q] = make_float2(-INFINITY, 0.f);
        if (q < a.nranks && t < a.tiles[q]) y[q] = a.part[q][(uint64_t)t * a.rows + row];
      }
#pragma unroll
      for (int q = 0; q < MAX_RANKS; ++q)
        if (q < a.nranks) x = merge_stats(x, y[q]);
    }
  }
  s[threadIdx.x] = x;
  __syncthreads();
  for (uint32_t half = slots / 2; half > 0; half /= 2) {
    if (slot < half) s[threadIdx.x] = merge_stats(s[threadIdx.x], s[threadIdx.x + half * rows_per_wg]);
    __syncthreads();
  }
  if (slot == 0 && row < a.rows) {
    x = s[r];
    const float lse = stats_shift(x.x) + logf(x.y);
    const int64_t t = a.target[row];
    const float loss = t >= 0 && (uint64_t)t < a.vocab ? lse - a.at[row] : 0.f;
    for (int q = 0; q < a.nranks; ++q) {
      a.loss[q][row] = loss;
      a.lse[q][row] = lse;
    }
  }
}

// The scale of a call's d: the largest finite |grad_loss| of the rows with
// loss (1 if there is none).  d / scale is what gets rounded to bf16.  With a
// mean loss every row has the same grad_loss, and each row's largest entry is
// about -grad_loss: stored as they are they would all be off by the same
// fraction, that constant's rounding, and so would dx and dw as a whole
// (measured at 3700 rows with loss: 0.0031 relative to the exact dw, with the
// scale 0.0024).  Over the scale that entry is -1.
__global__ __launch_bounds__(COMBINE_THREADS) void scale_kernel(const float* grad, const int64_t* target,
                                                                uint64_t vocab, uint32_t rows, float* out) {
  __shared__ float s[COMBINE_THREADS / 64];
  float top = 0.f;
  for (uint32_t i = threadIdx.x; i < rows; i += COMBINE_THREADS) {
    const float g = fabsf(grad[i]);
    const int64_t t = target[i];
    if (t >= 0 && (uint64_t)t < vocab && g < INFINITY) top = fmaxf(top, g);
  }
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < COMBINE_THREADS / 64; ++w) top = fmaxf(top, s[w]);
    *out = top > 0.f ? top : 1.0f;
  }
}

// d of all ranks, unless the caller says otherwise or 256 columns of each take more
constexpr uint64_t DEFAULT_PIECE_BYTES = 1ull << 30;

struct XentShape {
  uint64_t rows, hidden, vocab, es;
  uint64_t shard[MAX_RANKS], start[MAX_RANKS], max_shard;
  uint64_t part_tiles;  // partials per row and rank, at the narrowest tile that many rows may take
  uint64_t pack_bytes;  // copies of every rank's x and w, where their rows are not whole 16-byte chunks
  uint64_t live_bytes;  // the same with x copied always
};

XentShape shape_of(int n, size_t rows, size_t hidden, size_t vocab, int dtype) {
  XentShape s;
  s.rows = rows, s.hidden = hidden, s.vocab = vocab;
  s.es = dtype == DT_BF16 ? 2 : 4;
  const uint64_t b = (s.vocab + n - 1) / n;
  for (int r = 0; r < n; ++r) {
    s.start[r] = umin((uint64_t)r * b, s.vocab);
    s.shard[r] = umin((uint64_t)(r + 1) * b, s.vocab) - s.start[r];
  }
  s.max_shard = b;
  s.part_tiles = (b + min_tile_cols(rows) - 1) / min_tile_cols(rows);
  s.pack_bytes = s.live_bytes = 0;
  for (int r = 0; r < n; ++r) {
    const uint64_t w = Packer::bytes(s.shard[r], s.hidden, s.es);
    s.pack_bytes += Packer::bytes(s.rows, s.hidden, s.es) + w;
    s.live_bytes += Packer::copy_bytes(s.rows, s.hidden, s.es) + w;
  }
  return s;
}

ar_status check_shape(int n, size_t rows, size_t hidden, size_t vocab, int dtype) {
  if (n < 1 || n > MAX_RANKS || dtype < 0 || dtype > 2) return AR_ERR_INVALID;
  if (hidden < 1 || vocab < 1) return AR_ERR_INVALID;
  if (dtype == DT_I32) return AR_ERR_UNSUPPORTED;
  if (rows > LAYER_MAX_ROWS || hidden > LAYER_MAX_WIDTH || vocab > LAYER_MAX_ROWS) return AR_ERR_TOO_LARGE;
  return AR_OK;
}

// Vocabulary rows per rank and piece: the caller's, or as many as keep d of
// all ranks within DEFAULT_PIECE_BYTES; whole tiles, at least one (256 columns,
// however many rows there are).
uint64_t piece_of(const XentShape& s, int n, size_t piece) {
  uint64_t p = piece ? (uint64_t)piece : DEFAULT_PIECE_BYTES / umax(1, (uint64_t)n * s.rows * s.es);
  p = umin(p, LAYER_MAX_WIDTH);
  p = umax(256, p / 256 * 256);
  return umin(p, (s.max_shard + 7) / 8 * 8);
}

struct BackwardSpace {
  uint64_t piece, d_bytes, acc_bytes;  // per rank
  uint32_t fold;                       // d: rows down to its second terms, 0: none
  uint64_t share;                      // dx's shares
  uint64_t scale_bytes;                // the scale of d, of all ranks
  uint64_t bytes(int n) const { return (uint64_t)n * (d_bytes + acc_bytes + share) + scale_bytes; }
};
BackwardSpace space_of(const XentShape& s, int n, int dtype, size_t piece) {
  BackwardSpace b;
  b.piece = piece_of(s, n, piece);
  b.fold = fold_of(s.rows, dtype);
  b.d_bytes = layer_align((b.fold + s.rows) * b.piece * s.es);
  b.share = share_bytes(n, s.rows, s.hidden);
  b.scale_bytes = dtype == DT_BF16 && !b.fold ? layer_align(sizeof(float)) : 0;
  // fp32 gradients add up in dx itself
  b.acc_bytes = dtype == DT_BF16 && b.piece < s.max_shard ? layer_align(s.rows * s.hidden * 4) : 0;
  return b;
}

}  // namespace

extern "C" {

size_t ar_linear_cross_entropy_workspace(int nranks, size_t rows, size_t hidden, size_t vocab, ar_dtype dtype,
                                         int backward, size_t piece) {
  if (check_shape(nranks, rows, hidden, vocab, (int)dtype) != AR_OK || rows == 0) return 0;
  const XentShape s = shape_of(nranks, rows, hidden, vocab, (int)dtype);
  if (backward) {
    const BackwardSpace b = space_of(s, nranks, (int)dtype, piece);
    return (size_t)(b.bytes(nranks) + s.live_bytes);
  }
  return (size_t)(layer_align(s.rows * 4) + (uint64_t)nranks * layer_align(s.part_tiles * s.rows * 8) + s.pack_bytes);
}

ar_status ar_linear_cross_entropy(int nranks, const void* const* x, const void* const* w, const int64_t* target,
                                  float* const* loss, float* const* lse, size_t rows, size_t hidden, size_t vocab,
                                  ar_dtype dtype, void* workspace, size_t workspace_bytes, ar_stream_t stream) {
  const ar_status st = check_shape(nranks, rows, hidden, vocab, (int)dtype);
  if (st != AR_OK) return st;
  if (!x || !w || !loss || !lse) return AR_ERR_INVALID;
  if (rows == 0) return AR_OK;
  const XentShape s = shape_of(nranks, rows, hidden, vocab, (int)dtype);
  const uint64_t at_bytes = layer_align(s.rows * 4), part_bytes = layer_align(s.part_tiles * s.rows * 8);
  const uint64_t need = at_bytes + (uint64_t)nranks * part_bytes + s.pack_bytes;
  LayerBuffers b;
  for (int r = 0; r < nranks; ++r) {
    b.in(x[r], s.rows * s.hidden * s.es);
    b.in(w[r], s.shard[r] * s.hidden * s.es);
    b.out(loss[r], s.rows * 4, 4);
    b.out(lse[r], s.rows * 4, 4);
  }
  b.in(target, s.rows * 8, 8);
  b.out(workspace, need);
  if (!b.ok()) return AR_ERR_INVALID;
  if (workspace_bytes < need) return AR_ERR_TOO_LARGE;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return AR_ERR_HIP;
  char* ws = (char*)workspace;

  CombineArgs c = {};
  ProductPlan plan;
  plan.a.target = target;
  plan.a.vocab = s.vocab;
  Packer pack(ws + at_bytes + (uint64_t)nranks * part_bytes, s.es);
  for (int r = 0; r < nranks; ++r) {
    c.part[r] = (const float2*)(ws + at_bytes + (uint64_t)r * part_bytes);
    c.loss[r] = loss[r];
    c.lse[r] = lse[r];
    if (!s.shard[r]) continue;
    const Packer::Rows px = pack.rows(x[r], s.rows, s.hidden), pw = pack.rows(w[r], s.shard[r], s.hidden);
    Problem* p = plan.add(s.rows, s.shard[r], s.hidden, px.ld, pw.ld, 0);
    p->a[0] = px.p;
    p->b[0] = pw.p;
    p->c[0] = (char*)c.part[r];
    p->c[1] = ws;
    p->col0 = s.start[r];
  }
  const uint64_t cols = tile_cols(product_tile(PK_STATS, (int)dtype, plan, dev).tile);
  for (int r = 0; r < nranks; ++r) c.tiles[r] = (uint32_t)((s.shard[r] + cols - 1) / cols);
  c.max_tiles = c.tiles[0];  // the first shard is the longest
  c.at = (const float*)ws;
  c.target = target;
  c.vocab = s.vocab;
  c.rows = (uint32_t)s.rows;
  c.nranks = nranks;
  if (pack.launch((hipStream_t)stream) != hipSuccess) return AR_ERR_HIP;
  if (launch_products(PK_STATS, (int)dtype, plan, dev, (hipStream_t)stream) != hipSuccess) return AR_ERR_HIP;
  uint32_t per = 1;
  while (per < 64 && per < s.rows) per *= 2;
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((s.rows + per - 1) / per)), dim3(COMBINE_THREADS), 0,
                     (hipStream_t)stream, c, per);
  return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP;
}

ar_status ar_linear_cross_entropy_backward(int nranks, const float* grad_loss, const void* const* x,
                                           const void* const* w, const int64_t* target, const float* const* lse,
                                           void* const* dx, void* const* dw, size_t rows, size_t hidden, size_t vocab,
                                           ar_dtype dtype, size_t piece, void* workspace, size_t workspace_bytes,
                                           ar_stream_t stream) {
  const ar_status st = check_shape(nranks, rows, hidden, vocab, (int)dtype);
  if (st != AR_OK) return st;
  if (!x || !w || !lse || !dx || !dw) return AR_ERR_INVALID;
  const XentShape s = shape_of(nranks, rows, hidden, vocab, (int)dtype);
  const BackwardSpace sp = space_of(s, nranks, (int)dtype, piece);
  const uint64_t need = rows ? sp.bytes(nranks) + s.live_bytes : 0;
  const uint64_t xb = s.rows * s.hidden * s.es;
  LayerBuffers b;
  for (int r = 0; r < nranks; ++r) {
    b.in(x[r], xb);
    b.in(w[r], s.shard[r] * s.hidden * s.es);
    b.in(lse[r], s.rows * 4, 4);
    b.out(dx[r], xb);
    b.out(dw[r], s.shard[r] * s.hidden * s.es);
  }
  b.in(target, s.rows * 8, 8);
  b.in(grad_loss, s.rows * 4, 4);
  b.out(workspace, need);
  if (!b.ok()) return AR_ERR_INVALID;
  if (workspace_bytes < need) return AR_ERR_TOO_LARGE;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return AR_ERR_HIP;
  char* ws = (char*)workspace;
  const uint64_t pieces = (s.max_shard + sp.piece - 1) / sp.piece;
  Packer pack(ws + sp.bytes(nranks), s.es);
  Packer::Rows px[MAX_RANKS], pw[MAX_RANKS];
  // x is a sum's operand over the rows (dw): a row without loss has weight 0 there,
  // but 0 times what a padding row may hold (infinities, NaN) is not 0.  x is
  // read from a copy that has zeros in those rows.
  for (int r = 0; r < nranks; ++r) {  // (with no rows nothing is read, and nothing copied)
    px[r] = pack.live_rows(x[r], s.rows, s.hidden, target, s.vocab);
    pw[r] = pack.rows(w[r], rows ? s.shard[r] : 0, s.hidden);
  }
  if (pack.launch((hipStream_t)stream) != hipSuccess) return AR_ERR_HIP;
  // The logits are the forward pass's bits again: their sums run in the order
  // that pass's tile class takes (else lse and the logits differ in their
  // roundings, which d of a confident row, 1 - p, does not forgive).
  uint32_t k_parts = 0;
  if (rows) {
    ProductPlan plan;
    for (int r = 0; r < nranks; ++r)
      if (s.shard[r]) plan.add(s.rows, s.shard[r], s.hidden, px[r].ld, pw[r].ld, 0);
    k_parts = tile_k_parts(product_tile(PK_STATS, (int)dtype, plan, dev).tile);
  }
  const float* scale = nullptr;
  if (rows && sp.scale_bytes) {
    float* out = (float*)(ws + sp.bytes(nranks) - sp.scale_bytes);
    hipLaunchKernelGGL(scale_kernel, dim3(1), dim3(COMBINE_THREADS), 0, (hipStream_t)stream, grad_loss, target, s.vocab,
                       (uint32_t)s.rows, out);
    if (hipGetLastError() != hipSuccess) return AR_ERR_HIP;
    scale = out;
  }
  for (uint64_t i = 0; i < pieces; ++i) {
    const uint64_t first = i * sp.piece;
    ProductPlan d_plan, grads;
    d_plan.a.target = target;
    d_plan.a.grad = grad_loss;
    d_plan.a.vocab = s.vocab;
    d_plan.a.scale = grads.a.scale = scale;
    d_plan.k_parts = k_parts;
    grads.may_share = sp.share != 0;
    for (int r = 0; r < nranks; ++r) {
      // a rank without vocabulary still writes dx: a product with k = 0
      if (first >= umax(s.shard[r], 1)) continue;
      const uint64_t len = umin(sp.piece, s.shard[r] - first);
      char* d = ws + (uint64_t)r * sp.d_bytes;
      const char* wp = pw[r].p + first * pw[r].ld * s.es;
      Problem* p;
      if (len) {
        p = d_plan.add(s.rows, len, s.hidden, px[r].ld, pw[r].ld, sp.piece);
        p->a[0] = px[r].p;
        p->b[0] = wp;
        p->c[0] = d;
        p->a[1] = (const char*)lse[r];
        p->fold = sp.fold;
        p->col0 = s.start[r] + first;
      }
      p = grads.add(sp.fold + s.rows, s.hidden, len, sp.piece, pw[r].ld, s.hidden);
      p->fold = sp.fold;
      p->a[0] = d;
      p->b[0] = wp;
      p->c[0] = (char*)dx[r];
      p->c[1] = sp.acc_bytes ? ws + (uint64_t)nranks * sp.d_bytes + (uint64_t)r * sp.acc_bytes : (char*)dx[r];
      p->c[2] = ws + (uint64_t)nranks * (sp.d_bytes + sp.acc_bytes) + (uint64_t)r * sp.share;
      p->mode = (i ? GRAD_ADD : 0) | (first + len < s.shard[r] ? GRAD_PARTIAL : 0);
    }
    grads.head = grads.a.nprob;
    for (int r = 0; r < nranks; ++r) {
      if (first >= s.shard[r]) continue;
      const uint64_t len = umin(sp.piece, s.shard[r] - first);
      Problem* p = grads.add(len, s.hidden, s.rows, sp.piece, px[r].ld, s.hidden);
      p->nseg = sp.fold ? 2 : 1;
      p->a[0] = ws + (uint64_t)r * sp.d_bytes;
      p->a[1] = p->a[0] + sp.fold * sp.piece * s.es;
      p->b[0] = p->b[1] = px[r].p;
      p->c[0] = (char*)dw[r] + first * s.hidden * s.es;
      p->mode = GRAD_TN;
    }
    if (launch_products(PK_DLOGITS, (int)dtype, d_plan, dev, (hipStream_t)stream) != hipSuccess ||
        launch_grads((int)dtype, grads, dev, (hipStream_t)stream) != hipSuccess)
      return AR_ERR_HIP;
  }
  return AR_OK;
}

}  // extern "C"
