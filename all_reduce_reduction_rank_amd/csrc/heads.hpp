// heads.hpp -- what the operators on attention heads share: shape checks,
// kernels chosen by type and head size, the 8-bit cache's pages and codes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/ar.h"
#include "layer.hpp"
#include "schedule.hpp"

namespace ar {

constexpr uint64_t MAX_HEADS = 1024;

inline bool head_dim_ok(uint64_t dim) { return dim == 64 || dim == 128 || dim == 256; }

// Rows `stride` elements apart, each `width` wide and whole 16-byte chunks.
inline bool stride_ok(uint64_t stride, uint64_t width, uint64_t es) {
  return stride >= width && stride * es % 16 == 0 && stride < (1ull << 31);
}

// Bytes from the first to the last element of such rows.
inline uint64_t span_bytes(uint64_t rows, uint64_t stride, uint64_t width, uint64_t es) {
  return rows ? ((rows - 1) * stride + width) * es : 0;
}

// f(type constant, head_dim constant)
template <class F>
void by_head_dim(int dtype, uint64_t dim, F f) {
  auto with = [&](auto dt) {
    if (dim == 64) f(dt, std::integral_constant<int, 64>{});
    else if (dim == 128) f(dt, std::integral_constant<int, 128>{});
    else f(dt, std::integral_constant<int, 256>{});
  };
  if (dtype == DT_BF16) with(std::integral_constant<int, DT_BF16>{});
  else with(std::integral_constant<int, DT_F32>{});
}

// A launch may have fewer than 2^32 threads along x.  Work items beyond that go
// along z, in `folds` layers of as many as x holds (the last one partly empty:
// kernels check their items).
struct Fold {
  uint32_t x, folds;
};

inline Fold fold_items(uint64_t items, uint32_t threads) {
  const uint64_t most = (1ull << 32) / threads - 1;
  const uint64_t x = items < most ? items : most;
  return {(uint32_t)x, (uint32_t)(x ? (items + x - 1) / x : 1)};
}

// z holds the ranks and the layers: a workgroup's item, and its rank in *r.
__device__ __forceinline__ uint32_t item_of(uint32_t nranks, uint32_t* r) {
  uint32_t item = blockIdx.x, z = blockIdx.z;
  while (z >= nranks) z -= nranks, item += gridDim.x;
  *r = z;
  return item;
}

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// Two floats to bf16, nearest even, NaN kept (one instruction).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const v2bf v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

// ------------------------------------------------------------ paged cache

// Rows and pages of a call's sequences (ar_paged_rows), as kernels take them.
struct Paged {
  const int32_t* table;
  const int32_t* first;
  const int32_t* at;
  uint64_t table_stride;
  uint32_t width, seqs, rows;
  uint32_t pages, page_shift;  // page = 1 << page_shift
};

// Bytes of one (page, head) of codes; where it lies.
__device__ __forceinline__ uint64_t page_at(uint32_t id, uint32_t kv_heads, uint32_t head, uint32_t bytes) {
  return ((uint64_t)id * kv_heads + head) * bytes;
}

// Entry of the table for tokens j << page_shift on of sequence s: a page if it
// is below p.pages.  (Compared where it is used and not here, so that a loop may
// ask for it ahead of time without waiting for it.)
__device__ __forceinline__ uint32_t page_id(const Paged& p, uint32_t s, uint64_t j) {
  uint32_t id = ~0u;
  if (j < p.width) id = (uint32_t)p.table[s * p.table_stride + j];
  return id;
}

__device__ __forceinline__ uint32_t first_row(const Paged& p, uint32_t s) {
  const int32_t f = p.first[s];
  return f < 0 ? 0u : (uint32_t)f < p.rows ? (uint32_t)f : p.rows;
}

// Work items are numbered without knowing the lengths: sequence s owns the
// items from base(s) = floor(first[s] * mul / div) + extra * s on, which leaves
// it room for the ceil(n mul / div) + extra - 1 it may need.  The sequence of
// an item is found by every wave on its own: its lanes look at 64 sequences at
// a time, first at every 64th part of those in question, and count the ones that
// start at or before the item: one memory latency up to 64 sequences, two up to
// 4096, four at most (65536 sequences of one token stored: 0.42 ms; with all of them
// looked at in turn 22 ms).  Returns seqs if no sequence owns the item; n = its rows, at = its entry
// of p.at, local = the item's number within the sequence.  (Where `first`
// decreases the count names some sequence, whose rows are checked as any.)
__device__ __forceinline__ uint64_t item_base(uint64_t first, uint32_t s, uint32_t mul, uint32_t div, uint32_t extra) {
  return first * mul / div + (uint64_t)extra * s;
}

__device__ __forceinline__ uint32_t find_sequence(const Paged& p, uint64_t item, uint32_t mul, uint32_t div,
                                                  uint32_t extra, uint32_t* row0, uint32_t* n, uint64_t* local,
                                                  int32_t* at) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t s0 = 0, span = p.seqs;  // the owner is one of [s0, s0 + span)
  while (span > 64) {
    const uint32_t part = (span + 63) / 64, s = s0 + lane * part;
    const uint64_t who = __ballot(lane * part < span && item_base(first_row(p, s), s, mul, div, extra) <= item);
    const uint32_t c = __popcll(who);
    if (!c) return p.seqs;
    s0 += (c - 1) * part;
    span -= (c - 1) * part;
    if (span > part) span = part;
  }
  const uint32_t s = s0 + lane;
  // what the owner will need is loaded along, for the same latency
  uint32_t a = 0, b = 0;
  int32_t x = 0;
  if (lane < span) a = first_row(p, s), b = first_row(p, s + 1), x = p.at[s];
  const uint32_t c = __popcll(__ballot(lane < span && item_base(a, s, mul, div, extra) <= item));
  if (!c) return p.seqs;
  *row0 = __builtin_amdgcn_readlane(a, c - 1);
  *n = __builtin_amdgcn_readlane(b, c - 1);
  *at = __builtin_amdgcn_readlane(x, c - 1);
  if (*n <= *row0) return p.seqs;
  const uint32_t owner = __builtin_amdgcn_readfirstlane(s0 + c - 1);
  *n -= *row0;
  const uint64_t base = item_base(*row0, owner, mul, div, extra);
  if (item < base) return p.seqs;
  *local = item - base;
  return owner;
}

inline uint64_t item_count(uint64_t rows, uint64_t seqs, uint64_t mul, uint64_t div, uint64_t extra) {
  return rows * mul / div + extra * seqs;
}

// ------------------------------------------------------------------- codes

constexpr uint32_t SCALE_MIN = 1, SCALE_MAX = 254;

__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }  // 2^(byte - 127), byte 1 .. 254

// The smallest byte with m <= 448 * 2^(byte - 127): 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t scale_byte(float m) {
  const uint32_t u = __float_as_uint(m), e = u >> 23;  // m >= 0
  const int b = (int)e - 8 + ((u & 0x7fffff) > 0x600000 ? 1 : 0);
  return b < (int)SCALE_MIN ? SCALE_MIN : (uint32_t)b;
}

// Codes of four values of magnitude at most 448; NaN where `x` is not finite.
__device__ __forceinline__ uint32_t codes_of(const float* x, float inv_scale) {
  int w = 0;
  const float y[4] = {x[0] * inv_scale, x[1] * inv_scale, x[2] * inv_scale, x[3] * inv_scale};
  w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
  uint32_t r = (uint32_t)w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!(fabsf(x[i]) < __builtin_inff())) r = (r & ~(0xffu << (8 * i))) | (0x7fu << (8 * i));
  return r;
}

typedef float v2fl __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void values_of(uint32_t codes, float scale, float* x) {
  const v2fl lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
  const v2fl hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
  x[0] = lo[0] * scale, x[1] = lo[1] * scale, x[2] = hi[0] * scale, x[3] = hi[1] * scale;
}

// The host's checks of a cache and of a call's sequences.
ar_status check_cache(const ar_kv_cache* c);
ar_status check_rows(const ar_kv_cache* c, const ar_paged_rows* p);
Paged paged_of(const ar_kv_cache* c, const ar_paged_rows* p);
// Their buffers; the cache is written or read.
void add_cache(LayerBuffers& b, const ar_kv_cache* c, bool written);
void add_rows(LayerBuffers& b, const ar_paged_rows* p);

}  // namespace ar
