// cache.hip -- the 8-bit key/value cache of the attention operators: storing
// new tokens (ar_cache_write) and reading tokens back (ar_cache_read).
//
// A page and head has one scale, a power of two: the smallest that brings the
// largest new magnitude to 448 or less, and no smaller than what the page has.
// Dividing by it is exact, so a code is one rounding of the value; when it
// grows, the codes of the page's earlier tokens move by whole binades and only
// those that become subnormal are rounded.
//
// Both are bound by memory, or by latency for a few tokens.  One workgroup owns
// a page and head of keys or of values, so a scale has one writer and nothing is
// atomic.  Values are kept with tokens running fastest, as the product with the
// softmax weights reads them; a page is turned in LDS.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/ar.h"
#include "device.hpp"
#include "heads.hpp"
#include "layer.hpp"

using namespace ar;

namespace {

constexpr int THREADS = 256;

struct CacheArgs {
  const char* x[2][MAX_RANKS];  // new keys, values (write); results (read)
  uint8_t* codes[2][MAX_RANKS];
  uint8_t* scale[2][MAX_RANKS];
  uint64_t pitch[2];  // bytes from row to row
  Paged p;
  uint32_t kv_heads, nranks;
};

// A workgroup's page: rows row .. row + (hi - lo) of the call are the page's
// tokens lo .. hi - 1.
struct Piece {
  uint32_t row, lo, hi, id;
};

// Item -> page of a sequence.  A sequence's n tokens lie on at most
// floor(n / page) + 2 pages.
__device__ __forceinline__ bool piece_of(const Paged& p, uint64_t item, Piece* out) {
  uint32_t row0, n;
  uint64_t local;
  int32_t at;
  const uint32_t s = find_sequence(p, item, 1, 1u << p.page_shift, 2, &row0, &n, &local, &at);
  if (s >= p.seqs) return false;
  const uint64_t start = at < 0 ? 0 : (uint64_t)at, end = start + n;
  const uint64_t j = (start >> p.page_shift) + local, t0 = j << p.page_shift;
  if (t0 >= end) return false;
  const uint64_t lo = start > t0 ? start : t0, hi = end < t0 + (1ull << p.page_shift) ? end : t0 + (1ull << p.page_shift);
  out->row = row0 + (uint32_t)(lo - start);
  out->lo = (uint32_t)(lo - t0);
  out->hi = (uint32_t)(hi - t0);
  out->id = page_id(p, s, j);
  return true;
}

// Eight elements of a row, as they are stored.
template <int DT>
struct Eight {
  uint4 w[DT == DT_BF16 ? 1 : 2];
};

template <int DT>
__device__ __forceinline__ Eight<DT> load8(const char* p) {
  Eight<DT> r;
  r.w[0] = ld16(p);
  if constexpr (DT != DT_BF16) r.w[1] = ld16(p + 16);
  return r;
}

template <int DT>
__device__ __forceinline__ void widen(const Eight<DT>& v, float* f) {
  const uint32_t w[4] = {v.w[0].x, v.w[0].y, v.w[0].z, v.w[0].w};
  if constexpr (DT == DT_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  } else {
    const uint32_t u[4] = {v.w[1].x, v.w[1].y, v.w[1].z, v.w[1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]), f[4 + i] = __uint_as_float(u[i]);
  }
}

template <int DT>
__device__ __forceinline__ void store8(char* p, const float* f) {
  if (DT == DT_BF16) {
    st16(p, make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      st16(p + 16 * i, make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                  __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3])));
  }
}

// Four words of four bytes, turned: byte i of word j becomes byte j of word i.
__device__ __forceinline__ void turn4(uint32_t* w) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602);
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602);
  w[0] = __builtin_amdgcn_perm(c, a, 0x05040100), w[1] = __builtin_amdgcn_perm(c, a, 0x07060302);
  w[2] = __builtin_amdgcn_perm(d, b, 0x05040100), w[3] = __builtin_amdgcn_perm(d, b, 0x07060302);
}

// Four codes at another scale: what they stand for, rounded again.
__device__ __forceinline__ uint32_t rescaled(uint32_t codes, float from, float inv_to) {
  float x[4];
  values_of(codes, from, x);
  return codes_of(x, inv_to);
}

// The workgroup's largest value, and thread 0's byte for everyone.
__device__ float block_max(float m, float* s, uint32_t* byte) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = m;
  if (threadIdx.x == 0) s[THREADS / 64] = __uint_as_float(*byte);
  __syncthreads();
  *byte = __float_as_uint(s[THREADS / 64]);
  m = s[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) m = fmaxf(m, s[w]);
  return m;
}

// Tokens a workgroup has in registers at a time: BATCH of each thread.  A page of
// 64 tokens of 128 values is one batch and read once; what is longer is read a
// second time, from L2.
constexpr int BATCH = 4;

// Bytes of the tokens [lo, hi) in a word that holds tokens 4 q .. 4 q + 3.
__device__ __forceinline__ uint32_t bytes_of(uint32_t q, uint32_t lo, uint32_t hi) {
  uint32_t m = 0;
#pragma unroll
  for (uint32_t e = 0; e < 4; ++e)
    if (4 * q + e >= lo && 4 * q + e < hi) m |= 0xffu << (8 * e);
  return m;
}

template <int DT, int DIM>
__global__ __launch_bounds__(THREADS) void write_kernel(CacheArgs a) {
  constexpr uint32_t ES = DT == DT_BF16 ? 2 : 4, LANES = DIM / 8, ROWS = THREADS / LANES;  // lanes of a token, tokens a pass
  constexpr uint32_t PITCH = DIM + 4;                                                      // of a token's codes in LDS
  extern __shared__ uint8_t tile[];                                                        // values: [page][PITCH]
  __shared__ float maxima[THREADS / 64 + 1];
  const uint32_t kind = blockIdx.y & 1, head = blockIdx.y >> 1;
  uint32_t r;
  Piece pc;
  if (!piece_of(a.p, item_of(a.nranks, &r), &pc)) return;
  const uint32_t page = 1u << a.p.page_shift, count = pc.hi - pc.lo;
  const uint32_t lane = threadIdx.x % LANES, row = threadIdx.x / LANES;
  const char* x = a.x[kind][r] + (uint64_t)pc.row * a.pitch[kind] + (uint64_t)head * (DIM * ES) + lane * 8 * ES;
  Eight<DT> v[BATCH];
  auto load = [&](uint32_t i0) {
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const uint32_t i = i0 + row + j * ROWS;
      if (i < count) v[j] = load8<DT>(x + (uint64_t)i * a.pitch[kind]);
    }
  };
  load(0);  // (does not wait for the page's number)
  if (pc.id >= a.p.pages) return;
  uint8_t* codes = a.codes[kind][r] + page_at(pc.id, a.kv_heads, head, page * DIM);
  uint8_t* scale = a.scale[kind][r] + (uint64_t)pc.id * a.kv_heads + head;
  // one thread reads the byte and writes it, in that order
  uint32_t held = threadIdx.x == 0 ? *scale : 0;
  // Values: words q0 .. of every dimension change.  A thread's first ones are asked
  // for here where some of their bytes stay.
  const uint32_t q1 = (pc.hi + 3) / 4, q0 = pc.lo / 4;
  uint32_t old[4] = {};
  if (kind == 1 && threadIdx.x < (q1 - q0) * (DIM / 4)) {
    const uint32_t words = q1 - q0, dq = threadIdx.x / words, q = q0 + threadIdx.x - dq * words;
    if (bytes_of(q, pc.lo, pc.hi) != ~0u)
#pragma unroll
      for (int e = 0; e < 4; ++e) old[e] = *(const uint32_t*)(codes + (4 * dq + e) * page + q * 4);
  }

  float m = 0.f;
  for (uint32_t i0 = 0; i0 < count; i0 += BATCH * ROWS) {
    if (i0) load(i0);
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
      if (i0 + row + j * ROWS < count) {
        float f[8];
        widen<DT>(v[j], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = fabsf(f[e]);
          m = fmaxf(m, w < __builtin_inff() ? w : 0.f);
        }
      }
  }
  uint32_t byte = scale_byte(block_max(m, maxima, &held));
  const uint32_t before = held < SCALE_MIN ? SCALE_MIN : held > SCALE_MAX ? SCALE_MAX : held;
  const bool grows = pc.lo > 0 && byte > before;
  if (pc.lo > 0 && byte < before) byte = before;
  const float inv = scale_of(254 - byte < SCALE_MIN ? SCALE_MIN : 254 - byte), from = scale_of(before);
  const float half = 254 - byte < SCALE_MIN ? 0.5f : 1.f;  // 2^-127 is not a normal number
  if (threadIdx.x == 0) *scale = (uint8_t)byte;

  for (uint32_t i0 = 0; i0 < count; i0 += BATCH * ROWS) {
    if (count > BATCH * ROWS) load(i0);
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const uint32_t i = i0 + row + j * ROWS;
      if (i >= count) continue;
      float f[8];
      widen<DT>(v[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= half;
      const uint2 w = make_uint2(codes_of(f, inv), codes_of(f + 4, inv));
      if (kind == 0) {
        *(uint2*)(codes + (pc.lo + i) * DIM + lane * 8) = w;
      } else {
        uint32_t* t = (uint32_t*)(tile + i * PITCH + lane * 8);
        t[0] = w.x, t[1] = w.y;
      }
    }
  }
  if (kind == 0) {
    if (grows)
      for (uint32_t i = threadIdx.x * 4; i < pc.lo * DIM; i += THREADS * 4) {
        uint32_t* at = (uint32_t*)(codes + i);
        *at = rescaled(*at, from * half, inv);
      }
    return;
  }
  __syncthreads();
  // Four dimensions of four tokens per item, turned in registers.
  const uint32_t words = q1 - q0;
  for (uint32_t i = threadIdx.x; i < words * (DIM / 4); i += THREADS) {
    const uint32_t dq = i / words, q = q0 + i - dq * words, fresh = bytes_of(q, pc.lo, pc.hi);
    uint32_t w[4];
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) {
      const uint32_t t = 4 * q + e;
      w[e] = t >= pc.lo && t < pc.hi ? *(const uint32_t*)(tile + (t - pc.lo) * PITCH + 4 * dq) : 0;
    }
    turn4(w);
    if (fresh != ~0u) {
      // tokens before lo are the page's (at its new scale), those from hi on stay as they are
      const uint32_t first = bytes_of(q, 0, pc.lo);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (i >= THREADS) old[e] = *(const uint32_t*)(codes + (4 * dq + e) * page + q * 4);
        const uint32_t moved = grows ? rescaled(old[e], from * half, inv) : old[e];
        w[e] = (w[e] & fresh) | (moved & first) | (old[e] & ~(fresh | first));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) *(uint32_t*)(codes + (4 * dq + e) * page + q * 4) = w[e];
  }
  if (grows)  // whole words of earlier tokens
    for (uint32_t i = threadIdx.x; i < q0 * DIM; i += THREADS) {
      uint32_t* at = (uint32_t*)(codes + i / q0 * page + i % q0 * 4);
      *at = rescaled(*at, from * half, inv);
    }
}

template <int DT, int DIM>
__global__ __launch_bounds__(THREADS) void read_kernel(CacheArgs a) {
  constexpr uint32_t ES = DT == DT_BF16 ? 2 : 4, LANES = DIM / 8, ROWS = THREADS / LANES, PITCH = DIM + 4;
  extern __shared__ uint8_t tile[];
  const uint32_t kind = blockIdx.y & 1, head = blockIdx.y >> 1;
  uint32_t r;
  Piece pc;
  if (!piece_of(a.p, item_of(a.nranks, &r), &pc)) return;
  const uint32_t page = 1u << a.p.page_shift, count = pc.hi - pc.lo;
  const bool there = pc.id < a.p.pages;
  const uint32_t lane = threadIdx.x % LANES, row = threadIdx.x / LANES;
  char* x = (char*)a.x[kind][r] + (uint64_t)pc.row * a.pitch[kind] + (uint64_t)head * (DIM * ES) + lane * 8 * ES;
  const uint8_t* codes = a.codes[kind][r] + page_at(there ? pc.id : 0, a.kv_heads, head, page * DIM);
  uint32_t byte = 127;
  if (there) byte = a.scale[kind][r][(uint64_t)pc.id * a.kv_heads + head];
  const uint32_t q0 = pc.lo / 4, words = (pc.hi + 3) / 4 - q0;
  if (kind == 1 && there) {
    // Four dimensions of four tokens per item, BATCH items of a thread in flight.
    for (uint32_t i0 = threadIdx.x; i0 < words * (DIM / 4); i0 += BATCH * THREADS) {
      uint32_t w[BATCH][4];
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        const uint32_t i = i0 + j * THREADS, dq = i / words, q = i - dq * words;
        if (i < words * (DIM / 4))
#pragma unroll
          for (int e = 0; e < 4; ++e) w[j][e] = *(const uint32_t*)(codes + (4 * dq + e) * page + (q0 + q) * 4);
      }
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        const uint32_t i = i0 + j * THREADS, dq = i / words, q = i - dq * words;
        if (i >= words * (DIM / 4)) continue;
        turn4(w[j]);
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) *(uint32_t*)(tile + (4 * q + e) * PITCH + 4 * dq) = w[j][e];
      }
    }
    __syncthreads();
  }
  const float scale = scale_of(byte < SCALE_MIN ? SCALE_MIN : byte > SCALE_MAX ? SCALE_MAX : byte);
  for (uint32_t i0 = row; i0 < count; i0 += BATCH * ROWS) {
    uint2 w[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const uint32_t i = i0 + j * ROWS;
      w[j] = make_uint2(0, 0);
      if (i >= count || !there) continue;
      if (kind == 0) {
        w[j] = *(const uint2*)(codes + (pc.lo + i) * DIM + lane * 8);
      } else {
        const uint32_t* t = (const uint32_t*)(tile + (i + pc.lo % 4) * PITCH + lane * 8);
        w[j] = make_uint2(t[0], t[1]);
      }
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const uint32_t i = i0 + j * ROWS;
      if (i >= count) continue;
      float f[8];
      values_of(w[j].x, scale, f);
      values_of(w[j].y, scale, f + 4);
      store8<DT>(x + (uint64_t)i * a.pitch[kind], f);
    }
  }
}

}  // namespace

namespace ar {

ar_status check_cache(const ar_kv_cache* c) {
  if (!c || c->nranks < 1 || c->nranks > MAX_RANKS || !c->k || !c->v || !c->k_scale || !c->v_scale) return AR_ERR_INVALID;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return AR_ERR_UNSUPPORTED;
  if (!head_dim_ok(c->head_dim)) return AR_ERR_UNSUPPORTED;
  if (c->kv_heads < 1) return AR_ERR_INVALID;
  if (c->kv_heads > MAX_HEADS || c->pages >= (1ull << 31)) return AR_ERR_TOO_LARGE;
  if (c->pages * c->kv_heads * c->page * c->head_dim >= (1ull << 47)) return AR_ERR_TOO_LARGE;
  return AR_OK;
}

ar_status check_rows(const ar_kv_cache* c, const ar_paged_rows* p) {
  if (!p) return AR_ERR_INVALID;
  if (p->rows > LAYER_MAX_ROWS || p->seqs > (1ull << 20) || p->width > (1ull << 31) ||
      p->width * c->page >= (1ull << 31) || p->table_stride >= (1ull << 31))
    return AR_ERR_TOO_LARGE;
  if (p->seqs && (!p->first || !p->at || (uintptr_t)p->first % 4 || (uintptr_t)p->at % 4)) return AR_ERR_INVALID;
  if (p->seqs && p->width && (!p->table || (uintptr_t)p->table % 4 || (p->seqs > 1 && p->table_stride < p->width)))
    return AR_ERR_INVALID;
  return AR_OK;
}

Paged paged_of(const ar_kv_cache* c, const ar_paged_rows* p) {
  Paged r;
  r.table = p->table;
  r.first = p->first;
  r.at = p->at;
  r.table_stride = p->table_stride;
  r.width = (uint32_t)p->width;
  r.seqs = (uint32_t)p->seqs;
  r.rows = (uint32_t)p->rows;
  r.pages = (uint32_t)c->pages;
  r.page_shift = (uint32_t)__builtin_ctzll(c->page);
  return r;
}

void add_cache(LayerBuffers& b, const ar_kv_cache* c, bool written) {
  const uint64_t heads = c->pages * c->kv_heads, bytes = heads * c->page * c->head_dim;
  for (int r = 0; r < c->nranks; ++r) {
    const void* codes[2] = {c->k[r], c->v[r]};
    const void* scales[2] = {c->k_scale[r], c->v_scale[r]};
    for (int i = 0; i < 2; ++i) {
      if (written) b.out(codes[i], bytes), b.out(scales[i], heads, 1);
      else b.in(codes[i], bytes), b.in(scales[i], heads, 1);
    }
  }
}

void add_rows(LayerBuffers& b, const ar_paged_rows* p) {
  b.in(p->first, p->seqs ? (p->seqs + 1) * 4 : 0, 4);
  b.in(p->at, p->seqs * 4, 4);
  b.in(p->table, p->seqs && p->width ? ((p->seqs - 1) * p->table_stride + p->width) * 4 : 0, 4);
}

}  // namespace ar

namespace {

// What a write and a read share: checks, arguments, the grid.
ar_status cache_call(const ar_kv_cache* c, const void* const* k, size_t k_stride, const void* const* v, size_t v_stride,
                     const ar_paged_rows* p, int dtype, bool write, hipStream_t stream) {
  ar_status st = check_cache(c);
  if (st == AR_OK) st = check_rows(c, p);
  if (st != AR_OK) return st;
  if (dtype < 0 || dtype > 2 || !k || !v) return AR_ERR_INVALID;
  if (dtype == DT_I32) return AR_ERR_UNSUPPORTED;
  if (p->rows == 0 || p->seqs == 0) return AR_OK;
  const uint64_t es = dtype == DT_BF16 ? 2 : 4, width = c->kv_heads * c->head_dim;
  if (!stride_ok(k_stride, width, es) || !stride_ok(v_stride, width, es)) return AR_ERR_INVALID;
  CacheArgs a;
  LayerBuffers b;
  for (int r = 0; r < c->nranks; ++r) {
    a.x[0][r] = (const char*)k[r];
    a.x[1][r] = (const char*)v[r];
    a.codes[0][r] = (uint8_t*)c->k[r];
    a.codes[1][r] = (uint8_t*)c->v[r];
    a.scale[0][r] = (uint8_t*)c->k_scale[r];
    a.scale[1][r] = (uint8_t*)c->v_scale[r];
    const uint64_t kb = span_bytes(p->rows, k_stride, width, es), vb = span_bytes(p->rows, v_stride, width, es);
    if (write) b.in(k[r], kb), b.in(v[r], vb);
    else b.out(k[r], kb), b.out(v[r], vb);
  }
  add_cache(b, c, write);
  add_rows(b, p);
  if (!b.ok()) return AR_ERR_INVALID;
  a.pitch[0] = k_stride * es;
  a.pitch[1] = v_stride * es;
  a.p = paged_of(c, p);
  a.kv_heads = (uint32_t)c->kv_heads;
  a.nranks = (uint32_t)c->nranks;
  const Fold fold = fold_items(item_count(p->rows, p->seqs, 1, c->page, 2), THREADS);
  const dim3 grid(fold.x, 2 * a.kv_heads, a.nranks * fold.folds);
  const uint32_t lds = (uint32_t)(c->page * (c->head_dim + 4));
  by_head_dim(dtype, c->head_dim, [&](auto dt, auto dim) {
    if (write) write_kernel<decltype(dt)::value, decltype(dim)::value><<<grid, THREADS, lds, stream>>>(a);
    else read_kernel<decltype(dt)::value, decltype(dim)::value><<<grid, THREADS, lds, stream>>>(a);
  });
  return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP;
}

}  // namespace

extern "C" {

ar_status ar_cache_write(const ar_kv_cache* cache, const void* const* k, size_t k_stride, const void* const* v,
                         size_t v_stride, const ar_paged_rows* rows, ar_dtype dtype, ar_stream_t stream) {
  return cache_call(cache, k, k_stride, v, v_stride, rows, (int)dtype, true, (hipStream_t)stream);
}

ar_status ar_cache_read(const ar_kv_cache* cache, void* const* k, void* const* v, const ar_paged_rows* rows,
                        ar_dtype dtype, ar_stream_t stream) {
  const size_t width = cache ? cache->kv_heads * cache->head_dim : 0;
  return cache_call(cache, (const void* const*)k, width, (const void* const*)v, width, rows, (int)dtype, false,
                    (hipStream_t)stream);
}

}  // extern "C"
