// attention.hip -- attention over the 8-bit paged cache (ar_cache_attention).
//
//   z_j = scale q . k_j over the tokens a row sees, out = sum_j p_j v_j / sum_j p_j,
//   p_j = exp(z_j - m), in one pass over the tokens with a running maximum.
//
// The query heads that share a key/value head are rows of one product: packed
// row rho of a sequence is query row rho / group, head rho % group of the
// group, so that a few tokens still fill a tile and codes are read once for
// the whole group.
//
// Products run on the matrix cores in bf16.  e4m3 codes times a power of two
// are bf16 numbers, so keys and values enter exactly; fp32 queries enter as
// three bf16 terms, the softmax weights as one to three (see the kernels).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/ar.h"
#include "device.hpp"
#include "heads.hpp"
#include "layer.hpp"

using namespace ar;

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr uint32_t TOKENS = 64;  // of a step along the cache
constexpr float LN2 = 0.69314718055994530942f, LOG2E = 1.44269504088896340736f;

struct AttnArgs {
  const char* q[MAX_RANKS];
  char* out[MAX_RANKS];
  float* lse[MAX_RANKS];
  const uint8_t* k[MAX_RANKS];
  const uint8_t* v[MAX_RANKS];
  const uint8_t* k_scale[MAX_RANKS];
  const uint8_t* v_scale[MAX_RANKS];
  uint64_t q_pitch;  // bytes
  Paged p;
  uint32_t kv_heads, heads, group;
  uint32_t splits, min_steps;  // shares of a tile's tokens: at most `splits`, of at least `min_steps` steps
  uint32_t tiles;              // row tiles of a head (bound)
  float scale;                 // times log2(e)
  int32_t causal;
  uint32_t window;
  float* part;   // [rank][kv head][tile][split][rows of a tile][dim]: sum p v of a share
  float2* stat;  // [rank][kv head][tile][split][rows of a tile]: its m (of log2) and sum p
};

// A tile of packed rows of one sequence and the tokens its rows see.
struct Tile {
  uint32_t s, row0, n;  // sequence, its first row in the call, its rows
  uint32_t r0, rows;    // packed rows r0 .. r0 + rows - 1
  int64_t length;       // cached tokens
  int64_t lo, hi;       // tokens some row sees lie in [lo, hi)
  uint32_t begin, steps;  // steps of TOKENS tokens from token `begin` on
};

__device__ __forceinline__ bool tile_of(const AttnArgs& a, uint32_t tile, uint32_t bm, Tile* t) {
  uint64_t local;
  t->s = find_sequence(a.p, tile, a.group, bm, 1, &t->row0, &t->n, &local);
  if (t->s >= a.p.seqs) return false;
  const uint64_t rows = (uint64_t)t->n * a.group, r0 = local * bm;
  if (r0 >= rows) return false;
  t->r0 = (uint32_t)r0;
  t->rows = (uint32_t)(rows - r0 < bm ? rows - r0 : bm);
  const int64_t cap = (int64_t)a.p.width << a.p.page_shift;
  int64_t len = a.p.at[t->s];
  len = len < 0 ? 0 : len < cap ? len : cap;
  t->length = len;
  t->lo = 0;
  t->hi = len;
  if (a.causal) {
    const int64_t last = len - t->n + (t->r0 + t->rows - 1) / a.group + 1;
    t->hi = last < 0 ? 0 : last < len ? last : len;
    if (a.window) {
      const int64_t first = len - t->n + t->r0 / a.group + 1 - (int64_t)a.window;
      t->lo = first < 0 ? 0 : first < t->hi ? first : t->hi;
    }
  }
  t->begin = (uint32_t)(t->lo & ~(int64_t)(TOKENS - 1));
  t->steps = t->hi > t->lo ? (uint32_t)((t->hi - t->begin + TOKENS - 1) / TOKENS) : 0;
  return true;
}

__device__ __forceinline__ uint32_t share_steps(const AttnArgs& a, uint32_t steps) {
  const uint32_t per = (steps + a.splits - 1) / a.splits;
  return per > a.min_steps ? per : a.min_steps;
}

// Eight codes (two words) as bf16 numbers, exact.
__device__ __forceinline__ v8bf widen8(uint32_t lo, uint32_t hi, float scale) {
  v4u w;
  w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
  w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
  w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
  w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
  return __builtin_bit_cast(v8bf, w);
}

__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// x in TERMS bf16 terms: each holds what the ones before it left.
template <int TERMS>
__device__ __forceinline__ void split8(float* x, v8bf* out) {
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    v4u w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
      if (t + 1 < TERMS) x[2 * i] -= low_of(w[i]), x[2 * i + 1] -= high_of(w[i]);
    }
    out[t] = __builtin_bit_cast(v8bf, w);
  }
}

// A bf16 pair's numbers that are not finite become 1 and the others 0
// (count), or they become 0 and the others stay.
__device__ __forceinline__ v8bf sift(v8bf x, bool count) {
  v4u w = __builtin_bit_cast(v4u, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (w[i] & 0x7f80u) == 0x7f80u ? 0xffffu : 0u, hi = (w[i] & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u;
    w[i] = count ? (0x3f803f80u & (lo | hi)) : (w[i] & ~(lo | hi));
  }
  return __builtin_bit_cast(v8bf, w);
}

__device__ __forceinline__ float byte_scale(uint32_t b) { return scale_of(b < SCALE_MIN ? SCALE_MIN : b > SCALE_MAX ? SCALE_MAX : b); }

// Bytes of a 16-token block of codes that lie outside tokens [lo, hi) become 0;
// `at` is the block's first token.
__device__ __forceinline__ uint4 clear_outside(uint4 w, int64_t at, int64_t lo, int64_t hi) {
  uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (at + 4 * i + e < lo || at + 4 * i + e >= hi) x[i] &= ~(0xffu << (8 * e));
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// ---- few rows: 16 rows per workgroup, its four waves share the tokens ----
//
// Each wave takes every fourth step of 64 tokens straight from memory to
// registers, with a softmax of its own, joined at the end; a long cache is
// shared among workgroups and joined by a second kernel.  Bound by memory: a
// step is 64 x 2 x dim bytes of codes, loaded 16 bytes per lane one step ahead.
//
// Matrix instructions 16x16x32, keys as the first operand: S^T[token][row].
// The order of k is free as long as both operands share it, and so is the
// order of tokens; both are chosen so that lanes load contiguous bytes and
// weights stay in the lanes that hold them.  With lane = 16 g + c:
//   keys   step a (0..3), row c of the operand: token 16 (c / 4) + 4 a + c % 4,
//          k: dim / 4 contiguous values from g dim / 4 on
//   S^T    lane (g, c) holds tokens 16 g + 4 a + i (i = 0..3) of row c
//   values operand row c: dimension 16 t + c, k of group g: tokens 16 g ..
//          16 g + 15, which are one 16-byte load (a page is whole blocks of 16)
//   O^T    lane (g, c) holds dimensions 16 t + 4 g + i of row c
//
// What a row does not see must not reach it: its weight is 0, but 0 times a NaN
// is not.  A wave that ends with a NaN goes over its tokens twice more, once to
// count the numbers that are not finite among those that each row sees, once
// without them.
template <int DT, int DIM>
__global__ __launch_bounds__(256) void few_rows_kernel(AttnArgs a) {
  constexpr int WAVES = 4, BM = 16;
  constexpr int KSTEPS = DIM / 32, KW = DIM / 64;  // instructions of q . k; 16-byte loads of a key
  constexpr int DT_TILES = DIM / 16;
  constexpr int QT = DT == DT_BF16 ? 1 : 3;  // terms of q
  constexpr int PT = DT == DT_BF16 ? 2 : 3;  // terms of the weights
  constexpr uint32_t ES = DT == DT_BF16 ? 2 : 4;
  constexpr int PITCH = DIM + 4;
  __shared__ float o_s[WAVES][BM][PITCH];
  __shared__ float m_s[WAVES][BM], l_s[WAVES][BM];

  const uint32_t split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits;
  const uint32_t h = blockIdx.y, r = blockIdx.z;
  Tile t;
  if (!tile_of(a, tile, BM, &t)) return;
  const uint32_t per = share_steps(a, t.steps), step0 = split * per;
  if (split && step0 >= t.steps) return;
  const uint32_t step1 = step0 + per < t.steps ? step0 + per : t.steps;
  const bool shared = t.steps > per;

  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const uint8_t* kc = a.k[r];
  const uint8_t* vc = a.v[r];
  const uint32_t page_bytes = DIM << a.p.page_shift;

  // This lane's row and the tokens it sees.
  const uint32_t rho = t.r0 + c;
  const bool real = c < t.rows;
  const uint32_t qrow = real ? rho / a.group : 0, qhead = h * a.group + (real ? rho - qrow * a.group : 0);
  int64_t see0 = 0, see1 = real ? t.length : 0;
  if (a.causal && real) {
    const int64_t e = t.length - t.n + qrow + 1;
    see1 = e < 0 ? 0 : e < t.length ? e : t.length;
    if (a.window && e > (int64_t)a.window) see0 = e - a.window;
  }
  v8bf q[KSTEPS][QT];
  {
    const char* at = a.q[r] + (uint64_t)(t.row0 + qrow) * a.q_pitch + (uint64_t)qhead * (DIM * ES) + g * (DIM / 4) * ES;
#pragma unroll
    for (int s = 0; s < KSTEPS; ++s) {
      if (DT == DT_BF16) {
        const uint4 w = real ? ld16(at + s * 16) : make_uint4(0, 0, 0, 0);
        q[s][0] = __builtin_bit_cast(v8bf, w);
      } else {
        const uint4 w = real ? ld16(at + s * 32) : make_uint4(0, 0, 0, 0), u = real ? ld16(at + s * 32 + 16) : make_uint4(0, 0, 0, 0);
        float x[8] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w),
                      __uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
        split8<QT>(x, q[s]);
      }
    }
  }
  // Tokens that every row sees: no mask within [all0, all1).
  int64_t all0 = 0, all1 = t.length;
  if (a.causal) {
    const int64_t e = t.length - t.n + t.r0 / a.group + 1;
    all1 = e < 0 ? 0 : e < t.length ? e : t.length;
    const int64_t f = t.length - t.n + (t.r0 + t.rows - 1) / a.group + 1 - (int64_t)a.window;
    if (a.window && f > 0) all0 = f;
  }

  v4f o[DT_TILES];
  float m, l;
  uint4 kw[4][KW], vw[DT_TILES];
  uint32_t kid, vid;      // pages of the step to load next
  float ks, vs;
  bool there;             // this lane's block of values is on a page
  const uint32_t kb = 16 * (c >> 2), koff = c & 3;  // this lane's key block, row in a group of four

  auto ids = [&](uint32_t step) {
    const uint64_t base = (uint64_t)t.begin + (uint64_t)step * TOKENS;
    kid = page_id(a.p, t.s, (base + kb) >> a.p.page_shift);
    vid = page_id(a.p, t.s, (base + 16 * g) >> a.p.page_shift);
  };
  auto load_k = [&](uint32_t step) {
    const uint64_t base = (uint64_t)t.begin + (uint64_t)step * TOKENS + kb;
    const uint32_t off = (uint32_t)base & ((1u << a.p.page_shift) - 1);
    if (kid < a.p.pages) {
      const uint8_t* at = kc + page_at(kid, a.kv_heads, h, page_bytes) + (off + koff) * DIM + g * (DIM / 4);
      ks = byte_scale(a.k_scale[r][(uint64_t)kid * a.kv_heads + h]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < KW; ++j) kw[i][j] = ld16((const char*)at + i * 4 * DIM + j * 16);
    } else {
      ks = 1.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < KW; ++j) kw[i][j] = make_uint4(0, 0, 0, 0);
    }
  };
  auto load_v = [&](uint32_t step, uint32_t id) {
    const uint64_t base = (uint64_t)t.begin + (uint64_t)step * TOKENS + 16 * g;
    const uint32_t off = (uint32_t)base & ((1u << a.p.page_shift) - 1);
    there = id < a.p.pages;
    if (there) {
      const uint8_t* at = vc + page_at(id, a.kv_heads, h, page_bytes) + (c << a.p.page_shift) + off;
      vs = byte_scale(a.v_scale[r][(uint64_t)id * a.kv_heads + h]);
#pragma unroll
      for (int i = 0; i < DT_TILES; ++i) vw[i] = ld16((const char*)at + ((16 * i) << a.p.page_shift));
    } else {
      vs = 1.f;
#pragma unroll
      for (int i = 0; i < DT_TILES; ++i) vw[i] = make_uint4(0, 0, 0, 0);
    }
  };

  // One pass over this wave's steps.  MODE 0: the sums; 1: numbers that are not
  // finite among the values a row sees; 2: the sums without those.
  auto sweep = [&](auto mode) {
    constexpr int MODE = decltype(mode)::value;
#pragma unroll
    for (int i = 0; i < DT_TILES; ++i) o[i] = (v4f){0.f, 0.f, 0.f, 0.f};
    m = -INFINITY;
    l = 0.f;
    uint32_t step = step0 + wave;
    if (step >= step1) return;
    ids(step);
    load_k(step);
    load_v(step, vid);
    for (; step < step1; step += WAVES) {
      const int64_t base = (int64_t)t.begin + (int64_t)step * TOKENS;
      const bool more = step + WAVES < step1;
      if (more) ids(step + WAVES);
      v4f s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KSTEPS; ++j) {
          const uint4 w = kw[i][j / 2];
          const v8bf k8 = j % 2 ? widen8(w.z, w.w, ks) : widen8(w.x, w.y, ks);
#pragma unroll
          for (int x = QT - 1; x >= 0; --x) s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8, q[j][x], s[i], 0, 0, 0);
        }
      }
      if (more) load_k(step + WAVES);
      const bool mask = base < all0 || base + TOKENS > all1 || __any(!there);
      const int64_t first = base + 16 * g;
      float p[16];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float z = s[i][e] * a.scale;
          if (MODE == 1) z = 0.f;
          if (mask) {
            const int64_t at = first + 4 * i + e;
            if (at < see0 || at >= see1 || !there) z = -INFINITY;
          }
          p[4 * i + e] = z;
        }
      if (MODE == 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = p[i] == 0.f ? 1.f : 0.f;
      } else {
        float top = p[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, p[i]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float next = fmaxf(m, top), shift = next == -INFINITY ? 0.f : next;
        if (__any(next > m)) {
          const float f = __builtin_amdgcn_exp2f(m - shift);  // m -inf: 0
          l *= f;
#pragma unroll
          for (int i = 0; i < DT_TILES; ++i) o[i] *= f;
        }
        m = next;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          p[i] = __builtin_amdgcn_exp2f(p[i] - shift);
          l += p[i];
        }
      }
      v8bf w[2][PT];
      split8<PT>(p, w[0]);
      split8<PT>(p + 8, w[1]);
      if (base < t.lo || base + TOKENS > t.hi) {
#pragma unroll
        for (int i = 0; i < DT_TILES; ++i) vw[i] = clear_outside(vw[i], first, t.lo, t.hi);
      }
#pragma unroll
      for (int i = 0; i < DT_TILES; ++i) {
        v8bf lo = widen8(vw[i].x, vw[i].y, vs), hi = widen8(vw[i].z, vw[i].w, vs);
        if (MODE) lo = sift(lo, MODE == 1), hi = sift(hi, MODE == 1);
#pragma unroll
        for (int x = PT - 1; x >= 0; --x) {
          o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, w[0][x], o[i], 0, 0, 0);
          o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, w[1][x], o[i], 0, 0, 0);
        }
      }
      if (more) load_v(step + WAVES, vid);
    }
  };

  sweep(std::integral_constant<int, 0>{});
  float worst = 0.f;
#pragma unroll
  for (int i = 0; i < DT_TILES; ++i) worst += o[i][0] * 0.f + o[i][1] * 0.f + o[i][2] * 0.f + o[i][3] * 0.f;
  if (__any(!(worst == 0.f))) {
    uint32_t bad[(DT_TILES * 4 + 31) / 32];
    sweep(std::integral_constant<int, 1>{});
#pragma unroll
    for (int i = 0; i < (DT_TILES * 4 + 31) / 32; ++i) bad[i] = 0;
#pragma unroll
    for (int i = 0; i < DT_TILES * 4; ++i) bad[i / 32] |= (o[i / 4][i % 4] > 0.f ? 1u : 0u) << (i % 32);
    sweep(std::integral_constant<int, 2>{});
#pragma unroll
    for (int i = 0; i < DT_TILES * 4; ++i)
      if (bad[i / 32] >> (i % 32) & 1) o[i / 4][i % 4] = NAN;
  }

  // Join the waves (and the lane groups' sums of p).
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g == 0) m_s[wave][c] = m, l_s[wave][c] = l;
#pragma unroll
  for (int i = 0; i < DT_TILES; ++i) *(v4f*)&o_s[wave][c][16 * i + 4 * g] = o[i];
  __syncthreads();
  const uint64_t slot = (((uint64_t)r * a.kv_heads + h) * a.tiles + tile) * a.splits + split;
  for (uint32_t i = threadIdx.x; i < BM * (DIM / 4); i += 256) {
    const uint32_t row = i / (DIM / 4), d = i % (DIM / 4) * 4;
    if (row >= t.rows) break;
    float top = m_s[0][row];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) top = fmaxf(top, m_s[w][row]);
    const float shift = top == -INFINITY ? 0.f : top;
    float total = 0.f;
    v4f sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const float f = __builtin_amdgcn_exp2f(m_s[w][row] - shift);
      total += l_s[w][row] * f;
      sum += *(const v4f*)&o_s[w][row][d] * f;
    }
    if (shared) {
      *(v4f*)(a.part + (slot * BM + row) * DIM + d) = sum;
      if (d == 0) a.stat[slot * BM + row] = make_float2(top, total);
    } else {
      const uint32_t packed = t.r0 + row, qr = packed / a.group, head = h * a.group + packed % a.group;
      const float inv = total == 0.f ? 0.f : 1.f / total;
      sum *= inv;
      const uint64_t at = ((uint64_t)(t.row0 + qr) * a.heads + head) * DIM + d;
      if (DT == DT_BF16) *(uint2*)(a.out[r] + at * 2) = make_uint2(pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]));
      else *(v4f*)(a.out[r] + at * 4) = sum;
      if (d == 0 && a.lse[r]) a.lse[r][(uint64_t)(t.row0 + qr) * a.heads + head] = total == 0.f ? -INFINITY : (shift + log2f(total)) * LN2;
    }
  }
}

// Joins the shares of a tile, BM rows of DIM: one workgroup per row tile, four
// dimensions per thread.
template <int DT, int DIM>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, uint32_t bm) {
  const uint32_t tile = blockIdx.x, h = blockIdx.y, r = blockIdx.z;
  Tile t;
  if (!tile_of(a, tile, bm, &t)) return;
  const uint32_t per = share_steps(a, t.steps);
  if (t.steps <= per) return;  // one share: stored whole
  const uint32_t shares = (t.steps + per - 1) / per;
  const uint64_t slot = (((uint64_t)r * a.kv_heads + h) * a.tiles + tile) * a.splits;
  for (uint32_t i = threadIdx.x; i < t.rows * (DIM / 4); i += 256) {
    const uint32_t row = i / (DIM / 4), d = i % (DIM / 4) * 4;
    float top = -INFINITY, total = 0.f;
    for (uint32_t s = 0; s < shares; ++s) top = fmaxf(top, a.stat[(slot + s) * bm + row].x);
    const float shift = top == -INFINITY ? 0.f : top;
    v4f sum = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t s = 0; s < shares; ++s) {
      const float2 st = a.stat[(slot + s) * bm + row];
      const float f = __builtin_amdgcn_exp2f(st.x - shift);
      total += st.y * f;
      sum += *(const v4f*)(a.part + ((slot + s) * bm + row) * DIM + d) * f;
    }
    const uint32_t packed = t.r0 + row, qr = packed / a.group, head = h * a.group + packed % a.group;
    sum *= total == 0.f ? 0.f : 1.f / total;
    const uint64_t at = ((uint64_t)(t.row0 + qr) * a.heads + head) * DIM + d;
    if (DT == DT_BF16) *(uint2*)(a.out[r] + at * 2) = make_uint2(pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]));
    else *(v4f*)(a.out[r] + at * 4) = sum;
    if (d == 0 && a.lse[r]) a.lse[r][(uint64_t)(t.row0 + qr) * a.heads + head] = total == 0.f ? -INFINITY : (shift + log2f(total)) * LN2;
  }
}

// How a call is cut.
struct AttnPlan {
  uint32_t bm, tiles, splits, min_steps;
  uint64_t part_bytes, stat_bytes;
  uint64_t bytes() const { return part_bytes + stat_bytes; }
};

AttnPlan plan_of(int n, uint64_t seqs, uint64_t rows, uint64_t tokens, uint64_t heads, uint64_t kv_heads, uint64_t dim) {
  AttnPlan p;
  const uint64_t group = heads / kv_heads;
  p.bm = 16;
  p.tiles = (uint32_t)item_count(rows, seqs, group, p.bm, 1);
  // Tiles that may be real: a sequence's last one is counted twice above.
  const uint64_t real = umax(1, umin(p.tiles, (rows * group + p.bm - 1) / p.bm + seqs - 1));
  const uint64_t steps = (tokens + TOKENS - 1) / TOKENS;
  p.min_steps = 16;
  p.splits = (uint32_t)umax(1, umin((steps + p.min_steps - 1) / p.min_steps, (1024 + real * n * kv_heads - 1) / (real * n * kv_heads)));
  const uint64_t slots = p.splits > 1 ? (uint64_t)n * kv_heads * p.tiles * p.splits : 0;
  p.part_bytes = layer_align(slots * p.bm * dim * 4);
  p.stat_bytes = layer_align(slots * p.bm * 8);
  return p;
}

ar_status check_heads(const ar_kv_cache* c, size_t rows, size_t heads, int dtype) {
  if (dtype < 0 || dtype > 2) return AR_ERR_INVALID;
  if (dtype == DT_I32) return AR_ERR_UNSUPPORTED;
  if (heads < 1 || heads % c->kv_heads) return AR_ERR_INVALID;
  if (heads > MAX_HEADS || rows * heads > LAYER_MAX_ROWS) return AR_ERR_TOO_LARGE;
  return AR_OK;
}

}  // namespace

extern "C" {

size_t ar_cache_attention_workspace(const ar_kv_cache* cache, size_t seqs, size_t rows, size_t width, size_t heads,
                                    size_t max_rows, ar_dtype dtype) {
  if (check_cache(cache) != AR_OK || rows > LAYER_MAX_ROWS || seqs > (1ull << 20) || width > (1ull << 31) ||
      width * cache->page >= (1ull << 31) || check_heads(cache, rows, heads, (int)dtype) != AR_OK || !rows || !seqs)
    return 0;
  (void)max_rows;
  return (size_t)plan_of(cache->nranks, seqs, rows, width * cache->page, heads, cache->kv_heads, cache->head_dim).bytes();
}

ar_status ar_cache_attention(const ar_kv_cache* cache, const void* const* q, size_t q_stride,
                             const ar_paged_rows* rows, void* const* out, float* const* lse, size_t heads,
                             float scale, int causal, size_t window, size_t max_rows, ar_dtype dtype,
                             void* workspace, size_t workspace_bytes, ar_stream_t stream) {
  ar_status st = check_cache(cache);
  if (st == AR_OK) st = check_rows(cache, rows);
  if (st == AR_OK) st = check_heads(cache, rows->rows, heads, (int)dtype);
  if (st != AR_OK) return st;
  if (!q || !out || causal < 0 || causal > 1 || (window && !causal) || !(fabsf(scale) < INFINITY)) return AR_ERR_INVALID;
  if (rows->rows == 0 || rows->seqs == 0) return AR_OK;
  const uint64_t es = dtype == AR_BF16 ? 2 : 4, width = heads * cache->head_dim;
  if (!stride_ok(q_stride, width, es)) return AR_ERR_INVALID;
  const int n = cache->nranks;
  const AttnPlan plan = plan_of(n, rows->seqs, rows->rows, rows->width * cache->page, heads, cache->kv_heads, cache->head_dim);
  (void)max_rows;
  AttnArgs a;
  LayerBuffers b;
  for (int r = 0; r < n; ++r) {
    a.q[r] = (const char*)q[r];
    a.out[r] = (char*)out[r];
    a.lse[r] = lse ? lse[r] : nullptr;
    a.k[r] = (const uint8_t*)cache->k[r];
    a.v[r] = (const uint8_t*)cache->v[r];
    a.k_scale[r] = (const uint8_t*)cache->k_scale[r];
    a.v_scale[r] = (const uint8_t*)cache->v_scale[r];
    b.in(q[r], span_bytes(rows->rows, q_stride, width, es));
    b.out(out[r], rows->rows * width * es);
    if (lse) b.out(lse[r], rows->rows * heads * 4, 4);
  }
  add_cache(b, cache, false);
  add_rows(b, rows);
  b.out(workspace, plan.bytes());
  if (!b.ok()) return AR_ERR_INVALID;
  if (workspace_bytes < plan.bytes()) return AR_ERR_TOO_LARGE;
  a.q_pitch = q_stride * es;
  a.p = paged_of(cache, rows);
  a.kv_heads = (uint32_t)cache->kv_heads;
  a.heads = (uint32_t)heads;
  a.group = (uint32_t)(heads / cache->kv_heads);
  a.splits = plan.splits;
  a.min_steps = plan.min_steps;
  a.tiles = plan.tiles;
  a.scale = scale * LOG2E;
  a.causal = causal;
  a.window = (uint32_t)umin(window, 0x7fffffff);
  a.part = (float*)workspace;
  a.stat = (float2*)((char*)workspace + plan.part_bytes);
  const dim3 grid(plan.tiles * plan.splits, a.kv_heads, n), joins(plan.tiles, a.kv_heads, n);
  by_head_dim((int)dtype, cache->head_dim, [&](auto dt, auto dim) {
    constexpr int DT = decltype(dt)::value, DIM = decltype(dim)::value;
    few_rows_kernel<DT, DIM><<<grid, 256, 0, (hipStream_t)stream>>>(a);
    if (plan.splits > 1) join_kernel<DT, DIM><<<joins, 256, 0, (hipStream_t)stream>>>(a, plan.bm);
  });
  return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP;
}

}  // extern "C"
