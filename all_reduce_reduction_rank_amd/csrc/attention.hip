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
typedef float v16f __attribute__((ext_vector_type(16)));
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
  uint32_t kv_heads, heads, group, nranks;
  uint32_t splits, min_steps;  // shares of a tile's tokens: at most `splits`, of at least `min_steps` steps
  uint32_t tiles;              // row tiles of a head (bound)
  // z in units of log2: factor * (q . k), factor > 0; a negative scale turns the
  // queries' signs instead (a multiply-add from the raw product then gives the
  // exponent, and the largest product is the largest z)
  float factor;
  uint32_t flip;
  int32_t causal;
  int32_t window;
  float* part;   // [rank][kv head][tile][split][rows of a tile][dim]: sum p v of a share
  float2* stat;  // [rank][kv head][tile][split][rows of a tile]: its m (of log2) and sum p
};

// A tile of packed rows of one sequence and the tokens its rows see.
struct Tile {
  uint32_t s, row0, n;  // sequence, its first row in the call, its rows
  uint32_t r0, rows;    // packed rows r0 .. r0 + rows - 1
  int32_t length;       // cached tokens (below 2^31, as every position)
  int32_t lo, hi;       // tokens some row sees lie in [lo, hi)
  uint32_t begin, steps;  // steps of TOKENS tokens from token `begin` on
};

__device__ __forceinline__ bool tile_of(const AttnArgs& a, uint32_t tile, uint32_t bm, Tile* t) {
  uint64_t local;
  int32_t len;
  t->s = find_sequence(a.p, tile, a.group, bm, 1, &t->row0, &t->n, &local, &len);
  if (t->s >= a.p.seqs) return false;
  const uint64_t rows = (uint64_t)t->n * a.group, r0 = local * bm;
  if (r0 >= rows) return false;
  t->r0 = (uint32_t)r0;
  t->rows = (uint32_t)(rows - r0 < bm ? rows - r0 : bm);
  const int32_t cap = (int32_t)(a.p.width << a.p.page_shift);
  len = len < 0 ? 0 : len < cap ? len : cap;
  t->length = len;
  t->lo = 0;
  t->hi = len;
  if (a.causal) {
    const int32_t n = (int32_t)t->n, last = len - n + (int32_t)((t->r0 + t->rows - 1) / a.group) + 1;
    t->hi = last < 0 ? 0 : last < len ? last : len;
    if (a.window) {
      const int32_t end = len - n + (int32_t)(t->r0 / a.group) + 1, first = end > a.window ? end - a.window : 0;
      t->lo = first < t->hi ? first : t->hi;
    }
  }
  t->begin = (uint32_t)t->lo & ~(TOKENS - 1);
  t->steps = t->hi > t->lo ? ((uint32_t)t->hi - t->begin + TOKENS - 1) / TOKENS : 0;
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

// x in TERMS bf16 terms: each holds what the ones before it left.  WIDE: x may be any
// fp32 number; those beyond bf16's largest would round to infinity and leave NaN, so
// the first term stops there.
template <int TERMS, bool WIDE = false>
__device__ __forceinline__ void split8(float* x, v8bf* out) {
  constexpr float MOST = 0x1.fep+127f;
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    v4u w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (WIDE && t == 0) w[i] = pack_bf16(__builtin_amdgcn_fmed3f(x[2 * i], -MOST, MOST), __builtin_amdgcn_fmed3f(x[2 * i + 1], -MOST, MOST));
      else w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
      if (t + 1 < TERMS) x[2 * i] -= low_of(w[i]), x[2 * i + 1] -= high_of(w[i]);
    }
    out[t] = __builtin_bit_cast(v8bf, w);
  }
}

// x rounded to bf16, and the sum of what that gives added to *sum.
__device__ __forceinline__ v8bf rounded8(const float* x, float* sum) {
  const v2bf one = {(__bf16)1.f, (__bf16)1.f};
  v4u w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    *sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, (uint32_t)w[i]), one, *sum, false);
  }
  return __builtin_bit_cast(v8bf, w);
}

__device__ __forceinline__ uint4 flipped(const uint4& w, uint32_t f) { return make_uint4(w.x ^ f, w.y ^ f, w.z ^ f, w.w ^ f); }

__device__ __forceinline__ uint32_t clamp_byte(uint32_t b) { return b < SCALE_MIN ? SCALE_MIN : b > SCALE_MAX ? SCALE_MAX : b; }
__device__ __forceinline__ float byte_scale(uint32_t b) { return scale_of(clamp_byte(b)); }

// ---- what a row does not see ----
//
// Its weight is 0, but 0 times a NaN or an infinity is NaN. Codes of tokens that no
// row of a tile sees are cleared in the steps where a mask runs through the tile.
// Codes that stand for no number are cleared there too where some rows see the token
// and others do not; the rows that do get their NaN at the end, from another look at
// those steps. (In all other steps every row sees every token.) With a NaN that rows
// see in the first and the last 64 tokens: a prompt of 1500 tokens takes the time it
// takes without; with rows done again in plain loops it took 135 times as long.

// The tokens [all0, all1) that every row of a tile sees.
struct Mask {
  int32_t all0, all1;
  __device__ __forceinline__ Mask(const Tile& t, const AttnArgs& a) {
    all0 = 0, all1 = t.length;
    if (a.causal) {
      const int32_t end = t.length - (int32_t)t.n + 1;
      const int32_t e = end + (int32_t)(t.r0 / a.group), f = end + (int32_t)((t.r0 + t.rows - 1) / a.group);
      all1 = e < 0 ? 0 : e;
      if (a.window && f > a.window) all0 = f - a.window;
    }
  }
  __device__ __forceinline__ bool step(int32_t base) const { return base < all0 || base > all1 - (int32_t)TOKENS; }
  __device__ __forceinline__ bool token(int32_t at) const { return at < all0 || at >= all1; }
};

// The smallest magnitude of a code that stands for no finite number: NaN, or with
// scales of 2^120 and more 2^128 and above.
__device__ __forceinline__ uint32_t not_finite_from(uint32_t byte) {
  return byte < 247 ? 0x7fu : 0x78u - 8 * (byte - 247);
}

// The high bit of every byte whose code is one of those.
__device__ __forceinline__ uint32_t not_finite(uint32_t codes, uint32_t from) {
  return ((codes & 0x7f7f7f7fu) + (0x80u - from) * 0x01010101u) & 0x80808080u;
}

// Bytes of a 16-token block of codes that lie outside tokens [lo, hi) become 0;
// `at` is the block's first token.
__device__ __forceinline__ uint4 clear_outside(uint4 w, int32_t at, int32_t lo, int32_t hi) {
  uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (at + 4 * i + e < lo || at + 4 * i + e >= hi) x[i] &= ~(0xffu << (8 * e));
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// Clears those of a block that some rows do not see; *taken becomes 1 if there are any.
__device__ __forceinline__ uint4 clear_unseen(uint4 w, uint32_t from, int32_t at, const Mask& m, uint32_t* taken) {
  uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t bad = not_finite(x[i], from);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((bad >> (8 * e + 7) & 1) && m.token(at + 4 * i + e)) x[i] &= ~(0xffu << (8 * e)), *taken = 1;
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// A bit for each token of a block that some rows do not see and that holds no number.
__device__ __forceinline__ uint16_t hidden_bits(uint4 w, uint32_t from, int32_t at, const Mask& m) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if ((not_finite(x[i / 4], from) >> (8 * (i % 4) + 7) & 1) && m.token(at + i)) bits |= 1u << i;
  return (uint16_t)bits;
}

// Bits of the tokens [from, to) of a step.
__device__ __forceinline__ uint64_t token_bits(int32_t from, int32_t to) {
  const uint64_t below = to >= 64 ? ~0ull : to > 0 ? (1ull << to) - 1 : 0;
  return from >= 64 ? 0 : from > 0 ? below & (~0ull << from) : below;
}

// A dimension's tokens of a step, 16 bits of each block, written by four lanes and read as one.
typedef uint16_t __attribute__((may_alias)) bits16;
typedef uint64_t __attribute__((may_alias)) bits64;

// ---- few rows: 16 rows per workgroup, its four or eight waves share the tokens ----
//
// The waves take the steps of 64 tokens in turn, straight from memory to
// registers, each with a softmax of its own, joined at the end; a long cache is
// shared among workgroups and joined by a second kernel.  Bound by memory: a
// step is 64 x 2 x dim bytes of codes, loaded 16 bytes per lane one step ahead
// (64 sequences of 8192 tokens, 8 key heads of 128: 198 us, 5.4 TB/s; with
// entries and scales waited for as they were loaded 271).
//
// Matrix instructions 16x16x32, keys as the first operand: S^T[token][row].
// The order of k is free as long as both operands share it, and so is the
// order of tokens; both are chosen so that lanes load contiguous bytes and
// weights stay in the lanes that hold them.  With lane = 16 g + c:
//   keys   step a (0..3), row c of the operand: token 16 (c / 4) + 4 a + c % 4,
//          k: 16 contiguous values of every 64, from 16 g on, so that a load
//          takes 64 contiguous bytes of each key
//   S^T    lane (g, c) holds tokens 16 g + 4 a + i (i = 0..3) of row c
//   values operand row c: dimension 16 t + c, k of group g: tokens 16 g ..
//          16 g + 15, which are one 16-byte load (a page is whole blocks of 16)
//   O^T    lane (g, c) holds dimensions 16 t + 4 g + i of row c
//
template <int DT, int DIM, int WAVES>
__global__ __launch_bounds__(64 * WAVES, WAVES == 8 || DT == DT_BF16 && DIM <= 128 || DIM == 64 ? 2 : 1) void few_rows_kernel(AttnArgs a) {
  constexpr int BM = 16;
  constexpr int KSTEPS = DIM / 32, KW = DIM / 64;  // instructions of q . k; 16-byte loads of a key
  constexpr int DT_TILES = DIM / 16;
  constexpr int QT = DT == DT_BF16 ? 1 : 3;  // terms of q
  constexpr int PT = DT == DT_BF16 ? 2 : 3;  // terms of the weights
  constexpr uint32_t ES = DT == DT_BF16 ? 2 : 4;
  constexpr int PITCH = DIM + 4;
  __shared__ float o_s[WAVES][BM][PITCH];
  __shared__ float m_s[WAVES][BM], l_s[WAVES][BM];
  // One term of q stays in registers, three would not fit beside the rest.
  constexpr bool Q_LDS = QT > 1;
  __shared__ uint4 q_s[Q_LDS ? KSTEPS * QT * 64 : 1];

  uint32_t r;
  const uint32_t item = item_of(a.nranks, &r), split = item % a.splits, tile = item / a.splits, h = blockIdx.y;
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
  int32_t see0 = 0, see1 = real ? t.length : 0;
  if (a.causal && real) {
    const int32_t e = t.length - (int32_t)t.n + (int32_t)qrow + 1;
    see1 = e < 0 ? 0 : e;
    if (a.window && e > a.window) see0 = e - a.window;
  }
  v8bf q[Q_LDS ? 1 : KSTEPS];
  {
    const char* at = a.q[r] + (uint64_t)(t.row0 + qrow) * a.q_pitch + (uint64_t)qhead * (DIM * ES) + g * 16 * ES;
    if constexpr (!Q_LDS) {
#pragma unroll
      for (int s = 0; s < KSTEPS; ++s)
        q[s] = __builtin_bit_cast(v8bf, flipped(real ? ld16(at + (s / 2 * 64 + s % 2 * 8) * 2) : make_uint4(0, 0, 0, 0), a.flip));
    } else {
      for (int s = wave; s < KSTEPS; s += WAVES) {
        const char* from = at + (s / 2 * 64 + s % 2 * 8) * 4;
        const uint4 w = real ? ld16(from) : make_uint4(0, 0, 0, 0), u = real ? ld16(from + 16) : make_uint4(0, 0, 0, 0);
        float x[8] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w),
                      __uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
        if (a.flip)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = -x[e];
        v8bf terms[QT];
        split8<QT, true>(x, terms);
#pragma unroll
        for (int y = 0; y < QT; ++y) q_s[(s * QT + y) * 64 + lane] = __builtin_bit_cast(uint4, terms[y]);
      }
      __syncthreads();
    }
  }
  const Mask seen(t, a);
  const bool differ = seen.all0 > t.lo || seen.all1 < t.hi;  // some rows do not see tokens that others see
  uint32_t taken = 0;

  v4f o[DT_TILES];
  float m, l;
  uint4 kw[4][KW], vw[DT_TILES];
  // What a load brings is not touched before its step, so that nothing waits:
  // the table's entries of the step to load next, the scales' bytes of the one
  // that is loaded.
  uint32_t kid, vid, kbyte, vbyte;
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
      const uint8_t* at = kc + page_at(kid, a.kv_heads, h, page_bytes) + (off + koff) * DIM + g * 16;
      kbyte = a.k_scale[r][(uint64_t)kid * a.kv_heads + h];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < KW; ++j) kw[i][j] = ld16((const char*)at + i * 4 * DIM + j * 64);
    } else {
      kbyte = 127;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < KW; ++j) kw[i][j] = make_uint4(0, 0, 0, 0);
    }
  };
  auto load_v = [&](uint32_t step) {
    const uint64_t base = (uint64_t)t.begin + (uint64_t)step * TOKENS + 16 * g;
    const uint32_t off = (uint32_t)base & ((1u << a.p.page_shift) - 1);
    there = vid < a.p.pages;
    if (there) {
      const uint8_t* at = vc + page_at(vid, a.kv_heads, h, page_bytes) + (c << a.p.page_shift) + off;
      vbyte = a.v_scale[r][(uint64_t)vid * a.kv_heads + h];
#pragma unroll
      for (int i = 0; i < DT_TILES; ++i) vw[i] = ld16((const char*)at + ((16 * i) << a.p.page_shift));
    } else {
      vbyte = 127;
#pragma unroll
      for (int i = 0; i < DT_TILES; ++i) vw[i] = make_uint4(0, 0, 0, 0);
    }
  };

  {
#pragma unroll
    for (int i = 0; i < DT_TILES; ++i) o[i] = (v4f){0.f, 0.f, 0.f, 0.f};
    m = -INFINITY;
    l = 0.f;
    uint32_t step = step0 + wave;
    if (step < step1) {
      ids(step);
      load_k(step);
      load_v(step);
      ids(step + WAVES);
    }
    for (; step < step1; step += WAVES) {
      const int32_t base = (int32_t)(t.begin + step * TOKENS);
      const bool more = step + WAVES < step1;
      const float ks = byte_scale(kbyte);
      v4f s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < KSTEPS; ++j) {
        v8bf qj[QT];
#pragma unroll
        for (int x = 0; x < QT; ++x) {
          if constexpr (Q_LDS) qj[x] = __builtin_bit_cast(v8bf, q_s[(j * QT + x) * 64 + lane]);
          else qj[x] = q[j];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = kw[i][j / 2];
          const v8bf k8 = j % 2 ? widen8(w.z, w.w, ks) : widen8(w.x, w.y, ks);
#pragma unroll
          for (int x = QT - 1; x >= 0; --x) s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8, qj[x], s[i], 0, 0, 0);
        }
      }
      if (more) load_k(step + WAVES);
      const bool mask = seen.step(base) || __any(!there);
      const int32_t first = base + 16 * (int32_t)g;
      float p[16];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float z = s[i][e];
          if (mask) {
            const int32_t at = first + 4 * i + e;
            if (at < see0 || at >= see1 || !there) z = -INFINITY;
          }
          p[4 * i + e] = z;
        }
      {
        float top = p[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, p[i]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        // The maximum follows only when it has grown by more than 2^8: weights of
        // up to that are as good.
        if (__any((top - m) * a.factor > 8.f)) {
          const float next = fmaxf(m, top), f = next == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - next) * a.factor);
          m = next;
          l *= f;
#pragma unroll
          for (int i = 0; i < DT_TILES; ++i) o[i] *= f;
        }
        const float shift = m == -INFINITY ? 0.f : m * a.factor;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[i], a.factor, -shift));
          l += p[i];
        }
      }
      v8bf w[2][PT];
      split8<PT>(p, w[0]);
      split8<PT>(p + 8, w[1]);
      if (base < t.lo || base > t.hi - (int32_t)TOKENS) {
#pragma unroll
        for (int i = 0; i < DT_TILES; ++i) vw[i] = clear_outside(vw[i], first, t.lo, t.hi);
      }
      // (looked for first: taking them out costs 4 us of a decode step)
      if (differ && seen.step(base)) {
        const uint32_t from = not_finite_from(clamp_byte(vbyte));
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < DT_TILES; ++i)
          bad |= not_finite(vw[i].x, from) | not_finite(vw[i].y, from) | not_finite(vw[i].z, from) | not_finite(vw[i].w, from);
        if (__any(bad != 0)) {
#pragma unroll
          for (int i = 0; i < DT_TILES; ++i) vw[i] = clear_unseen(vw[i], from, first, seen, &taken);
        }
      }
      const float vs = byte_scale(vbyte);
#pragma unroll
      for (int i = 0; i < DT_TILES; ++i) {
        const v8bf lo = widen8(vw[i].x, vw[i].y, vs), hi = widen8(vw[i].z, vw[i].w, vs);
        // fp32 payloads: a step's sum on its own, so that a long sequence rounds the
        // whole sum once a step and not once an instruction
        v4f sum = PT == 3 ? (v4f){0.f, 0.f, 0.f, 0.f} : o[i];
#pragma unroll
        for (int x = PT - 1; x >= 0; --x) {
          sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, w[0][x], sum, 0, 0, 0);
          sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, w[1][x], sum, 0, 0, 0);
        }
        o[i] = PT == 3 ? o[i] + sum : sum;
      }
      if (more) {
        load_v(step + WAVES);
        ids(step + 2 * WAVES);
      }
    }
  }

  if (__any(taken)) {
    static_assert(DIM * 8 <= BM * PITCH * 4, "a wave's part of o_s, free until the waves are joined, holds a step's bits");
    bits16* hidden = (bits16*)o_s[wave];  // [DIM][4]
#pragma nounroll
    for (uint32_t step = step0 + wave; step < step1; step += WAVES) {
      const int32_t base = (int32_t)(t.begin + step * TOKENS);
      if (!seen.step(base)) continue;
      ids(step);
      load_v(step);
#pragma unroll
      for (int i = 0; i < DT_TILES; ++i) hidden[(16 * i + c) * 4 + g] = hidden_bits(vw[i], not_finite_from(clamp_byte(vbyte)), base + 16 * (int32_t)g, seen);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const uint64_t own = token_bits(see0 - base, see1 - base);
#pragma unroll
      for (int i = 0; i < DT_TILES; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (((const bits64*)hidden)[16 * i + 4 * g + e] & own) o[i][e] = __builtin_nanf("");
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }

  const uint64_t slot = (((uint64_t)r * a.kv_heads + h) * a.tiles + tile) * a.splits + split;
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);

  // Join the waves.
  if (g == 0) m_s[wave][c] = m * a.factor, l_s[wave][c] = l;
#pragma unroll
  for (int i = 0; i < DT_TILES; ++i) *(v4f*)&o_s[wave][c][16 * i + 4 * g] = o[i];
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < BM * (DIM / 4); i += 64 * WAVES) {
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

// ---- many rows: 128 rows per workgroup, 32 per wave, the codes shared in LDS ----
//
// Bound by the vector units and the matrix cores in turn: the softmax, and the
// waits of two waves per SIMD that share both.  The codes are widened once, on
// their way into LDS; widened by every wave from codes in LDS they cost more
// than the larger LDS reads (prompt of 8192 tokens, 40 heads of 128: 941 us, 815
// so; 795 to 830 by the machine's clock now, 0.83 to 0.87 PFLOP/s).  The e4m3 instructions with block scales would take the keys' codes
// as they are, but their sums over 64 products keep fewer than fp32's bits
// (scores off by 2^-18 of their terms' size, measured).  A step of 64 tokens is
// loaded to registers one step ahead and stored to the other of two LDS buffers.
//
// Matrix instructions 32x32x16, keys as the first operand, with lane = 32 h + c:
//   S^T    operand row i of x (0, 1) is token 32 ((i >> 2) & 1) + 16 x +
//          4 (i >> 3) + (i & 3): lane (h, c) then holds tokens 32 h + 16 x +
//          0 .. 15 of row c, which is the order the weights enter the second
//          product in, without leaving their lane
//   keys   k of half h: 8 contiguous values of every 16, from 8 h on
//   values operand row: dimension 32 t + c, k of half h: tokens 32 h .. + 31
// LDS rows (a token's key, a dimension's 64 values) hold their 16-byte chunks
// permuted, so that the 16 rows that 16 neighbouring lanes read lie on 16 chunks
// of the 256 bytes of banks: values two rows to 256 bytes, hence by the row's
// number over 2; keys, whose rows a wave reads in the order above, by the bits
// that differ there.
__device__ __forceinline__ uint32_t key_turn(uint32_t key, uint32_t row_chunks) {
  return ((key & 3) | (key >> 3 & 4) | (key << 1 & 8)) & (row_chunks - 1);
}

template <int DT, int DIM>
__global__ __launch_bounds__(256, (DT == DT_BF16 && DIM <= 128) || DIM == 64 ? 2 : 1) void many_rows_kernel(AttnArgs a) {
  constexpr int WAVES = 4, THREADS = 64 * WAVES, BM = 32 * WAVES;
  constexpr int KSTEPS = DIM / 16, DT_TILES = DIM / 32;
  constexpr int KCHUNKS = DIM / 16;               // 16-byte chunks of a key
  constexpr int NC = 4 * DIM / THREADS;           // chunks a thread moves, of keys and of values
  constexpr int QT = DT == DT_BF16 ? 1 : 3, PT = DT == DT_BF16 ? 1 : 3;
  constexpr uint32_t ES = DT == DT_BF16 ? 2 : 4;
  constexpr int KROW = DIM / 8;                   // LDS chunks of a key
  __shared__ uint4 k_s[2][8 * DIM], v_s[2][8 * DIM];  // bf16
  __shared__ uint32_t there_s[2][4];                  // the 16-token blocks: on a page

  const uint32_t columns = a.kv_heads * a.nranks;
  uint32_t b = blockIdx.x;
  if (blockIdx.z) b += blockIdx.z * gridDim.x;  // (below 2^32: the host checks)
  const uint32_t column = b % columns, item = b / columns;
  const uint32_t h = column % a.kv_heads, r = column / a.kv_heads;
  // (past the last item `tile` is beyond every sequence's)
  const uint32_t split = item % a.splits, tile = a.tiles - 1 - item / a.splits;
  Tile t;
  if (!tile_of(a, tile, BM, &t)) return;
  const uint32_t per = share_steps(a, t.steps), step0 = split * per;
  if (split && step0 >= t.steps) return;
  const uint32_t step1 = step0 + per < t.steps ? step0 + per : t.steps;
  const bool shared = t.steps > per;

  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, hf = lane >> 5, c = lane & 31;
  const uint32_t page_bytes = DIM << a.p.page_shift;

  // This lane's row, the tokens it sees and those its wave's rows see.
  const uint32_t wr = wave * 32, row = wr + c, rho = t.r0 + row;
  const bool real = row < t.rows;
  const uint32_t qrow = real ? rho / a.group : 0, qhead = h * a.group + (real ? rho - qrow * a.group : 0);
  int32_t see0 = 0, see1 = real ? t.length : 0, some0 = 0, some1 = wr < t.rows ? t.length : 0, all0 = 0, all1 = t.length;
  if (a.causal && wr < t.rows) {
    const int32_t end = t.length - (int32_t)t.n + 1;
    const uint32_t last = t.r0 + (wr + 31 < t.rows ? wr + 31 : t.rows - 1);
    const int32_t e = end + (int32_t)qrow, e0 = end + (int32_t)((t.r0 + wr) / a.group), e1 = end + (int32_t)(last / a.group);
    if (real) see1 = e < 0 ? 0 : e;
    all1 = e0 < 0 ? 0 : e0;
    some1 = e1 < 0 ? 0 : e1;
    if (a.window) {
      see0 = e > a.window ? e - a.window : 0;
      some0 = e0 > a.window ? e0 - a.window : 0;
      all0 = e1 > a.window ? e1 - a.window : 0;
    }
  }
  const Mask seen(t, a);
  uint32_t taken = 0;
  v8bf q[KSTEPS][QT];
  {
    const char* at = a.q[r] + (uint64_t)(t.row0 + qrow) * a.q_pitch + (uint64_t)qhead * (DIM * ES) + hf * 8 * ES;
#pragma unroll
    for (int s = 0; s < KSTEPS; ++s) {
      if (DT == DT_BF16) {
        q[s][0] = __builtin_bit_cast(v8bf, flipped(real ? ld16(at + s * 32) : make_uint4(0, 0, 0, 0), a.flip));
      } else {
        const uint4 w = real ? ld16(at + s * 64) : make_uint4(0, 0, 0, 0), u = real ? ld16(at + s * 64 + 16) : make_uint4(0, 0, 0, 0);
        float x[8] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w),
                      __uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
        if (a.flip)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = -x[e];
        split8<QT, true>(x, q[s]);
      }
    }
  }

  v16f o[DT_TILES];
  // l: sum of the weights; lr: of the weights as they are multiplied.  One bf16
  // term is off by up to 2^-8 of it (a second one costs a quarter of the kernel's time:
  // prompt of 8192 tokens 829 -> 1065 us); over lr a row that one token dominates has
  // that error in both and loses it.  lse goes by l.
  float m, l, lr;
  // Of the blocks of 16 tokens, lane by lane block tid % 4: the page of the step to
  // load next, the scales of the one that is loaded (as the entries, not touched
  // before their step).  A wave's chunk i of keys lies in one block and takes both
  // from a lane that has them: held by every lane for its own chunks they were
  // short of registers with heads of 256, and waited for where they moved.
  uint32_t vid, kbyte, vbyte;
  uint4 kx[NC], vx[NC];
  bool there;  // block tid % 4 is on a page
  const uint32_t wave64 = __builtin_amdgcn_readfirstlane(tid & ~63u);
  auto key_block = [&](int i) { return (wave64 + i * THREADS) / DIM; };
  // A page of 64 tokens or more holds a whole step: one page, the same for
  // every thread, whose address scalar registers keep.
  const bool whole = a.p.page_shift >= 6;
  auto ids = [&](uint32_t step) {
    const uint64_t base = (uint64_t)t.begin + (uint64_t)step * TOKENS;
    vid = page_id(a.p, t.s, (whole ? base : base + 16 * (tid & 3)) >> a.p.page_shift);
  };
  auto load = [&](uint32_t step) {
    const uint32_t base = t.begin + step * TOKENS, in_page = (1u << a.p.page_shift) - 1;
    there = vid < a.p.pages;
    kbyte = vbyte = 127;
    if (whole) {
      const uint32_t id = __builtin_amdgcn_readfirstlane(vid);
      if (id < a.p.pages) {
        const uint64_t at = page_at(id, a.kv_heads, h, page_bytes);
        const uint8_t* kp = a.k[r] + at + (base & in_page) * DIM;
        const uint8_t* vp = a.v[r] + at + (base & in_page);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          kx[i] = ld16((const char*)kp + (tid + i * THREADS) * 16);
          vx[i] = ld16((const char*)vp + (((tid + i * THREADS) / 4) << a.p.page_shift) + 16 * (tid & 3));
        }
        kbyte = a.k_scale[r][(uint64_t)id * a.kv_heads + h];
        vbyte = a.v_scale[r][(uint64_t)id * a.kv_heads + h];
      } else {
#pragma unroll
        for (int i = 0; i < NC; ++i) kx[i] = vx[i] = make_uint4(0, 0, 0, 0);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const uint32_t ch = tid + i * THREADS, id = __builtin_amdgcn_readlane(vid, key_block(i));
      kx[i] = make_uint4(0, 0, 0, 0);
      if (id < a.p.pages)
        kx[i] = ld16((const char*)a.k[r] + page_at(id, a.kv_heads, h, page_bytes) + ((base + ch / KCHUNKS) & in_page) * DIM +
                     ch % KCHUNKS * 16);
    }
    const uint8_t* at = a.v[r] + page_at(there ? vid : 0, a.kv_heads, h, page_bytes) + ((base + 16 * (tid & 3)) & in_page);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      vx[i] = make_uint4(0, 0, 0, 0);
      if (there) vx[i] = ld16((const char*)at + (((tid + i * THREADS) / 4) << a.p.page_shift));
    }
    if (there) {
      kbyte = a.k_scale[r][(uint64_t)vid * a.kv_heads + h];
      vbyte = a.v_scale[r][(uint64_t)vid * a.kv_heads + h];
    }
  };
  auto store = [&](uint32_t step, uint32_t buf) {
    const int32_t base = (int32_t)(t.begin + step * TOKENS);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const uint32_t ch = tid + i * THREADS, kr = ch / KCHUNKS, vr = ch / 4;
      const float ks = byte_scale(__builtin_amdgcn_readlane(kbyte, key_block(i))), vs = byte_scale(vbyte);
      uint4* kt = k_s[buf] + kr * KROW;
      kt[(ch % KCHUNKS * 2) ^ key_turn(kr, KROW)] = __builtin_bit_cast(uint4, widen8(kx[i].x, kx[i].y, ks));
      kt[(ch % KCHUNKS * 2 + 1) ^ key_turn(kr, KROW)] = __builtin_bit_cast(uint4, widen8(kx[i].z, kx[i].w, ks));
      uint4 w = vx[i];
      if (seen.step(base)) {
        const int32_t first = base + 16 * (int32_t)(tid & 3);
        const uint32_t from = not_finite_from(clamp_byte(vbyte));
        w = clear_outside(w, first, t.lo, t.hi);
        if (not_finite(w.x, from) | not_finite(w.y, from) | not_finite(w.z, from) | not_finite(w.w, from))
          w = clear_unseen(w, from, first, seen, &taken);
      }
      uint4* vt = v_s[buf] + vr * 8;
      vt[(2 * (tid & 3)) ^ ((vr >> 1) & 7)] = __builtin_bit_cast(uint4, widen8(w.x, w.y, vs));
      vt[(2 * (tid & 3) + 1) ^ ((vr >> 1) & 7)] = __builtin_bit_cast(uint4, widen8(w.z, w.w, vs));
    }
    if (tid < 4) there_s[buf][tid] = there;
  };

  const uint32_t kt = 32 * ((c >> 2) & 1) + 4 * (c >> 3) + (c & 3);  // this lane's key of x = 0
  // where its chunks lie in LDS: the chunk's number is exclusive-ored in
  const uint32_t ka0 = kt * KROW + (hf ^ key_turn(kt, KROW));
  const uint32_t va0 = c * 8 + ((4 * hf) ^ ((c >> 1) & 7));
  {
#pragma unroll
    for (int i = 0; i < DT_TILES; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[i][e] = 0.f;
    m = -INFINITY;
    l = lr = 0.f;
    if (step0 < step1) {
      ids(step0);
      load(step0);
      if (step0 + 1 < step1) ids(step0 + 1);
      store(step0, 0);
    }
    __syncthreads();
    for (uint32_t step = step0; step < step1; ++step) {
      const uint32_t buf = (step - step0) & 1;
      const bool more = step + 1 < step1;
      if (more) {
        load(step + 1);
        if (step + 2 < step1) ids(step + 2);
      }
      const int32_t base = (int32_t)(t.begin + step * TOKENS);
      if (base < some1 && base > some0 - (int32_t)TOKENS) {
        const bool gap = !there_s[buf][2 * hf] || !there_s[buf][2 * hf + 1];
        const bool mask = base < all0 || base > all1 - (int32_t)TOKENS || __any(gap);
        float p[2][16];
        v16f s[2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[x][e] = 0.f;
#pragma unroll
        for (int j = 0; j < KSTEPS; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const v8bf k8 = __builtin_bit_cast(v8bf, k_s[buf][(ka0 ^ (2 * j)) + x * 16 * KROW]);
#pragma unroll
            for (int y = QT - 1; y >= 0; --y) s[x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k8, q[j][y], s[x], 0, 0, 0);
          }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 16; ++e) p[x][e] = s[x][e];
        if (mask) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // tokens first + e with from <= e < to
            const int32_t first = base + 32 * (int32_t)hf + 16 * x, from = see0 - first;
            const int32_t to = there_s[buf][2 * hf + x] ? see1 - first : -1;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e < from || e >= to) p[x][e] = -INFINITY;
          }
        }
        {
          float top = p[0][0];
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, p[x][e]);
          top = fmaxf(top, __shfl_xor(top, 32));
          // The maximum follows only when it has grown by more than 2^8: weights
          // of up to that are as good, and rescaling the sums costs as much as
          // the rest of the softmax.
          if (__any((top - m) * a.factor > 8.f)) {
            const float next = fmaxf(m, top), f = next == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - next) * a.factor);
            m = next;
            l *= f;
            lr *= f;
#pragma unroll
            for (int i = 0; i < DT_TILES; ++i) o[i] *= f;
          }
        }
        const float shift = m == -INFINITY ? 0.f : m * a.factor;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            p[x][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[x][e], a.factor, -shift));
            l += p[x][e];
          }
          v8bf w[2][PT];
          if (PT == 1) {
            w[0][0] = rounded8(p[x], &lr);
            w[1][0] = rounded8(p[x] + 8, &lr);
          } else {
            split8<PT>(p[x], w[0]);
            split8<PT>(p[x] + 8, w[1]);
          }
#pragma unroll
          for (int i = 0; i < DT_TILES; ++i) {
            v16f sum;  // (as above: half a step's sum on its own)
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[e] = PT == 3 ? 0.f : o[i][e];
            const v8bf v0 = __builtin_bit_cast(v8bf, v_s[buf][(va0 ^ (2 * x)) + 256 * i]);
            const v8bf v1 = __builtin_bit_cast(v8bf, v_s[buf][(va0 ^ (2 * x + 1)) + 256 * i]);
#pragma unroll
            for (int y = PT - 1; y >= 0; --y) {
              sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v0, w[0][y], sum, 0, 0, 0);
              sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v1, w[1][y], sum, 0, 0, 0);
            }
            if (PT == 3) o[i] += sum;
            else o[i] = sum;
          }
        }
      }
      if (more) store(step + 1, buf ^ 1);
      __syncthreads();
    }
  }

  if (__syncthreads_or(taken)) {
    bits16* hidden = (bits16*)v_s;  // [DIM][4]
#pragma nounroll
    for (uint32_t step = step0; step < step1; ++step) {
      const int32_t base = (int32_t)(t.begin + step * TOKENS);
      if (!seen.step(base)) continue;
      ids(step);
      load(step);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NC; ++i)
        hidden[tid + i * THREADS] = hidden_bits(vx[i], not_finite_from(clamp_byte(vbyte)), base + 16 * (int32_t)(tid & 3), seen);
      __syncthreads();
      const uint64_t own = token_bits(see0 - base, see1 - base);
#pragma unroll
      for (int i = 0; i < DT_TILES; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (((const bits64*)hidden)[32 * i + 8 * (e / 4) + 4 * hf + e % 4] & own) o[i][e] = __builtin_nanf("");
    }
  }

  const uint64_t slot = ((((uint64_t)r * a.kv_heads + h) * a.tiles + tile) * a.splits + split) * BM;
  l += __shfl_xor(l, 32);
  if (PT == 1) lr += __shfl_xor(lr, 32);
  else lr = l;
  if (!real) return;
  if (shared) {
    const float f = lr == 0.f ? 0.f : l / lr;  // sums that go with l
#pragma unroll
    for (int i = 0; i < DT_TILES; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const v4f x = (v4f){o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]} * f;
        *(v4f*)(a.part + (slot + row) * DIM + 32 * i + 8 * e + 4 * hf) = x;
      }
    if (hf == 0) a.stat[slot + row] = make_float2(m * a.factor, l);
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / lr;
  const uint64_t at = ((uint64_t)(t.row0 + qrow) * a.heads + qhead) * DIM;
#pragma unroll
  for (int i = 0; i < DT_TILES; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const v4f x = (v4f){o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]} * inv;
      const uint64_t d = at + 32 * i + 8 * e + 4 * hf;
      if (DT == DT_BF16) *(uint2*)(a.out[r] + d * 2) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
      else *(v4f*)(a.out[r] + d * 4) = x;
    }
  if (hf == 0 && a.lse[r])
    a.lse[r][(uint64_t)(t.row0 + qrow) * a.heads + qhead] = l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m * a.factor) + log2f(l)) * LN2;
}

// Joins the shares of a tile, 16 rows per workgroup, four dimensions per thread.
constexpr uint32_t JOIN_ROWS = 16;

template <int DT, int DIM>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, uint32_t bm) {
  const uint32_t parts = bm / JOIN_ROWS, tile = blockIdx.x / parts, row0 = blockIdx.x % parts * JOIN_ROWS;
  const uint32_t h = blockIdx.y, r = blockIdx.z;
  Tile t;
  if (!tile_of(a, tile, bm, &t)) return;
  const uint32_t per = share_steps(a, t.steps);
  if (t.steps <= per) return;  // one share: stored whole
  const uint32_t shares = (t.steps + per - 1) / per;
  const uint64_t slot = (((uint64_t)r * a.kv_heads + h) * a.tiles + tile) * a.splits;
#pragma unroll
  for (uint32_t i = threadIdx.x; i < JOIN_ROWS * (DIM / 4); i += 256) {
    const uint32_t row = row0 + i / (DIM / 4), d = i % (DIM / 4) * 4;
    if (row >= t.rows) break;
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

constexpr bool eight_waves_fit(int dtype, uint64_t dim) { return dim == 64 || (dim == 128 && dtype == DT_BF16); }

// How a call is cut.
struct AttnPlan {
  bool few;
  uint32_t bm, tiles, splits, min_steps, waves;
  uint64_t part_bytes, stat_bytes;
  uint64_t bytes() const { return part_bytes + stat_bytes; }
};

AttnPlan plan_of(const ar_kv_cache* c, uint64_t seqs, uint64_t rows, uint64_t width, uint64_t heads, uint64_t window,
                 uint64_t max_rows, int dtype) {
  AttnPlan p;
  const uint64_t group = heads / c->kv_heads, columns = c->kv_heads * c->nranks;
  // Packed rows of a sequence: by the caller's word, or the mean.  Either kernel is
  // right for any number.  Tiles of 16 rows read the codes again for each 16, from
  // L2 beyond the first, and multiply twice; tiles of 128 are mostly empty with few
  // rows and start slowly.  (90 fp32 rows: 18 us against 45; 80 bf16 rows over 9000
  // tokens: 38 against 50; 32 sequences of 100 rows over 4000 tokens: 271 against
  // 159; 2 sequences of 100 rows over 200 tokens: 10 against 17.)  The table's width
  // stands for the lengths, which only the device knows.
  const uint64_t packed = (max_rows ? umin(max_rows, rows) : (rows + seqs - 1) / seqs) * group;
  const bool small = (rows * group / 16 + seqs) * columns <= 512 && width * c->page <= 1024;
  p.few = packed <= 96 || small;
  p.bm = p.few ? 16 : 128;
  p.tiles = (uint32_t)item_count(rows, seqs, group, p.bm, 1);
  // Tiles that may be real: a sequence's last one is counted twice above.
  const uint64_t real = umax(1, umin(p.tiles, (rows * group + p.bm - 1) / p.bm + seqs - 1)) * columns;
  // Steps of a tile, at most; a window's rows start and end inside one.
  uint64_t steps = (width * c->page + TOKENS - 1) / TOKENS;
  if (window) steps = umin(steps, (window + p.bm / group) / TOKENS + 2);
  p.min_steps = 8;
  p.waves = 4;
  const uint64_t most_splits = umax(1, (steps + p.min_steps - 1) / p.min_steps);
  // Workgroups that are resident together: two per CU, one where registers are short.
  // (Of 64 bf16 values a head three may be; shares for two were measured.)
  const uint64_t round = eight_waves_fit(dtype, c->head_dim) ? 512 : 256;
  if (p.few) {
    // One round of them if the tiles are few, else two: shares that fill a round
    // exactly leave CUs with one share too many (64 sequences of 8192 tokens, 8 key
    // heads of 128: one share each 234 us, two 198; 4 sequences of 32768: 16 shares
    // 56 us, 32 69).
    const uint64_t want = real < round / 2 ? round : 2 * round;
    p.splits = (uint32_t)umin(most_splits, (want + real - 1) / real);
    // Half a GPU's worth of tiles over not many tokens: eight waves of one workgroup
    // instead of a few workgroups and a second kernel to join them.  (Measured with 8 to
    // 480 tiles of heads of 64 and 128 over 2000 tokens: 128 tiles of 128 27 us shared, 21
    // so, 192 tiles 35 and 23, of 64 17 and 16, 21 and 17; equal within 4 % with 64
    // and 96 tiles; with 8 and 32, where the CUs' own bandwidth is short, 15 shared, 19 so;
    // with 480 tiles 49 and 59.  `real` counts a sequence's last tile up to twice: 176
    // tiles of 64 count as 344, and are better shared, 18 us and 22.)
    // Not where eight waves would be short of registers.
    const bool fits = eight_waves_fit(dtype, c->head_dim);
    if (p.splits > 1 && fits && real > 64 && real <= 256 && steps <= 48) p.waves = 8, p.splits = 1;
  } else {
    // Rounds of workgroups times the steps of each, where starting costs about four
    // steps more, and what joining costs, about six and more with the shares (42
    // fp32 rows of 256 over 20260 tokens, 8 tiles: 8 shares 550 us, 32 145).
    p.splits = 1;
    uint64_t best = (real + round - 1) / round * (steps + 4);
    for (uint64_t k = 2; k <= most_splits && k <= 64 && real < round; ++k) {
      const uint64_t cost = (real * k + round - 1) / round * ((steps + k - 1) / k + 4) + 6 + k / 8;
      if (cost < best) best = cost, p.splits = (uint32_t)k;
    }
  }
  const uint64_t slots = p.splits > 1 ? columns * p.tiles * p.splits : 0;
  p.part_bytes = layer_align(slots * p.bm * c->head_dim * 4);
  p.stat_bytes = layer_align(slots * p.bm * 8);
  return p;
}

ar_status check_heads(const ar_kv_cache* c, size_t rows, size_t seqs, size_t heads, int dtype) {
  if (dtype < 0 || dtype > 2) return AR_ERR_INVALID;
  if (dtype == DT_I32) return AR_ERR_UNSUPPORTED;
  if (heads < 1 || heads % c->kv_heads) return AR_ERR_INVALID;
  if (heads > MAX_HEADS || rows * heads > LAYER_MAX_ROWS) return AR_ERR_TOO_LARGE;
  // Tiles of every key head and rank are numbered in 32 bits.
  if (seqs * c->kv_heads * c->nranks > (1ull << 31)) return AR_ERR_TOO_LARGE;
  return AR_OK;
}

}  // namespace

extern "C" {

size_t ar_cache_attention_workspace(const ar_kv_cache* cache, size_t seqs, size_t rows, size_t width, size_t heads,
                                    size_t window, size_t max_rows, ar_dtype dtype) {
  if (check_cache(cache) != AR_OK || rows > LAYER_MAX_ROWS || seqs > (1ull << 20) || width > (1ull << 31) ||
      width * cache->page >= (1ull << 31) || check_heads(cache, rows, seqs, heads, (int)dtype) != AR_OK || !rows || !seqs)
    return 0;
  return (size_t)plan_of(cache, seqs, rows, width, heads, window, max_rows, (int)dtype).bytes();
}

ar_status ar_cache_attention(const ar_kv_cache* cache, const void* const* q, size_t q_stride,
                             const ar_paged_rows* rows, void* const* out, float* const* lse, size_t heads,
                             float scale, int causal, size_t window, size_t max_rows, ar_dtype dtype,
                             void* workspace, size_t workspace_bytes, ar_stream_t stream) {
  ar_status st = check_cache(cache);
  if (st == AR_OK) st = check_rows(cache, rows);
  if (st == AR_OK) st = check_heads(cache, rows->rows, rows->seqs, heads, (int)dtype);
  if (st != AR_OK) return st;
  if (!q || !out || causal < 0 || causal > 1 || (window && !causal) || !(fabsf(scale) < 1e38f)) return AR_ERR_INVALID;
  if (rows->rows == 0 || rows->seqs == 0) return AR_OK;
  const uint64_t es = dtype == AR_BF16 ? 2 : 4, width = heads * cache->head_dim;
  if (!stride_ok(q_stride, width, es)) return AR_ERR_INVALID;
  const int n = cache->nranks;
  const AttnPlan plan = plan_of(cache, rows->seqs, rows->rows, rows->width, heads, window, max_rows, (int)dtype);
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
  a.nranks = (uint32_t)n;
  a.group = (uint32_t)(heads / cache->kv_heads);
  a.splits = plan.splits;
  a.min_steps = plan.min_steps;
  a.tiles = plan.tiles;
  // (a factor of 0 would make NaN of what is masked; the smallest number there is makes
  // scores of less than 1e-6, whatever the products)
  a.factor = fmaxf(fabsf(scale * LOG2E), 0x1p-149f);
  a.flip = scale < 0.f ? 0x80008000u : 0u;
  a.causal = causal;
  a.window = (int32_t)umin(window, 0x7fffffff);
  a.part = (float*)workspace;
  a.stat = (float2*)((char*)workspace + plan.part_bytes);
  const Fold fold = fold_items((uint64_t)plan.tiles * plan.splits * (plan.few ? 1 : a.kv_heads * n), 64 * plan.waves);
  const dim3 grid(fold.x, plan.few ? a.kv_heads : 1, plan.few ? fold.folds * n : fold.folds);
  const dim3 joins(plan.tiles * (plan.bm / JOIN_ROWS), a.kv_heads, n);  // (few tiles, where they are shared)
  by_head_dim((int)dtype, cache->head_dim, [&](auto dt, auto dim) {
    constexpr int DT = decltype(dt)::value, DIM = decltype(dim)::value;
    if (plan.few) {
      if constexpr (eight_waves_fit(DT, DIM)) {
        if (plan.waves == 8) few_rows_kernel<DT, DIM, 8><<<grid, 512, 0, (hipStream_t)stream>>>(a);
        else few_rows_kernel<DT, DIM, 4><<<grid, 256, 0, (hipStream_t)stream>>>(a);
      } else {
        few_rows_kernel<DT, DIM, 4><<<grid, 256, 0, (hipStream_t)stream>>>(a);
      }
    } else many_rows_kernel<DT, DIM><<<grid, 256, 0, (hipStream_t)stream>>>(a);
    if (plan.splits > 1) join_kernel<DT, DIM><<<joins, 256, 0, (hipStream_t)stream>>>(a, plan.bm);
  });
  return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP;
}

}  // extern "C"
