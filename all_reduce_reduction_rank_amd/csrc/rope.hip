// rope.hip -- norms of queries and keys for each head with the rotation to
// their positions in one pass, and its gradients (ar_qk_norm_rope and its
// backward pass).
//
//   n = x / sqrt(mean(x^2) + eps), y = n w, out = R(a) y;  a(j) = pos freq[j]
//   backward: g = R(-a) dout, dn = g w, dx = (dn - n mean(dn n)) / sqrt(...),
//             dw = sum g n
//
// Both are bound by memory: every value is read once and written once
// (backward: two reads, one write).  head_dim / 8 lanes hold one head of one row,
// 8 values each in two pieces of 4 that lie rot / 2 apart, so that both values
// of a rotation's pair are in one lane (with neighbours in pairs, and in what is
// not rotated, the pieces are side by side); the sums over a head go through
// lane exchanges within rows of 16 lanes, which cost no LDS access.
//
// The angle of a far position needs more than fp32: pos * freq is formed in
// fp64 in turns, only its fraction goes on in fp32 (off by 2^-25 of half a turn at
// most, which adds a tenth to the error of an fp32 result).  That costs far more than
// the rest per value, so a workgroup computes the cosines and sines of its
// tokens once into LDS, for every head (forward: of every rank).
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

struct RopeArgs {
  const char* x[2][MAX_RANKS];   // queries, keys
  char* out[2][MAX_RANKS];       // backward: dx
  const char* dy[2][MAX_RANKS];  // backward
  const char* weight[2];
  const int64_t* pos;
  const float* freq;
  float* part;            // backward: [rank][2][blocks][dim] sums of g n
  uint64_t x_pitch[2];    // bytes from row to row
  uint64_t out_pitch[2];
  uint64_t dy_pitch[2];
  uint32_t rows, heads[2], rot;
  uint32_t tokens;  // of a workgroup (backward: of a pass)
  uint32_t blocks;  // backward: workgroups per rank
  int32_t nranks, pairs;
  float eps;
};

// The cosines and sines of `n` tokens from t0 on: [token][rot / 2].
__device__ void angles(const RopeArgs& a, uint32_t t0, uint32_t n, float2* table) {
  const uint32_t half = a.rot / 2;
  for (uint32_t i = threadIdx.x; i < n * half; i += THREADS) {
    const uint32_t t = t0 + i / half, j = i % half;
    // turns = pos freq / (2 pi); sincospi takes half turns
    const double turns = (double)a.pos[t] * (double)a.freq[j] * 0.15915494309189533577;
    const float f = (float)(2.0 * (turns - rint(turns)));
    float s, c;
    sincospif(f, &s, &c);
    table[i] = make_float2(c, s);
  }
}

constexpr int E = 8;  // values of a lane

// Four values of a row, and back.
template <int DT>
struct Piece {
  uint32_t w[DT == DT_BF16 ? 2 : 4];
};

template <int DT>
__device__ __forceinline__ Piece<DT> load4(const char* p) {
  Piece<DT> r;
  if constexpr (DT == DT_BF16) {
    const uint2 v = *(const uint2*)p;
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
    const uint4 v = *(const uint4*)p;
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void widen(const Piece<DT>& v, float* f) {
  if constexpr (DT == DT_BF16) {
#pragma unroll
    for (int i = 0; i < 2; ++i) f[2 * i] = __uint_as_float(v.w[i] << 16), f[2 * i + 1] = __uint_as_float(v.w[i] & 0xffff0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v.w[i]);
  }
}

// Results are not read again by this call: stored past the caches' turn
// (prompt of 4096 tokens, 8 x 6 heads of 128: 21.8 us stored plainly, 20.7 so; training
// step of 8192: 106 and 89).
template <int DT>
__device__ __forceinline__ void store4(char* p, const float* f) {
  typedef uint32_t v2u __attribute__((ext_vector_type(2)));
  if constexpr (DT == DT_BF16) {
    const v2u v = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
    __builtin_nontemporal_store(v, (v2u*)p);
  } else {
    st16_hint<true>(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
  }
}

template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, false));
}

// The sum over L neighbouring lanes, in each of them.
template <int L>
__device__ __forceinline__ float sum_lanes(float v) {
  v = add_dpp<0xb1>(v);   // quad_perm 1 0 3 2
  v = add_dpp<0x4e>(v);   // quad_perm 2 3 0 1
  v = add_dpp<0x141>(v);  // the other four of eight (row_half_mirror)
  if (L > 8) v = add_dpp<0x140>(v);  // the other eight of sixteen (row_mirror)
  if (L > 16) v += __shfl_xor(v, 16);
  return v;
}

// What a lane holds of a head.
struct Share {
  uint32_t at[2];  // first values of its pieces
  uint32_t turn;   // first entry of its token's table
  bool rotated;
};

__device__ __forceinline__ Share share_of(uint32_t lane, uint32_t rot, int pairs) {
  Share s;
  s.rotated = lane * E < rot;
  s.at[0] = lane * E, s.at[1] = lane * E + 4, s.turn = lane * 4;
  if (s.rotated && !pairs) s.at[0] = lane * 4, s.at[1] = rot / 2 + lane * 4;
  return s;
}

// y turned by the angles in cs (dir +1) or back (dir -1).
__device__ __forceinline__ void rotate(bool rotated, int pairs, const float2* cs, float dir, float* y) {
  if (!rotated) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = cs[i];
    const int j = pairs ? 2 * i : i, k = pairs ? 2 * i + 1 : i + 4;
    const float p = y[j], q = y[k], s = dir * v.y;
    y[j] = p * v.x - q * s;
    y[k] = q * v.x + p * s;
  }
}

// Forward.  A workgroup takes `tokens` rows of every rank: thread (row, head,
// lane) keeps its cosines, sines and weights over the ranks, whose loads go
// out together, the first ones before the cosines are made.
template <int DT, int DIM, bool PAIRS>
__global__ __launch_bounds__(THREADS) void rope_kernel(RopeArgs a) {
  constexpr int L = DIM / E, ES = DT == DT_BF16 ? 2 : 4;
  extern __shared__ float2 table[];
  uint32_t group = blockIdx.x;
  if (blockIdx.z) group += blockIdx.z * gridDim.x;
  const uint32_t t0 = group * a.tokens, half = a.rot / 2;
  if (t0 >= a.rows) return;
  const uint32_t n = min(a.tokens, a.rows - t0);
  const uint32_t heads = a.heads[0] + a.heads[1];
  const Share sh = share_of(threadIdx.x % L, a.rot, PAIRS);
  constexpr int R = MAX_RANKS;  // ranks whose loads are in flight together: all
  // every lane of a head takes part in its sums: whole heads per pass
  const uint32_t step = gridDim.y * (THREADS / L);
  uint32_t i = threadIdx.x / L + blockIdx.y * (THREADS / L);
  uint32_t t, hh;
  int kind;
  Piece<DT> v[R][2];
  auto load = [&] {
    t = i / heads, hh = i - t * heads;
    kind = hh >= a.heads[0];
    if (kind) hh -= a.heads[0];
    const uint64_t from = (uint64_t)(t0 + t) * a.x_pitch[kind] + (uint64_t)hh * (DIM * ES);
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (j < a.nranks) {
#pragma unroll
        for (int p = 0; p < 2; ++p) v[j][p] = load4<DT>(a.x[kind][j] + from + sh.at[p] * ES);
      }
  };
  if (i < n * heads) load();
  angles(a, t0, n, table);
  __syncthreads();
  while (i < n * heads) {
    float w[E];
    float2 cs[4];
#pragma unroll
    for (int p = 0; p < 2; ++p) widen<DT>(load4<DT>(a.weight[kind] + sh.at[p] * ES), w + 4 * p);
    if (sh.rotated)
#pragma unroll
      for (int p = 0; p < 4; ++p) cs[p] = table[t * half + sh.turn + p];
    const uint64_t to = (((uint64_t)(t0 + t) * a.heads[kind] + hh) * DIM) * ES;
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (j < a.nranks) {
        float x[E], q = 0.f;
#pragma unroll
        for (int p = 0; p < 2; ++p) widen<DT>(v[j][p], x + 4 * p);
#pragma unroll
        for (int e = 0; e < E; ++e) q += x[e] * x[e];
        const float inv = rsqrtf(sum_lanes<L>(q) * (1.0f / DIM) + a.eps);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = x[e] * inv * w[e];
        rotate(sh.rotated, PAIRS, cs, 1.f, x);
#pragma unroll
        for (int p = 0; p < 2; ++p) store4<DT>(a.out[kind][j] + to + sh.at[p] * ES, x + 4 * p);
      }
    i += step;
    if (i < n * heads) load();
  }
}

// Backward.  A workgroup takes every `blocks`-th group of `tokens` rows of one
// rank; a thread's values of a head are the same for all of them, so its share
// of dw stays in registers until the end, one sum for queries and one for keys.
template <int DT, int DIM, bool PAIRS>
__global__ __launch_bounds__(THREADS) void rope_backward_kernel(RopeArgs a) {
  constexpr int L = DIM / E, PER = THREADS / L, ES = DT == DT_BF16 ? 2 : 4;
  extern __shared__ float2 table[];
  const uint32_t half = a.rot / 2;
  const int r = blockIdx.y;
  const Share sh = share_of(threadIdx.x % L, a.rot, PAIRS);
  float dw[2][E] = {};
  for (uint64_t t0 = (uint64_t)blockIdx.x * a.tokens; t0 < a.rows; t0 += (uint64_t)a.blocks * a.tokens) {
    const uint32_t n = (uint32_t)min((uint64_t)a.tokens, a.rows - t0);
    angles(a, (uint32_t)t0, n, table);
    __syncthreads();
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const uint32_t heads = a.heads[kind];
      if (!heads) continue;
      float w[E];
#pragma unroll
      for (int p = 0; p < 2; ++p) widen<DT>(load4<DT>(a.weight[kind] + sh.at[p] * ES), w + 4 * p);
      for (uint32_t i = threadIdx.x / L; i < n * heads; i += PER) {
        const uint32_t t = i / heads, h = i - t * heads;
        const uint64_t row = t0 + t, at = (uint64_t)h * (DIM * ES);
        float x[E], g[E];
        float2 cs[4];
        Piece<DT> xv[2], gv[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          xv[p] = load4<DT>(a.x[kind][r] + row * a.x_pitch[kind] + at + sh.at[p] * ES);
          gv[p] = load4<DT>(a.dy[kind][r] + row * a.dy_pitch[kind] + at + sh.at[p] * ES);
        }
        if (sh.rotated)
#pragma unroll
          for (int p = 0; p < 4; ++p) cs[p] = table[t * half + sh.turn + p];
        float q = 0.f, dot = 0.f;
#pragma unroll
        for (int p = 0; p < 2; ++p) widen<DT>(xv[p], x + 4 * p), widen<DT>(gv[p], g + 4 * p);
#pragma unroll
        for (int e = 0; e < E; ++e) q += x[e] * x[e];
        const float inv = rsqrtf(sum_lanes<L>(q) * (1.0f / DIM) + a.eps);
        rotate(sh.rotated, PAIRS, cs, -1.f, g);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          x[e] *= inv;
          dw[kind][e] += g[e] * x[e];
          g[e] *= w[e];
          dot += g[e] * x[e];
        }
        dot = sum_lanes<L>(dot) * (1.0f / DIM);
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] = inv * (g[e] - x[e] * dot);
#pragma unroll
        for (int p = 0; p < 2; ++p)
          store4<DT>(a.out[kind][r] + row * a.out_pitch[kind] + at + sh.at[p] * ES, g + 4 * p);
      }
    }
    __syncthreads();  // the table is written again
  }
  // The lanes with the same values, then the waves, join their shares.
  __shared__ float s[2][THREADS / 64][DIM];
#pragma unroll
  for (int kind = 0; kind < 2; ++kind)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float v = dw[kind][e];
#pragma unroll
      for (int o = 32; o >= L; o >>= 1) v += __shfl_xor(v, o);
      if ((threadIdx.x & 63) < L) s[kind][threadIdx.x >> 6][sh.at[e / 4] + e % 4] = v;
    }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < 2 * DIM; i += THREADS) {
    const int kind = i / DIM, d = i % DIM;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) v += s[kind][w][d];
    a.part[(((uint64_t)r * 2 + kind) * a.blocks + blockIdx.x) * DIM + d] = v;
  }
}

struct SumArgs {
  const float* part;
  char* out[2][MAX_RANKS];
  uint32_t blocks, dim;
};

// 32 values of one rank's and kind's dw: the workgroups' shares, up to a thousand,
// added in fp64 and in a fixed order, 32 slices of them side by side, eight loads of
// a slice in flight.
constexpr uint32_t SUM_DIMS = 32, SUM_SLICES = 32;

template <int DT>
__global__ __launch_bounds__(SUM_DIMS * SUM_SLICES) void rope_weight_kernel(SumArgs a) {
  __shared__ double s[SUM_SLICES][SUM_DIMS];
  const uint32_t kind = blockIdx.x, r = blockIdx.y, lane = threadIdx.x % SUM_DIMS, slice = threadIdx.x / SUM_DIMS;
  const uint32_t d = blockIdx.z * SUM_DIMS + lane;
  const float* p = a.part + ((uint64_t)r * 2 + kind) * a.blocks * a.dim + d;
  double v = 0.;
#pragma unroll 8
  for (uint32_t b = slice; b < a.blocks; b += SUM_SLICES) v += p[(uint64_t)b * a.dim];
  s[slice][lane] = v;
  __syncthreads();
  if (slice == 0) {
    for (uint32_t i = 1; i < SUM_SLICES; ++i) v += s[i][lane];
    Elem<DT>::stf(a.out[kind][r] + (uint64_t)d * Elem<DT>::size, (float)v);
  }
}

// Workgroups per rank of the backward pass.  Enough to fill the 256 CUs
// several times over, few enough that their shares of dw stay small.
uint32_t backward_blocks(int nranks, uint64_t rows, uint64_t heads) {
  const uint64_t want = 1024 / nranks;
  const uint64_t useful = (rows * heads + 31) / 32;  // two passes of a workgroup's 16 heads of 128
  return (uint32_t)(useful < 1 ? 1 : useful < want ? useful : want);
}

uint64_t rope_workspace(int nranks, uint64_t rows, uint64_t heads, uint64_t dim) {
  return rows ? (uint64_t)nranks * 2 * backward_blocks(nranks, rows, heads) * dim * 4 : 0;
}

ar_status check_shape(int n, size_t rows, size_t heads, size_t kv_heads, size_t dim, size_t rot, int pairs, int dtype) {
  if (n < 1 || n > MAX_RANKS || dtype < 0 || dtype > 2 || pairs < 0 || pairs > 1) return AR_ERR_INVALID;
  if (heads < 1) return AR_ERR_INVALID;
  if (dtype == DT_I32 || !head_dim_ok(dim)) return AR_ERR_UNSUPPORTED;
  if (rot > dim || rot % 16) return AR_ERR_INVALID;
  if (heads > MAX_HEADS || kv_heads > MAX_HEADS || rows > LAYER_MAX_ROWS || rows * (heads + kv_heads) > LAYER_MAX_ROWS)
    return AR_ERR_TOO_LARGE;
  return AR_OK;
}

template <int DT, int DIM>
void launch_forward(const RopeArgs& a, dim3 grid, uint32_t lds, hipStream_t stream) {
  if (a.pairs) rope_kernel<DT, DIM, true><<<grid, THREADS, lds, stream>>>(a);
  else rope_kernel<DT, DIM, false><<<grid, THREADS, lds, stream>>>(a);
}

template <int DT, int DIM>
void launch_backward(const RopeArgs& a, dim3 grid, uint32_t lds, hipStream_t stream) {
  if (a.pairs) rope_backward_kernel<DT, DIM, true><<<grid, THREADS, lds, stream>>>(a);
  else rope_backward_kernel<DT, DIM, false><<<grid, THREADS, lds, stream>>>(a);
}

}  // namespace

extern "C" {

ar_status ar_qk_norm_rope(int nranks, const void* const* q, size_t q_stride, const void* const* k, size_t k_stride,
                          const void* q_weight, const void* k_weight, const int64_t* pos, const float* freq,
                          void* const* q_out, void* const* k_out, size_t rows, size_t heads, size_t kv_heads,
                          size_t head_dim, size_t rot, int pairs, float eps, ar_dtype dtype, ar_stream_t stream) {
  const ar_status st = check_shape(nranks, rows, heads, kv_heads, head_dim, rot, pairs, (int)dtype);
  if (st != AR_OK) return st;
  if (!q || !q_out || (kv_heads && (!k || !k_out))) return AR_ERR_INVALID;
  if (rows == 0) return AR_OK;
  const uint64_t es = dtype == AR_BF16 ? 2 : 4;
  if (!stride_ok(q_stride, heads * head_dim, es) || (kv_heads && !stride_ok(k_stride, kv_heads * head_dim, es)))
    return AR_ERR_INVALID;
  RopeArgs a = {};
  LayerBuffers b;
  for (int r = 0; r < nranks; ++r) {
    a.x[0][r] = (const char*)q[r];
    a.out[0][r] = (char*)q_out[r];
    b.in(q[r], span_bytes(rows, q_stride, heads * head_dim, es));
    b.out(q_out[r], rows * heads * head_dim * es);
    if (!kv_heads) continue;
    a.x[1][r] = (const char*)k[r];
    a.out[1][r] = (char*)k_out[r];
    b.in(k[r], span_bytes(rows, k_stride, kv_heads * head_dim, es));
    b.out(k_out[r], rows * kv_heads * head_dim * es);
  }
  b.in(q_weight, head_dim * es);
  if (kv_heads) b.in(k_weight, head_dim * es);
  if (rot) {
    b.in(pos, rows * 8, 8);
    b.in(freq, rot / 2 * 4, 4);
  }
  if (!b.ok()) return AR_ERR_INVALID;
  a.weight[0] = (const char*)q_weight;
  a.weight[1] = (const char*)k_weight;
  a.pos = pos;
  a.freq = freq;
  a.x_pitch[0] = q_stride * es;
  a.x_pitch[1] = k_stride * es;
  a.rows = (uint32_t)rows;
  a.heads[0] = (uint32_t)heads;
  a.heads[1] = (uint32_t)kv_heads;
  a.rot = (uint32_t)rot;
  a.nranks = nranks;
  a.pairs = pairs;
  a.eps = eps;
  // One pass a thread, or one token's heads shared by
  // several workgroups where there are few tokens.
  const uint64_t per_token = (heads + kv_heads) * head_dim / E;  // threads
  a.tokens = (uint32_t)umin(umax(THREADS / per_token, 1), 16);
  const uint32_t groups = (uint32_t)((rows + a.tokens - 1) / a.tokens);
  const uint64_t passes = (a.tokens * per_token + THREADS - 1) / THREADS;
  const uint32_t split = (uint32_t)umax(1, umin(passes, 512 / groups));
  const Fold fold = fold_items(groups, THREADS);
  const dim3 grid(fold.x, split, fold.folds);
  const uint32_t lds = a.tokens * (uint32_t)rot / 2 * 8;
  by_head_dim((int)dtype, head_dim, [&](auto dt, auto dim) {
    launch_forward<decltype(dt)::value, decltype(dim)::value>(a, grid, lds, (hipStream_t)stream);
  });
  return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP;
}

size_t ar_qk_norm_rope_workspace(int nranks, size_t rows, size_t heads, size_t kv_heads, size_t head_dim) {
  if (check_shape(nranks, rows, heads, kv_heads, head_dim, 0, 0, DT_F32) != AR_OK) return 0;
  return rope_workspace(nranks, rows, heads + kv_heads, head_dim);
}

ar_status ar_qk_norm_rope_backward(int nranks, const void* const* dq_out, const void* const* dk_out,
                                   const void* const* q, size_t q_stride, const void* const* k, size_t k_stride,
                                   const void* q_weight, const void* k_weight, const int64_t* pos, const float* freq,
                                   void* const* dq, size_t dq_stride, void* const* dk, size_t dk_stride,
                                   void* const* dq_weight, void* const* dk_weight, size_t rows, size_t heads,
                                   size_t kv_heads, size_t head_dim, size_t rot, int pairs, float eps, ar_dtype dtype,
                                   void* workspace, size_t workspace_bytes, ar_stream_t stream) {
  const ar_status st = check_shape(nranks, rows, heads, kv_heads, head_dim, rot, pairs, (int)dtype);
  if (st != AR_OK) return st;
  if (!dq_out || !q || !dq || !dq_weight) return AR_ERR_INVALID;
  if (kv_heads && (!dk_out || !k || !dk || !dk_weight)) return AR_ERR_INVALID;
  const uint64_t es = dtype == AR_BF16 ? 2 : 4;
  const uint64_t qw = heads * head_dim, kw = kv_heads * head_dim;
  if (rows && (!stride_ok(q_stride, qw, es) || !stride_ok(dq_stride, qw, es))) return AR_ERR_INVALID;
  if (rows && kv_heads && (!stride_ok(k_stride, kw, es) || !stride_ok(dk_stride, kw, es))) return AR_ERR_INVALID;
  const uint64_t need = rope_workspace(nranks, rows, heads + kv_heads, head_dim);
  RopeArgs a = {};
  SumArgs s = {};
  LayerBuffers b;
  for (int r = 0; r < nranks; ++r) {
    a.x[0][r] = (const char*)q[r];
    a.dy[0][r] = (const char*)dq_out[r];
    a.out[0][r] = (char*)dq[r];
    s.out[0][r] = (char*)dq_weight[r];
    b.in(q[r], span_bytes(rows, q_stride, qw, es));
    b.in(dq_out[r], rows * qw * es);
    b.out_rows(dq[r], rows, dq_stride * es, qw * es);
    b.out(dq_weight[r], head_dim * es);
    if (!kv_heads) continue;
    a.x[1][r] = (const char*)k[r];
    a.dy[1][r] = (const char*)dk_out[r];
    a.out[1][r] = (char*)dk[r];
    s.out[1][r] = (char*)dk_weight[r];
    b.in(k[r], span_bytes(rows, k_stride, kw, es));
    b.in(dk_out[r], rows * kw * es);
    b.out_rows(dk[r], rows, dk_stride * es, kw * es);
    b.out(dk_weight[r], head_dim * es);
  }
  b.in(q_weight, head_dim * es);
  if (kv_heads) b.in(k_weight, head_dim * es);
  if (rot) {
    b.in(pos, rows * 8, 8);
    b.in(freq, rot / 2 * 4, 4);
  }
  b.out(workspace, need);
  if (!b.ok()) return AR_ERR_INVALID;
  if (workspace_bytes < need) return AR_ERR_TOO_LARGE;
  a.weight[0] = (const char*)q_weight;
  a.weight[1] = (const char*)k_weight;
  a.pos = pos;
  a.freq = freq;
  a.part = (float*)workspace;
  a.x_pitch[0] = q_stride * es;
  a.x_pitch[1] = k_stride * es;
  a.dy_pitch[0] = qw * es;
  a.dy_pitch[1] = kw * es;
  a.out_pitch[0] = dq_stride * es;
  a.out_pitch[1] = dk_stride * es;
  a.rows = (uint32_t)rows;
  a.heads[0] = (uint32_t)heads;
  a.heads[1] = (uint32_t)kv_heads;
  a.rot = (uint32_t)rot;
  a.nranks = nranks;
  a.pairs = pairs;
  a.eps = eps;
  a.blocks = rows ? backward_blocks(nranks, rows, heads + kv_heads) : 0;
  a.tokens = rows ? (uint32_t)umin((rows + a.blocks - 1) / a.blocks, 16) : 0;
  if (rows) {
    const dim3 grid(a.blocks, nranks);
    const uint32_t lds = a.tokens * (uint32_t)rot / 2 * 8;
    by_head_dim((int)dtype, head_dim, [&](auto dt, auto dim) {
      launch_backward<decltype(dt)::value, decltype(dim)::value>(a, grid, lds, (hipStream_t)stream);
    });
    if (hipGetLastError() != hipSuccess) return AR_ERR_HIP;
  }
  s.part = a.part;
  s.blocks = a.blocks;
  s.dim = (uint32_t)head_dim;
  const dim3 grid(kv_heads ? 2 : 1, nranks, (uint32_t)head_dim / SUM_DIMS);
  if (dtype == AR_BF16) rope_weight_kernel<DT_BF16><<<grid, SUM_DIMS * SUM_SLICES, 0, (hipStream_t)stream>>>(s);
  else rope_weight_kernel<DT_F32><<<grid, SUM_DIMS * SUM_SLICES, 0, (hipStream_t)stream>>>(s);
  return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP;
}

}  // extern "C"
