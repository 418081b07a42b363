// rope.hip -- norms of queries and keys for each head with the rotation to
// their positions in one pass, and its gradients (ar_qk_norm_rope and its
// backward pass).
//
//   n = x / sqrt(mean(x^2) + eps), y = n w, out = R(a) y;  a(j) = pos freq[j]
//   backward: g = R(-a) dout, dn = g w, dx = (dn - n mean(dn n)) / sqrt(...),
//             dw = sum g n
//
// Both are bound by memory: every value is read once and written once
// (backward: two reads, one write), 16 bytes per lane.  head_dim / E lanes (E
// elements of 16 bytes) hold one head of one row; its sums go through lane
// exchanges, and so does a rotation's other half, which lies rot / 2 elements
// away in the same head.
//
// The angle of a far position needs more than fp32: pos * freq is formed in
// fp64 in turns, only its fraction goes on in fp32.  That costs far more than
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

template <int DT> constexpr int elems() { return DT == DT_BF16 ? 8 : 4; }

template <int DT>
__device__ __forceinline__ void widen(const uint4& v, float* f) {
  if (DT == DT_BF16) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
}

template <int DT>
__device__ __forceinline__ uint4 narrow(const float* f) {
  if (DT == DT_BF16)
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

template <int L>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

__device__ __forceinline__ uint4 from_lane(const uint4& v, int lane) {
  return make_uint4(__shfl((int)v.x, lane), __shfl((int)v.y, lane), __shfl((int)v.z, lane), __shfl((int)v.w, lane));
}

// Where chunk c of a head finds the other half of its rotation.
struct Turn {
  int partner;      // lane that holds the other half (the lane itself: none, or in pairs)
  float sign;       // of the sine term of a rotation: -1 in the first half, +1 in the second, 0 not rotated
  uint32_t at;      // first entry of the chunk in its token's table
  bool rotated;
};

template <int DT, int DIM>
__device__ __forceinline__ Turn turn_of(uint32_t chunk, uint32_t rot, int pairs) {
  constexpr int E = elems<DT>();
  const uint32_t rc = rot / E, hc = rc / 2, lane = threadIdx.x & 63;
  Turn t;
  t.rotated = chunk < rc;
  t.partner = (int)lane;
  t.sign = 0.f;
  t.at = 0;
  if (!t.rotated) return t;
  if (pairs) {
    t.at = chunk * (E / 2);
    return t;
  }
  t.partner = (int)(chunk < hc ? lane + hc : lane - hc);
  t.sign = chunk < hc ? -1.f : 1.f;
  t.at = (chunk < hc ? chunk : chunk - hc) * E;
  return t;
}

// y turned by the angles in cs (dir +1) or back (dir -1); other: the partner's y.
template <int DT>
__device__ __forceinline__ void rotate(const Turn& t, int pairs, const float2* cs, float dir, const float* other, float* y) {
  constexpr int E = elems<DT>();
  if (!t.rotated) return;
  if (pairs) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 v = cs[i];
      const float p = y[2 * i], q = y[2 * i + 1], s = dir * v.y;
      y[2 * i] = p * v.x - q * s;
      y[2 * i + 1] = q * v.x + p * s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float2 v = cs[i];
      y[i] = y[i] * v.x + other[i] * (dir * t.sign * v.y);
    }
  }
}

// Forward.  A workgroup takes `tokens` rows of every rank: thread (row, head,
// chunk) keeps its cosines, sines and weights over the ranks, whose loads go
// out together.
template <int DT, int DIM>
__global__ __launch_bounds__(THREADS) void rope_kernel(RopeArgs a) {
  constexpr int E = elems<DT>(), L = DIM / E;
  extern __shared__ float2 table[];
  const uint32_t t0 = blockIdx.x * a.tokens, half = a.rot / 2;
  const uint32_t n = min(a.tokens, a.rows - t0);
  angles(a, t0, n, table);
  __syncthreads();
  const uint32_t heads = a.heads[0] + a.heads[1], chunk = threadIdx.x % L;
  const Turn turn = turn_of<DT, DIM>(chunk, a.rot, a.pairs);
  const uint32_t other_chunk = chunk + turn.partner - (threadIdx.x & 63);
  // every lane of a head takes part in its exchanges: whole heads per pass
  for (uint32_t i = threadIdx.x / L + blockIdx.y * (THREADS / L); i < n * heads; i += gridDim.y * (THREADS / L)) {
    const uint32_t t = i / heads, h = i - t * heads;
    const int kind = h >= a.heads[0];
    const uint32_t hh = kind ? h - a.heads[0] : h;
    float w[E], wo[E];
    widen<DT>(ld16(a.weight[kind] + chunk * 16), w);
    widen<DT>(ld16(a.weight[kind] + other_chunk * 16), wo);
    const float2* cs = table + t * half + turn.at;
    const uint64_t from = (uint64_t)(t0 + t) * a.x_pitch[kind] + (uint64_t)hh * (L * 16) + chunk * 16;
    const uint64_t to = ((uint64_t)(t0 + t) * a.heads[kind] + hh) * (L * 16) + chunk * 16;
    constexpr int R = 4;  // ranks whose loads are in flight together
    for (int r0 = 0; r0 < a.nranks; r0 += R) {
      uint4 v[R];
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (r0 + j < a.nranks) v[j] = ld16(a.x[kind][r0 + j] + from);
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (r0 + j < a.nranks) {
          float x[E], o[E];
          widen<DT>(v[j], x);
          widen<DT>(from_lane(v[j], turn.partner), o);
          float q = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) q += x[e] * x[e];
          const float inv = 1.0f / sqrtf(sum_lanes<L>(q) * (1.0f / DIM) + a.eps);
#pragma unroll
          for (int e = 0; e < E; ++e) x[e] = x[e] * inv * w[e], o[e] = o[e] * inv * wo[e];
          rotate<DT>(turn, a.pairs, cs, 1.f, o, x);
          st16(a.out[kind][r0 + j] + to, narrow<DT>(x));
        }
    }
  }
}

// Backward.  A workgroup takes every `blocks`-th group of `tokens` rows of one
// rank; a thread's chunk is the same for all of them, so its share of dw stays
// in registers until the end, one sum for queries and one for keys.
template <int DT, int DIM>
__global__ __launch_bounds__(THREADS) void rope_backward_kernel(RopeArgs a) {
  constexpr int E = elems<DT>(), L = DIM / E, PER = THREADS / L;
  extern __shared__ float2 table[];
  const uint32_t half = a.rot / 2, chunk = threadIdx.x % L;
  const int r = blockIdx.y;
  const Turn turn = turn_of<DT, DIM>(chunk, a.rot, a.pairs);
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
      widen<DT>(ld16(a.weight[kind] + chunk * 16), w);
      for (uint32_t i = threadIdx.x / L; i < n * heads; i += PER) {
        const uint32_t t = i / heads, h = i - t * heads;
        const uint64_t row = t0 + t, at = (uint64_t)h * (L * 16) + chunk * 16;
        const uint4 xv = ld16(a.x[kind][r] + row * a.x_pitch[kind] + at);
        const uint4 gv = ld16(a.dy[kind][r] + row * a.dy_pitch[kind] + at);
        float x[E], g[E], o[E];
        widen<DT>(xv, x);
        widen<DT>(gv, g);
        widen<DT>(from_lane(gv, turn.partner), o);
        rotate<DT>(turn, a.pairs, table + t * half + turn.at, -1.f, o, g);
        float q = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) q += x[e] * x[e];
        const float inv = 1.0f / sqrtf(sum_lanes<L>(q) * (1.0f / DIM) + a.eps);
        float dot = 0.f;
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
        st16(a.out[kind][r] + row * a.out_pitch[kind] + at, narrow<DT>(g));
      }
    }
    __syncthreads();  // the table is written again
  }
  // The lanes of a chunk, then the waves, join their shares.
  __shared__ float s[2][THREADS / 64][DIM];
#pragma unroll
  for (int kind = 0; kind < 2; ++kind)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float v = dw[kind][e];
#pragma unroll
      for (int o = 32; o >= L; o >>= 1) v += __shfl_xor(v, o);
      if ((threadIdx.x & 63) < L) s[kind][threadIdx.x >> 6][chunk * E + e] = v;
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

// dw of one rank and kind: the workgroups' shares added in order, by
// 1024 / dim slices of them.
template <int DT>
__global__ __launch_bounds__(1024) void rope_weight_kernel(SumArgs a) {
  __shared__ float s[1024];
  const uint32_t kind = blockIdx.x, r = blockIdx.y, d = threadIdx.x % a.dim, slice = threadIdx.x / a.dim;
  const uint32_t slices = 1024 / a.dim;
  const float* p = a.part + ((uint64_t)r * 2 + kind) * a.blocks * a.dim;
  float v = 0.f;
  for (uint32_t b = slice; b < a.blocks; b += slices) v += p[(uint64_t)b * a.dim + d];
  s[threadIdx.x] = v;
  __syncthreads();
  if (slice == 0 && a.out[kind][r]) {
    for (uint32_t i = 1; i < slices; ++i) v += s[i * a.dim + d];
    Elem<DT>::stf(a.out[kind][r] + (uint64_t)d * Elem<DT>::size, v);
  }
}

// Workgroups per rank of the backward pass.  Enough to fill the 256 CUs
// several times over, few enough that their shares of dw stay small.
uint32_t backward_blocks(int nranks, uint64_t rows, uint64_t heads) {
  const uint64_t want = 1024 / nranks;
  const uint64_t useful = (rows * heads + 31) / 32;  // two passes of a workgroup's 16 heads
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
  rope_kernel<DT, DIM><<<grid, THREADS, lds, stream>>>(a);
}

template <int DT, int DIM>
void launch_backward(const RopeArgs& a, dim3 grid, uint32_t lds, hipStream_t stream) {
  rope_backward_kernel<DT, DIM><<<grid, THREADS, lds, stream>>>(a);
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
  // Two passes of 16-byte chunks a thread, or one token's heads shared by
  // several workgroups where there are few tokens.
  const uint64_t per_token = (heads + kv_heads) * head_dim * es / 16;  // threads
  a.tokens = (uint32_t)umin(umax(2 * THREADS / per_token, 1), 16);
  const uint32_t groups = (uint32_t)((rows + a.tokens - 1) / a.tokens);
  const uint64_t passes = (a.tokens * per_token + THREADS - 1) / THREADS;
  const uint32_t split = (uint32_t)umax(1, umin(passes, 512 / groups));
  const dim3 grid(groups, split);
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
  const dim3 grid(kv_heads ? 2 : 1, nranks);
  if (dtype == AR_BF16) rope_weight_kernel<DT_BF16><<<grid, 1024, 0, (hipStream_t)stream>>>(s);
  else rope_weight_kernel<DT_F32><<<grid, 1024, 0, (hipStream_t)stream>>>(s);
  return hipGetLastError() == hipSuccess ? AR_OK : AR_ERR_HIP;
}

}  // extern "C"
