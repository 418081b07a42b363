// product_kernels.hpp -- the product kernels of the layer operators: one kernel
// template over (type, layouts, epilogue, tile class), instantiated
// per payload type by products_bf16.hip and products_f32.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "products.hpp"

namespace ar {

namespace {

// Value and derivative of the gate's activation, fp32.
struct Act {
  float v, d;
};
template <uint32_t ACT, bool DERIV>
__device__ __forceinline__ Act activate(float z) {
  Act r;
  r.d = 0.f;
  if constexpr (ACT == ACT_SILU) {
    const float s = 1.0f / (1.0f + expf(-z));
    r.v = z * s;
    if (DERIV) r.d = s * (1.0f + z * (1.0f - s));
  } else if constexpr (ACT == ACT_GELU) {
    const float phi = 0.5f * erfcf(-0.70710678118654752f * z);  // erfc keeps the small tail's digits
    r.v = z * phi;
    if (DERIV) r.d = phi + z * 0.39894228040143268f * expf(-0.5f * z * z);
  } else {
    // tanh(y) = 2 s(2 y) - 1: (1 + tanh(y)) / 2 = s(2 y) = 1 / (1 + exp(-2 y))
    // beyond +-64 s is 0 or 1 exactly; the clamp keeps z^3 and z^2 finite
    const float k = 0.79788456080286536f, c = 0.044715f;
    const float y = z > 64.f ? 64.f : z < -64.f ? -64.f : z;
    const float s = 1.0f / (1.0f + expf(-2.0f * k * (y + c * y * y * y)));
    r.v = z * s;
    if (DERIV) r.d = s + 2.0f * y * s * (1.0f - s) * k * (1.0f + 3.0f * c * y * y);
  }
  return r;
}

// A target's column of a problem (columns col0 .. col0 + n of the vocabulary),
// or a value no column has.
__device__ __forceinline__ uint32_t target_column(int64_t target, uint64_t vocab, uint64_t col0, uint32_t n) {
  const uint64_t at = (uint64_t)target - col0;
  return target >= 0 && (uint64_t)target < vocab && at < n ? (uint32_t)at : 0xffffffffu;
}

// exp for probabilities.  bf16 gradients round far above the hardware
// exponential's error (about |z| 2^-24 relative); fp32 takes the exact one.
template <int DT>
__device__ __forceinline__ float exp_of(float z) {
  return DT == DT_BF16 ? __expf(z) : expf(z);
}

struct Nothing {};

// c[0] = the finished tile times `scale`, rounded once.
template <class P>
__device__ __forceinline__ void store_result(P& x, const Problem& p, float scale, uint32_t row0, uint32_t col0,
                                             char* smem) {
  constexpr int ES = KElem<P::DT>::ES, V = KElem<P::DT>::E;
  const bool vec = p.ldc % V == 0;
  const uint32_t m = p.m - p.fold;
  x.template hand_out<V, 2>(
      smem, p.fold, [](uint32_t, uint32_t) { return Nothing(); },
      [&](uint32_t r, uint32_t col, float* v, float*, Nothing) {
        const uint64_t row = (uint64_t)row0 + r;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] *= scale;
        if (row < m) store_row<P::DT, V, true>(p.c[0] + row * p.ldc * ES, (uint64_t)col0 + col, p.n, vec, v);
      });
}

template <class P>
__device__ __forceinline__ void store_tile(const Problem& p, float scale, uint32_t row0, uint32_t col0, char* smem) {
  P x;
  x.run(p, 0, row0, col0, smem);
  store_result(x, p, scale, row0, col0, smem);
}

// The fp32 sum of one share of K, for finish_kernel.  (In order: sums by atomics
// would change with the workgroups' timing.)
template <class P>
__device__ __forceinline__ void store_share(P& x, const Problem& p, uint32_t share, uint32_t row0, uint32_t col0,
                                            char* smem) {
  constexpr int V = KElem<P::DT>::E;
  const uint32_t m = p.m - p.fold;
  char* to = p.c[2] + (uint64_t)share * m * p.ldc * 4;
  x.template hand_out<V, 2>(
      smem, p.fold, [](uint32_t, uint32_t) { return Nothing(); },
      [&](uint32_t r, uint32_t col, float* v, float*, Nothing) {
        const uint64_t row = (uint64_t)row0 + r;
        if (row < m) store_row<DT_F32, V>(to + row * p.ldc * 4, (uint64_t)col0 + col, p.n, p.ldc % 4 == 0, v);
      });
}

// ACT: the gate's activation (gated kinds).
template <class P, int KIND, uint32_t ACT>
__global__ __launch_bounds__(P::NT) void product_kernel(const ProductArgs a) {
  __shared__ __align__(1024) char smem[P::LDS_BYTES];
  constexpr int DT = P::DT;
  constexpr int ES = KElem<DT>::ES;
  constexpr int V = KElem<DT>::E;  // values per 16-byte vector of the payload
  constexpr bool FOLDS = P::BM < Large::BM;  // may write second terms (product_tile keeps them from the large tile)
  uint32_t row0, col0, share;
  const Problem& p = a.p[locate<P>(a, &row0, &col0, &share)];
  if constexpr (KIND == PK_GRADS) {
    if (p.mode & GRAD_TN) {
      store_tile<typename P::TN_>(p, a.scale ? *a.scale : 1.0f, row0, col0, smem);
      return;
    }
  }
  P x;
  x.run(p, share, row0, col0, smem);
  if constexpr (KIND == PK_STORE_NT || KIND == PK_GRADS) {
    if (p.shares > 1) {
      store_share(x, p, share, row0, col0, smem);
      return;
    }
  }
  const uint32_t m = p.m, n = p.n;
  const uint64_t ldc = p.ldc;
  const bool vec = p.ldc % V == 0;
  auto nothing = [](uint32_t, uint32_t) { return Nothing(); };

  if constexpr (KIND == PK_STORE_NT) {
    store_result(x, p, 1.0f, row0, col0, smem);
  } else if constexpr (KIND == PK_GRADS) {
    const bool add = p.mode & GRAD_ADD, partial = p.mode & GRAD_PARTIAL;
    const float scale = a.scale ? *a.scale : 1.0f;
    if (!add && !partial) {
      store_result(x, p, scale, row0, col0, smem);
      return;
    }
    const uint32_t rows = m - p.fold;
    const bool fvec = p.ldc % 4 == 0;
    x.template hand_out<V, 4>(
        smem, p.fold,
        [&](uint32_t r, uint32_t col) {
          const uint64_t row = (uint64_t)row0 + r;
          Floats<V> o = {};
          if (add && row < rows) o = load_floats<V>(p.c[1] + row * ldc * 4, (uint64_t)col0 + col, n, fvec);
          return o;
        },
        [&](uint32_t r, uint32_t col, float* v, float*, const Floats<V>& o) {
          const uint64_t row = (uint64_t)row0 + r;
          if (row >= rows) return;
          // (the sum so far is scaled already)
#pragma unroll
          for (int e = 0; e < V; ++e) v[e] = add ? o.v[e] + v[e] * scale : v[e] * scale;
          if (partial) store_row<DT_F32, V>(p.c[1] + row * ldc * 4, (uint64_t)col0 + col, n, fvec, v);
          else store_row<DT, V>(p.c[0] + row * ldc * ES, (uint64_t)col0 + col, n, vec, v);
        });
  } else if constexpr (KIND == PK_GATED) {
    // h's storage has rows of whole chunks (ldc), of which the last columns
    // come out as zeros (their g and u are); g and u are n wide, fp32.
    x.template hand_out<V, 2>(smem, 0, nothing, [&](uint32_t r, uint32_t col, float* g, float* u, Nothing) {
      const uint64_t row = (uint64_t)row0 + r;
      if (row >= m) return;
      float h[V];
#pragma unroll
      for (int e = 0; e < V; ++e) h[e] = activate<ACT, false>(g[e]).v * u[e];
      char* to = p.c[0] + row * ldc * ES;
      store_terms<DT, V>(to, FOLDS && p.fold ? to + p.fold * ldc * ES : nullptr, (uint64_t)col0 + col, p.ldc, vec, h);
      if (p.c[1]) {
        store_row<DT_F32, V, true>(p.c[1] + row * (uint64_t)n * 4, (uint64_t)col0 + col, n, n % 4 == 0, g);
        store_row<DT_F32, V, true>(p.c[2] + row * (uint64_t)n * 4, (uint64_t)col0 + col, n, n % 4 == 0, u);
      }
    });
  } else if constexpr (KIND == PK_GATED_BWD) {
    struct Pre {
      Floats<V> g, u;
    };
    x.template hand_out<V, 4>(
        smem, 0,
        [&](uint32_t r, uint32_t col) {
          const uint64_t row = (uint64_t)row0 + r;
          Pre q = {};
          if (row < m) {
            q.g = load_floats<V>(p.a[1] + row * (uint64_t)n * 4, (uint64_t)col0 + col, n, n % 4 == 0);
            q.u = load_floats<V>(p.b[1] + row * (uint64_t)n * 4, (uint64_t)col0 + col, n, n % 4 == 0);
          }
          return q;
        },
        [&](uint32_t r, uint32_t col, float* dh, float*, const Pre& q) {
          const uint64_t row = (uint64_t)row0 + r;
          if (row >= m) return;
          float dg[V], du[V], h[V];
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const Act f = activate<ACT, true>(q.g.v[e]);
            dg[e] = dh[e] * q.u.v[e] * f.d;
            du[e] = dh[e] * f.v;
            h[e] = f.v * q.u.v[e];
          }
          const uint64_t to = row * ldc * ES, low = to + p.fold * ldc * ES;
          const bool two = FOLDS && p.fold != 0;
          store_terms<DT, V>(p.c[0] + to, two ? p.c[0] + low : nullptr, (uint64_t)col0 + col, p.ldc, vec, dg);
          store_terms<DT, V>(p.c[1] + to, two ? p.c[1] + low : nullptr, (uint64_t)col0 + col, p.ldc, vec, du);
          store_terms<DT, V>(p.c[2] + to, two ? p.c[2] + low : nullptr, (uint64_t)col0 + col, p.ldc, vec, h);
        });
  } else if constexpr (KIND == PK_DLOGITS) {
    struct Row {
      uint32_t at;  // the target's column in this problem, if it lies there
      float z, g;
      bool live;
    };
    x.template hand_out<V, 4>(
        smem, 0,
        [&](uint32_t r, uint32_t) {
          const uint64_t row = (uint64_t)row0 + r;
          Row q = {0xffffffffu, 0.f, 0.f, false};
          if (row < m) {
            const int64_t t = a.target[row];
            q.live = t >= 0 && (uint64_t)t < a.vocab;
            q.at = target_column(t, a.vocab, p.col0, n);
            q.z = ((const float*)p.a[1])[row];
            q.g = a.scale ? a.grad[row] / *a.scale : a.grad[row];
          }
          return q;
        },
        [&](uint32_t r, uint32_t col, float* v, float*, const Row& q) {
          const uint64_t row = (uint64_t)row0 + r;
          if (row >= m) return;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const uint32_t c = col0 + col + e;
            const float d = (exp_of<DT>(v[e] - q.z) - (c == q.at ? 1.0f : 0.0f)) * q.g;
            v[e] = q.live && c < n ? d : 0.f;  // columns n .. ldc: zeros
          }
          char* to = p.c[0] + row * ldc * ES;
          store_terms<DT, V, true>(to, FOLDS && p.fold ? to + p.fold * ldc * ES : nullptr, (uint64_t)col0 + col, p.ldc, vec, v);
        });
  } else if constexpr (P::WK > 1) {  // PK_STATS, K split over the waves
    float* at_target = (float*)p.c[1];
    x.template hand_out<V, 1>(
        smem, 0,
        [&](uint32_t r, uint32_t) {
          const uint64_t row = (uint64_t)row0 + r;
          return target_column(row < m ? a.target[row] : -1, a.vocab, p.col0, n);
        },
        [&](uint32_t r, uint32_t col, float* v, float*, uint32_t at) {
          // the COLS / V threads of a row are neighbours in a wave
          const uint64_t row = (uint64_t)row0 + r;
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const uint32_t c = col0 + col + e;
            if (c < n) top = fmaxf(top, v[e]);
            if (c == at && row < m) at_target[row] = v[e];
          }
#pragma unroll
          for (int o = 1; o < P::COLS / V; o *= 2) top = fmaxf(top, __shfl_xor(top, o));
          const float shift = stats_shift(top);
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (col0 + col + e < n) sum += exp_of<DT>(v[e] - shift);
#pragma unroll
          for (int o = 1; o < P::COLS / V; o *= 2) sum += __shfl_xor(sum, o);
          if (col == 0 && row < m) ((float2*)p.c[0])[(uint64_t)(col0 / P::COLS) * m + row] = make_float2(top, sum);
        });
  } else {  // PK_STATS
    __syncthreads();  // every wave is done with the tiles
    float2* part = (float2*)smem;  // [WN][BM]
    const uint32_t lane = threadIdx.x & 63;
    const int wn = uniform((int)(threadIdx.x / 64)) % P::WN;
#pragma unroll
    for (int i = 0; i < P::TM; ++i) {
      const uint32_t r = P::wave_row() + 16 * i + (lane & 15);
      const uint64_t row = (uint64_t)row0 + r;
      const uint32_t at = target_column(row < m ? a.target[row] : -1, a.vocab, p.col0, n);
      float top = -INFINITY, value = 0.f;
      bool hit = false;
#pragma unroll
      for (int j = 0; j < P::TN; ++j) {
        const uint32_t col = col0 + P::wave_col() + 16 * j + 4 * (lane >> 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = x.acc[i][j][e];
          top = col + e < n ? fmaxf(top, v) : top;
          value = col + e == at ? v : value;
          hit = hit || col + e == at;
        }
      }
      if (hit) ((float*)p.c[1])[row] = value;
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float shift = stats_shift(top);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < P::TN; ++j) {
        const uint32_t col = col0 + P::wave_col() + 16 * j + 4 * (lane >> 4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < n) sum += exp_of<DT>(x.acc[i][j][e] - shift);
      }
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (lane < 16) part[wn * P::BM + r] = make_float2(top, sum);
    }
    __syncthreads();
    for (uint32_t r = threadIdx.x; r < (uint32_t)P::BM; r += P::NT) {
      const uint64_t row = (uint64_t)row0 + r;
      if (row >= m) continue;
      float2 s = part[r];
#pragma unroll
      for (int w = 1; w < P::WN; ++w) s = merge_stats(s, part[w * P::BM + r]);
      ((float2*)p.c[0])[(uint64_t)(col0 / P::COLS) * m + row] = s;
    }
  }
}

constexpr int layout_b(int kind) { return kind >= PK_GATED_BWD ? L_R : L_K; }

// Adds the shares of the problems that have them, in order, and finishes as the
// product kernel would have: times scale, plus the sum so far (GRAD_ADD), as the
// result or as the sum (GRAD_PARTIAL).
template <int DT>
__global__ __launch_bounds__(256) void finish_kernel(const ProductArgs a, int32_t count) {
  const float scale = a.scale ? *a.scale : 1.0f;
  for (int q = 0; q < count; ++q) {
    const Problem& p = a.p[q];
    const uint64_t total = (uint64_t)(p.m - p.fold) * p.ldc;
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < total; i += gridDim.x * 256ull) {
      const float* part = (const float*)p.c[2] + i;
      float v = 0.f;
      for (uint32_t s = 0; s < p.shares; ++s) v += part[s * total];
      v *= scale;
      if (p.mode & GRAD_ADD) v = ((const float*)p.c[1])[i] + v;
      if (p.mode & GRAD_PARTIAL) ((float*)p.c[1])[i] = v;
      else if (DT == DT_BF16) ((uint16_t*)p.c[0])[i] = (uint16_t)bf16_round(v);
      else ((float*)p.c[0])[i] = v;
    }
  }
}

template <int KIND, int DT, class TILE, uint32_t ACT>
hipError_t launch(ProductPlan& plan, hipStream_t stream) {
  using P = Product<DT, L_K, layout_b(KIND), KIND == PK_GATED, TILE>;
  if (!plan.cut(P::BM, P::COLS)) return hipErrorInvalidValue;
  if (plan.tiles == 0) return hipSuccess;
  hipLaunchKernelGGL((product_kernel<P, KIND, ACT>), dim3((unsigned)plan.tiles), dim3(P::NT), 0, stream, plan.a);
  const hipError_t e = hipGetLastError();
  if constexpr (KIND == PK_STORE_NT || KIND == PK_GRADS) {
    if (e == hipSuccess && plan.a.p[0].shares > 1) {
      const uint64_t each = ((uint64_t)(plan.a.p[0].m - plan.a.p[0].fold) * plan.a.p[0].ldc + 255) / 256;
      hipLaunchKernelGGL(finish_kernel<DT>, dim3((unsigned)(each < 1024 ? each : 1024)), dim3(256), 0, stream, plan.a,
                         plan.sharing());
      return hipGetLastError();
    }
  }
  return e;
}

template <int KIND, int DT, uint32_t ACT = ACT_SILU>
hipError_t launch_kind(ProductPlan& plan, int device, hipStream_t stream) {
  const TileChoice choice = product_tile(KIND, DT, plan, device);
  const int tile = choice.tile;
  for (int i = 0; i < plan.sharing(); ++i) plan.a.p[i].shares = choice.shares;
  if constexpr (DT == DT_BF16) {  // classes of one type only
    if (tile == TILE_LARGE) return launch<KIND, DT, Large, ACT>(plan, stream);
    if (tile == TILE_FLAT) return launch<KIND, DT, Flat, ACT>(plan, stream);
  } else {
    if (tile == TILE_TALL) return launch<KIND, DT, Tall, ACT>(plan, stream);
  }
  switch (tile) {
    case TILE_SMALL: return launch<KIND, DT, Small, ACT>(plan, stream);
    case TILE_SPLIT: return launch<KIND, DT, Split, ACT>(plan, stream);
    case TILE_THIN: return launch<KIND, DT, Thin, ACT>(plan, stream);
  }
  return hipErrorInvalidValue;
}

template <int KIND, int DT>
hipError_t launch_gated(ProductPlan& plan, int device, hipStream_t stream) {
  switch (plan.a.act) {
    case ACT_SILU: return launch_kind<KIND, DT, ACT_SILU>(plan, device, stream);
    case ACT_GELU: return launch_kind<KIND, DT, ACT_GELU>(plan, device, stream);
    case ACT_GELU_TANH: return launch_kind<KIND, DT, ACT_GELU_TANH>(plan, device, stream);
  }
  return hipErrorInvalidValue;
}

template <int DT>
hipError_t launch_typed(int kind, ProductPlan& plan, int device, hipStream_t stream) {
  switch (kind) {
    case PK_GATED: return launch_gated<PK_GATED, DT>(plan, device, stream);
    case PK_STORE_NT: return launch_kind<PK_STORE_NT, DT>(plan, device, stream);
    case PK_STATS: return launch_kind<PK_STATS, DT>(plan, device, stream);
    case PK_DLOGITS: return launch_kind<PK_DLOGITS, DT>(plan, device, stream);
    case PK_GATED_BWD: return launch_gated<PK_GATED_BWD, DT>(plan, device, stream);
    case PK_GRADS: return launch_kind<PK_GRADS, DT>(plan, device, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

}  // namespace ar
