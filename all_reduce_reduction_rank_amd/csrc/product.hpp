// product.hpp -- the tile product shared by the tensor-parallel layer
// operators (ffn.hip, xent.hip): C = A B^T over tiles of BM x BN, fp32
// accumulate on the matrix cores, for the three operand layouts a layer and
// its gradients need.
//
// An operand is a matrix of "rows" (C's rows for A, C's columns for B) by k:
//   L_K: k runs fastest (row-major [rows, k], a linear layer's x and weights)
//   L_R: rows run fastest (row-major [k, rows]); a product that sums over
//        the tokens or over the output features reads its operand this way,
//        so no transposed copy is made.
// A tile of either operand takes BM (BN) x 128 bytes of LDS: 64 k of bf16 or
// 32 k of fp32.  Two buffers alternate: while the waves multiply one, the
// loads of the next K step land in the other.
//
// LDS layout and bank conflicts.  Tiles are written 16 bytes per lane in
// lane order (the direct global -> LDS loads allow nothing else), so the
// order is permuted on the global side: the 16-byte chunk at position p of
// an LDS row holds chunk p ^ f(row) of the matrix row.
//   L_K rows are 8 chunks; f = row & 7: the 16 rows a fragment read touches
//       fall on all 8 chunk columns.
//   L_R rows (one k each) are BM * esize / 16 chunks.  bf16 fragments come
//       from the transposing LDS read, whose 16-lane groups read 4 k x 32
//       bytes; f = 2 ((k & 3) + 4 ((k >> 3) & 1)) spreads the 8 rows of two
//       neighbouring groups over 256 bytes.  fp32 fragments are 4-byte reads
//       of 16 consecutive rows at 4 k; f = 4 ((k >> 2) & 3) puts the four
//       64-byte pieces side by side.
//
// Matrix instructions: 16x16x32 bf16 or four 16x16x4 fp32, one 16-byte
// fragment of each operand per step.  Both types place k alike (lane group q
// holds k = 8 q + j, or 4 q + j), so the layouts mix freely.  B goes in as
// the instruction's first operand: a lane then holds 4 consecutive columns of
// one row of C, and stores them as one vector.
//
// Bounds: the buffer descriptor of each K step ends at the last valid row
// (L_K) or the last valid k (L_R) of the tile, and lanes past K in an L_K row
// are sent past the end, so every out-of-range chunk reads as zero and
// nothing outside a matrix is touched.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "device.hpp"
#include "schedule.hpp"

namespace ar {

enum : int { L_K = 0, L_R = 1 };

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
// 16 bytes at any byte address (global memory reads need no alignment)
typedef uint32_t v4u_any __attribute__((ext_vector_type(4), aligned(1)));

typedef __attribute__((address_space(3))) char lds_char;

constexpr int KBYTES = 128;       // bytes of k per operand row and K step
constexpr uint32_t OUT_OF_RANGE = 0x7fffff00u;  // beyond every descriptor (at most 2^30 bytes)
constexpr int MAX_PROBLEMS = 3 * MAX_RANKS;

template <int DT>
struct KElem {
  static constexpr int ES = DT == DT_BF16 ? 2 : 4;  // bytes of an element
  static constexpr int E = 16 / ES;                 // elements of a 16-byte chunk
  static constexpr int BK = KBYTES / ES;            // k per step
};

// One product of a launch.  `first` .. `first` + tiles_m * tiles_n are its
// tiles in the launch.  With two K segments, C = a[0] b[0]^T + a[1] b[1]^T;
// a paired product has b[0] and b[1] side by side in every tile.
struct Problem {
  const char* a[2];
  const char* b[2];
  char* c[3];
  const char* e[2];
  uint64_t col0;  // first column's index in the whole matrix (vocabulary offset)
  uint32_t m, n, k;
  uint32_t lda, ldb, ldc;  // elements between rows of storage
  uint32_t tiles_m, tiles_n, first;
  uint32_t mode;  // epilogue variant
};

struct ProductArgs {
  Problem p[MAX_PROBLEMS];
  const int64_t* target;  // cross entropy: per row
  const float* grad;      // cross entropy: per row
  uint64_t vocab;         // cross entropy: targets outside [0, vocab) are ignored
  int32_t nprob, nseg;
  uint32_t tiles;  // of all problems
};

// Workgroup -> tile.  Workgroups go to the XCDs round robin; XCD x takes the
// x-th contiguous eighth of the tiles, so the tiles that share operand panels
// share an L2.
__device__ __forceinline__ uint32_t tile_of_block(uint32_t b, uint32_t tiles) {
  const uint32_t x = b % XCDS, i = b / XCDS;
  const uint32_t per = tiles / XCDS, extra = tiles % XCDS;
  return x * per + (x < extra ? x : extra) + i;
}

// Tile index within a problem -> (row tile, column tile): groups of GROUP row
// tiles, column by column, so that the ~32 tiles an XCD runs at once form a
// block and re-read few panels.
__device__ __forceinline__ void tile_coords(uint32_t t, uint32_t tiles_m, uint32_t tiles_n, uint32_t* tm,
                                            uint32_t* tn) {
  constexpr uint32_t GROUP = 8;
  const uint32_t g = t / (GROUP * tiles_n), rest = t % (GROUP * tiles_n);
  const uint32_t rows = tiles_m - g * GROUP < GROUP ? tiles_m - g * GROUP : GROUP;
  *tm = g * GROUP + rest % rows;
  *tn = rest / rows;
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }
template <class T>
__device__ __forceinline__ T* uniform(T* p) {
  const uint64_t x = (uint64_t)p;
  const uint32_t lo = uniform((uint32_t)x), hi = uniform((uint32_t)(x >> 32));
  return (T*)(((uint64_t)hi << 32) | lo);
}

// Buffer descriptor of `bytes` bytes from p on (raw 32-bit data; offsets past
// the end read as zero).
__device__ __forceinline__ v4u descriptor(const char* p, uint32_t bytes) {
  const uint64_t x = (uint64_t)p;
  return v4u{uniform((uint32_t)x), uniform((uint32_t)(x >> 32)) & 0xffffu, uniform(bytes), 0x00020000u};
}

// 16 bytes per lane from the buffer to LDS: lane l's land at dst + 16 l.
// `dst` is uniform over the wave.  Inline, so that the compiler does not wait
// for the load before the next LDS read of another buffer (the kernels wait
// themselves, before the barrier that publishes a buffer); there is no output
// register a load in flight could overwrite.
__device__ __forceinline__ void load_to_lds(v4u rsrc, uint32_t off, lds_char* dst) {
  const uint32_t at = uniform((uint32_t)(uintptr_t)dst);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(rsrc)
               : "m0");
}

// Loads one operand's tiles.  ROWS rows (of one matrix, or ROWS / 2 of each
// of two when PAIR) by 128 bytes of k, by NT threads.
template <int DT, int LAYOUT, int ROWS, int NT, bool PAIR, bool ALIGNED>
struct TileLoader {
  static constexpr int ES = KElem<DT>::ES, E = KElem<DT>::E, BK = KElem<DT>::BK;
  static constexpr int SLOTS = ROWS * 8 / NT;  // 16-byte chunks per thread
  static constexpr int CH = LAYOUT == L_K ? 8 : ROWS * ES / 16;  // chunks of an LDS row
  static_assert(!PAIR || (LAYOUT == L_K && (ROWS / 2) % (NT / 8) == 0), "a slot's rows lie in one matrix");
  static_assert(SLOTS >= 1, "");

  const char* base[2];  // row0's first element (L_K), or k 0 of row0 (L_R)
  uint32_t rows;        // rows left from row0 on
  uint32_t k;
  uint32_t ldbytes;

  __device__ __forceinline__ static uint32_t swz(uint32_t row) {
    if constexpr (LAYOUT == L_K) return row & 7;
    else if constexpr (DT == DT_BF16) return (2 * ((row & 3) + 4 * ((row >> 3) & 1))) & (CH - 1);
    else return (4 * ((row >> 2) & 3)) & (CH - 1);
  }

  __device__ __forceinline__ void init(const char* p0, const char* p1, uint32_t row0, uint32_t nrows, uint32_t kk,
                                       uint32_t ld) {
    ldbytes = ld * ES;
    k = kk;
    rows = nrows > row0 ? nrows - row0 : 0;
    const uint64_t off = LAYOUT == L_K ? (uint64_t)row0 * ldbytes : (uint64_t)row0 * ES;
    base[0] = p0 + off;
    base[1] = PAIR ? p1 + off : nullptr;
  }

  // Chunk of this thread's slot i: its LDS row and the chunk of the matrix
  // row it holds.
  __device__ __forceinline__ static void slot(int i, uint32_t* row, uint32_t* chunk) {
    const uint32_t p = (uint32_t)i * NT + threadIdx.x;
    *row = p / CH;
    *chunk = (p % CH) ^ swz(*row);
  }

  // Start the direct loads of K step k0 into LDS at `dst`.
  __device__ __forceinline__ void load_direct(uint32_t k0, lds_char* dst) const {
    const uint32_t wave = uniform(threadIdx.x / 64);
    v4u rsrc[2];
#pragma unroll
    for (int h = 0; h < (PAIR ? 2 : 1); ++h) {
      if constexpr (LAYOUT == L_K) {
        constexpr uint32_t R = PAIR ? ROWS / 2 : ROWS;
        const uint32_t bytes = (rows < R ? rows : R) * ldbytes;
        const uint32_t skip = k0 * ES;
        rsrc[h] = descriptor(base[h] + skip, bytes > skip ? bytes - skip : 0);
      } else {
        const uint32_t left = k > k0 ? k - k0 : 0;
        const uint32_t ks = left < (uint32_t)BK ? left : (uint32_t)BK;
        // the last k row ends with the matrix's last row (base is row0's column)
        // (to the end of its chunk: a row of storage is whole chunks)
        const uint32_t span = (rows < (uint32_t)ROWS ? rows : (uint32_t)ROWS) * ES;
        const uint32_t bytes = ks && rows ? (ks - 1) * ldbytes + ((span + 15) & ~15u) : 0;
        rsrc[h] = descriptor(base[h] + (uint64_t)k0 * ldbytes, bytes);
      }
    }
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      uint32_t row, chunk;
      slot(i, &row, &chunk);
      int h = 0;
      if constexpr (PAIR) {
        if (i >= SLOTS / 2) {
          h = 1;
          row -= ROWS / 2;
        }
      }
      uint32_t off = row * ldbytes + chunk * 16;
      if constexpr (LAYOUT == L_K) {
        if (k0 + chunk * E >= k) off = OUT_OF_RANGE;
      } else {
        if (chunk * E >= rows) off = OUT_OF_RANGE;
      }
      load_to_lds(rsrc[h], off, dst + ((uint32_t)i * NT + wave * 64) * 16);
    }
  }

  // Unaligned matrices (a row of partial chunks): the same chunks through
  // registers.  Whole chunks are one 16-byte load at any address; the chunk
  // that crosses the end of a row (of the matrix's rows, L_R) is gathered by
  // element, so no byte outside the matrix is read.
  __device__ __forceinline__ void load_regs(uint32_t k0, v4u* r) const {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      uint32_t row, chunk;
      slot(i, &row, &chunk);
      int h = 0;
      if constexpr (PAIR) {
        if (i >= SLOTS / 2) {
          h = 1;
          row -= ROWS / 2;
        }
      }
      int valid;
      const char* src;
      if constexpr (LAYOUT == L_K) {
        valid = row < rows ? (int)k - (int)(k0 + chunk * E) : 0;
        src = base[h] + (uint64_t)row * ldbytes + (uint64_t)(k0 + chunk * E) * ES;
      } else {
        valid = k0 + row < k ? (int)rows - (int)(chunk * E) : 0;
        src = base[h] + (uint64_t)(k0 + row) * ldbytes + chunk * 16;
      }
      v4u v = {0, 0, 0, 0};
      if (valid >= E) {
        v = *(const v4u_any*)src;
      } else if (valid > 0) {
#pragma unroll
        for (int j = 0; j < E; ++j) {
          if (j < valid) {
            if constexpr (DT == DT_BF16) v[j / 2] |= (uint32_t)((const uint16_t*)src)[j] << (16 * (j % 2));
            else v[j] = ((const uint32_t*)src)[j];
          }
        }
      }
      r[i] = v;
    }
  }
  __device__ __forceinline__ void store_regs(const v4u* r, lds_char* dst) const {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      *(__attribute__((address_space(3))) v4u*)(dst + ((uint32_t)i * NT + threadIdx.x) * 16) = r[i];
  }

  // Fragment of 16 rows from r0 on, K substep s (0, 1): 16 bytes per lane.
  __device__ __forceinline__ static v4u fragment(const lds_char* tile, int r0, int s) {
    const uint32_t lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
    if constexpr (LAYOUT == L_K) {
      const uint32_t chunk = (uint32_t)(s * 4) + q;
      return *(const __attribute__((address_space(3))) v4u*)(tile + (r0 + i) * KBYTES + ((chunk ^ (i & 7)) * 16));
    } else if constexpr (DT == DT_BF16) {
      constexpr uint32_t RB = ROWS * 2;
      const uint32_t kr = (uint32_t)s * 32 + 8 * q + i / 4;
      const uint32_t chunk = ((uint32_t)r0 / 8 + (i % 4) / 2) ^ swz(kr);
      const lds_char* p = tile + kr * RB + chunk * 16 + (i & 1) * 8;
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)p);
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(p + 4 * RB));
      typedef short v8s __attribute__((ext_vector_type(8)));
      const v8s both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(v4u, both);
    } else {
      constexpr uint32_t RB = ROWS * 4;
      v4u v;
      const uint32_t chunk = ((uint32_t)r0 / 4 + i / 4) ^ swz(4 * q);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = *(const __attribute__((address_space(3))) uint32_t*)(tile + ((uint32_t)s * 16 + 4 * q + j) * RB +
                                                                    chunk * 16 + (i & 3) * 4);
      return v;
    }
  }
};

template <int DT>
__device__ __forceinline__ v4f mma(v4u first, v4u second, v4f acc) {
  if constexpr (DT == DT_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, first), __builtin_bit_cast(v8bf, second),
                                                   acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(first[j]), __uint_as_float(second[j]), acc, 0, 0, 0);
    return acc;
  }
}

// Tile sizes.  WM x WN waves share the BM x BN tile.
struct Large {  // 8 waves of 128 x 64
  static constexpr int BM = 256, BN = 256, WM = 2, WN = 4;
};
struct Small {  // 4 waves of 64 x 64
  static constexpr int BM = 128, BN = 128, WM = 2, WN = 2;
};

template <int DT_, int LA_, int LB_, bool PAIR_, bool ALIGNED_, class TILE_>
struct Product {
  static constexpr int DT = DT_, LA = LA_, LB = LB_;
  static constexpr bool PAIR = PAIR_, ALIGNED = ALIGNED_;
  using TILE = TILE_;
  static constexpr int BM = TILE::BM, BN = TILE::BN, WM = TILE::WM, WN = TILE::WN;
  static constexpr int NT = 64 * WM * WN;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 blocks per wave
  static constexpr int COLS = PAIR ? BN / 2 : BN;             // columns of C a tile covers
  static constexpr int STAGE = (BM + BN) * KBYTES;
  static constexpr int LDS_BYTES = 2 * STAGE;

  using LoadA = TileLoader<DT, LA, BM, NT, false, ALIGNED>;
  using LoadB = TileLoader<DT, LB, BN, NT, PAIR, ALIGNED>;

  v4f acc[TM][TN];

  // This wave's first row in the A tile / its block j's first row in the B
  // tile.  A paired tile holds BN / 2 rows of b[0], then BN / 2 of b[1];
  // blocks j and j + TN / 2 of a wave are the same columns of the two.
  __device__ __forceinline__ static int wave_row() { return uniform((int)(threadIdx.x / 64)) / WN * (BM / WM); }
  __device__ __forceinline__ static int wave_col() {
    return uniform((int)(threadIdx.x / 64)) % WN * ((PAIR ? BN / 2 : BN) / WN);
  }
  __device__ __forceinline__ static int block_row(int j) {
    if constexpr (PAIR) return j < TN / 2 ? wave_col() + 16 * j : BN / 2 + wave_col() + 16 * (j - TN / 2);
    else return wave_col() + 16 * j;
  }

  __device__ __forceinline__ void step(const lds_char* lds) {
    const lds_char* ta = lds;
    const lds_char* tb = lds + BM * KBYTES;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      v4u fb[TN], fa[TM];
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[j] = LoadB::fragment(tb, block_row(j), s);
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[i] = LoadA::fragment(ta, wave_row() + 16 * i, s);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = mma<DT>(fb[j], fa[i], acc[i][j]);
    }
  }

  // Accumulate the tile at (row0, col0) of problem p.
  __device__ __forceinline__ void run(const Problem& p, int nseg, uint32_t row0, uint32_t col0, char* smem) {
    lds_char* lds = (lds_char*)smem;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    const uint32_t per = (p.k + KElem<DT>::BK - 1) / KElem<DT>::BK;
    const uint32_t steps = per * (uint32_t)nseg;
    if (steps == 0) return;
    LoadA la[2];
    LoadB lb[2];
    la[0].init(p.a[0], nullptr, row0, p.m, p.k, p.lda);
    lb[0].init(p.b[0], p.b[1], col0, p.n, p.k, p.ldb);
    la[1].init(p.a[1], nullptr, row0, p.m, p.k, p.lda);
    lb[1].init(p.b[1], nullptr, col0, p.n, p.k, p.ldb);
    auto start = [&](uint32_t t, lds_char* dst) {
      const bool second = t >= per;
      LoadA a = la[0];
      LoadB b = lb[0];
      if (second) {
        a.base[0] = la[1].base[0];
        b.base[0] = lb[1].base[0];
      }
      const uint32_t k0 = (second ? t - per : t) * KElem<DT>::BK;
      a.load_direct(k0, dst);
      b.load_direct(k0, dst + BM * KBYTES);
    };
    if constexpr (ALIGNED) {
      start(0, lds);
      for (uint32_t t = 0; t < steps; ++t) {
        // This wave's loads of step t have landed; behind the barrier
        // everyone's have, and the other buffer is free.
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (t + 1 < steps) start(t + 1, lds + ((t + 1) & 1) * STAGE);
        step(lds + (t & 1) * STAGE);
      }
    } else {
      v4u ra[LoadA::SLOTS], rb[LoadB::SLOTS];
      auto fetch = [&](uint32_t t) {
        const bool second = t >= per;
        LoadA a = la[0];
        LoadB b = lb[0];
        if (second) {
          a.base[0] = la[1].base[0];
          b.base[0] = lb[1].base[0];
        }
        const uint32_t k0 = (second ? t - per : t) * KElem<DT>::BK;
        a.load_regs(k0, ra);
        b.load_regs(k0, rb);
      };
      fetch(0);
      for (uint32_t t = 0; t < steps; ++t) {
        lds_char* buf = lds + (t & 1) * STAGE;
        la[0].store_regs(ra, buf);
        lb[0].store_regs(rb, buf + BM * KBYTES);
        __syncthreads();
        if (t + 1 < steps) fetch(t + 1);
        step(buf);
      }
    }
  }

  // Visit every group of 4 consecutive columns this lane holds:
  // f(row, col, i, j) with C's local row and first column; block j of a
  // paired product's second half is passed as its first half's partner.
  template <class F>
  __device__ __forceinline__ void visit(F&& f) {
    const uint32_t lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < (PAIR ? TN / 2 : TN); ++j)
        f((uint32_t)wave_row() + 16 * i + (lane & 15), (uint32_t)wave_col() + 16 * j + 4 * (lane >> 4), i, j);
  }
};

// Store 4 consecutive values of a row (n left in the row) as the payload type.
template <int DT>
__device__ __forceinline__ void store4(char* row, uint64_t col, uint32_t n, bool vec, const float* v) {
  if constexpr (DT == DT_BF16) {
    const uint32_t h[4] = {bf16_round(v[0]), bf16_round(v[1]), bf16_round(v[2]), bf16_round(v[3])};
    if (vec && col + 4 <= n) {
      *(uint2*)(row + col * 2) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    } else {
      for (int e = 0; e < 4; ++e)
        if (col + e < n) *(uint16_t*)(row + (col + e) * 2) = (uint16_t)h[e];
    }
  } else {
    if (vec && col + 4 <= n) {
      *(float4*)(row + col * 4) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      for (int e = 0; e < 4; ++e)
        if (col + e < n) *(float*)(row + (col + e) * 4) = v[e];
    }
  }
}

// Load 4 consecutive values of a row as floats (0 beyond n).
template <int DT>
__device__ __forceinline__ void load4(const char* row, uint64_t col, uint32_t n, bool vec, float* v) {
  if constexpr (DT == DT_BF16) {
    if (vec && col + 4 <= n) {
      const uint2 x = *(const uint2*)(row + col * 2);
      v[0] = __uint_as_float(x.x << 16);
      v[1] = __uint_as_float(x.x & 0xffff0000u);
      v[2] = __uint_as_float(x.y << 16);
      v[3] = __uint_as_float(x.y & 0xffff0000u);
    } else {
      for (int e = 0; e < 4; ++e)
        v[e] = col + e < n ? __uint_as_float((uint32_t)((const uint16_t*)row)[col + e] << 16) : 0.f;
    }
  } else {
    if (vec && col + 4 <= n) {
      const float4 x = *(const float4*)(row + col * 4);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      for (int e = 0; e < 4; ++e) v[e] = col + e < n ? ((const float*)row)[col + e] : 0.f;
    }
  }
}

// Find this workgroup's problem and tile.  Returns the problem's index.
template <class P>
__device__ __forceinline__ int locate(const ProductArgs& a, uint32_t* row0, uint32_t* col0) {
  const uint32_t t = tile_of_block(blockIdx.x, a.tiles);
  int q = 0;
  while (q + 1 < a.nprob && t >= a.p[q + 1].first) ++q;
  uint32_t tm, tn;
  tile_coords(t - a.p[q].first, a.p[q].tiles_m, a.p[q].tiles_n, &tm, &tn);
  *row0 = tm * P::BM;
  *col0 = tn * P::COLS;
  return q;
}

// ------------------------------------------------------------ host side

// Collects the problems of a launch.
struct ProductPlan {
  ProductArgs a;
  bool aligned = true;  // every operand's rows start on 16-byte boundaries
  uint64_t tiles = 0;

  ProductPlan() { memset(&a, 0, sizeof(a)); a.nseg = 1; }

  // Operand checks of p, then a place for it; `es`: element bytes.
  Problem* add(uint64_t m, uint64_t n, uint64_t k, uint64_t lda, uint64_t ldb, uint64_t ldc, uint64_t es) {
    Problem* p = &a.p[a.nprob++];
    p->m = (uint32_t)m, p->n = (uint32_t)n, p->k = (uint32_t)k;
    p->lda = (uint32_t)lda, p->ldb = (uint32_t)ldb, p->ldc = (uint32_t)ldc;
    if (k && ((lda * es) % 16 || (ldb * es) % 16)) aligned = false;
    return p;
  }
  // Tiles of every problem for a kernel whose tile covers bm x cols of C.
  bool cut(uint32_t bm, uint32_t cols) {
    tiles = 0;
    for (int i = 0; i < a.nprob; ++i) {
      Problem& p = a.p[i];
      p.tiles_m = (uint32_t)(((uint64_t)p.m + bm - 1) / bm);
      p.tiles_n = (uint32_t)(((uint64_t)p.n + cols - 1) / cols);
      p.first = (uint32_t)tiles;
      tiles += (uint64_t)p.tiles_m * p.tiles_n;
    }
    a.tiles = (uint32_t)tiles;
    return tiles < (1ull << 31);
  }
};

}  // namespace ar
