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
// A K step is 128 bytes of k of every row, two substeps of 64 (32 bf16 or 16
// fp32): one 16-byte fragment per lane and 16 rows each.  A ring of buffers
// holds K steps: the direct global -> LDS loads of the next ones are in flight
// while the waves multiply.
//
// LDS layout and bank conflicts.  Tiles are written 16 bytes per lane in
// lane order (the direct global -> LDS loads allow nothing else), so the
// order is permuted on the global side: the 16-byte chunk at position p of
// an LDS row holds chunk p ^ f(row) of the matrix row.
//   L_K rows are 8 chunks; f = row & 7: the 16 rows of a fragment read touch
//       every chunk column twice, 256 bytes apart (a kernel that reads nothing
//       else from LDS, the statistics of 4096 x 131072 logits, counts no conflict).
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

typedef __attribute__((address_space(3))) char lds_char;

constexpr int KB = 128;  // bytes of k per operand row and K step: a cache line, two substeps
constexpr uint32_t OUT_OF_RANGE = 0x7fffff00u;  // beyond every descriptor (at most 2^30 bytes)
constexpr int MAX_PROBLEMS = 4 * MAX_RANKS;
constexpr uint32_t MAX_SHARES = 16;  // of a tile's K

template <int DT>
struct KElem {
  static constexpr int ES = DT == DT_BF16 ? 2 : 4;  // bytes of an element
  static constexpr int E = 16 / ES;                 // elements of a 16-byte chunk
};

// One product of a launch.  `first` .. `first` + tiles_m * tiles_n are its
// tiles in the launch.  With two K segments, C = a[0] b[0]^T + a[1] b[1]^T;
// a paired product has b[0] and b[1] side by side in every tile.  Elsewhere
// a[1] and b[1] are what the epilogue reads.
struct Problem {
  const char* a[2];
  const char* b[2];
  char* c[3];
  uint64_t col0;  // first column's index in the whole matrix (vocabulary offset)
  uint32_t m, n, k;
  uint32_t lda, ldb, ldc;  // elements between rows of storage
  uint32_t tiles_m, tiles_n, first;
  uint32_t nseg;  // K segments
  // Rows in two bf16 terms, value + what its rounding left (kept so where there
  // are few of them): the products that write such a matrix put the second
  // terms `fold` rows below the first; those that read it as A have both in
  // one tile of 2 fold rows and add row r + fold to row r of the result.
  uint32_t fold;
  // Workgroups that share a tile's K; with more than one, each stores its fp32
  // sum to c[2] + its share's [rows, ldc] block, and a second kernel adds them.
  uint32_t shares;
  uint32_t mode;  // what the epilogue (and PK_GRADS' layout) goes by
};

struct ProductArgs {  // a kernel's arguments: at most 4 KB
  Problem p[MAX_PROBLEMS];
  const int64_t* target;  // cross entropy: per row
  const float* grad;      // cross entropy: per row
  uint64_t vocab;         // cross entropy: targets outside [0, vocab) are ignored
  const float* scale;     // cross entropy: one value; d is stored over it, dx and dw times it (null: 1)
  int32_t nprob;
  int32_t act;     // gated kinds
  uint32_t tiles;  // of all problems
  uint32_t head;   // of the problems that start first (ProductPlan::head)
};

static_assert(sizeof(ProductArgs) <= 4096, "");

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

// Buffer descriptor of `bytes` bytes from p on (raw 32-bit data; offsets past
// the end read as zero).
__device__ __forceinline__ v4u descriptor(const char* p, uint32_t bytes) {
  const uint64_t x = (uint64_t)p;
  return v4u{uniform((uint32_t)x), uniform((uint32_t)(x >> 32)) & 0xffffu, uniform(bytes), 0x00020000u};
}

// 16 bytes per lane from the buffer to LDS: lane l's land at dst + 16 l.
// `dst` and `soff` (added to every lane's offset) are uniform over the wave.  Inline, so that the compiler does not wait
// for the load before the next LDS read of another buffer (the kernels wait
// themselves, before the barrier that publishes a buffer); there is no output
// register a load in flight could overwrite.
__device__ __forceinline__ void load_to_lds(v4u rsrc, uint32_t off, uint32_t soff, lds_char* dst) {
  const uint32_t at = uniform((uint32_t)(uintptr_t)dst);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(at), "v"(off),
               "s"(rsrc), "s"(soff)
               : "m0");
}

// Loads one operand's tiles.  ROWS rows (of one matrix, or ROWS / 2 of each
// of two when PAIR) by KB bytes of k, by NT threads (thread `tid` of them).
template <int DT, int LAYOUT, int ROWS, int NT, bool PAIR>
struct TileLoader {
  static constexpr int ES = KElem<DT>::ES, E = KElem<DT>::E, BK = KB / ES;
  static constexpr int SLOTS = ROWS * (KB / 16) / NT;  // 16-byte chunks per thread
  static constexpr int CH = LAYOUT == L_K ? KB / 16 : ROWS * ES / 16;  // chunks of an LDS row
  // slots after which a thread's swizzle repeats (its rows are NT / CH apart)
  static constexpr int PERIOD = NT / CH >= 16 || SLOTS == 1 ? 1 : 16 / (NT / CH) < SLOTS ? 16 / (NT / CH) : SLOTS;
  static_assert(SLOTS % PERIOD == 0 && (!PAIR || (SLOTS / 2) % PERIOD == 0), "");
  static_assert(!PAIR || (LAYOUT == L_K && (ROWS / 2) % (NT / CH) == 0), "a slot's rows lie in one matrix");
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
    const uint32_t p = (uint32_t)i * NT + threadIdx.x % NT;
    *row = p / CH;
    *chunk = (p % CH) ^ swz(*row);
  }

  // Start the direct loads of K step k0 into LDS at `dst`.
  __device__ __forceinline__ void load_direct(uint32_t k0, lds_char* dst) const {
    const uint32_t wave = uniform(threadIdx.x % NT / 64);
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
    uint32_t off[PERIOD];
#pragma unroll
    for (int i = 0; i < PERIOD; ++i) {
      uint32_t row, chunk;
      slot(i, &row, &chunk);
      const bool in = LAYOUT == L_K ? k0 + chunk * E < k : chunk * E < rows;
      off[i] = in ? row * ldbytes + chunk * 16 : OUT_OF_RANGE;
    }
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int h = PAIR && i >= SLOTS / 2 ? 1 : 0;
      const uint32_t turn = (uint32_t)((h ? i - SLOTS / 2 : i) / PERIOD * PERIOD);
      load_to_lds(rsrc[h], off[i % PERIOD], turn * (NT / CH) * ldbytes, dst + ((uint32_t)i * NT + wave * 64) * 16);
    }
  }

  // Fragment of 16 rows from r0 on, substep s: 16 bytes per lane.
  __device__ __forceinline__ static v4u fragment(const lds_char* tile, int r0, int s) {
    const uint32_t lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
    if constexpr (LAYOUT == L_K) {
      return *(const __attribute__((address_space(3))) v4u*)(tile + (r0 + i) * KB + (((uint32_t)s * 4 + q) ^ swz(i)) * 16);
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

// One 16 x 16 block: acc += first second^T, element j of the fragments (fp32;
// bf16 takes the whole fragments at once).
template <int DT>
__device__ __forceinline__ v4f mma(v4u first, v4u second, v4f acc, int j) {
  if constexpr (DT == DT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, first), __builtin_bit_cast(v8bf, second),
                                                   acc, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(first[j]), __uint_as_float(second[j]), acc, 0, 0, 0);
}

// Tile classes.  WM x WN waves share the BM x BN tile and a ring of STAGES K
// steps in LDS.  With WK > 1, WK single waves take a part of K
// each, with a ring each and no barrier, and their sums are added in LDS: few
// rows or few tiles still have many loads in flight.
//
// KB is 128, a cache line: with 64 bytes a row, weights streamed for one token
// came at 4.3 TB/s, with lines at 5.4, and the loads alone of an 8192^3
// product at 12.4 TB/s however many were in flight, with lines at up to 18.7.
// The large tile, by parts of an 8192^3 product: its matrix instructions alone took
// 590 us (1.86 PFLOP/s, 1.8 GHz of 2.4), its loads alone 690, both with the LDS
// reads 840; five buffers of half steps, A one step further ahead, 32 x 32
// blocks, other orders of the half step and wave priorities all came within 3 %
// of that, 4 waves of 128 x 128 at 920.  Counters of whole kernels (feed-forward
// step of 8192 rows, loss of 4096): 1.9 to 2.2 GHz, matrix cores busy 0.37 to 0.56
// of the cycles, least where the epilogue moves most: with one workgroup on a CU
// no other's products run under it (K = 5120: statistics 1105 TFLOP/s, gate and
// up 933, gradient of the activation 792).
struct Large {  // 8 waves of 128 x 64, 128 KB of LDS: one workgroup per CU
  static constexpr int BM = 256, BN = 256, WM = 2, WN = 4, WK = 1, STAGES = 2;
};
struct Small {  // 4 waves of 64 x 64, 64 KB: two workgroups per CU
  static constexpr int BM = 128, BN = 128, WM = 2, WN = 2, WK = 1, STAGES = 2;
};
struct Tall {  // 4 waves of 64 x 32, 48 KB: three workgroups per CU (fp32, Flat's place)
  static constexpr int BM = 128, BN = 64, WM = 2, WN = 2, WK = 1, STAGES = 2;
};
struct Flat {  // 4 waves of 64 x 32, 72 KB: two workgroups per CU
  static constexpr int BM = 64, BN = 128, WM = 1, WN = 4, WK = 1, STAGES = 3;
};
struct Split {  // 4 waves, 64 x 64 each of a quarter of K, 128 KB
  static constexpr int BM = 64, BN = 64, WM = 1, WN = 1, WK = 4, STAGES = 2;
};
struct Thin {  // 4 waves, 16 x 32 each of a quarter of K, 72 KB: two workgroups per CU
  static constexpr int BM = 16, BN = 32, WM = 1, WN = 1, WK = 4, STAGES = 3;
};

template <int DT_, int LA_, int LB_, bool PAIR_, class TILE_>
struct Product {
  static constexpr int DT = DT_, LA = LA_, LB = LB_;
  static constexpr bool PAIR = PAIR_;
  using TILE = TILE_;
  using TN_ = Product<DT_, L_R, L_R, false, TILE_>;  // the same tile of a dy^T x product
  static constexpr int BM = TILE::BM, BN = TILE::BN, WM = TILE::WM, WN = TILE::WN;
  static constexpr int WK = TILE::WK;
  static constexpr int STAGES = TILE::STAGES;
  static_assert(WK == 1 || WM * WN == 1, "waves that split K work alone");
  static constexpr int GROUP = 64 * WM * WN, NT = GROUP * WK;  // threads of a ring, of the workgroup
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 blocks per wave
  static constexpr int COLS = PAIR ? BN / 2 : BN;             // columns of C a tile covers
  static constexpr int STAGE = (BM + BN) * KB, RING = STAGES * STAGE;
  static constexpr int LDS_BYTES = WK * RING;

  using LoadA = TileLoader<DT, LA, BM, GROUP, false>;
  using LoadB = TileLoader<DT, LB, BN, GROUP, PAIR>;
  static constexpr int LOADS = LoadA::SLOTS + LoadB::SLOTS;  // direct loads per thread and K step

  v4f acc[TM][TN];

  // This wave's first row in the A tile / its block j's first row in the B
  // tile.  A paired tile holds BN / 2 rows of b[0], then BN / 2 of b[1];
  // blocks j and j + TN / 2 of a wave are the same columns of the two.
  __device__ __forceinline__ static int wave_row() { return WM == 1 ? 0 : uniform((int)(threadIdx.x / 64)) / WN * (BM / WM); }
  __device__ __forceinline__ static int wave_col() {
    return WN == 1 ? 0 : uniform((int)(threadIdx.x / 64)) % WN * ((PAIR ? BN / 2 : BN) / WN);
  }
  __device__ __forceinline__ static int block_row(int j) {
    if constexpr (PAIR) return j < TN / 2 ? wave_col() + 16 * j : BN / 2 + wave_col() + 16 * (j - TN / 2);
    else return wave_col() + 16 * j;
  }

  // Fragment i of A and its share of B's fragments, of substep s.
  __device__ __forceinline__ static void read(const lds_char* buf, int s, v4u* fa, v4u* fb, int i) {
    fa[i] = LoadA::fragment(buf, wave_row() + 16 * i, s);
#pragma unroll
    for (int j = i * TN / TM; j < (i + 1) * TN / TM; ++j) fb[j] = LoadB::fragment(buf + BM * KB, block_row(j), s);
  }
  __device__ __forceinline__ void multiply(const v4u* fa, const v4u* fb, int i) {
#pragma unroll
    for (int e = 0; e < (DT == DT_BF16 ? 1 : 4); ++e)  // outermost: no product waits for the one before it
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mma<DT>(fb[j], fa[i], acc[i][j], e);
  }
  // Order of a step for the compiler: the LDS reads of the next step
  // spread evenly over the first half of the products, so that neither waits
  // for the other.
  static constexpr int READS_A = LA == L_K ? 1 : DT == DT_BF16 ? 2 : 4;
  static constexpr int READS_B = LB == L_K ? 1 : DT == DT_BF16 ? 2 : 4;
  template <int I>
  __device__ __forceinline__ static void interleave() {
    constexpr int R = TM * READS_A + TN * READS_B, M = TM * TN * (DT == DT_BF16 ? 1 : 4), Q = M / 2;
    if constexpr (I < R) {
      __builtin_amdgcn_sched_group_barrier(0x8, (I + 1) * Q / R - I * Q / R, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      interleave<I + 1>();
    } else {
      __builtin_amdgcn_sched_group_barrier(0x8, M - Q, 0);
    }
  }
  // Every load of this wave but the youngest N (all of them unless `more` are
  // behind) has landed, and so has every LDS read; then the barrier of the
  // waves that share the rings.
  template <int N>
  __device__ __forceinline__ static void landed(bool more) {
    if (N > 0 && more) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(N) : "memory");
    else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    if constexpr (WK == 1) {
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    }
  }

  // Accumulate the tile at (row0, col0) of problem p, share `share` of its K.
  //
  // A substep multiplies fragments that were read from LDS during the one
  // before, while it reads the next one's, so the matrix cores never wait for
  // an LDS read.  Before the last substep of step t every wave has read all
  // of t, and step t + 1 must have landed: one barrier there frees step t's
  // buffer for step t + STAGES and publishes t + 1.
  __device__ __forceinline__ void run(const Problem& p, uint32_t share, uint32_t row0, uint32_t col0, char* smem) {
    const int wk = WK == 1 ? 0 : uniform((int)(threadIdx.x / GROUP));
    lds_char* lds = (lds_char*)smem + wk * RING;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    constexpr uint32_t BK = LoadA::BK;
    const uint32_t per = (p.k + BK - 1) / BK;
    const uint32_t all = per * p.nseg;
    // this wave's part of the steps
    const uint32_t parts = WK * p.shares;
    const uint32_t part = (all + parts - 1) / parts;
    const uint32_t first = (share * WK + (uint32_t)wk) * part;
    const uint32_t steps = first >= all ? 0 : all - first < part ? all - first : part;
    if (steps == 0) return;
    LoadA la;
    LoadB lb;
    la.init(p.a[0], nullptr, row0, p.m, p.k, p.lda);
    lb.init(p.b[0], p.b[1], col0, p.n, p.k, p.ldb);
    // the second segment's operands lie where the first's do in their matrices
    const char* const second_a = p.a[1] + (la.base[0] - p.a[0]);
    const char* const second_b = p.b[1] + (lb.base[0] - p.b[0]);
    // Step t's segment, and its first k there.
    auto in_second = [&](uint32_t t) { return p.nseg > 1 && first + t >= per; };
    auto k_of = [&](uint32_t t) { return (in_second(t) ? first + t - per : first + t) * BK; };
    v4u fa[2][TM], fb[2][TN];
    auto start = [&](uint32_t t, lds_char* dst) {
      LoadA a = la;
      LoadB b = lb;
      a.base[0] = in_second(t) ? second_a : la.base[0];
      b.base[0] = in_second(t) ? second_b : lb.base[0];
      a.load_direct(k_of(t), dst);
      b.load_direct(k_of(t), dst + BM * KB);
    };
#pragma unroll
    for (uint32_t t = 0; t < (uint32_t)STAGES; ++t)
      if (t < steps) start(t, lds + t * STAGE);
    landed<(STAGES - 1) * LOADS>(steps >= (uint32_t)STAGES);
#pragma unroll
    for (int i = 0; i < TM; ++i) read(lds, 0, fa[0], fb[0], i);
    // Products of few rows in fp32 add up K in blocks: an error of 1.5e-6 of
    // a row over k = 6478 in one chain is that of the few values it has, and
    // no mean over many evens it out.
    constexpr bool BLOCKED = DT == DT_F32 && WK > 1;
    constexpr uint32_t BLOCK_STEPS = 4;
    v4f sum[BLOCKED ? TM : 1][BLOCKED ? TN : 1];
    if constexpr (BLOCKED) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) sum[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    uint32_t cur = 0;  // byte offset of step t's buffer
    // the two substeps' fragment sets alternate by name
    for (uint32_t t = 0; t < steps; ++t) {
      const uint32_t next = cur + STAGE == (uint32_t)RING ? 0 : cur + STAGE;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1) {
          landed<(STAGES - 2) * LOADS>(t + STAGES <= steps);
          if (t + STAGES < steps) start(t + STAGES, lds + cur);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          // (after the last step: stale, and not used)
          read(lds + (h ? next : cur), 1 - h, fa[1 - h], fb[1 - h], i);
          multiply(fa[h], fb[h], i);
        }
        interleave<0>();
      }
      cur = next;
      if constexpr (BLOCKED) {
        if (t % BLOCK_STEPS == BLOCK_STEPS - 1) {
#pragma unroll
          for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
              sum[i][j] += acc[i][j];
              acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
            }
        }
      }
    }
    if constexpr (BLOCKED) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] += sum[i][j];
    }
    landed<0>(false);
  }

  // Hand the finished tile out by rows: a lane of the accumulators holds 4
  // columns of 16 different rows, so they pass through LDS (fp32, at most
  // LDS_BYTES at a time) and every thread takes V consecutive columns at a
  // time, a wave whole rows: 16-byte loads and stores of whole lines.
  // (Straight from the accumulators, 32 bytes of a row per store, a
  // 256 x 256 tile took 73 us to write.)
  // pre(row, col) loads what f needs, for U groups at once, before any of
  // them is stored; f(row, col, v, w, x) gets the V values (w: of the paired
  // product) and pre's result.  Rows and columns count from the tile's corner.
  // 16-byte chunk c of a row sits at chunk c ^ (row & 15): the 16 rows of a
  // write and the neighbouring chunks of a read fall on different banks.
  // fold: row r + fold is added to row r (tiles of one phase; Problem::fold).
  template <int V, int U, class PRE, class F>
  __device__ __forceinline__ void hand_out(char* smem, uint32_t fold, PRE&& pre, F&& f) {
    constexpr int PHASES = (BM * BN * 4 * WK + LDS_BYTES - 1) / LDS_BYTES;
    constexpr int PART = TM / PHASES;  // blocks of a wave per phase
    constexpr int ROWS = PART * 16 * WM, UNITS = ROWS * (COLS / V), ROUNDS = (UNITS + NT * U - 1) / (NT * U);
    constexpr int SWZ = BN / 4 < 16 ? BN / 4 - 1 : 15;
    static_assert(TM % PHASES == 0 && (PHASES == 1 || WK == 1), "");
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t wk = WK == 1 ? 0 : threadIdx.x / GROUP;
    float4* t = (float4*)smem;
#pragma unroll
    for (int ph = 0; ph < PHASES; ++ph) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < PART; ++i) {
        const uint32_t r = (uint32_t)(wave_row() / (16 * TM) * (16 * PART) + 16 * i) + (lane & 15);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const v4f v = acc[ph * PART + i][j];
          const uint32_t chunk = (uint32_t)block_row(j) / 4 + (lane >> 4);
          t[(wk * ROWS + r) * (BN / 4) + (chunk ^ (r & SWZ))] = make_float4(v[0], v[1], v[2], v[3]);
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int round = 0; round < ROUNDS; ++round) {
        decltype(pre(0u, 0u)) x[U];
        uint32_t row[U], col[U], at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t unit = (uint32_t)((round * U + u) * NT) + threadIdx.x;
          const uint32_t r = unit / (COLS / V);
          at[u] = r;
          col[u] = unit % (COLS / V) * V;
          row[u] = r / (16 * PART) * (16 * TM) + ph * PART * 16 + r % (16 * PART);
          if (UNITS % (NT * U) == 0 || unit < (uint32_t)UNITS) x[u] = pre(row[u], col[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (UNITS % (NT * U) != 0 && at[u] >= (uint32_t)ROWS) continue;
          float v[V], w[V];
#pragma unroll
          for (int q = 0; q < V / 4; ++q) {
            const uint32_t chunk = col[u] / 4 + q, s = at[u] & SWZ;
            // the parts of K, added in order
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll
            for (int z = 0; z < WK; ++z) {
              const float4 y = t[(z * ROWS + at[u]) * (BN / 4) + (chunk ^ s)];
              a.x += y.x, a.y += y.y, a.z += y.z, a.w += y.w;
            }
            if (PHASES == 1 && !PAIR && fold) {
              const uint32_t r = (at[u] + fold) % ROWS;  // (rows from fold on are not wanted)
#pragma unroll
              for (int z = 0; z < WK; ++z) {
                const float4 y = t[(z * ROWS + r) * (BN / 4) + (chunk ^ (r & SWZ))];
                b.x += y.x, b.y += y.y, b.z += y.z, b.w += y.w;
              }
              a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
            }
            v[4 * q] = a.x, v[4 * q + 1] = a.y, v[4 * q + 2] = a.z, v[4 * q + 3] = a.w;
            if constexpr (PAIR) {
#pragma unroll
              for (int z = 0; z < WK; ++z) {
                const float4 y = t[(z * ROWS + at[u]) * (BN / 4) + ((chunk + BN / 8) ^ s)];
                b.x += y.x, b.y += y.y, b.z += y.z, b.w += y.w;
              }
              w[4 * q] = b.x, w[4 * q + 1] = b.y, w[4 * q + 2] = b.z, w[4 * q + 3] = b.w;
            }
          }
          f(row[u], col[u], v, w, x[u]);
        }
      }
    }
  }
};

// Store V consecutive values of a row as DT: columns col .. col + V of a row
// with n.  `vec`: the row's storage allows 16-byte (V * esize) stores.
// STREAM: non-temporal, for what this call reads no more, or not before as much
// again has been written (a feed-forward step [8192, 5120] x 8 x 1728: g and u
// stored so 2590 -> 2500 us, out 1160 -> 1115; d of a loss of 4096 x 131072
// 5600 -> 5400).
template <int DT, int V, bool STREAM = false>
__device__ __forceinline__ void store_row(char* row, uint64_t col, uint32_t n, bool vec, const float* v) {
  constexpr int ES = KElem<DT>::ES;
  static_assert(DT != DT_BF16 || V == 8, "a 16-byte store");
  char* p = row + col * ES;
  if (vec && col + V <= n) {
    if constexpr (DT == DT_BF16) {
      uint32_t h[V / 2];
#pragma unroll
      for (int e = 0; e < V / 2; ++e) h[e] = bf16_round(v[2 * e]) | (bf16_round(v[2 * e + 1]) << 16);
      const v4u x = {h[0], h[1], h[2], h[3]};
      if constexpr (STREAM) __builtin_nontemporal_store(x, (v4u*)p);
      else *(v4u*)p = x;
    } else {
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        const v4f x = {v[e], v[e + 1], v[e + 2], v[e + 3]};
        if constexpr (STREAM) __builtin_nontemporal_store(x, (v4f*)(p + e * 4));
        else *(v4f*)(p + e * 4) = x;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (col + e >= n) break;
      if constexpr (DT == DT_BF16) *(uint16_t*)(p + e * 2) = (uint16_t)bf16_round(v[e]);
      else *(float*)(p + e * 4) = v[e];
    }
  }
}

// The same in two terms: v rounded at `row`, the rest at `low` (if there is one).
template <int DT, int V, bool STREAM = false>
__device__ __forceinline__ void store_terms(char* row, char* low, uint64_t col, uint32_t n, bool vec, const float* v) {
  store_row<DT, V, STREAM>(row, col, n, vec, v);
  if (DT == DT_BF16 && low) {
    float rest[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float top = __uint_as_float(bf16_round(v[e]) << 16);
      rest[e] = fabsf(top) < INFINITY ? v[e] - top : 0.f;  // nothing to add to an infinity or a NaN
    }
    store_row<DT, V>(low, col, n, vec, rest);
  }
}

// V consecutive fp32 values of a row (0 beyond n).
template <int V>
struct Floats {
  float v[V];
};
template <int V>
__device__ __forceinline__ Floats<V> load_floats(const char* row, uint64_t col, uint32_t n, bool vec) {
  Floats<V> r;
  const float* p = (const float*)row + col;
  if (vec && col + V <= n) {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      const float4 x = *(const float4*)(p + e);
      r.v[e] = x.x, r.v[e + 1] = x.y, r.v[e + 2] = x.z, r.v[e + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) r.v[e] = col + e < n ? p[e] : 0.f;
  }
  return r;
}

// Find this workgroup's problem, tile and share of its K.  Returns the problem's
// index.
template <class P>
__device__ __forceinline__ int locate(const ProductArgs& a, uint32_t* row0, uint32_t* col0, uint32_t* share) {
  const uint32_t b = blockIdx.x;
  const uint32_t t = b < a.head ? tile_of_block(b, a.head) : a.head + tile_of_block(b - a.head, a.tiles - a.head);
  int q = 0;
  while (q + 1 < a.nprob && t >= a.p[q + 1].first) ++q;
  uint32_t tm, tn;
  const uint32_t at = t - a.p[q].first;
  *share = at % a.p[q].shares;
  tile_coords(at / a.p[q].shares, a.p[q].tiles_m, a.p[q].tiles_n, &tm, &tn);
  *row0 = tm * P::BM;
  *col0 = tn * P::COLS;
  return q;
}

// ------------------------------------------------------------ host side

// Collects the problems of a launch.
struct ProductPlan {
  ProductArgs a;
  uint64_t tiles = 0;
  // Room for shares: c[2] of the head problems (all of them, where head is 0)
  // holds MAX_SHARES blocks.
  bool may_share = false;
  // Order of the sums over K: 0 any; 1 one wave, 4 quarters added up.  Values
  // that are computed twice are the same bits twice in the same order.
  uint32_t k_parts = 0;
  // Problems before this one go first, spread over the XCDs by themselves:
  // where two sorts of tiles differ in length, the long ones start and the
  // short ones fill the end of the launch.
  int head = 0;

  ProductPlan() { memset(&a, 0, sizeof(a)); }

  // Problems whose K may be shared: the first ones.
  int sharing() const { return !may_share ? 0 : head ? head : a.nprob; }

  // Rows of both operands start on 16-byte boundaries (Packer).
  Problem* add(uint64_t m, uint64_t n, uint64_t k, uint64_t lda, uint64_t ldb, uint64_t ldc) {
    Problem* p = &a.p[a.nprob++];
    p->m = (uint32_t)m, p->n = (uint32_t)n, p->k = (uint32_t)k;
    p->lda = (uint32_t)lda, p->ldb = (uint32_t)ldb, p->ldc = (uint32_t)ldc;
    p->nseg = 1;
    p->shares = 1;
    return p;
  }
  // Tiles of every problem for a kernel whose tile covers bm x cols of C.
  bool cut(uint32_t bm, uint32_t cols) {
    tiles = 0;
    a.head = 0;
    for (int i = 0; i < a.nprob; ++i) {
      Problem& p = a.p[i];
      p.tiles_m = (uint32_t)(((uint64_t)p.m + bm - 1) / bm);
      p.tiles_n = (uint32_t)(((uint64_t)p.n + cols - 1) / cols);
      p.first = (uint32_t)tiles;
      if (i == head) a.head = (uint32_t)tiles;
      tiles += (uint64_t)p.tiles_m * p.tiles_n * p.shares;
    }
    a.tiles = (uint32_t)tiles;
    return tiles < (1ull << 31);
  }
};

}  // namespace ar
