// Attention of a chunk of new tokens over the paged cache: for every layer,
// token row n of sequence b (position pos = cached[b] + n - cu_q[b], its own
// row already in the cache) and query head, the members of row pos of the
// forward ("Depth-Staggered Fibonacci Spacing for Sparse Attention",
// Methodology: attended set, scaling, interpolation):
//   window rows pos-W+1 .. pos, sinks j < S with j <= pos, and per offset f
//   (1-w) row[pos-lo] + w row[pos-lo-1],  d = alpha f, lo = floor(d), w = d-lo,
//   while pos - ceil(d) >= 0;
//   s = scale q . k (+ beta on the offset members);  o = softmax(s) v.
// Keys are rotated in the cache and the queries by cache_append.
//
// 16-bit queries (k_chunk_tc): products on the tensor cores by mma.sync
// m16n8k16, one warp per block of 8 columns. A column is a (token, query head)
// pair that shares one key/value head: with G heads per key/value head a block
// holds 8/G consecutive tokens. Scores are S^T = K q^T (M = 16 gathered rows,
// N = 8 columns) and outputs O^T = V^T P^T (M = 16 head dims, N = 8 columns), so
// that eight columns, not sixteen, have to be filled.
//   - Gathered rows come in stages of 32 (36) by 16-byte asynchronous copies past the
//     L1 into the warp's own shared memory, two stages in flight, and become fragments
//     by ldmatrix (transposed for V). Rows that went from global memory into registers
//     directly took 10 % more: they need the registers that hide the latency.
//     Nothing waits but a warp for its own copies. tcgen05 has no form for the
//     gather: its A operand is a tile of 128 rows, of which a token's 15
//     interpolated pairs would fill a quarter.
//   - Window and sinks: tiles of 16 rows shared by all columns, masked, with a
//     running maximum and sum per column.
//   - Offsets, interpolated (KIND 0): for each token tiles of 8 offsets, row a of
//     offset g in row g of the tile and row b in row g + 8, so that one lane holds
//     both products and interpolates in registers. Only the token's own columns
//     of such a tile count; over the block's tokens a lane keeps its own.
//   - One query head per key head (KIND 3): 8 tokens in a row read 9 rows of an
//     offset, not 16, so a stage holds 4 offsets x 9 rows and serves 4 tiles of two
//     tokens each (16384 tokens, 16 heads of 64, window 12: 182 -> 170 us).
//   - Integer distances in the whole layer (KIND 1, 2): no row b. 16 offsets in a
//     tile of one token, or 8 of two; an offset inside the window is a window row a
//     second time and costs nothing but a larger score (16384 tokens behind 16384, 16
//     heads of 64: 164 -> 144 us at window 64; at 1024 the look at each score costs
//     more than the few tiles, 713 -> 770).
//   - Few blocks (one token each, a long window): the warps of up to eight CTAs share a
//     block's window, one of them takes the offsets, and the parts (o, m, l) meet in
//     shared memory, across CTAs through the cluster's.
// Bound: issue, and the latency of dependent instructions that five warps a scheduler
// leave: 3110 instructions per warp of 8 tokens at window 64, 56 % of the issue slots
// (interpolated at window 12: 3380, 59 %; the L1's data path 46 and 64 %, the tensor
// pipe 16 and 29 %).
// Rounding: products of 16-bit values are exact, sums fp32. The probabilities go into
// P V as sums of two bf16 values, off by 2^-16 of themselves at most. One alone cost the
// output a quarter more error than its own rounding (16384 tokens, 16 heads of 64,
// window 64: 2.06e-3 of its 2-norm against 1.66e-3 with both, which is what fp32
// probabilities give); the second product on the same fragments took 136 -> 144 us
// there, and a mixed batch over e4m3 rows of 128 from 110 to 113. e4m3 codes are
// exact in fp16, and so are the queries beside them after scaling by a power of two;
// there probabilities times row scales are sums of two fp16 values (2^-22), relative
// to the largest of the column.
// A masked probability is 0, and 0 * Inf or NaN is NaN: a block with a non-finite
// output is computed again query by query (one_query), from its members alone.
//
// 32-bit queries (k_chunk_f32, one_query): one warp per token and up to 4 query heads of
// a key/value head on the CUDA cores, chunks of 32 members: four lanes per member for
// the scores, lanes over head dims for the values. 4096 tokens, 16 heads of 64, window
// 12: 180 us; two groups of 8 of them: 176 us head by head, 91 in fours. Bound: the L1,
// whose data path is busy 76 % of the time (1800 instructions per token and head, 56 %
// of the issue slots): tokens share no rows, so each loads its 42 again.
#pragma once

#include <type_traits>

#include "sa_paged.cuh"

namespace sa {

struct ChunkArgs {
  int L, N, B, Hq, Hkv, n_pages, max_pages, W, n_off, S, blocks;
  int G, groups, per, shift;      // heads per kv head; column groups, heads in one, log2 tokens
  int team;                       // CTAs whose warps share a block; 0: a block per warp
  int inv_per;                    // ceil(256 / per): col * inv_per / 256 = col / per for col < 8
  FastDiv pd;
  float scale;
  int f[SA_MAX_OFFSETS];
  int64_t ql, qn, qh;
  const void* q; const void* kc; const void* vc; const float* ks; const float* vs;
  const float* alpha; const float* beta;
  const int* table; const int* cu; const int* cached;
  void* o; float* lse;
};

// One head dim per translation unit (sa_chunk_<D>.cu): the instances compile side by side.
template <int D>
cudaError_t launch_chunk_of(const ChunkArgs& a, bool f32, bool e4m3, cudaStream_t st);
template <int D>
cudaError_t chunk_error_of(unsigned* out, bool clear);

#ifdef SA_CHUNK_KERNELS
namespace {

__device__ unsigned g_chunk_err;

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One m16n8k16 product with fp32 sums, of bf16 (plain rows) or fp16 (e4m3 rows,
// whose codes are exact in fp16) operands.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16x2(lo, hi);
  }
}
// A pair as a sum of two 16-bit pairs: the rounded values and what that leaves, rounded.
template <bool F16>
__device__ __forceinline__ void split16(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack16<F16>(a, b);
  if constexpr (F16) {
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    lo = pack16<true>(a - h.x, b - h.y);
  } else {
    lo = pack16<false>(a - bf16lo(hi), b - bf16hi(hi));
  }
}

// Transpose of an 8x8 matrix of 16-bit values (lane (g, c) holds row g, columns
// 2c and 2c+1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int BYTES>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (BYTES == 16) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else if constexpr (BYTES == 8) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = u.x; w[1] = u.y;
  } else if constexpr (BYTES == 4) {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else {
    static_assert(BYTES == 2, "unsupported width");
    w[0] = __ldg(reinterpret_cast<const unsigned short*>(p));
  }
}

// Four e4m3 codes as two pairs of fp16 values: exact, NaN kept.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; "
      "cvt.rn.f16x2.e4m3x2 %1, b; }"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

// Past the L1: its data path is half of what the kernel waits for, and a row that passes
// through it crosses it twice (16384 tokens, 16 heads of 64: window 64 162 -> 144 us,
// interpolated, window 12 198 -> 170; 8 heads of 128: 198 -> 160).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
template <bool TRANS, int OFFSET>
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4 + %5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(OFFSET)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4 + %5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(OFFSET)
                 : "memory");
}
// Clusters of CTAs: this one's rank, a barrier, the address of what p is in the CTA of
// rank r, and a load from there.
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile(
      "barrier.cluster.arrive.release;\n\t"
      "barrier.cluster.wait.acquire;" ::: "memory");
  __syncwarp();
}
__device__ __forceinline__ uint32_t cluster_address(const void* p, int r) {
  uint32_t there;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(there)
      : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(r));
  return there;
}
__device__ __forceinline__ float load_cluster(uint32_t addr) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ float load_shared(uint32_t addr) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
  return x;
}

// P^T of a tile, rounded and what that leaves: p[0], p[1] for rows 0..7 and 8..15.
struct Weights {
  uint32_t hi[2], lo[2];
};

// A stage: 32 gathered rows (two tiles of 16) of K or V, in 16-byte chunks whose
// place is exchanged by row (so that eight rows of one chunk column, an ldmatrix
// phase, fall into different banks), and for e4m3 rows their scales.
template <int D, bool E4M3>
struct Stage {
  static constexpr int kRow = D * (E4M3 ? 1 : 2);       // bytes
  static constexpr int kChunks = kRow / 16;
  static constexpr int kTile = 16 * kRow;
  static constexpr int kRows = 36;                      // 32, and 4 more of shared stages
  static constexpr int kScales = kRows * kRow;          // the rows' key scales, then the values'
  static constexpr int kValues = kRows * 4;
  static constexpr int kBytes = kRows * kRow + (E4M3 ? 2 * kValues : 0);
  static __device__ __forceinline__ int place(int row, int chunk) {
    constexpr int kPer = kChunks >= 8 ? 1 : 8 / kChunks;
    constexpr int kMask = kChunks >= 8 ? 7 : kChunks - 1;
    return row * kRow + ((chunk ^ ((row / kPer) & kMask)) << 4);
  }
  // Copies the rows that the lanes name (pool rows; lane = row of the stage). Of
  // its place a lane keeps the part that does not depend on the pass (own = place
  // of its chunk in pass 0); `pool` points at its chunk of row 0.
  static __device__ __forceinline__ const uint8_t* row_at(const uint8_t* pool, int row) {
    const uint8_t* p;      // one instruction; as C++ it becomes two or three
    asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(p) : "r"(row), "n"(kRow), "l"(pool));
    return p;
  }
  static __device__ __forceinline__ int own() {
    const int lane = threadIdx.x & 31;
    return place(lane / kChunks, lane % kChunks);
  }
  static __device__ __forceinline__ void fill(uint32_t stage, int own, const uint8_t* pool,
                                              int row, bool two) {
    constexpr int kRows = 32 / kChunks;      // rows of a pass
    const int r0 = (threadIdx.x & 31) / kChunks;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if (i == kChunks / 2 && kChunks > 1 && !two) break;
      constexpr int kMask = kChunks >= 8 ? 7 : 0;      // passes of fewer than 8 rows
      const int turn = ((i * kRows) & kMask) << 4;
      const int r = __shfl_sync(0xffffffffu, row, i * kRows + r0);
      copy16(stage + (own ^ turn) + i * kRows * kRow, row_at(pool, r));
    }
  }
  // A shared stage: for 4 offsets o the 9 rows r that 8 consecutive tokens read (token
  // t rows t + 1 and t), row r of offset o at 9 o + r. A tile is two tokens of the four
  // offsets: as fragments see it rows r and r + 1 of each, so the exchange of chunks
  // goes by r % 2 + 2 o, and is the same for all tiles.
  static __device__ __forceinline__ int turn(int r, int o) {
    constexpr int kDown = kChunks >= 8 ? 0 : (kChunks == 4 ? 1 : (kChunks == 2 ? 2 : 3));
    return (((r & 1) ^ (2 * o)) >> kDown) << 4;
  }
  static __device__ __forceinline__ int shared_row(int o, int r) { return 9 * o + r; }
  static __device__ __forceinline__ int own_shared() {
    const int lane = threadIdx.x & 31, row = lane / kChunks;
    return shared_row(row >> 3, row & 7) * kRow +
           (((lane % kChunks) << 4) ^ turn(row, row >> 3));
  }
  // row: lane 8 o + r's row r of offset o; row8: lane o's row 8
  static __device__ __forceinline__ void fill_shared(uint32_t stage, int own, const uint8_t* pool,
                                                     int row, int row8) {
    constexpr int kPass = 32 / kChunks;      // rows of a pass
    const int r0 = (threadIdx.x & 31) / kChunks;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int at = i * kPass;              // its first row
      const int r = __shfl_sync(0xffffffffu, row, at + r0);
      copy16(stage + (own ^ turn(at, at >> 3)) + shared_row(at >> 3, at & 7) * kRow,
             row_at(pool, r));
    }
#pragma unroll
    for (int i = 0; i < (kPass >= 4 ? 1 : 4 / kPass); ++i) {
      const int fo = i * kPass + r0;
      const int r = __shfl_sync(0xffffffffu, row8, fo & 3);
      if (fo < 4)
        copy16(stage + shared_row(fo, 8) * kRow +
                   ((((threadIdx.x & 31) % kChunks) << 4) ^ turn(8, fo)),
               row_at(pool, r));
    }
  }
  // Lane offset of an ldmatrix of K or V of the tile of tokens 0 and 1; the tile of
  // tokens 2 j and 2 j + 1 is 2 j rows further.
  static __device__ __forceinline__ uint32_t shared_at(bool v) {
    const int lane = threadIdx.x & 31, mi = lane >> 3;
    const int half = v ? mi >> 1 : mi & 1, chunk = v ? mi & 1 : mi >> 1;
    const int fo = lane & 3, r = ((lane >> 2) & 1) + (half == 0);
    return shared_row(fo, r) * kRow + (((kChunks > 1 ? chunk : 0) << 4) ^ turn(r, fo));
  }
  // Lane offset of an ldmatrix of K (matrices: row halves, then chunks) or V
  // (chunks, then row halves); step s of the loop over chunk pairs is at ^ (s << 5).
  static __device__ __forceinline__ uint32_t lane_at(bool v) {
    const int lane = threadIdx.x & 31, mi = lane >> 3;
    const int half = v ? mi >> 1 : mi & 1, chunk = v ? mi & 1 : mi >> 1;
    return place((lane & 7) + 8 * half, kChunks > 1 ? chunk : 0);
  }
  // S^T of N tiles' 16 keys each, STEP bytes from one to the next, with the block's 8
  // columns: the tiles in turn, so that a product does not wait for the one before.
  template <int N, int STEP>
  static __device__ __forceinline__ void scores(uint32_t stage, uint32_t at,
                                                const uint32_t (&q)[D / 8], float (&s)[N][4]) {
#pragma unroll
    for (int t = 0; t < N; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
    constexpr int kPairs = (kChunks + 1) / 2;      // chunk pairs: 16 elements, 32 codes
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      uint32_t r[N][4];
      const uint32_t from = stage + (at ^ (i << 5));
      ldmatrix4<false, 0>(from, r[0]);
      if constexpr (N > 1) ldmatrix4<false, STEP>(from, r[1]);
      if constexpr (N > 2) ldmatrix4<false, 2 * STEP>(from, r[2]);
      if constexpr (N > 3) ldmatrix4<false, 3 * STEP>(from, r[3]);
      if constexpr (!E4M3) {
#pragma unroll
        for (int t = 0; t < N; ++t)
          mma16816<false>(s[t], r[t][0], r[t][1], r[t][2], r[t][3], q[2 * i], q[2 * i + 1]);
      } else {
#pragma unroll
        for (int j = 0; j < (kChunks > 1 ? 2 : 1); ++j)
#pragma unroll
          for (int t = 0; t < N; ++t) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x4(r[t][2 * j], a0, a2);
            e4m3x4_to_f16x4(r[t][2 * j + 1], a1, a3);
            mma16816<true>(s[t], a0, a1, a2, a3, q[4 * i + 2 * j], q[4 * i + 2 * j + 1]);
          }
      }
    }
  }
  // O^T += V^T P^T of a tile's 16 values.
  // Lane g's head dims of product j: 16 j + g and 16 j + 8 + g, for e4m3 rows
  // 16 j + 2 g and the next.
  template <int OFFSET>
  static __device__ __forceinline__ void add(uint32_t stage, uint32_t at, const Weights& p,
                                             float (&o)[D / 16][4]) {
    if constexpr (!E4M3) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t r[4];
        ldmatrix4<true, OFFSET>(stage + (at ^ (j << 5)), r);
        mma16816<false>(o[j], r[0], r[1], r[2], r[3], p.lo[0], p.lo[1]);
        mma16816<false>(o[j], r[0], r[1], r[2], r[3], p.hi[0], p.hi[1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < (kChunks + 1) / 2; ++i) {
        uint32_t r[4];
        ldmatrix4<true, OFFSET>(stage + (at ^ (i << 5)), r);
#pragma unroll
        for (int j = 0; j < (kChunks > 1 ? 2 : 1); ++j) {
          // two rows of a pair of codes to two pairs of rows of a code
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x4(__byte_perm(r[j], 0, 0x3120), a0, a1);
          e4m3x4_to_f16x4(__byte_perm(r[2 + j], 0, 0x3120), a2, a3);
          mma16816<true>(o[2 * i + j], a0, a1, a2, a3, p.lo[0], p.lo[1]);
          mma16816<true>(o[2 * i + j], a0, a1, a2, a3, p.hi[0], p.hi[1]);
        }
      }
    }
  }
  // add() of tile `tile` (a constant after unrolling), STEP bytes from one to the next.
  template <int STEP>
  static __device__ __forceinline__ void add_of(int tile, uint32_t stage, uint32_t at,
                                                const Weights& p, float (&o)[D / 16][4]) {
    if (tile == 0) add<0>(stage, at, p, o);
    if (tile == 1) add<STEP>(stage, at, p, o);
    if (tile == 2) add<2 * STEP>(stage, at, p, o);
    if (tile == 3) add<3 * STEP>(stage, at, p, o);
  }
};

template <typename QT, int D, bool E4M3>
__device__ __noinline__ void one_query(const ChunkArgs& a, int layer, int hq, int n, int b,
                                       int pos, bool inside);

// Bytes of a stage, and of a warp's shared memory: two stages, and (shared stages of
// interpolated distances) a score per lane of each. Plain rows of 128 without shared
// stages take 32 rows, which leaves the L1 24 KB more (16384 tokens, 32 heads over 4:
// 262 -> 249 us).
template <int D, bool E4M3>
__host__ __device__ __forceinline__ constexpr int stage_bytes(bool shared) {
  return !E4M3 && D == 128 && !shared ? 32 * Stage<D, E4M3>::kRow : Stage<D, E4M3>::kBytes;
}
template <int D, bool E4M3, int NT, bool TEAM>
__host__ __device__ __forceinline__ constexpr int warp_bytes(bool shared) {
  return 2 * stage_bytes<D, E4M3>(shared) + (!TEAM && shared ? NT * 4 * 32 * 4 : 0);
}

// A lane's walk over the pool rows that one member has for consecutive tokens:
// mostly the next row of the same page.
struct Walk {
  int row = 0, left = -1;      // the last row, and how many follow it in its page
};

// ---------------------------------------------------------------------------
// NT: pairs of offset tiles (16 offsets each), 0 .. 2. TEAM: the warps of a cluster of
// a.team CTAs share one block (an instance of its own: the shares cost the others 4 %).
// CTAs per SM, and with them the registers (96 a thread for five): more warps hide more
// of the latency until the spills cost as much. 16384 tokens, plain rows: 16 heads of 64,
// window 64 149 us with four, 144 with five, 178 with six; 32 heads of 128 over 4 261
// with four, 249 with three; 16 heads of 16 112 with five, 108 with six, 121 with eight.
// e4m3 rows of 128: 253 with three, 224 with four, 284 with five. Of teams there are at
// most four per SM (one token, 16 heads of 64, window 4096 by one CTA: 55 us with
// registers for five, 46 for four).
template <int D, bool E4M3, bool TEAM>
__host__ __device__ __forceinline__ constexpr int chunk_ctas() {
  return D == 128 ? (E4M3 ? 4 : 3) : TEAM ? 4 : D == 64 ? 5 : 6;
}
template <int D, bool E4M3, int NT, bool TEAM>
__global__ void __launch_bounds__(kWarps * 32, chunk_ctas<D, E4M3, TEAM>())
    k_chunk_tc(const __grid_constant__ ChunkArgs a) {
  using Y = Stage<D, E4M3>;
  extern __shared__ __align__(1024) uint8_t s_stages[];
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int warp = threadIdx.x >> 5;
  const int x = TEAM ? blockIdx.x / a.team : blockIdx.x * kWarps + warp;
  if (x >= a.blocks) return;
  const int h = blockIdx.y / a.groups, grp = blockIdx.y % a.groups, layer = blockIdx.z;

  // this block's tokens: rows n0 .. n0 + count - 1, positions from pos0
  const int b = find_sequence(a.cu, a.B, a.shift, x);
  const int first = __ldg(a.cu + b), past = min(__ldg(a.cu + b + 1), a.N);
  const long long n0l = (long long)first + ((long long)(x - (first >> a.shift) -
                                                        (a.shift ? b : 0)) << a.shift);
  if (first < 0 || n0l < first || n0l >= past) return;
  const int n0 = (int)n0l, count = min(1 << a.shift, past - n0);
  const long long posl = (long long)__ldg(a.cached + b) + (n0 - first);
  const bool inside = posl >= 0 && posl + count <= (long long)a.max_pages * a.pd.d;
  const int pos0 = inside ? (int)posl : 0;

  // offset geometry: lane k holds offset k
  int off_lo = 0, off_c = 0x7fffffff;
  float off_w = 0.f;
  bool ok = inside;
  if (NT > 0 && lane < a.n_off) {
    const OffGeo og = offset_geometry(__ldg(a.alpha + layer), a.f[lane]);
    off_lo = og.lo; off_c = og.c; off_w = og.w;
    ok = ok && og.ok;
  }
  ok = __all_sync(0xffffffffu, ok);
  const int* table = a.table + (size_t)b * a.max_pages;
  const size_t pool = (size_t)layer * a.n_pages * a.Hkv * a.pd.d;
  const size_t chunk = pool * Y::kRow + (lane % Y::kChunks) * 16;      // this lane's, of row 0
  const uint8_t* kb = reinterpret_cast<const uint8_t*>(a.kc) + chunk;
  const uint8_t* vb = reinterpret_cast<const uint8_t*>(a.vc) + chunk;
  const float* ks = E4M3 ? a.ks + pool : nullptr;
  const float* vs = E4M3 ? a.vs + pool : nullptr;
  bool lost = !inside;      // a position or page outside its range

  // column 2c + e of this lane: token tok[e] of the block, query head sub[e] of the
  // group, position qpos[e]
  const int heads = min(a.per, a.G - grp * a.per), head0 = h * a.G + grp * a.per;
  auto token_of = [&](int col) { return col * a.inv_per >> 8; };      // col / per, col < 8
  int tok[2], sub[2], qpos[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    tok[e] = token_of(2 * c + e);
    sub[e] = 2 * c + e - tok[e] * a.per;
    if (sub[e] >= heads || tok[e] >= count) tok[e] = -1;
    qpos[e] = tok[e] < 0 ? -(1 << 30) : pos0 + tok[e];
  }

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[D / 16][4];
#pragma unroll
  for (int j = 0; j < D / 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  const bool shares = a.shift == 3;      // 8 tokens of one head
  uint8_t* const own_smem = s_stages + warp * warp_bytes<D, E4M3, NT, TEAM>(shares);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(own_smem);
  const int hrow = h * a.pd.d, page_rows = a.Hkv * a.pd.d;
  // a team member's share: the last one has the offsets, the others every window_by-th
  // pair of window tiles from the window_at-th on (0: none)
  const int members = TEAM ? kWarps * a.team : 1, rank = TEAM ? cluster_rank() : 0;
  const int member = TEAM ? rank * kWarps + warp : 0;
  const bool offsets = member == members - 1;
  const int window_by = !TEAM ? 1 : NT == 0 ? members : offsets ? 0 : members - 1;
  const int window_at = TEAM && window_by ? member : 0;
  int n_far = a.n_off;                   // offsets that have rows of their own
  unsigned near_lo = 0, near_hi = 0;     // distances 0..31 and 32..63 folded into the window

  auto run = [&](auto kind) {
    // 0: interpolated distances; integer ones: 1: 16 offsets a tile, 2: up to 8
    // offsets left besides the folded ones, two tokens a tile; 3: interpolated, 8
    // tokens of one head, which share each other's rows
    constexpr int KIND = decltype(kind)::value;
    constexpr bool FLAT = KIND == 1 || KIND == 2;
    constexpr int STEP = KIND == 2 ? 4 : KIND + 1;      // tokens of an offset stage
    auto find = [&](int r, int& left) {
      const int lp = quotient(a.pd, r), in = r - lp * a.pd.d;
      int page = __ldg(table + lp);
      if ((unsigned)page >= (unsigned)a.n_pages) {
        lost = true;
        page = 0;
      }
      left = a.pd.d - 1 - in;
      return page * page_rows + hrow + in;
    };
    // Rows without a member take this row, the first token's own, with weight 0.
    int unused;
    const int fill = find(pos0, unused);

    // ---- stages, in the order in which they are used: offset keys; window keys and
    // values in turn; offset values ----
    const int own = Y::own();
    uint32_t in = ring, out = ring;
    const uint32_t flip_by = stage_bytes<D, E4M3>(shares);
    auto stage_in = [&](const uint8_t* rows, int row, bool two, bool keys) {
      Y::fill(in, own, rows, row, two);
      if constexpr (E4M3) {
        if (keys) copy4(in + Y::kScales + lane * 4, ks + row);
        copy4(in + Y::kScales + Y::kValues + lane * 4, vs + row);
      }
      in = ring + flip_by - (in - ring);
    };
    auto take = [&]() {      // the next stage to use, complete and visible to the warp
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      const uint32_t s = out;
      out = ring + flip_by - (out - ring);
      return s;
    };
    auto commit = []() { asm volatile("cp.async.commit_group;" ::: "memory"); };

    // Offset stages. Interpolated: one per (token, tile pair); tile i of the pair
    // has, for 8 offsets, rows a in 0..7 and rows b in 8..15. Integer distances: a
    // tile holds 16 offsets of one token, or 8 of two.
    int lo_[NT > 0 ? NT : 1], c_[NT > 0 ? NT : 1];      // of the row this lane looks up
    const int ahead = KIND == 2 ? lane >> 3 : (KIND == 1 ? lane >> 4 : 0);      // for token t + ahead
#pragma unroll
    for (int pair = 0; pair < NT; ++pair) {
      const int src = pair * 16 + (KIND == 2   ? lane & 7
                                   : KIND == 1 ? lane & 15
                                               : (lane >> 4) * 8 + (lane & 7));
      const bool isb = !FLAT && (lane & 8);
      lo_[pair] = __shfl_sync(0xffffffffu, off_lo, src) + isb;
      c_[pair] = __shfl_sync(0xffffffffu, off_c, src);
      if (!FLAT && __shfl_sync(0xffffffffu, off_w, src) == 0.f && isb)
        c_[pair] = 0x7fffffff;      // no second row
    }
    Walk walk[NT > 0 ? NT : 1];
    int next_t = 0;      // token of the next offset stage
    auto offset_in = [&](int pair, bool keys) {
      const int mine = next_t + ahead, p = pos0 + mine;
      const bool there = c_[pair] <= p && mine < count;
      Walk& w = walk[pair];
      if (there) {
        w.row += STEP;
        w.left -= STEP;
        if (w.left < 0) w.row = find(p - lo_[pair], w.left);
      }
      stage_in(keys ? kb : vb, there ? w.row : fill,
               FLAT ? next_t + STEP / 2 < count : pair * 16 + 8 < a.n_off, keys);
      if (pair == NT - 1) next_t += STEP;
    };
    // Shared stage `st`: lane 8 o + r has row r of offset 4 st + o, at position pos0 -
    // lo - 1 + r: row a of token r - 1 and row b of token r.
    const int own_shared = KIND == 3 ? Y::own_shared() : 0;
    int next_st = 0;
    auto shared_in = [&](bool keys) {
      const int src = next_st * 4 + (lane >> 3), r = lane & 7;
      const int lo = __shfl_sync(0xffffffffu, off_lo, src);
      const int cc = __shfl_sync(0xffffffffu, off_c, src);
      const float w = __shfl_sync(0xffffffffu, off_w, src);
      const int p = pos0 + r;
      const bool there = (r > 0 && r <= count && cc <= p - 1) || (w != 0.f && r < count && cc <= p);
      const int row = find(there ? p - lo - 1 : pos0, unused);
      const int lo8 = __shfl_sync(0xffffffffu, off_lo, next_st * 4 + (lane & 3));
      const int c8 = __shfl_sync(0xffffffffu, off_c, next_st * 4 + (lane & 3));
      const int row8 = find(count == 8 && c8 <= pos0 + 7 ? pos0 + 7 - lo8 : pos0, unused);
      Y::fill_shared(in, own_shared, keys ? kb : vb, row, row8);
      if constexpr (E4M3) {
        const uint32_t at = in + Y::kScales + Y::shared_row(lane >> 3, lane & 7) * 4;
        const uint32_t at8 = in + Y::kScales + Y::shared_row(lane & 3, 8) * 4;
        if (keys) {
          copy4(at, ks + row);
          if (lane < 4) copy4(at8, ks + row8);
        }
        copy4(at + Y::kValues, vs + row);
        if (lane < 4) copy4(at8 + Y::kValues, vs + row8);
      }
      in = ring + flip_by - (in - ring);
      ++next_st;
    };
    auto restart = [&]() {      // the values go over the same tokens again
      next_t = next_st = 0;
#pragma unroll
      for (int pair = 0; pair < NT; ++pair) walk[pair] = Walk();
    };
    auto rows_in = [&](int pair, bool keys) {
      if constexpr (KIND == 3)
        shared_in(keys);
      else
        offset_in(pair, keys);
    };
    const int n_off = KIND == 3 ? (a.n_off + 3) / 4
                      : (KIND == 2 && n_far == 0) || !offsets ? 0 : NT * ((count + STEP - 1) / STEP);

    // Window tiles of 16 rows from `base`, the sinks as tile -1 before them.
    const int last = pos0 + count - 1;
    const int base = max(0, pos0 - (a.W - 1));
    const int t_first = (a.S > 0 ? -1 : 0) + 2 * window_at, t_step = 2 * window_by;
    const int t_past = !TEAM || window_by ? (last - base) / 16 + 1 : t_first;
    int win_row = 0, win_t = t_first;      // rows and first tile of the last key stage
    auto window_in = [&](int t0, bool keys) {
      if (keys) {
        const int t = t0 + (lane >> 4);      // this lane's tile
        const int r = (t < 0 ? 0 : base + t * 16) + (lane & 15);
        const bool there = r <= last && (t >= 0 || r < a.S);
        win_row = find(there ? r : pos0, unused);
        win_t = t0;
      }
      stage_in(keys ? kb : vb, win_row, win_t + 1 < t_past, keys);
    };
    // stage k of the whole order for k = 0 and 1, and from then on two ahead
    // (a team's member may have no offsets, or no window)
    const int n_win = t_first < t_past ? 2 : 0;      // its first key and value stage
    auto after_keys = [&](int k) {      // stage k >= n_off, for k up to n_off + 1
      if (k < n_off + n_win)
        window_in(t_first, k == n_off);
      else if (NT > 0 && k - n_win < 2 * n_off) {
        if (k - n_win == n_off) restart();
        rows_in(NT == 2 ? (k - n_win - n_off) & 1 : 0, false);
      }
    };
    auto issue = [&](int k) {      // stage k <= n_off + 1 (of tile pair k % NT)
      if (NT > 0 && k < n_off)
        rows_in(NT == 2 ? k & 1 : 0, true);
      else
        after_keys(k);
      commit();
    };
    issue(0);
    issue(1);

    // Query fragments of column g. For e4m3 rows in fp16, times a power of two that
    // brings the column's largest element to [2^14, 2^15): an element loses bits
    // only where it is 2^28 times smaller.
    uint32_t q[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) q[i] = 0u;
    {
      const int t = token_of(g), hh = g - t * a.per;
      if (hh < heads && t < count) {
        const uint8_t* qp = reinterpret_cast<const uint8_t*>(
            reinterpret_cast<const __nv_bfloat16*>(a.q) + layer * a.ql + (n0 + t) * a.qn +
            (head0 + hh) * a.qh);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          if constexpr (E4M3) {      // elements 16 i + 4 c ..
            load_words<8>(qp + i * 32 + c * 8, q + 2 * i);
          } else {                   // 16 i + 2 c .. and 8 further
            load_words<4>(qp + i * 32 + c * 4, q + 2 * i);
            load_words<4>(qp + i * 32 + 16 + c * 4, q + 2 * i + 1);
          }
        }
      }
    }
    float scale[2] = {a.scale * kLog2e, a.scale * kLog2e};      // of the lane's two columns
    if constexpr (E4M3) {
      __nv_bfloat162 top2 = __float2bfloat162_rn(0.f);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&q[i])));
      float top = fmaxf(__low2float(top2), __high2float(top2));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int e = (int)(__float_as_uint(top) >> 23) - 127;          // 2^e <= top < 2^(e+1)
      e = e < -100 || e > 127 ? 14 : e;                         // zeros, infinities: as they are
      const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
      const float down = __uint_as_float((uint32_t)(e - 14 + 127) << 23);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) q[i] = pack16<true>(bf16lo(q[i]) * up, bf16hi(q[i]) * up);
      scale[0] *= __shfl_sync(0xffffffffu, down, 8 * c);
      scale[1] *= __shfl_sync(0xffffffffu, down, 8 * c + 4);
    }
    const uint32_t at_k = Y::lane_at(false), at_v = Y::lane_at(true);
    // scales of the stage's rows i * 16 + half * 8 + g: keys 0, values 1
    auto row_scale = [&](uint32_t stage, int which, int i, int half) {
      return load_shared(stage + Y::kScales + which * Y::kValues + (i * 16 + half * 8 + g) * 4);
    };
    auto shared_scale = [&](uint32_t stage, int which, bool next) {      // of the lane's own token
      return load_shared(stage + Y::kScales + which * Y::kValues +
                         Y::shared_row(g & 3, 2 * c + (g >> 2) + next) * 4);
    };
    auto log_scale = [](float x) {      // 2^-100 at least; NaN does not matter here
      float y;
      asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(fabsf(x), 7.9e-31f)));
      return y;
    };

    // Running reference m and sum l of each of the lane's columns; o the outputs
    // times l. For e4m3 rows the reference is the maximum of score + log2(value
    // scale): the weights that go into P V, probability * value scale, are then at
    // most 1 and fit fp16 whatever the scales.
    constexpr int NS = NT > 0 && KIND < 2 ? 2 * NT : 1;
    float beta[2] = {0.f, 0.f};
    if (NT > 0 && a.beta) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (tok[e] >= 0)
          beta[e] = kLog2e * __ldg(a.beta + ((size_t)layer * a.N + n0 + tok[e]) * a.Hq + head0 +
                                   sub[e]);
    }
    // a folded offset is its window row a second time: log2(1 + 2^beta) more score
    [[maybe_unused]] float extra[2] = {0.f, 0.f};
    if (KIND == 2 && (near_lo | near_hi)) {
#pragma unroll
      for (int e = 0; e < 2; ++e)      // (from the larger of the two terms)
        extra[e] = fmaxf(beta[e], 0.f) + log2f(1.f + exp2f(-fabsf(beta[e])));
    }
    [[maybe_unused]] float sig[NS][2], wg[NS];      // scores, and weights of row b, of offset 8 i + g
    // KIND 3: a lane has offset g % 4 of each stage for one token, 2c + mine. The loops
    // stay loops (four of them unrolled did not fit the instruction cache), so the
    // scores wait in shared memory.
    [[maybe_unused]] float* const ps = reinterpret_cast<float*>(own_smem + 2 * flip_by) + lane;
    [[maybe_unused]] const int mine = g >> 2;
    if constexpr (KIND == 3) {
      // ---- offset scores, rows shared by the tokens ----
      const uint32_t at = Y::shared_at(false);
      const int at_pos = mine ? qpos[1] : qpos[0];
      const float at_scale = mine ? scale[1] : scale[0], at_beta = mine ? beta[1] : beta[0];
      float top = -INFINITY;
#pragma unroll 1
      for (int st = 0; st < n_off; ++st) {
        const uint32_t stage = take();
        const float w = __shfl_sync(0xffffffffu, off_w, st * 4 + (g & 3));
        const int cc = __shfl_sync(0xffffffffu, off_c, st * 4 + (g & 3));
        float wa = 1.f - w, wb = w, y = 0.f, vl = 0.f;
        if constexpr (E4M3) {
          wa *= shared_scale(stage, 0, true);
          wb *= shared_scale(stage, 0, false);
          vl = log_scale(shared_scale(stage, 1, true));
          if (w != 0.f) vl = fmaxf(vl, log_scale(shared_scale(stage, 1, false)));
        }
        float s[4][4];      // of tokens 2 j and 2 j + 1
        Y::template scores<4, 2 * Y::kRow>(stage, at, q, s);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c == j)
            y = mine ? fmaf(wb, s[j][3], wa * s[j][1]) : fmaf(wb, s[j][2], wa * s[j][0]);
        y = cc <= at_pos ? fmaf(y, at_scale, at_beta) : -INFINITY;
        ps[st * 32] = y;
        top = fmaxf(top, y + vl);
        __syncwarp();
        issue(st + 2);
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
      const float other = __shfl_xor_sync(0xffffffffu, top, 16);
      m[0] = mine ? other : top;
      m[1] = mine ? top : other;
    } else if constexpr (NT > 0) {
      // ---- offset scores: a lane keeps its own columns' ----
      float vl[NS][2];
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        wg[i] = FLAT ? 0.f : __shfl_sync(0xffffffffu, off_w, i * 8 + g);
        sig[i][0] = sig[i][1] = vl[i][0] = vl[i][1] = 0.f;
      }
      int k = 2;      // the stage after the next
#pragma unroll 1
      for (int t = 0; k < n_off + 2; t += STEP) {
#pragma unroll
        for (int pair = 0; pair < NT; ++pair, ++k) {
          const bool second = FLAT ? t + STEP / 2 < count : pair * 16 + 8 < a.n_off;
          const uint32_t stage = take();
          float both[2][4];      // (an absent second tile: not used)
          Y::template scores<2, Y::kTile>(stage, at_k, q, both);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i == 1 && !second) continue;
            const float(&s)[4] = both[i];
            float va = 0.f, vc = 0.f, ka = 1.f, kc = 1.f;
            if constexpr (E4M3) {
              ka = row_scale(stage, 0, i, 0);
              kc = row_scale(stage, 0, i, 1);
              va = log_scale(row_scale(stage, 1, i, 0));
              vc = log_scale(row_scale(stage, 1, i, 1));
            }
            if constexpr (KIND == 2) {      // rows g and g + 8: offset g of two tokens
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (tok[e] == t + 2 * i) {
                  sig[0][e] = s[e] * ka;
                  vl[0][e] = va;
                }
                if (tok[e] == t + 2 * i + 1) {
                  sig[0][e] = s[2 + e] * kc;
                  vl[0][e] = vc;
                }
              }
            } else if constexpr (FLAT) {      // offsets 16 pair + g and 8 further
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (tok[e] == t + i) {
                  sig[2 * pair][e] = s[e] * ka;
                  sig[2 * pair + 1][e] = s[2 + e] * kc;
                  vl[2 * pair][e] = va;
                  vl[2 * pair + 1][e] = vc;
                }
            } else {      // (a weight of 0 times a non-finite score: found at the end)
              const float wb = wg[2 * pair + i] * kc, wa = (1.f - wg[2 * pair + i]) * ka;
              if (wg[2 * pair + i] != 0.f) va = fmaxf(va, vc);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (tok[e] == t) {
                  sig[2 * pair + i][e] = fmaf(wb, s[2 + e], wa * s[e]);
                  vl[2 * pair + i][e] = va;
                }
            }
          }
          __syncwarp();
          issue(k);
        }
      }
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int c_of = __shfl_sync(0xffffffffu, off_c, i * 8 + g);
        const int cc = offsets ? c_of : 0x7fffffff;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sig[i][e] = cc <= qpos[e] ? fmaf(sig[i][e], scale[e], beta[e]) : -INFINITY;
          m[e] = fmaxf(m[e], E4M3 ? sig[i][e] + vl[i][e] : sig[i][e]);
        }
      }
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) {
        m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], d));
        m[1] = fmaxf(m[1], __shfl_xor_sync(0xffffffffu, m[1], d));
      }
    }

    // P^T of half a tile from the lane's two columns of a row
    auto transposed = [](Weights& p, int half, float a, float b) {
      split16<E4M3>(a, b, p.hi[half], p.lo[half]);
      p.hi[half] = transpose8(p.hi[half]);
      p.lo[half] = transpose8(p.lo[half]);
    };

    // ---- window and sinks, two tiles of 16 rows at a time ----
#pragma unroll 1
    for (int t0 = t_first; t0 < t_past; t0 += t_step) {
      const bool second = t0 + 1 < t_past, more = t0 + t_step < t_past;
      float s[2][4], nm[2] = {-INFINITY, -INFINITY};
      uint32_t stage = take();
      Y::template scores<2, Y::kTile>(stage, at_k, q, s);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i == 1 && !second) {
          s[1][0] = s[1][1] = s[1][2] = s[1][3] = -INFINITY;
          continue;
        }
        const int t = t0 + i;
        float ka[2] = {scale[0], scale[1]}, kc[2] = {scale[0], scale[1]}, va = 0.f, vc = 0.f;
        if constexpr (E4M3) {
          const float x0 = row_scale(stage, 0, i, 0), x1 = row_scale(stage, 0, i, 1);
          ka[0] *= x0; ka[1] *= x0; kc[0] *= x1; kc[1] *= x1;
          va = log_scale(row_scale(stage, 1, i, 0));
          vc = log_scale(row_scale(stage, 1, i, 1));
        }
        // lags of rows g and g + 8 from the two columns' positions (negative, so
        // large unsigned, where there is no column); sinks have no far edge, and
        // beyond the last one stand at a position past all
        const int r0 = t < 0 ? (g < a.S ? g : 1 << 29) : base + t * 16 + g;
        const int r1 = t < 0 ? (g + 8 < a.S ? g + 8 : 1 << 29) : r0 + 8;
        const unsigned far = t < 0 ? 0x7fffffffu : (unsigned)a.W;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[i][e] = (unsigned)(qpos[e] - r0) < far ? s[i][e] * ka[e] : -INFINITY;
          s[i][2 + e] = (unsigned)(qpos[e] - r1) < far ? s[i][2 + e] * kc[e] : -INFINITY;
          if (KIND == 2 && (near_lo | near_hi)) {      // (uniform)
            const int l0 = qpos[e] - r0, l1 = qpos[e] - r1;
            if (t >= 0 && (unsigned)l0 < 64u && ((l0 < 32 ? near_lo : near_hi) >> (l0 & 31) & 1u))
              s[i][e] += extra[e];
            if (t >= 0 && (unsigned)l1 < 64u && ((l1 < 32 ? near_lo : near_hi) >> (l1 & 31) & 1u))
              s[i][2 + e] += extra[e];
          }
          nm[e] = fmaxf(nm[e], E4M3 ? fmaxf(s[i][e] + va, s[i][2 + e] + vc)
                                    : fmaxf(s[i][e], s[i][2 + e]));
        }
      }
      __syncwarp();
      if (more)
        window_in(t0 + t_step, true);
      else if (NT > 0 && n_off > 0) {
        restart();
        rows_in(0, false);
      }
      commit();
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) {
        nm[0] = fmaxf(nm[0], __shfl_xor_sync(0xffffffffu, nm[0], d));
        nm[1] = fmaxf(nm[1], __shfl_xor_sync(0xffffffffu, nm[1], d));
      }
      if (__any_sync(0xffffffffu, nm[0] > m[0] || nm[1] > m[1])) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          nm[e] = fmaxf(nm[e], m[e]);
          const float f = exp2_approx(m[e] - (nm[e] == -INFINITY ? 0.f : nm[e]));
          m[e] = nm[e];
          l[e] *= f;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            o[j][e] *= f;
            o[j][2 + e] *= f;
          }
        }
      }
      const float z0 = m[0] == -INFINITY ? 0.f : m[0], z1 = m[1] == -INFINITY ? 0.f : m[1];
      stage = take();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i == 1 && !second) continue;
        float p[4] = {exp2_approx(s[i][0] - z0), exp2_approx(s[i][1] - z1),
                      exp2_approx(s[i][2] - z0), exp2_approx(s[i][3] - z1)};
        l[0] += p[0] + p[2];
        l[1] += p[1] + p[3];
        if constexpr (E4M3) {
          const float va = row_scale(stage, 1, i, 0), vc = row_scale(stage, 1, i, 1);
          p[0] *= va; p[1] *= va; p[2] *= vc; p[3] *= vc;
        }
        Weights pt;
        transposed(pt, 0, p[0], p[1]);
        transposed(pt, 1, p[2], p[3]);
        Y::template add_of<Y::kTile>(i, stage, at_v, pt, o);
      }
      __syncwarp();
      if (more)
        window_in(t0 + t_step, false);
      else if (NT > 0 && n_off > 1)
        rows_in(NT - 1, false);
      commit();
    }

    // ---- offset values ----
    if constexpr (KIND == 3) {
      const float z0 = m[0] == -INFINITY ? 0.f : m[0], z1 = m[1] == -INFINITY ? 0.f : m[1];
      // P^T of a tile: lane (g, c) has column (token) g, rows 2c and 2c + 1: offsets
      // 2 (c % 2) and the next of token 2 j + c / 2
      const int from = ((g & 1) * 4 + 2 * (c & 1)) * 4 + (g >> 1);
      const uint32_t at = Y::shared_at(true);
      float sum = 0.f;
#pragma unroll 1
      for (int st = 0; st < n_off; ++st) {
        const float p = exp2_approx(ps[st * 32] - (mine ? z1 : z0));
        sum += p;
        const uint32_t stage = take();
        const float w = __shfl_sync(0xffffffffu, off_w, st * 4 + (g & 3));
        float pa = p * (1.f - w), pb = p * w;
        if constexpr (E4M3) {
          pa *= shared_scale(stage, 1, true);
          pb *= shared_scale(stage, 1, false);
        }
        const float a0 = __shfl_sync(0xffffffffu, pa, from);
        const float a1 = __shfl_sync(0xffffffffu, pa, from + 4);
        const float b0 = __shfl_sync(0xffffffffu, pb, from);
        const float b1 = __shfl_sync(0xffffffffu, pb, from + 4);
        Weights f;
        split16<E4M3>(a0, a1, f.hi[0], f.lo[0]);
        split16<E4M3>(b0, b1, f.hi[1], f.lo[1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (2 * j >= count) continue;      // uniform
          const bool on = g == 2 * j + (c >> 1);
          const Weights p = {{on ? f.hi[0] : 0u, on ? f.hi[1] : 0u},
                             {on ? f.lo[0] : 0u, on ? f.lo[1] : 0u}};
          Y::template add_of<2 * Y::kRow>(j, stage, at, p, o);
        }
        __syncwarp();
        if (st + 2 < n_off) rows_in(0, false);
        commit();
      }
      l[0] += mine ? 0.f : sum;
      l[1] += mine ? sum : 0.f;
    } else if constexpr (NT > 0) {
      const float z0 = m[0] == -INFINITY ? 0.f : m[0], z1 = m[1] == -INFINITY ? 0.f : m[1];
      // P^T of all columns (plain rows): lane (g, c) has column g, rows 2c and 2c + 1;
      // a token's product takes its own columns of it
      [[maybe_unused]] Weights pt[NS];      // halves: rows a and b
      const int tok_g = token_of(g);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        sig[i][0] = exp2_approx(sig[i][0] - z0);
        sig[i][1] = exp2_approx(sig[i][1] - z1);
        l[0] += sig[i][0];
        l[1] += sig[i][1];
        if constexpr (!E4M3) {
          const float wb = wg[i], wa = 1.f - wb;
          transposed(pt[i], 0, sig[i][0] * wa, sig[i][1] * wa);
          if (!FLAT) transposed(pt[i], 1, sig[i][0] * wb, sig[i][1] * wb);
        }
      }
      int k = 2;
#pragma unroll 1
      for (int t = 0; k < n_off + 2; t += STEP) {
#pragma unroll
        for (int pair = 0; pair < NT; ++pair, ++k) {
          const bool second = FLAT ? t + STEP / 2 < count : pair * 16 + 8 < a.n_off;
          const uint32_t stage = take();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i == 1 && !second) continue;
            // tokens and offsets of rows 0..7 and 8..15
            const int at = KIND == 2 ? t + 2 * i : (FLAT ? t + i : t);
            const int bt = KIND == 2 ? at + 1 : at;
            const int ia = KIND == 2 ? 0 : (FLAT ? 2 * pair : 2 * pair + i);
            const int ib = KIND == 1 ? 2 * pair + 1 : ia;
            Weights p;
            if constexpr (E4M3) {
              const float wb = FLAT ? 1.f : wg[ia], wa = FLAT ? 1.f : 1.f - wb;
              const float va = row_scale(stage, 1, i, 0) * wa, vc = row_scale(stage, 1, i, 1) * wb;
              transposed(p, 0, tok[0] == at ? sig[ia][0] * va : 0.f,
                         tok[1] == at ? sig[ia][1] * va : 0.f);
              transposed(p, 1, tok[0] == bt ? sig[ib][0] * vc : 0.f,
                         tok[1] == bt ? sig[ib][1] * vc : 0.f);
            } else {
              constexpr int hb = FLAT ? 0 : 1;
              p.hi[0] = tok_g == at ? pt[ia].hi[0] : 0u;
              p.lo[0] = tok_g == at ? pt[ia].lo[0] : 0u;
              p.hi[1] = tok_g == bt ? pt[ib].hi[hb] : 0u;
              p.lo[1] = tok_g == bt ? pt[ib].lo[hb] : 0u;
            }
            Y::template add_of<Y::kTile>(i, stage, at_v, p, o);
          }
          __syncwarp();
          if (k < n_off) rows_in(pair, false);
          commit();
        }
      }
    }
  };
  if (ok) {
    if (NT == 0) {
      run(std::integral_constant<int, 1>());
    } else if (!__all_sync(0xffffffffu, off_w == 0.f)) {
      if constexpr (!TEAM && NT > 0) {
        if (shares && count > 3)
          run(std::integral_constant<int, 3>());
        else
          run(std::integral_constant<int, 0>());
      } else {
        run(std::integral_constant<int, 0>());
      }
    } else {
      // Integer distances: an offset inside the window is a window row a second time.
      // Such offsets (the first of each distance) are folded into the window's scores
      // where that leaves at most 8 others, which then go two tokens to a tile.
      if constexpr (NT == 1) {
        const bool listed = lane < a.n_off;
        const unsigned same = __match_any_sync(0xffffffffu, listed ? off_lo : -1 - lane);
        const bool near = listed && off_lo < min(a.W, 64) && __ffs(same) == lane + 1;
        unsigned far = __ballot_sync(0xffffffffu, listed && !near);
        if (!TEAM && count > 2 && (far == 0 || (a.n_off > 8 && __popc(far) <= 8))) {
          near_lo = __reduce_or_sync(0xffffffffu, near && off_lo < 32 ? 1u << off_lo : 0u);
          near_hi = __reduce_or_sync(0xffffffffu, near && off_lo >= 32 ? 1u << (off_lo & 31) : 0u);
        } else {
          far = __ballot_sync(0xffffffffu, listed);
        }
        n_far = __popc(far);
        if (n_far <= 8) {      // the others, in order, to lanes 0 .. n_far - 1
          int* list = reinterpret_cast<int*>(own_smem);
          if (far >> lane & 1u) list[__popc(far & ((1u << lane) - 1u))] = off_lo;
          __syncwarp();
          off_lo = lane < n_far ? list[lane] : 0;
          off_c = lane < n_far ? off_lo : 0x7fffffff;
          __syncwarp();
        }
      }
      if constexpr (NT == 1) {
        if (n_far <= 8)
          run(std::integral_constant<int, 2>());
        else
          run(std::integral_constant<int, 1>());
      } else {
        run(std::integral_constant<int, 1>());
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if constexpr (TEAM) {      // each CTA's first member joins its parts, then the first CTA's these
    constexpr int kPart = D / 4 + 4;      // floats of a lane's part
    static_assert(kPart * 32 * 4 <= 2 * 32 * Y::kRow, "a part fits a warp's stages");
    auto publish = [&]() {
      float* mine = reinterpret_cast<float*>(own_smem) + lane;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) mine[(4 * j + e) * 32] = o[j][e];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mine[(D / 4 + e) * 32] = m[e];
        mine[(D / 4 + 2 + e) * 32] = l[e];
      }
      if (__any_sync(0xffffffffu, lost) && lane == 0) {
        mine[(D / 4) * 32] = __int_as_float(0x7fc00000);      // tells who joins it
        atomicOr(&g_chunk_err, kErrPage);
      }
    };
    auto absorb = [&](auto part) {      // part(i): its float i
      const bool theirs = __shfl_sync(0xffffffffu, part(D / 4) != part(D / 4), 0);
      lost = lost || theirs;      // (every lane shuffles, lost or not)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mp = part(D / 4 + e), top = fmaxf(m[e], mp);
        const float z = top == -INFINITY ? 0.f : top;
        const float f = exp2_approx(m[e] - z), fp = exp2_approx(mp - z);
        m[e] = top;
        l[e] = l[e] * f + part(D / 4 + 2 + e) * fp;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          o[j][e] = o[j][e] * f + part(4 * j + e) * fp;
          o[j][2 + e] = o[j][2 + e] * f + part(4 * j + 2 + e) * fp;
        }
      }
    };
    if (warp > 0) publish();
    __syncthreads();      // (the returns before are the same for all of the team)
    if (warp > 0) return;
    for (int w = 1; w < kWarps; ++w) {
      const float* part = reinterpret_cast<const float*>(
                              s_stages + w * warp_bytes<D, E4M3, NT, TEAM>(shares)) + lane;
      absorb([&](int i) { return part[i * 32]; });
    }
    if (a.team > 1) {      // (the barriers count the warps that have not returned)
      if (rank > 0) publish();
      cluster_barrier();
      if (rank == 0)
        for (int r = 1; r < a.team; ++r) {
          const uint32_t part = cluster_address(own_smem, r) + lane * 4;
          absorb([&](int i) { return load_cluster(part + i * 128); });
        }
      cluster_barrier();      // what was read stays until then
      if (rank > 0) return;
    }
  }
#pragma unroll
  for (int d = 4; d <= 16; d <<= 1) {
    l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
    l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
  }
  const bool nan = __any_sync(0xffffffffu, lost) || !ok;

  // A weight of 0 does not hide an infinity or a NaN: when an output is not
  // finite, the block's queries are computed again from their own members alone.
  float odd[2] = {l[0], l[1]};      // times 0: 0 for finite values only
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    odd[e] *= 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
      odd[e] = fmaf(o[j][e], 0.f, fmaf(o[j][2 + e], 0.f, odd[e]));
  }
  if (!nan && __any_sync(0xffffffffu, (tok[0] >= 0 && odd[0] != 0.f) ||
                                          (tok[1] >= 0 && odd[1] != 0.f))) {
    for (int col = 0; col < count * a.per; ++col) {
      const int t = token_of(col), hh = col - t * a.per;
      if (hh < heads)
        one_query<__nv_bfloat16, D, E4M3>(a, layer, head0 + hh, n0 + t, b, pos0 + t, true);
    }
    return;
  }

  // Outputs through shared memory: one row per column, 16 bytes apart in banks,
  // then 16 bytes a lane of consecutive head dims.
  constexpr int kOut = D * 2 + 16;
  uint8_t* const out = own_smem;
  static_assert(8 * kOut <= 2 * 32 * Y::kRow, "the output tile fits the stages");
  __syncwarp();
  const float bad = __int_as_float(0x7fc00000);
  const float inv0 = nan ? bad : 1.f / l[0], inv1 = nan ? bad : 1.f / l[1];
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    if constexpr (E4M3) {      // head dims 16 j + 2 g and the next
      *reinterpret_cast<uint32_t*>(out + (2 * c) * kOut + (16 * j + 2 * g) * 2) =
          pack_bf16x2(o[j][0] * inv0, o[j][2] * inv0);
      *reinterpret_cast<uint32_t*>(out + (2 * c + 1) * kOut + (16 * j + 2 * g) * 2) =
          pack_bf16x2(o[j][1] * inv1, o[j][3] * inv1);
    } else {                   // transposed: column g, head dims 2c and 2c + 1 of eight
      *reinterpret_cast<uint32_t*>(out + g * kOut + (16 * j + 2 * c) * 2) =
          transpose8(pack_bf16x2(o[j][0] * inv0, o[j][1] * inv1));
      *reinterpret_cast<uint32_t*>(out + g * kOut + (16 * j + 8 + 2 * c) * 2) =
          transpose8(pack_bf16x2(o[j][2] * inv0, o[j][3] * inv1));
    }
  }
  __syncwarp();
  constexpr int kPer = D / 8;      // 16-byte chunks of a row
  const size_t out0 = ((size_t)layer * a.N + n0) * a.Hq + head0;
#pragma unroll
  for (int i = 0; i < 8 * kPer / 32 || i == 0; ++i) {
    const int id = i * 32 + lane, col = id / kPer, t = token_of(col), hh = col - t * a.per;
    if (id < 8 * kPer && t < count && hh < heads)
      *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.o) +
                                (out0 + t * a.Hq + hh) * D + (id % kPer) * 8) =
          *reinterpret_cast<const uint4*>(out + col * kOut + (id % kPer) * 16);
  }
  if (a.lse && g == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (tok[e] >= 0)
        a.lse[out0 + tok[e] * a.Hq + sub[e]] = nan ? bad : kLn2 * (m[e] + log2f(l[e]));
  }
  if (__any_sync(0xffffffffu, lost) && lane == 0) atomicOr(&g_chunk_err, kErrPage);
}

// ---------------------------------------------------------------------------
// 32-bit queries, and the queries that meet infinities or NaN.

// NE consecutive elements of a cache row from element e0, as stored.
template <bool E4M3, bool BF16, int NE>
__device__ __forceinline__ void load_part(const uint8_t* base, int D, int row, int e0,
                                          float (&x)[NE]) {
  if constexpr (E4M3) {
    const uint8_t* p = base + (size_t)row * D + e0;
    if constexpr (NE == 1) {
      float unused;
      e4m3x2_to_float2(__ldg(p), x[0], unused);
    } else {
      constexpr int STEP = NE < 16 ? NE : 16, NW = STEP < 4 ? 1 : STEP / 4;
#pragma unroll
      for (int i = 0; i < NE / STEP; ++i) {
        uint32_t u[NW];
        load_words<STEP>(p + i * STEP, u);
#pragma unroll
        for (int j = 0; j < STEP / 2; ++j)
          e4m3x2_to_float2((u[j / 2] >> (16 * (j & 1))) & 0xffffu, x[i * STEP + 2 * j],
                           x[i * STEP + 2 * j + 1]);
      }
    }
  } else if constexpr (BF16) {
    load_row<__nv_bfloat16, NE>(reinterpret_cast<const __nv_bfloat16*>(base) + (size_t)row * D + e0,
                                x);
  } else {
    const float* p = reinterpret_cast<const float*>(base) + (size_t)row * D + e0;
    if constexpr (NE == 1)
      x[0] = __ldg(p);
    else if constexpr (NE == 2) {
      const float2 u = __ldg(reinterpret_cast<const float2*>(p));
      x[0] = u.x; x[1] = u.y;
    } else
      load_row<float, NE>(p, x);
  }
}

// NH query heads (from hq on, `live` of them) of one key/value head and one token (row n
// of sequence b at position pos) by one warp: members 32 at a time, and no row but
// their members' is touched.
template <typename QT, int D, bool E4M3, int NH>
__device__ __forceinline__ void query_heads(const ChunkArgs& a, int layer, int hq, int live, int n,
                                            int b, int pos, bool inside) {
  constexpr bool BF16 = !E4M3 && sizeof(QT) == 2;
  constexpr int QE = D / 4;                        // elements of a row per quad lane
  constexpr int VE = D >= 32 ? D / 32 : 1;         // value elements per lane
  constexpr int SPLIT = D >= 32 ? 1 : 2;           // D = 16: two members at a time
  constexpr int BATCH = NH == 1 || D == 128 ? 2 : 4;      // value rows whose loads are in flight
  const int lane = threadIdx.x & 31, part = lane & 3, mm = lane >> 2;
  const int h = hq / a.G;

  int off_lo = 0, off_c = 0x7fffffff;
  float off_w = 0.f;
  bool ok = inside;
  if (lane < a.n_off) {
    const OffGeo og = offset_geometry(__ldg(a.alpha + layer), a.f[lane]);
    off_lo = og.lo; off_c = og.c; off_w = og.w;
    ok = ok && og.ok;
  }
  ok = __all_sync(0xffffffffu, ok);
  bool lost = !inside;
  const int* table = a.table + (size_t)b * a.max_pages;
  const size_t pool = (size_t)layer * a.n_pages * a.Hkv * a.pd.d;
  constexpr int kElt = E4M3 ? 1 : (int)sizeof(QT);
  const uint8_t* kb = reinterpret_cast<const uint8_t*>(a.kc) + pool * D * kElt;
  const uint8_t* vb = reinterpret_cast<const uint8_t*>(a.vc) + pool * D * kElt;

  const size_t at = ((size_t)layer * a.N + n) * a.Hq + hq;
  float q[NH][QE], beta[NH], m[NH], l[NH], o[NH][VE];
#pragma unroll
  for (int j = 0; j < NH; ++j) {
    const int jj = min(j, live - 1);      // idle heads repeat the last one
    load_row<QT, QE>(reinterpret_cast<const QT*>(a.q) + layer * a.ql + n * a.qn +
                         (hq + jj) * a.qh + part * QE, q[j]);
    beta[j] = a.beta ? __ldg(a.beta + at + jj) : 0.f;
    m[j] = -INFINITY;
    l[j] = 0.f;
#pragma unroll
    for (int i = 0; i < VE; ++i) o[j][i] = 0.f;
  }
  const int nw = min(a.W, pos + 1), ns = min(a.S, pos + 1);
  const int total = ok ? nw + ns + a.n_off : 0;
  const int d0 = (D >= 32 ? lane : (lane & 15)) * VE;

  for (int m0 = 0; m0 < total; m0 += 32) {
    // lane's member m0 + lane: rows, weights
    const int mem = m0 + lane;
    const int k = mem - nw - ns;
    const int lo = __shfl_sync(0xffffffffu, off_lo, k & 31);
    const int cc = __shfl_sync(0xffffffffu, off_c, k & 31);
    const float w = __shfl_sync(0xffffffffu, off_w, k & 31);
    int ra = -1, rb = -1;
    if (mem < nw) {
      ra = pos - mem;
    } else if (k < 0) {
      ra = mem - nw;
    } else if (k < a.n_off && cc <= pos) {
      ra = pos - lo;
      if (w != 0.f) rb = ra - 1;
    }
    float wa = 1.f, wb = 0.f;
    const bool off = k >= 0;
    if (rb >= 0) { wa = 1.f - w; wb = w; }
    if (ra >= 0) { ra = pool_row(table, a.pd, ra, a.n_pages, a.Hkv, h); lost |= ra < 0; }
    if (rb >= 0) { rb = pool_row(table, a.pd, rb, a.n_pages, a.Hkv, h); lost |= rb < 0; }
    float ka = wa, kc = wb, va = wa, vc = wb;
    if constexpr (E4M3) {
      if (ra >= 0) { ka *= __ldg(a.ks + pool + ra); va *= __ldg(a.vs + pool + ra); }
      if (rb >= 0) { kc *= __ldg(a.ks + pool + rb); vc *= __ldg(a.vs + pool + rb); }
    }
    // scores: 8 members at a time, four lanes each
    float s[NH], p[NH];
#pragma unroll
    for (int j = 0; j < NH; ++j) s[j] = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ia = __shfl_sync(0xffffffffu, ra, i * 8 + mm);
      const int ib = __shfl_sync(0xffffffffu, rb, i * 8 + mm);
      const float xa = __shfl_sync(0xffffffffu, ka, i * 8 + mm);
      const float xb = __shfl_sync(0xffffffffu, kc, i * 8 + mm);
      float dot[NH];
#pragma unroll
      for (int j = 0; j < NH; ++j) dot[j] = 0.f;
#pragma unroll
      for (int row = 0; row < 2; ++row) {
        const int at_row = row ? ib : ia;
        if (at_row < 0) continue;
        float x[QE];
        load_part<E4M3, BF16, QE>(kb, D, at_row, part * QE, x);
#pragma unroll
        for (int j = 0; j < NH; ++j) {
          float t = 0.f;
#pragma unroll
          for (int e = 0; e < QE; ++e) t = fmaf(q[j][e], x[e], t);
          dot[j] = fmaf(t, row ? xb : xa, dot[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < NH; ++j) {
        dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], 1);
        dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], 2);
        const float mine = __shfl_sync(0xffffffffu, dot[j], (lane & 7) * 4);
        if ((lane >> 3) == i) s[j] = mine;
      }
    }
#pragma unroll
    for (int j = 0; j < NH; ++j) {
      s[j] = ra >= 0 ? (s[j] * a.scale + (off ? beta[j] : 0.f)) * kLog2e : -INFINITY;
      float nm = s[j];
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, d));
      nm = fmaxf(m[j], nm);
      const float z = nm == -INFINITY ? 0.f : nm;
      const float f = exp2f(m[j] - z);
      p[j] = exp2f(s[j] - z);
      m[j] = nm;
      l[j] = l[j] * f + p[j];
#pragma unroll
      for (int i = 0; i < VE; ++i) o[j][i] *= f;
    }
    // values: lanes over head dims; an interpolated value is formed once for all heads
    if constexpr (NH == 1) {      // (the probability is part of the rows' weights)
      va *= p[0];
      vc *= p[0];
    }
    const int here = min(32, total - m0);
    for (int i0 = 0; i0 < here; i0 += BATCH * SPLIT) {
      float xa[BATCH][VE], xb[BATCH][VE];
      int src[BATCH];
      bool ina[BATCH], inb[BATCH];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        src[u] = (i0 + u * SPLIT + (SPLIT == 2 ? lane >> 4 : 0)) & 31;
        const int ia = __shfl_sync(0xffffffffu, ra, src[u]);
        const int ib = __shfl_sync(0xffffffffu, rb, src[u]);
        ina[u] = i0 + u * SPLIT < here && ia >= 0;
        inb[u] = ina[u] && ib >= 0;
        if (ina[u]) load_part<E4M3, BF16, VE>(vb, D, ia, d0, xa[u]);
        if (inb[u]) load_part<E4M3, BF16, VE>(vb, D, ib, d0, xb[u]);
      }
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const float ya = __shfl_sync(0xffffffffu, va, src[u]);
        const float yb = __shfl_sync(0xffffffffu, vc, src[u]);
        if (inb[u]) {
#pragma unroll
          for (int e = 0; e < VE; ++e) xa[u][e] = fmaf(yb, xb[u][e], ya * xa[u][e]);
        } else if (ina[u]) {
#pragma unroll
          for (int e = 0; e < VE; ++e) xa[u][e] *= ya;
        }
#pragma unroll
        for (int j = 0; j < NH; ++j) {
          const float pj = NH == 1 ? 1.f : __shfl_sync(0xffffffffu, p[j], src[u]);
          if (ina[u]) {
#pragma unroll
            for (int e = 0; e < VE; ++e) o[j][e] = fmaf(pj, xa[u][e], o[j][e]);
          }
        }
      }
    }
  }
  const bool nan = __any_sync(0xffffffffu, lost) || !ok;
  const float bad = __int_as_float(0x7fc00000);
#pragma unroll
  for (int j = 0; j < NH; ++j) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], d);
    if constexpr (SPLIT == 2) o[j][0] += __shfl_xor_sync(0xffffffffu, o[j][0], 16);
    if (j >= live) continue;
    const float inv = nan ? bad : 1.f / l[j];
    if (D >= 32 || lane < 16) {
#pragma unroll
      for (int e = 0; e < VE; ++e) o[j][e] *= inv;
      store_row<QT, VE>(reinterpret_cast<QT*>(a.o) + (at + j) * D + d0, o[j]);
    }
    if (lane == 0 && a.lse) a.lse[at + j] = nan ? bad : kLn2 * m[j] + logf(l[j]);
  }
  if (lost) atomicOr(&g_chunk_err, kErrPage);
}

// One query out of a block of k_chunk_tc.
template <typename QT, int D, bool E4M3>
__device__ __noinline__ void one_query(const ChunkArgs& a, int layer, int hq, int n, int b,
                                       int pos, bool inside) {
  query_heads<QT, D, E4M3, 1>(a, layer, hq, 1, n, b, pos, inside);
}

template <int D, bool E4M3, int NH>
__global__ void __launch_bounds__(kWarps * 32) k_chunk_f32(const __grid_constant__ ChunkArgs a) {
  const int n = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (n >= a.N) return;
  const int per = (a.G + NH - 1) / NH;      // groups of NH heads per key/value head
  const int h = blockIdx.y / per, j = (blockIdx.y % per) * NH;
  const int b = find_sequence(a.cu, a.B, 0, n);
  const int first = __ldg(a.cu + b);
  if (first < 0 || n < first || n >= __ldg(a.cu + b + 1)) return;
  const long long posl = (long long)__ldg(a.cached + b) + (n - first);
  const bool inside = posl >= 0 && posl < (long long)a.max_pages * a.pd.d;
  query_heads<float, D, E4M3, NH>(a, blockIdx.z, h * a.G + j, min(NH, a.G - j), n, b,
                                  inside ? (int)posl : 0, inside);
}

// Heads of a group by one warp: a row is loaded once for all of them; as many as the
// registers hold (4, at D = 128 2) where warps enough remain for 16 per SM.
template <int D, bool E4M3, int NH>
cudaError_t launch_f32(const ChunkArgs& a, cudaStream_t st) {
  const long long warps = (long long)a.N * a.Hkv * ((a.G + NH - 1) / NH) * a.L;
  if constexpr (NH > 1) {
    if (a.G < NH || warps < 148 * 16) return launch_f32<D, E4M3, NH / 2>(a, st);
  }
  const dim3 grid((a.N + kWarps - 1) / kWarps, a.Hkv * ((a.G + NH - 1) / NH), a.L);
  k_chunk_f32<D, E4M3, NH><<<grid, kWarps * 32, 0, st>>>(a);
  return cudaSuccess;
}

template <int D, bool E4M3, int NT, bool TEAM>
cudaError_t launch_tc(const ChunkArgs& a, cudaStream_t st) {
  const int smem = kWarps * warp_bytes<D, E4M3, NT, TEAM>(a.shift == 3);
  // The limit is the process's: the instance's largest size whatever this call needs, so
  // that calls of several threads do not lower it for each other.
  constexpr int most = kWarps * warp_bytes<D, E4M3, NT, TEAM>(true);
  static_assert(most >= kWarps * warp_bytes<D, E4M3, NT, TEAM>(false), "shared stages are larger");
  if (most > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        k_chunk_tc<D, E4M3, NT, TEAM>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(TEAM ? a.blocks * a.team : (a.blocks + kWarps - 1) / kWarps, a.Hkv * a.groups,
                  a.L);
  if (TEAM && a.team > 1) {
    cudaLaunchAttribute cluster = {};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim = {(unsigned)a.team, 1, 1};
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(kWarps * 32);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = &cluster;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, k_chunk_tc<D, E4M3, NT, TEAM>, a);
  }
  k_chunk_tc<D, E4M3, NT, TEAM><<<grid, kWarps * 32, smem, st>>>(a);
  return cudaSuccess;
}

template <int D, bool E4M3, int NT>
cudaError_t launch_nt(const ChunkArgs& a, cudaStream_t st) {
  return a.team > 0 ? launch_tc<D, E4M3, NT, true>(a, st) : launch_tc<D, E4M3, NT, false>(a, st);
}

template <int D, bool E4M3>
cudaError_t launch_t(const ChunkArgs& a, bool f32, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  trace_mark("chunk_attn", st, true);
  if (f32) {
    e = launch_f32<D, E4M3, D == 128 ? 2 : 4>(a, st);
  } else {
    e = a.n_off == 0    ? launch_nt<D, E4M3, 0>(a, st)
        : a.n_off <= 16 ? launch_nt<D, E4M3, 1>(a, st)
                        : launch_nt<D, E4M3, 2>(a, st);
  }
  trace_mark("chunk_attn", st, false);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

template <int D>
cudaError_t launch_chunk_of(const ChunkArgs& a, bool f32, bool e4m3, cudaStream_t st) {
  return e4m3 ? launch_t<D, true>(a, f32, st) : launch_t<D, false>(a, f32, st);
}

template <int D>
cudaError_t chunk_error_of(unsigned* out, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_chunk_err, sizeof(unsigned));
  if (e != cudaSuccess || !clear || *out == 0) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_chunk_err, &zero, sizeof(unsigned));
}
#endif  // SA_CHUNK_KERNELS

}  // namespace sa
