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
// that eight columns, not sixteen, have to be filled. Gathered rows go straight
// from global memory into A fragments: the contraction index of a product may be
// permuted, so a lane takes 16 contiguous bytes of its row (and the query
// fragments the same), and a pair of V rows becomes a fragment by byte
// permutes. Nothing is staged, no barrier is needed, and a row read by several
// tokens is an L1 hit. tcgen05 has no form for this gather: its A operand is a
// tile of 128 rows in tensor or shared memory, of which a token's 15 interpolated
// pairs would fill a quarter, after a copy through shared memory.
//   - Window and sinks: tiles of 16 rows shared by all columns, masked, with a
//     running maximum and sum per column.
//   - Offsets: for each token tiles of 8 offsets, row a of offset g in row g of
//     the tile and row b in row g + 8, so that one lane holds both dot products
//     and interpolates in registers. Only the token's own columns of such a
//     tile count: over the block's tokens a lane keeps just its own two
//     columns, 2 scores per tile in all.
// Rounding: products of 16-bit (or e4m3) values are exact, sums fp32; the
// probabilities are rounded to bf16 for P V (2^-9 each, below the output's own
// rounding on average), their sum is not. e4m3 codes are used as bf16 values, the
// row scales (powers of two) multiply the scores and the probabilities.
// A masked probability is 0, and 0 * Inf or NaN is NaN: when a block of several
// tokens ends with a non-finite output, its tokens are computed again one by
// one, where no masked row is loaded at all.
//
// 32-bit queries (k_chunk_f32): one warp per (token, query head) on the CUDA
// cores, chunks of 32 members: four lanes per member for the scores, lanes over
// head dims for the values.
#include "sa_paged.cuh"

namespace sa {

namespace {

__device__ unsigned g_chunk_err;

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct ChunkArgs {
  int L, N, B, Hq, Hkv, n_pages, max_pages, W, n_off, S, blocks;
  int G, groups, per, shift;      // heads per kv head; column groups, heads in one, log2 tokens
  FastDiv pd;
  float scale;
  int f[SA_MAX_OFFSETS];
  int64_t ql, qn, qh;
  const void* q; const void* kc; const void* vc; const float* ks; const float* vs;
  const float* alpha; const float* beta;
  const int* table; const int* cu; const int* cached;
  void* o; float* lse;
};

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

// Lane layouts of a row of D elements, in pieces of at most 16 bytes of the
// cache's type.
//   K (and q): lane c of a quad holds KP pieces of KE elements, piece i at
//              element (4 i + c) KE;
//   V (and o): lane g of eight holds VP pieces of VE elements, piece i at
//              element (8 i + g) VE.
template <int D, bool E4M3>
struct Lay {
  static constexpr int kElt = E4M3 ? 1 : 2, kRow = D * kElt;      // bytes
  static constexpr int kFull = 16 / kElt;
  static constexpr int KE = D / 4 < kFull ? D / 4 : kFull, KP = D / 4 / KE;
  static constexpr int VE = D / 8 < kFull ? D / 8 : kFull, VP = D / 8 / VE;
  static constexpr int KW = D / 4 * kElt / 4;                     // words of a K part
  static constexpr int VN = VE * kElt < 4 ? 1 : VE * kElt / 4;    // words of a V piece
};

// Two e4m3 codes as two fp16 values: exact, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t h;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(h) : "r"(two));
  return h;
}

// K parts of 16 rows: this lane's of rows g (a) and g + 8 (b) of the tile.
template <int D, bool E4M3>
struct KTile {
  using Y = Lay<D, E4M3>;
  uint32_t a[Y::KW], b[Y::KW];
  __device__ __forceinline__ void load(const uint8_t* lane_base, int ra, int rb) {
    const uint8_t* pa = lane_base + (int64_t)ra * Y::kRow;
    const uint8_t* pb = lane_base + (int64_t)rb * Y::kRow;
    constexpr int PB = Y::KE * Y::kElt;      // bytes of a piece
#pragma unroll
    for (int i = 0; i < Y::KP; ++i) {
      load_words<PB>(pa + i * 4 * PB, a + i * (PB / 4));
      load_words<PB>(pb + i * 4 * PB, b + i * (PB / 4));
    }
  }
  // S^T of the 16 rows with the block's 8 columns
  __device__ __forceinline__ void scores(const uint32_t (&q)[D / 8], float (&s)[4]) const {
    s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      if constexpr (E4M3)
        mma16816<true>(s, e4m3x2_to_f16x2(a[i] & 0xffffu), e4m3x2_to_f16x2(b[i] & 0xffffu),
                       e4m3x2_to_f16x2(a[i] >> 16), e4m3x2_to_f16x2(b[i] >> 16), q[2 * i],
                       q[2 * i + 1]);
      else
        mma16816<false>(s, a[2 * i], b[2 * i], a[2 * i + 1], b[2 * i + 1], q[2 * i],
                        q[2 * i + 1]);
    }
  }
};

// V parts of 16 rows: this lane's of rows 2c, 2c+1, 2c+8 and 2c+9 of the tile.
template <int D, bool E4M3>
struct VTile {
  using Y = Lay<D, E4M3>;
  uint32_t u[4][Y::VP * Y::VN];
  __device__ __forceinline__ void load(const uint8_t* lane_base, int r, int row) {
    const uint8_t* p = lane_base + (int64_t)row * Y::kRow;
    constexpr int PB = Y::VE * Y::kElt;
#pragma unroll
    for (int i = 0; i < Y::VP; ++i) load_words<PB>(p + i * 8 * PB, u[r] + i * Y::VN);
  }
  // O^T += V^T P^T; p0 and p1: the fragments of P^T
  __device__ __forceinline__ void add(uint32_t p0, uint32_t p1, float (&o)[D / 16][4]) const {
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {      // head dims 2j and 2j + 1 of this lane's list
      if constexpr (E4M3) {
        const int w = j / 2;
        const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
        const uint32_t x = __byte_perm(u[0][w], u[1][w], sel);
        const uint32_t y = __byte_perm(u[2][w], u[3][w], sel);
        mma16816<true>(o[j], e4m3x2_to_f16x2(x & 0xffffu), e4m3x2_to_f16x2(x >> 16),
                       e4m3x2_to_f16x2(y & 0xffffu), e4m3x2_to_f16x2(y >> 16), p0, p1);
      } else {
        mma16816<false>(o[j], __byte_perm(u[0][j], u[1][j], 0x5410),
                        __byte_perm(u[0][j], u[1][j], 0x7632),
                        __byte_perm(u[2][j], u[3][j], 0x5410),
                        __byte_perm(u[2][j], u[3][j], 0x7632), p0, p1);
      }
    }
  }
};

// A lane's walk over the rows that one member has for consecutive tokens: one
// more row per token, in the same page mostly.
struct Walk {
  int row, left;      // pool row of the last token served; rows after it in its page
};

template <typename QT, int D, bool E4M3>
__device__ __noinline__ void one_query(const ChunkArgs& a, int layer, int hq, int n, int b,
                                       int pos, bool inside);

// ---------------------------------------------------------------------------
// NT: pairs of offset tiles (16 offsets each), 0 .. 2.
template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kWarps * 32) k_chunk_tc(const __grid_constant__ ChunkArgs a) {
  using Y = Lay<D, E4M3>;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int x = blockIdx.x * kWarps + (threadIdx.x >> 5);
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

  // column 2c + e of this lane: token tok[e] of the block, query head head[e]
  const int heads = min(a.per, a.G - grp * a.per);
  int tok[2], head[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int col = 2 * c + e;
    tok[e] = col / a.per;
    const int hh = col - tok[e] * a.per;
    head[e] = h * a.G + grp * a.per + hh;
    if (hh >= heads || tok[e] >= count) tok[e] = -1;
  }

  // offset geometry: lane k holds offset k
  int off_lo = 0, off_c = 0x7fffffff;
  float off_w = 0.f;
  bool ok = inside;
  if (NT > 0 && lane < a.n_off) {
    const OffGeo og = offset_geometry(__ldg(a.alpha + layer), a.f[lane]);
    off_lo = og.lo; off_c = og.c; off_w = og.w;
    ok = ok && og.ok;
  }
  const int* table = a.table + (size_t)b * a.max_pages;
  const size_t pool = (size_t)layer * a.n_pages * a.Hkv * a.pd.d;
  const uint8_t* kb = reinterpret_cast<const uint8_t*>(a.kc) + pool * Y::kRow + c * Y::KE * Y::kElt;
  const uint8_t* vb = reinterpret_cast<const uint8_t*>(a.vc) + pool * Y::kRow + g * Y::VE * Y::kElt;
  const float* ks = E4M3 ? a.ks + pool : nullptr;
  const float* vs = E4M3 ? a.vs + pool : nullptr;
  bool lost = !inside;      // a position or page outside its range
  ok = __all_sync(0xffffffffu, ok);

  // query fragments: column g of the block. For e4m3 rows in fp16, times a power
  // of two that brings the column's largest element to [2^14, 2^15): an element
  // loses bits only where it is 2^28 times smaller.
  uint32_t q[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) q[i] = 0u;
  {
    const int t = g / a.per, hh = g - t * a.per;
    if (hh < heads && t < count) {
      const __nv_bfloat16* qp = reinterpret_cast<const __nv_bfloat16*>(a.q) + layer * a.ql +
                                (n0 + t) * a.qn + (h * a.G + grp * a.per + hh) * a.qh;
#pragma unroll
      for (int i = 0; i < Y::KP; ++i) {
        const uint8_t* p = reinterpret_cast<const uint8_t*>(qp + (4 * i + c) * Y::KE);
        if constexpr (Y::KE == 16) {
          load_words<16>(p, q + i * 8);
          load_words<16>(p + 16, q + i * 8 + 4);
        } else {
          load_words<Y::KE * 2>(p, q + i * (Y::KE / 2));
        }
      }
    }
  }
  float scale[2] = {a.scale * kLog2e, a.scale * kLog2e};      // of the lane's two columns
  if constexpr (E4M3) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      top = fmaxf(top, fmaxf(fabsf(bf16lo(q[i])), fabsf(bf16hi(q[i]))));
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
  float beta[2] = {0.f, 0.f};
  if (a.beta) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (tok[e] >= 0)
        beta[e] = kLog2e * __ldg(a.beta + ((size_t)layer * a.N + n0 + tok[e]) * a.Hq + head[e]);
  }

  // Running reference m and sum l of each of the lane's columns; o the outputs
  // times l. For e4m3 rows the reference is the maximum of score + log2(value
  // scale): the weights that go into P V, probability * value scale, are then at
  // most 1 and fit fp16 whatever the scales.
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[D / 16][4];
#pragma unroll
  for (int j = 0; j < D / 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float sig[NT > 0 ? 2 * NT : 1][2];

  if (ok) {
    auto find = [&](int r, int& left) {
      const int lp = quotient(a.pd, r), in = r - lp * a.pd.d;
      const int page = __ldg(table + lp);
      left = a.pd.d - 1 - in;
      if ((unsigned)page >= (unsigned)a.n_pages) {
        lost = true;
        left = 0;
        return 0;
      }
      return (page * a.Hkv + h) * a.pd.d + in;
    };
    auto step_to = [&](Walk& w, int r, int by) {      // from row r - by to row r
      if (w.left >= by) {
        w.row += by;
        w.left -= by;
      } else {
        w.row = find(r, w.left);
      }
    };
    // Rows without a member take this row, the first token's own, with weight 0.
    int unused;
    const int fill = find(pos0, unused);
    const bool flat = __all_sync(0xffffffffu, off_w == 0.f);      // integer distances only

    // ---- offset scores -------------------------------------------------------
    // A tile pair serves 16 offsets. Interpolated: tile i holds, for 8 offsets,
    // rows a in 0..7 and rows b in 8..15, and lane c of quad g looks up row a (c
    // even) or b (c odd) of offset g of tile c / 2. Integer distances only: one
    // tile per token holds 16 offsets; lanes 0..15 look up the rows of token t,
    // lanes 16..31 those of t + 1.
    int lo_[NT > 0 ? NT : 1], c_[NT > 0 ? NT : 1];
    float w_[NT > 0 ? 2 * NT : 1];
    bool two = true;
#pragma unroll
    for (int pair = 0; pair < NT; ++pair) {
      const int src = pair * 16 + (flat ? lane & 15 : (c >> 1) * 8 + g);
      const float w = __shfl_sync(0xffffffffu, off_w, src);
      lo_[pair] = __shfl_sync(0xffffffffu, off_lo, src) + (flat ? 0 : c & 1);
      c_[pair] = __shfl_sync(0xffffffffu, off_c, src);
      if (!flat && (c & 1) && w == 0.f) c_[pair] = 0x7fffffff;      // no second row
      w_[2 * pair] = __shfl_sync(0xffffffffu, off_w, pair * 16 + g);
      w_[2 * pair + 1] = __shfl_sync(0xffffffffu, off_w, pair * 16 + 8 + g);
    }
    (void)two;
    const int ahead = flat ? lane >> 4 : 0;       // this lane serves token t + ahead
    const int stride = flat ? 2 : 1;

    if constexpr (NT > 0) {
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) sig[i][0] = sig[i][1] = -INFINITY;
      Walk w[NT];
#pragma unroll
      for (int pair = 0; pair < NT; ++pair) w[pair] = {0, -1};
      // scores of a tile, times its rows' scales; ra, rb < 0: no member
      auto tile_scores = [&](const KTile<D, E4M3>& k, int ra, int rb, float (&s)[4]) {
        k.scores(q, s);
        if constexpr (E4M3) {
          const float ka = __ldg(ks + (ra ^ (ra >> 31))), kc = __ldg(ks + (rb ^ (rb >> 31)));
          s[0] *= ka; s[1] *= ka; s[2] *= kc; s[3] *= kc;
        }
      };
      auto log_scale = [&](int r) {
        return __log2f(fmaxf(fabsf(__ldg(vs + (r ^ (r >> 31)))), 7.9e-31f));
      };
      for (int t = 0; t < count; t += stride) {
#pragma unroll
        for (int pair = 0; pair < NT; ++pair) {
          const int p = pos0 + t + ahead;
          int row = ~fill;
          if (c_[pair] <= p && t + ahead < count) {
            step_to(w[pair], p - lo_[pair], stride);
            row = w[pair].row;
          }
          if (flat) {
            // tiles of tokens t and t + 1
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (t + i >= count) continue;
              const int ra = __shfl_sync(0xffffffffu, row, i * 16 + g);
              const int rb = __shfl_sync(0xffffffffu, row, i * 16 + 8 + g);
              KTile<D, E4M3> k;
              k.load(kb, ra ^ (ra >> 31), rb ^ (rb >> 31));
              float s[4];
              tile_scores(k, ra, rb, s);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (tok[e] == t + i) {
                  if (ra >= 0) sig[2 * pair][e] = fmaf(s[e], scale[e], beta[e]);
                  if (rb >= 0) sig[2 * pair + 1][e] = fmaf(s[2 + e], scale[e], beta[e]);
                }
              }
              if constexpr (E4M3) {
                const float va = log_scale(ra), vc = log_scale(rb);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (tok[e] == t + i)
                    m[e] = fmaxf(m[e], fmaxf(sig[2 * pair][e] + va, sig[2 * pair + 1][e] + vc));
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (i == 1 && pair * 16 + 8 >= a.n_off) continue;
              const int ra = __shfl_sync(0xffffffffu, row, (lane & 28) + 2 * i);
              const int rb = __shfl_sync(0xffffffffu, row, (lane & 28) + 2 * i + 1);
              KTile<D, E4M3> k;
              k.load(kb, ra ^ (ra >> 31), rb ^ (rb >> 31));
              float s[4];
              tile_scores(k, ra, rb, s);
              const float wb = w_[2 * pair + i], wa = 1.f - wb;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float y = rb >= 0 ? wa * s[e] + wb * s[2 + e] : s[e];
                if (ra >= 0 && tok[e] == t) sig[2 * pair + i][e] = fmaf(y, scale[e], beta[e]);
              }
              if constexpr (E4M3) {
                float va = log_scale(ra);
                if (rb >= 0) va = fmaxf(va, log_scale(rb));
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (tok[e] == t) m[e] = fmaxf(m[e], sig[2 * pair + i][e] + va);
              }
            }
          }
        }
      }
      if constexpr (!E4M3) {
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
          m[0] = fmaxf(m[0], sig[i][0]);
          m[1] = fmaxf(m[1], sig[i][1]);
        }
      }
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) {
        m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], d));
        m[1] = fmaxf(m[1], __shfl_xor_sync(0xffffffffu, m[1], d));
      }
    }

    // ---- sinks (tile -1) and window, two tiles of 16 rows at a time -------------
    const int last = pos0 + count - 1;
    const int base = max(0, pos0 - (a.W - 1));
    const int tiles = (last - base) / 16 + 1;
    for (int t0 = a.S > 0 ? -1 : 0; t0 < tiles; t0 += 2) {
      const int mine = t0 + (lane >> 4);      // the tile this lane looks a row up for
      const int r_ = mine < 0 ? lane & 15 : base + mine * 16 + (lane & 15);
      const bool in = r_ <= last && (mine < 0 ? r_ < a.S : mine < tiles);
      const int row = in ? find(r_, unused) : fill;
      const bool second = t0 + 1 < tiles;
      float s[2][4], lv[2][2];
      int rk[2][2];
      KTile<D, E4M3> k[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        rk[i][0] = __shfl_sync(0xffffffffu, row, i * 16 + g);
        rk[i][1] = __shfl_sync(0xffffffffu, row, i * 16 + 8 + g);
        if (i == 0 || second) k[i].load(kb, rk[i][0], rk[i][1]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i == 1 && !second) {
          s[1][0] = s[1][1] = s[1][2] = s[1][3] = -INFINITY;
          continue;
        }
        k[i].scores(q, s[i]);
        const int t = t0 + i;
        float ka[2] = {scale[0], scale[1]}, kc[2] = {scale[0], scale[1]};
        if constexpr (E4M3) {
          const float x0 = __ldg(ks + rk[i][0]), x1 = __ldg(ks + rk[i][1]);
          ka[0] *= x0; ka[1] *= x0; kc[0] *= x1; kc[1] *= x1;
        }
        // lags of rows r and r + 8 from the two columns' positions; sinks have no
        // far edge but a last row
        const int r = t < 0 ? g : base + t * 16 + g;
        const unsigned far = t < 0 ? 0x7fffffffu : (unsigned)a.W;
        const bool ea = t >= 0 || r < a.S, eb = t >= 0 || r + 8 < a.S;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int lag = pos0 + tok[e] - r;
          const bool on = tok[e] >= 0;
          s[i][e] = on && ea && (unsigned)lag < far ? s[i][e] * ka[e] : -INFINITY;
          s[i][2 + e] = on && eb && (unsigned)(lag - 8) < far ? s[i][2 + e] * kc[e] : -INFINITY;
        }
        if constexpr (E4M3) {
          lv[i][0] = __ldg(vs + rk[i][0]);
          lv[i][1] = __ldg(vs + rk[i][1]);
        }
      }
      float nm[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (E4M3) {
          nm[e] = -INFINITY;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (i == 0 || second) {
              nm[e] = fmaxf(nm[e], s[i][e] + __log2f(fmaxf(fabsf(lv[i][0]), 7.9e-31f)));
              nm[e] = fmaxf(nm[e], s[i][2 + e] + __log2f(fmaxf(fabsf(lv[i][1]), 7.9e-31f)));
            }
        } else {
          nm[e] = fmaxf(fmaxf(s[0][e], s[0][2 + e]), fmaxf(s[1][e], s[1][2 + e]));
        }
      }
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
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i == 1 && !second) continue;
        VTile<D, E4M3> v;
        v.load(vb, 0, __shfl_sync(0xffffffffu, row, i * 16 + 2 * c));
        v.load(vb, 1, __shfl_sync(0xffffffffu, row, i * 16 + 2 * c + 1));
        v.load(vb, 2, __shfl_sync(0xffffffffu, row, i * 16 + 2 * c + 8));
        v.load(vb, 3, __shfl_sync(0xffffffffu, row, i * 16 + 2 * c + 9));
        float p[4] = {exp2_approx(s[i][0] - z0), exp2_approx(s[i][1] - z1),
                      exp2_approx(s[i][2] - z0), exp2_approx(s[i][3] - z1)};
        l[0] += p[0] + p[2];
        l[1] += p[1] + p[3];
        if constexpr (E4M3) {
          p[0] = s[i][0] == -INFINITY ? 0.f : p[0] * lv[i][0];
          p[1] = s[i][1] == -INFINITY ? 0.f : p[1] * lv[i][0];
          p[2] = s[i][2] == -INFINITY ? 0.f : p[2] * lv[i][1];
          p[3] = s[i][3] == -INFINITY ? 0.f : p[3] * lv[i][1];
        }
        v.add(transpose8(pack16<E4M3>(p[0], p[1])), transpose8(pack16<E4M3>(p[2], p[3])), o);
      }
    }

    // ---- offset values -----------------------------------------------------------
    if constexpr (NT > 0) {
      const float z0 = m[0] == -INFINITY ? 0.f : m[0], z1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) {
        sig[i][0] = exp2_approx(sig[i][0] - z0);
        sig[i][1] = exp2_approx(sig[i][1] - z1);
        l[0] += sig[i][0];
        l[1] += sig[i][1];
      }
      Walk w[NT];
#pragma unroll
      for (int pair = 0; pair < NT; ++pair) w[pair] = {0, -1};
      for (int t = 0; t < count; t += stride) {
#pragma unroll
        for (int pair = 0; pair < NT; ++pair) {
          const int p = pos0 + t + ahead;
          int row = fill;
          if (c_[pair] <= p && t + ahead < count) {
            step_to(w[pair], p - lo_[pair], stride);
            row = w[pair].row;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // interpolated: tile i of the pair; flat: the tile of token t + i
            if (flat ? t + i >= count : (i == 1 && pair * 16 + 8 >= a.n_off)) continue;
            const int s0 = flat ? i * 16 + 2 * c : 8 * c + 2 * i;
            const int dn = flat ? 1 : 4, db = flat ? 8 : 1;      // next row; row + 8
            VTile<D, E4M3> v;
            v.load(vb, 0, __shfl_sync(0xffffffffu, row, s0));
            v.load(vb, 1, __shfl_sync(0xffffffffu, row, s0 + dn));
            v.load(vb, 2, __shfl_sync(0xffffffffu, row, s0 + db));
            v.load(vb, 3, __shfl_sync(0xffffffffu, row, s0 + dn + db));
            const int at = flat ? t + i : t;
            const bool on0 = tok[0] == at, on1 = tok[1] == at;
            float pa0, pa1, pb0, pb1;
            if (flat) {
              pa0 = sig[2 * pair][0]; pa1 = sig[2 * pair][1];
              pb0 = sig[2 * pair + 1][0]; pb1 = sig[2 * pair + 1][1];
            } else {
              const float wb = w_[2 * pair + i], wa = 1.f - wb;
              pa0 = sig[2 * pair + i][0]; pa1 = sig[2 * pair + i][1];
              pb0 = pa0 * wb; pb1 = pa1 * wb;
              pa0 *= wa; pa1 *= wa;
            }
            if constexpr (E4M3) {
              const float va = __ldg(vs + __shfl_sync(0xffffffffu, row,
                                                      flat ? i * 16 + g : (lane & 28) + 2 * i));
              const float vc = __ldg(vs + __shfl_sync(0xffffffffu, row,
                                                      flat ? i * 16 + 8 + g
                                                           : (lane & 28) + 2 * i + 1));
              pa0 = pa0 == 0.f ? 0.f : pa0 * va;
              pa1 = pa1 == 0.f ? 0.f : pa1 * va;
              pb0 = pb0 == 0.f ? 0.f : pb0 * vc;
              pb1 = pb1 == 0.f ? 0.f : pb1 * vc;
            }
            v.add(transpose8(pack16<E4M3>(on0 ? pa0 : 0.f, on1 ? pa1 : 0.f)),
                  transpose8(pack16<E4M3>(on0 ? pb0 : 0.f, on1 ? pb1 : 0.f)), o);
          }
        }
      }
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
  float odd = 0.f;      // x - x is 0 for finite x only
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    if (tok[0] >= 0) odd += (o[j][0] - o[j][0]) + (o[j][2] - o[j][2]);
    if (tok[1] >= 0) odd += (o[j][1] - o[j][1]) + (o[j][3] - o[j][3]);
  }
  if (!nan && __any_sync(0xffffffffu, odd != 0.f)) {
    for (int col = 0; col < count * a.per; ++col) {
      const int t = col / a.per, hh = col - t * a.per;
      if (hh < heads)
        one_query<__nv_bfloat16, D, E4M3>(a, layer, h * a.G + grp * a.per + hh, n0 + t, b,
                                          pos0 + t, true);
    }
    return;
  }

#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (tok[e] < 0) continue;
    const size_t at = ((size_t)layer * a.N + n0 + tok[e]) * a.Hq + head[e];
    const float bad = __int_as_float(0x7fc00000);
    const float inv = nan ? bad : 1.f / l[e];
    __nv_bfloat16* op = reinterpret_cast<__nv_bfloat16*>(a.o) + at * D;
#pragma unroll
    for (int i = 0; i < Y::VP; ++i) {
      float y[Y::VE];
#pragma unroll
      for (int j = 0; j < Y::VE / 2; ++j) {
        y[2 * j] = o[i * (Y::VE / 2) + j][e] * inv;
        y[2 * j + 1] = o[i * (Y::VE / 2) + j][2 + e] * inv;
      }
      store_row<__nv_bfloat16, Y::VE>(op + (8 * i + g) * Y::VE, y);
    }
    if (g == 0 && a.lse) a.lse[at] = nan ? bad : kLn2 * (m[e] + log2f(l[e]));
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

// One query (token row n of sequence b at position pos, query head hq) by one
// warp: members 32 at a time, and no row but its members' is touched.
template <typename QT, int D, bool E4M3>
__device__ __noinline__ void one_query(const ChunkArgs& a, int layer, int hq, int n, int b,
                                       int pos, bool inside) {
  constexpr bool BF16 = !E4M3 && sizeof(QT) == 2;
  constexpr int QE = D / 4;                        // elements of a row per quad lane
  constexpr int VE = D >= 32 ? D / 32 : 1;         // value elements per lane
  constexpr int SPLIT = D >= 32 ? 1 : 2;           // D = 16: two members at a time
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

  float q[QE];
  load_row<QT, QE>(reinterpret_cast<const QT*>(a.q) + layer * a.ql + n * a.qn + hq * a.qh +
                       part * QE, q);
  const size_t at = ((size_t)layer * a.N + n) * a.Hq + hq;
  const float beta = a.beta ? __ldg(a.beta + at) : 0.f;
  const int nw = min(a.W, pos + 1), ns = min(a.S, pos + 1);
  const int total = ok ? nw + ns + a.n_off : 0;

  float m = -INFINITY, l = 0.f, o[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) o[i] = 0.f;
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
    float s = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ia = __shfl_sync(0xffffffffu, ra, i * 8 + mm);
      const int ib = __shfl_sync(0xffffffffu, rb, i * 8 + mm);
      const float xa = __shfl_sync(0xffffffffu, ka, i * 8 + mm);
      const float xb = __shfl_sync(0xffffffffu, kc, i * 8 + mm);
      float dot = 0.f;
      if (ia >= 0) {
        float x[QE];
        load_part<E4M3, BF16, QE>(kb, D, ia, part * QE, x);
        float t = 0.f;
#pragma unroll
        for (int e = 0; e < QE; ++e) t = fmaf(q[e], x[e], t);
        dot = t * xa;
      }
      if (ib >= 0) {
        float x[QE];
        load_part<E4M3, BF16, QE>(kb, D, ib, part * QE, x);
        float t = 0.f;
#pragma unroll
        for (int e = 0; e < QE; ++e) t = fmaf(q[e], x[e], t);
        dot = fmaf(t, xb, dot);
      }
      dot += __shfl_xor_sync(0xffffffffu, dot, 1);
      dot += __shfl_xor_sync(0xffffffffu, dot, 2);
      const float mine = __shfl_sync(0xffffffffu, dot, (lane & 7) * 4);
      if ((lane >> 3) == i) s = mine;
    }
    s = ra >= 0 ? (s * a.scale + (off ? beta : 0.f)) * kLog2e : -INFINITY;
    float nm = s;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, d));
    nm = fmaxf(m, nm);
    const float z = nm == -INFINITY ? 0.f : nm;
    const float f = exp2f(m - z), p = exp2f(s - z);
    m = nm;
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < VE; ++i) o[i] *= f;
    va *= p;
    vc *= p;
    const int here = min(32, total - m0);
    for (int i = 0; i < here; i += SPLIT) {
      const int src = i + (SPLIT == 2 ? lane >> 4 : 0);
      const int ia = __shfl_sync(0xffffffffu, ra, src & 31);
      const int ib = __shfl_sync(0xffffffffu, rb, src & 31);
      const float xa = __shfl_sync(0xffffffffu, va, src & 31);
      const float xb = __shfl_sync(0xffffffffu, vc, src & 31);
      if (ia >= 0) {
        float x[VE];
        load_part<E4M3, BF16, VE>(vb, D, ia, d0, x);
#pragma unroll
        for (int e = 0; e < VE; ++e) o[e] = fmaf(xa, x[e], o[e]);
      }
      if (ib >= 0) {
        float x[VE];
        load_part<E4M3, BF16, VE>(vb, D, ib, d0, x);
#pragma unroll
        for (int e = 0; e < VE; ++e) o[e] = fmaf(xb, x[e], o[e]);
      }
    }
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  if constexpr (SPLIT == 2) o[0] += __shfl_xor_sync(0xffffffffu, o[0], 16);
  const bool nan = __any_sync(0xffffffffu, lost) || !ok;
  const float bad = __int_as_float(0x7fc00000);
  const float inv = nan ? bad : 1.f / l;
  if (D >= 32 || lane < 16) {
#pragma unroll
    for (int e = 0; e < VE; ++e) o[e] *= inv;
    store_row<QT, VE>(reinterpret_cast<QT*>(a.o) + at * D + d0, o);
  }
  if (lane == 0 && a.lse) a.lse[at] = nan ? bad : kLn2 * m + logf(l);
  if (lost) atomicOr(&g_chunk_err, kErrPage);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) k_chunk_f32(const __grid_constant__ ChunkArgs a) {
  const int n = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (n >= a.N) return;
  const int b = find_sequence(a.cu, a.B, 0, n);
  const int first = __ldg(a.cu + b);
  if (first < 0 || n < first || n >= __ldg(a.cu + b + 1)) return;
  const long long posl = (long long)__ldg(a.cached + b) + (n - first);
  const bool inside = posl >= 0 && posl < (long long)a.max_pages * a.pd.d;
  one_query<float, D, E4M3>(a, blockIdx.z, blockIdx.y, n, b, inside ? (int)posl : 0, inside);
}

template <int D, bool E4M3>
cudaError_t launch_t(const ChunkArgs& a, bool f32, cudaStream_t st) {
  trace_mark("chunk_attn", st, true);
  if (f32) {
    const dim3 grid((a.N + kWarps - 1) / kWarps, a.Hq, a.L);
    k_chunk_f32<D, E4M3><<<grid, kWarps * 32, 0, st>>>(a);
  } else {
    const dim3 grid((a.blocks + kWarps - 1) / kWarps, a.Hkv * a.groups, a.L);
    if (a.n_off == 0)
      k_chunk_tc<D, E4M3, 0><<<grid, kWarps * 32, 0, st>>>(a);
    else if (a.n_off <= 16)
      k_chunk_tc<D, E4M3, 1><<<grid, kWarps * 32, 0, st>>>(a);
    else
      k_chunk_tc<D, E4M3, 2><<<grid, kWarps * 32, 0, st>>>(a);
  }
  trace_mark("chunk_attn", st, false);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk_attn(const PagedProblem& p, const PagedPtrs& c, const ChunkPtrs& x,
                              cudaStream_t st) {
  ChunkArgs a = {};
  a.L = p.L; a.N = p.N; a.B = p.B; a.Hq = p.Hq; a.Hkv = p.Hkv; a.n_pages = p.n_pages;
  a.max_pages = p.max_pages;
  a.W = x.W; a.n_off = x.n_off; a.S = x.S; a.scale = x.scale;
  for (int k = 0; k < x.n_off; ++k) a.f[k] = x.f[k];
  a.pd = fast_div(p.page_size);
  a.ql = x.qs.layer; a.qn = x.qs.row; a.qh = x.qs.head;
  a.q = x.q; a.kc = c.k; a.vc = c.v; a.ks = c.k_scale; a.vs = c.v_scale;
  a.alpha = x.alpha; a.beta = x.beta;
  a.table = c.table; a.cu = x.cu_q; a.cached = x.cached;
  a.o = x.o; a.lse = x.lse;
  // columns: the heads of a key/value head in equal groups of at most 8, and
  // as many tokens as fill 8 columns (a power of two, for find_sequence)
  a.G = p.Hq / p.Hkv;
  a.groups = (a.G + 7) / 8;
  a.per = (a.G + a.groups - 1) / a.groups;
  a.shift = a.per == 1 ? 3 : (a.per == 2 ? 2 : (a.per <= 4 ? 1 : 0));
  a.blocks = a.shift ? (p.N >> a.shift) + p.B : p.N;
  const bool f32 = p.dtype == SA_DTYPE_F32, q8 = p.format == SA_CACHE_E4M3;
  switch (p.D) {
    case 16: return q8 ? launch_t<16, true>(a, f32, st) : launch_t<16, false>(a, f32, st);
    case 32: return q8 ? launch_t<32, true>(a, f32, st) : launch_t<32, false>(a, f32, st);
    case 64: return q8 ? launch_t<64, true>(a, f32, st) : launch_t<64, false>(a, f32, st);
    default: return q8 ? launch_t<128, true>(a, f32, st) : launch_t<128, false>(a, f32, st);
  }
}

cudaError_t chunk_read_error(unsigned* out, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_chunk_err, sizeof(unsigned));
  if (e != cudaSuccess || !clear || *out == 0) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_chunk_err, &zero, sizeof(unsigned));
}

}  // namespace sa
