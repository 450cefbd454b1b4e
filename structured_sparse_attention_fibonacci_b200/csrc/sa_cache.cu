// The paged key/value cache: new tokens are written into its pages (with the
// norm and the rotation of their queries and keys in the same pass), and the
// rows of whole sequences are read back.
//
// Append. Per token row n of sequence b at position pos = cached[b] + n -
// cu_q[b], with RoPE as in the forward (rotate-half pairs, integer positions):
//   q'_h = R(pos) norm(q_h; q_weight),  k'_h = R(pos) norm(k_h; k_weight),
//   norm(x; w) = x / sqrt(mean(x^2) + eps) * w   (without weights: x),
// q' is returned; k' and v go to slot pos % page_size of page
// page_table[b][pos / page_size]. 8-bit rows hold e4m3 codes of x / s and s.
// Keys are kept rotated: a row is rotated once when written instead of by each
// of the ~W + 30 queries that read it.
//
// Bound: HBM bytes (16 flops per loaded pair). One warp per (token, layer):
// D/16 lanes hold one head's row, 16 elements each (8 pairs j, j + D/2), so the
// rotation stays inside a lane and the cosines, loaded once per warp, serve
// every head of the token; the norm and the 8-bit maximum cost log2(D/16)
// shuffles. A decode step has few tokens: the rows are then split over
// `parts` warps per token. Measured with the norm for 5446 tokens x 4 layers of 32 +
// 8 heads of 128: into e4m3 491 MB in 92 us, 5.4 TB/s of 6.55, into plain bf16 pages 93
// us; fp32 170 us into plain pages, 151 into e4m3. 16384 tokens x 4 layers of 8 + 8
// heads of 64: e4m3 84 us (68 without the norm), plain bf16 82 (70), fp32 into plain
// pages 128 (123). Half the issue slots go to the norm, the rotation and the
// conversions.
#include "sa_paged.cuh"

namespace sa {

namespace {

__device__ unsigned g_cache_err;

constexpr int kAppendWarps = 4;

struct AppendArgs {
  int N, B, Hq, Hkv, n_pages, max_pages, parts;
  FastDiv pd;
  float eps;
  int64_t ql, qn, qh, kl, kn, kh, vl, vn, vh;     // strides in elements
  const void* q; const void* k; const void* v;
  const float* qw; const float* kw;
  const int* table; const int* cu; const int* cached;
  const float2* rope;
  void* q_out; void* kc; void* vc; float* ks; float* vs;
};

// A thread's copies in flight: its own 16 elements of the next rows, as 16-byte chunks
// in slots of shared memory that no other thread touches (so no barrier is needed).
// (Two rows a thread in registers, beside the 60 that the arithmetic takes, and five CTAs
// per SM: 103 us where this takes 91; four stages 94, seven CTAs 99, eight 115: spills.)
template <typename T>
struct Ahead {
  static constexpr int kChunks = sizeof(T);      // 8 elements from j0, 8 from j0 + D / 2
  static constexpr int kStages = sizeof(T) == 2 ? 3 : 2;
  static constexpr int kStage = kChunks * kAppendWarps * 32 * 16;
  // (fp32: half a sector at a time, so through the L1)
  static __device__ __forceinline__ void copy(uint32_t dst, const T* src) {
    if constexpr (sizeof(T) == 2)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  }
};
template <typename T>
__device__ __forceinline__ void read8(const uint8_t* slot, float (&x)[8]) {
#pragma unroll
  for (int c = 0; c < (int)sizeof(T) / 2; ++c) {
    const uint4 u = *reinterpret_cast<const uint4*>(slot + c * kAppendWarps * 32 * 16);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (sizeof(T) == 4) {
        x[4 * c + e] = __uint_as_float(w[e]);
      } else {
        x[2 * e] = bf16lo(w[e]);
        x[2 * e + 1] = bf16hi(w[e]);
      }
    }
  }
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <typename T, int D, bool E4M3, bool NORM>
__global__ void __launch_bounds__(kAppendWarps * 32, 6) k_cache_append(const AppendArgs a) {
  constexpr int LANES = D / 16, ROWS = 32 / LANES, HALF = D / 2;
  using Y = Ahead<T>;
  __shared__ __align__(16) uint8_t s_ring[Y::kStages * Y::kStage];
  const int lane = threadIdx.x & 31, sub = lane % LANES, grp = lane / LANES;
  const long long wid = (long long)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int layer = blockIdx.y;
  if (wid >= (long long)a.N * a.parts) return;
  const int n = (int)(wid / a.parts), part = (int)(wid % a.parts);
  const int j0 = sub * 8;
  const int rows = a.Hq + 2 * a.Hkv, stride = a.parts * ROWS;
  const T* q = reinterpret_cast<const T*>(a.q) + layer * a.ql + n * a.qn + j0;
  const T* k = reinterpret_cast<const T*>(a.k) + layer * a.kl + n * a.kn + j0;
  const T* v = reinterpret_cast<const T*>(a.v) + layer * a.vl + n * a.vn + j0;
  // Rows in turn: q heads, k heads, v heads. Every group of the warp takes part in
  // the shuffles; one without a row takes the last one again and does not store it.
  int next = part * ROWS, slot_in = 0, slot = 0;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(s_ring) + threadIdx.x * 16;
  auto issue = [&]() {
    if (next < rows) {
      const int r = min(next + grp, rows - 1);
      const T* from = r < a.Hq           ? q + r * a.qh
                      : r < a.Hq + a.Hkv ? k + (r - a.Hq) * a.kh
                                         : v + (r - a.Hq - a.Hkv) * a.vh;
#pragma unroll
      for (int c = 0; c < Y::kChunks; ++c)
        Y::copy(mine + slot_in + c * kAppendWarps * 32 * 16,
                from + c / (Y::kChunks / 2) * HALF + c % (Y::kChunks / 2) * (16 / (int)sizeof(T)));
      next += stride;
      slot_in = slot_in + Y::kStage == Y::kStages * Y::kStage ? 0 : slot_in + Y::kStage;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < Y::kStages - 1; ++i) issue();      // before the sequence is known

  const int b = find_sequence(a.cu, a.B, 0, n);
  const int first = __ldg(a.cu + b);
  if (n < first || n >= __ldg(a.cu + b + 1)) {      // a row behind the last sequence
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  const long long pos = (long long)__ldg(a.cached + b) + (n - first);
  const bool inside = pos >= 0 && pos < (long long)a.max_pages * a.pd.d;
  int page = -1, lp = 0;
  if (inside) {
    lp = quotient(a.pd, (int)pos);
    page = __ldg(a.table + (size_t)b * a.max_pages + lp);
  }
  const bool have = (unsigned)page < (unsigned)a.n_pages;
  if (!have && lane == 0) atomicOr(&g_cache_err, kErrPage);

  float2 cs[8];
  if (inside) {
    load_cs<8>(a.rope + (size_t)pos * HALF + j0, cs);
  } else {      // no such position: the query becomes NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = make_float2(__int_as_float(0x7fc00000), 0.f);
  }
  const int row_slot = (int)pos - lp * a.pd.d;
  float w1[8], w2[8];
  int weights_of = -1;
#pragma unroll 1
  for (int r0 = part * ROWS; r0 < rows; r0 += stride) {
    issue();
    asm volatile("cp.async.wait_group %0;" ::"n"(Y::kStages - 1) : "memory");
    const uint8_t* from = s_ring + slot + threadIdx.x * 16;
    slot = slot + Y::kStage == Y::kStages * Y::kStage ? 0 : slot + Y::kStage;
    const bool live = r0 + grp < rows;
    const int r = min(r0 + grp, rows - 1);
    const int what = r < a.Hq ? 0 : (r < a.Hq + a.Hkv ? 1 : 2);       // q, k, v
    float x1[8], x2[8];
    read8<T>(from, x1);
    read8<T>(from + Y::kStage / 2, x2);
    if constexpr (NORM) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x1[i], x1[i], fmaf(x2[i], x2[i], ss));
      ss = group_sum<LANES>(ss);
      if (what < 2) {
        if (weights_of != what) {
          const float* w = (what == 0 ? a.qw : a.kw) + (size_t)layer * D + j0;
          load_row<float, 8>(w, w1);
          load_row<float, 8>(w + HALF, w2);
          weights_of = what;
        }
        const float rstd = inverse_sqrt(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x1[i] = x1[i] * rstd * w1[i];
          x2[i] = x2[i] * rstd * w2[i];
        }
      }
    }
    if (what < 2) rope_fwd<8>(x1, x2, cs);
    if (what == 0) {      // (a lane group without a row is never here: v rows are last)
      T* dst = reinterpret_cast<T*>(a.q_out) + (((size_t)layer * a.N + n) * a.Hq + r) * D + j0;
      store_row<T, 8>(dst, x1);
      store_row<T, 8>(dst + HALF, x2);
    }
    if (r0 + ROWS <= a.Hq) continue;      // queries only (uniform)
    float scale = 1.f;
    if constexpr (E4M3) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max_nan(m, max_nan(fabsf(x1[i]), fabsf(x2[i])));
      scale = e4m3_scale(group_max<LANES>(m));
    }
    if (what > 0 && live && have) {
      const int h = what == 1 ? r - a.Hq : r - a.Hq - a.Hkv;
      const size_t row = (((size_t)layer * a.n_pages + page) * a.Hkv + h) * a.pd.d + row_slot;
      if constexpr (E4M3) {
        const float inv = 1.f / scale;     // a power of two: exact
        uint8_t* dst = reinterpret_cast<uint8_t*>(what == 1 ? a.kc : a.vc) + row * D + j0;
        uint2 u;
        u.x = float4_to_e4m3x4(x1[0] * inv, x1[1] * inv, x1[2] * inv, x1[3] * inv);
        u.y = float4_to_e4m3x4(x1[4] * inv, x1[5] * inv, x1[6] * inv, x1[7] * inv);
        *reinterpret_cast<uint2*>(dst) = u;
        u.x = float4_to_e4m3x4(x2[0] * inv, x2[1] * inv, x2[2] * inv, x2[3] * inv);
        u.y = float4_to_e4m3x4(x2[4] * inv, x2[5] * inv, x2[6] * inv, x2[7] * inv);
        *reinterpret_cast<uint2*>(dst + HALF) = u;
        if (sub == 0) (what == 1 ? a.ks : a.vs)[row] = scale;
      } else {
        T* dst = reinterpret_cast<T*>(what == 1 ? a.kc : a.vc) + row * D + j0;
        store_row<T, 8>(dst, x1);
        store_row<T, 8>(dst + HALF, x2);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Read back: rows 0 .. lengths[b] - 1 of every sequence, both tensors, to
// contiguous [L][B][Hkv][rows][D]; rows from lengths[b] on stay as they are.
// Bound: HBM bytes. D/8 lanes per row, so that a warp's 16-byte stores are
// contiguous; a thread moves kReadRows rows of both tensors, loads first. 4 x 8192 rows
// x 16 layers x 8 heads of 64: e4m3 to bf16 248 us (floor 251 at the copy rate of 6.55
// TB/s, a reference and not a bound: this reads a third of what it moves), plain bf16
// 320 (328), e4m3 to fp32 531 (415).
constexpr int kReadThreads = 256;
constexpr int kReadRows = 4;

struct ReadArgs {
  int B, Hkv, n_pages, max_pages, rows;
  FastDiv pd;
  const int* table; const int* lengths;
  const void* kc; const void* vc; const float* ks; const float* vs;
  void* k; void* v;
};

template <typename T, bool E4M3>
struct Held {      // 8 elements of a cache row and its scale
  uint4 u, u2;
  float s;
};

template <typename T, bool E4M3, int D>
__device__ __forceinline__ void fetch(const void* c, const float* sc, size_t row, int e0,
                                      Held<T, E4M3>& x) {
  if constexpr (E4M3) {
    const uint2 t = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(c) +
                                                         row * D + e0));
    x.u.x = t.x; x.u.y = t.y;
    x.s = __ldg(sc + row);
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(c) + row * D + e0);
    x.u = __ldg(p);
    if constexpr (sizeof(T) == 4) x.u2 = __ldg(p + 1);
  }
}

template <typename T, bool E4M3>
__device__ __forceinline__ void put(T* dst, const Held<T, E4M3>& x) {
  if constexpr (E4M3) {
    float f[8];
    e4m3x2_to_float2(x.u.x & 0xffffu, f[0], f[1]);
    e4m3x2_to_float2(x.u.x >> 16, f[2], f[3]);
    e4m3x2_to_float2(x.u.y & 0xffffu, f[4], f[5]);
    e4m3x2_to_float2(x.u.y >> 16, f[6], f[7]);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= x.s;
    store_row<T, 8>(dst, f);
  } else {
    *reinterpret_cast<uint4*>(dst) = x.u;
    if constexpr (sizeof(T) == 4) reinterpret_cast<uint4*>(dst)[1] = x.u2;
  }
}

template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(kReadThreads) k_cache_read(const ReadArgs a) {
  constexpr int LANES = D / 8, PER = kReadThreads / LANES;      // rows per pass of the CTA
  const int e0 = (threadIdx.x % LANES) * 8, g = threadIdx.x / LANES;
  const int b = blockIdx.y / a.Hkv, h = blockIdx.y % a.Hkv, layer = blockIdx.z;
  const int len = min(__ldg(a.lengths + b), a.rows);
  const int r0 = blockIdx.x * (PER * kReadRows) + g;
  const int* table = a.table + (size_t)b * a.max_pages;
  const size_t base = (size_t)layer * a.n_pages * a.Hkv * a.pd.d;
  const long long cap = (long long)a.max_pages * a.pd.d;
  Held<T, E4M3> k[kReadRows], v[kReadRows];
  int at[kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int r = r0 + i * PER;
    at[i] = (r < len && r < cap) ? pool_row(table, a.pd, r, a.n_pages, a.Hkv, h) : -1;
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i)
    if (at[i] >= 0) {
      fetch<T, E4M3, D>(a.kc, a.ks, base + at[i], e0, k[i]);
      fetch<T, E4M3, D>(a.vc, a.vs, base + at[i], e0, v[i]);
    }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int r = r0 + i * PER;
    if (r >= len) continue;
    const size_t out = ((((size_t)layer * a.B + b) * a.Hkv + h) * a.rows + r) * D + e0;
    T* ko = reinterpret_cast<T*>(a.k) + out;
    T* vo = reinterpret_cast<T*>(a.v) + out;
    if (at[i] >= 0) {
      put<T, E4M3>(ko, k[i]);
      put<T, E4M3>(vo, v[i]);
    } else {      // no such page: NaN, and the error word
      float nan[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) nan[e] = __int_as_float(0x7fc00000);
      store_row<T, 8>(ko, nan);
      store_row<T, 8>(vo, nan);
      atomicOr(&g_cache_err, kErrPage);
    }
  }
}

template <typename T, int D, bool E4M3>
cudaError_t append_t(const AppendArgs& a, int L, bool norm, cudaStream_t st) {
  const long long warps = (long long)a.N * a.parts;
  const dim3 grid((unsigned)((warps + kAppendWarps - 1) / kAppendWarps), L);
  trace_mark("cache_append", st, true);
  if (norm)
    k_cache_append<T, D, E4M3, true><<<grid, kAppendWarps * 32, 0, st>>>(a);
  else
    k_cache_append<T, D, E4M3, false><<<grid, kAppendWarps * 32, 0, st>>>(a);
  trace_mark("cache_append", st, false);
  return cudaGetLastError();
}

template <typename T, int D, bool E4M3>
cudaError_t read_t(const ReadArgs& a, int L, cudaStream_t st) {
  constexpr int per = kReadThreads / (D / 8) * kReadRows;
  const dim3 grid((a.rows + per - 1) / per, a.B * a.Hkv, L);
  trace_mark("cache_read", st, true);
  k_cache_read<T, E4M3, D><<<grid, kReadThreads, 0, st>>>(a);
  trace_mark("cache_read", st, false);
  return cudaGetLastError();
}

}  // namespace

#define SA_BY_TYPE(FN, p, ...)                                                          \
  const bool f32 = (p).dtype == SA_DTYPE_F32, q8 = (p).format == SA_CACHE_E4M3;         \
  switch ((p).D) {                                                                      \
    case 16: SA_BY_TYPE_D(FN, 16, __VA_ARGS__)                                          \
    case 32: SA_BY_TYPE_D(FN, 32, __VA_ARGS__)                                          \
    case 64: SA_BY_TYPE_D(FN, 64, __VA_ARGS__)                                          \
    default: SA_BY_TYPE_D(FN, 128, __VA_ARGS__)                                         \
  }
#define SA_BY_TYPE_D(FN, DD, ...)                                                       \
  if (f32) return q8 ? FN<float, DD, true>(__VA_ARGS__) : FN<float, DD, false>(__VA_ARGS__); \
  return q8 ? FN<__nv_bfloat16, DD, true>(__VA_ARGS__) : FN<__nv_bfloat16, DD, false>(__VA_ARGS__);

cudaError_t launch_cache_append(const PagedProblem& p, const PagedPtrs& c, const AppendPtrs& x,
                                cudaStream_t st) {
  AppendArgs a = {};
  a.N = p.N; a.B = p.B; a.Hq = p.Hq; a.Hkv = p.Hkv; a.n_pages = p.n_pages;
  a.max_pages = p.max_pages;
  a.pd = fast_div(p.page_size);
  a.eps = x.eps;
  a.ql = x.qs.layer; a.qn = x.qs.row; a.qh = x.qs.head;
  a.kl = x.ks.layer; a.kn = x.ks.row; a.kh = x.ks.head;
  a.vl = x.vs.layer; a.vn = x.vs.row; a.vh = x.vs.head;
  a.q = x.q; a.k = x.k; a.v = x.v; a.qw = x.q_weight; a.kw = x.k_weight;
  a.table = c.table; a.cu = x.cu_q; a.cached = x.cached; a.rope = x.rope;
  a.q_out = x.q_out; a.kc = c.k; a.vc = c.v; a.ks = c.k_scale; a.vs = c.v_scale;
  // few tokens: one pass over the rows per warp
  const int per = 512 / p.D, passes = (p.Hq + 2 * p.Hkv + per - 1) / per;
  a.parts = 1;
  while (a.parts < passes && (long long)p.N * p.L * a.parts < 148 * 16) a.parts *= 2;
  if (a.parts > passes) a.parts = passes;
  const bool norm = x.q_weight != nullptr;
  SA_BY_TYPE(append_t, p, a, p.L, norm, st)
}

cudaError_t launch_cache_read(const PagedProblem& p, const PagedPtrs& c, const int* lengths,
                              int rows, void* k, void* v, cudaStream_t st) {
  ReadArgs a = {};
  a.B = p.B; a.Hkv = p.Hkv; a.n_pages = p.n_pages; a.max_pages = p.max_pages; a.rows = rows;
  a.pd = fast_div(p.page_size);
  a.table = c.table; a.lengths = lengths;
  a.kc = c.k; a.vc = c.v; a.ks = c.k_scale; a.vs = c.v_scale;
  a.k = k; a.v = v;
  SA_BY_TYPE(read_t, p, a, p.L, st)
}

cudaError_t cache_read_error(unsigned* out, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_cache_err, sizeof(unsigned));
  if (e != cudaSuccess || !clear || *out == 0) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_cache_err, &zero, sizeof(unsigned));
}

}  // namespace sa
