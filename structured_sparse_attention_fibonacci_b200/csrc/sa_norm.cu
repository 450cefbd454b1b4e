// Norms of queries and keys per head, with the position rotation in the same
// pass, and their gradients. For every row x (head dim D) of q and k:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = R(pos) (n * w)
// with one weight vector per layer and tensor, R the rotate-half rotation at the
// row's position (left out where the attention that follows rotates by itself,
// as sparse_attn_fwd does). Backward, g = R(pos)^T dy:
//   dw = sum over rows of g * n,   dx = r (g w - n mean(g w n)).
//
// Bound: HBM bytes (x, y; backward x, dy, dx): about 8 and 16 flops per element
// against the ~11 an element's 2 to 4 bytes allow on the fp32 pipe. D/16 lanes
// hold a row, 16 elements each (8 pairs j, j + D/2): two 16-byte loads of a bf16
// row per lane, log2(D/16) shuffles per sum, and the rotation inside a lane. A
// lane group walks the heads of one token, so that its cosines are loaded once.
// The backward accumulates dw in registers over all rows a thread sees, then per
// CTA in shared memory; a second kernel adds the CTAs' partials in a fixed order
// and in 64 bits (no atomics: results do not depend on scheduling).
#include <algorithm>

#include "sa_device.cuh"
#include "sa_internal.h"

namespace sa {

namespace {

constexpr int kThreads = 256;

struct NormArgs {
  int Hq, Hkv, T, tokens, pos0, chunk, n_q;      // tokens = B * T
  float eps;
  sa_head_strides qs, ks, dqs, dks;
  const void* q; const void* k; const float* qw; const float* kw;
  const void* dqo; const void* dko;              // backward: gradients of the outputs
  void* qo; void* ko;                            // outputs, or dq and dk
  const float2* rope;
  float* part;                                   // [L][blocks][D]
};

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D>
__device__ __forceinline__ float inverse_rms(const float (&x1)[8], const float (&x2)[8],
                                             float eps) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(x1[i], x1[i], fmaf(x2[i], x2[i], s));
  return inverse_sqrt(row_sum<D / 16>(s) * (1.f / D) + eps);
}

template <typename T, int D, bool NORM, bool ROT>
__global__ void __launch_bounds__(kThreads) k_qk_norm(const NormArgs a) {
  constexpr int LANES = D / 16, HALF = D / 2, PER = kThreads / LANES;
  const int j0 = (threadIdx.x % LANES) * 8, layer = blockIdx.z;
  const int p_ = blockIdx.x * PER + threadIdx.x / LANES;
  const bool live = p_ < a.tokens;
  const int p = live ? p_ : a.tokens - 1;        // idle groups recompute, and do not store
  const int b = p / a.T, t = p - b * a.T;
  float2 cs[8];
  if constexpr (ROT) load_cs<8>(a.rope + (size_t)(a.pos0 + t) * HALF + j0, cs);
  const int h1 = min(a.Hq + a.Hkv, (int)(blockIdx.y + 1) * a.chunk);
  float w1[8], w2[8];
  int have = -1;
#pragma unroll 2
  for (int hh = blockIdx.y * a.chunk; hh < h1; ++hh) {
    const bool is_k = hh >= a.Hq;
    const int h = is_k ? hh - a.Hq : hh;
    const sa_head_strides& s = is_k ? a.ks : a.qs;
    const T* src = reinterpret_cast<const T*>(is_k ? a.k : a.q) + layer * s.layer + b * s.batch +
                   h * s.head + t * s.row + j0;
    float x1[8], x2[8];
    load_row<T, 8>(src, x1);
    load_row<T, 8>(src + HALF, x2);
    if constexpr (NORM) {
      if (have != (int)is_k) {
        const float* w = (is_k ? a.kw : a.qw) + (size_t)layer * D + j0;
        load_row<float, 8>(w, w1);
        load_row<float, 8>(w + HALF, w2);
        have = is_k;
      }
      const float r = inverse_rms<D>(x1, x2, a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x1[i] = x1[i] * r * w1[i];
        x2[i] = x2[i] * r * w2[i];
      }
    }
    if constexpr (ROT) rope_fwd<8>(x1, x2, cs);
    if (live) {
      const int H = is_k ? a.Hkv : a.Hq;
      const size_t B = a.tokens / a.T;
      T* dst = reinterpret_cast<T*>(is_k ? a.ko : a.qo) +
               (((layer * B + b) * H + h) * a.T + t) * (size_t)D + j0;
      store_row<T, 8>(dst, x1);
      store_row<T, 8>(dst + HALF, x2);
    }
  }
}

// A thread's copies in flight: its own 16-byte chunks of the next rows' x and dy, in
// slots of shared memory that no other thread touches (so no barrier is needed).
// Registers would hold 16 KB an SM in flight beside the 100 that the arithmetic
// takes; at 1 us of latency 6.5 TB/s need 44 KB.
template <typename T>
struct Ahead {
  static constexpr int kChunks = sizeof(T) / 2 * 4;       // of x1, x2, dy1, dy2
  static constexpr int kStages = sizeof(T) == 2 ? 4 : 3;
  static constexpr int kBytes = kStages * kChunks * kThreads * 16;
};

template <typename T>
__device__ __forceinline__ void read8(const uint8_t* slot, float (&x)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(slot);
  if constexpr (sizeof(T) == 2) {
    x[0] = bf16lo(u.x); x[1] = bf16hi(u.x); x[2] = bf16lo(u.y); x[3] = bf16hi(u.y);
    x[4] = bf16lo(u.z); x[5] = bf16hi(u.z); x[6] = bf16lo(u.w); x[7] = bf16hi(u.w);
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(slot + kThreads * 16);
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    x[4] = __uint_as_float(v.x); x[5] = __uint_as_float(v.y);
    x[6] = __uint_as_float(v.z); x[7] = __uint_as_float(v.w);
  }
}

// CTAs 0 .. n_q - 1 of a layer take q, the rest k; each a run of consecutive
// (token tile, head) items, so that a tile's cosines serve its heads.
template <typename T, int D, bool NORM, bool ROT>
__global__ void __launch_bounds__(kThreads, 2) k_qk_norm_bwd(const NormArgs a) {
  constexpr int LANES = D / 16, HALF = D / 2, PER = kThreads / LANES;
  using Y = Ahead<T>;
  extern __shared__ __align__(16) uint8_t s_ring[];
  __shared__ float s_part[kThreads / 32][D];
  const int sub = threadIdx.x % LANES, j0 = sub * 8, layer = blockIdx.y;
  const bool is_k = (int)blockIdx.x >= a.n_q;
  const int blk = is_k ? blockIdx.x - a.n_q : blockIdx.x;
  const int blks = is_k ? gridDim.x - a.n_q : a.n_q;
  const int H = is_k ? a.Hkv : a.Hq;
  const sa_head_strides& s = is_k ? a.ks : a.qs;
  const sa_head_strides& ds = is_k ? a.dks : a.dqs;
  const T* x = reinterpret_cast<const T*>(is_k ? a.k : a.q) + layer * s.layer + j0;
  const T* dy = reinterpret_cast<const T*>(is_k ? a.dko : a.dqo) + layer * ds.layer + j0;
  const size_t B = a.tokens / a.T;
  T* dx = reinterpret_cast<T*>(is_k ? a.ko : a.qo) + (size_t)layer * B * H * a.T * D + j0;
  float w1[8], w2[8], dw1[8], dw2[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw1[i] = dw2[i] = 0.f;
  if constexpr (NORM) {
    const float* w = (is_k ? a.kw : a.qw) + (size_t)layer * D + j0;
    load_row<float, 8>(w, w1);
    load_row<float, 8>(w + HALF, w2);
  }
  const long long items = (long long)((a.tokens + PER - 1) / PER) * H;
  const long long i0 = items * blk / blks, i1 = items * (blk + 1) / blks;

  // A walk over the items; b, t: this lane group's token (the last one again, and
  // not live, behind the end).
  struct At {
    int tile, h, b, t;
    bool live;
  };
  auto place = [&](At& p) {
    const int n = p.tile * PER + threadIdx.x / LANES;
    p.live = n < a.tokens;
    const int c = p.live ? n : a.tokens - 1;
    p.b = c / a.T;
    p.t = c - p.b * a.T;
  };
  auto step = [&](At& p) {      // whether the tile changed
    if (++p.h < H) return false;
    p.h = 0;
    ++p.tile;
    place(p);
    return true;
  };
  At in;
  in.tile = (int)(i0 / H);
  in.h = (int)(i0 - (long long)in.tile * H);
  place(in);
  At at = in;
  long long next = i0;
  int slot_in = 0, slot = 0;
  auto issue = [&]() {
    if (next < i1) {
      const T* xp = x + in.b * s.batch + in.h * s.head + in.t * s.row;
      const T* gp = dy + in.b * ds.batch + in.h * ds.head + in.t * ds.row;
      const uint32_t dst = (uint32_t)__cvta_generic_to_shared(s_ring) +
                           (slot_in * Y::kChunks * kThreads + threadIdx.x) * 16;
      const T* part[4] = {xp, xp + HALF, gp, gp + HALF};
#pragma unroll
      for (int c = 0; c < Y::kChunks; ++c)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + c * kThreads * 16),
                     "l"(part[c / (Y::kChunks / 4)] + (c % (Y::kChunks / 4)) * (16 / (int)sizeof(T)))
                     : "memory");
      step(in);
      slot_in = slot_in + 1 == Y::kStages ? 0 : slot_in + 1;
    }
    ++next;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < Y::kStages - 1; ++i) issue();
  float2 cs[8];
  if constexpr (ROT) load_cs<8>(a.rope + (size_t)(a.pos0 + at.t) * HALF + j0, cs);
  for (long long it = i0; it < i1; ++it) {
    issue();      // into the slot that the last round has read
    asm volatile("cp.async.wait_group %0;" ::"n"(Y::kStages - 1) : "memory");
    const uint8_t* from = s_ring + (slot * Y::kChunks * kThreads + threadIdx.x) * 16;
    slot = slot + 1 == Y::kStages ? 0 : slot + 1;
    float x1[8], x2[8], g1[8], g2[8];
    constexpr int kHalf = Y::kChunks / 4 * kThreads * 16;
    read8<T>(from, x1);
    read8<T>(from + kHalf, x2);
    read8<T>(from + 2 * kHalf, g1);
    read8<T>(from + 3 * kHalf, g2);
    if constexpr (ROT) rope_bwd<8>(g1, g2, cs);
    if constexpr (NORM) {
      float ss = 0.f, sg = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(x1[i], x1[i], fmaf(x2[i], x2[i], ss));
        sg = fmaf(g1[i] * w1[i], x1[i], fmaf(g2[i] * w2[i], x2[i], sg));
      }
      ss = row_sum<LANES>(ss);
      sg = row_sum<LANES>(sg);
      const float r = inverse_sqrt(ss * (1.f / D) + a.eps);
      const float mean = sg * r * (1.f / D);                 // of g w n
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n1 = x1[i] * r, n2 = x2[i] * r;
        if (at.live) {
          dw1[i] = fmaf(g1[i], n1, dw1[i]);
          dw2[i] = fmaf(g2[i], n2, dw2[i]);
        }
        g1[i] = r * (g1[i] * w1[i] - n1 * mean);
        g2[i] = r * (g2[i] * w2[i] - n2 * mean);
      }
    }
    if (at.live) {
      T* dst = dx + (((size_t)at.b * H + at.h) * a.T + at.t) * D;
      store_row<T, 8>(dst, g1);
      store_row<T, 8>(dst + HALF, g2);
    }
    const bool moved = step(at);
    if (ROT && moved) load_cs<8>(a.rope + (size_t)(a.pos0 + at.t) * HALF + j0, cs);
  }
  if constexpr (NORM) {
    cudaTriggerProgrammaticLaunchCompletion();      // k_qk_norm_dw may take its place
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw1[i] += __shfl_xor_sync(0xffffffffu, dw1[i], o);
        dw2[i] += __shfl_xor_sync(0xffffffffu, dw2[i], o);
      }
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) < LANES) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s_part[warp][j0 + i] = dw1[i];
        s_part[warp][HALF + j0 + i] = dw2[i];
      }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) sum += s_part[w][d];
      a.part[((size_t)layer * gridDim.x + blockIdx.x) * D + d] = sum;
    }
  }
}

// dw of one (layer, tensor): 1024 / D slices add every (1024 / D)-th partial, then
// meet in shared memory.
constexpr int kDwThreads = 1024;
template <int D>
__global__ void __launch_bounds__(kDwThreads) k_qk_norm_dw(const float* part, int n_q, int blocks,
                                                         float* dqw, float* dkw) {
  constexpr int SL = kDwThreads / D;
  __shared__ double s_sum[SL][D];
  const int layer = blockIdx.y, d = threadIdx.x % D, sl = threadIdx.x / D;
  const bool is_k = blockIdx.x == 1;
  const int lo = is_k ? n_q : 0, hi = is_k ? blocks : n_q;
  const float* p = part + (size_t)layer * blocks * D + d;
  double sum = 0.0;
  cudaGridDependencySynchronize();      // every partial is written
#pragma unroll 8
  for (int i = lo + sl; i < hi; i += SL) sum += (double)p[(size_t)i * D];
  s_sum[sl][d] = sum;
  __syncthreads();
  if (sl == 0) {
    for (int i = 1; i < SL; ++i) sum += s_sum[i][d];
    (is_k ? dkw : dqw)[(size_t)layer * D + d] = (float)sum;
  }
}

// CTAs per layer of the backward: 1 to 4 times the 296 that the GPU holds, over all
// layers, so that a CTA has 16 items or more where there are that many; at least
// one per tensor. Long runs even out over several waves (16 x 8 x (8 + 8) x 1024 rows
// of 64: 164 us with one wave, 141 with two, 130 with four), short ones pay for
// each CTA's start and partial sums (2 x 3 x (12 + 4) x 777 rows of 128: 18, 21, 26;
// all before the early launch of the second kernel, which takes 1 to 2 us off).
// Beyond that as many as leave a CTA about 64 items: a thread adds a row of each to its
// fp32 sums of dw, whose error would else grow with the batch (it is at most (rows +
// 24) 2^-24 of the terms' sizes; the partial sums are added in 64 bits). 8 x (8 + 8) x
// 65536 rows of 64: 505 us with four waves, 497 so.
struct BwdGrid {
  int n_q, blocks;
};
BwdGrid bwd_grid(const NormProblem& p) {
  const long long per = kThreads / (p.D / 16);
  const long long tiles = ((long long)p.B * p.T + per - 1) / per;
  const long long waves =
      std::min(4LL, std::max(1LL, tiles * (p.Hq + p.Hkv) * p.L / (296 * 16)));
  const long long want = std::max({2LL, (296 * waves + p.L - 1) / p.L,
                                   (tiles * (p.Hq + p.Hkv) + 63) / 64});
  const long long q = std::max(1LL, std::min(tiles * p.Hq, want * p.Hq / (p.Hq + p.Hkv)));
  const long long k = std::max(1LL, std::min(tiles * p.Hkv, want - want * p.Hq / (p.Hq + p.Hkv)));
  return {(int)q, (int)(q + k)};
}

template <typename T, int D, bool NORM, bool ROT>
cudaError_t fwd_v(const NormArgs& a, const dim3& grid, cudaStream_t st) {
  trace_mark("qk_norm_rope", st, true);
  k_qk_norm<T, D, NORM, ROT><<<grid, kThreads, 0, st>>>(a);
  trace_mark("qk_norm_rope", st, false);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t fwd_t(const NormProblem& p, const NormArgs& a, cudaStream_t st) {
  constexpr int per = kThreads / (D / 16);
  NormArgs x = a;
  // heads walked by one lane group: up to 8 while 8 CTAs per SM remain
  const long long tiles = ((long long)a.tokens + per - 1) / per;
  const int H = p.Hq + p.Hkv;
  x.chunk = 8;
  while (x.chunk > 1 && tiles * p.L * ((H + x.chunk - 1) / x.chunk) < 148 * 8) x.chunk /= 2;
  const dim3 grid((unsigned)tiles, (H + x.chunk - 1) / x.chunk, p.L);
  if (!a.qw) return fwd_v<T, D, false, true>(x, grid, st);
  return p.rotate ? fwd_v<T, D, true, true>(x, grid, st) : fwd_v<T, D, true, false>(x, grid, st);
}

template <typename T, int D, bool NORM, bool ROT>
cudaError_t bwd_v(const NormProblem& p, const NormArgs& a, float* dqw, float* dkw, cudaStream_t st,
                  int* launches) {
  const BwdGrid g = bwd_grid(p);
  trace_mark("qk_norm_rope_bwd", st, true);
  const cudaError_t e =
      cudaFuncSetAttribute(k_qk_norm_bwd<T, D, NORM, ROT>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, Ahead<T>::kBytes);
  if (e != cudaSuccess) return e;
  k_qk_norm_bwd<T, D, NORM, ROT><<<dim3(g.blocks, p.L), kThreads, Ahead<T>::kBytes, st>>>(a);
  trace_mark("qk_norm_rope_bwd", st, false);
  ++*launches;
  if constexpr (NORM) {
    trace_mark("qk_norm_dw", st, true);
    // Launched before the first kernel has ended, and waits for it, so that its launch
    // is hidden (2 x 3 x (12 + 4) x 777 rows of 128: 17.7 -> 16.5 us).
    cudaLaunchAttribute early = {};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(2, p.L);
    c.blockDim = dim3(kDwThreads);
    c.stream = st;
    c.attrs = &early;
    c.numAttrs = 1;
    const cudaError_t dw = cudaLaunchKernelEx(&c, k_qk_norm_dw<D>, (const float*)a.part, g.n_q,
                                              g.blocks, dqw, dkw);
    if (dw != cudaSuccess) return dw;
    trace_mark("qk_norm_dw", st, false);
    ++*launches;
  }
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t bwd_t(const NormProblem& p, const NormArgs& a, float* dqw, float* dkw, cudaStream_t st,
                  int* n) {
  if (!a.qw) return bwd_v<T, D, false, true>(p, a, dqw, dkw, st, n);
  return p.rotate ? bwd_v<T, D, true, true>(p, a, dqw, dkw, st, n)
                  : bwd_v<T, D, true, false>(p, a, dqw, dkw, st, n);
}

NormArgs make_args(const NormProblem& p, const NormPtrs& x) {
  NormArgs a = {};
  a.Hq = p.Hq; a.Hkv = p.Hkv; a.T = p.T; a.tokens = p.B * p.T; a.pos0 = p.pos0; a.eps = p.eps;
  a.qs = x.qs; a.ks = x.ks; a.dqs = x.dqs; a.dks = x.dks;
  a.q = x.q; a.k = x.k; a.qw = x.q_weight; a.kw = x.k_weight;
  a.dqo = x.dq_out; a.dko = x.dk_out; a.qo = x.q_dst; a.ko = x.k_dst; a.rope = x.rope;
  return a;
}

}  // namespace

size_t qk_norm_workspace(const NormProblem& p) {
  return (size_t)p.L * bwd_grid(p).blocks * p.D * sizeof(float);
}

cudaError_t launch_qk_norm(const NormProblem& p, const NormPtrs& x, cudaStream_t st) {
  const NormArgs a = make_args(p, x);
  const bool f32 = p.dtype == SA_DTYPE_F32;
  switch (p.D) {
    case 16: return f32 ? fwd_t<float, 16>(p, a, st) : fwd_t<__nv_bfloat16, 16>(p, a, st);
    case 32: return f32 ? fwd_t<float, 32>(p, a, st) : fwd_t<__nv_bfloat16, 32>(p, a, st);
    case 64: return f32 ? fwd_t<float, 64>(p, a, st) : fwd_t<__nv_bfloat16, 64>(p, a, st);
    default: return f32 ? fwd_t<float, 128>(p, a, st) : fwd_t<__nv_bfloat16, 128>(p, a, st);
  }
}

cudaError_t launch_qk_norm_bwd(const NormProblem& p, const NormPtrs& x, float* dqw, float* dkw,
                               void* ws, cudaStream_t st, int* n) {
  NormArgs a = make_args(p, x);
  a.part = reinterpret_cast<float*>(ws);
  a.n_q = bwd_grid(p).n_q;
  const bool f32 = p.dtype == SA_DTYPE_F32;
  switch (p.D) {
    case 16: return f32 ? bwd_t<float, 16>(p, a, dqw, dkw, st, n)
                        : bwd_t<__nv_bfloat16, 16>(p, a, dqw, dkw, st, n);
    case 32: return f32 ? bwd_t<float, 32>(p, a, dqw, dkw, st, n)
                        : bwd_t<__nv_bfloat16, 32>(p, a, dqw, dkw, st, n);
    case 64: return f32 ? bwd_t<float, 64>(p, a, dqw, dkw, st, n)
                        : bwd_t<__nv_bfloat16, 64>(p, a, dqw, dkw, st, n);
    default: return f32 ? bwd_t<float, 128>(p, a, dqw, dkw, st, n)
                        : bwd_t<__nv_bfloat16, 128>(p, a, dqw, dkw, st, n);
  }
}

}  // namespace sa
