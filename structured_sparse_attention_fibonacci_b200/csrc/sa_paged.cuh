// Device helpers of the paged key/value cache: where a row lies, which
// sequence a new token belongs to, and the 8-bit rows.
//
// Layout (include/sparse_attn.h): pages [L][n_pages][Hkv][page_size][D], so
// that the rows of one head inside a page are contiguous: a query's window and
// the two rows of an interpolated offset are then runs of whole rows.
#pragma once

#include <cuda_fp8.h>

#include "sa_device.cuh"
#include "sa_internal.h"

namespace sa {

// n / d for 0 <= n < 2^31 by one multiplication: with l = ceil(log2 d) and
// mul = ceil(2^(31+l) / d) < 2^32 the error n * (mul * d - 2^(31+l)) stays below
// 2^(31+l), so floor(n * mul / 2^(31+l)) is exact.
struct FastDiv {
  uint32_t mul, shift;
  int d;
};
inline FastDiv fast_div(int d) {
  uint32_t l = 0;
  while ((1ll << l) < d) ++l;
  FastDiv f;
  f.d = d;
  f.shift = l;
  f.mul = (uint32_t)(((1ull << (31 + l)) + (uint64_t)d - 1) / (uint64_t)d);
  return f;
}
__device__ __forceinline__ int quotient(const FastDiv& f, int n) {
  return (int)(__umulhi((uint32_t)n * 2u, f.mul) >> f.shift);
}

// Device error word bits of the paged kernels.
constexpr unsigned kErrPage = 8u;    // a page index or a position outside its range

// Page-pool row of position r of a sequence for key/value head h, inside one
// layer's pool, or -1 when the page table names no such page.
__device__ __forceinline__ int pool_row(const int* __restrict__ table_row, const FastDiv& pd, int r,
                                        int n_pages, int Hkv, int h) {
  const int lp = quotient(pd, r);
  const int page = __ldg(table_row + lp);
  if ((unsigned)page >= (unsigned)n_pages) return -1;
  return (page * Hkv + h) * pd.d + (r - lp * pd.d);
}

// The last b in [0, B) with (cu[b] >> shift) + (shift ? b : 0) <= x: with
// shift = 0 the sequence that row x belongs to (rows cu[b] .. cu[b+1]-1); with
// shift > 0 the sequence of block x, when every sequence's rows are cut into
// blocks of 2^shift and sequence b's blocks start at (cu[b] >> shift) + b. (A
// sequence of n rows has ceil(n / 2^shift) blocks, at most the distance to the
// next start, so starts need no prefix sum; unused block numbers hold none.)
// All 32 lanes take part; 32 candidates per step.
__device__ __forceinline__ int find_sequence(const int* __restrict__ cu, int B, int shift, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const long long idx = (long long)lo + (long long)lane * step;
    const bool le = idx < hi && (__ldg(cu + idx) >> shift) + (shift ? (int)idx : 0) <= x;
    const unsigned m = __ballot_sync(0xffffffffu, le) | 1u;
    lo += (31 - __clz(m)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// ---- 8-bit rows -------------------------------------------------------------
// Smallest power of two s >= 2^-100 with amax / s <= 448, the largest e4m3
// value: 448 = 1.75 * 2^8, so the exponent of amax = m 2^E goes down by 8 where
// m <= 1.75 and by 7 where it is above; the addition carries exactly then. A
// power of two keeps the division exact and costs nothing in a floating-point
// code: relative steps are the same under any scale, only the subnormal floor
// moves. NaN where amax is not finite.
__device__ __forceinline__ float e4m3_scale(float amax) {
  if (!(amax < INFINITY)) return __int_as_float(0x7fc00000);
  int e = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 127 - 8;
  e = max(e, -100);
  return __int_as_float((e + 127) << 23);
}

// Two e4m3 codes (low byte first) to fp32; exact, NaN kept.
__device__ __forceinline__ void e4m3x2_to_float2(uint32_t two, float& a, float& b) {
  uint32_t h;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(h) : "r"(two));
  const __half2 x = *reinterpret_cast<const __half2*>(&h);
  a = __low2float(x);
  b = __high2float(x);
}

// Four fp32 values to four e4m3 codes, first in the low byte.
__device__ __forceinline__ uint32_t float4_to_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

}  // namespace sa
