// Attention of a chunk of new tokens over the paged cache: choice of the kernel
// instance. The kernels are in sa_chunk.cuh.
#include <algorithm>

#include "sa_chunk.cuh"

namespace sa {

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
  a.inv_per = (256 + a.per - 1) / a.per;
  a.shift = a.per == 1 ? 3 : (a.per == 2 ? 2 : (a.per <= 4 ? 1 : 0));
  a.blocks = a.shift ? (p.N >> a.shift) + p.B : p.N;
  const long long warps = (long long)a.blocks * a.Hkv * a.groups * a.L;
  const long long rows = std::min((long long)x.W, (long long)p.max_pages * p.page_size) +
                         (1 << a.shift) - 1;
  // Few blocks, as in a decode step, and a window of three tiles or more (the sinks
  // are one): a CTA's warps share a block while all CTAs are resident at once, four
  // per SM, of plain rows of 128 three. One token each of 8 sequences of 16 heads of 64
  // with 4 sinks (128 blocks): 8.4 -> 6.4 us at window 64, 14.5 -> 8.3 at 256, 38 -> 12
  // at 1024; of 32 sequences (512 blocks) 8.9 -> 7.2, 14.8 -> 9.6, 42 -> 26. Past the
  // limit (640 blocks) a block per warp: 9.3 us where sharing takes 11.2 at window 64,
  // 16.2 against 16.4 at 256, 45 against 44 at 1024. (Blocks are estimated here, up to
  // an eighth too many. With a window of one pair of tiles the join costs what it
  // saves.)
  // Clusters of two, four or eight CTAs share it where each of their warps has more
  // than four pairs left (one token, 16 heads, window 512: 10.8 us by one CTA, 8.7 by
  // two; 1024: 15.4 and 9.2; 4096: 46 by one, 13.1 by eight).
  const bool f32 = p.dtype == SA_DTYPE_F32, q8 = p.format == SA_CACHE_E4M3;
  const long long tiles = (rows + 15) / 16 + (x.S > 0), pairs = (tiles + 1) / 2;
  const long long room = 148 * (p.D == 128 && !q8 ? 3 : 4);
  a.team = tiles >= 3 && warps <= room ? 1 : 0;
  while (a.team > 0 && a.team < 8 && pairs > 4 * (4 * a.team - 1) && warps * a.team * 2 <= room)
    a.team *= 2;
  switch (p.D) {
    case 16: return launch_chunk_of<16>(a, f32, q8, st);
    case 32: return launch_chunk_of<32>(a, f32, q8, st);
    case 64: return launch_chunk_of<64>(a, f32, q8, st);
    default: return launch_chunk_of<128>(a, f32, q8, st);
  }
}

cudaError_t chunk_read_error(unsigned* out, bool clear) {
  unsigned w[4] = {0, 0, 0, 0};
  cudaError_t e = chunk_error_of<16>(w, clear);
  if (e == cudaSuccess) e = chunk_error_of<32>(w + 1, clear);
  if (e == cudaSuccess) e = chunk_error_of<64>(w + 2, clear);
  if (e == cudaSuccess) e = chunk_error_of<128>(w + 3, clear);
  *out = w[0] | w[1] | w[2] | w[3];
  return e;
}

}  // namespace sa
