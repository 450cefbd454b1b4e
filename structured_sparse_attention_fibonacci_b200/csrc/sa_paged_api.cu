// C entry points of the query/key norm, the paged cache and the chunk attention:
// argument validation and dispatch. The contract is in include/sparse_attn.h.
#include <math.h>

#include "sa_internal.h"
#include "sparse_attn.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool usable(const void* p, uintptr_t a) { return p && aligned(p, a); }

bool head_dim(int D) { return D == 16 || D == 32 || D == 64 || D == 128; }
bool known(sa_dtype t) { return t == SA_DTYPE_F32 || t == SA_DTYPE_BF16; }
int64_t element(sa_dtype t) { return t == SA_DTYPE_F32 ? 4 : 2; }

bool rows16(const sa_head_strides* s, sa_dtype t) {
  const int64_t e = element(t);
  return s && s->layer * e % 16 == 0 && s->batch * e % 16 == 0 && s->head * e % 16 == 0 &&
         s->row * e % 16 == 0;
}
bool rows16(const sa_row_strides* s, sa_dtype t) {
  const int64_t e = element(t);
  return s && s->layer * e % 16 == 0 && s->row * e % 16 == 0 && s->head * e % 16 == 0;
}

// Weights: both (16-byte aligned) or neither.
bool weights_ok(const float* qw, const float* kw) {
  return (!qw && !kw) || (usable(qw, 16) && usable(kw, 16));
}

sa_status norm_problem(const sa_qk_norm_params* p, sa::NormProblem* x) {
  if (!p) return SA_ERR_INVALID_ARG;
  if (p->L < 1 || p->B < 0 || p->T < 0 || p->Hq < 1 || p->Hkv < 1 || p->pos0 < 0)
    return SA_ERR_INVALID_ARG;
  if (!known(p->dtype) || !(p->eps >= 0.f) || !isfinite(p->eps)) return SA_ERR_INVALID_ARG;
  if (!(p->rope_base > 0.f) || !isfinite(p->rope_base)) return SA_ERR_INVALID_ARG;
  if (!head_dim(p->D)) return SA_ERR_UNSUPPORTED;
  if ((int64_t)p->pos0 + p->T > (1 << 24)) return SA_ERR_UNSUPPORTED;
  if ((int64_t)p->B * p->T > (1LL << 30) || p->L > 65535 || (int64_t)p->Hq + p->Hkv > 65535)
    return SA_ERR_UNSUPPORTED;
  *x = {p->L, p->B, p->Hq, p->Hkv, p->T, p->D, p->pos0, p->rotate != 0, p->eps, p->dtype};
  return SA_OK;
}

sa_status paged_problem(const sa_paged_params* p, const sa_pages* c, sa::PagedProblem* x,
                        sa::PagedPtrs* y) {
  if (!p || !c) return SA_ERR_INVALID_ARG;
  if (p->L < 1 || p->N < 0 || p->B < 0 || p->Hq < 1 || p->Hkv < 1 || p->Hq % p->Hkv)
    return SA_ERR_INVALID_ARG;
  if (p->n_pages < 1 || p->page_size < 1 || p->max_pages < 1) return SA_ERR_INVALID_ARG;
  if (!known(p->dtype) || (p->format != SA_CACHE_PLAIN && p->format != SA_CACHE_E4M3))
    return SA_ERR_INVALID_ARG;
  if (!head_dim(p->D)) return SA_ERR_UNSUPPORTED;
  if ((int64_t)p->max_pages * p->page_size > (1 << 24)) return SA_ERR_UNSUPPORTED;
  if ((double)p->n_pages * p->Hkv * p->page_size >= 2147483648.0) return SA_ERR_UNSUPPORTED;
  if (p->L > 65535 || (int64_t)p->Hq + 2LL * p->Hkv > 65535) return SA_ERR_UNSUPPORTED;
  if (p->N > (1 << 30) || p->B > (1 << 30)) return SA_ERR_UNSUPPORTED;
  if (!usable(c->k, 16) || !usable(c->v, 16)) return SA_ERR_INVALID_ARG;
  if (p->format == SA_CACHE_E4M3 ? (!usable(c->k_scale, 4) || !usable(c->v_scale, 4))
                                 : (c->k_scale || c->v_scale))
    return SA_ERR_INVALID_ARG;
  if (p->B > 0 && !usable(c->page_table, 4)) return SA_ERR_INVALID_ARG;
  *x = {p->L, p->N, p->B, p->Hq, p->Hkv, p->D, p->n_pages, p->page_size, p->max_pages,
        p->dtype, p->format};
  *y = {c->k, c->v, c->k_scale, c->v_scale, c->page_table};
  return SA_OK;
}

}  // namespace

extern "C" {

size_t sparse_attn_qk_norm_workspace_size(const sa_qk_norm_params* p) {
  sa::NormProblem x;
  if (norm_problem(p, &x) != SA_OK || x.B == 0 || x.T == 0) return 0;
  return sa::qk_norm_workspace(x);
}

sa_status sparse_attn_qk_norm_rope(const sa_qk_norm_params* p, const void* q,
                                   const sa_head_strides* q_strides, const void* k,
                                   const sa_head_strides* k_strides, const float* q_weight,
                                   const float* k_weight, void* q_out, void* k_out, void* stream) {
  sa::NormProblem x;
  sa_status s = norm_problem(p, &x);
  if (s != SA_OK) return s;
  if (!weights_ok(q_weight, k_weight) || (!q_weight && !x.rotate)) return SA_ERR_INVALID_ARG;
  if (!rows16(q_strides, x.dtype) || !rows16(k_strides, x.dtype)) return SA_ERR_INVALID_ARG;
  if (x.B == 0 || x.T == 0) {
    sa::set_last_launches(0);
    return SA_OK;
  }
  if (!usable(q, 16) || !usable(k, 16) || !usable(q_out, 16) || !usable(k_out, 16))
    return SA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  sa::NormPtrs a = {};
  a.q = q; a.k = k; a.qs = *q_strides; a.ks = *k_strides;
  a.q_weight = q_weight; a.k_weight = k_weight; a.q_dst = q_out; a.k_dst = k_out;
  if (x.rotate && (s = sa::rope_table_for(x.pos0 + x.T, x.D, p->rope_base, st, &a.rope)) != SA_OK)
    return s;
  if (sa::launch_qk_norm(x, a, st) != cudaSuccess) return SA_ERR_CUDA;
  sa::set_last_launches(1);
  return SA_OK;
}

sa_status sparse_attn_qk_norm_rope_bwd(const sa_qk_norm_params* p, const void* q,
                                       const sa_head_strides* q_strides, const void* k,
                                       const sa_head_strides* k_strides, const float* q_weight,
                                       const float* k_weight, const void* dq_out,
                                       const sa_head_strides* dq_out_strides, const void* dk_out,
                                       const sa_head_strides* dk_out_strides, void* dq, void* dk,
                                       float* dq_weight, float* dk_weight, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  sa::NormProblem x;
  sa_status s = norm_problem(p, &x);
  if (s != SA_OK) return s;
  if (!weights_ok(q_weight, k_weight) || (!q_weight && !x.rotate)) return SA_ERR_INVALID_ARG;
  if (q_weight ? (!usable(dq_weight, 4) || !usable(dk_weight, 4)) : (dq_weight || dk_weight))
    return SA_ERR_INVALID_ARG;
  if (!rows16(q_strides, x.dtype) || !rows16(k_strides, x.dtype) ||
      !rows16(dq_out_strides, x.dtype) || !rows16(dk_out_strides, x.dtype))
    return SA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (x.B == 0 || x.T == 0) {
    const size_t n = (size_t)x.L * x.D * sizeof(float);
    if (q_weight && (cudaMemsetAsync(dq_weight, 0, n, st) != cudaSuccess ||
                     cudaMemsetAsync(dk_weight, 0, n, st) != cudaSuccess))
      return SA_ERR_CUDA;
    sa::set_last_launches(0);
    return SA_OK;
  }
  const void* arrays[] = {q, k, dq_out, dk_out, dq, dk};
  for (const void* a : arrays)
    if (!usable(a, 16)) return SA_ERR_INVALID_ARG;
  if (q_weight && (workspace_bytes < sa::qk_norm_workspace(x) || !usable(workspace, 16)))
    return SA_ERR_WORKSPACE;
  sa::NormPtrs a = {};
  a.q = q; a.k = k; a.qs = *q_strides; a.ks = *k_strides;
  a.q_weight = q_weight; a.k_weight = k_weight;
  a.dq_out = dq_out; a.dk_out = dk_out; a.dqs = *dq_out_strides; a.dks = *dk_out_strides;
  a.q_dst = dq; a.k_dst = dk;
  if (x.rotate && (s = sa::rope_table_for(x.pos0 + x.T, x.D, p->rope_base, st, &a.rope)) != SA_OK)
    return s;
  int launches = 0;
  if (sa::launch_qk_norm_bwd(x, a, dq_weight, dk_weight, workspace, st, &launches) != cudaSuccess)
    return SA_ERR_CUDA;
  sa::set_last_launches(launches);
  return SA_OK;
}

sa_status sparse_attn_cache_append(const sa_paged_params* p, const sa_pages* pages,
                                   const int32_t* cu_q, const int32_t* cached, const void* q,
                                   const sa_row_strides* q_strides, const void* k,
                                   const sa_row_strides* k_strides, const void* v,
                                   const sa_row_strides* v_strides, const float* q_weight,
                                   const float* k_weight, float eps, float rope_base, void* q_out,
                                   void* stream) {
  sa::PagedProblem x;
  sa::PagedPtrs c;
  sa_status s = paged_problem(p, pages, &x, &c);
  if (s != SA_OK) return s;
  if (!weights_ok(q_weight, k_weight) || !(eps >= 0.f) || !isfinite(eps)) return SA_ERR_INVALID_ARG;
  if (!(rope_base > 0.f) || !isfinite(rope_base)) return SA_ERR_INVALID_ARG;
  if (!rows16(q_strides, x.dtype) || !rows16(k_strides, x.dtype) || !rows16(v_strides, x.dtype))
    return SA_ERR_INVALID_ARG;
  if (x.N == 0 || x.B == 0) {
    sa::set_last_launches(0);
    return SA_OK;
  }
  if (!usable(q, 16) || !usable(k, 16) || !usable(v, 16) || !usable(q_out, 16) ||
      !usable(cu_q, 4) || !usable(cached, 4))
    return SA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  sa::AppendPtrs a = {q, k, v, *q_strides, *k_strides, *v_strides, q_weight, k_weight, eps,
                      cu_q, cached, nullptr, q_out};
  if ((s = sa::rope_table_for(x.max_pages * x.page_size, x.D, rope_base, st, &a.rope)) != SA_OK)
    return s;
  if (sa::launch_cache_append(x, c, a, st) != cudaSuccess) return SA_ERR_CUDA;
  sa::set_last_launches(1);
  return SA_OK;
}

sa_status sparse_attn_cache_read(const sa_paged_params* p, const sa_pages* pages,
                                 const int32_t* lengths, int32_t rows, void* k, void* v,
                                 void* stream) {
  sa::PagedProblem x;
  sa::PagedPtrs c;
  sa_status s = paged_problem(p, pages, &x, &c);
  if (s != SA_OK) return s;
  if (rows < 0) return SA_ERR_INVALID_ARG;
  if ((int64_t)x.B * x.Hkv > 65535 || rows > (1 << 24)) return SA_ERR_UNSUPPORTED;
  if (rows == 0 || x.B == 0) {
    sa::set_last_launches(0);
    return SA_OK;
  }
  if (!usable(lengths, 4) || !usable(k, 16) || !usable(v, 16)) return SA_ERR_INVALID_ARG;
  if (sa::launch_cache_read(x, c, lengths, rows, k, v, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return SA_ERR_CUDA;
  sa::set_last_launches(1);
  return SA_OK;
}

sa_status sparse_attn_chunk(const sa_paged_params* p, const sa_pages* pages, const int32_t* cu_q,
                            const int32_t* cached, const void* q, const sa_row_strides* q_strides,
                            const float* alpha, const float* beta, int32_t window,
                            int32_t n_offsets, const int32_t* offsets, int32_t n_sinks,
                            float scale, void* o, float* lse, void* stream) {
  sa::PagedProblem x;
  sa::PagedPtrs c;
  sa_status s = paged_problem(p, pages, &x, &c);
  if (s != SA_OK) return s;
  if (window < 1 || n_offsets < 0 || n_sinks < 0 || !isfinite(scale)) return SA_ERR_INVALID_ARG;
  if (n_offsets > SA_MAX_OFFSETS || n_sinks > SA_MAX_SINKS) return SA_ERR_UNSUPPORTED;
  if (n_offsets > 0 && !offsets) return SA_ERR_INVALID_ARG;
  if (!rows16(q_strides, x.dtype)) return SA_ERR_INVALID_ARG;
  sa::ChunkPtrs a = {};
  for (int k = 0; k < n_offsets; ++k) {
    if (offsets[k] < 1) return SA_ERR_INVALID_ARG;
    a.f[k] = offsets[k];
  }
  if (x.N == 0 || x.B == 0) {
    sa::set_last_launches(0);
    return SA_OK;
  }
  if (!usable(q, 16) || !usable(o, 16) || !usable(cu_q, 4) || !usable(cached, 4) ||
      !usable(alpha, 4) || !aligned(beta, 4) || !aligned(lse, 4))
    return SA_ERR_INVALID_ARG;
  a.q = q; a.qs = *q_strides; a.cu_q = cu_q; a.cached = cached;
  a.alpha = alpha; a.beta = beta;
  a.W = window; a.n_off = n_offsets; a.S = n_sinks;
  a.scale = scale > 0.f ? scale : (float)(1.0 / sqrt((double)x.D));
  a.o = o; a.lse = lse;
  if (sa::launch_chunk_attn(x, c, a, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return SA_ERR_CUDA;
  sa::set_last_launches(1);
  return SA_OK;
}

}  // extern "C"
