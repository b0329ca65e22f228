// api_serving.cu -- C ABI of the grouped-query draft's serving step: host
// validation, workspace layout and dispatch of dflash_qk_norm_rope (+ backward),
// dflash_cache_append, dflash_attn_paged, dflash_attn_tree, dflash_verify, dflash_sample,
// dflash_tree_accept, and of what moves and hands out the cache's pages.
#include <math.h>
#include <string.h>

#include <initializer_list>

#include "common.cuh"
#include "internal.h"

using namespace dflash;

namespace {

bool aligned(const void* p, size_t b) { return ((uintptr_t)p % b) == 0; }
dflash_status_t launched(cudaError_t e) { return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA; }
dflash_status_t check_dtype(dflash_dtype_t t) {
  return t == DFLASH_BF16 || t == DFLASH_FP32 ? DFLASH_OK : DFLASH_ERR_DTYPE;
}
dflash_status_t check_ws(const void* ws, size_t bytes, size_t need) {
  return bytes < need || (need > 0 && (!ws || !aligned(ws, 256))) ? DFLASH_ERR_WORKSPACE : DFLASH_OK;
}
dflash_status_t check_head(int D) {
  if (D <= 0) return DFLASH_ERR_SHAPE;
  return D % 8 == 0 && D <= DFLASH_PAGED_MAX_D ? DFLASH_OK : DFLASH_ERR_UNSUPPORTED;
}

// Norm, rotation and strides of a call over `T` tokens with these heads.
dflash_status_t check_rotation(const dflash_rope_dims_t* d, int D, const float* cos_sin) {
  if (d->rot_dim < 0 || d->rot_dim > D || d->rot_dim % 2 != 0 || d->max_pos < 0) return DFLASH_ERR_SHAPE;
  if (!(d->eps >= 0.f) || isinf(d->eps)) return DFLASH_ERR_INVALID;
  if (d->rot_dim > 0 && !cos_sin) return DFLASH_ERR_INVALID;
  return cos_sin && !aligned(cos_sin, 4) ? DFLASH_ERR_ALIGN : DFLASH_OK;
}
// Token stride of a tensor with `heads` heads: 0 selects the contiguous one.
dflash_status_t resolve_stride(int64_t given, int heads, int D, long long* out) {
  const long long least = (long long)heads * D;
  *out = given == 0 ? least : given;
  return *out < least ? DFLASH_ERR_SHAPE : DFLASH_OK;
}
dflash_status_t check_tensor(const void* p, size_t esz) {
  if (!p) return DFLASH_ERR_INVALID;
  return aligned(p, esz) ? DFLASH_OK : DFLASH_ERR_ALIGN;
}

// Whole numbers that a call reads or writes, n of them.
struct Ints {
  const int32_t* p;
  long long n;
};
// Whether what a call writes overlaps what it reads, or one result another: CTAs read some while others write.
bool overlap(std::initializer_list<Ints> written, std::initializer_list<Ints> read) {
  auto meet = [](const Ints& x, const Ints& y) {
    const uintptr_t a = (uintptr_t)x.p, b = (uintptr_t)y.p;
    return x.p && y.p && x.n > 0 && y.n > 0 && a < b + sizeof(int32_t) * (size_t)y.n && b < a + sizeof(int32_t) * (size_t)x.n;
  };
  for (auto w = written.begin(); w != written.end(); ++w) {
    for (const Ints& r : read)
      if (meet(*w, r)) return true;
    for (auto v = written.begin(); v != w; ++v)
      if (meet(*w, *v)) return true;
  }
  return false;
}

#define TRY(call)                                 \
  do {                                            \
    const dflash_status_t st_ = (call);           \
    if (st_ != DFLASH_OK) return st_;             \
  } while (0)

dflash_status_t check_rope(const dflash_rope_dims_t* d, dflash_dtype_t dtype, const float* cos_sin,
                           const int32_t* positions, RopeArgs* a) {
  TRY(check_dtype(dtype));
  if (!d) return DFLASH_ERR_INVALID;
  if (d->T < 0 || d->H_q < 0 || d->H_kv < 0) return DFLASH_ERR_SHAPE;
  if (d->H_q > 65535 || d->H_kv > 65535 || d->T >= 1 << 30) return DFLASH_ERR_UNSUPPORTED;
  TRY(check_head(d->D));
  memset(a, 0, sizeof *a);
  a->T = d->T;
  a->Hq = d->H_q;
  a->Hkv = d->H_kv;
  a->D = d->D;
  a->rot = d->rot_dim;
  a->max_pos = d->max_pos;
  a->interleaved = d->interleaved != 0;
  a->eps = d->eps;
  TRY(resolve_stride(d->q_stride, d->H_q, d->D, &a->qs));
  TRY(resolve_stride(d->k_stride, d->H_kv, d->D, &a->ks));
  if (d->T == 0 || d->H_q + d->H_kv == 0) {
    if (d->rot_dim < 0 || d->rot_dim > d->D || d->rot_dim % 2 != 0) return DFLASH_ERR_SHAPE;
    return DFLASH_OK;
  }
  TRY(check_rotation(d, d->D, cos_sin));
  if (d->rot_dim > 0) TRY(check_tensor(positions, 4));
  a->cs = cos_sin;
  a->pos = positions;
  a->err = device_error_word();
  return DFLASH_OK;
}

dflash_status_t check_paged(const dflash_paged_dims_t* d, dflash_dtype_t dtype) {
  TRY(check_dtype(dtype));
  if (!d) return DFLASH_ERR_INVALID;
  if (d->R < 0 || d->H_q <= 0 || d->H_kv <= 0 || d->H_q % d->H_kv != 0 || d->total_q < 0 || d->max_q_len < 0 ||
      d->num_pages < 0 || d->page_size <= 0 || d->max_pages < 0)
    return DFLASH_ERR_SHAPE;
  TRY(check_head(d->D));
  if (d->H_q > 65535) return DFLASH_ERR_UNSUPPORTED;
  // the kernels' 32-bit indexes of requests go some strips beyond the last one
  if (d->R > 1 << 30) return DFLASH_ERR_UNSUPPORTED;
  // positions and rows of a request have to fit the kernels' 32-bit row arithmetic
  if ((long long)d->max_pages * d->page_size >= (1ll << 31) - 1024) return DFLASH_ERR_UNSUPPORTED;
  if ((long long)d->max_q_len * (d->H_q / d->H_kv) >= (1ll << 31) - 1024) return DFLASH_ERR_UNSUPPORTED;
  const long long page = (long long)d->page_size * d->H_kv * d->D;
  const int vec = dtype == DFLASH_BF16 ? 8 : 4;
  for (const int64_t s : {d->k_page_stride, d->v_page_stride}) {
    if (s != 0 && s < page) return DFLASH_ERR_SHAPE;
    if (s % vec != 0) return DFLASH_ERR_ALIGN;
    if (s > 0 && d->num_pages > 0 && s > (1ll << 60) / d->num_pages) return DFLASH_ERR_UNSUPPORTED;
  }
  return DFLASH_OK;
}

dflash_status_t check_table(const dflash_paged_dims_t* d, const int32_t* table, const int32_t* kv_lens,
                            const int32_t* q_offsets) {
  TRY(check_tensor(kv_lens, 4));
  TRY(check_tensor(q_offsets, 4));
  return d->max_pages > 0 ? check_tensor(table, 4) : DFLASH_OK;
}

size_t paged_ws(const dflash_paged_dims_t* d, dflash_dtype_t dtype) {
  return paged_workspace_bytes(dtype == DFLASH_BF16, d->H_q, d->H_kv, d->D, d->max_q_len, d->page_size);
}

// Attention over the pages, of a tree where `tree` is set (parents is required then).
dflash_status_t attend(const dflash_paged_dims_t* dims, dflash_dtype_t dtype, const void* q, const void* k_cache,
                       const void* v_cache, const int32_t* page_table, const int32_t* kv_lens, const int32_t* q_offsets,
                       bool tree, const int32_t* parents, int causal, float scale, void* out, float* lse,
                       void* workspace, size_t ws_bytes, dflash_stream_t stream) {
  TRY(check_paged(dims, dtype));
  if (isnan(scale) || isinf(scale)) return DFLASH_ERR_INVALID;
  if (dims->R == 0 || dims->total_q == 0) return DFLASH_OK;
  if (dims->max_q_len == 0) return DFLASH_ERR_SHAPE;
  if (!q || !out || (dims->num_pages > 0 && (!k_cache || !v_cache))) return DFLASH_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(lse, 4))
    return DFLASH_ERR_ALIGN;
  TRY(check_table(dims, page_table, kv_lens, q_offsets));
  if (tree) TRY(check_tensor(parents, 4));
  TRY(check_ws(workspace, ws_bytes, paged_ws(dims, dtype)));
  const long long page = (long long)dims->page_size * dims->H_kv * dims->D;
  PagedArgs a;
  memset(&a, 0, sizeof a);
  a.q = q;
  a.kc = k_cache;
  a.vc = v_cache;
  a.table = page_table;
  a.kv_lens = kv_lens;
  a.q_off = q_offsets;
  a.out = out;
  a.lse = lse;
  a.R = dims->R;
  a.Hq = dims->H_q;
  a.Hkv = dims->H_kv;
  a.G = dims->H_q / dims->H_kv;
  a.D = dims->D;
  a.total_q = dims->total_q;
  a.max_q = dims->max_q_len;
  a.num_pages = dims->num_pages;
  a.P = dims->page_size;
  a.max_pages = dims->max_pages;
  a.kps = dims->k_page_stride ? dims->k_page_stride : page;
  a.vps = dims->v_page_stride ? dims->v_page_stride : page;
  a.causal = causal != 0;
  a.parents = tree ? parents : nullptr;
  a.scale_log2 = (float)((scale > 0.f ? (double)scale : 1.0 / sqrt((double)dims->D)) * 1.4426950408889634);
  a.err = device_error_word();
  a.wait_ns = wait_budget_ns();
  a.stall_cta = stalled_cta();
  return launched(launch_attn_paged(a, dtype == DFLASH_BF16, workspace, (cudaStream_t)stream));
}

// The cache of a call that reads neither queries' heads nor max_q_len, and without `requests` nothing but the pages.
dflash_status_t check_cache(const dflash_paged_dims_t* dims, dflash_dtype_t dtype, bool requests) {
  if (!dims) return check_paged(dims, dtype);
  dflash_paged_dims_t d = *dims;
  d.H_q = d.H_kv;
  d.max_q_len = 0;
  if (!requests) d.R = d.total_q = d.max_pages = 0;
  return check_paged(&d, dtype);
}

// Layers of a cache: strides in 16-byte vectors, and the cache's pointers.
struct Layers {
  long long kps, vps, kls, vls;
  int row;
};
dflash_status_t check_layers(const dflash_paged_dims_t* d, const dflash_layers_t* l, dflash_dtype_t dtype,
                             const void* kc, const void* vc, Layers* out) {
  if (!l) return DFLASH_ERR_INVALID;
  if (l->L < 0) return DFLASH_ERR_SHAPE;
  if (l->L > 32767) return DFLASH_ERR_UNSUPPORTED;
  const long long vec = dtype == DFLASH_BF16 ? 8 : 4, row = (long long)d->H_kv * d->D, page = row * d->page_size;
  const long long kps = d->k_page_stride ? d->k_page_stride : page, vps = d->v_page_stride ? d->v_page_stride : page;
  if (row / vec >= 1 << 30 || (d->num_pages > 0 && page > (1ll << 60) / d->num_pages)) return DFLASH_ERR_UNSUPPORTED;
  const long long k_all = d->num_pages > 0 ? (d->num_pages - 1) * kps + page : 0;
  const long long v_all = d->num_pages > 0 ? (d->num_pages - 1) * vps + page : 0;
  const long long kls = l->k_layer_stride ? l->k_layer_stride : d->num_pages * kps;
  const long long vls = l->v_layer_stride ? l->v_layer_stride : d->num_pages * vps;
  // layers may lie in one another's gaps between pages (one tensor's [pages, L, ...]), or one behind the other
  const bool k_in = kls > 0 && kls >= page && (d->num_pages <= 1 || (l->L - 1) * kls + page <= kps);
  const bool v_in = vls > 0 && vls >= page && (d->num_pages <= 1 || (l->L - 1) * vls + page <= vps);
  if (kls < 0 || vls < 0 || (l->L > 1 && ((kls < k_all && !k_in) || (vls < v_all && !v_in)))) return DFLASH_ERR_SHAPE;
  if (kls % vec != 0 || vls % vec != 0) return DFLASH_ERR_ALIGN;
  if (l->L > 0 && (kls > (1ll << 60) / l->L || vls > (1ll << 60) / l->L)) return DFLASH_ERR_UNSUPPORTED;
  if (d->num_pages > 0 && l->L > 0) {
    if (!kc || !vc) return DFLASH_ERR_INVALID;
    if (!aligned(kc, 16) || !aligned(vc, 16)) return DFLASH_ERR_ALIGN;
  }
  *out = Layers{kps / vec, vps / vec, kls / vec, vls / vec, (int)(row / vec)};
  return DFLASH_OK;
}

dflash_status_t check_pool(const dflash_pool_dims_t* d, int items) {
  if (!d) return DFLASH_ERR_INVALID;
  if (d->R < 0 || d->max_pages < 0 || d->page_size <= 0 || d->num_pages < 0 || items < 0) return DFLASH_ERR_SHAPE;
  if (d->R > DFLASH_POOL_MAX_ROWS || items > DFLASH_POOL_MAX_ROWS || d->num_pages > 1 << 30) return DFLASH_ERR_UNSUPPORTED;
  if ((long long)d->R * d->max_pages >= 1ll << 31 || (long long)d->max_pages * d->page_size >= (1ll << 31) - 1024)
    return DFLASH_ERR_UNSUPPORTED;
  return DFLASH_OK;
}
dflash_status_t pool_args(const dflash_pool_dims_t* d, int32_t* table, int32_t* refs, int32_t* missing,
                          void* ws, size_t ws_bytes, PoolArgs* a) {
  if (d->R > 0 && d->max_pages > 0) TRY(check_tensor(table, 4));
  if (d->num_pages > 0) TRY(check_tensor(refs, 4));
  TRY(check_tensor(missing, 4));
  TRY(check_ws(ws, ws_bytes, pool_workspace_bytes(d->num_pages)));
  *a = PoolArgs{table, refs, missing, static_cast<int32_t*>(ws), d->R, d->max_pages, d->page_size, d->num_pages,
                aligned(refs, 16), device_error_word()};
  return DFLASH_OK;
}

}  // namespace

extern "C" {

dflash_status_t dflash_qk_norm_rope(const dflash_rope_dims_t* dims, dflash_dtype_t dtype, const void* q,
                                    const void* k, const void* q_norm, const void* k_norm, const float* cos_sin,
                                    const int32_t* positions, void* q_out, void* k_out, dflash_stream_t stream) {
  RopeArgs a;
  TRY(check_rope(dims, dtype, cos_sin, positions, &a));
  if (a.T == 0 || a.Hq + a.Hkv == 0) return DFLASH_OK;
  const size_t esz = dtype == DFLASH_BF16 ? 2 : 4;
  if (a.Hq > 0) {
    TRY(check_tensor(q, esz));
    TRY(check_tensor(q_out, esz));
    if (q_norm) TRY(check_tensor(q_norm, esz));
  }
  if (a.Hkv > 0) {
    TRY(check_tensor(k, esz));
    TRY(check_tensor(k_out, esz));
    if (k_norm) TRY(check_tensor(k_norm, esz));
  }
  a.q = q;
  a.k = k;
  a.wq = q_norm;
  a.wk = k_norm;
  a.qo = q_out;
  a.ko = k_out;
  return launched(launch_qk_norm_rope(a, dtype == DFLASH_BF16, false, (cudaStream_t)stream));
}

size_t dflash_qk_norm_rope_workspace_size(const dflash_rope_dims_t* dims) {
  if (!dims || check_head(dims->D) != DFLASH_OK) return 0;
  return rope_bwd_workspace_bytes(dims->D);
}

dflash_status_t dflash_qk_norm_rope_backward(const dflash_rope_dims_t* dims, dflash_dtype_t dtype, const void* q,
                                             const void* k, const void* q_norm, const void* k_norm,
                                             const float* cos_sin, const int32_t* positions, const void* dq_out,
                                             const void* dk_out, void* dq, void* dk, float* dq_norm, float* dk_norm,
                                             void* workspace, size_t ws_bytes, dflash_stream_t stream) {
  RopeArgs a;
  TRY(check_rope(dims, dtype, cos_sin, positions, &a));
  if (q_norm) TRY(check_tensor(dq_norm, 4));
  if (k_norm) TRY(check_tensor(dk_norm, 4));
  const size_t esz = dtype == DFLASH_BF16 ? 2 : 4;
  if (a.T == 0 || a.Hq + a.Hkv == 0) {
    cudaError_t e = cudaSuccess;
    if (q_norm) e = cudaMemsetAsync(dq_norm, 0, sizeof(float) * a.D, (cudaStream_t)stream);
    if (e == cudaSuccess && k_norm) e = cudaMemsetAsync(dk_norm, 0, sizeof(float) * a.D, (cudaStream_t)stream);
    return launched(e);
  }
  if (a.Hq > 0) {
    TRY(check_tensor(dq_out, esz));
    TRY(check_tensor(dq, esz));
    if (q_norm) {
      TRY(check_tensor(q, esz));
      TRY(check_tensor(q_norm, esz));
    }
  }
  if (a.Hkv > 0) {
    TRY(check_tensor(dk_out, esz));
    TRY(check_tensor(dk, esz));
    if (k_norm) {
      TRY(check_tensor(k, esz));
      TRY(check_tensor(k_norm, esz));
    }
  }
  TRY(check_ws(workspace, ws_bytes, rope_bwd_workspace_bytes(a.D)));
  a.q = q_norm ? q : nullptr;
  a.k = k_norm ? k : nullptr;
  a.wq = q_norm;
  a.wk = k_norm;
  a.dqo = dq_out;
  a.dko = dk_out;
  a.qo = dq;
  a.ko = dk;
  a.dw_part = static_cast<float*>(workspace);
  return launched(launch_qk_norm_rope_bwd(a, dtype == DFLASH_BF16, q_norm ? dq_norm : nullptr,
                                          k_norm ? dk_norm : nullptr, (cudaStream_t)stream));
}

dflash_status_t dflash_cache_append(const dflash_paged_dims_t* dims, const dflash_rope_dims_t* rope,
                                    dflash_dtype_t dtype, const void* q, const void* k, const void* v,
                                    int64_t v_stride, const void* q_norm, const void* k_norm, const float* cos_sin,
                                    const int32_t* page_table, const int32_t* kv_lens, const int32_t* q_offsets,
                                    void* q_out, void* k_cache, void* v_cache, dflash_stream_t stream) {
  TRY(check_paged(dims, dtype));
  if (!rope) return DFLASH_ERR_INVALID;
  const size_t esz = dtype == DFLASH_BF16 ? 2 : 4;
  RopeArgs a;
  memset(&a, 0, sizeof a);
  a.T = dims->total_q;
  a.Hq = q ? dims->H_q : 0;
  a.Hkv = dims->H_kv;
  a.D = dims->D;
  TRY(check_rotation(rope, a.D, cos_sin));
  TRY(resolve_stride(rope->q_stride, a.Hq, a.D, &a.qs));
  TRY(resolve_stride(rope->k_stride, a.Hkv, a.D, &a.ks));
  TRY(resolve_stride(v_stride, a.Hkv, a.D, &a.vs));
  if (dims->R == 0 || dims->total_q == 0) return DFLASH_OK;
  if (q) {
    TRY(check_tensor(q, esz));
    TRY(check_tensor(q_out, esz));
    if (q_norm) TRY(check_tensor(q_norm, esz));
  }
  TRY(check_tensor(k, esz));
  TRY(check_tensor(v, esz));
  if (k_norm) TRY(check_tensor(k_norm, esz));
  TRY(check_table(dims, page_table, kv_lens, q_offsets));
  if (dims->num_pages > 0) {
    if (!k_cache || !v_cache) return DFLASH_ERR_INVALID;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return DFLASH_ERR_ALIGN;
  }
  const long long page = (long long)dims->page_size * dims->H_kv * dims->D;
  a.q = q;
  a.k = k;
  a.v = v;
  a.wq = q_norm;
  a.wk = k_norm;
  a.cs = cos_sin;
  a.qo = q_out;
  a.rot = rope->rot_dim;
  a.max_pos = rope->max_pos;
  a.interleaved = rope->interleaved != 0;
  a.eps = rope->eps;
  a.kc = k_cache;
  a.vc = v_cache;
  a.kps = dims->k_page_stride ? dims->k_page_stride : page;
  a.vps = dims->v_page_stride ? dims->v_page_stride : page;
  a.table = page_table;
  a.kv_lens = kv_lens;
  a.q_off = q_offsets;
  a.R = dims->R;
  a.P = dims->page_size;
  a.max_pages = dims->max_pages;
  a.num_pages = dims->num_pages;
  a.err = device_error_word();
  return launched(launch_qk_norm_rope(a, dtype == DFLASH_BF16, true, (cudaStream_t)stream));
}

size_t dflash_attn_paged_workspace_size(const dflash_paged_dims_t* dims, dflash_dtype_t dtype) {
  return check_paged(dims, dtype) == DFLASH_OK ? paged_ws(dims, dtype) : 0;
}

dflash_status_t dflash_attn_paged(const dflash_paged_dims_t* dims, dflash_dtype_t dtype, const void* q,
                                  const void* k_cache, const void* v_cache, const int32_t* page_table,
                                  const int32_t* kv_lens, const int32_t* q_offsets, int causal, float scale, void* out,
                                  float* lse, void* workspace, size_t ws_bytes, dflash_stream_t stream) {
  return attend(dims, dtype, q, k_cache, v_cache, page_table, kv_lens, q_offsets, false, nullptr, causal, scale, out,
                lse, workspace, ws_bytes, stream);
}

dflash_status_t dflash_attn_tree(const dflash_paged_dims_t* dims, dflash_dtype_t dtype, const void* q,
                                 const void* k_cache, const void* v_cache, const int32_t* page_table,
                                 const int32_t* kv_lens, const int32_t* q_offsets, const int32_t* parents, float scale,
                                 void* out, float* lse, void* workspace, size_t ws_bytes, dflash_stream_t stream) {
  return attend(dims, dtype, q, k_cache, v_cache, page_table, kv_lens, q_offsets, true, parents, 1, scale, out, lse,
                workspace, ws_bytes, stream);
}

dflash_status_t dflash_verify(const dflash_verify_dims_t* dims, const float* target_probs, const float* draft_probs,
                              const int32_t* draft_tokens, const int32_t* draft_offsets, const float* accept_u,
                              const float* sample_u, int32_t* out_tokens, int32_t* num_accepted,
                              dflash_stream_t stream) {
  if (!dims) return DFLASH_ERR_INVALID;
  if (dims->R < 0 || dims->V <= 0 || dims->total_draft < 0 || dims->max_draft < 0) return DFLASH_ERR_SHAPE;
  // (the kernel's indexes along a row of out_tokens are 32 bits and go a block's width beyond it)
  if (dims->V > (1 << 30) || dims->R > (1 << 24) || dims->max_draft > (1 << 30)) return DFLASH_ERR_UNSUPPORTED;
  VerifyArgs a;
  memset(&a, 0, sizeof a);
  a.ps = dims->target_stride ? dims->target_stride : dims->V;
  a.qs = dims->draft_stride ? dims->draft_stride : dims->V;
  if (a.ps < dims->V || a.qs < dims->V) return DFLASH_ERR_SHAPE;
  if (dims->R == 0) return DFLASH_OK;
  TRY(check_tensor(target_probs, 4));
  if (draft_probs) TRY(check_tensor(draft_probs, 4));
  TRY(check_tensor(draft_offsets, 4));
  TRY(check_tensor(sample_u, 4));
  TRY(check_tensor(out_tokens, 4));
  TRY(check_tensor(num_accepted, 4));
  if (dims->total_draft > 0) {
    TRY(check_tensor(draft_tokens, 4));
    TRY(check_tensor(accept_u, 4));
  }
  a.p = target_probs;
  a.q = draft_probs;
  a.tokens = draft_tokens;
  a.offsets = draft_offsets;
  a.u = accept_u;
  a.s = sample_u;
  a.out = out_tokens;
  a.acc = num_accepted;
  a.R = dims->R;
  a.V = dims->V;
  a.total = dims->total_draft;
  a.max_draft = dims->max_draft;
  a.err = device_error_word();
  return launched(launch_verify(a, (cudaStream_t)stream));
}

dflash_status_t dflash_sample(const dflash_sample_dims_t* dims, dflash_dtype_t dtype, const void* logits,
                              const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                              const float* min_p, int32_t* tokens, float* probs, dflash_stream_t stream) {
  TRY(check_dtype(dtype));
  if (!dims) return DFLASH_ERR_INVALID;
  if (dims->N < 0 || dims->V <= 0) return DFLASH_ERR_SHAPE;
  if (dims->V > DFLASH_SAMPLE_MAX_V || dims->N > (1 << 24)) return DFLASH_ERR_UNSUPPORTED;
  SampleArgs a;
  memset(&a, 0, sizeof a);
  a.xs = dims->logits_stride ? dims->logits_stride : dims->V;
  a.ps = dims->probs_stride ? dims->probs_stride : dims->V;
  if (a.xs < dims->V || a.ps < dims->V) return DFLASH_ERR_SHAPE;
  if (dims->N == 0) return DFLASH_OK;
  TRY(check_tensor(logits, dtype == DFLASH_BF16 ? 2 : 4));
  TRY(check_tensor(u, 4));
  TRY(check_tensor(tokens, 4));
  if (!aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(probs, 4))
    return DFLASH_ERR_ALIGN;
  a.x = logits;
  a.u = u;
  a.temp = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.tokens = tokens;
  a.probs = probs;
  a.N = dims->N;
  a.V = dims->V;
  a.err = device_error_word();
  return launched(launch_sample(a, dtype == DFLASH_BF16, (cudaStream_t)stream));
}

dflash_status_t dflash_tree_accept(const dflash_accept_dims_t* dims, const int32_t* sampled, const int32_t* tokens,
                                   const int32_t* parents, const int32_t* q_offsets, int32_t* path,
                                   int32_t* out_tokens, int32_t* num_accepted, dflash_stream_t stream) {
  if (!dims) return DFLASH_ERR_INVALID;
  if (dims->R < 0 || dims->total < 0 || dims->max_path <= 0) return DFLASH_ERR_SHAPE;
  if (dims->R > 1 << 30 || dims->max_path > 1 << 30) return DFLASH_ERR_UNSUPPORTED;
  if (dims->R == 0) return DFLASH_OK;
  if (dims->total > 0) {
    TRY(check_tensor(sampled, 4));
    TRY(check_tensor(tokens, 4));
    TRY(check_tensor(parents, 4));
  }
  TRY(check_tensor(q_offsets, 4));
  TRY(check_tensor(path, 4));
  TRY(check_tensor(out_tokens, 4));
  TRY(check_tensor(num_accepted, 4));
  const long long R = dims->R, T = dims->total, cells = R * dims->max_path;
  if (overlap({{path, cells}, {out_tokens, cells}, {num_accepted, R}},
              {{sampled, T}, {tokens, T}, {parents, T}, {q_offsets, R + 1}}))
    return DFLASH_ERR_INVALID;
  const AcceptArgs a = {sampled, tokens, parents, q_offsets, path, out_tokens, num_accepted,
                        dims->R, dims->total, dims->max_path, device_error_word()};
  return launched(launch_tree_accept(a, (cudaStream_t)stream));
}

dflash_status_t dflash_cache_compact(const dflash_paged_dims_t* dims, const dflash_layers_t* layers,
                                     dflash_dtype_t dtype, const int32_t* page_table, const int32_t* kv_lens,
                                     const int32_t* q_offsets, const int32_t* path, int max_path,
                                     const int32_t* num_accepted, void* k_cache, void* v_cache, int32_t* new_lens,
                                     dflash_stream_t stream) {
  TRY(check_cache(dims, dtype, true));
  Layers l;
  TRY(check_layers(dims, layers, dtype, k_cache, v_cache, &l));
  if (max_path <= 0) return DFLASH_ERR_SHAPE;
  if (max_path > 1 << 30) return DFLASH_ERR_UNSUPPORTED;
  if (dims->R == 0) return DFLASH_OK;
  if (layers->L == 0) return DFLASH_ERR_SHAPE;  // the new lengths come from the layers' call
  TRY(check_table(dims, page_table, kv_lens, q_offsets));
  TRY(check_tensor(path, 4));
  TRY(check_tensor(num_accepted, 4));
  TRY(check_tensor(new_lens, 4));
  const long long R = dims->R;
  if (overlap({{new_lens, R}}, {{page_table, R * dims->max_pages}, {kv_lens, R}, {q_offsets, R + 1}, {path, R * max_path},
                                {num_accepted, R}}))
    return DFLASH_ERR_INVALID;
  const CompactArgs a = {k_cache, v_cache, page_table, kv_lens, q_offsets, path, num_accepted, new_lens,
                         l.kps, l.vps, l.kls, l.vls, dims->R, dims->total_q, dims->page_size, dims->max_pages,
                         dims->num_pages, max_path, layers->L, l.row, device_error_word()};
  return launched(launch_cache_compact(a, (cudaStream_t)stream));
}

dflash_status_t dflash_cache_copy(const dflash_paged_dims_t* dims, const dflash_layers_t* layers,
                                  dflash_dtype_t dtype, int n, const int32_t* src, const int32_t* dst,
                                  const int32_t* rows, void* k_cache, void* v_cache, dflash_stream_t stream) {
  TRY(check_cache(dims, dtype, false));
  Layers l;
  TRY(check_layers(dims, layers, dtype, k_cache, v_cache, &l));
  if (n < 0) return DFLASH_ERR_SHAPE;
  if (n > 1 << 30) return DFLASH_ERR_UNSUPPORTED;
  if (n == 0 || layers->L == 0) return DFLASH_OK;
  TRY(check_tensor(src, 4));
  TRY(check_tensor(dst, 4));
  if (!aligned(rows, 4)) return DFLASH_ERR_ALIGN;
  const CopyArgs a = {k_cache, v_cache, src, dst, rows, l.kps, l.vps, l.kls, l.vls,
                      n, dims->page_size, dims->num_pages, layers->L, l.row, device_error_word()};
  return launched(launch_cache_copy(a, (cudaStream_t)stream));
}

size_t dflash_pages_workspace_size(const dflash_pool_dims_t* dims) {
  return check_pool(dims, 0) == DFLASH_OK ? pool_workspace_bytes(dims->num_pages) : 0;
}

dflash_status_t dflash_pages_resize(const dflash_pool_dims_t* dims, int32_t* page_table, const int32_t* old_lens,
                                    const int32_t* new_lens, int32_t* refs, int32_t* missing, void* workspace,
                                    size_t ws_bytes, dflash_stream_t stream) {
  TRY(check_pool(dims, 0));
  PoolArgs a;
  TRY(pool_args(dims, page_table, refs, missing, workspace, ws_bytes, &a));
  if (dims->R > 0) {
    TRY(check_tensor(old_lens, 4));
    TRY(check_tensor(new_lens, 4));
  }
  const long long R = dims->R;
  if (overlap({{page_table, R * dims->max_pages}, {refs, dims->num_pages}, {missing, 1}}, {{old_lens, R}, {new_lens, R}}))
    return DFLASH_ERR_INVALID;
  return launched(launch_pages_resize(a, old_lens, new_lens, (cudaStream_t)stream));
}

dflash_status_t dflash_pages_fork(const dflash_pool_dims_t* dims, int32_t* page_table, int32_t* lens, int n,
                                  const int32_t* src, const int32_t* dst, int32_t* refs, int32_t* copy_src,
                                  int32_t* copy_dst, int32_t* copy_rows, int32_t* missing, void* workspace,
                                  size_t ws_bytes, dflash_stream_t stream) {
  TRY(check_pool(dims, n));
  PoolArgs a;
  TRY(pool_args(dims, page_table, refs, missing, workspace, ws_bytes, &a));
  if (dims->R > 0) TRY(check_tensor(lens, 4));
  if (n > 0)
    for (const int32_t* p : {src, dst, (const int32_t*)copy_src, (const int32_t*)copy_dst, (const int32_t*)copy_rows})
      TRY(check_tensor(p, 4));
  const long long R = dims->R;
  if (overlap({{page_table, R * dims->max_pages}, {lens, R}, {refs, dims->num_pages}, {copy_src, n}, {copy_dst, n},
               {copy_rows, n}, {missing, 1}}, {{src, n}, {dst, n}}))
    return DFLASH_ERR_INVALID;
  const ForkArgs f = {src, dst, lens, copy_src, copy_dst, copy_rows, n};
  return launched(launch_pages_fork(a, f, (cudaStream_t)stream));
}

}  // extern "C"
