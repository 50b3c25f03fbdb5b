// api_serving.cu -- the C-ABI of the serving operators (declared in
// include/dspark.h): argument checks, workspace layout, launches.
#include <cuda_runtime.h>
#include <math.h>

#include "../../include/dspark.h"
#include "kernels.h"
#include "serving.h"

using namespace dspark;

namespace {

constexpr float kLog2e = 1.4426950408889634f;  // the kernels' exponentials are powers of two

int check_workspace(const void* ws, size_t have, size_t need) {
  return !ws || have < need || ((uintptr_t)ws & 255u) ? DSPARK_ERR_WORKSPACE : DSPARK_OK;
}

int esize_of(int dtype) { return dtype == DSPARK_BF16 ? 2 : 4; }

int check_cache(const dspark_cache* c, int layer) {
  if (!c || !c->k || !c->v) return DSPARK_ERR_INVALID_ARG;
  if (c->dtype != DSPARK_F32 && c->dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARG;
  if (c->layers <= 0 || c->n_pages <= 0 || c->page_size <= 0 || c->heads <= 0 || c->head_dim <= 0)
    return DSPARK_ERR_INVALID_ARG;
  if (layer < 0 || layer >= c->layers) return DSPARK_ERR_INVALID_ARG;
  if (c->page_stride <= 0 || c->token_stride <= 0 || c->head_stride <= 0 || c->layer_stride < 0)
    return DSPARK_ERR_INVALID_ARG;
  const uintptr_t a = (uintptr_t)(esize_of(c->dtype) - 1);
  if (((uintptr_t)c->k & a) || ((uintptr_t)c->v & a)) return DSPARK_ERR_INVALID_ARG;
  if (c->head_dim > 256 || c->heads > 1024 || c->page_size > 65536 || c->n_pages > kMaxCount ||
      (long long)c->page_size * c->heads * c->head_dim > (1ll << 30))
    return unsupported("head_dim <= 256, heads <= 1024, page_size <= 65536, n_pages <= 2^31 - 2^16, 2^30 elements a page");
  return DSPARK_OK;
}

int check_tables(int R, int max_pages) {
  if (R <= 0 || max_pages <= 0) return DSPARK_ERR_INVALID_ARG;
  if (R > 65535 || (long long)R * max_pages >= (1ll << 31))
    return unsupported("R <= 65535, R * max_pages < 2^31");
  return DSPARK_OK;
}

CacheView layer_view(const dspark_cache* c, int layer) {
  CacheView v;
  const size_t at = (size_t)layer * (size_t)c->layer_stride * esize_of(c->dtype);
  v.k = (char*)c->k + at;
  v.v = (char*)c->v + at;
  v.n_pages = c->n_pages;
  v.page_size = c->page_size;
  v.heads = c->heads;
  v.head_dim = c->head_dim;
  v.page_stride = c->page_stride;
  v.token_stride = c->token_stride;
  v.head_stride = c->head_stride;
  return v;
}

PagePool pool_of(const dspark_cache* c) {
  return PagePool{layer_view(c, 0), esize_of(c->dtype), c->layers, c->layer_stride};
}

int check_meta(const dspark_cache* cache, const PageMeta& m, void* workspace, size_t bytes) {
  int st = check_cache(cache, 0);
  if (st != DSPARK_OK) return st;
  if (!m.table || !m.kv_len || !m.refcount || !m.table_out || !m.kv_len_out || !m.refcount_out)
    return DSPARK_ERR_INVALID_ARG;
  st = check_tables(m.R, m.max_pages);
  if (st != DSPARK_OK) return st;
  return check_workspace(workspace, bytes, pages_workspace_layout(m.R, m.n_pages).total);
}

}  // namespace

extern "C" {

int dspark_cache_append(const dspark_cache* cache, int layer, const void* k_new, const void* v_new,
                        long long new_token_stride, long long new_head_stride,
                        const int32_t* q_offsets, const int32_t* kv_len, const int32_t* page_table,
                        int R, int n_tokens, int max_pages, void* workspace, size_t workspace_bytes,
                        void* stream) {
  int st = check_cache(cache, layer);
  if (st != DSPARK_OK) return st;
  if (!q_offsets || !kv_len || !page_table) return DSPARK_ERR_INVALID_ARG;
  if (n_tokens != 0 && (!k_new || !v_new)) return DSPARK_ERR_INVALID_ARG;
  if (n_tokens < 0 || new_token_stride < 0 || new_head_stride < 0) return DSPARK_ERR_INVALID_ARG;
  const uintptr_t a = (uintptr_t)(esize_of(cache->dtype) - 1);
  if (((uintptr_t)k_new & a) || ((uintptr_t)v_new & a)) return DSPARK_ERR_INVALID_ARG;
  st = check_tables(R, max_pages);
  if (st != DSPARK_OK) return st;
  if (n_tokens > kMaxCount) return unsupported("n_tokens <= 2^31 - 2^16");
  st = check_workspace(workspace, workspace_bytes, 256);
  if (st != DSPARK_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  prof_begin(kKindAppend, s);
  const cudaError_t e = launch_cache_append(
      layer_view(cache, layer), esize_of(cache->dtype), k_new, v_new, new_token_stride,
      new_head_stride, ChunkArgs{q_offsets, kv_len, page_table, R, n_tokens, max_pages},
      (int*)workspace, s);
  prof_end(s);
  return e != cudaSuccess ? cuda_fail(e, "cache_append") : DSPARK_OK;
}

size_t dspark_paged_attention_workspace_bytes(const dspark_cache* cache) {
  if (!cache || cache->head_dim <= 0 || cache->head_dim > 256) return 0;
  return attention_workspace_bytes(cache->dtype, cache->head_dim);
}

int dspark_paged_attention(const void* q, long long q_token_stride, long long q_head_stride, int Hq,
                           const dspark_cache* cache, int layer, const int32_t* q_offsets,
                           const int32_t* kv_len, const int32_t* page_table, int R, int n_tokens,
                           int max_pages, float scale, void* out, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  int st = check_cache(cache, layer);
  if (st != DSPARK_OK) return st;
  if (!q_offsets || !kv_len || !page_table) return DSPARK_ERR_INVALID_ARG;
  if (n_tokens != 0 && (!q || !out || !lse)) return DSPARK_ERR_INVALID_ARG;
  if (n_tokens < 0 || q_token_stride < 0 || q_head_stride < 0) return DSPARK_ERR_INVALID_ARG;
  if (Hq <= 0 || Hq % cache->heads != 0 || !isfinite(scale * kLog2e)) return DSPARK_ERR_INVALID_ARG;
  const uintptr_t a = (uintptr_t)(esize_of(cache->dtype) - 1);
  if (((uintptr_t)q & a) || ((uintptr_t)out & 15u)) return DSPARK_ERR_INVALID_ARG;
  st = check_tables(R, max_pages);
  if (st != DSPARK_OK) return st;
  if ((long long)n_tokens * Hq > kMaxCount) return unsupported("n_tokens * Hq <= 2^31 - 2^16");
  st = check_workspace(workspace, workspace_bytes, dspark_paged_attention_workspace_bytes(cache));
  if (st != DSPARK_OK) return st;
  AttnArgs p;
  p.a = ChunkArgs{q_offsets, kv_len, page_table, R, n_tokens, max_pages};
  p.c = layer_view(cache, layer);
  p.q = q;
  p.q_token_stride = q_token_stride;
  p.q_head_stride = q_head_stride;
  p.Hq = Hq;
  p.G = Hq / cache->heads;
  p.dtype = cache->dtype;
  p.scale = scale;
  p.out = out;
  p.lse = lse;
  cudaStream_t s = (cudaStream_t)stream;
  prof_begin(kKindAttention, s);
  const cudaError_t e = launch_paged_attention(p, (char*)workspace, s);
  prof_end(s);
  return e != cudaSuccess ? cuda_fail(e, "paged_attention") : DSPARK_OK;
}

size_t dspark_pages_workspace_bytes(int R, int n_pages) {
  if (R <= 0 || n_pages <= 0) return 0;
  return pages_workspace_layout(R, n_pages).total;
}

int dspark_pages_resize(const dspark_cache* cache, const int32_t* page_table, const int32_t* kv_len,
                        const int32_t* new_len, const int32_t* refcount, int R, int max_pages,
                        int32_t* page_table_out, int32_t* kv_len_out, int32_t* refcount_out,
                        int32_t* free_pages, void* workspace, size_t workspace_bytes, void* stream) {
  if (!cache || !new_len || !free_pages) return DSPARK_ERR_INVALID_ARG;
  const PageMeta m{page_table, kv_len, refcount, page_table_out, kv_len_out, refcount_out,
                   R, max_pages, cache->n_pages, cache->page_size};
  const int st = check_meta(cache, m, workspace, workspace_bytes);
  if (st != DSPARK_OK) return st;
  const PagesWorkspace w = pages_workspace_layout(R, cache->n_pages);
  char* ws = (char*)workspace;
  cudaStream_t s = (cudaStream_t)stream;
  prof_begin(kKindPages, s);
  const cudaError_t e = launch_pages_resize(pool_of(cache), m, new_len, free_pages, ws, w, s);
  prof_end(s);
  return e != cudaSuccess ? cuda_fail(e, "pages_resize") : DSPARK_OK;
}

int dspark_pages_fork(const dspark_cache* cache, const int32_t* page_table, const int32_t* kv_len,
                      const int32_t* refcount, const int32_t* parent, const int32_t* child, int n,
                      int R, int max_pages, int32_t* page_table_out, int32_t* kv_len_out,
                      int32_t* refcount_out, int32_t* free_pages, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (!cache || !free_pages || (n != 0 && (!parent || !child))) return DSPARK_ERR_INVALID_ARG;
  if (n < 0 || n > R) return DSPARK_ERR_INVALID_ARG;
  const PageMeta m{page_table, kv_len, refcount, page_table_out, kv_len_out, refcount_out,
                   R, max_pages, cache->n_pages, cache->page_size};
  const int st = check_meta(cache, m, workspace, workspace_bytes);
  if (st != DSPARK_OK) return st;
  const PagesWorkspace w = pages_workspace_layout(R, cache->n_pages);
  char* ws = (char*)workspace;
  cudaStream_t s = (cudaStream_t)stream;
  prof_begin(kKindPages, s);
  const cudaError_t e =
      launch_pages_fork(pool_of(cache), m, parent, child, n, free_pages, ws, w, s);
  prof_end(s);
  return e != cudaSuccess ? cuda_fail(e, "pages_fork") : DSPARK_OK;
}

int dspark_pages_compact(const dspark_cache* cache, const int32_t* page_table,
                         const int32_t* kv_len, const int32_t* refcount, int R, int max_pages,
                         int32_t* page_table_out, int32_t* refcount_out, int32_t* page_map,
                         int32_t* n_live, void* workspace, size_t workspace_bytes, void* stream) {
  if (!cache || !page_map || !n_live) return DSPARK_ERR_INVALID_ARG;
  const PageMeta m{page_table, kv_len, refcount, page_table_out, (int32_t*)kv_len, refcount_out,
                   R, max_pages, cache->n_pages, cache->page_size};
  const int st = check_meta(cache, m, workspace, workspace_bytes);
  if (st != DSPARK_OK) return st;
  const PagesWorkspace w = pages_workspace_layout(R, cache->n_pages);
  char* ws = (char*)workspace;
  cudaStream_t s = (cudaStream_t)stream;
  prof_begin(kKindPages, s);
  const cudaError_t e = launch_pages_compact(pool_of(cache), m, page_map, n_live, ws, w, s);
  prof_end(s);
  return e != cudaSuccess ? cuda_fail(e, "pages_compact") : DSPARK_OK;
}

int dspark_pages_copy(const dspark_cache* cache, const int32_t* src, const int32_t* dst, int n,
                      void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_cache(cache, 0);
  if (st != DSPARK_OK) return st;
  if (n < 0 || (n != 0 && (!src || !dst))) return DSPARK_ERR_INVALID_ARG;
  st = check_workspace(workspace, workspace_bytes, 256);
  if (st != DSPARK_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  prof_begin(kKindPages, s);
  const cudaError_t e = launch_pages_copy(pool_of(cache), src, dst, n, (int*)workspace, s);
  prof_end(s);
  return e != cudaSuccess ? cuda_fail(e, "pages_copy") : DSPARK_OK;
}

size_t dspark_logprobs_workspace_bytes(int n_rows, int V) {
  if (n_rows <= 0 || V <= 0) return 0;
  return logprobs_workspace_layout(n_rows, V).total;
}

int dspark_logprobs(const void* Z, int dtype, long long row_stride, const int32_t* tokens,
                    int n_rows, int V, float temperature, int top, float* logp, float* entropy,
                    float* lse, int32_t* top_ids, float* top_logp, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!Z || !tokens || !logp || !entropy || !lse) return DSPARK_ERR_INVALID_ARG;
  if (top < 0 || (top > 0 && (!top_ids || !top_logp))) return DSPARK_ERR_INVALID_ARG;
  if (n_rows <= 0 || V <= 0 || row_stride < V) return DSPARK_ERR_INVALID_ARG;
  if (!(temperature > 0.0f) || !isfinite(temperature) || !isfinite(1.0f / temperature * kLog2e))
    return DSPARK_ERR_INVALID_ARG;
  if (dtype != DSPARK_F32 && dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARG;
  if (V % 8 != 0 || V > (1 << 30) || n_rows > (1 << 30) || top > 32 || top > V)
    return unsupported("V % 8 == 0, V <= 2^30, n_rows <= 2^30, top <= min(32, V)");
  if (((uintptr_t)Z & 15u) || (row_stride * esize_of(dtype)) % 16 != 0) return DSPARK_ERR_INVALID_ARG;
  const LogprobsWorkspace w = logprobs_workspace_layout(n_rows, V);
  const int st = check_workspace(workspace, workspace_bytes, w.total);
  if (st != DSPARK_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  prof_begin(kKindLogprobs, s);
  const cudaError_t e = launch_logprobs(Z, dtype, row_stride, tokens, n_rows, V, 1.0f / temperature, top,
                                  logp, entropy, lse, top_ids, top_logp, (char*)workspace, w, s);
  prof_end(s);
  return e != cudaSuccess ? cuda_fail(e, "logprobs") : DSPARK_OK;
}

}  // extern "C"
