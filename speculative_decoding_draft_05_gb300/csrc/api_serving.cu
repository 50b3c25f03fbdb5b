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

bool is_dtype(int dtype) { return dtype == DSPARK_F32 || dtype == DSPARK_BF16; }
bool is_fp4(const dspark_cache* c) { return c->dtype == DSPARK_FP4; }

// A factor of a 4-bit cache: its products with any scale, and their inverses, stay normal.
bool is_factor(float f) { return f >= 0x1p-60f && f <= 0x1p60f; }

// any: of any type, else fp32 or bf16.
int check_cache(const dspark_cache* c, int layer, bool any = false) {
  if (!c || !c->k || !c->v) return DSPARK_ERR_INVALID_ARG;
  if (!is_dtype(c->dtype) && !(any && is_fp4(c))) return DSPARK_ERR_INVALID_ARG;
  if (c->layers <= 0 || c->n_pages <= 0 || c->page_size <= 0 || c->heads <= 0 || c->head_dim <= 0)
    return DSPARK_ERR_INVALID_ARG;
  if (layer < 0 || layer >= c->layers) return DSPARK_ERR_INVALID_ARG;
  if (c->page_stride <= 0 || c->token_stride <= 0 || c->head_stride <= 0 || c->layer_stride < 0)
    return DSPARK_ERR_INVALID_ARG;
  const uintptr_t a = is_fp4(c) ? 15u : (uintptr_t)(esize_of(c->dtype) - 1);
  if (((uintptr_t)c->k & a) || ((uintptr_t)c->v & a)) return DSPARK_ERR_INVALID_ARG;
  if (is_fp4(c)) {
    if (c->token_stride != 9ll * c->head_dim || ((c->layer_stride | c->page_stride | c->head_stride) & 15))
      return DSPARK_ERR_INVALID_ARG;
    if (c->head_dim % 32 != 0 || c->page_size % 16 != 0)
      return unsupported("a 4-bit cache: head_dim % 32 == 0, page_size % 16 == 0");
  }
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
  const size_t at = (size_t)layer * (size_t)c->layer_stride * (is_fp4(c) ? 1 : esize_of(c->dtype));
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
  if (is_fp4(c)) {  // rows of 9 D / 16 bytes a position, in pairs of bytes, heads first
    CacheView v = layer_view(c, 0);
    v.head_dim = 9 * c->head_dim / 32;
    v.token_stride = v.head_dim;
    v.page_stride /= 2;
    v.head_stride /= 2;
    return PagePool{v, 2, c->layers, c->layer_stride / 2};
  }
  return PagePool{layer_view(c, 0), esize_of(c->dtype), c->layers, c->layer_stride};
}

int check_meta(const dspark_cache* cache, const PageMeta& m, void* workspace, size_t bytes) {
  int st = check_cache(cache, 0, true);
  if (st != DSPARK_OK) return st;
  if (!m.table || !m.kv_len || !m.refcount || !m.table_out || !m.kv_len_out || !m.refcount_out)
    return DSPARK_ERR_INVALID_ARG;
  st = check_tables(m.R, m.max_pages);
  if (st != DSPARK_OK) return st;
  return check_workspace(workspace, bytes, pages_workspace_layout(m.R, m.n_pages).total);
}

// Whether rows of D elements at t * token + h * head (t < T, h < H) do not lie one over the other.
bool rows_apart(long long token, long long head, int T, int H, int D) {
  if ((H > 1 && head < D) || (T > 1 && token < D)) return false;
  if (H == 1 || T == 1 || (token - D) / head >= H - 1 || (head - D) / token >= T - 1) return true;
  for (int h = 1; h < H; ++h) {  // heads h apart: the tokens apart that come nearest
    const __int128 at = (__int128)h * head, t = at / token, over = at - t * token;
    if ((t < T && over < D) || (t + 1 < T && token - over < D)) return false;
  }
  return true;
}

// Attention of either kind of cache, which is checked already.  dtype: of q and out.
int attend(const void* q, long long q_token_stride, long long q_head_stride, int Hq, int dtype,
           const dspark_cache* cache, int layer, float k_factor, float v_factor,
           const int32_t* q_offsets, const int32_t* kv_len, const int32_t* page_table, int R,
           int n_tokens, int max_pages, float scale, void* out, float* lse, void* workspace,
           size_t workspace_bytes, size_t need, void* stream) {
  if (!q_offsets || !kv_len || !page_table) return DSPARK_ERR_INVALID_ARG;
  if (n_tokens != 0 && (!q || !out || !lse)) return DSPARK_ERR_INVALID_ARG;
  if (n_tokens < 0 || q_token_stride < 0 || q_head_stride < 0) return DSPARK_ERR_INVALID_ARG;
  if (Hq <= 0 || Hq % cache->heads != 0 || !isfinite(scale * k_factor * kLog2e)) return DSPARK_ERR_INVALID_ARG;
  const uintptr_t a = (uintptr_t)(esize_of(dtype) - 1);
  if (((uintptr_t)q & a) || ((uintptr_t)out & 15u)) return DSPARK_ERR_INVALID_ARG;
  int st = check_tables(R, max_pages);
  if (st != DSPARK_OK) return st;
  if ((long long)n_tokens * Hq > kMaxCount) return unsupported("n_tokens * Hq <= 2^31 - 2^16");
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != DSPARK_OK) return st;
  AttnArgs p;
  p.a = ChunkArgs{q_offsets, kv_len, page_table, R, n_tokens, max_pages};
  p.c = layer_view(cache, layer);
  p.q = q;
  p.q_token_stride = q_token_stride;
  p.q_head_stride = q_head_stride;
  p.Hq = Hq;
  p.G = Hq / cache->heads;
  p.dtype = dtype;
  p.scale = scale * k_factor;
  p.out = out;
  p.lse = lse;
  p.fp4 = is_fp4(cache);
  p.v_factor = v_factor;
  cudaStream_t s = (cudaStream_t)stream;
  prof_begin(kKindAttention, s);
  const cudaError_t e = launch_paged_attention(p, (char*)workspace, s);
  prof_end(s);
  return e != cudaSuccess ? cuda_fail(e, "paged_attention") : DSPARK_OK;
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
  if (!cache || is_fp4(cache) || cache->head_dim <= 0 || cache->head_dim > 256) return 0;
  return attention_workspace_bytes(cache->dtype, cache->head_dim);
}

int dspark_paged_attention(const void* q, long long q_token_stride, long long q_head_stride, int Hq,
                           const dspark_cache* cache, int layer, const int32_t* q_offsets,
                           const int32_t* kv_len, const int32_t* page_table, int R, int n_tokens,
                           int max_pages, float scale, void* out, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const int st = check_cache(cache, layer);
  if (st != DSPARK_OK) return st;
  return attend(q, q_token_stride, q_head_stride, Hq, cache->dtype, cache, layer, 1.0f, 1.0f, q_offsets, kv_len,
                page_table, R, n_tokens, max_pages, scale, out, lse, workspace, workspace_bytes,
                dspark_paged_attention_workspace_bytes(cache), stream);
}

size_t dspark_paged_attention_fp4_workspace_bytes(const dspark_cache* cache, int dtype) {
  if (!cache || !is_fp4(cache) || !is_dtype(dtype) || cache->head_dim <= 0 || cache->head_dim > 256) return 0;
  return attention_fp4_workspace_bytes(dtype, cache->head_dim);
}

int dspark_paged_attention_fp4(const void* q, long long q_token_stride, long long q_head_stride, int Hq,
                               int dtype, const dspark_cache* cache, int layer, float k_factor,
                               float v_factor, const int32_t* q_offsets, const int32_t* kv_len,
                               const int32_t* page_table, int R, int n_tokens, int max_pages,
                               float scale, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const int st = check_cache(cache, layer, true);
  if (st != DSPARK_OK) return st;
  if (!is_fp4(cache) || !is_dtype(dtype) || !is_factor(k_factor) || !is_factor(v_factor))
    return DSPARK_ERR_INVALID_ARG;
  return attend(q, q_token_stride, q_head_stride, Hq, dtype, cache, layer, k_factor, v_factor, q_offsets, kv_len,
                page_table, R, n_tokens, max_pages, scale, out, lse, workspace, workspace_bytes,
                attention_fp4_workspace_bytes(dtype, cache->head_dim), stream);
}

int dspark_cache_append_rotary(const dspark_cache* cache, int layer, float k_factor, float v_factor,
                               const dspark_rotary* rotary, int dtype, const void* k_new,
                               const void* v_new, long long new_token_stride,
                               long long new_head_stride, const void* q, long long q_token_stride,
                               long long q_head_stride, int Hq, void* q_out,
                               long long q_out_token_stride, long long q_out_head_stride,
                               const int32_t* q_offsets, const int32_t* kv_len,
                               const int32_t* page_table, int R, int n_tokens, int max_pages,
                               void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_cache(cache, layer, true);
  if (st != DSPARK_OK) return st;
  if (!is_dtype(dtype) || (!is_fp4(cache) && dtype != cache->dtype)) return DSPARK_ERR_INVALID_ARG;
  if (is_fp4(cache) && (!is_factor(k_factor) || !is_factor(v_factor))) return DSPARK_ERR_INVALID_ARG;
  if (!q_offsets || !kv_len || !page_table) return DSPARK_ERR_INVALID_ARG;
  if (n_tokens != 0 && (!k_new || !v_new)) return DSPARK_ERR_INVALID_ARG;
  if (n_tokens < 0 || new_token_stride < 0 || new_head_stride < 0 || Hq < 0) return DSPARK_ERR_INVALID_ARG;
  if (Hq > 0 && n_tokens != 0 && (!q || !q_out)) return DSPARK_ERR_INVALID_ARG;
  if (Hq > 0 && (q_token_stride < 0 || q_head_stride < 0 || q_out_token_stride < 0 || q_out_head_stride < 0))
    return DSPARK_ERR_INVALID_ARG;
  if (Hq > 0 && n_tokens != 0 && q == q_out && (q_token_stride != q_out_token_stride || q_head_stride != q_out_head_stride))
    return DSPARK_ERR_INVALID_ARG;
  if (Hq > 0 && n_tokens != 0 && !rows_apart(q_out_token_stride, q_out_head_stride, n_tokens, Hq, cache->head_dim))
    return DSPARK_ERR_INVALID_ARG;
  const uintptr_t a = (uintptr_t)(esize_of(dtype) - 1);
  if (((uintptr_t)k_new & a) || ((uintptr_t)v_new & a) || ((uintptr_t)q & a) || ((uintptr_t)q_out & a))
    return DSPARK_ERR_INVALID_ARG;
  if (rotary && (!rotary->cos_sin || ((uintptr_t)rotary->cos_sin & 3u) || rotary->n_positions <= 0 ||
                 rotary->dim <= 0 || rotary->dim % 2 != 0 || rotary->dim > cache->head_dim))
    return DSPARK_ERR_INVALID_ARG;
  st = check_tables(R, max_pages);
  if (st != DSPARK_OK) return st;
  if (n_tokens > kMaxCount || (long long)n_tokens * Hq > kMaxCount)
    return unsupported("n_tokens, n_tokens * Hq <= 2^31 - 2^16");
  st = check_workspace(workspace, workspace_bytes, 256);
  if (st != DSPARK_OK) return st;
  RotaryAppendArgs p;
  p.c = layer_view(cache, layer);
  p.a = ChunkArgs{q_offsets, kv_len, page_table, R, n_tokens, max_pages};
  p.k_new = k_new;
  p.v_new = v_new;
  p.q = q;
  p.q_out = q_out;
  p.tok_stride = new_token_stride;
  p.head_stride = new_head_stride;
  p.q_tok = q_token_stride;
  p.q_head = q_head_stride;
  p.qo_tok = q_out_token_stride;
  p.qo_head = q_out_head_stride;
  p.Hq = Hq;
  p.cos_sin = rotary ? rotary->cos_sin : nullptr;
  p.positions = rotary ? rotary->positions : nullptr;
  p.rot = rotary ? rotary->dim : 0;
  p.n_positions = rotary ? rotary->n_positions : 0;
  p.interleaved = rotary && rotary->interleaved;
  p.k_factor = is_fp4(cache) ? make_float2(k_factor, 1.0f / k_factor) : make_float2(1.0f, 1.0f);
  p.v_factor = is_fp4(cache) ? make_float2(v_factor, 1.0f / v_factor) : make_float2(1.0f, 1.0f);
  p.status = (int*)workspace;
  cudaStream_t s = (cudaStream_t)stream;
  prof_begin(kKindAppend, s);
  const cudaError_t e = launch_append_rotary(p, dtype, is_fp4(cache), s);
  prof_end(s);
  return e != cudaSuccess ? cuda_fail(e, "cache_append_rotary") : DSPARK_OK;
}

int dspark_cache_read(const dspark_cache* cache, int layer, float k_factor, float v_factor, int dtype,
                      const int32_t* q_offsets, const int32_t* kv_len, const int32_t* page_table,
                      int R, int n_tokens, int max_pages, void* k_out, void* v_out, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int st = check_cache(cache, layer, true);
  if (st != DSPARK_OK) return st;
  if (!is_dtype(dtype) || (!is_fp4(cache) && dtype != cache->dtype)) return DSPARK_ERR_INVALID_ARG;
  if (is_fp4(cache) && (!is_factor(k_factor) || !is_factor(v_factor))) return DSPARK_ERR_INVALID_ARG;
  if (!q_offsets || !kv_len || !page_table || n_tokens < 0) return DSPARK_ERR_INVALID_ARG;
  if (n_tokens != 0 && (!k_out || !v_out)) return DSPARK_ERR_INVALID_ARG;
  if (((uintptr_t)k_out | (uintptr_t)v_out) & 15u) return DSPARK_ERR_INVALID_ARG;
  st = check_tables(R, max_pages);
  if (st != DSPARK_OK) return st;
  if (n_tokens > kMaxCount) return unsupported("n_tokens <= 2^31 - 2^16");
  st = check_workspace(workspace, workspace_bytes, 256);
  if (st != DSPARK_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  prof_begin(kKindAppend, s);
  const cudaError_t e = launch_cache_read(
      CacheReadArgs{layer_view(cache, layer), ChunkArgs{q_offsets, kv_len, page_table, R, n_tokens, max_pages},
                    k_out, v_out, k_factor, v_factor, (int*)workspace},
      esize_of(dtype), is_fp4(cache), s);
  prof_end(s);
  return e != cudaSuccess ? cuda_fail(e, "cache_read") : DSPARK_OK;
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
  int st = check_cache(cache, 0, true);
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
