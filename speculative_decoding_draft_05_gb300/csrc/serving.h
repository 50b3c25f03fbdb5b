// serving.h -- host-side launchers of the serving operators (paged K/V cache,
// attention over it, page management, token log-probabilities), internal to
// libdspark.so.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/dspark.h"

namespace dspark {

// Shared by the C-ABI files (defined in api.cu).
int cuda_fail(cudaError_t e, const char* where);
int unsupported(const char* why);  // sets dspark_last_error's text
void prof_begin(int kind, cudaStream_t s);
void prof_end(cudaStream_t s);

inline size_t align_up256(size_t x) { return (x + 255) & ~(size_t)255; }

// One layer's K and V (or, for page copies, layer 0's) as kernels see them.
// Strides in elements; K and V share them.
struct CacheView {
  void* k;
  void* v;
  int n_pages, page_size, heads, head_dim;
  long long page_stride, token_stride, head_stride;
};

// Positions that a request may have: what its row of the table holds, and at most
// 2^31 - 2^16, so that rounding a length up to whole pages (of up to 2^16
// positions) or tiles stays an int.  (Without that bound a page count of a length
// near 2^31 came out negative, and table entries before the row would be written.)
// The same bound holds for what kernels step through: the pages of a pool, the
// rows of a chunk.
constexpr int kMaxCount = 0x7fff0000;
constexpr int kMaxPositions = kMaxCount;
__host__ __device__ __forceinline__ int most_positions(int max_pages, int page_size) {
  const long long n = (long long)max_pages * page_size;
  return n > kMaxPositions ? kMaxPositions : (int)n;
}

// The chunk of new tokens and the lengths of a call.
struct ChunkArgs {
  const int32_t* q_offsets;   // [R + 1]
  const int32_t* kv_len;      // [R]
  const int32_t* page_table;  // [R, max_pages]
  int R, n_tokens, max_pages;
};

cudaError_t launch_cache_append(const CacheView& c, int esize, const void* k_new, const void* v_new,
                                long long new_token_stride, long long new_head_stride,
                                const ChunkArgs& a, int* status, cudaStream_t s);

// Page management.  Workspace (byte offsets, 256-aligned): words (the status
// word first), per-request or per-pair scratch, the free list and copy list.
struct PagesWorkspace {
  size_t words, start, len, owner, list, src, dst, total;
};
PagesWorkspace pages_workspace_layout(int R, int n_pages);

// The cache as page copies see it: layer 0's view and the step between layers.
struct PagePool {
  CacheView c;
  int esize, layers;
  long long layer_stride;
};
struct PageMeta {
  const int32_t *table, *kv_len, *refcount;
  int32_t *table_out, *kv_len_out, *refcount_out;
  int R, max_pages, n_pages, page_size;
};
cudaError_t launch_pages_resize(const PagePool& pool, const PageMeta& m, const int32_t* new_len,
                                int32_t* free_pages, char* ws, const PagesWorkspace& w,
                                cudaStream_t s);
cudaError_t launch_pages_fork(const PagePool& pool, const PageMeta& m, const int32_t* parent,
                              const int32_t* child, int n, int32_t* free_pages, char* ws,
                              const PagesWorkspace& w, cudaStream_t s);
cudaError_t launch_pages_compact(const PagePool& pool, const PageMeta& m, int32_t* page_map,
                                 int32_t* n_live, char* ws, const PagesWorkspace& w,
                                 cudaStream_t s);
// Pages src[i] -> dst[i], i < n, of K and V in all layers.
cudaError_t launch_pages_copy(const PagePool& pool, const int32_t* src, const int32_t* dst, int n,
                              int* status, cudaStream_t s);

// Token log-probabilities.
struct LogprobsWorkspace {
  size_t rows, parts, gmax, total;
};
LogprobsWorkspace logprobs_workspace_layout(int n_rows, int V);
cudaError_t launch_logprobs(const void* Z, int dtype, long long row_stride, const int32_t* tokens,
                            int n_rows, int V, float invT, int top, float* logp, float* entropy,
                            float* lse, int32_t* top_ids, float* top_logp, char* ws,
                            const LogprobsWorkspace& w, cudaStream_t s);

// Attention over the paged cache.
struct AttnArgs {
  ChunkArgs a;
  CacheView c;
  const void* q;
  long long q_token_stride, q_head_stride;  // elements
  int Hq, G, dtype;
  float scale;
  void* out;    // [n_tokens, Hq, D]
  float* lse;   // [n_tokens, Hq]
};
size_t attention_workspace_bytes(int dtype, int head_dim);
cudaError_t launch_paged_attention(const AttnArgs& a, char* ws, cudaStream_t s);

// The kernels here may be launched while the one before them in the stream ends:
// the launch, and what stands before this wait, then cost nothing.  What that
// one wrote (and all before it) is read, and anything written, after the wait,
// and never by the non-coherent path (__ldg, const __restrict__ parameters): that
// asks for data that nothing writes while the kernel runs, which it does before
// the wait too.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
inline cudaLaunchConfig_t overlapped_launch(dim3 grid, int threads, int smem, cudaStream_t s,
                                            cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace dspark
