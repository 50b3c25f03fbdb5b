// pages.cu -- writing new tokens' K and V into the paged cache, and the
// management of its pages: reserving and freeing (resize), forking, compacting,
// copying.
//
// The tables (page table, lengths, reference counts) are small next to the
// cache; what costs there is latency, so each operation is one kernel of one
// thread-block cluster (8 CTAs x 1024 threads, phases separated by the
// hardware's cluster barrier) and the copy kernel behind it, instead of a
// chain of launches.  Which page an allocation takes depends on nothing but the
// inputs: the lowest free ids, in the order of the requests, found by a prefix
// sum over the counts.
//
// Bounds and figures: the cluster kernels are chains of dependent reads (resize
// of 512 requests over 40,000 pages: 16 us in a graph, 22 us a call from Python,
// whose host side is the longer.  In a graph 11 of them where no length changes; 3
// more for growth, one for releases and one for 19 split pages; compact of 2000
// pages 10 us); the copies and
// the append move bytes: 262 MB of pages read and written in 80 us (6.5 TB/s),
// prompts of 8 k and 16 k new tokens of 8 x 128 (119 MB each way) in 37 us, 4.8 k
// tokens of 512 requests in 7 us, four dependent look-ups behind their loads.
#include <cooperative_groups.h>

#include "append.cuh"
#include "common.cuh"
#include "serving.h"

namespace cg = cooperative_groups;

namespace dspark {

namespace {

constexpr int kClusterCtas = 8;
constexpr int kPageThreads = 1024;
constexpr int kPageWarps = kPageThreads / 32;

// Words at the start of the workspace.  The table kernels run in one cluster
// and leave what the copy kernel behind them (which ends every call) needs:
// each CTA's status bits and count of pages that became free, the number of
// copies, and the free pages without those.
enum { kWordStatus = 0, kWordCopies = 1, kWordFree = 2, kWordFlags = 8, kWordFreed = 16 };

// (a: a length, at most kMaxPositions, or a number of pages, at most as much)
__device__ __forceinline__ int ceil_div(int a, int b) { return (int)(((unsigned)a + b - 1) / b); }

__device__ __forceinline__ int warp_sum_int(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ int warp_scan_incl(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Exclusive prefix of v over the CTA's threads; *total gets the sum.  Uses
// sm[0 .. kPageWarps].
__device__ __forceinline__ int block_scan_excl(int v, int* sm, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int incl = warp_scan_incl(v);
  if (lane == 31) sm[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int w = sm[lane];
    const int wi = warp_scan_incl(w);
    sm[lane] = wi - w;
    if (lane == 31) sm[kPageWarps] = wi;
  }
  __syncthreads();
  const int r = sm[warp] + incl - v;
  *total = sm[kPageWarps];
  __syncthreads();
  return r;
}

// A warp's contiguous share of the pages, in cluster order (CTA rank, warp).
__device__ __forceinline__ void page_share(int n_pages, int rank, int& lo, int& hi) {
  const int warps = kClusterCtas * kPageWarps;
  const int per = ceil_div(ceil_div(n_pages, warps), 32) * 32;
  const long long a = (long long)(rank * kPageWarps + (int)(threadIdx.x >> 5)) * per;
  lo = a < n_pages ? (int)a : n_pages;
  hi = a + per < n_pages ? (int)(a + per) : n_pages;
}

// N counts per warp -> this warp's exclusive prefixes over the whole cluster
// and the cluster's totals, with one cluster barrier.  sm[N][kPageWarps + 1] is
// this call's own; no CTA may leave the kernel before a further barrier (the
// others read its totals).
template <int N>
__device__ __forceinline__ void cluster_prefix(cg::cluster_group& cl, const int (&warp_count)[N],
                                               int (*sm)[kPageWarps + 1], int (&prefix)[N],
                                               int (&total)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0)
    for (int k = 0; k < N; ++k) sm[k][warp] = warp_count[k];
  __syncthreads();
  if (warp < N) {
    const int w = sm[warp][lane];
    const int wi = warp_scan_incl(w);
    sm[warp][lane] = wi - w;
    if (lane == 31) sm[warp][kPageWarps] = wi;  // this CTA's total
  }
  cl.sync();
  const int rank = (int)cl.block_rank();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    int before = 0, all = 0;
#pragma unroll
    for (int c = 0; c < kClusterCtas; ++c) {
      const int t = *cl.map_shared_rank(&sm[k][kPageWarps], c);
      all += t;
      if (c < rank) before += t;
    }
    prefix[k] = before + sm[k][warp];
    total[k] = all;
  }
}

// Counts the pages of [lo, hi) for which pred(p) holds, by one warp.
template <typename Pred>
__device__ __forceinline__ int warp_count(int lo, int hi, Pred pred) {
  const int lane = threadIdx.x & 31;
  int n = 0;
#pragma unroll 4
  for (int p = lo + lane; p < hi; p += 32) n += pred(p) ? 1 : 0;
  return warp_sum_int(n);
}

// Calls put(rank, p) for the pages of [lo, hi) with pred(p), in order, ranks
// from `at`, as long as rank < most.
template <typename Pred, typename Put>
__device__ __forceinline__ void warp_list(int lo, int hi, int at, int most, Pred pred, Put put) {
  const int lane = threadIdx.x & 31;
  for (int b = lo; b < hi && at < most; b += 32) {
    const int p = b + lane;
    const bool y = p < hi && pred(p);
    const unsigned m = __ballot_sync(0xffffffffu, y);
    const int r = at + __popc(m & ((1u << lane) - 1u));
    if (y && r < most) put(r, p);
    at += __popc(m);
  }
}

__device__ __forceinline__ int clamp_len(int n, int most, int* status) {
  if (n < 0 || n > most) {
    flag_status(status, DSPARK_DEV_BAD_INPUT);
    return n < 0 ? 0 : most;
  }
  return n;
}

// Copies the tables into the outputs where those are arrays of their own.
struct MetaCopy {
  const int32_t* from[3];
  int32_t* to[3];
  size_t n[3];
};
__device__ __forceinline__ void copy_meta(const MetaCopy& c, size_t t, size_t T) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (c.from[k] == c.to[k]) continue;
    const bool vec = (((uintptr_t)c.from[k] | (uintptr_t)c.to[k]) & 15u) == 0;
    const size_t n4 = vec ? c.n[k] / 4 : 0;
#pragma unroll 4
    for (size_t i = t; i < n4; i += T) ((int4*)c.to[k])[i] = ((const int4*)c.from[k])[i];
    for (size_t i = 4 * n4 + t; i < c.n[k]; i += T) c.to[k][i] = c.from[k][i];
  }
}
__global__ void __launch_bounds__(256) meta_copy_kernel(const MetaCopy c) {
  copy_meta(c, (size_t)blockIdx.x * blockDim.x + threadIdx.x, (size_t)gridDim.x * blockDim.x);
}

// What the copy kernels do beside the copies, as the end of a call.
struct CopyTail {
  const int* words;     // the table kernel's words (null: a plain copy)
  int32_t* free_pages;  // resize, fork: gets the free pages
  PageMeta m;           // compact: the table is rewritten through page_map
  const int32_t* page_map;
};

// One page of one layer's K or V per (copy, layer, K/V); 16-byte pieces where a
// page is one dense block on 16-byte boundaries.
struct CopyArgs {
  CacheView c;
  int layers, esize, n_max;
  long long layer_stride;
  const int32_t *src, *dst;
  int* status;
  CopyTail tail;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;  // 16-byte loads in flight a thread

// Number of copies; before it, the tail of a table kernel's call.
__device__ __forceinline__ int copy_begin(const CopyArgs& a) {
  const CopyTail& t = a.tail;
  if (!t.words) return a.n_max;
  wait_for_previous();
  if (t.free_pages && blockIdx.x == 0 && threadIdx.x == 0) {
    int f = 0, freed = 0;
    for (int i = 0; i < kClusterCtas; ++i) {
      f |= __ldcg(t.words + kWordFlags + i);
      freed += __ldcg(t.words + kWordFreed + i);
    }
    *t.free_pages = __ldcg(t.words + kWordFree) + freed;
    *a.status = f;
  }
  if (t.page_map) {
    const PageMeta& m = t.m;
    const size_t n = (size_t)m.R * m.max_pages;
    const int most = most_positions(m.max_pages, m.page_size);
    for (size_t i = (size_t)blockIdx.x * kCopyThreads + threadIdx.x; i < n;
         i += (size_t)gridDim.x * kCopyThreads) {
      const int r = (int)(i / m.max_pages), j = (int)(i - (size_t)r * m.max_pages);
      int p = m.table[i];
      const int L = clamp_len(m.kv_len[r], most, a.status);
      if (j < ceil_div(L, m.page_size)) {
        const int q = p >= 0 && p < m.n_pages ? __ldcg(t.page_map + p) : -1;
        if (q < 0)
          flag_status(a.status, DSPARK_DEV_BAD_INPUT);
        else
          p = q;
      }
      m.table_out[i] = p;
    }
  }
  const int n = __ldcg(t.words + kWordCopies);
  return n < a.n_max ? n : a.n_max;
}

// Copy i's pages; false: nothing to copy (in a call of dspark_pages_copy, out of range).
__device__ __forceinline__ bool copy_pair(const CopyArgs& a, int i, bool flag, int& s, int& d) {
  s = __ldcg(a.src + i), d = __ldcg(a.dst + i);
  if (s >= 0 && s < a.c.n_pages && d >= 0 && d < a.c.n_pages) return true;
  if (!a.tail.words && flag) flag_status(a.status, DSPARK_DEV_BAD_INPUT);
  return false;
}

// The copies of n pairs by `teams` teams of kThreads threads (a CTA, or a
// warp), of which this is number `team` and `t` its thread.
template <int kThreads>
__device__ __forceinline__ void copy_dense(const CopyArgs& a, int n, int team, int teams, int t) {
  const int vecs = (int)((size_t)a.c.page_size * a.c.heads * a.c.head_dim * a.esize / 16);
  const int piece = kThreads * kCopyUnroll;
  const int pieces = (vecs + piece - 1) / piece;
  const long long units = (long long)n * 2 * a.layers * pieces;
  // As many teams as share the units evenly: a last round that few of them had
  // work in would leave the memory idle.
  const long long rounds = (units + teams - 1) / teams;
  const int used = rounds > 0 ? (int)((units + rounds - 1) / rounds) : 0;
  if (team >= used) return;
  for (long long u = team; u < units; u += used) {
    const int pc = (int)(u % pieces);
    long long w = u / pieces;
    const bool is_v = w & 1;
    w >>= 1;
    const int layer = (int)(w % a.layers), i = (int)(w / a.layers);
    int s, d;
    if (!copy_pair(a, i, t == 0, s, d)) continue;
    char* base = (char*)(is_v ? a.c.v : a.c.k);
    const uint4* from =
        (const uint4*)(base + (layer * a.layer_stride + s * a.c.page_stride) * a.esize);
    uint4* to = (uint4*)(base + (layer * a.layer_stride + d * a.c.page_stride) * a.esize);
    const int v0 = pc * piece + t;
    uint4 x[kCopyUnroll];
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k)
      if (v0 + k * kThreads < vecs) x[k] = __ldcs(&from[v0 + k * kThreads]);
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k)
      if (v0 + k * kThreads < vecs) __stcs(&to[v0 + k * kThreads], x[k]);
  }
}

__global__ void __launch_bounds__(kCopyThreads) pages_copy_dense_kernel(const CopyArgs a) {
  copy_dense<kCopyThreads>(a, copy_begin(a), blockIdx.x, gridDim.x, threadIdx.x);
}

// Any strides: element by element, the head dimension over the lanes.
template <typename E>
__device__ __forceinline__ void copy_rows(const CopyArgs& a, int n, int warp, int warps) {
  const int rows = a.c.page_size * a.c.heads;
  const long long units = (long long)n * 2 * a.layers * rows;
  const int lane = threadIdx.x & 31;
  for (long long u = warp; u < units; u += warps) {
    const int row = (int)(u % rows);
    long long w = u / rows;
    const bool is_v = w & 1;
    w >>= 1;
    const int layer = (int)(w % a.layers), i = (int)(w / a.layers);
    int s, d;
    if (!copy_pair(a, i, lane == 0, s, d)) continue;
    E* base = (E*)(is_v ? a.c.v : a.c.k) + layer * a.layer_stride +
              (row / a.c.heads) * a.c.token_stride + (row % a.c.heads) * a.c.head_stride;
    const E* from = base + s * a.c.page_stride;
    E* to = base + d * a.c.page_stride;
    for (int e = lane; e < a.c.head_dim; e += 32) to[e] = from[e];
  }
}
template <typename E>
__global__ void __launch_bounds__(kCopyThreads) pages_copy_rows_kernel(const CopyArgs a) {
  copy_rows<E>(a, copy_begin(a), blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5),
               gridDim.x * (kCopyThreads / 32));
}

struct ResizeArgs {
  PageMeta m;
  MetaCopy copy;  // done here first (all from == to: not)
  const int32_t* new_len;
  int* words;
  int* start;  // [R]: first allocation of the request
  int* cow;    // [R]: copies before it; bit 31: it copies a shared page
  int* list;   // [n_pages]: the lowest free pages in order
  int* src;    // [R] copy list
  int* dst;
  int32_t* free_pages;
  CopyArgs pages;  // the copies, where this kernel makes them itself
  int copy_here;   // 0: the copy kernel behind it does, 1: dense pages, 2: row by row
};

__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kPageThreads, 1)
pages_resize_kernel(const ResizeArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ int sm[1][kPageWarps + 1], scan[kPageWarps + 1], flags, freed, need_sm, copies_sm;
  const int rank = (int)cl.block_rank();
  const int lane = threadIdx.x & 31;
  const int gthread = rank * kPageThreads + (int)threadIdx.x;
  const int gwarp = rank * kPageWarps + (threadIdx.x >> 5), warps = kClusterCtas * kPageWarps;
  const PageMeta& m = a.m;
  const int S = m.page_size, P = m.max_pages;
  const int most = most_positions(P, S);
  int* const rc = m.refcount_out;
  int* const status = &flags;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) flags = freed = 0;
  wait_for_previous();
  __syncthreads();
  copy_meta(a.copy, gthread, kClusterCtas * kPageThreads);
  cl.sync();

  // CTA 0's first requests, for step 2: lengths and a grower's partly filled
  // last page (no release touches either).
  int pre_L = 0, pre_N = 0, pre_p = -1;
  if (rank == 0 && (int)threadIdx.x < m.R) {
    pre_L = clamp_len(m.kv_len[threadIdx.x], most, status);
    pre_N = clamp_len(a.new_len[threadIdx.x], most, status);
    if (pre_N > pre_L && pre_L % S != 0)
      pre_p = __ldcg(&m.table_out[(size_t)threadIdx.x * P + pre_L / S]);
  }

  // 1. Pages past the new length lose a reference.
  for (int r = gwarp; r < m.R; r += warps) {
    const int L = clamp_len(m.kv_len[r], most, status), N = clamp_len(a.new_len[r], most, status);
    int32_t* row = m.table_out + (size_t)r * P;
    for (int j = ceil_div(N, S) + lane; j < ceil_div(L, S); j += 32) {
      const int p = row[j];
      if (p < 0 || p >= m.n_pages)
        flag_status(status, DSPARK_DEV_BAD_INPUT);
      else
        atomicSub(&rc[p], 1);
      row[j] = -1;
    }
  }
  cl.sync();

  // 2. Free pages of this warp's share; the requests' needs, in order, by CTA 0.
  int lo, hi;
  page_share(m.n_pages, rank, lo, hi);
  const auto is_free = [&](int p) { return __ldcg(&rc[p]) == 0; };
  const int mine[1] = {warp_count(lo, hi, is_free)};
  if (rank == 0) {
    int base = 0, copies = 0;
    for (int r0 = 0; r0 < m.R; r0 += kPageThreads) {
      const int r = r0 + (int)threadIdx.x;
      int need = 0, cow = 0;
      if (r < m.R) {
        const int L = r0 == 0 ? pre_L : clamp_len(m.kv_len[r], most, status);
        const int N = r0 == 0 ? pre_N : clamp_len(a.new_len[r], most, status);
        if (N > L) {
          if (L % S != 0) {
            const int p = r0 == 0 ? pre_p : __ldcg(&m.table_out[(size_t)r * P + L / S]);
            if (p < 0 || p >= m.n_pages)
              flag_status(status, DSPARK_DEV_BAD_INPUT);
            else
              cow = __ldcg(&rc[p]) > 1 ? 1 : 0;
          }
          need = cow + ceil_div(N, S) - ceil_div(L, S);
        }
      }
      int total, n_cow;
      const int at = block_scan_excl(need, scan, &total);
      const int ci = block_scan_excl(cow, scan, &n_cow);
      if (r < m.R) {
        a.start[r] = base + at;
        a.cow[r] = (int)((unsigned)(copies + ci) | (cow ? 0x80000000u : 0u));
      }
      base += total;
      copies += n_cow;
    }
    if (threadIdx.x == 0) {
      need_sm = base;
      copies_sm = copies;
      a.words[kWordCopies] = copies;
    }
  }
  int at[1], n_free[1];
  cluster_prefix<1>(cl, mine, sm, at, n_free);
  const int need_all = *cl.map_shared_rank(&need_sm, 0);
  const int copies = *cl.map_shared_rank(&copies_sm, 0);
  if (need_all > n_free[0] && threadIdx.x == 0 && rank == 0) flag_status(status, DSPARK_DEV_NO_PAGES);

  // 3. The lowest free pages, as many as are wanted.
  warp_list(lo, hi, at[0], need_all, is_free, [&](int i, int p) { a.list[i] = p; });
  cl.sync();

  // 4. Each request takes its share of the list.
  for (int r = gwarp; r < m.R; r += warps) {
    const int L = clamp_len(m.kv_len[r], most, status), N = clamp_len(a.new_len[r], most, status);
    int out_len = N;
    if (N > L) {
      const unsigned cw = (unsigned)__ldcg(&a.cow[r]);
      const int cow = (int)(cw >> 31), first = __ldcg(&a.start[r]);
      const int old = ceil_div(L, S), need = cow + ceil_div(N, S) - old;
      int got = n_free[0] - first;
      got = got < 0 ? 0 : got > need ? need : got;
      int32_t* row = m.table_out + (size_t)r * P;
      int from = -1, to = -1;
      if (cow && got == 0) {
        out_len = L;
      } else {
        const int grown = got - cow;
        for (int j = lane; j < grown; j += 32) {
          const int p = __ldcg(&a.list[first + cow + j]);
          row[old + j] = p;
          rc[p] = 1;
        }
        if (cow && lane == 0) {
          from = __ldcg(&row[L / S]);
          to = __ldcg(&a.list[first]);
          row[L / S] = to;
          rc[to] = 1;
          if (atomicSub(&rc[from], 1) == 1) atomicAdd(&freed, 1);
        }
        const long long room = (long long)(old + grown) * S;
        out_len = room < N ? (int)room : N;
      }
      if (cow && lane == 0) {
        a.src[cw & 0x7fffffffu] = from;
        a.dst[cw & 0x7fffffffu] = to;  // -1: not copied, the pool ran out
      }
    }
    __syncwarp();
    if (lane == 0) m.kv_len_out[r] = out_len;
  }
  const int left = n_free[0] - (need_all < n_free[0] ? need_all : n_free[0]);
  if (!a.copy_here) {
    __syncthreads();
    if (threadIdx.x == 0) {
      a.words[kWordFlags + rank] = flags;
      a.words[kWordFreed + rank] = freed;
      if (rank == 0) a.words[kWordFree] = left;
    }
    return;
  }
  cl.sync();
  if (copies) {
    if (a.copy_here == 1)
      copy_dense<32>(a.pages, copies, gwarp, warps, lane);
    else if (a.pages.esize == 2)
      copy_rows<uint16_t>(a.pages, copies, gwarp, warps);
    else
      copy_rows<uint32_t>(a.pages, copies, gwarp, warps);
  }
  if (rank == 0 && threadIdx.x == 0) {
    int f = 0, more = 0;
    for (int c = 0; c < kClusterCtas; ++c) {
      f |= *cl.map_shared_rank(&flags, c);
      more += *cl.map_shared_rank(&freed, c);
    }
    a.words[kWordStatus] = f;
    *a.free_pages = left + more;
  }
  cl.sync();  // (rank 0 reads the others' shared memory)
}

struct ForkArgs {
  PageMeta m;
  MetaCopy copy;
  const int32_t *parent, *child;
  int n;
  int* words;
  int* start;  // [n <= R]: first allocation
  int* len;    // [n] the parent's length, -1: the pair is skipped
  int* owner;  // [R]: the first pair that names a child
  int* list;
  int* src;
  int* dst;
};

__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kPageThreads, 1)
pages_fork_kernel(const ForkArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ int sm[1][kPageWarps + 1], scan[kPageWarps + 1], flags, need_sm;
  const int rank = (int)cl.block_rank();
  const int lane = threadIdx.x & 31;
  const int gwarp = rank * kPageWarps + (threadIdx.x >> 5), warps = kClusterCtas * kPageWarps;
  const PageMeta& m = a.m;
  const int S = m.page_size, P = m.max_pages;
  const int most = most_positions(P, S);
  int* const rc = m.refcount_out;
  int* const status = &flags;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) flags = 0;
  wait_for_previous();
  __syncthreads();
  // Up to the last barrier only the inputs are read and, where the outputs are
  // arrays of their own, those filled from them.
  int lo, hi;
  page_share(m.n_pages, rank, lo, hi);
  const auto is_free = [&](int p) { return m.refcount[p] == 0; };
  const int mine[1] = {warp_count(lo, hi, is_free)};
  // The pairs' needs, in order, by CTA 0.  A pair whose child holds pages, is
  // named twice or is out of range is skipped and flagged.
  if (rank == 0) {
    for (int r = threadIdx.x; r < m.R; r += kPageThreads) a.owner[r] = 0x7fffffff;
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += kPageThreads) {
      const int c = a.child[i];
      if (c >= 0 && c < m.R) atomicMin(&a.owner[c], i);
    }
    __syncthreads();
    int base = 0;
    for (int i0 = 0; i0 < a.n; i0 += kPageThreads) {
      const int i = i0 + (int)threadIdx.x;
      int need = 0, L = -1;
      if (i < a.n) {
        const int p = a.parent[i], c = a.child[i];
        const bool ok = p >= 0 && p < m.R && c >= 0 && c < m.R && m.kv_len[c] == 0 &&
                        __ldcg(&a.owner[c]) == i;
        if (ok) {
          L = clamp_len(m.kv_len[p], most, status);
          need = L % S != 0 ? 1 : 0;
          if (need) {
            const int q = m.table[(size_t)p * P + L / S];
            if (q < 0 || q >= m.n_pages) {
              flag_status(status, DSPARK_DEV_BAD_INPUT);
              L = L / S * S;
              need = 0;
            }
          }
        } else {
          flag_status(status, DSPARK_DEV_BAD_INPUT);
        }
      }
      int total;
      const int at = block_scan_excl(need, scan, &total);
      if (i < a.n) {
        a.start[i] = base + at;
        a.len[i] = L;
      }
      base += total;
    }
    if (threadIdx.x == 0) {
      need_sm = base;
      a.words[kWordCopies] = base;
    }
  } else {
    copy_meta(a.copy, gwarp * 32 + lane - kPageThreads, (kClusterCtas - 1) * kPageThreads);
  }
  int at[1], n_free[1];
  cluster_prefix<1>(cl, mine, sm, at, n_free);
  const int need_all = *cl.map_shared_rank(&need_sm, 0);
  if (need_all > n_free[0] && threadIdx.x == 0 && rank == 0) flag_status(status, DSPARK_DEV_NO_PAGES);
  warp_list(lo, hi, at[0], need_all, is_free, [&](int i, int p) { a.list[i] = p; });
  cl.sync();

  for (int i = gwarp; i < a.n; i += warps) {
    const int L = __ldcg(&a.len[i]);
    if (L < 0) continue;
    const int32_t* from = m.table_out + (size_t)a.parent[i] * P;
    int32_t* to = m.table_out + (size_t)a.child[i] * P;
    const int full = L / S;
    for (int j = lane; j < full; j += 32) {
      const int p = __ldcg(&from[j]);
      if (p < 0 || p >= m.n_pages)
        flag_status(status, DSPARK_DEV_BAD_INPUT);
      else
        atomicAdd(&rc[p], 1);
      to[j] = p;
    }
    if (lane == 0) {
      int out_len = full * S;
      if (L % S != 0) {
        const int k = __ldcg(&a.start[i]);  // also this copy's place in the list
        int p = -1;
        if (k < n_free[0]) {
          p = __ldcg(&a.list[k]);
          to[full] = p;
          rc[p] = 1;
          out_len = L;
        }
        a.src[k] = __ldcg(&from[full]);
        a.dst[k] = p;
      }
      m.kv_len_out[a.child[i]] = out_len;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    a.words[kWordFlags + rank] = flags;
    a.words[kWordFreed + rank] = 0;
    if (rank == 0) a.words[kWordFree] = n_free[0] - (need_all < n_free[0] ? need_all : n_free[0]);
  }
}

struct CompactArgs {
  PageMeta m;
  MetaCopy copy;
  int32_t* page_map;
  int32_t* n_live;
  int* words;
  int* src;
  int* dst;
};

// Lists the moves: the i-th live page with id >= n_live goes to the i-th free
// id < n_live, where n_live is the number of live pages.
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kPageThreads, 1)
pages_compact_kernel(const CompactArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ int sm1[1][kPageWarps + 1], sm2[2][kPageWarps + 1];
  const int rank = (int)cl.block_rank();
  const int lane = threadIdx.x & 31;
  const PageMeta& m = a.m;
  const int32_t* rc = m.refcount;
  int lo, hi, none[1], live[1], at[2], n[2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_previous();
  page_share(m.n_pages, rank, lo, hi);
  copy_meta(a.copy, rank * kPageThreads + (int)threadIdx.x, kClusterCtas * kPageThreads);
  const int n_mine[1] = {warp_count(lo, hi, [&](int p) { return rc[p] > 0; })};
  cluster_prefix<1>(cl, n_mine, sm1, none, live);
  const int n_live = live[0];
  const auto high = [&](int p) { return p >= n_live && rc[p] > 0; };
  const auto low = [&](int p) { return p < n_live && rc[p] <= 0; };
  const int n_both[2] = {warp_count(lo, hi, high), warp_count(lo, hi, low)};
  cluster_prefix<2>(cl, n_both, sm2, at, n);
  warp_list(lo, hi, at[0], n[0], high, [&](int i, int p) { a.src[i] = p; });
  warp_list(lo, hi, at[1], n[1], low, [&](int i, int p) { a.dst[i] = p; });
  for (int p = lo + lane; p < hi; p += 32)
    if (!high(p)) a.page_map[p] = rc[p] > 0 ? p : -1;
  cl.sync();
  for (int i = rank * kPageThreads + (int)threadIdx.x; i < n[0]; i += kClusterCtas * kPageThreads) {
    const int s = __ldcg(&a.src[i]), d = __ldcg(&a.dst[i]);
    a.page_map[s] = d;
    m.refcount_out[d] = __ldcg(&rc[s]);
    m.refcount_out[s] = 0;
  }
  if (rank == 0 && threadIdx.x == 0) {
    *a.n_live = n_live;
    a.words[kWordCopies] = n[0];
    a.words[kWordStatus] = 0;  // (raised by the table rewrite behind this kernel)
  }
}

MetaCopy meta_args(const PageMeta& m, bool table, bool len) {
  MetaCopy c;
  c.from[0] = m.table, c.to[0] = table ? m.table_out : (int32_t*)m.table;
  c.n[0] = (size_t)m.R * m.max_pages;
  c.from[1] = m.kv_len, c.to[1] = len ? m.kv_len_out : (int32_t*)m.kv_len, c.n[1] = (size_t)m.R;
  c.from[2] = m.refcount, c.to[2] = m.refcount_out;
  c.n[2] = (size_t)m.n_pages;
  return c;
}

// Tables of up to kMetaInKernel entries are copied by the cluster kernel
// itself, larger ones by a launch of their own over all SMs.  A resize whose
// outputs are arrays of their own, inside a CUDA graph, with / without the extra
// launch: 32 k entries 11.5 / 11.1 us, 262 k 11.4 / 13.4, 1 M 14.9 / 24.1; outside
// a graph the launch costs the host 3 us more.
constexpr size_t kMetaInKernel = 1u << 17;
// A resize copies the shared pages that it has to split in the cluster kernel
// where even all requests' pages come to this many bytes: about as far as a call
// that has to split all of them loses no more by it than one that splits none
// gains.  In a graph, 256 requests, in the kernel / by the second launch:
//                      1 MB         2 MB         4 MB         8 MB         16 MB
//   no split         8.8 / 10.0   8.8 / 10.0   8.8 / 10.1   8.7 / 10.7   8.8 / 11.0
//   every 16th      12.5 / 11.4  12.5 / 11.4  12.4 / 11.4  12.5 / 12.2  13.9 / 12.4
//   all             14.3 / 12.5  16.9 / 12.5  22.4 / 12.5  33.6 / 14.4  55.2 / 17.8
// Calls outside a graph, outputs given: none 9.1 / 10.7 .. 11.1, all 14.9 / 12.4
// (1 MB), 23.0 / 12.5 (4 MB), 34.2 / 14.4 (8 MB).
constexpr size_t kCopyInKernel = 1u << 20;
cudaError_t split_meta(MetaCopy* c, cudaStream_t s) {
  size_t most = 0, all = 0;
  for (int k = 0; k < 3; ++k)
    if (c->from[k] != c->to[k]) {
      most = most < c->n[k] ? c->n[k] : most;
      all += c->n[k];
    }
  if (all <= kMetaInKernel) return cudaSuccess;
  size_t ctas = (most + 1023) / 1024;
  if (ctas > 608) ctas = 608;
  meta_copy_kernel<<<(int)ctas, 256, 0, s>>>(*c);
  for (int k = 0; k < 3; ++k) c->from[k] = c->to[k];
  return cudaGetLastError();
}

// ------------------------------------------------------------------ append
struct AppendArgs {
  CacheView c;
  ChunkArgs a;
  const void *k_new, *v_new;
  long long tok_stride, head_stride;  // of the new rows
  int* status;
};

// One warp a token: VE elements (16 bytes, or one where alignment does not
// allow) a lane and step.  The first kAppendAhead steps' rows are loaded before
// the token's request, position and page are looked up (four dependent loads).
constexpr int kAppendAhead = 4;
template <typename E, int VE>
__global__ void __launch_bounds__(256) cache_append_kernel(const AppendArgs p) {
  struct alignas(sizeof(E) * VE) Vec {
    E e[VE];
  };
  const int lane = threadIdx.x & 31;
  const int S = p.c.page_size;
  const int per_head = p.c.head_dim / VE, n = p.c.heads * per_head;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (attention over the cache mostly follows)
  wait_for_previous();
  if (blockIdx.x == 0) {
    append_status(p.c, p.a, p.status);
    return;
  }
  for (int t = (blockIdx.x - 1) * 8 + (threadIdx.x >> 5); t < p.a.n_tokens; t += (gridDim.x - 1) * 8) {
    const E* kn = (const E*)p.k_new + t * p.tok_stride;
    const E* vn = (const E*)p.v_new + t * p.tok_stride;
    Vec kx[kAppendAhead], vx[kAppendAhead];
#pragma unroll
    for (int k = 0; k < kAppendAhead; ++k) {
      const int i = lane + 32 * k;
      if (i < n) {
        const int h = i / per_head, d = (i - h * per_head) * VE;
        kx[k] = *(const Vec*)(kn + h * p.head_stride + d);
        vx[k] = *(const Vec*)(vn + h * p.head_stride + d);
      }
    }
    const int r = find_request(p.a.q_offsets, p.a.R, t);
    const int end = p.a.q_offsets[r + 1];
    const long long pos = (long long)p.a.kv_len[r] - end + t;
    const long long slot = pos / S;
    int page = -1;
    if (t >= p.a.q_offsets[r] && t < end && pos >= 0 && pos < most_positions(p.a.max_pages, S))
      page = p.a.page_table[(size_t)r * p.a.max_pages + slot];
    if (page < 0 || page >= p.c.n_pages) continue;  // flagged by CTA 0, or padding
    const long long dst0 = page * p.c.page_stride + (pos - slot * S) * p.c.token_stride;
#pragma unroll
    for (int k = 0; k < kAppendAhead; ++k) {
      const int i = lane + 32 * k;
      if (i < n) {
        const int h = i / per_head, d = (i - h * per_head) * VE;
        *(Vec*)((E*)p.c.k + dst0 + h * p.c.head_stride + d) = kx[k];
        *(Vec*)((E*)p.c.v + dst0 + h * p.c.head_stride + d) = vx[k];
      }
    }
#pragma unroll 4
    for (int i = lane + 32 * kAppendAhead; i < n; i += 32) {
      const int h = i / per_head, d = (i - h * per_head) * VE;
      const Vec a = *(const Vec*)(kn + h * p.head_stride + d);
      const Vec b = *(const Vec*)(vn + h * p.head_stride + d);
      *(Vec*)((E*)p.c.k + dst0 + h * p.c.head_stride + d) = a;
      *(Vec*)((E*)p.c.v + dst0 + h * p.c.head_stride + d) = b;
    }
  }
}

bool dense_page(const CacheView& c) {
  const long long D = c.head_dim;
  const bool thd = (c.heads == 1 || c.head_stride == D) &&
                   (c.page_size == 1 || c.token_stride == c.heads * D);
  const bool htd = (c.page_size == 1 || c.token_stride == D) &&
                   (c.heads == 1 || c.head_stride == c.page_size * D);
  return thd || htd;
}

}  // namespace

PagesWorkspace pages_workspace_layout(int R, int n_pages) {
  PagesWorkspace w;
  const size_t lists = (size_t)(R > n_pages ? R : n_pages) * sizeof(int);
  w.words = 0;
  w.start = 256;
  w.len = align_up256(w.start + (size_t)R * sizeof(int));
  w.owner = align_up256(w.len + (size_t)R * sizeof(int));
  w.list = align_up256(w.owner + (size_t)R * sizeof(int));
  w.src = align_up256(w.list + (size_t)n_pages * sizeof(int));
  w.dst = align_up256(w.src + lists);
  w.total = align_up256(w.dst + lists);
  return w;
}

static size_t page_bytes_of(const CopyArgs& a) {
  return (size_t)a.c.page_size * a.c.heads * a.c.head_dim * a.esize;
}

// Whether pages are dense blocks that move in 16-byte pieces.
static bool copy_vec(const CopyArgs& a) {
  const CacheView& c = a.c;
  return dense_page(c) && page_bytes_of(a) % 16 == 0 && (c.page_stride * a.esize) % 16 == 0 &&
         (a.layer_stride * a.esize) % 16 == 0 && (((uintptr_t)c.k | (uintptr_t)c.v) & 15u) == 0;
}

static cudaError_t launch_copy(const CopyArgs& a, cudaStream_t s) {
  const CacheView& c = a.c;
  const size_t page_bytes = page_bytes_of(a);
  const bool vec = copy_vec(a);
  const long long per = vec ? (long long)((page_bytes / 16 + kCopyThreads * kCopyUnroll - 1) /
                                          (kCopyThreads * kCopyUnroll))
                            : ((long long)c.page_size * c.heads + 7) / 8;
  // Up to 8 CTAs an SM.
  const long long units = per * 2 * a.layers * (a.n_max > 0 ? a.n_max : 1);
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg =
      overlapped_launch(dim3((unsigned)(units < 1216 ? units : 1216)), kCopyThreads, 0, s, &attr);
  if (!a.tail.words) cfg.numAttrs = 0;  // (a plain copy does not wait)
  return cudaLaunchKernelEx(&cfg, vec            ? pages_copy_dense_kernel
                                  : a.esize == 2 ? pages_copy_rows_kernel<uint16_t>
                                                 : pages_copy_rows_kernel<uint32_t>,
                            a);
}

cudaError_t launch_pages_resize(const PagePool& pool, const PageMeta& m, const int32_t* new_len,
                                int32_t* free_pages, char* ws, const PagesWorkspace& w,
                                cudaStream_t s) {
  int* words = (int*)(ws + w.words);
  ResizeArgs a{m, meta_args(m, true, false), new_len, words, (int*)(ws + w.start),
               (int*)(ws + w.owner), (int*)(ws + w.list), (int*)(ws + w.src), (int*)(ws + w.dst),
               free_pages, CopyArgs{}, 0};
  a.pages = CopyArgs{pool.c, pool.layers, pool.esize, m.R, pool.layer_stride, a.src, a.dst,
                     words, CopyTail{words, free_pages, m, nullptr}};
  if ((size_t)m.R * 2 * pool.layers * page_bytes_of(a.pages) <= kCopyInKernel)
    a.copy_here = copy_vec(a.pages) ? 1 : 2;
  cudaError_t e = split_meta(&a.copy, s);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = overlapped_launch(dim3(kClusterCtas), kPageThreads, 0, s, &attr);
  e = cudaLaunchKernelEx(&cfg, pages_resize_kernel, a);
  if (e != cudaSuccess || a.copy_here) return e;
  return launch_copy(a.pages, s);
}

cudaError_t launch_pages_fork(const PagePool& pool, const PageMeta& m, const int32_t* parent,
                              const int32_t* child, int n, int32_t* free_pages, char* ws,
                              const PagesWorkspace& w, cudaStream_t s) {
  int* words = (int*)(ws + w.words);
  ForkArgs a{m, meta_args(m, true, true), parent, child, n, words, (int*)(ws + w.start),
             (int*)(ws + w.len), (int*)(ws + w.owner), (int*)(ws + w.list), (int*)(ws + w.src),
             (int*)(ws + w.dst)};
  cudaError_t e = split_meta(&a.copy, s);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = overlapped_launch(dim3(kClusterCtas), kPageThreads, 0, s, &attr);
  e = cudaLaunchKernelEx(&cfg, pages_fork_kernel, a);
  if (e != cudaSuccess) return e;
  return launch_copy(CopyArgs{pool.c, pool.layers, pool.esize, n, pool.layer_stride, a.src, a.dst,
                              words, CopyTail{words, free_pages, m, nullptr}}, s);
}

cudaError_t launch_pages_compact(const PagePool& pool, const PageMeta& m, int32_t* page_map,
                                 int32_t* n_live, char* ws, const PagesWorkspace& w, cudaStream_t s) {
  int* words = (int*)(ws + w.words);
  CompactArgs a{m, meta_args(m, false, false), page_map, n_live, words, (int*)(ws + w.src),
                (int*)(ws + w.dst)};
  cudaError_t e = split_meta(&a.copy, s);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = overlapped_launch(dim3(kClusterCtas), kPageThreads, 0, s, &attr);
  e = cudaLaunchKernelEx(&cfg, pages_compact_kernel, a);
  if (e != cudaSuccess) return e;
  return launch_copy(CopyArgs{pool.c, pool.layers, pool.esize, m.n_pages, pool.layer_stride, a.src,
                              a.dst, words, CopyTail{words, nullptr, m, page_map}}, s);
}

cudaError_t launch_pages_copy(const PagePool& pool, const int32_t* src, const int32_t* dst, int n,
                              int* status, cudaStream_t s) {
  const cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int), s);
  if (e != cudaSuccess || n == 0) return e;
  return launch_copy(CopyArgs{pool.c, pool.layers, pool.esize, n, pool.layer_stride, src, dst, status,
                              CopyTail{}}, s);
}

cudaError_t launch_cache_append(const CacheView& c, int esize, const void* k_new, const void* v_new,
                                long long new_token_stride, long long new_head_stride,
                                const ChunkArgs& a, int* status, cudaStream_t s) {
  AppendArgs p{c, a, k_new, v_new, new_token_stride, new_head_stride, status};
  const int ve = 16 / esize;
  const bool vec = c.head_dim % ve == 0 && c.page_stride % ve == 0 && c.token_stride % ve == 0 &&
                   c.head_stride % ve == 0 && new_token_stride % ve == 0 &&
                   new_head_stride % ve == 0 &&
                   (((uintptr_t)c.k | (uintptr_t)c.v | (uintptr_t)k_new | (uintptr_t)v_new) & 15u) == 0;
  int ctas = (a.n_tokens + 7) / 8;
  ctas = (ctas < 1215 ? ctas : 1215) + 1;  // (the first one for the status word: also without tokens)
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = overlapped_launch(dim3(ctas), 256, 0, s, &attr);
  if (esize == 2)
    return vec ? cudaLaunchKernelEx(&cfg, cache_append_kernel<uint16_t, 8>, p)
               : cudaLaunchKernelEx(&cfg, cache_append_kernel<uint16_t, 1>, p);
  return vec ? cudaLaunchKernelEx(&cfg, cache_append_kernel<uint32_t, 4>, p)
             : cudaLaunchKernelEx(&cfg, cache_append_kernel<uint32_t, 1>, p);
}

}  // namespace dspark
