// append.cuh -- what the kernels share that write a chunk's rows into the cache
// or read them back: which request a row belongs to, and the status word.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "serving.h"

namespace dspark {

// The request whose chunk holds token t: the largest r with q_offsets[r] <= t
// (later empty requests have larger offsets or follow it with the same one).
// 32 probes a step: two dependent loads for up to 1024 requests.
__device__ __forceinline__ int find_request(const int32_t* off, int R, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = R;  // off[lo] <= t (taken as given for lo = 0), off[hi] > t
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step;
    const bool le = i < hi && off[i] <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, le));
    const int nlo = lo + k * step;
    const int nhi = nlo + step;
    lo = nlo;
    hi = nhi < hi ? nhi : hi;
  }
  return lo;
}

// Whether any new token has no place in the cache, or an offset lies past the
// rows given (the positions counted for them stay unwritten), by one CTA, request
// by request (a request a thread, its further pages by the warp): the status word,
// which so needs no clearing before the launch (a launch of its own cost 2 of 12
// us for 512 requests).  `bad`: what a thread has found amiss before.
__device__ __forceinline__ void append_status(const CacheView& c, const ChunkArgs& a, int* status,
                                              bool bad = false) {
  const int lane = threadIdx.x & 31, S = c.page_size;
  const auto check = [&](int r, long long j) {
    const int page = a.page_table[(size_t)r * a.max_pages + j];
    bad |= page < 0 || page >= c.n_pages;
  };
  for (int r0 = 0; r0 < a.R; r0 += blockDim.x) {  // a request a thread
    const int r = r0 + (int)threadIdx.x;
    long long s0 = 0, s1 = -1;  // the pages that its tokens go to
    if (r < a.R) {
      const int b = a.q_offsets[r], e = a.q_offsets[r + 1], L = a.kv_len[r];
      bad |= b > e || e > a.n_tokens || (r == 0 && b != 0);
      const int t0 = b < 0 ? 0 : b, t1 = e < a.n_tokens ? e : a.n_tokens;
      if (t0 < t1) {
        const long long base = (long long)L - e;  // a token's position less its number
        bad |= base + t0 < 0;
        s0 = base + t0 < 0 ? 0 : (base + t0) / S;
        const long long last = base + t1 - 1, most = most_positions(a.max_pages, S);
        bad |= last >= most;
        s1 = last < 0 ? -1 : (last < most ? last : most - 1) / S;
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (s0 + k <= s1) check(r, s0 + k);
    for (unsigned more = __ballot_sync(0xffffffffu, s0 + 2 <= s1); more; more &= more - 1) {
      const int src = __ffs(more) - 1;
      const long long j0 = __shfl_sync(0xffffffffu, s0, src) + 2, j1 = __shfl_sync(0xffffffffu, s1, src);
      const int row = __shfl_sync(0xffffffffu, r, src);
#pragma unroll 4
      for (long long j = j0 + lane; j <= j1; j += 32) check(row, j);
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) *status = any ? DSPARK_DEV_BAD_INPUT : 0;
}

// A row's place: its position, and its page (-1: it has none) and slot there.
struct RowPlace {
  long long pos;
  int page, slot;
};
__device__ __forceinline__ RowPlace find_place(const CacheView& c, const ChunkArgs& a, int t) {
  const int r = find_request(a.q_offsets, a.R, t);
  const int end = a.q_offsets[r + 1];
  RowPlace p;
  p.pos = (long long)a.kv_len[r] - end + t;
  p.page = -1;
  p.slot = 0;
  if (t >= a.q_offsets[r] && t < end && p.pos >= 0 && p.pos < most_positions(a.max_pages, c.page_size)) {
    const int j = (int)p.pos / c.page_size;
    p.slot = (int)p.pos - j * c.page_size;
    p.page = a.page_table[(size_t)r * a.max_pages + j];
    if (p.page >= c.n_pages) p.page = -1;
  }
  return p;
}

}  // namespace dspark
