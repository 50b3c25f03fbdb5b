// attention.cuh -- what the kernels of attention over the paged cache share:
// the division of the work and the partial results that a division leaves.
//
// An item is a block of up to `mr` rows of one request's chunk for one K/V head.
// A row is (token, query head of the group): row = token * G + g, so all G
// query heads that share a K/V head read its tiles once.  An item walks its
// keys in tiles of TN; its work is counted as one unit a tile (an item without
// keys has one) and `item_units` more for its start and end.  The units of
// all items, in the order request, row block, head, tile, are cut into equal
// contiguous shares, one a CTA: short and long requests, many rows and few,
// all load every SM alike.  An item cut by a share's end leaves partial results
// (max, sum, unnormalised output in fp32), which the combine kernel adds in
// the order of the shares, so results do not depend on timing.
#pragma once

#include "common.cuh"
#include "serving.h"

namespace dspark {

constexpr int kAttnMaxCtas = 320;  // CTAs of one attention launch, at most (attn_share counts on it)

// Rows of most requests for a K/V head, as far as the host can tell: twice the mean.
inline long long attn_likely_rows(const AttnArgs& a) {
  const long long all = (long long)a.a.n_tokens * a.G, twice = 2 * all / a.a.R;
  return twice < 1 ? 1 : twice < all ? twice : all;
}

// Units that an item counts beyond its tiles, for its start and end (Q, merging
// the streams, writing the result): three for long chunks, whose items are 256
// rows, else one.  Measured (us) at 0, 1, 2, 3 units:
//   decoding, 16 requests of 200 .. 2048 positions      32.6   32.3  33.9  34.8
//   verifying, 128 requests of 100 .. 600 positions     88.9   81.7  80.4  82.0
//   prefill, 2 requests of 2901 .. 4096 tokens           438    436   433   430
inline int attn_item_units(const AttnArgs& a) { return attn_likely_rows(a) > 256 ? 3 : 1; }

// A cut item, written by the first CTA whose share begins inside it.
struct CutItem {
  int pieces;       // slot 1 of the CTA before, slot 0 of this one and those after; 0: no such item
  int row0, rows;   // rows of the block within the chunk
  int h, q0;        // K/V head, the chunk's first token
  int pad[3];
};

// Workspace of a launch of `ctas` CTAs: status word, per-CTA status bits, cut
// items, partial (m, l) and O.  Nothing in it has to be cleared before a call.
struct AttnWorkspace {
  size_t flags, cuts, stats, out, total;
};
inline AttnWorkspace attn_workspace_layout(int MR, int D, int ctas) {
  AttnWorkspace w;
  w.flags = 256;
  w.cuts = align_up256(w.flags + ctas * sizeof(int));
  w.stats = align_up256(w.cuts + ctas * sizeof(CutItem));
  w.out = align_up256(w.stats + (size_t)ctas * 2 * MR * sizeof(float2));
  w.total = align_up256(w.out + (size_t)ctas * 2 * MR * D * sizeof(float));
  return w;
}

struct AttnParams {
  AttnArgs a;
  int* status;       // written by the combine
  int* flags;        // [grid] status bits of each CTA
  CutItem* cuts;     // [grid]
  float2* stats;     // [grid][2][MR] (m, l), m in log2 units
  float* part;       // [grid][2][MR][D]
  float scale_log2;  // scale * log2(e)
  int item_units;    // units of an item beyond its tiles
  int mr;            // rows of an item, at most (partial results are MR >= mr rows apart)
};

struct AttnRequest {
  int q0, n, L;  // first token, chunk length, cached positions
};

__device__ __forceinline__ AttnRequest attn_request(const ChunkArgs& a, int page_size, int r,
                                                    int* status) {
  AttnRequest q;
  int b = a.q_offsets[r], e = a.q_offsets[r + 1], L = a.kv_len[r];
  const int most = most_positions(a.max_pages, page_size);
  if (b < 0 || e < b || e > a.n_tokens || L < 0 || L > most || (r == 0 && b != 0)) {
    flag_status(status, DSPARK_DEV_BAD_INPUT);
    b = b < 0 ? 0 : b > a.n_tokens ? a.n_tokens : b;
    e = e < b ? b : e > a.n_tokens ? a.n_tokens : e;
    L = L < 0 ? 0 : L > most ? most : L;
  }
  q.q0 = b;
  q.n = e - b;
  q.L = L;
  return q;
}

// Keys that the rows of block m see: positions 0 .. end - 1.
__device__ __forceinline__ int attn_item_end(const AttnRequest& q, int G, int mr, int m) {
  int last = ((m + 1) * mr - 1) / G;
  last = last < q.n - 1 ? last : q.n - 1;
  const int end = q.L - q.n + last + 1;
  return end < 0 ? 0 : end;
}

template <int TN>
__device__ __forceinline__ int attn_tiles(int end) {
  return end <= TN ? 1 : (end + TN - 1) / TN;
}

// Row blocks of a request.
__device__ __forceinline__ int attn_blocks(const AttnRequest& q, int G, int mr) {
  return (int)(((long long)q.n * G + mr - 1) / mr);
}

// First unit of CTA c's share.  With fewer units than CTAs the first `units`
// CTAs get one each, so that no share between two others is empty.
__device__ __forceinline__ long long attn_share(long long units, int ctas, int c) {
  const long long n = units < ctas ? units : ctas;
  if (c >= n) return units;
  if (units < (1 << 23)) return (unsigned)(units * c) / (unsigned)n;  // (c < 320: below 2^32)
  return units * c / n;
}

// The walk of one CTA (or one warp role of it) over its share.
template <int TN>
struct AttnWalk {
  AttnRequest q;
  int r, m, h;       // current item: request, row block, K/V head
  int end, n_tiles;  // its keys and tiles
  int pos;           // the piece's first unit within the item
  int left;          // units of the share from there on
  int extra;         // item_units

  __device__ __forceinline__ bool done() const { return left <= 0; }
  // (the item's first item_units units stand for no tile)
  __device__ __forceinline__ int first_tile() const {
    return pos > extra ? pos - extra : 0;
  }
  __device__ __forceinline__ int last_tile() const {  // one past the piece's last tile
    const int e = pos + left - extra;
    return e < n_tiles ? e : n_tiles;
  }
  // A share that ends before the item's first tile has nothing of it.
  __device__ __forceinline__ void drop_empty() {
    if (left > 0 && last_tile() <= first_tile()) left = 0;
  }
  __device__ __forceinline__ int block_rows(const AttnParams& p) const {
    const long long rest = (long long)q.n * p.a.G - (long long)m * p.mr;
    return rest < p.mr ? (int)rest : p.mr;
  }

  // flags: the CTA's status bits.
  __device__ __forceinline__ void next(const AttnParams& p, int* flags) {
    left -= n_tiles + extra - pos;
    if (done()) return;
    pos = 0;
    if (++h >= p.a.c.heads) {
      h = 0;
      if ((long long)(++m) * p.mr >= (long long)q.n * p.a.G) {
        m = 0;
        do {
          if (++r >= p.a.a.R) {  // (not reached: the units count the items)
            left = 0;
            return;
          }
          q = attn_request(p.a.a, p.a.c.page_size, r, flags);
        } while (q.n == 0);
      }
      end = attn_item_end(q, p.a.G, p.mr, m);
      n_tiles = attn_tiles<TN>(end);
    }
    drop_empty();
  }
};

// What a CTA's threads work out together at the start: where its walk begins.
template <int TN>
struct AttnStart {
  AttnWalk<TN> walk;
  long long u0;  // the unit of the first item's first tile
  long long units, scan[33];
};

// All threads of the CTA (a multiple of 32, at most 1024).  *flags (shared
// memory) collects the CTA's status bits.  Ends with a barrier.
//
// A prefix sum of the requests' units, one request a thread (or a run of
// them); a request of many row blocks is summed by its thread's whole warp.
template <int TN>
__device__ __forceinline__ void attn_plan(const AttnParams& p, AttnStart<TN>* st, int* flags) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int R = p.a.a.R, G = p.a.G, Hkv = p.a.c.heads;
  const int per = (R + (int)blockDim.x - 1) / (int)blockDim.x;
  const int r0 = (int)threadIdx.x * per;
  // Units of the thread's i-th request, which all lanes of the warp call for
  // together.  (With one request a thread the second call finds it in q.)
  auto units_of = [&](int i, AttnRequest& q, bool again) -> long long {
    const int r = r0 + i;
    if (!again || per > 1) {
      q = AttnRequest{0, 0, 0};
      if (r < R) q = attn_request(p.a.a, p.a.c.page_size, r, flags);
    }
    const int blocks = attn_blocks(q, G, p.mr);
    long long u = blocks == 1 ? attn_tiles<TN>(q.L) + p.item_units : 0;
    for (unsigned todo = __ballot_sync(0xffffffffu, blocks > 1); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const AttnRequest w{0, __shfl_sync(0xffffffffu, q.n, src), __shfl_sync(0xffffffffu, q.L, src)};
      const int nb = __shfl_sync(0xffffffffu, blocks, src);
      long long sum = 0;
      for (int m = lane; m < nb; m += 32)
        sum += attn_tiles<TN>(attn_item_end(w, G, p.mr, m)) + p.item_units;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == src) u = sum;
    }
    return u * Hkv;
  };
  long long mine = 0;
  AttnRequest q;
  for (int i = 0; i < per; ++i) mine += units_of(i, q, false);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) st->scan[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const long long own = lane < warps ? st->scan[lane] : 0;
    long long v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane < warps) st->scan[lane] = v - own;
    if (lane == 31) st->units = v;
  }
  __syncthreads();
  const long long units = st->units;
  const long long start = attn_share(units, gridDim.x, blockIdx.x);
  const int left = (int)(attn_share(units, gridDim.x, blockIdx.x + 1) - start);
  if (left <= 0) {
    if (threadIdx.x == 0) st->walk.left = 0;
  } else {
    long long at = st->scan[warp] + incl - mine;  // the thread's first unit
    if (__any_sync(0xffffffffu, start >= at && start < at + mine)) {  // one warp
      for (int i = 0; i < per; ++i) {
        const long long k = units_of(i, q, true);
        const bool here = start >= at && start < at + k;  // one lane, for one i
        const unsigned who = __ballot_sync(0xffffffffu, here);
        if (who) {
          // The row block, 32 at a time: the warp's lanes each weigh one.
          const int src = __ffs(who) - 1;
          AttnWalk<TN> w;
          w.q.q0 = __shfl_sync(0xffffffffu, q.q0, src);
          w.q.n = __shfl_sync(0xffffffffu, q.n, src);
          w.q.L = __shfl_sync(0xffffffffu, q.L, src);
          w.r = __shfl_sync(0xffffffffu, r0, src) + i;
          long long base = __shfl_sync(0xffffffffu, at, src);
          const int blocks = attn_blocks(w.q, G, p.mr);
          for (int m0 = 0; m0 < blocks; m0 += 32) {
            w.m = m0 + lane;
            w.end = attn_item_end(w.q, G, p.mr, w.m);
            w.n_tiles = attn_tiles<TN>(w.end);
            const int item = w.n_tiles + p.item_units;
            const long long own = w.m < blocks ? (long long)item * Hkv : 0;
            long long upto = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const long long v = __shfl_up_sync(0xffffffffu, upto, o);
              if (lane >= o) upto += v;
            }
            const long long first = base + upto - own;
            if (start >= first && start < first + own) {
              const long long d = start - first;
              w.h = d >> 31 ? (int)(d / item) : (int)d / item;
              w.pos = (int)(d - (long long)w.h * item);
              w.left = left;
              w.extra = p.item_units;
              w.drop_empty();
              st->walk = w;
              st->u0 = first + (long long)w.h * item + p.item_units;
            }
            base += __shfl_sync(0xffffffffu, upto, 31);
          }
        }
        at += k;
      }
    }
  }
  __syncthreads();
}

// Written once a CTA: the item that its share begins inside of, if it is the
// first share to do so (the CTA before holds the item's first tile).
template <int TN>
__device__ __forceinline__ void attn_write_cut(const AttnParams& p, const AttnStart<TN>& st) {
  const AttnWalk<TN>& w = st.walk;
  CutItem c;
  c.pieces = 0;
  if (!w.done() && w.first_tile() > 0 &&
      st.u0 >= attn_share(st.units, gridDim.x, (int)blockIdx.x - 1)) {
    // The last piece is in the share that holds the item's last unit.
    const long long end = st.u0 + w.n_tiles, shares = st.units < gridDim.x ? st.units : gridDim.x;
    const int last = (int)((end * shares - 1) / st.units);
    c.pieces = last - (int)blockIdx.x + 2;
    c.row0 = w.m * p.mr, c.rows = w.block_rows(p);
    c.h = w.h, c.q0 = w.q.q0;
  }
  p.cuts[blockIdx.x] = c;
}

// Where the walk's current piece of its item goes: -1 whole (straight to the
// output), 0 the item began in an earlier share, 1 it goes on in a later one.
template <int TN>
__device__ __forceinline__ int attn_slot(const AttnWalk<TN>& w) {
  if (w.first_tile() > 0) return 0;
  return w.last_tile() < w.n_tiles ? 1 : -1;
}

cudaError_t launch_attn_combine(const AttnParams& p, int MR, int ctas, cudaStream_t s);

// The tensor-core path (attention_tc.cu).
bool attention_tc_supported(const AttnArgs& a);
size_t attention_tc_workspace_bytes(int head_dim);
cudaError_t launch_attention_tc(const AttnArgs& a, char* ws, cudaStream_t s);

}  // namespace dspark
