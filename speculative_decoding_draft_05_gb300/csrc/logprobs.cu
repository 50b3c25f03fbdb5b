// logprobs.cu -- log-probabilities of given tokens, entropy and the top
// alternatives of logit rows.
//
// With x_v = Z_v / T, m = max x, s = sum e^{x-m}, t = sum (x-m) e^{x-m}:
//   lse = m + ln s,  logp = x_token - lse,  H = lse - sum p x = ln s - t / s.
// (m, s, t) of two parts merge by rescaling to the larger m, so the row is read
// once, in chunks of 4096 ids that warps take independently of one another.
// The same pass leaves the largest logit of every group of 256 consecutive ids
// (594 groups at V = 151,936).  The k best ids lie in the k groups whose best
// id comes first: a group left out has k groups before it, each with an id that
// beats all of its own.  So the second kernel reads k groups again instead of
// sorting the row.
#include "common.cuh"
#include "serving.h"

namespace dspark {

namespace {

constexpr int kGroupIds = 256;      // ids a group: 32 lanes x 8
constexpr int kChunkGroups = 16;    // groups a warp's chunk
constexpr int kChunkIds = kGroupIds * kChunkGroups;
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kBlockGroups = 4;     // groups a warp reads at a time: 2 KB of bf16 in flight
constexpr int kBlockIds = kGroupIds * kBlockGroups;
constexpr int kRowCtas = 4;         // CTAs an SM
constexpr int kListRows = 12288;    // rows a CTA lists at a time
constexpr int kFinishWarps = 4;     // rows a CTA of the second kernel
constexpr int kShortRows = 4096;    // rows that a launch of one warp a row takes (one CTA checks all tokens)
constexpr int kMaxCand = 256;       // ids that the second kernel ranks at once
constexpr int kMaxPicked = 64;      // and groups that they may come from
constexpr uint32_t kSpent = 0xffd5a5a5u;  // a NaN that no maximum gives: a group all of whose ids are drawn
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Largest value over the warp; a NaN never wins.
__device__ __forceinline__ float warp_max_redux(float v) {
  float d;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
  return d;
}

// 8 consecutive logits, one lane's share of a group.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs((const float4*)p), b = __ldcs((const float4*)p + 1);
  }
  __device__ __forceinline__ void fill_low() {
    a = b = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
  }
  __device__ __forceinline__ f32x2 pair(int i) const {
    return i == 0 ? pack2(a.x, a.y) : i == 1 ? pack2(a.z, a.w) : i == 2 ? pack2(b.x, b.y) : pack2(b.z, b.w);
  }
  __device__ __forceinline__ float max() const {
    return fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = __ldcs((const uint4*)p); }
  __device__ __forceinline__ void fill_low() {
    q = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
  }
  __device__ __forceinline__ f32x2 pair(int i) const {
    const uint32_t w = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  __device__ __forceinline__ float max() const {  // (packed maxima: four instructions)
    __nv_bfloat162 v[4];
    memcpy(v, &q, 16);
    const __nv_bfloat162 m = __hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
};

// Exclusive prefix of v over the CTA's 256 threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* sm, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sm[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) {
    const int t = sm[w];
    all += t;
    if (w < warp) before += t;
  }
  *total = all;
  return before + incl - v;
}

// A warp's running sums over a chunk.
struct Sums {
  float m, s, t;  // largest logit; this lane's sums relative to it, t in units of log2
};

// A block of up to kBlockIds ids in registers: 8 of each group a lane.
template <typename T>
struct Block {
  Eight<T> x[kBlockGroups];
  __device__ __forceinline__ void load(const T* row, int v0, int V) {
    const T* p = row + v0 + (threadIdx.x & 31) * 8;
    if (v0 + kBlockIds <= V) {
#pragma unroll
      for (int k = 0; k < kBlockGroups; ++k) x[k].load(p + k * kGroupIds);
    } else {
#pragma unroll
      for (int k = 0; k < kBlockGroups; ++k) {
        const int v = v0 + k * kGroupIds + (threadIdx.x & 31) * 8;  // V % 8 == 0: all 8 ids or none
        if (v < V)
          x[k].load(p + k * kGroupIds);
        else
          x[k].fill_low();
      }
    }
  }
};

// Adds a block, whose first id is v0, to the sums and writes its groups'
// largest logits.  Per 8 logits a lane: the maximum (packed for bf16, one warp
// reduction), and packed pairs through y = x c - m c, p = 2^y, s += p, t += p y.
// A masked id makes p y = 0 * -inf = NaN: a block whose t is NaN is summed
// again with y held above -1e30.
template <typename T>
__device__ __forceinline__ void block_sums(const Block<T>& b, int v0, int V, float c, float* gmax,
                                           Sums& a) {
  const int lane = threadIdx.x & 31;
  // (a group of nothing but NaN may leave a NaN, which the readers take for -inf)
  float best = -INFINITY, mine = 0.0f;
#pragma unroll
  for (int k = 0; k < kBlockGroups; ++k) {
    const float g = warp_max_redux(b.x[k].max());
    best = fmaxf(best, g);
    if (lane == k) mine = g;
  }
  if (lane < kBlockGroups && v0 + lane * kGroupIds < V) gmax[v0 / kGroupIds + lane] = mine;
  if (best > a.m) {  // the same for all lanes
    const float d = (a.m - best) * c, f = ex2(d);  // m = -inf: the sums are 0
    a.t = a.m == -INFINITY ? 0.0f : f * (a.t + d * a.s);
    a.s *= f;
    a.m = best;
  }
  const float mm = a.m == -INFINITY ? 0.0f : a.m;
  const f32x2 c2 = pack2(c, c), mc2 = pack2(-mm * c, -mm * c);
  f32x2 s2[2] = {0ull, 0ull}, t2[2] = {0ull, 0ull};
#pragma unroll
  for (int k = 0; k < kBlockGroups; ++k) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f32x2 y = fma2(b.x[k].pair(e), c2, mc2);
      float y0, y1;
      unpack2(y, y0, y1);
      const f32x2 p = pack2(ex2(y0), ex2(y1));
      s2[e & 1] = add2(s2[e & 1], p);
      t2[e & 1] = fma2(p, y, t2[e & 1]);
    }
  }
  float sa, sb, ta, tb;
  unpack2(add2(s2[0], s2[1]), sa, sb);
  unpack2(add2(t2[0], t2[1]), ta, tb);
  sa += sb;
  ta += tb;
  if (__any_sync(0xffffffffu, isnan(ta)) || fabsf(mm) >= 1e30f) {  // (|m| c could overflow)
    sa = ta = 0.0f;
#pragma unroll
    for (int k = 0; k < kBlockGroups; ++k) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x0, x1;
        unpack2(b.x[k].pair(e), x0, x1);
        const float y0 = (x0 - mm) * c, y1 = (x1 - mm) * c;
        const float p0 = ex2(y0), p1 = ex2(y1);
        sa += p0 + p1;
        ta = fmaf(p0, fmaxf(y0, -1e30f), ta);
        ta = fmaf(p1, fmaxf(y1, -1e30f), ta);
      }
    }
  }
  a.s += sa;
  a.t += ta;
}

struct RowOutputs {
  float *logp, *entropy, *lse;  // [n_rows]
  int32_t* top_ids;             // [n_rows, top]
  float* top_logp;
  int top;
};

__device__ __forceinline__ void skip_row(const RowOutputs& o, int r) {
  const int lane = threadIdx.x & 31;
  const float nan = __int_as_float(0x7fc00000);
  if (lane == 0) o.logp[r] = o.entropy[r] = o.lse[r] = nan;
  if (lane < o.top) {
    o.top_ids[(size_t)r * o.top + lane] = -1;
    o.top_logp[(size_t)r * o.top + lane] = nan;
  }
}

// The wanted rows' chunks, dealt out to all warps in turn, so that the whole
// GPU reads one moving window of memory (contiguous shares a CTA, hundreds of
// places of a 2.6 GB array at once, took 214 us where this takes 156, with the
// same ring of copies).  Every CTA lists the wanted rows itself, by a prefix sum
// over the tokens (a few us beside a launch and a list in memory).
template <typename T>
__global__ void __launch_bounds__(kRowThreads, kRowCtas)
logprobs_stream_kernel(const T* __restrict__ Z, long long row_stride,
                       const int32_t* __restrict__ tokens, int n_rows, int V, int chunks,
                       int groups, float c, float4* parts, float* gmax, int* rows_wanted,
                       const RowOutputs o, int* status) {
  __shared__ int sm[kRowWarps];
  __shared__ uint16_t list[kListRows];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool bad = false;
  // Rows without a token get their results here.
  for (int r = blockIdx.x * kRowWarps + warp; r < n_rows; r += gridDim.x * kRowWarps)
    if (__ldg(tokens + r) < 0) skip_row(o, r);
  int listed = 0;
  // A window of rows at a time (one, up to kListRows rows).
  for (int w0 = 0; w0 < n_rows; w0 += kListRows) {
    const int rows = min(kListRows, n_rows - w0);
    const int seg = (rows + kRowThreads - 1) / kRowThreads;
    const int r0 = min(rows, (int)threadIdx.x * seg), r1 = min(rows, r0 + seg);
    int mine = 0;
#pragma unroll 8
    for (int r = r0; r < r1; ++r) {
      const int tok = __ldg(tokens + w0 + r);
      mine += tok >= 0 ? 1 : 0;
      bad |= tok >= V;
    }
    int n;
    int k = block_scan(mine, sm, &n);
#pragma unroll 8
    for (int r = r0; r < r1; ++r)
      if (__ldg(tokens + w0 + r) >= 0) list[k++] = (uint16_t)r;
    __syncthreads();
    if (blockIdx.x == 0)  // the second kernel's list: [0] how many, then the rows
      for (int i = threadIdx.x; i < n; i += kRowThreads) rows_wanted[1 + listed + i] = w0 + list[i];
    listed += n;
    const long long units = (long long)n * chunks;
    const int all_warps = gridDim.x * kRowWarps, me = blockIdx.x * kRowWarps + warp;
    const int dk = all_warps / chunks, dch = all_warps - dk * chunks;
    int i = me / chunks, ch = me - i * chunks;
    for (long long u = me; u < units; u += all_warps) {
      const int row = w0 + list[i];
      const T* z = Z + (long long)row * row_stride;
      Sums acc{-INFINITY, 0.0f, 0.0f};
      const int v0 = ch * kChunkIds, v1 = min(V, v0 + kChunkIds);
      for (int v = v0; v < v1; v += kBlockIds) {
        Block<T> b;
        b.load(z, v, V);
        block_sums(b, v, V, c, gmax + (size_t)row * groups, acc);
      }
      const float s = warp_sum(acc.s), t = warp_sum(acc.t);
      if (lane == 0) parts[(size_t)row * chunks + ch] = make_float4(acc.m, s, t, 0.0f);
      i += dk;
      ch += dch;
      if (ch >= chunks) ch -= chunks, ++i;
    }
    __syncthreads();
  }
  const int any_bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *status = any_bad ? DSPARK_DEV_BAD_INPUT : 0;
    rows_wanted[0] = listed;
  }
}

// Order of the alternatives as unsigned keys: larger logit, larger key; NaN
// counts as -inf, -0 as 0; 0 stands for "none".
__device__ __forceinline__ uint32_t rank_key(float x) {
  return key_ord(isnan(x) ? -INFINITY : x + 0.0f);
}

// The 32 lanes' values, sorted downwards.
__device__ __forceinline__ uint32_t warp_sort_desc(uint32_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const uint32_t u = __shfl_xor_sync(0xffffffffu, v, j);
      const bool down = (lane & k) == 0;       // this block of k sorts downwards
      const bool low = (lane & j) == 0;        // this lane is the pair's first
      v = down == low ? max(u, v) : min(u, v);
    }
  }
  return v;
}

// What one warp needs of shared memory to find a row's alternatives.
struct RowScratch {
  unsigned long long cand[kMaxCand];  // key, then ~id: the larger comes first
  int picked[kMaxPicked], n_cand;
};

// Row r's results from its sums, by one warp; gm: its groups' largest logits (changed).
template <typename T>
__device__ __forceinline__ void finish_row(const T* row, int r, float x_tok, int V, int groups,
                                           float invT, float m, float s, float t, float* gm,
                                           const RowOutputs& o, RowScratch& sm) {
  const int lane = threadIdx.x & 31, top = o.top;
  int32_t* top_ids = o.top_ids;
  float* top_logp = o.top_logp;
  const float ln_s = logf(s);
  if (lane == 0) {
    o.logp[r] = (x_tok - m) * invT - ln_s;
    o.entropy[r] = ln_s - t / s * kLn2;
    o.lse[r] = m * invT + ln_s;
  }
  if (top == 0) return;

  // Alternatives.  A threshold that at least `top` ids reach: the top-th largest
  // of the lanes' two largest values each, over the groups' maxima, or over the
  // ids' eights where there are few groups.  The ids at or above it (a few
  // times `top` of them) are collected and ranked by counting.
  unsigned long long* cand = sm.cand;
  int* picked = sm.picked;
  int& n_cand_s = sm.n_cand;
  uint32_t best = 0, second = 0;
  auto rank_in = [&](uint32_t k) {
    second = max(second, min(best, k));
    best = max(best, k);
  };
  if (groups >= 64) {
#pragma unroll 8
    for (int g = lane; g < groups; g += 32) rank_in(rank_key(gm[g]));
  } else {
#pragma unroll 4
    for (int v = lane * 8; v < V; v += kGroupIds) {
      Eight<T> x;
      x.load(row + v);
      rank_in(rank_key(x.max()));
    }
  }
  // (the 32 largest of two sorted 32s: the larger of each pair, one list reversed)
  best = warp_sort_desc(best);
  second = warp_sort_desc(second);
  best = warp_sort_desc(max(best, __shfl_xor_sync(0xffffffffu, second, 31)));
  const uint32_t floor_key = __shfl_sync(0xffffffffu, best, top - 1);
  if (lane == 0) n_cand_s = 0;
  int n_cand = kMaxCand + 1;
  if (floor_key > key_ord(-INFINITY)) {
    const float floor_x = ord_key(floor_key);
    int n_picked = 0;
#pragma unroll 4
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const bool y = g0 + lane < groups && gm[g0 + lane] >= floor_x;
      const unsigned b = __ballot_sync(0xffffffffu, y);
      const int at = n_picked + __popc(b & ((1u << lane) - 1u));
      if (y && at < kMaxPicked) picked[at] = g0 + lane;
      n_picked += __popc(b);
    }
    __syncwarp();
    if (n_picked <= kMaxPicked) {
      constexpr int kBatch = sizeof(T) == 2 ? 8 : 4;  // groups in flight
      for (int i0 = 0; i0 < n_picked; i0 += kBatch) {
        Eight<T> x[kBatch];
        int v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          v[k] = i0 + k < n_picked ? picked[i0 + k] * kGroupIds + lane * 8 : V;
          if (v[k] < V)
            x[k].load(row + v[k]);
          else
            x[k].fill_low();
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (x[k].max() >= floor_x) {  // few lanes
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float f[2];
              unpack2(x[k].pair(e), f[0], f[1]);
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (f[h] >= floor_x) {
                  const int at = atomicAdd(&n_cand_s, 1);
                  if (at < kMaxCand)
                    cand[at] = (unsigned long long)rank_key(f[h]) << 32 | ~(uint32_t)(v[k] + 2 * e + h);
                }
            }
          }
      }
      __syncwarp();
      n_cand = n_cand_s;
    }
  }
  if (n_cand <= kMaxCand) {
    for (int i = lane; i < n_cand; i += 32) {
      const unsigned long long own = cand[i];
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < n_cand; ++j) rank += cand[j] > own ? 1 : 0;
      if (rank < top) {
        top_ids[(size_t)r * top + rank] = (int)~(uint32_t)own;
        top_logp[(size_t)r * top + rank] = (ord_key((uint32_t)(own >> 32)) - m) * invT - ln_s;
      }
    }
    return;
  }
  // Many ids tie at the threshold, or fewer than `top` are finite (or V < 256):
  // one at a time, from the group whose head comes first.  Drawn are the ids
  // up to the last drawn one in the order, so an id is open if it comes after.
  uint32_t last_key = 0xffffffffu;
  int last_id = -1;
  for (int k = 0; k < top; ++k) {
    uint32_t hk = 0;
    int hg = 0x7fffffff;
#pragma unroll 4
    for (int g = lane; g < groups; g += 32) {
      const uint32_t q = __float_as_uint(gm[g]) == kSpent ? 0u : rank_key(gm[g]);
      if (q > hk) hk = q, hg = g;
    }
    const uint32_t key = __reduce_max_sync(0xffffffffu, hk);
    const int g = __reduce_min_sync(0xffffffffu, hk == key ? hg : 0x7fffffff);
    if (key == 0 || g >= groups) break;  // (not reached: top <= V)
    const int v = g * kGroupIds + lane * 8;
    uint32_t q[8];
    int at = 0x7fffffff;
#pragma unroll
    for (int e = 7; e >= 0; --e) {
      q[e] = v < V ? rank_key(to_f32(row[v + e])) : 0u;
      if (q[e] > last_key || (q[e] == last_key && v + e <= last_id)) q[e] = 0;
      if (q[e] == key) at = v + e;
    }
    const int id = __reduce_min_sync(0xffffffffu, at);
    uint32_t next = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (v + e != id) next = max(next, q[e]);
    next = __reduce_max_sync(0xffffffffu, next);
    if (lane == 0) {
      gm[g] = next ? ord_key(next) : __uint_as_float(kSpent);
      top_ids[(size_t)r * top + k] = id;
      top_logp[(size_t)r * top + k] = (ord_key(key) - m) * invT - ln_s;
    }
    last_key = key, last_id = id;
    __syncwarp();
  }
}

// Merges the chunks of a wanted row and finishes it: one warp a row, the first
// CTAs (the list keeps the SMs evenly loaded: with the rows in place, most of a
// CTA's warps would have none).
template <typename T>
__global__ void __launch_bounds__(kFinishWarps * 32)
logprobs_finish_kernel(const T* __restrict__ Z, long long row_stride,
                       const int32_t* __restrict__ tokens, int V, int chunks, int groups, float c,
                       float invT, const float4* parts, float* gmax, const int* rows_wanted,
                       const RowOutputs o) {
  __shared__ RowScratch scratch[kFinishWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = blockIdx.x * kFinishWarps + warp;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int r = __ldcg(rows_wanted + 1 + i);  // (read with the count: a row of the list or, past it, unused)
  if (i >= __ldcg(rows_wanted)) return;
  const int tok = __ldg(tokens + r);
  const T* row = Z + (long long)r * row_stride;
  const float x_tok = tok < V ? to_f32(row[tok]) : __int_as_float(0x7fc00000);

  float m = -INFINITY, s = 0.0f, t = 0.0f;
  for (int k = lane; k < chunks; k += 32) {
    const float4 p = parts[(size_t)r * chunks + k];
    if (p.x > m) {
      const float d = (m - p.x) * c, f = ex2(d);
      t = m == -INFINITY ? 0.0f : f * (t + d * s);
      s *= f;
      m = p.x;
    }
    if (p.x != -INFINITY) {
      const float d = (p.x - m) * c, f = ex2(d);
      s += f * p.y;
      t += f > 0.0f ? f * (p.z + d * p.y) : 0.0f;
    } else {
      s += p.y;  // 0, or NaN where the chunk held one
      t += p.z;
    }
  }
  const float all = warp_max(m);
  if (m != -INFINITY) {
    const float d = (m - all) * c, f = ex2(d);
    t = f > 0.0f ? f * (t + d * s) : 0.0f;
    s *= f;
  }
  finish_row(row, r, x_tok, V, groups, invT, all, warp_sum(s), warp_sum(t),
             gmax + (size_t)r * groups, o, scratch[warp]);
}

// Rows of one chunk: sums and results by the same warp, in one launch.
template <typename T>
__global__ void __launch_bounds__(kFinishWarps * 32)
logprobs_short_kernel(const T* __restrict__ Z, long long row_stride,
                      const int32_t* __restrict__ tokens, int n_rows, int V, int groups, float c,
                      float invT, float* gmax, const RowOutputs o, int* status) {
  __shared__ RowScratch scratch[kFinishWarps];
  const int warp = threadIdx.x >> 5, r = blockIdx.x * kFinishWarps + warp;
  if (blockIdx.x == 0) {  // the status word, from all tokens
    bool bad = false;
    for (int i = threadIdx.x; i < n_rows; i += kFinishWarps * 32) bad |= __ldg(tokens + i) >= V;
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) *status = any ? DSPARK_DEV_BAD_INPUT : 0;
  }
  if (r >= n_rows) return;
  const int tok = __ldg(tokens + r);
  if (tok < 0) {
    skip_row(o, r);
    return;
  }
  const T* row = Z + (long long)r * row_stride;
  const float x_tok = tok < V ? to_f32(row[tok]) : __int_as_float(0x7fc00000);
  float* gm = gmax + (size_t)r * groups;
  Sums acc{-INFINITY, 0.0f, 0.0f};
  for (int v = 0; v < V; v += kBlockIds) {
    Block<T> b;
    b.load(row, v, V);
    block_sums(b, v, V, c, gm, acc);
  }
  __syncwarp();
  finish_row(row, r, x_tok, V, groups, invT, acc.m, warp_sum(acc.s), warp_sum(acc.t), gm, o,
             scratch[warp]);
}

int groups_of(int V) { return (V + kGroupIds - 1) / kGroupIds; }
int chunks_of(int V) { return (V + kChunkIds - 1) / kChunkIds; }

template <typename T>
cudaError_t launch(const void* Z, long long row_stride, const int32_t* tokens, int n_rows, int V,
                   float invT, const RowOutputs& o, char* ws, const LogprobsWorkspace& w,
                   cudaStream_t s) {
  float4* parts = (float4*)(ws + w.parts);
  float* gmax = (float*)(ws + w.gmax);
  int* rows_wanted = (int*)(ws + w.rows);
  const int chunks = chunks_of(V), groups = groups_of(V);
  const float c = invT * kLog2e;
  const int row_ctas = (n_rows + kFinishWarps - 1) / kFinishWarps;
  if (chunks == 1 && n_rows <= kShortRows) {
    logprobs_short_kernel<T><<<row_ctas, kFinishWarps * 32, 0, s>>>(
        (const T*)Z, row_stride, tokens, n_rows, V, groups, c, invT, gmax, o, (int*)ws);
    return cudaGetLastError();
  }
  long long ctas = ((long long)n_rows * chunks + kRowWarps - 1) / kRowWarps;
  if (ctas > 152 * kRowCtas) ctas = 152 * kRowCtas;
  logprobs_stream_kernel<T><<<(int)ctas, kRowThreads, 0, s>>>(
      (const T*)Z, row_stride, tokens, n_rows, V, chunks, groups, c, parts, gmax, rows_wanted, o,
      (int*)ws);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(row_ctas);
  cfg.blockDim = dim3(kFinishWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_finish_kernel<T>, (const T*)Z, row_stride, tokens, V,
                            chunks, groups, c, invT, (const float4*)parts, gmax,
                            (const int*)rows_wanted, o);
}

}  // namespace

LogprobsWorkspace logprobs_workspace_layout(int n_rows, int V) {
  LogprobsWorkspace w;
  w.rows = 256;
  // (read up to a whole CTA of the second kernel past the last row)
  w.parts = align_up256(w.rows + ((size_t)n_rows + 1 + kFinishWarps) * sizeof(int));
  w.gmax = align_up256(w.parts + (size_t)n_rows * chunks_of(V) * sizeof(float4));
  w.total = align_up256(w.gmax + (size_t)n_rows * groups_of(V) * sizeof(float));
  return w;
}

cudaError_t launch_logprobs(const void* Z, int dtype, long long row_stride, const int32_t* tokens,
                            int n_rows, int V, float invT, int top, float* logp, float* entropy,
                            float* lse, int32_t* top_ids, float* top_logp, char* ws,
                            const LogprobsWorkspace& w, cudaStream_t s) {
  const RowOutputs o{logp, entropy, lse, top_ids, top_logp, top};
  return dtype == DSPARK_BF16
             ? launch<__nv_bfloat16>(Z, row_stride, tokens, n_rows, V, invT, o, ws, w, s)
             : launch<float>(Z, row_stride, tokens, n_rows, V, invT, o, ws, w, s);
}

}  // namespace dspark
