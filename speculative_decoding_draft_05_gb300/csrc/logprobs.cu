// logprobs.cu -- log-probabilities of given tokens, entropy and the top
// alternatives of logit rows.
//
// With x_v = Z_v / T, m = max x, s = sum e^{x-m}, t = sum (x-m) e^{x-m}:
//   lse = m + ln s,  logp = x_token - lse,  H = lse - sum p x = ln s - t / s.
// (m, s, t) of two parts merge by rescaling to the larger m, so the row is read
// once, in blocks of 4 KB that warps take independently of one another.
// The same pass leaves the largest logit of every group of 256 consecutive ids
// (594 groups at V = 151,936).  The k best ids lie in the k groups whose best
// id comes first: a group left out has k groups before it, each with an id that
// beats all of its own.  So the second kernel reads k groups again, or fewer,
// instead of sorting the row.
//
// Bound by the read of the logits.  512 requests of 17 rows, 2567 of them
// wanted, V = 151,936: 780 MB of bf16 in 121 us without alternatives (6.45 TB/s),
// 129 us with 20 a row; fp32 (1.56 GB) 239 us.
#include "common.cuh"
#include "serving.h"

namespace dspark {

namespace {

constexpr int kGroupIds = 256;      // ids a group: 32 lanes x 8
constexpr int kBlockBytes = 4096;   // what a warp reads at a time: 8 groups of bf16, 4 of fp32
constexpr int kRowThreads = 512;    // one CTA an SM: 126 registers a thread, all that there are
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kListRows = 16384;    // rows a CTA lists at a time
constexpr int kFinishWarps = 4;     // rows a CTA of the second kernel
constexpr int kFinishCtas = 5;      // its CTAs an SM
constexpr int kShortIds = 4096;     // rows that one warp sums and finishes in one launch: up to this long,
constexpr int kShortRows = 4096;    // and up to so many (one CTA checks all tokens)
constexpr int kTile = 20;           // group maxima in flight a lane: 640 groups
constexpr int kTileGroups = kTile * 32;
constexpr int kMaxCand = 256;       // ids that the second kernel ranks at once
constexpr int kMaxEights = 128;     // the eights of ids that they may come from,
constexpr int kMaxPicked = 64;      // and groups
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

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
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

// Exclusive prefix of v over the CTA's threads; *total gets the sum.
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

template <typename T>
__host__ __device__ constexpr int block_ids() {
  return kBlockBytes / (int)sizeof(T);
}

// A block in registers: 8 consecutive ids of each group a lane.
template <typename T>
struct Block {
  static constexpr int kGroups = block_ids<T>() / kGroupIds;
  Eight<T> x[kGroups];
  __device__ __forceinline__ void load(const T* row, int v0, int V) {
    const int lane = threadIdx.x & 31;
    const T* p = row + v0 + lane * 8;
    if (v0 + block_ids<T>() <= V) {
#pragma unroll
      for (int k = 0; k < kGroups; ++k) x[k].load(p + k * kGroupIds);
    } else {
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        if (v0 + k * kGroupIds + lane * 8 < V)  // V % 8 == 0: all 8 ids or none
          x[k].load(p + k * kGroupIds);
        else
          x[k].fill_low();
      }
    }
  }
};

// Part of a row: largest logit, sum of p and sum of p y relative to it (y in units of log2).
struct Part {
  float m, s, t;
};

__device__ __forceinline__ void merge(Part& a, float m, float s, float t, float c) {
  if (m > a.m) {
    const float d = (a.m - m) * c, f = ex2(d);
    a.t = a.m == -INFINITY ? 0.0f : f > 0.0f ? f * (a.t + d * a.s) : 0.0f;
    a.s *= f;
    a.m = m;
  }
  if (m != -INFINITY) {
    const float d = (m - a.m) * c, f = ex2(d);
    a.s += f * s;
    a.t += f > 0.0f ? f * (t + d * s) : 0.0f;
  } else {
    a.s += s;  // 0, or NaN where the part held one
    a.t += t;
  }
}

// A block's part, by the whole warp, the same in all lanes; its groups' largest
// logits go to gm[g0 ...].  Per 8 logits a lane: the maximum (packed for bf16,
// one warp reduction), and packed pairs through y = (x - m) c, p = 2^y, s += p,
// t += p max(y, -1e30): a masked id's y is -inf, and p y would be 0 * -inf.  (Summing
// the blocks that have one a second time instead, from what the first pass left
// NaN, made such rows half as long again: 90 us for 60 at 1000 rows.)  x - m first, then times c: x c
// alone overflows where masks hold the type's lowest value.
template <typename T>
__device__ __forceinline__ Part block_part(const Block<T>& b, int g0, int groups, float c, float* gm) {
  constexpr int kGroups = Block<T>::kGroups;
  const int lane = threadIdx.x & 31;
  // (a group of nothing but NaN may leave a NaN, which the readers take for -inf)
  float best = -INFINITY, mine = 0.0f;
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const float g = warp_max_redux(b.x[k].max());
    best = fmaxf(best, g);
    if (lane == k) mine = g;
  }
  if (lane < kGroups && g0 + lane < groups) gm[g0 + lane] = mine;
  const float mm = best == -INFINITY ? 0.0f : best;
  const f32x2 c2 = pack2(c, c), m2 = pack2(-mm, -mm);
  f32x2 s2[2] = {0ull, 0ull}, t2[2] = {0ull, 0ull};
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f32x2 y = mul2(add2(b.x[k].pair(e), m2), c2);
      float y0, y1;
      unpack2(y, y0, y1);
      const f32x2 p = pack2(ex2(y0), ex2(y1));
      s2[e & 1] = add2(s2[e & 1], p);
      t2[e & 1] = fma2(p, pack2(fmaxf(y0, -1e30f), fmaxf(y1, -1e30f)), t2[e & 1]);
    }
  }
  float s, t, sb, tb;
  unpack2(add2(s2[0], s2[1]), s, sb);
  unpack2(add2(t2[0], t2[1]), t, tb);
  s += sb;
  t += tb;
  // Both sums over the warp: the lower half takes s, the upper t.
  const bool up = lane & 16;
  float mix = up ? t : s;
  mix += __shfl_xor_sync(0xffffffffu, up ? s : t, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) mix += __shfl_xor_sync(0xffffffffu, mix, o);
  return Part{best, __shfl_sync(0xffffffffu, mix, 0), __shfl_sync(0xffffffffu, mix, 16)};
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

// The wanted rows' blocks, dealt out to all warps in turn, so that the whole
// GPU reads one moving window of memory and no warp has more than one block
// more than another (contiguous shares a CTA, hundreds of places of a 2.6 GB
// array at once, took a third longer).  16 warps an SM with 4 KB blocks and the
// next one loaded ahead beat 32 warps with 2 KB and no load ahead, 144 to 159
// us, and 2 KB with, 151 us: what a block costs besides its ids' own arithmetic
// (the reductions over the warp) counts as much as the bytes in flight.  Every
// CTA lists the wanted rows itself, by a prefix sum over the tokens (a few us
// beside a launch and a list in memory).
template <typename T>
__global__ void __launch_bounds__(kRowThreads, 1)
logprobs_stream_kernel(const T* Z, long long row_stride,
                       const int32_t* tokens, int n_rows, int V, int blocks,
                       int groups, float c, float4* parts, float* gmax, int* rows_wanted,
                       const RowOutputs o, int* status) {
  __shared__ int sm[kRowWarps];
  __shared__ uint16_t list[kListRows];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool bad = false;
  // Rows without a token get their results here.
  for (int r = blockIdx.x * kRowWarps + warp; r < n_rows; r += gridDim.x * kRowWarps)
    if (tokens[r] < 0) skip_row(o, r);
  int listed = 0;
  // A window of rows at a time (one, up to kListRows rows).
  for (int w0 = 0; w0 < n_rows; w0 += kListRows) {
    const int rows = min(kListRows, n_rows - w0);
    const int seg = (rows + kRowThreads - 1) / kRowThreads;
    const int r0 = min(rows, (int)threadIdx.x * seg), r1 = min(rows, r0 + seg);
    int mine = 0;
#pragma unroll 8
    for (int r = r0; r < r1; ++r) {
      const int tok = tokens[w0 + r];
      mine += tok >= 0 ? 1 : 0;
      bad |= tok >= V;
    }
    int n;
    int k = block_scan(mine, sm, &n);
#pragma unroll 8
    for (int r = r0; r < r1; ++r)
      if (tokens[w0 + r] >= 0) list[k++] = (uint16_t)r;
    __syncthreads();
    if (blockIdx.x == 0)  // the second kernel's list: [0] how many, then the rows
      for (int i = threadIdx.x; i < n; i += kRowThreads) rows_wanted[1 + listed + i] = w0 + list[i];
    listed += n;
    // (The rows do not overlap, so the blocks of any array that fits the memory
    // count far below 2^32.)  The next block is loaded before the current one is
    // summed: 128 KB in flight an SM.
    const unsigned units = (unsigned)n * (unsigned)blocks;
    const int step = gridDim.x * kRowWarps, di = step / blocks, dj = step - di * blocks;
    unsigned u = warp * gridDim.x + blockIdx.x;
    int i = (int)(u / (unsigned)blocks), j = (int)(u - (unsigned)i * blocks);
    Block<T> b;
    if (u < units) b.load(Z + (long long)(w0 + list[i]) * row_stride, j * block_ids<T>(), V);
#pragma unroll 1
    for (; u < units; u += step) {
      const int row = w0 + list[i], at = j;
      i += di;
      j += dj;
      if (j >= blocks) j -= blocks, ++i;
      Block<T> next;
      if (u + step < units)
        next.load(Z + (long long)(w0 + list[i]) * row_stride, j * block_ids<T>(), V);
      const Part p = block_part(b, at * Block<T>::kGroups, groups, c,
                                gmax + (size_t)row * groups);
      if (lane == 0) parts[(size_t)row * blocks + at] = make_float4(p.m, p.s, p.t, 0.0f);
      b = next;
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
__device__ __forceinline__ float warp_sort_desc(float v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, v, j);
      const bool down = (lane & k) == 0;       // this block of k sorts downwards
      const bool low = (lane & j) == 0;        // this lane is the pair's first
      v = down == low ? fmaxf(u, v) : fminf(u, v);
    }
  }
  return v;
}

// The 32 lanes' values, a sequence that falls and then rises or the other way
// round, sorted downwards.
__device__ __forceinline__ float warp_merge_desc(float v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, j);
    v = (lane & j) == 0 ? fmaxf(u, v) : fminf(u, v);
  }
  return v;
}

// Up to kTileGroups of a row's group maxima, all loads in flight at once; -inf
// past the last group.  Neighbours lie in different lanes: vocabularies are
// often in the order of frequency, and then so are the best groups.
struct GroupTile {
  float q[kTile];
  __device__ __forceinline__ void load(const float* gm, int g0, int groups) {
#pragma unroll
    for (int k = 0; k < kTile; ++k) {
      const int g = g0 + k * 32 + ((int)threadIdx.x & 31);
      q[k] = g < groups ? gm[g] : -INFINITY;
    }
  }
};

// Each lane's two largest values so far (a NaN counts as -inf), and the 32
// largest of all of them.
struct TopTwo {
  float best = -INFINITY, second = -INFINITY;
  __device__ __forceinline__ void add(float x) {
    x = fmaxf(x, -INFINITY);
    second = fmaxf(second, fminf(best, x));
    best = fmaxf(best, x);
  }
  // (of two sorted 32s: the larger of each pair, one list reversed)
  __device__ __forceinline__ float sorted() const {
    const float a = warp_sort_desc(best), b = warp_sort_desc(second);
    return warp_merge_desc(fmaxf(a, __shfl_xor_sync(0xffffffffu, b, 31)));
  }
};

// What one warp needs of shared memory to find a row's alternatives.
struct RowScratch {
  unsigned long long cand[kMaxCand];  // key, then ~id: the larger comes first
  int eights[kMaxEights], picked[kMaxPicked];
};

// Row r's results from its sums, by one warp; gm: its groups' largest logits
// (changed), of which `tile` holds the first kTileGroups.
template <typename T>
__device__ __forceinline__ void finish_row(const T* row, int r, float x_tok, int V, int groups,
                                           float invT, const Part& sum, float* gm, GroupTile& tile,
                                           const RowOutputs& o, RowScratch& sm) {
  const int lane = threadIdx.x & 31, top = o.top;
  int32_t* top_ids = o.top_ids;
  float* top_logp = o.top_logp;
  const float m = sum.m, ln_s = logf(sum.s);
  if (lane == 0) {
    o.logp[r] = (x_tok - m) * invT - ln_s;
    o.entropy[r] = ln_s - sum.t / sum.s * kLn2;
    o.lse[r] = m * invT + ln_s;
  }
  if (top == 0) return;

  // Alternatives.  A first threshold that at least `top` ids reach: the top-th
  // largest of the lanes' two largest values each, over the groups' maxima.  The
  // groups with the largest maxima are read, as many as fit the registers; the
  // maxima of their eights raise the threshold in the same way.  Then the other
  // groups that reach it, often few: in a vocabulary in the order of frequency
  // the first groups hold most of the best ids.  The eights that reach it are
  // listed and looked through by all lanes, and the ids that do (top of them
  // and few more) are ranked by counting.  Rows of less than 64 groups start at
  // the eights.
  constexpr int kBatch = sizeof(T) == 2 ? 12 : 6;  // groups in flight
  unsigned long long* cand = sm.cand;
  const unsigned below = (1u << lane) - 1u;
  float floor_x;
  int n_eights = 0;
  auto list_eight = [&](bool y, int v) {
    const unsigned b = __ballot_sync(0xffffffffu, y);
    const int at = n_eights + __popc(b & below);
    if (y && at < kMaxEights) sm.eights[at] = v;
    n_eights += __popc(b);
  };
  if (groups >= 64) {
    TopTwo lanes;
    for (int g0 = 0;;) {
#pragma unroll
      for (int k = 0; k < kTile; ++k) lanes.add(tile.q[k]);
      g0 += kTileGroups;
      if (g0 >= groups) break;
      tile.load(gm, g0, groups);
    }
    const float heads = lanes.sorted();
    const float first = __shfl_sync(0xffffffffu, heads, min(top, kBatch) - 1);
    floor_x = __shfl_sync(0xffffffffu, heads, top - 1);
    int n_picked = 0;
    // Groups whose maximum is at least lo and not at least hi, behind those picked.
    auto pick = [&](float lo, float hi) {
      for (int g0 = 0; g0 < groups; g0 += kTileGroups) {
        if (groups > kTileGroups) tile.load(gm, g0, groups);
#pragma unroll
        for (int k = 0; k < kTile; ++k) {
          const bool y = tile.q[k] >= lo && !(tile.q[k] >= hi);
          const unsigned b = __ballot_sync(0xffffffffu, y);
          if (b) {
            const int at = n_picked + __popc(b & below);
            if (y && at < kMaxPicked) sm.picked[at] = g0 + k * 32 + lane;
            n_picked += __popc(b);
          }
        }
      }
      __syncwarp();
    };
    if (floor_x > -INFINITY) pick(first, __int_as_float(0x7fc00000));  // (nothing is at least NaN)
    int i0 = 0;
    while (i0 < n_picked && n_picked <= kMaxPicked) {
      const int end = min(n_picked, i0 + kBatch);
      Eight<T> x[kBatch];
      int v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        v[k] = i0 + k < end ? sm.picked[i0 + k] * kGroupIds + lane * 8 : V;
        if (v[k] < V)
          x[k].load(row + v[k]);
        else
          x[k].fill_low();
      }
      if (i0 == 0 && top > 1) {
        TopTwo lanes2;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) lanes2.add(x[k].max());
        floor_x = fmaxf(floor_x, __shfl_sync(0xffffffffu, lanes2.sorted(), top - 1));
        pick(floor_x, first);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) list_eight(x[k].max() >= floor_x, v[k]);
      i0 = end;
    }
    if (n_picked > kMaxPicked) n_eights = kMaxEights + 1;
  } else {
    TopTwo lanes;
#pragma unroll 4
    for (int v = lane * 8; v < V; v += kGroupIds) {
      Eight<T> x;
      x.load(row + v);
      lanes.add(x.max());
    }
    floor_x = __shfl_sync(0xffffffffu, lanes.sorted(), top - 1);
#pragma unroll 4
    for (int v0 = 0; v0 < V; v0 += kGroupIds) {
      const int v = v0 + lane * 8;
      Eight<T> x;
      if (v < V)
        x.load(row + v);
      else
        x.fill_low();
      list_eight(v < V && x.max() >= floor_x, v);
    }
  }
  __syncwarp();
  if (floor_x > -INFINITY && n_eights <= kMaxEights) {
    int n_cand = 0;
    for (int i0 = 0; i0 < n_eights; i0 += 32) {  // four at a time, eight loads in flight
      float f[8];
      int id[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + k * 4 + (lane >> 3);
        id[k] = i < n_eights ? sm.eights[i] + (lane & 7) : -1;
        f[k] = id[k] >= 0 ? to_f32(row[id[k]]) : -INFINITY;  // (below the threshold)
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool y = f[k] >= floor_x;
        const unsigned b = __ballot_sync(0xffffffffu, y);
        const int at = n_cand + __popc(b & below);
        if (y && at < kMaxCand)
          cand[at] = (unsigned long long)rank_key(f[k]) << 32 | ~(uint32_t)id[k];
        n_cand += __popc(b);
      }
    }
    __syncwarp();
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
  }
  // Many ids tie at the threshold, or fewer than `top` are finite:
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

// Merges the parts of a wanted row and finishes it: one warp a row, the first
// CTAs (the list keeps the SMs evenly loaded: with the rows in place, most of a
// CTA's warps would have none).
template <typename T>
__global__ void __launch_bounds__(kFinishWarps * 32, kFinishCtas)
logprobs_finish_kernel(const T* Z, long long row_stride,
                       const int32_t* tokens, int V, int blocks, int groups, float c,
                       float invT, const float4* parts, float* gmax, const int* rows_wanted,
                       const RowOutputs o) {
  __shared__ RowScratch scratch[kFinishWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = blockIdx.x * kFinishWarps + warp;
  wait_for_previous();
  const int r = __ldcg(rows_wanted + 1 + i);  // (read with the count: a row of the list or, past it, unused)
  if (i >= __ldcg(rows_wanted)) return;
  float* gm = gmax + (size_t)r * groups;
  const float4* part = parts + (size_t)r * blocks;
  const int tok = tokens[r];
  GroupTile tile;
  tile.load(gm, 0, groups);
  const T* row = Z + (long long)r * row_stride;
  const float x_tok = tok < V ? to_f32(row[tok]) : __int_as_float(0x7fc00000);

  Part sum{-INFINITY, 0.0f, 0.0f};
  for (int k0 = 0; k0 < blocks; k0 += 128) {
    float4 p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      p[k] = k0 + k * 32 + lane < blocks ? part[k0 + k * 32 + lane]
                                         : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < 4; ++k) merge(sum, p[k].x, p[k].y, p[k].z, c);
  }
  const float all = warp_max(sum.m);
  if (sum.m != -INFINITY) {
    const float d = (sum.m - all) * c, f = ex2(d);
    sum.t = f > 0.0f ? f * (sum.t + d * sum.s) : 0.0f;
    sum.s *= f;
  }
  const Part row_sum{all, warp_sum(sum.s), warp_sum(sum.t)};
  finish_row(row, r, x_tok, V, groups, invT, row_sum, gm, tile, o, scratch[warp]);
}

// Short rows: sums and results by the same warp, in one launch.
template <typename T>
__global__ void __launch_bounds__(kFinishWarps * 32)
logprobs_short_kernel(const T* Z, long long row_stride,
                      const int32_t* tokens, int n_rows, int V, int groups, float c,
                      float invT, float* gmax, const RowOutputs o, int* status) {
  __shared__ RowScratch scratch[kFinishWarps];
  const int warp = threadIdx.x >> 5, r = blockIdx.x * kFinishWarps + warp;
  wait_for_previous();
  if (blockIdx.x == 0) {  // the status word, from all tokens
    bool bad = false;
    for (int i = threadIdx.x; i < n_rows; i += kFinishWarps * 32) bad |= tokens[i] >= V;
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) *status = any ? DSPARK_DEV_BAD_INPUT : 0;
  }
  if (r >= n_rows) return;
  const int tok = tokens[r];
  if (tok < 0) {
    skip_row(o, r);
    return;
  }
  const T* row = Z + (long long)r * row_stride;
  const float x_tok = tok < V ? to_f32(row[tok]) : __int_as_float(0x7fc00000);
  float* gm = gmax + (size_t)r * groups;
  Part sum{-INFINITY, 0.0f, 0.0f};
  for (int v = 0; v < V; v += block_ids<T>()) {
    Block<T> b;
    b.load(row, v, V);
    const Part p = block_part(b, v / kGroupIds, groups, c, gm);
    merge(sum, p.m, p.s, p.t, c);
  }
  __syncwarp();
  GroupTile tile;
  finish_row(row, r, x_tok, V, groups, invT, sum, gm, tile, o, scratch[warp]);
}

int groups_of(int V) { return (V + kGroupIds - 1) / kGroupIds; }
template <typename T>
int blocks_of(int V) {
  return (V + block_ids<T>() - 1) / block_ids<T>();
}

template <typename T>
cudaError_t launch(const void* Z, long long row_stride, const int32_t* tokens, int n_rows, int V,
                   float invT, const RowOutputs& o, char* ws, const LogprobsWorkspace& w,
                   cudaStream_t s) {
  float4* parts = (float4*)(ws + w.parts);
  float* gmax = (float*)(ws + w.gmax);
  int* rows_wanted = (int*)(ws + w.rows);
  const int blocks = blocks_of<T>(V), groups = groups_of(V);
  const float c = invT * kLog2e;
  const int row_ctas = (n_rows + kFinishWarps - 1) / kFinishWarps;
  cudaLaunchAttribute attr;
  if (V <= kShortIds && n_rows <= kShortRows) {
    const cudaLaunchConfig_t cfg = overlapped_launch(dim3(row_ctas), kFinishWarps * 32, 0, s, &attr);
    return cudaLaunchKernelEx(&cfg, logprobs_short_kernel<T>, (const T*)Z, row_stride, tokens, n_rows,
                              V, groups, c, invT, gmax, o, (int*)ws);
  }
  const long long units = (long long)n_rows * blocks;  // few: a block an SM first
  const cudaLaunchConfig_t stream_cfg =
      overlapped_launch(dim3((unsigned)(units < 152 ? units : 152)), kRowThreads, 0, s, &attr);
  const cudaError_t e = cudaLaunchKernelEx(&stream_cfg, logprobs_stream_kernel<T>, (const T*)Z, row_stride,
                                           tokens, n_rows, V, blocks, groups, c, parts, gmax,
                                           rows_wanted, o, (int*)ws);
  if (e != cudaSuccess) return e;
  const cudaLaunchConfig_t cfg = overlapped_launch(dim3(row_ctas), kFinishWarps * 32, 0, s, &attr);
  return cudaLaunchKernelEx(&cfg, logprobs_finish_kernel<T>, (const T*)Z, row_stride, tokens, V,
                            blocks, groups, c, invT, (const float4*)parts, gmax,
                            (const int*)rows_wanted, o);
}

}  // namespace

LogprobsWorkspace logprobs_workspace_layout(int n_rows, int V) {
  LogprobsWorkspace w;
  w.rows = 256;
  // (read up to a whole CTA of the second kernel past the last row)
  w.parts = align_up256(w.rows + ((size_t)n_rows + 1 + kFinishWarps) * sizeof(int));
  w.gmax = align_up256(w.parts + (size_t)n_rows * blocks_of<float>(V) * sizeof(float4));
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
