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
constexpr int kListRows = 1024;     // wanted rows a CTA lists at a time
constexpr int kMaxTop = 32;
constexpr int kSmemGroups = 2048;   // group maxima that the second kernel keeps in shared memory
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

// (m, s, t) of one chunk of a row by one warp (m: the largest logit; t in units
// of log2), and the groups' largest logits.  Per 8 logits a lane: one 16-byte
// load, the maximum (packed for bf16, one warp reduction), and packed pairs
// through y = x c - m c, p = 2^y, s += p, t += p y.  A masked id makes p y =
// 0 * -inf = NaN: a block of 1024 ids whose t is NaN is summed again from its
// registers with y held above -1e30.
template <typename T>
__device__ __forceinline__ void chunk_sums(const T* row, int v0, int v1, float c, float* gmax,
                                           float4* part) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, s = 0.0f, t = 0.0f;
  const f32x2 c2 = pack2(c, c);
  constexpr int kU = 4;
  for (int b = v0; b < v1; b += kU * kGroupIds) {
    Eight<T> x[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int v = b + k * kGroupIds + lane * 8;  // V % 8 == 0: all 8 ids or none
      if (v < v1)
        x[k].load(row + v);
      else
        x[k].fill_low();
    }
    float best = -INFINITY;
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const float g = warp_max_redux(fmaxf(x[k].max(), -INFINITY));  // (NaN counts as -inf)
      if (lane == 0 && b + k * kGroupIds < v1) gmax[b / kGroupIds + k] = g;
      best = fmaxf(best, g);
    }
    if (best > m) {  // the same for all lanes
      const float d = (m - best) * c, f = ex2(d);  // m = -inf: the sums are 0
      t = m == -INFINITY ? 0.0f : f * (t + d * s);
      s *= f;
      m = best;
    }
    const float mm = m == -INFINITY ? 0.0f : m;
    const f32x2 mc2 = pack2(-mm * c, -mm * c);
    f32x2 s2[2] = {0ull, 0ull}, t2[2] = {0ull, 0ull};
#pragma unroll
    for (int k = 0; k < kU; ++k) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f32x2 y = fma2(x[k].pair(e), c2, mc2);
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
      for (int k = 0; k < kU; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x0, x1;
          unpack2(x[k].pair(e), x0, x1);
          const float y0 = (x0 - mm) * c, y1 = (x1 - mm) * c;
          const float p0 = ex2(y0), p1 = ex2(y1);
          sa += p0 + p1;
          ta = fmaf(p0, fmaxf(y0, -1e30f), ta);
          ta = fmaf(p1, fmaxf(y1, -1e30f), ta);
        }
      }
    }
    s += sa;
    t += ta;
  }
  s = warp_sum(s);
  t = warp_sum(t);
  if (lane == 0) *part = make_float4(m, s, t, 0.0f);
}

// The wanted rows' chunks, in equal contiguous shares a CTA.  Every CTA finds
// its rows itself, by a prefix sum over the tokens (a few us beside a launch
// and a list in memory).
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
logprobs_stream_kernel(const T* __restrict__ Z, long long row_stride,
                       const int32_t* __restrict__ tokens, int n_rows, int V, int chunks,
                       int groups, float c, float4* parts, float* gmax, int* status) {
  __shared__ int sm[kRowWarps], list[kListRows];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int seg = (n_rows + kRowThreads - 1) / kRowThreads;
  const int r0 = min(n_rows, (int)threadIdx.x * seg), r1 = min(n_rows, r0 + seg);
  int mine = 0;
  bool bad = false;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    const int tok = __ldg(tokens + r);
    mine += tok >= 0 ? 1 : 0;
    bad |= tok >= V;
  }
  int n;
  const int first = block_scan(mine, sm, &n);
  const int any_bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = any_bad ? DSPARK_DEV_BAD_INPUT : 0;

  const long long units = (long long)n * chunks;
  const long long u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  for (long long k0 = u0 / chunks; k0 * chunks < u1; k0 += kListRows) {
    const long long k1 = k0 + kListRows;  // wanted rows k0 .. k1 - 1 of all
    if (first < k1 && first + mine > k0) {
      long long k = first;
      for (int r = r0; r < r1; ++r)
        if (__ldg(tokens + r) >= 0) {
          if (k >= k0 && k < k1) list[k - k0] = r;
          ++k;
        }
    }
    __syncthreads();
    const long long a = u0 > k0 * chunks ? u0 : k0 * chunks, b = u1 < k1 * chunks ? u1 : k1 * chunks;
    for (long long u = a + (threadIdx.x >> 5); u < b; u += kRowWarps) {
      const int i = (int)(u / chunks - k0), ch = (int)(u % chunks);
      const int r = list[i];
      const int v0 = ch * kChunkIds, v1 = min(V, v0 + kChunkIds);
      chunk_sums(Z + (long long)r * row_stride, v0, v1, c, gmax + (size_t)r * groups,
                 parts + (size_t)r * chunks + ch);
    }
    __syncthreads();
  }
}

// Order of the alternatives as unsigned keys: larger logit, larger key; NaN
// counts as -inf, -0 as 0; 0 stands for "none".
__device__ __forceinline__ uint32_t rank_key(float x) {
  return key_ord(isnan(x) ? -INFINITY : x + 0.0f);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// One warp a row: merges the chunks; picks the `top` best groups by their
// largest logits; fetches them into shared memory, all at once; then draws the
// alternatives one by one: the best head among the picked groups, the lowest
// id that has it, and that group's next head.
template <typename T>
__global__ void __launch_bounds__(32)
logprobs_finish_kernel(const T* __restrict__ Z, long long row_stride,
                       const int32_t* __restrict__ tokens, int V, int chunks, int groups, float c,
                       float invT, int top, const float4* parts, float* gmax, float* logp,
                       float* entropy, float* lse_out, int32_t* top_ids, float* top_logp) {
  extern __shared__ uint4 smem4[];
  const int r = blockIdx.x, lane = threadIdx.x;
  const int tok = __ldg(tokens + r);
  const T* row = Z + (long long)r * row_stride;
  const float nan = __int_as_float(0x7fc00000);
  if (tok < 0) {
    if (lane == 0) logp[r] = entropy[r] = lse_out[r] = nan;
    if (lane < top) {
      top_ids[(size_t)r * top + lane] = -1;
      top_logp[(size_t)r * top + lane] = nan;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const float x_tok = tok < V ? to_f32(row[tok]) : nan;
  asm volatile("griddepcontrol.wait;" ::: "memory");

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
  {
    const float all = warp_max(m);
    if (m != -INFINITY) {
      const float d = (m - all) * c, f = ex2(d);
      t = f > 0.0f ? f * (t + d * s) : 0.0f;
      s *= f;
    }
    m = all;
  }
  s = warp_sum(s);
  t = warp_sum(t);
  const float ln_s = logf(s);
  if (lane == 0) {
    logp[r] = (x_tok - m) * invT - ln_s;
    entropy[r] = ln_s - t / s * kLn2;
    lse_out[r] = m * invT + ln_s;
  }
  if (top == 0) return;

  // Shared memory: the picked groups' logits, the ids drawn from them (a bit an
  // id), and the group maxima's keys where they fit (else in gmax itself).
  T* stage = (T*)smem4;                                  // [top][256]
  uint8_t* drawn = (uint8_t*)(stage + top * kGroupIds);  // [top][32]
  uint32_t* keys = groups <= kSmemGroups ? (uint32_t*)(drawn + kMaxTop * 32)
                                         : (uint32_t*)(gmax + (size_t)r * groups);
  const float* gm = gmax + (size_t)r * groups;
  uint32_t bk = 0;  // this lane's best remaining group: key and index
  int bg = 0x7fffffff;
#pragma unroll 8
  for (int g = lane; g < groups; g += 32) {
    const uint32_t k = rank_key(gm[g]);
    keys[g] = k;
    if (k > bk) bk = k, bg = g;  // (ties: the lower index)
  }
  const int n_sel = min(top, groups);
  uint32_t head = 0;  // lane i < n_sel: the key of picked group i's best id not drawn yet
  int sel = 0;        // and that group
  for (int i = 0; i < n_sel; ++i) {
    const uint32_t k = __reduce_max_sync(0xffffffffu, bk);
    const int g = __reduce_min_sync(0xffffffffu, bk == k ? bg : 0x7fffffff);
    if (lane == i) head = k, sel = g;
    if (bg == g && bk == k) {
      keys[g] = 0;
      bk = 0, bg = 0x7fffffff;
      for (int j = lane; j < groups; j += 32) {
        const uint32_t q = keys[j];
        if (q > bk) bk = q, bg = j;
      }
    }
  }
  const uint32_t stage_s = (uint32_t)__cvta_generic_to_shared(stage);
  for (int i = 0; i < n_sel; ++i) {
    const int v = __shfl_sync(0xffffffffu, sel, i) * kGroupIds + lane * 8;
    if (v < V) {
      const uint32_t d = stage_s + (uint32_t)((i * kGroupIds + lane * 8) * sizeof(T));
      cp_async16(d, row + v);
      if (sizeof(T) == 4) cp_async16(d + 16, row + v + 4);
    }
    drawn[i * 32 + lane] = v < V ? 0 : 0xff;  // ids past V are never drawn
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  int my_id = -1;
  float my_x = nan;
  for (int k = 0; k < top; ++k) {
    const uint32_t hk = __reduce_max_sync(0xffffffffu, head);
    if (hk == 0) break;  // (not reached: top <= V)
    const int g = __reduce_min_sync(0xffffffffu, head == hk ? sel : 0x7fffffff);
    const int i = __ffs(__ballot_sync(0xffffffffu, head == hk && sel == g && lane < n_sel)) - 1;
    uint32_t taken = drawn[i * 32 + lane];
    const T* x = stage + i * kGroupIds + lane * 8;
    uint32_t q[8];
    int at = 0x7fffffff;  // this lane's lowest open id with the head's key
#pragma unroll
    for (int e = 7; e >= 0; --e) {
      q[e] = taken >> e & 1u ? 0u : rank_key(to_f32(x[e]));
      if (q[e] == hk) at = lane * 8 + e;
    }
    const int id = __reduce_min_sync(0xffffffffu, at);
    uint32_t next = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (lane * 8 + e != id && q[e] > next) next = q[e];
    if (id >> 3 == lane) drawn[i * 32 + lane] = (uint8_t)(taken | 1u << (id & 7));
    next = __reduce_max_sync(0xffffffffu, next);
    if (lane == i) head = next;
    if (lane == k) my_id = g * kGroupIds + id, my_x = ord_key(hk);
    __syncwarp();
  }
  if (lane < top) {
    top_ids[(size_t)r * top + lane] = my_id;
    top_logp[(size_t)r * top + lane] = (my_x - m) * invT - ln_s;
  }
}

int groups_of(int V) { return (V + kGroupIds - 1) / kGroupIds; }
int chunks_of(int V) { return (V + kChunkIds - 1) / kChunkIds; }

template <typename T>
cudaError_t launch(const void* Z, long long row_stride, const int32_t* tokens, int n_rows, int V,
                   float invT, int top, float* logp, float* entropy, float* lse, int32_t* top_ids,
                   float* top_logp, char* ws, const LogprobsWorkspace& w, cudaStream_t s) {
  float4* parts = (float4*)(ws + w.parts);
  float* gmax = (float*)(ws + w.gmax);
  const int chunks = chunks_of(V), groups = groups_of(V);
  const float c = invT * kLog2e;
  long long ctas = ((long long)n_rows * chunks + kRowWarps - 1) / kRowWarps;
  if (ctas > 152 * 6) ctas = 152 * 6;
  logprobs_stream_kernel<T><<<(int)ctas, kRowThreads, 0, s>>>(
      (const T*)Z, row_stride, tokens, n_rows, V, chunks, groups, c, parts, gmax, (int*)ws);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_rows);
  cfg.blockDim = dim3(32);
  cfg.dynamicSmemBytes = (size_t)top * kGroupIds * sizeof(T) + kMaxTop * 32 +
                         (groups <= kSmemGroups ? (size_t)groups * 4 : 0);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_finish_kernel<T>, (const T*)Z, row_stride, tokens, V,
                            chunks, groups, c, invT, top, (const float4*)parts, gmax, logp, entropy,
                            lse, top_ids, top_logp);
}

}  // namespace

LogprobsWorkspace logprobs_workspace_layout(int n_rows, int V) {
  LogprobsWorkspace w;
  w.parts = 256;
  w.gmax = align_up256(w.parts + (size_t)n_rows * chunks_of(V) * sizeof(float4));
  w.total = align_up256(w.gmax + (size_t)n_rows * groups_of(V) * sizeof(float));
  return w;
}

cudaError_t launch_logprobs(const void* Z, int dtype, long long row_stride, const int32_t* tokens,
                            int n_rows, int V, float invT, int top, float* logp, float* entropy,
                            float* lse, int32_t* top_ids, float* top_logp, char* ws,
                            const LogprobsWorkspace& w, cudaStream_t s) {
  return dtype == DSPARK_BF16
             ? launch<__nv_bfloat16>(Z, row_stride, tokens, n_rows, V, invT, top, logp, entropy,
                                     lse, top_ids, top_logp, ws, w, s)
             : launch<float>(Z, row_stride, tokens, n_rows, V, invT, top, logp, entropy, lse,
                             top_ids, top_logp, ws, w, s);
}

}  // namespace dspark
