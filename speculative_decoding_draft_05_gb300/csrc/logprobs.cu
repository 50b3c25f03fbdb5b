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

constexpr int kGroupIds = 256;                    // ids a group: 32 lanes x 8
constexpr int kChunkGroups = 16;                  // groups a warp's chunk
constexpr int kChunkIds = kGroupIds * kChunkGroups;
constexpr int kRowThreads = 256;
constexpr int kMaxTop = 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 8 consecutive logits (one lane's share of a group) as floats.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldcs((const float4*)p), b = __ldcs((const float4*)p + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 a = __ldcs((const uint4*)p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// The wanted rows (token >= 0), in order, and empty results for the others.
__global__ void __launch_bounds__(1024)
logprobs_rows_kernel(const int32_t* tokens, int n_rows, int top, int* count, int* list, float* logp,
                     float* entropy, float* lse, int32_t* top_ids, float* top_logp) {
  __shared__ int sm[33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int base = 0;
  for (int r0 = 0; r0 < n_rows; r0 += 1024) {
    const int r = r0 + (int)threadIdx.x;
    const bool want = r < n_rows && tokens[r] >= 0;
    const unsigned b = __ballot_sync(0xffffffffu, want);
    if (lane == 0) sm[warp] = __popc(b);
    __syncthreads();
    if (warp == 0) {
      int v = sm[lane];
      const int own = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      sm[lane] = v - own;
      if (lane == 31) sm[32] = v;
    }
    __syncthreads();
    if (want) list[base + sm[warp] + __popc(b & ((1u << lane) - 1u))] = r;
    if (r < n_rows && !want) {
      const float nan = __int_as_float(0x7fc00000);
      logp[r] = nan;
      entropy[r] = nan;
      lse[r] = nan;
      for (int i = 0; i < top; ++i) {
        top_ids[(size_t)r * top + i] = -1;
        top_logp[(size_t)r * top + i] = nan;
      }
    }
    base += sm[32];
    __syncthreads();
  }
  if (threadIdx.x == 0) *count = base;
}

// (m, s, t) of one chunk of a row by one warp (m: the largest logit; t in units
// of log2), and the groups' largest logits.
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
logprobs_stream_kernel(const T* __restrict__ Z, long long row_stride, const int* count,
                       const int* list, int V, int chunks, int groups, float c, float4* parts,
                       float* gmax) {
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * (kRowThreads / 32);
  const long long units = (long long)*count * chunks;
  for (long long u = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); u < units;
       u += warps) {
    const int i = (int)(u / chunks), ch = (int)(u - (long long)i * chunks);
    const T* row = Z + (long long)list[i] * row_stride;
    const int v0 = ch * kChunkIds, v1 = min(V, v0 + kChunkIds);
    float m = -INFINITY, s = 0.0f, t = 0.0f;  // largest logit; this lane's sums relative to it
    constexpr int kU = 4;
    for (int b = v0; b < v1; b += kU * kGroupIds) {
      float x[kU][8];
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        const int v = b + k * kGroupIds + lane * 8;  // V % 8 == 0: all 8 ids or none
        if (v < v1) {
          load8(row + v, x[k]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[k][e] = -INFINITY;
        }
      }
      float best = -INFINITY;
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        float g = fmaxf(fmaxf(fmaxf(x[k][0], x[k][1]), fmaxf(x[k][2], x[k][3])),
                        fmaxf(fmaxf(x[k][4], x[k][5]), fmaxf(x[k][6], x[k][7])));
        g = warp_max(fmaxf(g, -INFINITY));  // (NaN counts as -inf)
        const int j = b / kGroupIds + k;
        if (lane == 0 && j < groups) gmax[(size_t)i * groups + j] = g;
        best = fmaxf(best, g);
      }
      if (best > m) {  // the same for all lanes
        const float d = (m - best) * c, f = ex2(d);  // m = -inf: the sums are 0
        t = m == -INFINITY ? 0.0f : f * (t + d * s);
        s *= f;
        m = best;
      }
      const float mm = m == -INFINITY ? 0.0f : m;
      const float mc = mm * c;
      if (fabsf(mm) < 1e30f) {
#pragma unroll
        for (int k = 0; k < kU; ++k) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float y = fmaf(x[k][e], c, -mc);
            const float p = ex2(y);
            s += p;
            t = fmaf(p, fmaxf(y, -1e30f), t);  // a masked id: 0 * -1e30, not 0 * -inf
          }
        }
      } else {  // m c could overflow (a row masked with the type's lowest value)
#pragma unroll
        for (int k = 0; k < kU; ++k) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float y = (x[k][e] - mm) * c;
            const float p = ex2(y);
            s += p;
            t = fmaf(p, fmaxf(y, -1e30f), t);
          }
        }
      }
    }
    s = warp_sum(s);
    t = warp_sum(t);
    if (lane == 0) parts[(size_t)i * chunks + ch] = make_float4(m, s, t, 0.0f);
  }
}

// Comes (a, ia) before (b, ib) in the order of the alternatives?  NaN logits
// have been replaced by -inf.
__device__ __forceinline__ bool before(float a, int ia, float b, int ib) {
  return a > b || (a == b && ia < ib);
}

// One warp a row: merges the chunks, then draws the alternatives one by one
// from the groups' heads.  Lane l holds the heads of groups l, l + 32, ...: the
// best of them stays in registers, the rest in gmax (which the row owns).
template <typename T>
__global__ void __launch_bounds__(32)
logprobs_finish_kernel(const T* __restrict__ Z, long long row_stride, const int32_t* tokens,
                       const int* count, const int* list, int V, int chunks, int groups, float c,
                       float invT, int top, const float4* parts, float* gmax, float* logp, float* entropy,
                       float* lse_out, int32_t* top_ids, float* top_logp, int* status) {
  const int i = blockIdx.x, lane = threadIdx.x;
  if (i >= *count) return;
  const int r = list[i];
  const T* row = Z + (long long)r * row_stride;

  float m = -INFINITY, s = 0.0f, t = 0.0f;
  for (int k = lane; k < chunks; k += 32) {
    const float4 p = parts[(size_t)i * chunks + k];
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
    const int tok = tokens[r];
    if (tok >= V) flag_status(status, DSPARK_DEV_BAD_INPUT);
    const float x = tok < V ? to_f32(row[tok]) : __int_as_float(0x7fc00000);
    logp[r] = (x - m) * invT - ln_s;
    entropy[r] = ln_s - t / s * kLn2;
    lse_out[r] = m * invT + ln_s;  // (all masked: -inf - inf)
  }
  if (top == 0) return;

  float* gm = gmax + (size_t)i * groups;
  // heads: the id of each lane's best group; `taken` ids of a group come before
  // its head, so the next head is the best id after the last one taken.
  for (int k = 0; k < top; ++k) {
    float bv = -INFINITY;
    int bg = 0x7fffffff;
    for (int g = lane; g < groups; g += 32) {
      const float v = gm[g];
      // a group that is used up carries NaN and never comes first
      if (v > bv || (v == bv && g < bg)) {
        bv = v;
        bg = g;
      }
    }
    warp_argmax(bv, bg);
    if (bg >= groups) break;  // (not reached: top <= V, so some group has an id left)
    // The head: the first id with value bv that has not been taken.  Taken ids
    // of this group are among top_ids written so far with this group.
    const int v = bg * kGroupIds + lane * 8;
    float x[8];
    if (v < V) {
      load8(row + v, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __int_as_float(0x7fc00000);
    }
    unsigned open = v < V ? 0xffu : 0u;  // ids of this lane that may still be drawn
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (isnan(x[e])) x[e] = -INFINITY;
    for (int q = 0; q < k; ++q) {
      const int id = top_ids[(size_t)r * top + q];
      if (id >= v && id < v + 8) open &= ~(1u << (id - v));
    }
    float h1 = -INFINITY, h2 = -INFINITY;
    int i1 = 0x7fffffff, i2 = 0x7fffffff;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (!(open >> e & 1u)) continue;
      if (before(x[e], v + e, h1, i1)) {
        h2 = h1, i2 = i1;
        h1 = x[e], i1 = v + e;
      } else if (before(x[e], v + e, h2, i2)) {
        h2 = x[e], i2 = v + e;
      }
    }
    float w1 = h1;
    int j1 = i1;
    warp_argmax(w1, j1);
    // the group's next head: the drawn lane offers its second id
    float w2 = j1 == i1 ? h2 : h1;
    int j2 = j1 == i1 ? i2 : i1;
    warp_argmax(w2, j2);
    if (lane == 0) {
      top_ids[(size_t)r * top + k] = j1;
      top_logp[(size_t)r * top + k] = (w1 - m) * invT - ln_s;
      gm[bg] = j2 == 0x7fffffff ? __int_as_float(0x7fc00000) : w2;
    }
    __syncwarp();
  }
}

int groups_of(int V) { return (V + kGroupIds - 1) / kGroupIds; }
int chunks_of(int V) { return (V + kChunkIds - 1) / kChunkIds; }

}  // namespace

LogprobsWorkspace logprobs_workspace_layout(int n_rows, int V) {
  LogprobsWorkspace w;
  w.count = 4;
  w.list = 256;
  w.parts = align_up256(w.list + (size_t)n_rows * sizeof(int));
  w.gmax = align_up256(w.parts + (size_t)n_rows * chunks_of(V) * sizeof(float4));
  w.total = align_up256(w.gmax + (size_t)n_rows * groups_of(V) * sizeof(float));
  return w;
}

cudaError_t launch_logprobs(const void* Z, int dtype, long long row_stride, const int32_t* tokens,
                            int n_rows, int V, float invT, int top, float* logp, float* entropy,
                            float* lse, int32_t* top_ids, float* top_logp, char* ws,
                            const LogprobsWorkspace& w, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(ws, 0, 4, s);
  if (e != cudaSuccess) return e;
  int* count = (int*)(ws + w.count);
  int* list = (int*)(ws + w.list);
  float4* parts = (float4*)(ws + w.parts);
  float* gmax = (float*)(ws + w.gmax);
  const int chunks = chunks_of(V), groups = groups_of(V);
  const float c = invT * kLog2e;
  logprobs_rows_kernel<<<1, 1024, 0, s>>>(tokens, n_rows, top, count, list, logp, entropy, lse,
                                          top_ids, top_logp);
  long long ctas = ((long long)n_rows * chunks + kRowThreads / 32 - 1) / (kRowThreads / 32);
  if (ctas > 152 * 6) ctas = 152 * 6;
  if (dtype == DSPARK_BF16) {
    typedef __nv_bfloat16 T;
    logprobs_stream_kernel<T><<<(int)ctas, kRowThreads, 0, s>>>((const T*)Z, row_stride, count, list,
                                                               V, chunks, groups, c, parts, gmax);
    logprobs_finish_kernel<T><<<n_rows, 32, 0, s>>>((const T*)Z, row_stride, tokens, count, list, V,
                                                    chunks, groups, c, invT, top, parts, gmax, logp,
                                                    entropy, lse, top_ids, top_logp, (int*)ws);
  } else {
    typedef float T;
    logprobs_stream_kernel<T><<<(int)ctas, kRowThreads, 0, s>>>((const T*)Z, row_stride, count, list,
                                                               V, chunks, groups, c, parts, gmax);
    logprobs_finish_kernel<T><<<n_rows, 32, 0, s>>>((const T*)Z, row_stride, tokens, count, list, V,
                                                    chunks, groups, c, invT, top, parts, gmax, logp,
                                                    entropy, lse, top_ids, top_logp, (int*)ws);
  }
  return cudaGetLastError();
}

}  // namespace dspark
