// attention.cu -- attention of a chunk of new tokens over the paged K/V cache:
// the CUDA-core kernel (fp32, and the bf16 shapes that the tensor-core kernel
// does not take) and the combine of cut items.
//
// Token i of request r's chunk sits at position L - n + i and sees the cached
// positions up to its own.  For each row, over the keys j in tiles:
//   s_j = scale q . k_j,  m' = max(m, s_j),  l = l e^{m-m'} + e^{s_j-m'},
//   o = o e^{m-m'} + e^{s_j-m'} v_j;   out = o / l,  lse = m + ln l.
// A row that sees no key gets out = 0 and lse = -inf.
#include <type_traits>

#include "attention.cuh"

namespace dspark {

namespace {

constexpr int kMR = 32;  // rows of an item: 8 warps x 4 rows
constexpr int kTN = 32;  // keys of a tile: one a lane
constexpr int kThreads = 256;
constexpr int kRowsPerWarp = 4;
constexpr float kLn2 = 0.6931471805599453f;

// One warp holds 4 rows: lane j scores key j of the tile (K from shared memory,
// row stride D + 4 floats, free of bank conflicts for 16-byte reads), then
// lanes hold output columns lane + 32 i.
template <typename T, int NI>  // NI = ceil(D / 32)
__global__ void __launch_bounds__(kThreads)
attention_simt_kernel(const AttnParams p) {
  extern __shared__ float4 smem4[];
  __shared__ AttnStart<kTN> st;
  __shared__ int flags;
  __shared__ __align__(16) float sp[kThreads / 32][kTN][kRowsPerWarp];  // probabilities of a warp's rows
  const int D = p.a.c.head_dim, ld = NI * 32 + 4;
  float* sq = (float*)smem4;       // [kMR][ld], scaled by scale * log2 e
  float* sk = sq + kMR * ld;       // [kTN][ld]
  float* sv = sk + kTN * ld;       // [kTN][ld]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int S = p.a.c.page_size, G = p.a.G;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) flags = 0;
  __syncthreads();
  attn_plan<kTN>(p, &st, &flags);
  AttnWalk<kTN> w = st.walk;
  if (threadIdx.x == 0) attn_write_cut(p, st);

  for (; !w.done(); w.next(p, &flags)) {
    const int rows = w.block_rows(p), row0 = w.m * kMR;
    __syncthreads();
    for (int i = threadIdx.x; i < kMR * NI * 32; i += kThreads) {
      const int a = i / (NI * 32), d = i - a * (NI * 32);
      float x = 0.0f;
      if (a < rows && d < D) {
        const int tok = (row0 + a) / G, g = (row0 + a) - tok * G;
        x = to_f32(((const T*)p.a.q)[(long long)(w.q.q0 + tok) * p.a.q_token_stride +
                                     (long long)(w.h * G + g) * p.a.q_head_stride + d]);
      }
      sq[a * ld + d] = x;
    }
    float m[kRowsPerWarp], l[kRowsPerWarp], o[kRowsPerWarp][NI];
    int lim[kRowsPerWarp];  // keys that the row sees
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
      const int a = warp * kRowsPerWarp + i;
      m[i] = -INFINITY, l[i] = 0.0f;
      lim[i] = a < rows ? w.q.L - w.q.n + (row0 + a) / G + 1 : 0;
#pragma unroll
      for (int k = 0; k < NI; ++k) o[i][k] = 0.0f;
    }
    for (int t = w.first_tile(); t < w.last_tile(); ++t) {
      const int j0 = t * kTN;
      __syncthreads();
      // K and V of the tile; positions at or past `end` read as zeros.
      for (int a = warp; a < kTN; a += kThreads / 32) {
        const int j = j0 + a;
        int page = -1;
        if (j < w.end) {
          page = p.a.a.page_table[(size_t)w.r * p.a.a.max_pages + j / S];
          if (page < 0 || page >= p.a.c.n_pages) {
            if (lane == 0) flag_status(&flags, DSPARK_DEV_BAD_INPUT);
            page = page < 0 ? 0 : p.a.c.n_pages - 1;
          }
        }
        const long long at = page * p.a.c.page_stride + (j % S) * p.a.c.token_stride +
                             w.h * p.a.c.head_stride;
#pragma unroll
        for (int k = 0; k < NI; ++k) {
          const int d = lane + 32 * k;
          const bool in = page >= 0 && d < D;
          sk[a * ld + d] = in ? to_f32(((const T*)p.a.c.k)[at + d]) : 0.0f;
          sv[a * ld + d] = in ? to_f32(((const T*)p.a.c.v)[at + d]) : 0.0f;
        }
      }
      __syncthreads();
      if (warp * kRowsPerWarp < rows) {
        float s[kRowsPerWarp] = {};
        const float4* kr = (const float4*)(sk + lane * ld);
#pragma unroll 4
        for (int d = 0; d < NI * 8; ++d) {
          const float4 kx = kr[d];
#pragma unroll
          for (int i = 0; i < kRowsPerWarp; ++i) {
            const float4 qx = ((const float4*)(sq + (warp * kRowsPerWarp + i) * ld))[d];
            s[i] = fmaf(qx.x, kx.x, s[i]);
            s[i] = fmaf(qx.y, kx.y, s[i]);
            s[i] = fmaf(qx.z, kx.z, s[i]);
            s[i] = fmaf(qx.w, kx.w, s[i]);
          }
        }
        float f[kRowsPerWarp];
#pragma unroll
        for (int i = 0; i < kRowsPerWarp; ++i) {
          const float x = j0 + lane < lim[i] ? s[i] * p.scale_log2 : -INFINITY;
          const float mt = fmaxf(m[i], warp_max(x));
          const float ms = mt == -INFINITY ? 0.0f : mt;
          f[i] = exp2f(m[i] - ms);
          const float e = exp2f(x - ms);
          l[i] = l[i] * f[i] + warp_sum(e);
          m[i] = mt;
          sp[warp][lane][i] = e;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kRowsPerWarp; ++i)
#pragma unroll
          for (int k = 0; k < NI; ++k) o[i][k] *= f[i];
#pragma unroll 4
        for (int j = 0; j < kTN; ++j) {
          const float4 e = *(const float4*)sp[warp][j];
#pragma unroll
          for (int k = 0; k < NI; ++k) {
            const float v = sv[j * ld + lane + 32 * k];
            o[0][k] = fmaf(e.x, v, o[0][k]);
            o[1][k] = fmaf(e.y, v, o[1][k]);
            o[2][k] = fmaf(e.z, v, o[2][k]);
            o[3][k] = fmaf(e.w, v, o[3][k]);
          }
        }
        __syncwarp();
      }
    }
    const int slot = attn_slot(w);
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
      const int a = warp * kRowsPerWarp + i;
      if (a >= rows) continue;
      if (slot < 0) {
        const int tok = (row0 + a) / G, g = (row0 + a) - tok * G;
        const size_t at = (size_t)(w.q.q0 + tok) * p.a.Hq + w.h * G + g;
        const float inv = l[i] > 0.0f ? 1.0f / l[i] : l[i] == 0.0f ? 0.0f : l[i];
#pragma unroll
        for (int k = 0; k < NI; ++k)
          if (lane + 32 * k < D) {
            const float y = o[i][k] * inv;
            if (std::is_same<T, float>::value)
              ((float*)p.a.out)[at * D + lane + 32 * k] = y;
            else
              ((__nv_bfloat16*)p.a.out)[at * D + lane + 32 * k] = __float2bfloat16(y);
          }
        if (lane == 0) p.a.lse[at] = l[i] == 0.0f ? -INFINITY : m[i] * kLn2 + logf(l[i]);
      } else {
        const size_t at = ((size_t)blockIdx.x * 2 + slot) * kMR + a;
#pragma unroll
        for (int k = 0; k < NI; ++k)
          if (lane + 32 * k < D) p.part[at * D + lane + 32 * k] = o[i][k];
        if (lane == 0) p.stats[at] = make_float2(m[i], l[i]);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) p.flags[blockIdx.x] = flags;
}

// Adds the pieces of the items that shares cut.  Block (b, y): the item that
// CTA b + 1's share is the first to begin inside of; its warps take the rows in
// turn.  (As many blocks as the likely rows fill: for decoding, with a few rows
// an item, blocks without a row cost more than they save others.)  VE columns a
// lane and step: four where rows are whole 16-byte vectors.  Bound by the read
// of the pieces, which the attention kernel has just left in L2.
template <typename T, int NI, int VE>
__global__ void __launch_bounds__(256, NI * VE <= 4 ? 6 : 4)
attention_combine_kernel(const AttnParams p, int MR, int ctas) {
  struct alignas(4 * VE) Vec {
    float e[VE];
  };
  struct alignas(sizeof(T) * VE) Out {
    T e[VE];
  };
  constexpr int kAhead = 2;  // pieces in flight (four left room for half as many rows an SM: 436 for 429 us)
  // Launched while the attention kernel runs; everything below reads what it wrote.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) {  // the call's status word
    int f = 0;
    for (int i = threadIdx.x; i < ctas; i += 32) f |= __ldcg(p.flags + i);
    f = __reduce_or_sync(0xffffffffu, f);
    if (threadIdx.x == 0) *p.status = f;
  }
  const int c = blockIdx.x + 1;
  if (c >= ctas) return;
  const CutItem it = p.cuts[c];
  const int n = it.pieces;
  if (n == 0) return;
  const int lane = threadIdx.x & 31, D = p.a.c.head_dim, G = p.a.G;
  for (int a = blockIdx.y * 8 + (threadIdx.x >> 5); a < it.rows; a += gridDim.y * 8) {
    const auto at = [&](int i) {
      return (i == 0 ? (size_t)(c - 1) * 2 + 1 : (size_t)(c - 1 + i) * 2) * MR + a;
    };
    Vec v[kAhead][NI];
    auto load = [&](int i0) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int k = 0; k < NI; ++k) {
          v[i][k] = Vec{};
          if (i0 + i < n && (lane + 32 * k) * VE < D)
            v[i][k] = ((const Vec*)(p.part + at(i0 + i) * D))[lane + 32 * k];
        }
    };
    load(0);
    // The weights of 32 pieces at a time, one a lane.
    const float2 none = make_float2(-INFINITY, 0.0f);
    float2 st = lane < n ? p.stats[at(lane)] : none;
    float m = st.x, l = 0.0f;
    for (int i = lane + 32; i < n; i += 32) m = fmaxf(m, p.stats[at(i)].x);
    m = warp_max(m);
    const float ms = m == -INFINITY ? 0.0f : m;
    float o[NI][VE] = {};
    for (int i0 = 0; i0 < n; i0 += 32) {
      if (i0 > 0) st = i0 + lane < n ? p.stats[at(i0 + lane)] : none;
      const float f = exp2f(st.x - ms);
      l += warp_sum(st.y * f);
      for (int i1 = 0; i1 < 32 && i0 + i1 < n; i1 += kAhead) {
        if (i0 + i1 > 0) load(i0 + i1);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const float w = __shfl_sync(0xffffffffu, f, i1 + i);
#pragma unroll
          for (int k = 0; k < NI; ++k)
#pragma unroll
            for (int e = 0; e < VE; ++e) o[k][e] = fmaf(v[i][k].e[e], w, o[k][e]);
        }
      }
    }
    const int row = it.row0 + a, tok = row / G, g = row - tok * G;
    const size_t dst = (size_t)(it.q0 + tok) * p.a.Hq + it.h * G + g;
    const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
#pragma unroll
    for (int k = 0; k < NI; ++k)
      if ((lane + 32 * k) * VE < D) {
        Out y;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          if constexpr (std::is_same<T, float>::value)
            y.e[e] = o[k][e] * inv;
          else
            y.e[e] = __float2bfloat16(o[k][e] * inv);
        }
        ((Out*)((T*)p.a.out + dst * D))[lane + 32 * k] = y;
      }
    if (lane == 0) p.a.lse[dst] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
  }
}

template <typename T>
cudaError_t launch_combine(const cudaLaunchConfig_t& cfg, const AttnParams& p, int MR, int ctas) {
  const int D = p.a.c.head_dim;
  if (D % 4 == 0)
    return D <= 128 ? cudaLaunchKernelEx(&cfg, attention_combine_kernel<T, 1, 4>, p, MR, ctas)
                    : cudaLaunchKernelEx(&cfg, attention_combine_kernel<T, 2, 4>, p, MR, ctas);
  return D <= 128 ? cudaLaunchKernelEx(&cfg, attention_combine_kernel<T, 4, 1>, p, MR, ctas)
                  : cudaLaunchKernelEx(&cfg, attention_combine_kernel<T, 8, 1>, p, MR, ctas);
}

constexpr int kSimtCtas = 304;

template <typename T, int NI>
cudaError_t launch_simt(const AttnParams& p, cudaStream_t s) {
  const int smem = 3 * kMR * (NI * 32 + 4) * (int)sizeof(float);
  static const cudaError_t attr = cudaFuncSetAttribute(
      attention_simt_kernel<T, NI>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (attr != cudaSuccess) return attr;
  attention_simt_kernel<T, NI><<<kSimtCtas, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_simt_dim(const AttnParams& p, cudaStream_t s) {
  const int ni = (p.a.c.head_dim + 31) / 32;
  if (ni <= 1) return launch_simt<T, 1>(p, s);
  if (ni <= 2) return launch_simt<T, 2>(p, s);
  if (ni <= 4) return launch_simt<T, 4>(p, s);
  return launch_simt<T, 8>(p, s);
}

}  // namespace

cudaError_t launch_attn_combine(const AttnParams& p, int MR, int ctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const long long rows = attn_likely_rows(p.a);
  cfg.gridDim = dim3(ctas > 1 ? ctas - 1 : 1, (unsigned)((rows < MR ? rows : MR) + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.a.dtype == DSPARK_BF16 ? launch_combine<__nv_bfloat16>(cfg, p, MR, ctas)
                                  : launch_combine<float>(cfg, p, MR, ctas);
}

size_t attention_workspace_bytes(int dtype, int head_dim) {
  const size_t simt = attn_workspace_layout(kMR, head_dim).total;
  if (dtype != DSPARK_BF16 || head_dim > 128) return simt;
  const size_t tc = attention_tc_workspace_bytes(head_dim);
  return tc > simt ? tc : simt;
}

cudaError_t launch_paged_attention(const AttnArgs& a, char* ws, cudaStream_t s) {
  if (a.a.n_tokens == 0) return cudaMemsetAsync(ws, 0, sizeof(int), s);
  if (attention_tc_supported(a)) return launch_attention_tc(a, ws, s);
  const AttnWorkspace w = attn_workspace_layout(kMR, a.c.head_dim);
  AttnParams p{a, (int*)ws, (int*)(ws + w.flags), (CutItem*)(ws + w.cuts),
               (float2*)(ws + w.stats), (float*)(ws + w.out), a.scale * 1.4426950408889634f,
               attn_item_units(a), kMR};
  const cudaError_t e = a.dtype == DSPARK_BF16 ? launch_simt_dim<__nv_bfloat16>(p, s) : launch_simt_dim<float>(p, s);
  if (e != cudaSuccess) return e;
  return launch_attn_combine(p, kMR, kSimtCtas, s);
}

}  // namespace dspark
