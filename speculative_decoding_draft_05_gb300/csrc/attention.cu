// attention.cu -- attention of a chunk of new tokens over the paged K/V cache:
// the CUDA-core kernel (fp32, and the bf16 shapes that the tensor-core kernel
// does not take) and the combine of cut items.
//
// Token i of request r's chunk sits at position L - n + i and sees the cached
// positions up to its own.  For each row, over the keys j in tiles:
//   s_j = scale q . k_j,  m' = max(m, s_j),  l = l e^{m-m'} + e^{s_j-m'},
//   o = o e^{m-m'} + e^{s_j-m'} v_j;   out = o / l,  lse = m + ln l.
// A row that sees no key gets out = 0 and lse = -inf.
//
// Bound by shared memory's rate where rows are many (a chunk of 1024 fp32 tokens:
// 31 TFLOP/s), by latency and the reads where they are few (decoding of 128 fp32
// requests of 200 .. 2048 positions, 1.13 GB: 285 us, 4.0 TB/s; bf16 with head_dim
// 256, prompts of 2901 + 4096 tokens: 59 ms, 22 TFLOP/s).
#include <type_traits>

#include "attention.cuh"
#include "fp4.cuh"
#include "per_device.h"

namespace dspark {

namespace {

constexpr int kMR = 64;  // rows of an item: 8 warps x 8 rows
constexpr int kTN = 32;  // keys of a tile: one a lane
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerWarp = 8;  // at most
constexpr int kProbPairs = 128;  // (e, e) pairs of a warp in shared memory
constexpr float kSlackLog2 = 8.0f;
constexpr float kLn2 = 0.6931471805599453f;

// Columns d .. d + 3 of a row of D values as floats, zeros past D; `vec`: rows
// are whole, aligned 4-value vectors.
__device__ __forceinline__ float4 load4(const float* row, int d, int D, bool vec) {
  if (vec) return d < D ? *(const float4*)(row + d) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  return make_float4(d < D ? row[d] : 0.0f, d + 1 < D ? row[d + 1] : 0.0f,
                     d + 2 < D ? row[d + 2] : 0.0f, d + 3 < D ? row[d + 3] : 0.0f);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* row, int d, int D, bool vec) {
  if (vec) {
    const uint2 q = d < D ? *(const uint2*)(row + d) : make_uint2(0u, 0u);
    return make_float4(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u),
                       __uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u));
  }
  return make_float4(d < D ? to_f32(row[d]) : 0.0f, d + 1 < D ? to_f32(row[d + 1]) : 0.0f,
                     d + 2 < D ? to_f32(row[d + 2]) : 0.0f, d + 3 < D ? to_f32(row[d + 3]) : 0.0f);
}

// Four elements of a 4-bit row (two bytes of codes), times their scale and the factor.
__device__ __forceinline__ float4 values4_fp4(uint32_t codes, uint32_t scale, float factor) {
  uint32_t h[2];
  fp4x4_to_half(codes, h);
  const float s = e4m3_to_float(scale) * factor;
  return make_float4(half_lo(h[0]) * s, half_hi(h[0]) * s, half_lo(h[1]) * s, half_hi(h[1]) * s);
}

// A warp's rows: reference m (the same in all lanes), this lane's part of the
// sum l, and the output columns 2 lane + 64 k and the next.
template <int NP>
struct Rows {
  float m[kRowsPerWarp], l[kRowsPerWarp];
  int lim[kRowsPerWarp];  // keys that the row sees
  f32x2 o[kRowsPerWarp][NP];
};

// One tile for RW rows.  Lane j scores key j (K from shared memory, row stride
// ld = D + 4 floats: free of bank conflicts for 16-byte reads).  The reference
// follows the maximum only where that lies 2^8 or more above it: mostly once.
// Probabilities pass through shared memory as pairs (e, e), the operands of
// packed products with two columns of V.
template <int NI, int RW>
__device__ __forceinline__ void simt_tile(Rows<NI / 2>& r, const float* sq, const float* sk,
                                          const float* sv, f32x2* sp, int j0, float scale_log2) {
  constexpr int ld = NI * 32 + 4;
  const int lane = threadIdx.x & 31;
  f32x2 s2[RW] = {};
  const ulonglong2* kr = (const ulonglong2*)(sk + lane * ld);
#pragma unroll 8
  for (int d = 0; d < NI * 8; ++d) {
    const ulonglong2 kx = kr[d];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const ulonglong2 qx = ((const ulonglong2*)(sq + i * ld))[d];
      s2[i] = fma2(qx.x, kx.x, s2[i]);
      s2[i] = fma2(qx.y, kx.y, s2[i]);
    }
  }
  float x[RW];
  bool up = false;
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    float a, b;
    unpack2(s2[i], a, b);
    x[i] = j0 + lane < r.lim[i] ? (a + b) * scale_log2 : -INFINITY;
    up |= x[i] > r.m[i] + kSlackLog2;
  }
  if (__any_sync(0xffffffffu, up)) {
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const float mt = fmaxf(r.m[i], warp_max(x[i]));
      const float f = mt == -INFINITY ? 1.0f : exp2f(r.m[i] - mt);
      r.m[i] = mt;
      r.l[i] *= f;
#pragma unroll
      for (int k = 0; k < NI / 2; ++k) r.o[i][k] = mul2(r.o[i][k], pack2(f, f));
    }
  }
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    x[i] = exp2f(x[i] - (r.m[i] == -INFINITY ? 0.0f : r.m[i]));
    r.l[i] += x[i];
  }
  constexpr int kKeys = RW <= 4 ? kTN : kProbPairs / RW;  // at a time
#pragma unroll 1
  for (int h = 0; h < kTN; h += kKeys) {
    if (kKeys == kTN || (lane >= h && lane < h + kKeys)) {
#pragma unroll
      for (int i = 0; i < RW; ++i) sp[(lane - h) * RW + i] = pack2(x[i], x[i]);
    }
    __syncwarp();
    const float* vh = sv + h * ld + 2 * lane;
#pragma unroll 8
    for (int j = 0; j < kKeys; ++j) {
      f32x2 e[RW];
      if (RW == 1) {
        e[0] = sp[j];
      } else {
#pragma unroll
        for (int i = 0; i + 1 < RW; i += 2) {
          const ulonglong2 q = *(const ulonglong2*)&sp[j * RW + i];
          e[i] = q.x, e[i + 1] = q.y;
        }
      }
#pragma unroll
      for (int k = 0; k < NI / 2; ++k) {
        const f32x2 v = *(const f32x2*)(vh + j * ld + 64 * k);
#pragma unroll
        for (int i = 0; i < RW; ++i) r.o[i][k] = fma2(e[i], v, r.o[i][k]);
      }
    }
    __syncwarp();
  }
}

// Keys [from, to) of a tile, those that some rows of the block see and some do not
// (positions of the chunk itself): 0 times a V that is not finite would reach the
// latter, so such a V is cleared and the rows that do see it become NaN at the end.
template <int NI>
__device__ __forceinline__ void hide_bad_v(float* sv, int j0, int from, int to, int* bad_from) {
  constexpr int ld = NI * 32 + 4;
  const int lane = threadIdx.x & 31;
  for (int j = from + (int)(threadIdx.x >> 5); j < to; j += kWarps) {
    float* v = sv + j * ld;
    bool bad = false;
#pragma unroll
    for (int d = 0; d < NI; ++d) bad |= (__float_as_uint(v[d * 32 + lane]) & 0x7f800000u) == 0x7f800000u;
    if (!__any_sync(0xffffffffu, bad)) continue;
#pragma unroll
    for (int d = 0; d < NI; ++d) v[d * 32 + lane] = 0.0f;
    if (lane == 0) atomicMin(bad_from, j0 + j);
  }
}

__device__ __forceinline__ void copy16(float* dst, const float* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}

// The rows of an item are spread over the warps, one, two, four or eight a warp;
// a tile of K and V is on its way to shared memory while the one before is
// worked on, and the pages of the one after are looked up.
// FP4: codes become floats as they are put into shared memory, which then holds what it does for
// an fp32 cache; for many rows of fp32 queries, whose precision the tensor cores do not have, or of wide heads.
// Codes wait in registers while the tile before is worked on (loaded and converted at once, chunks
// of up to 17 tokens, four heads of 256, of 16 requests of 2000 .. 3900 positions: 1552 us for 1271).
template <typename T, int NI, bool FP4>  // NI = ceil(D / 32), 2, 4 or 8
__global__ void __launch_bounds__(kThreads, NI <= 4 ? 2 : 1)
attention_simt_kernel(const AttnParams p, const Divider by_page, const bool vec) {
  extern __shared__ float4 smem4[];
  __shared__ AttnStart<kTN> st;
  // Of the item: keys that all rows of the block see, the first tile with others,
  // and the first of those whose V is not finite (hide_bad_v).  Not in registers:
  // there they cost what fp32 decoding of 128 requests shows, 290 us for 286.
  __shared__ int flags, all_see, t_hidden, bad_from;
  __shared__ __align__(16) f32x2 sp[kWarps][kProbPairs];  // probabilities of a warp's rows
  constexpr int ld = NI * 32 + 4;
  constexpr int kPer = NI * 8;               // threads a row, four columns each
  constexpr int kPass = kThreads / kPer;     // rows a pass of the CTA; NI passes a tile
  const int D = p.a.c.head_dim;
  float* sq = (float*)smem4;       // [kMR][ld]
  float* skv = sq + kMR * ld;      // [2] K, V: [kTN][ld] each
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lr = threadIdx.x / kPer, lc = (threadIdx.x % kPer) * 4;  // first row and column it loads
  const int S = p.a.c.page_size, G = p.a.G;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) flags = 0;
  __syncthreads();
  wait_for_previous();
  attn_plan<kTN>(p, &st, &flags);
  AttnWalk<kTN> w = st.walk;
  if (threadIdx.x == 0) attn_write_cut(p, st);

  for (; !w.done(); w.next(p, &flags)) {
    const int rows = w.block_rows(p), row0 = w.m * kMR, t1 = w.last_tile();
    const int rw = rows <= kWarps ? 1 : rows <= 2 * kWarps ? 2 : rows <= 4 * kWarps ? 4 : 8;
    const int32_t* table = p.a.a.page_table + (size_t)w.r * p.a.a.max_pages;
    int page[NI];
    auto look_up = [&](int t) {  // the pages of tile t's rows; -1: past the item's keys
#pragma unroll
      for (int u = 0; u < NI; ++u) {
        const int j = t * kTN + lr + u * kPass;
        page[u] = t < t1 && j < w.end ? table[by_page(j)] : -1;
      }
    };
    auto load = [&](int t) {  // into buffer t & 1; positions at or past `end` become zeros
      float* sk = skv + (t & 1) * 2 * kTN * ld + lr * ld + lc;
#pragma unroll
      for (int u = 0; u < NI; ++u) {
        const int j = t * kTN + lr + u * kPass;
        float* k = sk + u * kPass * ld;
        float* v = k + kTN * ld;
        if (t < t1 && j < w.end) {
          int pg = page[u];
          if (pg < 0 || pg >= p.a.c.n_pages) {
            flag_status(&flags, DSPARK_DEV_BAD_INPUT);
            pg = pg < 0 ? 0 : p.a.c.n_pages - 1;
          }
          const long long at = pg * p.a.c.page_stride + (j - by_page(j) * S) * p.a.c.token_stride +
                               w.h * p.a.c.head_stride;
          if (std::is_same<T, float>::value && vec && lc < D) {
            copy16(k, (const float*)p.a.c.k + at + lc);
            copy16(v, (const float*)p.a.c.v + at + lc);
          } else {
            *(float4*)k = load4((const T*)p.a.c.k + at, lc, D, vec);
            *(float4*)v = load4((const T*)p.a.c.v + at, lc, D, vec);
          }
        } else {
          *(float4*)k = *(float4*)v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
      }
    };
    // FP4: tile t's codes and scales to registers, and as floats from there into its buffer.
    uint32_t codes[FP4 ? NI : 1], scales[FP4 ? NI : 1];  // of K, and V's above
    auto fetch = [&](int t) {
#pragma unroll
      for (int u = 0; u < NI; ++u) {
        const int j = t * kTN + lr + u * kPass;
        codes[u] = scales[u] = 0u;
        if (t >= t1 || j >= w.end || lc >= D) continue;
        int pg = page[u];
        if (pg < 0 || pg >= p.a.c.n_pages) {
          flag_status(&flags, DSPARK_DEV_BAD_INPUT);
          pg = pg < 0 ? 0 : p.a.c.n_pages - 1;
        }
        const int slot = j - by_page(j) * S;
        const long long at = pg * p.a.c.page_stride + w.h * p.a.c.head_stride;
        const long long c = at + fp4_codes_at(slot, D) + lc / 2, s = at + fp4_scales_at(slot, D) + lc / 16;
        const uint8_t *kb = (const uint8_t*)p.a.c.k, *vb = (const uint8_t*)p.a.c.v;
        codes[u] = *(const uint16_t*)(kb + c) | (uint32_t)*(const uint16_t*)(vb + c) << 16;
        scales[u] = kb[s] | (uint32_t)vb[s] << 8;
      }
    };
    auto put = [&](int t) {
      float* sk = skv + (t & 1) * 2 * kTN * ld + lr * ld + lc;
#pragma unroll
      for (int u = 0; u < NI; ++u) {
        float* k = sk + u * kPass * ld;
        *(float4*)k = values4_fp4(codes[u] & 0xffffu, scales[u], 1.0f);
        *(float4*)(k + kTN * ld) = values4_fp4(codes[u] >> 16, scales[u] >> 8, p.a.v_factor);
      }
    };
    __syncthreads();  // (the item before is done with both buffers and bad_from)
    if (threadIdx.x == 0) {
      const int a = w.q.L - w.q.n + row0 / G + 1;
      all_see = a;
      t_hidden = a < w.end ? max(a, 0) / kTN : 0x7fffffff;
      bad_from = 0x7fffffff;
    }
    look_up(w.first_tile());
    if constexpr (FP4)
      fetch(w.first_tile());
    else
      load(w.first_tile());
    look_up(w.first_tile() + 1);
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
    Rows<NI / 2> r;
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
      const int a = warp * rw + i;
      r.m[i] = -INFINITY, r.l[i] = 0.0f;
      r.lim[i] = i < rw && a < rows ? w.q.L - w.q.n + (row0 + a) / G + 1 : 0;
#pragma unroll
      for (int k = 0; k < NI / 2; ++k) r.o[i][k] = 0ull;
    }
    for (int t = w.first_tile(); t < t1; ++t) {
      // (all are past tile t - 1 behind the barrier, which was in the buffer of t + 1)
      if constexpr (FP4) {
        put(t);
        __syncthreads();
        fetch(t + 1);
      } else {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        load(t + 1);
      }
      look_up(t + 2);
      if (t >= t_hidden) {
        hide_bad_v<NI>(skv + ((t & 1) * 2 + 1) * kTN * ld, t * kTN, max(all_see - t * kTN, 0),
                       min(w.end - t * kTN, kTN), &bad_from);
        __syncthreads();
      }
      if (warp * rw < rows) {
        const float* q = sq + warp * rw * ld;
        const float* sk = skv + (t & 1) * 2 * kTN * ld;
        const float* sv = sk + kTN * ld;
        if (rw == 1)
          simt_tile<NI, 1>(r, q, sk, sv, sp[warp], t * kTN, p.scale_log2);
        else if (rw == 2)
          simt_tile<NI, 2>(r, q, sk, sv, sp[warp], t * kTN, p.scale_log2);
        else if (rw == 4)
          simt_tile<NI, 4>(r, q, sk, sv, sp[warp], t * kTN, p.scale_log2);
        else
          simt_tile<NI, 8>(r, q, sk, sv, sp[warp], t * kTN, p.scale_log2);
      }
    }
    const int slot = attn_slot(w);
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
      const int a = warp * rw + i;
      if (i >= rw || a >= rows) continue;
      const float sum = warp_sum(r.l[i]), l = r.lim[i] > bad_from ? __int_as_float(0x7fc00000) : sum;
      const int tok = (row0 + a) / G, g = (row0 + a) - tok * G;
      const size_t out = (size_t)(w.q.q0 + tok) * p.a.Hq + w.h * G + g;
      const size_t part = ((size_t)blockIdx.x * 2 + slot) * kMR + a;
      const float inv = slot >= 0 ? 1.0f : l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
#pragma unroll
      for (int k = 0; k < NI / 2; ++k) {
        float y[2];
        unpack2(r.o[i][k], y[0], y[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = 2 * lane + 64 * k + e;
          if (d >= D) continue;
          if (slot >= 0)
            p.part[part * D + d] = y[e];
          else if constexpr (std::is_same<T, float>::value)
            ((float*)p.a.out)[out * D + d] = y[e] * inv;
          else
            ((__nv_bfloat16*)p.a.out)[out * D + d] = __float2bfloat16(y[e] * inv);
        }
      }
      if (lane == 0) {
        if (slot >= 0)
          p.stats[part] = make_float2(r.m[i], l);
        else
          p.a.lse[out] = l == 0.0f ? -INFINITY : r.m[i] * kLn2 + logf(l);
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_previous();  // everything below reads what the attention kernel wrote
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

constexpr int kSimtCtas = 304;  // two an SM
static_assert(kSimtCtas <= kAttnMaxCtas, "");

template <typename T, int NI, bool FP4>
cudaError_t launch_simt(const AttnParams& p, cudaStream_t s) {
  const int smem = (kMR + 4 * kTN) * (NI * 32 + 4) * (int)sizeof(float);
  const cudaError_t attr = once_per_device([=] { return allow_smem(attention_simt_kernel<T, NI, FP4>, smem); });
  if (attr != cudaSuccess) return attr;
  // Rows that are whole 16-byte (fp32) or 8-byte (bf16) vectors load as such.
  const CacheView& c = p.a.c;
  const bool vec = c.head_dim % 4 == 0 && c.page_stride % 4 == 0 && c.token_stride % 4 == 0 &&
                   c.head_stride % 4 == 0 &&
                   (((uintptr_t)c.k | (uintptr_t)c.v) & (4 * sizeof(T) - 1)) == 0;
  cudaLaunchAttribute attr_pdl;
  const cudaLaunchConfig_t cfg = overlapped_launch(dim3(kSimtCtas), kThreads, smem, s, &attr_pdl);
  return cudaLaunchKernelEx(&cfg, attention_simt_kernel<T, NI, FP4>, p, Divider((unsigned)c.page_size), vec);
}

template <typename T, bool FP4>
cudaError_t launch_simt_dim(const AttnParams& p, cudaStream_t s) {
  const int ni = (p.a.c.head_dim + 31) / 32;
  if constexpr (!FP4 || sizeof(T) == 4) {  // (bf16 queries over a 4-bit cache: only wide heads come here)
    if (ni <= 2) return launch_simt<T, 2, FP4>(p, s);
    if (ni <= 4) return launch_simt<T, 4, FP4>(p, s);
  }
  return launch_simt<T, 8, FP4>(p, s);
}

}  // namespace

cudaError_t launch_attn_combine(const AttnParams& p, int MR, int ctas, cudaStream_t s) {
  const long long rows = attn_likely_rows(p.a);
  const dim3 grid(ctas > 1 ? ctas - 1 : 1, (unsigned)((rows < MR ? rows : MR) + 7) / 8);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = overlapped_launch(grid, 256, 0, s, &attr);
  return p.a.dtype == DSPARK_BF16 ? launch_combine<__nv_bfloat16>(cfg, p, MR, ctas)
                                  : launch_combine<float>(cfg, p, MR, ctas);
}

size_t attention_workspace_bytes(int dtype, int head_dim) {
  const size_t simt = attn_workspace_layout(kMR, head_dim, kSimtCtas).total;
  if (dtype != DSPARK_BF16 || head_dim > 128) return simt;
  const size_t tc = attention_tc_workspace_bytes(head_dim);
  return tc > simt ? tc : simt;
}

size_t attention_fp4_workspace_bytes(int dtype, int head_dim) {
  if (dtype != DSPARK_BF16 || head_dim > 128) {
    const size_t few = attention_fp4_simt_workspace_bytes(head_dim);
    const size_t many = attn_workspace_layout(kMR, head_dim, kSimtCtas).total;
    return few > many ? few : many;
  }
  const size_t rows = attention_fp4_rows_workspace_bytes(head_dim), tc = attention_tc_workspace_bytes(head_dim);
  return tc > rows ? tc : rows;
}

cudaError_t launch_paged_attention(const AttnArgs& a, char* ws, cudaStream_t s) {
  if (a.fp4 && attention_fp4_few_rows(a)) return launch_attention_fp4_rows(a, ws, s);
  if (attention_tc_fp4_supported(a)) return launch_attention_tc_fp4(a, ws, s);
  if (attention_fp4_simt_few_rows(a)) return launch_attention_fp4_simt(a, ws, s);
  if (!a.fp4 && attention_tc_supported(a)) return launch_attention_tc(a, ws, s);
  const AttnWorkspace w = attn_workspace_layout(kMR, a.c.head_dim, kSimtCtas);
  AttnParams p{a, (int*)ws, (int*)(ws + w.flags), (CutItem*)(ws + w.cuts),
               (float2*)(ws + w.stats), (float*)(ws + w.out), a.scale * 1.4426950408889634f,
               attn_item_units(a), kMR};
  const bool bf = a.dtype == DSPARK_BF16;
  const cudaError_t e = a.fp4 ? bf ? launch_simt_dim<__nv_bfloat16, true>(p, s) : launch_simt_dim<float, true>(p, s)
                        : bf  ? launch_simt_dim<__nv_bfloat16, false>(p, s)
                              : launch_simt_dim<float, false>(p, s);
  if (e != cudaSuccess) return e;
  return launch_attn_combine(p, kMR, kSimtCtas, s);
}

}  // namespace dspark
