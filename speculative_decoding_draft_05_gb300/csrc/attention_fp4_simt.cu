// attention_fp4_simt.cu -- attention of few rows a K/V head over the 4-bit paged cache on CUDA cores: fp32
// queries, whose precision the tensor cores do not have, and heads wider than 128.
//
// A warp takes a block of 16 keys at a time and all rows of the item.  Scores: a lane has half of a
// key's row, decodes it and multiplies it with every row of Q (from shared memory); sums
// and probabilities are fp32.  Output: a lane has pairs of columns, decodes them key by key and adds
// them with the probabilities, which pass through shared memory as pairs, the operands of packed products.
// So a code is decoded once for all rows, all warps work whatever rows there are, and nothing is kept as floats.
// (The kernel for more rows, in attention.cu, puts tiles of floats in shared memory and spreads the rows over
// the warps: with one to four rows most of them have none.)
//
// As in the kernel for bf16 (attention_fp4.cu), a CTA walks its share in tiles of 128 keys, a warp brings its own
// blocks by asynchronous copies into a ring of its own, and a piece's eight partial results meet in shared memory.
//
// What bounds it: the issue of instructions (57 % of the slots; 1365 for a block of 16 keys of 128 and four
// rows), and what waits for shared memory.  Decoding in fp32, 16 requests of 2000 .. 3900 positions, 32 query heads over
// 8 of 128: 52 us, 59 MB; bf16 heads of 256: 119 us.
#include <type_traits>

#include "attention.cuh"
#include "f32x2.cuh"
#include "fp4.cuh"
#include "per_device.h"

namespace dspark {

namespace {

constexpr int kWarps = 8;
constexpr int kTN = kWarps * kFp4Block;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxRows = 8;  // of an item
constexpr float kSlackLog2 = 8.0f;
constexpr float kLn2 = 0.6931471805599453f;

template <int NI, int RW>
struct Shape {
  static constexpr int kPerSm = NI <= 4 ? 2 : 1;
  static constexpr int kCtas = 152 * kPerSm;
  static constexpr int kD = 32 * NI;                  // or fewer columns
  static constexpr int kStage = 2 * 9 * kD;           // K, V of a warp's 16 keys
  static constexpr int kRow = kD + 4;                 // floats of a row of partial results
  static constexpr int kMerge = kWarps * RW * kRow * 4;
  static constexpr int kQRow = kD + 8;                // two halves, four floats apart in their banks
  static constexpr int kQ = RW * kQRow * 4;
  static constexpr int kProb = kWarps * kFp4Block * RW * 8;
  static constexpr int kRoom = 232448 / kPerSm - kMerge - kQ - kProb - 4096;
  static constexpr int kFit = kRoom / (kWarps * kStage);
  static constexpr int kStages = kFit >= 6 ? 6 : kFit;
  static constexpr int kBytes = kMerge + kQ + kProb + kStages * kWarps * kStage;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {  // all but the last N groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct SimtParams {
  explicit SimtParams(const AttnArgs& a) : p{a}, by_page((unsigned)a.c.page_size) {}
  AttnParams p;
  Divider by_page;
};

// (Of 128 registers; items of eight rows spill 52 bytes with heads of 128, 20 with 64.)
template <typename T, int NI, int RW>  // head_dim up to 32 NI; RW rows an item
__global__ void __launch_bounds__(kThreads, NI <= 4 ? 2 : 1)
attention_fp4_simt_kernel(const __grid_constant__ SimtParams fp) {
  using Sh = Shape<NI, RW>;
  constexpr int NP = NI / 2;               // pairs of columns a lane
  constexpr int kCols = NI >= 4 ? 4 : 2;   // of which so many columns follow one another
  constexpr int kRuns = NI / kCols;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ AttnStart<kTN> st;
  __shared__ float2 stats[kWarps][RW];
  __shared__ int flags, bad_from;
  const AttnParams& p = fp.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, D = p.a.c.head_dim, S = p.a.c.page_size;
  const int block = fp4_block_bytes(D);
  float* buf = (float*)smem;
  float* sq = (float*)(smem + Sh::kMerge);
  f32x2* sp = (f32x2*)(smem + Sh::kMerge + Sh::kQ) + warp * kFp4Block * RW;  // the warp's [16][RW]
  uint8_t* ring = smem + Sh::kMerge + Sh::kQ + Sh::kProb + warp * Sh::kStages * Sh::kStage;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) flags = 0;
  __syncthreads();
  wait_for_previous();
  attn_plan<kTN>(p, &st, &flags);
  AttnWalk<kTN> w = st.walk;
  if (threadIdx.x == 0) attn_write_cut(p, st);

  // Loads: groups of copies, the warp's block of a tile each.  The page of a tile is looked up one tile ahead.
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  const int chunks = block / 16;  // of 16 bytes: of K, and of V
  uint32_t stage = 0;
  int page = 0;
  auto look_up = [&](int t) {
    const int key = t * kTN + warp * kFp4Block;
    page = t < w.last_tile() && key < w.end
               ? p.a.a.page_table[(size_t)w.r * p.a.a.max_pages + fp.by_page(key)] : 0;
  };
  auto load = [&](int t) {
    const int key = t * kTN + warp * kFp4Block;
    int pg = page;
    look_up(t + 1);
    if (t < w.last_tile() && key < w.end) {
      if (pg < 0 || pg >= p.a.c.n_pages) {
        if (lane == 0) flag_status(&flags, DSPARK_DEV_BAD_INPUT);
        pg = pg < 0 ? 0 : p.a.c.n_pages - 1;
      }
      const long long at = pg * p.a.c.page_stride + w.h * p.a.c.head_stride +
                           (long long)((key - fp.by_page(key) * S) / kFp4Block) * block;
      const uint8_t *k = (const uint8_t*)p.a.c.k + at, *v = (const uint8_t*)p.a.c.v + at;
      const uint32_t dst = ring_at + stage * Sh::kStage;
      for (int i = lane; i < 2 * chunks; i += 32)
        copy16(dst + i * 16, i < chunks ? k + i * 16 : v + (i - chunks) * 16);
    }
    copy_commit();
    stage = stage + 1 == Sh::kStages ? 0 : stage + 1;
  };

  const int key_l = lane & 15, half = lane >> 4;
  const int G = p.a.G, words = D / 16;  // of half a row
  for (; !w.done(); w.next(p, &flags)) {
    const int rows = w.block_rows(p), row0 = w.m * p.mr, t1 = w.last_tile();
    const int n0 = w.q.L - w.q.n + 1;  // keys that the chunk's first token sees
    const int all_see = n0 + row0 / G;
    stage = 0;
    look_up(w.first_tile());
#pragma unroll 1
    for (int i = 0; i < Sh::kStages; ++i) load(w.first_tile() + i);
    __syncthreads();  // (the piece before is merged)
    if (threadIdx.x == 0) bad_from = 0x7fffffff;
    for (int i = threadIdx.x; i < RW * D; i += kThreads) {
      const int a = i / D, d = i - a * D;
      float x = 0.0f;
      if (a < rows) {
        const int tok = (row0 + a) / G, g = (row0 + a) - tok * G;
        x = to_f32(((const T*)p.a.q)[(long long)(w.q.q0 + tok) * p.a.q_token_stride +
                                     (long long)(w.h * G + g) * p.a.q_head_stride + d]);
      }
      sq[a * Sh::kQRow + d + (d >= D / 2 ? 4 : 0)] = x;
    }
    __syncthreads();
    f32x2 o[RW][NP];
    float m[RW], l[RW];
    int lim[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      m[i] = -INFINITY, l[i] = 0.0f;
      lim[i] = i < rows ? n0 + (row0 + i) / G : 0;
#pragma unroll
      for (int k = 0; k < NP; ++k) o[i][k] = 0ull;
    }
#pragma unroll 1
    for (int t = w.first_tile(); t < t1; ++t) {
      copy_wait<Sh::kStages - 1>();
      __syncwarp();
      const int k0 = t * kTN + warp * kFp4Block;
      if (k0 < w.end) {
        const uint8_t* kb = ring + stage * Sh::kStage;
        const uint8_t* vb = kb + block;
        f32x2 s2[RW] = {};
        {
          const uint8_t* codes = kb + key_l * (D / 2) + half * (D / 4);
          const uint8_t* scales = kb + 8 * D + key_l * (D / 16) + half * (D / 32);
          const float* q = sq + half * (D / 2 + 4);
#pragma unroll 4
          for (int u = 0; u < words; u += 2) {  // 16 elements, of one scale
            const uint2 c = *(const uint2*)(codes + u * 4);
            const uint32_t f = e4m3x2_to_half(scales[u / 2] * 0x101u);
            uint32_t h[8];
            fp4x8_to_half(c.x, h);
            fp4x8_to_half(c.y, h + 4);
            f32x2 x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t y = hmul2(h[e], f);  // (exact)
              x[e] = pack2(half_lo(y), half_hi(y));
            }
#pragma unroll
            for (int i = 0; i < RW; ++i) {
              const ulonglong2* qr = (const ulonglong2*)(q + i * Sh::kQRow + u * 8);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const ulonglong2 y = qr[e];
                s2[i] = fma2(y.x, x[2 * e], s2[i]);
                s2[i] = fma2(y.y, x[2 * e + 1], s2[i]);
              }
            }
          }
        }
        float x[RW];
        bool up = false;
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          float a, b;
          unpack2(s2[i], a, b);
          a += b;
          a += __shfl_xor_sync(0xffffffffu, a, 16);
          x[i] = k0 + key_l < lim[i] ? a * p.scale_log2 : -INFINITY;
          up |= x[i] > m[i] + kSlackLog2;
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int i = 0; i < RW; ++i) {
            float mt = x[i];
#pragma unroll
            for (int d = 1; d < 16; d *= 2) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, d));
            mt = fmaxf(mt, m[i]);
            const float f = mt == -INFINITY ? 1.0f : exp2f(m[i] - mt);
            m[i] = mt;
            l[i] *= f;
#pragma unroll
            for (int k = 0; k < NP; ++k) o[i][k] = mul2(o[i][k], pack2(f, f));
          }
        }
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          x[i] = exp2f(x[i] - (m[i] == -INFINITY ? 0.0f : m[i]));
          l[i] += x[i];
          if (half == 0) sp[key_l * RW + i] = pack2(x[i], x[i]);
        }
        __syncwarp();
        auto add = [&](int j, auto masked) {
          f32x2 v[NP];
#pragma unroll
          for (int k = 0; k < kRuns; ++k) {
            const int d = kCols * (lane + 32 * k);
            v[kCols / 2 * k] = v[kCols / 2 * k + kCols / 2 - 1] = 0ull;
            if (d < D) {
              uint32_t sc = vb[8 * D + j * (D / 16) + (d >> 4)];
              if (masked.value && k0 + j >= all_see) {
                // Past the item's end: any bytes.  Where some rows of the block do not see the key, a scale
                // that is NaN is hidden from them, and makes the others NaN below.
                if (k0 + j >= w.end) {
                  sc = 0u;
                } else if ((sc & 0x7fu) == 0x7fu) {
                  atomicMin(&bad_from, k0 + j);
                  sc = 0u;
                }
              }
              const uint8_t* at = vb + j * (D / 2) + (d >> 1);
              uint32_t h[2];
              fp4x4_to_half(kCols == 4 ? *(const uint16_t*)at : *at, h);
              const uint32_t f = e4m3x2_to_half(sc * 0x101u);
#pragma unroll
              for (int e = 0; e < kCols / 2; ++e) {
                const uint32_t y = hmul2(h[e], f);
                v[kCols / 2 * k + e] = pack2(half_lo(y), half_hi(y));
              }
            }
          }
#pragma unroll
          for (int i = 0; i < RW; ++i) {
            const f32x2 e = sp[j * RW + i];
#pragma unroll
            for (int k = 0; k < NP; ++k) o[i][k] = fma2(e, v[k], o[i][k]);
          }
        };
        if (k0 + kFp4Block > all_see) {
#pragma unroll 1
          for (int j = 0; j < kFp4Block; ++j) add(j, std::true_type{});
        } else {
#pragma unroll 4
          for (int j = 0; j < kFp4Block; ++j) add(j, std::false_type{});
        }
      }
      __syncwarp();  // (the stage and the probabilities are read)
      load(t + Sh::kStages);
    }
    copy_wait<0>();

    // The eight warps' results.
#pragma unroll
    for (int i = 0; i < RW; ++i) {
#pragma unroll
      for (int d = 1; d < 16; d *= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      if (lane == 0) stats[warp][i] = make_float2(m[i], l[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) top = fmaxf(top, stats[x][i].x);
      const float f = m[i] == -INFINITY ? 0.0f : exp2f(m[i] - top);
#pragma unroll
      for (int k = 0; k < NP; ++k)
        *(f32x2*)(buf + (warp * RW + i) * Sh::kRow + kCols * (lane + 32 * (k / (kCols / 2))) + 2 * (k % (kCols / 2))) =
            mul2(o[i][k], pack2(f, f));
    }
    __syncthreads();
    const int where = attn_slot(w);
    for (int i = threadIdx.x; i < RW * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      if (r >= rows) break;
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float4 v = *(const float4*)(buf + (x * RW + r) * Sh::kRow + d);
        y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
        top = fmaxf(top, stats[x][r].x);
      }
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float2 q = stats[x][r];
        sum += q.x == -INFINITY ? q.y : q.y * exp2f(q.x - top);  // (q.y: 0, or NaN)
      }
      const int tok = (row0 + r) / G, g = (row0 + r) - tok * G;
      if (n0 + tok > bad_from) sum = __int_as_float(0x7fc00000);
      if (where < 0) {
        const size_t out = (size_t)(w.q.q0 + tok) * p.a.Hq + w.h * G + g;
        const float inv = sum > 0.0f ? p.a.v_factor / sum : sum == 0.0f ? 0.0f : sum;
        if constexpr (sizeof(T) == 4) {
          *(float4*)((float*)p.a.out + out * D + d) = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
        } else {
          const __nv_bfloat162 a = __floats2bfloat162_rn(y.x * inv, y.y * inv);
          const __nv_bfloat162 b = __floats2bfloat162_rn(y.z * inv, y.w * inv);
          *(uint2*)((__nv_bfloat16*)p.a.out + out * D + d) = make_uint2(*(const uint32_t*)&a, *(const uint32_t*)&b);
        }
        if (d == 0) p.a.lse[out] = sum == 0.0f ? -INFINITY : top * kLn2 + logf(sum);
      } else {
        const size_t part = ((size_t)blockIdx.x * 2 + where) * kMaxRows + r;
        const float f = p.a.v_factor;
        *(float4*)(p.part + part * D + d) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
        if (d == 0) p.stats[part] = make_float2(top, sum);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) p.flags[blockIdx.x] = flags;
}

template <typename T, int NI, int RW>
cudaError_t launch(SimtParams fp, char* ws, cudaStream_t s) {
  using Sh = Shape<NI, RW>;
  static_assert(Sh::kCtas <= kAttnMaxCtas && Sh::kStages >= 2 && Sh::kPerSm * (Sh::kBytes + 4096) <= 233472, "");
  const AttnWorkspace w = attn_workspace_layout(kMaxRows, fp.p.a.c.head_dim, Sh::kCtas);
  AttnParams& p = fp.p;
  p.status = (int*)ws;
  p.flags = (int*)(ws + w.flags);
  p.cuts = (CutItem*)(ws + w.cuts);
  p.stats = (float2*)(ws + w.stats);
  p.part = (float*)(ws + w.out);
  p.mr = RW;
  const cudaError_t attr = once_per_device([] { return allow_smem(attention_fp4_simt_kernel<T, NI, RW>, Sh::kBytes); });
  if (attr != cudaSuccess) return attr;
  cudaLaunchAttribute attr_pdl;
  const cudaLaunchConfig_t cfg = overlapped_launch(dim3(Sh::kCtas), kThreads, Sh::kBytes, s, &attr_pdl);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attention_fp4_simt_kernel<T, NI, RW>, fp);
  return e != cudaSuccess ? e : launch_attn_combine(p, kMaxRows, Sh::kCtas, s);
}

template <typename T, int NI>
cudaError_t launch_rows(const SimtParams& fp, char* ws, cudaStream_t s) {
  const long long rows = attention_fp4_rows(fp.p.a);
  if (rows <= 1) return launch<T, NI, 1>(fp, ws, s);
  return rows <= 4 ? launch<T, NI, 4>(fp, ws, s) : launch<T, NI, 8>(fp, ws, s);
}

}  // namespace

// Few rows here, in items of eight, more in attention.cu, in items of 64: chunks of one length fill those, uneven
// ones leave much of them empty.  So the rule has a bound for either, of rows as attention_fp4_rows counts them, for
// heads up to 64 and for wider ones.  Measured (us), here / there, 16 requests of 1000 .. 2000 positions, four query
// heads of each of eight K/V heads:
//   chunks alike, rows    8          16         24         32         40         48         64
//   fp32, heads of 64     36 / 54    64 / 67    85 / 79    107 / 92   128 / 108  148 / 126  191 / 146
//   fp32, heads of 128    48 / 92    86 / 110   116 / 133  148 / 147  179 / 191  209 / 218  273 / 236
//   bf16, heads of 256    90 / 238   174 / 278  244 / 314  320 / 348  393 / 473  468 / 508  618 / 589
// and 64 requests of 200 .. 3000 positions:
//   fp32, heads of 64     109 / 211  223 / 261  320 / 304  418 / 353             615 / 494  810 / 589
//   fp32, heads of 128    158 / 457  315 / 521  456 / 591  603 / 668             878 / 955  1166 / 1032
// Uneven chunks, 16 requests as above, by the count (the mean and a third):
//   fp32, heads of 64     15: 51 / 72      48: 123 / 129    64: 154 / 163    82: 196 / 183    98: 218 / 218
//   fp32, heads of 128    20: 90 / 129     43: 160 / 214    80: 260 / 304    134: 422 / 448   175: 528 / 550
//   bf16, heads of 256    20: 178 / 326    56: 411 / 627    98: 721 / 825    140: 1001 / 1120
// and 64 requests:
//   fp32, heads of 64     40: 392 / 527    74: 740 / 786    82: 798 / 816    114: 1127 / 1058
//   fp32, heads of 128    45: 629 / 989    84: 1149 / 1432  145: 1859 / 2047 153: 2155 / 2332
bool attention_fp4_simt_few_rows(const AttnArgs& a) {
  if (!a.fp4 || (a.dtype == DSPARK_BF16 && a.c.head_dim <= 128) || a.a.n_tokens == 0) return false;
  const bool narrow = a.c.head_dim <= 64;
  const int most = attention_even_chunks(a) ? (narrow ? 20 : 48) : (narrow ? 80 : 160);
  return attention_fp4_rows(a) <= most;
}

size_t attention_fp4_simt_workspace_bytes(int head_dim) {
  return attn_workspace_layout(kMaxRows, head_dim, kAttnMaxCtas).total;
}

cudaError_t launch_attention_fp4_simt(const AttnArgs& a, char* ws, cudaStream_t s) {
  SimtParams fp(a);
  fp.p.scale_log2 = a.scale * 1.4426950408889634f;
  fp.p.item_units = 1;
  if (a.dtype == DSPARK_BF16) return launch_rows<__nv_bfloat16, 8>(fp, ws, s);
  if (a.c.head_dim <= 64) return launch_rows<float, 2>(fp, ws, s);
  if (a.c.head_dim <= 128) return launch_rows<float, 4>(fp, ws, s);
  return launch_rows<float, 8>(fp, ws, s);
}

}  // namespace dspark
