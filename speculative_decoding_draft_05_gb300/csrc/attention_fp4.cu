// attention_fp4.cu -- attention of few rows a K/V head over the 4-bit paged cache
// (bf16 queries, head_dim up to 128): decoding, and short chunks.
//
// Codes times scales are exact in fp16, so both products are of fp16 operands
// with fp32 sums, and codes become operands in registers: shared memory holds
// what the cache holds, 9 bytes for 16 elements, and is read once.
//   S^T = K Q^T: the 16 keys of a block are the rows of the product, 8 query
//     rows its columns.  The order of head_dim along the sum is free, so a
//     thread takes a contiguous quarter of a key's codes, and Q is laid out alike.
//   O^T = V^T P^T: S^T's fragments, transposed in registers, are its second
//     operand.  The order of V's columns over the rows of the product is free too:
//     a thread takes a contiguous eighth of a key's codes, and pairs of
//     keys are interleaved code by code before the conversion.
// Queries are multiplied by a power of two a row that brings the largest into fp16's
// upper range, which the scores' factor takes back: exact but for elements below
// 2^-28 of the row's largest.
//
// Softmax: p = 2^{s - m} with m 8 below the maximum of the first block that the row
// sees, moved (O and l rescaled) only when a score lies more than 15 above it: p < 2^15
// fits fp16, and what underflows is below 2^-32 of the largest.  l sums p before rounding.
//
// A CTA walks its share in tiles of 128 keys, a block of 16 keys a warp.  A warp brings its
// own blocks (9 head_dim bytes each, K's and V's) by asynchronous copies into a ring of its
// own, so that within a piece no warp waits for another.  (A warp that brought all of them by bulk
// copies took 150 cycles to issue each, and was the bottleneck: 173 us for decoding of 64.)
// A piece's eight partial results meet in shared memory, while the next piece's first
// tiles are on their way.
//
// What bounds it: with much to read the issue of instructions, 416 a block of 16 keys of 128 and
// warp, most of them conversions, scaling and products (decoding, 64 requests of 1000 .. 16384
// positions, 64 query heads over 8, 607 MB: 151 us, 4.0 TB/s, 63 % of the issue slots); with
// little, latency (16 requests of 200 .. 2048 positions, 24 MB: 18.7 us with the combine).
#include <cuda_fp16.h>

#include "attention.cuh"
#include "fp4.cuh"
#include "per_device.h"

namespace dspark {

namespace {

constexpr int kWarps = 8;
constexpr int kTN = kWarps * kFp4Block;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxRows = 16;  // of an item
constexpr float kRise = 15.0f, kBelow = 8.0f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D, int NB>
struct Shape {
  static constexpr int kCtas = 152 * 2;               // two an SM
  static constexpr int kBlock = 9 * D;
  static constexpr int kStage = 2 * kBlock;           // K, V of a warp's 16 keys
  static constexpr int kRow = D + 4;                  // floats of a row of partial results
  static constexpr int kMerge = kWarps * 8 * kRow * 4;
  static constexpr int kQ = NB > 1 ? NB * D / 16 * 32 * 8 : 0;  // Q's fragments, where registers have no room
  static constexpr int kRoom = 232448 / 2 - 2 * kQ - 4096;
  static constexpr int kFit = (kRoom - kMerge) / (kWarps * kStage);
  static constexpr int kTiles = NB == 1 ? 2 : 1;      // worked on side by side
  static constexpr int kStages = kFit >= 8 ? 8 : NB == 1 ? kFit & ~1 : kFit;
  static constexpr int kBytes = kMerge + 2 * kQ + kStages * kWarps * kStage;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {  // all but the last N groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// N consecutive 32-bit words.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 4) {
    const uint4 x = *(const uint4*)p;
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *(const uint2*)p;
    w[0] = x.x, w[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = ((const uint32_t*)p)[i];
  }
}

struct Fp4Params {
  explicit Fp4Params(const AttnArgs& a) : p{a}, by_page((unsigned)a.c.page_size) {}
  AttnParams p;
  Divider by_page;
  int q_vec;  // q's rows are whole 16-byte vectors
};

// (Of 128 registers; heads of 128 spill 8 bytes, and 104 with two blocks of rows, whose sums take 32 registers more.)
template <int D, int NB>  // NB blocks of 8 rows an item
__global__ void __launch_bounds__(kThreads, 2)
attention_fp4_kernel(const __grid_constant__ Fp4Params fp) {
  using Sh = Shape<D, NB>;
  constexpr int kSteps = D / 16;  // of the first product; tiles of 16 columns of the second
  constexpr int KW = D / 32;      // words of K's codes a thread and key
  constexpr int VW = (KW + 1) / 2;  // of V's
  constexpr int kPer = D / 8;     // columns of O a thread and row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ AttnStart<kTN> st;
  __shared__ float2 stats[2][kWarps][8 * NB];  // by the parity of the piece
  __shared__ int flags, bad_from[2];
  const AttnParams& p = fp.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + Sh::kMerge + 2 * Sh::kQ + warp * Sh::kStages * Sh::kStage;  // the warp's

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    flags = 0;
    bad_from[0] = bad_from[1] = 0x7fffffff;
  }
  __syncthreads();
  wait_for_previous();
  attn_plan<kTN>(p, &st, &flags);
  AttnWalk<kTN> w = st.walk;
  if (threadIdx.x == 0) attn_write_cut(p, st);

  // Loads of the walk's piece, the warp's block of a tile each: groups of copies, one a tile.
  const int S = p.a.c.page_size;
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  int ids = 0, ids_next = 0;  // pages of 32 tiles, a lane each, and of the 32 after
  auto look_up = [&](const AttnWalk<kTN>& c, int t) {
    const int key = (t + lane) * kTN + warp * kFp4Block;
    return key < c.end && t + lane < c.last_tile() ? p.a.a.page_table[(size_t)c.r * p.a.a.max_pages + fp.by_page(key)] : 0;
  };
  uint32_t stage = 0;  // of the ring
  auto load = [&](const AttnWalk<kTN>& c, int t) {  // tile t: called in order from the piece's first
    const int i = (t - c.first_tile()) & 31;
    if (i == 0) {
      ids = t == c.first_tile() ? look_up(c, t) : ids_next;
      ids_next = look_up(c, t + 32);
    }
    const int key = t * kTN + warp * kFp4Block;
    int pg = __shfl_sync(0xffffffffu, ids, i);
    if (key < c.end) {
      if (pg < 0 || pg >= p.a.c.n_pages) {
        if (lane == 0) flag_status(&flags, DSPARK_DEV_BAD_INPUT);
        pg = pg < 0 ? 0 : p.a.c.n_pages - 1;
      }
      const long long at = pg * p.a.c.page_stride + c.h * p.a.c.head_stride +
                           (key - fp.by_page(key) * S) / kFp4Block * Sh::kBlock + lane * 16;
      const uint8_t *k = (const uint8_t*)p.a.c.k + at, *v = (const uint8_t*)p.a.c.v + at - Sh::kBlock;
      const uint32_t dst = ring_at + stage * Sh::kStage + lane * 16;
      constexpr int kChunks = Sh::kBlock / 16;  // of K; then V's
#pragma unroll
      for (int j = 0; j < (2 * kChunks + 31) / 32; ++j) {
        const int c0 = 32 * j;
        if (c0 + 32 <= 2 * kChunks || c0 + lane < 2 * kChunks)
          copy16(dst + 512 * j, (c0 + 32 <= kChunks || (c0 < kChunks && c0 + lane < kChunks) ? k : v) + 512 * j);
      }
    }
    copy_commit();
    stage = stage + 1 == Sh::kStages ? 0 : stage + 1;
  };
  auto load_none = [&] {
    copy_commit();
    stage = stage + 1 == Sh::kStages ? 0 : stage + 1;
  };
  auto load_first = [&](const AttnWalk<kTN>& c) {
#pragma unroll 1
    for (int i = 0; i < Sh::kStages; ++i) {
      if (!c.done() && c.first_tile() + i < c.last_tile())
        load(c, c.first_tile() + i);
      else
        load_none();
    }
  };
  load_first(w);
  {
    const int g = lane >> 2, t4 = lane & 3;
    // Slot s of a block's eight keys holds key s ^ (s >> 1 & 1): rows of both
    // parities meet in the reads of V, whose 64-byte rows would else fall on the same banks.
    const int key_a = g ^ ((g >> 1) & 1);            // of the first product's row g (and 8 more)
    const int key_v = 2 * t4 ^ (t4 & 1);             // of the second's columns 2 t4 (and 8 more)
    const int key_w = key_v ^ 1;                     // and 2 t4 + 1
    const int G = p.a.G;
    uint32_t piece = 0;
    for (; !w.done(); ++piece) {
      const int rows = w.block_rows(p), row0 = w.m * p.mr, t1 = w.last_tile();
      const int n0 = w.q.L - w.q.n + 1;  // keys that the chunk's first token sees
      const int all_see = n0 + row0 / G;
      uint32_t qf[NB == 1 ? kSteps : 1][2];
      uint2* q_frags = (uint2*)(smem + Sh::kMerge + (piece & 1) * Sh::kQ);  // [NB][kSteps][32]
      float sc[NB][2];   // of the thread's columns: rows 2 t4 and 2 t4 + 1
      int lim[NB][2];    // keys that they see
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int a = 8 * b + g;
        const bool live = a < rows;
        uint32_t raw[kSteps * 2];
#pragma unroll
        for (int i = 0; i < kSteps * 2; ++i) raw[i] = 0u;
        if (live) {
          const unsigned row = row0 + a, tok = row / (unsigned)G, hq = row - tok * G;
          const uint16_t* src = (const uint16_t*)p.a.q + (long long)(w.q.q0 + tok) * p.a.q_token_stride +
                                (long long)(w.h * G + hq) * p.a.q_head_stride + t4 * (D / 4);
          if (fp.q_vec) {
#pragma unroll
            for (int i = 0; i < kSteps / 2; ++i) {
              const uint4 x = ((const uint4*)src)[i];
              raw[4 * i] = x.x, raw[4 * i + 1] = x.y, raw[4 * i + 2] = x.z, raw[4 * i + 3] = x.w;
            }
          } else {
#pragma unroll
            for (int i = 0; i < kSteps * 2; ++i) raw[i] = src[2 * i] | (uint32_t)src[2 * i + 1] << 16;
          }
        }
        uint32_t top = 0;  // the row's largest magnitude, as bf16 bits
#pragma unroll
        for (int i = 0; i < kSteps * 2; ++i) top = max(top, max(raw[i] & 0x7fffu, (raw[i] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^k that brings it to 2^14 .. 2^15 (field 141 - (its - 127)), as far as 2^-k is normal
        const int field = (int)(top >> 7), up = field == 255 ? 127 : min(268 - field, 253);
        const float f = __uint_as_float((uint32_t)up << 23);
        const float back = __uint_as_float((uint32_t)(254 - up) << 23) * p.scale_log2;
#pragma unroll
        for (int i = 0; i < kSteps * 2; ++i)
          raw[i] = pack_half(__uint_as_float(raw[i] << 16) * f, __uint_as_float(raw[i] & 0xffff0000u) * f);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          if constexpr (NB == 1)
            qf[i][0] = raw[2 * i], qf[i][1] = raw[2 * i + 1];
          else if (warp == 0)
            q_frags[(b * kSteps + i) * 32 + lane] = make_uint2(raw[2 * i], raw[2 * i + 1]);
        }
        const int lim_a = live ? n0 + (int)((unsigned)(row0 + a) / (unsigned)G) : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sc[b][i] = __shfl_sync(0xffffffffu, back, (2 * t4 + i) * 4);
          lim[b][i] = __shfl_sync(0xffffffffu, lim_a, (2 * t4 + i) * 4);
        }
      }
      // (Those of the piece before the last are not read any more: its merge is behind.)
      if (NB > 1) __syncthreads();
      float o[NB][kSteps][4], m[NB][2], l[NB][2];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) o[b][i][0] = o[b][i][1] = o[b][i][2] = o[b][i][3] = 0.0f;
        m[b][0] = m[b][1] = -INFINITY;
        l[b][0] = l[b][1] = 0.0f;
      }

      constexpr int U = Sh::kTiles;
      for (int t = w.first_tile(); t < t1; t += U) {
        copy_wait<Sh::kStages - U>();
        __syncwarp();
        // U tiles at a time: their chains of products run side by side.  (A tile past the piece's
        // last, like keys past the item's end, has any bytes, and is masked.)
        int k0[U];
        const uint8_t* kb[U];
        bool masked = false;
#pragma unroll
        for (int c = 0; c < U; ++c) {
          k0[c] = t + c < t1 ? (t + c) * kTN + warp * kFp4Block : 0x7fffff00;  // (past any length)
          kb[c] = ring + (stage + c) * Sh::kStage;
          masked |= k0[c] + kFp4Block > all_see;
        }
        if (k0[0] < w.end) {
          // S^T, each of a block's by two chains of products
          float s[U][NB][2][4] = {};
#pragma unroll
          for (int c = 0; c < U; ++c) {
            uint32_t lo[KW], hi[KW];
            load_words<KW>(kb[c] + key_a * (D / 2) + t4 * (D / 8), lo);
            load_words<KW>(kb[c] + (key_a + 8) * (D / 2) + t4 * (D / 8), hi);
            const uint8_t* ks = kb[c] + 8 * D + key_a * (D / 16);
            uint32_t slo = 0, shi = 0;
            if (KW == 4) {
              slo = e4m3x2_to_half(*(const uint16_t*)(ks + 2 * t4));
              shi = e4m3x2_to_half(*(const uint16_t*)(ks + 8 * (D / 16) + 2 * t4));
            }
#pragma unroll
            for (int j = 0; j < KW; ++j) {
              uint32_t fl, fh;  // the scale twice
              if (KW == 4) {
                fl = __byte_perm(slo, 0, j < 2 ? 0x1010 : 0x3232);
                fh = __byte_perm(shi, 0, j < 2 ? 0x1010 : 0x3232);
              } else {
                const int grp = (t4 * KW + j) >> 1;
                fl = e4m3x2_to_half(ks[grp] * 0x101u);
                fh = e4m3x2_to_half(ks[8 * (D / 16) + grp] * 0x101u);
              }
              uint32_t xl[4], xh[4];
              fp4x8_to_half(lo[j], xl);
              fp4x8_to_half(hi[j], xh);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t a[4] = {hmul2(xl[2 * h], fl), hmul2(xh[2 * h], fh), hmul2(xl[2 * h + 1], fl),
                                       hmul2(xh[2 * h + 1], fh)};
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                  if constexpr (NB == 1) {
                    mma16816(s[c][b][h], a, qf[2 * j + h][0], qf[2 * j + h][1]);
                  } else {
                    const uint2 q = q_frags[(b * kSteps + 2 * j + h) * 32 + lane];
                    mma16816(s[c][b][h], a, q.x, q.y);
                  }
                }
              }
            }
          }
          // P^T
          uint32_t pf[U][NB][2];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float x[U][4], x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
            for (int c = 0; c < U; ++c)
#pragma unroll
              for (int i = 0; i < 4; ++i) x[c][i] = (s[c][b][0][i] + s[c][b][1][i]) * sc[b][i & 1];
            if (masked) {
#pragma unroll
              for (int c = 0; c < U; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (k0[c] + key_a + 8 * (i >> 1) >= lim[b][i & 1]) x[c][i] = -INFINITY;
            }
#pragma unroll
            for (int c = 0; c < U; ++c) {
              x0 = fmaxf(x0, fmaxf(x[c][0], x[c][2]));
              x1 = fmaxf(x1, fmaxf(x[c][1], x[c][3]));
            }
            if (__any_sync(0xffffffffu, x0 > m[b][0] + kRise || x1 > m[b][1] + kRise)) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float mx = i ? x1 : x0;
#pragma unroll
                for (int d = 4; d < 32; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                if (mx > m[b][i] + kRise) {
                  const float mn = mx - kBelow, f = ex2(m[b][i] - mn);
                  m[b][i] = mn;
                  l[b][i] *= f;
#pragma unroll
                  for (int k = 0; k < kSteps; ++k) o[b][k][i] *= f, o[b][k][i + 2] *= f;
                }
              }
            }
            const float m0 = m[b][0] == -INFINITY ? 0.0f : m[b][0], m1 = m[b][1] == -INFINITY ? 0.0f : m[b][1];
#pragma unroll
            for (int c = 0; c < U; ++c) {
#pragma unroll
              for (int i = 0; i < 4; ++i) x[c][i] = ex2(x[c][i] - (i & 1 ? m1 : m0));
              l[b][0] += x[c][0] + x[c][2];
              l[b][1] += x[c][1] + x[c][3];
              pf[c][b][0] = transpose8x8(pack_half(x[c][0], x[c][1]));
              pf[c][b][1] = transpose8x8(pack_half(x[c][2], x[c][3]));
            }
          }
          // O^T
#pragma unroll
          for (int c = 0; c < U; ++c) {
            const uint8_t* vb = kb[c] + Sh::kBlock;
            constexpr int VS = KW == 3 ? 3 : 1;
            uint32_t v[4][VW], vs[4][VS];  // keys key_v, key_w, and 8 more
            auto key_of = [&](int i) { return (i & 1 ? key_w : key_v) + 8 * (i >> 1); };
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint8_t* row = vb + key_of(i) * (D / 2) + g * (D / 16);
              if constexpr (KW == 4 || KW == 2) {
                load_words<VW>(row, v[i]);
              } else {
                v[i][0] = *(const uint16_t*)row;
                if (KW == 3) {
                  v[i][0] |= (uint32_t)((const uint16_t*)row)[1] << 16;
                  v[i][VW - 1] = ((const uint16_t*)row)[2];
                }
              }
              const uint8_t* scale = vb + 8 * D + key_of(i) * (D / 16);
#pragma unroll
              for (int u = 0; u < VS; ++u) vs[i][u] = scale[KW == 3 ? (3 * g + u) >> 2 : g * KW >> 2];
            }
            if (masked) {
              // Past the item's end: any bytes.  Where some rows of the block do not see the
              // key, a scale that is NaN is hidden from them, and makes the others NaN below.
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = k0[c] + key_of(i);
#pragma unroll
                for (int u = 0; u < VS; ++u)
                  if (key >= all_see && (key >= w.end || (vs[i][u] & 0x7fu) == 0x7fu)) {
                    if (key < w.end) atomicMin(&bad_from[piece & 1], key);
                    vs[i][u] = 0u;
                  }
              }
            }
            uint32_t f0[VS], f1[VS];
#pragma unroll
            for (int u = 0; u < VS; ++u) {
              f0[u] = e4m3x2_to_half(vs[0][u] | vs[1][u] << 8);
              f1[u] = e4m3x2_to_half(vs[2][u] | vs[3][u] << 8);
            }
#pragma unroll
            for (int wi = 0; wi < VW; ++wi) {
              // Code by code: even columns in x, odd ones in y, the pair's two keys beside one another.
              uint32_t x[2][4], y[2][4];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t a = v[2 * i][wi], e = v[2 * i + 1][wi];
                fp4x8_to_half((a & 0x0f0f0f0fu) | ((e << 4) & 0xf0f0f0f0u), x[i]);
                fp4x8_to_half(((a >> 4) & 0x0f0f0f0fu) | (e & 0xf0f0f0f0u), y[i]);
              }
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int mt = 4 * wi + q;
                if (mt >= kSteps) break;
                const int u = KW == 3 ? mt >> 1 : 0;
                const uint32_t a[4] = {hmul2(x[0][q], f0[u]), hmul2(y[0][q], f0[u]), hmul2(x[1][q], f1[u]),
                                       hmul2(y[1][q], f1[u])};
#pragma unroll
                for (int b = 0; b < NB; ++b) mma16816(o[b][mt], a, pf[c][b][0], pf[c][b][1]);
              }
            }
          }
        }
        __syncwarp();  // (the stages are read)
#pragma unroll 1
        for (int c = 0; c < U; ++c) {
          if (t + Sh::kStages + c < t1)
            load(w, t + Sh::kStages + c);
          else
            load_none();
        }
      }

      // The next piece's first tiles, then this one's results.
      const AttnWalk<kTN> cur = w;
      w.next(p, &flags);
      load_first(w);

      // The eight warps' results.  (stats and bad_from of two pieces take turns: a warp
      // writes those of piece n + 2 after the barriers of piece n + 1.)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int d = 4; d < 32; d *= 2) l[b][i] += __shfl_xor_sync(0xffffffffu, l[b][i], d);
          if (g == 0) stats[piece & 1][warp][8 * b + 2 * t4 + i] = make_float2(m[b][i], l[b][i]);
        }
      const int where = attn_slot(cur);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (8 * b >= rows) break;
        __syncthreads();  // stats; the block before is read
        if (b == 0 && threadIdx.x == 0) bad_from[(piece + 1) & 1] = 0x7fffffff;  // (none is at the next piece yet)
        float* buf = (float*)smem;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int a = 2 * t4 + i;
          float top = -INFINITY;
#pragma unroll
          for (int x = 0; x < kWarps; ++x) top = fmaxf(top, stats[piece & 1][x][8 * b + a].x);
          const float f = m[b][i] == -INFINITY ? 0.0f : ex2(m[b][i] - top);
          float* dst = buf + (warp * 8 + a) * Sh::kRow + g * kPer;
#pragma unroll
          for (int k = 0; k < kSteps; k += 2) {
            const float4 v = make_float4(o[b][k][i] * f, o[b][k][i + 2] * f, o[b][k + 1][i] * f, o[b][k + 1][i + 2] * f);
            *(float4*)(dst + 2 * k) = v;
          }
        }
        __syncthreads();
        const int bad = *(volatile int*)&bad_from[piece & 1];
        for (int i = threadIdx.x; i < 8 * (D / 4); i += kWarps * 32) {
          const int a = i / (D / 4), d = i % (D / 4) * 4, r = 8 * b + a;
          if (r >= rows) continue;
          float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          float top = -INFINITY, sum = 0.0f;
#pragma unroll
          for (int x = 0; x < kWarps; ++x) {
            const float4 v = *(const float4*)(buf + (x * 8 + a) * Sh::kRow + d);
            y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
            top = fmaxf(top, stats[piece & 1][x][r].x);
          }
#pragma unroll
          for (int x = 0; x < kWarps; ++x) {
            const float2 q = stats[piece & 1][x][r];
            sum += q.x == -INFINITY ? q.y : q.y * ex2(q.x - top);  // (q.y: 0, or NaN)
          }
          const unsigned row = row0 + r, tok = row / (unsigned)G, hq = row - tok * G;
          if (n0 + (int)tok > bad) sum = __int_as_float(0x7fc00000);
          if (where < 0) {
            const size_t out = (size_t)(cur.q.q0 + tok) * p.a.Hq + cur.h * G + hq;
            const float inv = sum > 0.0f ? p.a.v_factor / sum : sum == 0.0f ? 0.0f : sum;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x * inv, y.y * inv);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(y.z * inv, y.w * inv);
            *(uint2*)((__nv_bfloat16*)p.a.out + out * D + d) = make_uint2(*(const uint32_t*)&lo, *(const uint32_t*)&hi);
            if (d == 0) p.a.lse[out] = sum == 0.0f ? -INFINITY : top * kLn2 + logf(sum);
          } else {
            const size_t part = ((size_t)blockIdx.x * 2 + where) * kMaxRows + r;
            const float f = p.a.v_factor;
            *(float4*)(p.part + part * D + d) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
            if (d == 0) p.stats[part] = make_float2(top, sum);
          }
        }
      }
    }
  }
  copy_wait<0>();
  __syncthreads();
  if (threadIdx.x == 0) p.flags[blockIdx.x] = flags;
}

template <int D, int NB>
cudaError_t launch(Fp4Params fp, char* ws, cudaStream_t s) {
  using Sh = Shape<D, NB>;
  static_assert(Sh::kCtas <= kAttnMaxCtas && Sh::kStages >= 2 * Sh::kTiles && 2 * (Sh::kBytes + 4096) <= 233472, "");
  const AttnWorkspace w = attn_workspace_layout(kMaxRows, D, Sh::kCtas);
  AttnParams& p = fp.p;
  p.status = (int*)ws;
  p.flags = (int*)(ws + w.flags);
  p.cuts = (CutItem*)(ws + w.cuts);
  p.stats = (float2*)(ws + w.stats);
  p.part = (float*)(ws + w.out);
  p.mr = 8 * NB;
  const cudaError_t attr = once_per_device([] { return allow_smem(attention_fp4_kernel<D, NB>, Sh::kBytes); });
  if (attr != cudaSuccess) return attr;
  cudaLaunchAttribute attr_pdl;
  const cudaLaunchConfig_t cfg = overlapped_launch(dim3(Sh::kCtas), kThreads, Sh::kBytes, s, &attr_pdl);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attention_fp4_kernel<D, NB>, fp);
  return e != cudaSuccess ? e : launch_attn_combine(p, kMaxRows, Sh::kCtas, s);
}

template <int D>
cudaError_t launch_rows(const Fp4Params& fp, char* ws, cudaStream_t s) {
  return attention_fp4_rows(fp.p.a) <= 8 ? launch<D, 1>(fp, ws, s) : launch<D, 2>(fp, ws, s);
}

}  // namespace

// Rows of most requests, as far as the host can tell.  Where there are no more tokens than requests, a
// token's.  Where they divide evenly, as many tokens each: chunks of one length, which a fixed number of drafted
// tokens gives, or rows padded to the longest.  Else the mean and a third, as a chunk longer than the mean takes
// another item.
bool attention_even_chunks(const AttnArgs& a) { return a.a.n_tokens <= a.a.R || a.a.n_tokens % a.a.R == 0; }
long long attention_fp4_rows(const AttnArgs& a) {
  if (a.a.n_tokens <= a.a.R) return a.G;
  const long long all = (long long)a.a.n_tokens * a.G;
  return attention_even_chunks(a) ? all / a.a.R : (all + all / 3 + a.a.R - 1) / a.a.R;
}

size_t attention_fp4_rows_workspace_bytes(int head_dim) {
  return attn_workspace_layout(kMaxRows, head_dim, kAttnMaxCtas).total;
}

// Up to 16 rows a request here, by the count above, and of them up to 8 in items of 8; more in attention_tc.cu,
// whose products are of 128 rows whatever there are.  Measured (us), items of 8 / of 16 / there, requests of 2000
// .. 8192 positions (32 of them) and of 100 .. 600 (128), eight K/V heads of 128:
//   chunks alike    8 rows   56 / 76 / 100     47 / 53 / 83
//                   12       112 / 80 / 101    93 / 62 / 85
//                   16       113 / 83 / 102    95 / 66 / 84
//                   20       154 / 157 / 103   130 / 119 / 85
//   uneven, on average 7.6   66 / 77 / 99      56 / 53 / 83       (counted as 10)
//                   11.2                       79 / 66 / 83       (15)
//                   13.2     114 / 104 / 101                      (18)
//                   14.6                       96 / 82 / 83       (20)
//                   18 .. 20 132 / 118 / 103   121 / 106 / 84
bool attention_fp4_few_rows(const AttnArgs& a) {
  if (a.dtype != DSPARK_BF16 || a.c.head_dim > 128) return false;
  return a.a.n_tokens == 0 || attention_fp4_rows(a) <= kMaxRows;  // (without tokens a call only checks its offsets)
}

cudaError_t launch_attention_fp4_rows(const AttnArgs& a, char* ws, cudaStream_t s) {
  Fp4Params fp(a);
  fp.p.scale_log2 = a.scale * 1.4426950408889634f;
  fp.p.item_units = 1;
  fp.q_vec = ((uintptr_t)a.q & 15u) == 0 && a.q_head_stride % 8 == 0 && a.q_token_stride % 8 == 0;
  switch (a.c.head_dim) {
    case 32: return launch_rows<32>(fp, ws, s);
    case 64: return launch_rows<64>(fp, ws, s);
    case 96: return launch_rows<96>(fp, ws, s);
    default: return launch_rows<128>(fp, ws, s);
  }
}

}  // namespace dspark
