// rows.cu -- a chunk's rows into the cache with the position rotation applied on
// the way (bf16, fp32 and 4-bit caches), and rows of the cache back as values.
//
// Rotation of pair i of a row at position p, with c, s = cos_sin[p][i], [p][rot / 2 + i]:
//   (a, b) -> (a c - b s, b c + a s),   pairs (i, i + rot / 2) or (2 i, 2 i + 1).
// Quantisation of a group y of 16 (after the rotation, divided by the factor):
//   scale = e4m3(max |y| / 6), code_j = e2m1(y_j / scale), both nearest, ties to even.
// K's rotated values are kept exact enough for that (rotated_odd), so that the
// stored bytes are those of the formula in infinite precision.
//
// Bound by memory: a row is read once and written once; the chain before a store
// (request, length, page: four dependent loads, then the table's row) is
// hidden by the rows of other warps, and by loading a row's K and V ahead of it.
#include <type_traits>

#include "append.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "serving.h"

namespace dspark {

namespace {

constexpr int kWarps = 8;  // of a CTA; a token a warp

template <typename T>
struct alignas(16) Vec16 {  // 16 bytes
  T e[16 / sizeof(T)];
};

template <typename T>
__device__ __forceinline__ T to_type(float x);
template <>
__device__ __forceinline__ float to_type<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_type<__nv_bfloat16>(float x) { return __float2bfloat16(x); }

// N consecutive elements as they lie in memory (a whole number of 16-byte vectors).
template <typename T, int N>
struct Group {
  static constexpr int kPer = 16 / sizeof(T), kVecs = N / kPer;
  Vec16<T> v[kVecs];
  __device__ __forceinline__ void load(const T* src) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = ((const Vec16<T>*)src)[i];
  }
  __device__ __forceinline__ void store(T* dst) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) ((Vec16<T>*)dst)[i] = v[i];
  }
  __device__ __forceinline__ float get(int i) const { return to_f32(v[i / kPer].e[i % kPer]); }
  __device__ __forceinline__ void set(int i, float x) { v[i / kPer].e[i % kPer] = to_type<T>(x); }
};

// Codes and scale of a group of 16, by two neighbouring lanes of `mask` with eight values each.
__device__ __forceinline__ void store_fp4(unsigned mask, const float* y, const float2& f, uint8_t* codes,
                                          uint8_t* scale) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(y[i]) & 0x7fffffffu);
  amax = max(amax, __shfl_xor_sync(mask, amax, 1));
  const Fp4Scale s = fp4_scale(amax, f.x, f.y);
  uint32_t w = 0u;
  if (s.inverse != 0.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w |= floats_to_fp4x2(fp4_quotient(y[2 * i], s), fp4_quotient(y[2 * i + 1], s)) << (8 * i);
  }
  *(uint32_t*)codes = w;
  if (!(threadIdx.x & 1)) *scale = (uint8_t)s.byte;
}

// Where a token's rows go in the cache.
struct CacheRow {
  long long at, codes, scales;  // the row of head 0: its element (or byte) offset
};
template <bool FP4>
__device__ __forceinline__ CacheRow cache_row(const CacheView& c, const RowPlace& pl) {
  CacheRow r;
  r.at = pl.page * c.page_stride + (FP4 ? 0 : pl.slot * c.token_stride);
  r.codes = FP4 ? r.at + fp4_codes_at(pl.slot, c.head_dim) : 0;
  r.scales = FP4 ? r.at + fp4_scales_at(pl.slot, c.head_dim) : 0;
  return r;
}

// The status word, by one CTA: rows without a place, and positions that the table lacks.
__device__ __forceinline__ void rotary_status(const RotaryAppendArgs& p) {
  bool bad = false;
  if (p.rot > 0 && p.positions) {
    int end = p.a.q_offsets[p.a.R];
    end = end < p.a.n_tokens ? end : p.a.n_tokens;
    for (int t = threadIdx.x; t < end; t += blockDim.x) {
      const int pos = p.positions[t];
      bad |= pos < 0 || pos >= p.n_positions;
    }
  } else if (p.rot > 0) {
    for (int r = threadIdx.x; r < p.a.R; r += blockDim.x)
      bad |= p.a.q_offsets[r + 1] > p.a.q_offsets[r] && p.a.kv_len[r] > p.n_positions;
  }
  append_status(p.c, p.a, p.status, bad);
}

// The row of the table for a token; false: the token is left out.
__device__ __forceinline__ bool table_row(const RotaryAppendArgs& p, const RowPlace& pl, int t,
                                          const float** cs) {
  if (pl.page < 0) return false;
  if (p.rot == 0) return true;
  const long long pos = p.positions ? p.positions[t] : pl.pos;
  if (pos < 0 || pos >= p.n_positions) return false;
  *cs = p.cos_sin + pos * p.rot;
  return true;
}

// Any sizes, strides, alignments and pairs: a row passes through shared memory
// and is then taken element by element, the head dimension over the lanes.
template <typename T, bool FP4>
__global__ void __launch_bounds__(kWarps * 32) append_rotary_any_kernel(const RotaryAppendArgs p) {
  __shared__ float rows[kWarps][256];
  const int lane = threadIdx.x & 31, D = p.c.head_dim, half = p.rot / 2;
  float* row = rows[threadIdx.x >> 5];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_previous();
  if (blockIdx.x == 0) {
    rotary_status(p);
    return;
  }
  for (int t = (blockIdx.x - 1) * kWarps + (threadIdx.x >> 5); t < p.a.n_tokens; t += (gridDim.x - 1) * kWarps) {
    const RowPlace pl = find_place(p.c, p.a, t);
    const float* cs = nullptr;
    if (!table_row(p, pl, t, &cs)) continue;
    const CacheRow at = cache_row<FP4>(p.c, pl);
    const auto load = [&](const T* src) {
      __syncwarp();
      for (int d = lane; d < D; d += 32) row[d] = to_f32(src[d]);
      __syncwarp();
    };
    const auto value = [&](int d, auto exact) -> float {  // of the rotated row
      if (d >= p.rot) return row[d];
      const bool first = p.interleaved ? !(d & 1) : d < half;
      const int i = p.interleaved ? d >> 1 : first ? d : d - half;
      const float x = row[d], y = row[p.interleaved ? d ^ 1 : first ? d + half : d - half];
      const float c = cs[i], s = first ? -cs[half + i] : cs[half + i];
      return exact ? rotated_odd(x, c, y, s) : fmaf(x, c, y * s);
    };
    const auto put = [&](void* base, int h, int d, float y, float2 f) {  // a warp's 32 elements of a head
      if constexpr (FP4) {
        uint32_t amax = __float_as_uint(y) & 0x7fffffffu;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const Fp4Scale s = fp4_scale(amax, f.x, f.y);
        const float z = s.inverse != 0.0f ? fp4_quotient(y, s) : 0.0f;
        const float z1 = __shfl_down_sync(0xffffffffu, z, 1);
        uint8_t* b = (uint8_t*)base + h * p.c.head_stride;
        if (!(lane & 1)) b[at.codes + d / 2] = (uint8_t)floats_to_fp4x2(z, z1);
        if (!(lane & 15)) b[at.scales + d / 16] = (uint8_t)s.byte;
      } else {
        if (d < D) ((T*)base)[at.at + h * p.c.head_stride + d] = to_type<T>(y);
      }
    };
    for (int h = 0; h < p.c.heads; ++h) {
      load((const T*)p.k_new + t * p.tok_stride + h * p.head_stride);
      for (int d = lane; d - lane < D; d += 32)
        put(p.c.k, h, d, d < D ? value(d, std::integral_constant<bool, FP4>{}) : 0.0f, p.k_factor);
      const T* vn = (const T*)p.v_new + t * p.tok_stride + h * p.head_stride;
      for (int d = lane; d - lane < D; d += 32) put(p.c.v, h, d, d < D ? to_f32(vn[d]) : 0.0f, p.v_factor);
    }
    for (int h = 0; h < p.Hq; ++h) {
      load((const T*)p.q + t * p.q_tok + h * p.q_head);
      for (int d = lane; d < D; d += 32)
        ((T*)p.q_out)[t * p.qo_tok + h * p.qo_head + d] = to_type<T>(value(d, std::false_type{}));
    }
  }
}

// Rows of whole groups of 16 on 16-byte boundaries, pairs whose groups are whole too:
// a lane takes eight columns and the eight that they are paired with (or, interleaved
// or past the rotated part, eight alone), so that rotation crosses no lanes; two
// neighbours have a 4-bit group.  K and V are on their way before the token's place is
// looked up, then the queries, four units a lane at a time.
template <typename T, bool FP4, bool Inter>
__global__ void __launch_bounds__(kWarps * 32, 2) append_rotary_kernel(const RotaryAppendArgs p, const Divider by_units, const Divider by_chunks) {
  typedef Group<T, 8> Cols;
  constexpr int kKAhead = sizeof(T) == 2 ? 2 : 1, kVAhead = 2 * kKAhead, kQ = 2;  // units a lane at a time
  const int lane = threadIdx.x & 31, D = p.c.head_dim, half = p.rot / 2;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_previous();
  if (blockIdx.x == 0) {
    rotary_status(p);
    return;
  }
  // Units of a row: those that are rotated first.  A unit's columns begin at d0 and, if it is a pair, d0 + half.
  // (Both counts are even: neighbouring lanes have neighbouring units of the same row.)
  const int turned = Inter ? p.rot / 8 : p.rot / 16, units = turned + (D - p.rot) / 8;
  const int n = p.c.heads * units, chunks = D / 8, nv = p.c.heads * chunks, nq = p.Hq * units;
  struct Unit {
    int h, d0;
    bool turn;
  };
  const auto unit = [&](int i) {
    const int h = by_units(i), j = i - h * units;
    return Unit{h, j < turned ? 8 * j : p.rot + 8 * (j - turned), j < turned};
  };
  for (int t = (blockIdx.x - 1) * kWarps + (threadIdx.x >> 5); t < p.a.n_tokens; t += (gridDim.x - 1) * kWarps) {
    const T* kn = (const T*)p.k_new + t * p.tok_stride;
    const T* vn = (const T*)p.v_new + t * p.tok_stride;
    const T* qn = (const T*)p.q + t * p.q_tok;
    T* qo = (T*)p.q_out + t * p.qo_tok;
    const auto load = [&](const T* row, const Unit& u, Cols& a, Cols& b) {
      a.load(row + u.d0);
      if (!Inter && u.turn) b.load(row + u.d0 + half);
    };
    const auto v_at = [&](int i) {
      const int h = by_chunks(i);
      return h * p.head_stride + (i - h * chunks) * 8;
    };
    Cols ka[kKAhead], kb[kKAhead], va[kVAhead];
#pragma unroll
    for (int k = 0; k < kKAhead; ++k)
      if (lane + 32 * k < n) {
        const Unit u = unit(lane + 32 * k);
        load(kn + u.h * p.head_stride, u, ka[k], kb[k]);
      }
#pragma unroll
    for (int k = 0; k < kVAhead; ++k)
      if (lane + 32 * k < nv) va[k].load(vn + v_at(lane + 32 * k));
    const RowPlace pl = find_place(p.c, p.a, t);
    const float* cs = nullptr;
    if (!table_row(p, pl, t, &cs)) continue;
    const CacheRow at = cache_row<FP4>(p.c, pl);
    constexpr int kAngles = Inter ? 4 : 8;
    float c[kAngles], s[kAngles];  // of the unit at column `cd`
    int cd = -1;
    const auto angles = [&](const Unit& u) {
      if (!u.turn || cd == u.d0) return;
      cd = u.d0;
      const float4* from = (const float4*)(cs + (Inter ? u.d0 / 2 : u.d0));
#pragma unroll
      for (int i = 0; i < kAngles; i += 4) {
        const float4 x = from[i / 4], y = *(const float4*)((const float*)(from + i / 4) + half);
        c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
        s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
      }
    };
    // One rotated value: rounded to odd for the choice of codes, else in fp32.
    const auto value = [](float x, float c, float y, float s, auto exact) {
      return exact ? rotated_odd(x, c, y, s) : fmaf(x, c, y * s);
    };
    const auto rotate = [&](const Unit& u, const Cols& a, const Cols& b, float* x, float* y, auto exact) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = a.get(i), y[i] = Inter || !u.turn ? 0.0f : b.get(i);
      if (!u.turn) return;
      if (Inter) {
#pragma unroll
        for (int i = 0; i < kAngles; ++i) {
          const float e = x[2 * i % 8], o = x[(2 * i + 1) % 8];
          x[2 * i % 8] = value(e, c[i], o, -s[i], exact);
          x[(2 * i + 1) % 8] = value(o, c[i], e, s[i], exact);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kAngles; ++i) {
          const float e = x[i], o = y[i];
          x[i] = value(e, c[i], o, -s[i], exact);
          y[i] = value(o, c[i], e, s[i], exact);
        }
      }
    };
    const auto store = [&](T* row, const Unit& u, const float* x, const float* y) {
      Cols g;
#pragma unroll
      for (int i = 0; i < 8; ++i) g.set(i, x[i]);
      g.store(row + u.d0);
      if (!Inter && u.turn) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g.set(i, y[i]);
        g.store(row + u.d0 + half);
      }
    };
    // mask: the lanes that have one (both of a group, as their units are in range together).
    const auto put_k = [&](unsigned mask, int i, const Cols& a, const Cols& b) {
      const Unit u = unit(i);
      float x[8], y[8];
      angles(u);
      rotate(u, a, b, x, y, std::integral_constant<bool, FP4>{});
      if constexpr (FP4) {
        uint8_t* base = (uint8_t*)p.c.k + u.h * p.c.head_stride;
        store_fp4(mask, x, p.k_factor, base + at.codes + u.d0 / 2, base + at.scales + u.d0 / 16);
        if (!Inter) {
          const unsigned pairs = __ballot_sync(mask, u.turn);
          if (u.turn)
            store_fp4(pairs, y, p.k_factor, base + at.codes + (u.d0 + half) / 2, base + at.scales + (u.d0 + half) / 16);
        }
      } else {
        store((T*)p.c.k + at.at + u.h * p.c.head_stride, u, x, y);
      }
    };
    const auto put_v = [&](unsigned mask, int i, const Cols& g) {
      const int h = by_chunks(i), j = i - h * chunks;
      if constexpr (FP4) {
        uint8_t* base = (uint8_t*)p.c.v + h * p.c.head_stride;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = g.get(e);
        store_fp4(mask, x, p.v_factor, base + at.codes + j * 4, base + at.scales + j / 2);
      } else {
        g.store((T*)p.c.v + at.at + h * p.c.head_stride + j * 8);
      }
    };
#pragma unroll
    for (int k = 0; k < kKAhead; ++k) {
      const unsigned mask = __ballot_sync(0xffffffffu, lane + 32 * k < n);
      if (lane + 32 * k < n) put_k(mask, lane + 32 * k, ka[k], kb[k]);
    }
#pragma unroll 1
    for (int i0 = 32 * kKAhead; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      const unsigned mask = __ballot_sync(0xffffffffu, i < n);
      if (i < n) {
        const Unit u = unit(i);
        load(kn + u.h * p.head_stride, u, ka[0], kb[0]);
        put_k(mask, i, ka[0], kb[0]);
      }
    }
#pragma unroll
    for (int k = 0; k < kVAhead; ++k) {
      const unsigned mask = __ballot_sync(0xffffffffu, lane + 32 * k < nv);
      if (lane + 32 * k < nv) put_v(mask, lane + 32 * k, va[k]);
    }
#pragma unroll 1
    for (int i0 = 32 * kVAhead; i0 < nv; i0 += 32) {
      const int i = i0 + lane;
      const unsigned mask = __ballot_sync(0xffffffffu, i < nv);
      if (i < nv) {
        va[0].load(vn + v_at(i));
        put_v(mask, i, va[0]);
      }
    }
#pragma unroll 1
    for (int i0 = lane; i0 < nq; i0 += 32 * kQ) {
      Cols a[kQ], b[kQ];
#pragma unroll
      for (int k = 0; k < kQ; ++k)
        if (i0 + 32 * k < nq) {
          const Unit u = unit(i0 + 32 * k);
          load(qn + u.h * p.q_head, u, a[k], b[k]);
        }
#pragma unroll
      for (int k = 0; k < kQ; ++k)
        if (i0 + 32 * k < nq) {
          const Unit u = unit(i0 + 32 * k);
          float x[8], y[8];
          angles(u);
          rotate(u, a[k], b[k], x, y, std::false_type{});
          store(qo + u.h * p.qo_head, u, x, y);
        }
    }
  }
}

// ------------------------------------------------------------------ read
// Rows of the cache as values: a row a warp; 4-bit rows in groups of 16, a group a lane.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) read_fp4_kernel(const CacheReadArgs p) {
  const int lane = threadIdx.x & 31, D = p.c.head_dim;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_previous();
  if (blockIdx.x == 0) {
    append_status(p.c, p.a, p.status);
    return;
  }
  const int groups = D / 16, n = p.c.heads * groups;
  for (int t = (blockIdx.x - 1) * kWarps + (threadIdx.x >> 5); t < p.a.n_tokens; t += (gridDim.x - 1) * kWarps) {
    const RowPlace pl = find_place(p.c, p.a, t);
    if (pl.page < 0) continue;
    const CacheRow at = cache_row<true>(p.c, pl);
    for (int i = lane; i < 2 * n; i += 32) {
      const bool is_v = i >= n;
      const int u = is_v ? i - n : i, h = u / groups, g = u - h * groups;
      const uint8_t* src = (const uint8_t*)(is_v ? p.c.v : p.c.k) + h * p.c.head_stride;
      const uint2 w = *(const uint2*)(src + at.codes + g * 8);
      const float s = e4m3_to_float(src[at.scales + g]), f = is_v ? p.v_factor : p.k_factor;
      uint32_t x[8];
      fp4x8_to_half(w.x, x);
      fp4x8_to_half(w.y, x + 4);
      Group<T, 16> out;
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // (code x scale is exact in 32 bits; the factor rounds once)
        out.set(2 * j, half_lo(x[j]) * s * f);
        out.set(2 * j + 1, half_hi(x[j]) * s * f);
      }
      out.store((T*)(is_v ? p.v_out : p.k_out) + ((long long)t * p.c.heads + h) * D + g * 16);
    }
  }
}

// bf16 and fp32: VE elements (16 bytes, or one where alignment does not allow) a lane and step.
template <typename E, int VE>
__global__ void __launch_bounds__(kWarps * 32) read_rows_kernel(const CacheReadArgs p) {
  struct alignas(sizeof(E) * VE) Vec {
    E e[VE];
  };
  const int lane = threadIdx.x & 31, D = p.c.head_dim;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_previous();
  if (blockIdx.x == 0) {
    append_status(p.c, p.a, p.status);
    return;
  }
  const int per_head = D / VE, n = p.c.heads * per_head;
  for (int t = (blockIdx.x - 1) * kWarps + (threadIdx.x >> 5); t < p.a.n_tokens; t += (gridDim.x - 1) * kWarps) {
    const RowPlace pl = find_place(p.c, p.a, t);
    if (pl.page < 0) continue;
    const long long at = cache_row<false>(p.c, pl).at, to = (long long)t * p.c.heads * D;
#pragma unroll 4
    for (int i = lane; i < n; i += 32) {
      const int h = i / per_head, d = (i - h * per_head) * VE;
      const Vec a = *(const Vec*)((const E*)p.c.k + at + h * p.c.head_stride + d);
      const Vec b = *(const Vec*)((const E*)p.c.v + at + h * p.c.head_stride + d);
      *(Vec*)((E*)p.k_out + to + i * VE) = a;
      *(Vec*)((E*)p.v_out + to + i * VE) = b;
    }
  }
}

int row_ctas(int n_tokens) {  // (the first one for the status word: also without tokens)
  const int ctas = (n_tokens + kWarps - 1) / kWarps;
  return (ctas < 1215 ? ctas : 1215) + 1;
}

}  // namespace

// Whether rows are whole groups on 16-byte boundaries, and pairs lie in whole groups.
static bool whole_groups(const RotaryAppendArgs& p, int esize, bool fp4) {
  const CacheView& c = p.c;
  const int ve = 16 / esize;
  uintptr_t at = (uintptr_t)p.k_new | (uintptr_t)p.v_new | (uintptr_t)p.cos_sin;
  long long strides = p.tok_stride | p.head_stride;
  if (p.Hq > 0) at |= (uintptr_t)p.q | (uintptr_t)p.q_out, strides |= p.q_tok | p.q_head | p.qo_tok | p.qo_head;
  if (!fp4) at |= (uintptr_t)c.k | (uintptr_t)c.v, strides |= c.page_stride | c.token_stride | c.head_stride;
  return c.head_dim % 16 == 0 && p.rot % (p.interleaved ? 16 : 32) == 0 && strides % ve == 0 && (at & 15u) == 0;
}

template <typename T, bool FP4>
static cudaError_t launch_append(const RotaryAppendArgs& p, const cudaLaunchConfig_t& cfg) {
  const int pairs = p.rot / (p.interleaved ? 8 : 16);
  const Divider by_units((unsigned)(pairs + (p.c.head_dim - p.rot) / 8)), by_chunks((unsigned)p.c.head_dim / 8);
  if (!whole_groups(p, sizeof(T), FP4)) return cudaLaunchKernelEx(&cfg, append_rotary_any_kernel<T, FP4>, p);
  return p.interleaved ? cudaLaunchKernelEx(&cfg, append_rotary_kernel<T, FP4, true>, p, by_units, by_chunks)
                       : cudaLaunchKernelEx(&cfg, append_rotary_kernel<T, FP4, false>, p, by_units, by_chunks);
}

cudaError_t launch_append_rotary(const RotaryAppendArgs& p, int dtype, bool fp4, cudaStream_t s) {
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = overlapped_launch(dim3(row_ctas(p.a.n_tokens)), kWarps * 32, 0, s, &attr);
  if (dtype == DSPARK_BF16)
    return fp4 ? launch_append<__nv_bfloat16, true>(p, cfg) : launch_append<__nv_bfloat16, false>(p, cfg);
  return fp4 ? launch_append<float, true>(p, cfg) : launch_append<float, false>(p, cfg);
}

cudaError_t launch_cache_read(const CacheReadArgs& p, int esize, bool fp4, cudaStream_t s) {
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = overlapped_launch(dim3(row_ctas(p.a.n_tokens)), kWarps * 32, 0, s, &attr);
  if (fp4)
    return esize == 2 ? cudaLaunchKernelEx(&cfg, read_fp4_kernel<__nv_bfloat16>, p)
                      : cudaLaunchKernelEx(&cfg, read_fp4_kernel<float>, p);
  const CacheView& c = p.c;
  const int ve = 16 / esize;
  const bool vec = c.head_dim % ve == 0 && c.page_stride % ve == 0 && c.token_stride % ve == 0 &&
                   c.head_stride % ve == 0 && (((uintptr_t)c.k | (uintptr_t)c.v) & 15u) == 0;
  if (esize == 2)
    return vec ? cudaLaunchKernelEx(&cfg, read_rows_kernel<uint16_t, 8>, p)
               : cudaLaunchKernelEx(&cfg, read_rows_kernel<uint16_t, 1>, p);
  return vec ? cudaLaunchKernelEx(&cfg, read_rows_kernel<uint32_t, 4>, p)
             : cudaLaunchKernelEx(&cfg, read_rows_kernel<uint32_t, 1>, p);
}

}  // namespace dspark
