// rows.cu -- a chunk's rows into the cache with the position rotation applied on
// the way (bf16, fp32 and 4-bit caches), and rows of the cache back as values.
//
// Rotation of pair i of a row at position p, with c, s = cos_sin[p][i], [p][rot / 2 + i]:
//   (a, b) -> (a c - b s, b c + a s),   pairs (i, i + rot / 2) or (2 i, 2 i + 1).
// Quantisation of a group y of 16 (after the rotation, divided by the factor):
//   scale = e4m3(max |y| / 6), code_j = e2m1(y_j / scale), both nearest, ties to even.
// K's rotated values are kept exact enough for that (rotated_odd: to about 2^-46 of the
// products), so that the stored bytes are those of the formula.
//
// Bound by memory: a row is read once and written once; the chain before a store
// (request, length, page: four dependent loads, then the table's row) is
// hidden by the rows of other warps, and by loading a row's K and V ahead of it.
// Measured, 32 query and 8 K/V heads of 128: 4868 tokens of 512 requests into a bf16
// cache 25.5 us in a graph (122 MB, 4.8 TB/s); prompts of 16,384 tokens into a bf16 cache 70 us
// (411 MB, 5.9 TB/s; of half-rotated heads 89), into a 4-bit one 79 us (362 MB, 4.6 TB/s, half of the
// issue slots taken by rotation, error bound and conversions; half-rotated 101); reading 36,321
// positions of a 4-bit cache 35 us (191 MB, 5.5 TB/s).
#include <type_traits>

#include "append.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "serving.h"

namespace dspark {

namespace {

constexpr int kWarps = 8;  // of a CTA; a token a warp

template <typename T>
__device__ __forceinline__ T to_type(float x);
template <>
__device__ __forceinline__ float to_type<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_type<__nv_bfloat16>(float x) { return __float2bfloat16(x); }

// Eight consecutive elements as they lie in memory: one or two 16-byte vectors.
template <typename T>
struct Cols {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* src) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = ((const uint4*)src)[i];
  }
  __device__ __forceinline__ void store(T* dst) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) ((uint4*)dst)[i] = v[i];
  }
  __device__ __forceinline__ uint32_t& word(int i) {
    uint4& q = v[i / 4];
    return i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w;
  }
  __device__ __forceinline__ f32x2 get(int i) {  // elements 2 i and 2 i + 1
    if constexpr (sizeof(T) == 2) {
      const uint32_t w = word(i);
      return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
      return pack2(__uint_as_float(word(2 * i)), __uint_as_float(word(2 * i + 1)));
    }
  }
  __device__ __forceinline__ void set(int i, f32x2 y) {
    float y0, y1;
    unpack2(y, y0, y1);
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(y0, y1);
      word(i) = *(const uint32_t*)&h;
    } else {
      word(2 * i) = __float_as_uint(y0), word(2 * i + 1) = __float_as_uint(y1);
    }
  }
};

// The largest magnitude of eight values, as bits; what is not a number counts as the largest.
__device__ __forceinline__ uint32_t largest8(const float* y) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(y[i])), "f"(fabsf(y[i + 1])));
  return __float_as_uint(m) & 0x7fffffffu;
}

// Eight codes of a group whose scale is s.  (fp4_quotient, two at a time; its bound in a branch, as most groups
// need none.  16,384 tokens: 78.6 us without it, 79.3 so; where such groups have scalar code of their own
// whole heads take 80.5 and half-rotated ones 127 for 101.)
__device__ __forceinline__ uint32_t codes8(const float* y, const Fp4Scale& s) {
  if (s.inverse == 0.0f) return 0u;
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = y[i];
  if (s.byte == kFp4LargestScale) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = at_most_8(z[i], s);
  }
  const f32x2 inv = pack2(s.inverse, s.inverse), value = pack2(-s.value, -s.value);
  uint32_t w = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 x = pack2(z[2 * i], z[2 * i + 1]), q = mul2(x, inv);
    float q0, q1;
    unpack2(fma2(fma2(q, value, x), inv, q), q0, q1);
    w |= floats_to_fp4x2(q0, q1) << (8 * i);
  }
  return w;
}

// Codes and scale of a group of 16, by two neighbouring lanes of `mask` with eight values each.
__device__ __forceinline__ void store_fp4(unsigned mask, const float* y, const float2& f, uint8_t* codes,
                                          uint8_t* scale) {
  uint32_t amax = largest8(y);
  amax = max(amax, __shfl_xor_sync(mask, amax, 1));
  const Fp4Scale s = fp4_scale(amax, f.x, f.y);
  *(uint32_t*)codes = codes8(y, s);
  if (!(threadIdx.x & 1)) *scale = (uint8_t)s.byte;
}

// The same for values that may be off by `error`: false, and nothing written, if one of the mask's
// groups might then get another scale or another code.  (Any lane of the mask: all are told.)
__device__ __forceinline__ bool store_fp4_if_sure(unsigned mask, const float* y, float error, const float2& f,
                                                  uint8_t* codes, uint8_t* scale) {
  uint32_t amax = largest8(y);
  amax = max(amax, __shfl_xor_sync(mask, amax, 1));
  const float a = __uint_as_float(amax);
  const Fp4Scale s = fp4_scale(amax, f.x, f.y);
  bool sure = fp4_scale_byte(fmaxf(a - error, 0.0f), f.y) == fp4_scale_byte(a + error, f.y);
  // Codes at both ends of each value's range.  (The quotient itself is off by 2^-22 of 6.5 at most.)
  const float d = error * s.inverse + 4e-6f;
  const f32x2 inv = pack2(s.inverse, s.inverse), up = pack2(d, d), down = pack2(-d, -d);
  uint32_t lo = 0u, hi = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 q = mul2(pack2(y[2 * i], y[2 * i + 1]), inv);
    float q0, q1;
    unpack2(add2(q, down), q0, q1);
    lo |= floats_to_fp4x2(q0, q1) << (8 * i);
    unpack2(add2(q, up), q0, q1);
    hi |= floats_to_fp4x2(q0, q1) << (8 * i);
  }
  // (A zero's sign does not count.  A group that is not finite, or all zero, is the exact path's.)
  const uint32_t diff = (lo ^ hi) & 0x77777777u, sign = (lo ^ hi) & 0x88888888u;
  sure = sure && diff == 0u && !(sign & ((lo << 1 | lo << 2 | lo << 3))) && amax < 0x7f800000u && s.inverse != 0.0f;
  if (!__all_sync(mask, sure)) return false;
  *(uint32_t*)codes = lo;
  if (!(threadIdx.x & 1)) *scale = (uint8_t)s.byte;
  return true;
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

// Any sizes, strides, alignments and pairs: a warp has some heads of a token's K and V, or of its
// queries; a row passes through shared memory and is then taken element by element, the
// head dimension over the lanes.  (A token always a warp: 64 tokens of 48 rows of 96 36 us for 4.7.)
template <typename T, bool FP4>
__global__ void __launch_bounds__(kWarps * 32) append_rotary_any_kernel(const RotaryAppendArgs p, int parts) {
  __shared__ float rows[kWarps][256];
  const int lane = threadIdx.x & 31, D = p.c.head_dim, half = p.rot / 2;
  float* row = rows[threadIdx.x >> 5];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_previous();
  if (blockIdx.x == 0) {
    rotary_status(p);
    return;
  }
  const int heads = p.c.heads + p.Hq;
  const long long jobs = (long long)p.a.n_tokens * parts;  // of every so many heads
  for (long long job = (blockIdx.x - 1) * kWarps + (threadIdx.x >> 5); job < jobs; job += (gridDim.x - 1) * kWarps) {
    const int t = (int)(job / parts), part = (int)(job - (long long)t * parts);
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
    for (int h = part; h < heads; h += parts) {
      if (h < p.c.heads) {
        load((const T*)p.k_new + t * p.tok_stride + h * p.head_stride);
        for (int d = lane; d - lane < D; d += 32)
          put(p.c.k, h, d, d < D ? value(d, std::integral_constant<bool, FP4>{}) : 0.0f, p.k_factor);
        const T* vn = (const T*)p.v_new + t * p.tok_stride + h * p.head_stride;
        for (int d = lane; d - lane < D; d += 32) put(p.c.v, h, d, d < D ? to_f32(vn[d]) : 0.0f, p.v_factor);
      } else {
        const int q = h - p.c.heads;
        load((const T*)p.q + t * p.q_tok + q * p.q_head);
        for (int d = lane; d < D; d += 32)
          ((T*)p.q_out)[t * p.qo_tok + q * p.qo_head + d] = to_type<T>(value(d, std::false_type{}));
      }
    }
  }
}

// Rows of whole groups of 16 on 16-byte boundaries, pairs of whole eights:
// a lane takes units of eight rotated columns and the eight that they are paired with (or,
// interleaved, eight alone), so that rotation crosses no lanes, and chunks of eight of what is
// not rotated; two neighbours have a 4-bit group.  A warp has a token's K and V, or a part
// of its queries; its rows are on their way before the token's place is looked up.
struct RowSteps {
  int units, step_h, step_j;  // rotated units of a row; 32 of them are step_h rows and step_j units
  int q_units, q_step_h, q_step_j;  // of Q
  int plain;                  // chunks of a row of K or Q that are not rotated
  int parts;                  // warps a token
  Divider by_units, by_q_units, by_plain, by_chunks, by_parts;
};
template <bool Wide>
constexpr int kQUnits = Wide ? 4 : 2;  // units a lane of a part of the queries
// A token is dealt to as many warps as run at once in all (two CTAs an SM): one for K, V and
// the queries, or one for K and V and the others for the queries, for the latency. More only
// repeat the look-ups of the token's place.  Measured (us) in a graph, by the warps a token, 32
// query and 8 K/V heads of 128:
//   tokens                 256: 1     2     5      608: 1     2     3     4     5      1216: 1     2     3      2432: 1     2
//   bf16                   5.5   4.5   3.4        6.2   4.8   4.0   4.1   5.6          8.1   7.0   7.5          13.4  15.4
//   bf16 to 4 bits         8.0   5.7   5.8        8.8   6.2   6.5   6.6   9.7         10.4   7.5  10.8          15.1  16.5
//   fp32                   8.0   6.2   5.6       11.4   8.5   8.1   7.4  10.5         16.0  12.5  16.5          22.2  22.4
constexpr int kWarpsAtOnce = 152 * 2 * kWarps;
enum Pairs {
  kHalves,      // (i, i + rot / 2): a unit is eight columns and those they are paired with
  kNeighbours,  // (2 i, 2 i + 1): eight columns
  kHalf,        // as kHalves, but a unit of K is eight columns, and the others are looked at: for 4-bit groups
                // of both halves, where rot / 2 is no multiple of 16.  (Not of Q, which may be rotated in place.)
};
template <typename T, bool FP4, Pairs P, bool Full>  // Full: the whole head is rotated
__global__ void __launch_bounds__(kWarps * 32, 2)
append_rotary_kernel(const RotaryAppendArgs p, const RowSteps rs) {
  constexpr bool Inter = P == kNeighbours;
  constexpr Pairs kOfQ = P == kHalf ? kHalves : P;
  // Units a lane at a time (interleaved ones are half as much; more in partly rotated rows: prompts into a
  // bf16 cache 86 -> 93 us).  Two CTAs an SM leave 128 registers.  Of whole heads in halves only fp32 rows spill
  // (8 bytes, into 4 bits 184), interleaved ones up to 64 bytes; partly rotated halves spill 68 (bf16), 132
  // (fp32) and 232 .. 244 (into 4 bits), a part of what they take longer.
  constexpr int kAhead = kQUnits<Inter && Full>, kKAhead = (sizeof(T) == 2 ? 2 : 1) * (Inter && Full ? 2 : 1);
  constexpr int kVAhead = sizeof(T) == 2 ? 4 : 1, kMore = Full || sizeof(T) == 4 ? 1 : 2;
  const int lane = threadIdx.x & 31, D = p.c.head_dim, half = p.rot / 2;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_previous();
  if (blockIdx.x == 0) {
    rotary_status(p);
    return;
  }
  // Strides as 32-bit numbers (the launcher checks).
  const int k_head = (int)p.head_stride, q_head = (int)p.q_head, qo_head = (int)p.qo_head, c_head = (int)p.c.head_stride;
  struct Unit {
    int h, j;
  };
  const auto next = [&](Unit u, int units, int step_h, int step_j) {  // 32 units on
    u.h += step_h, u.j += step_j;
    if (u.j >= units) u.j -= units, ++u.h;
    return u;
  };
  const auto load = [&](const T* row, const Unit& u, Cols<T>& a, Cols<T>& b, auto pairs) {
    a.load(row + 8 * u.j);
    if (pairs == kHalves) b.load(row + 8 * u.j + half);
    if (pairs == kHalf) b.load(row + 8 * u.j + (8 * u.j < half ? half : -half));
  };
  Unit first;
  first.h = rs.by_units(lane);
  first.j = lane - first.h * rs.units;

  const int jobs = p.a.n_tokens * rs.parts;
  for (int job = (blockIdx.x - 1) * kWarps + (threadIdx.x >> 5); job < jobs; job += (gridDim.x - 1) * kWarps) {
    const int t = rs.by_parts(job), part = job - t * rs.parts;
    const float* cs = nullptr;
    constexpr int kAngles = Inter ? 2 : 4;  // pairs of them, of the unit `at_j`
    f32x2 c[kAngles], s[kAngles];
    int at_j = -1;
    float largest = 1.0f;  // of their magnitudes and 1 (4-bit)
    const auto minus = [](f32x2 x) { return x ^ 0x8000000080000000ull; };
    const auto angles = [&](const Unit& u, auto pairs) {
      if (at_j == u.j) return;
      at_j = u.j;
      const bool second = pairs == kHalf && 8 * u.j >= half;
      const float* from = cs + (Inter ? 4 : 8) * u.j - (second ? half : 0);
#pragma unroll
      for (int i = 0; i < kAngles; i += 2) {
        const float4 x = *(const float4*)(from + 2 * i), y = *(const float4*)(from + half + 2 * i);
        c[i] = pack2(x.x, x.y), c[i + 1] = pack2(x.z, x.w);
        s[i] = pack2(y.x, y.y), s[i + 1] = pack2(y.z, y.w);
        if (pairs == kHalf && !second) s[i] = minus(s[i]), s[i + 1] = minus(s[i + 1]);
      }
      if constexpr (FP4) {
        largest = 1.0f;
#pragma unroll
        for (int i = 0; i < kAngles; ++i) {
          float x0, x1;
          unpack2(c[i], x0, x1);
          largest = fmaxf(largest, fmaxf(fabsf(x0), fabsf(x1)));
          unpack2(s[i], x0, x1);
          largest = fmaxf(largest, fmaxf(fabsf(x0), fabsf(x1)));
        }
      }
    };
    // The unit's columns (and those paired with them, y) rotated, as fp32 pairs: the plain products and sum.
    const auto rotate = [&](Cols<T>& a, Cols<T>& b, f32x2* x, f32x2* y, auto pairs) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = a.get(i);
      if (Inter) {  // pair i is (x0, x1) of x[i]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float e, o, ci[2], si[2];
          unpack2(x[i], e, o);
          unpack2(c[i / 2 % kAngles], ci[0], ci[1]);
          unpack2(s[i / 2 % kAngles], si[0], si[1]);
          x[i] = pack2(fmaf(e, ci[i & 1], -o * si[i & 1]), fmaf(o, ci[i & 1], e * si[i & 1]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x2 e = x[i], o = b.get(i), si = s[i % kAngles];
          x[i] = fma2(e, c[i % kAngles], mul2(o, pairs == kHalf ? si : minus(si)));
          if (pairs == kHalves) y[i] = fma2(o, c[i % kAngles], mul2(e, si));
        }
      }
    };
    // Units i0 .. of the queries, kAhead a lane.
    const std::integral_constant<Pairs, kOfQ> of_q;
    const auto queries = [&](int i0, auto find) {
      const int n = p.Hq * rs.q_units - i0;
      const T* row = (const T*)p.q + t * p.q_tok;
      T* to = (T*)p.q_out + t * p.qo_tok;
      Unit u[kAhead];
      Cols<T> a[kAhead], b[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (k > 0) {
          u[k] = next(u[k - 1], rs.q_units, rs.q_step_h, rs.q_step_j);
        } else {
          u[0].h = rs.by_q_units(i0 + lane), u[0].j = i0 + lane - u[0].h * rs.q_units;
        }
        if (lane + 32 * k < n) load(row + (long long)u[k].h * q_head, u[k], a[k], b[k], of_q);
      }
      if (!find()) return;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (lane + 32 * k < n) {
          f32x2 x[4], y[4];
          angles(u[k], of_q);
          rotate(a[k], b[k], x, y, of_q);
          T* dst = to + (long long)u[k].h * qo_head + 8 * u[k].j;
          Cols<T> g;
#pragma unroll
          for (int i = 0; i < 4; ++i) g.set(i, x[i]);
          g.store(dst);
          if (kOfQ == kHalves) {
#pragma unroll
            for (int i = 0; i < 4; ++i) g.set(i, y[i]);
            g.store(dst + half);
          }
        }
      }
    };
    // Part i of n of the queries.  find: whether the token has a place, looked up behind the first loads.
    // (What is not rotated stands already where q_out is q.)
    const auto some_queries = [&](int i, int n, auto find) {
#pragma unroll 1
      for (int i0 = i * 32 * kAhead; i0 < p.Hq * rs.q_units; i0 += n * 32 * kAhead) queries(i0, find);
      if constexpr (!Full) {
        if (p.q == p.q_out) return;
#pragma unroll 1
        for (int i0 = i * 32 * kVAhead; i0 < p.Hq * rs.plain; i0 += n * 32 * kVAhead) {
          Cols<T> g[kVAhead];
          const auto at = [&](int k, int head) {
            const int c = i0 + lane + 32 * k, h = rs.by_plain(c);
            return (long long)h * head + p.rot + (c - h * rs.plain) * 8;
          };
#pragma unroll
          for (int k = 0; k < kVAhead; ++k)
            if (i0 + lane + 32 * k < p.Hq * rs.plain) g[k].load((const T*)p.q + t * p.q_tok + at(k, q_head));
          if (!find()) return;
#pragma unroll
          for (int k = 0; k < kVAhead; ++k)
            if (i0 + lane + 32 * k < p.Hq * rs.plain) g[k].store((T*)p.q_out + t * p.qo_tok + at(k, qo_head));
        }
      }
    };
    if (part > 0) {
      int place = 0;  // 0 not looked up yet, 1, -1
      some_queries(part - 1, rs.parts - 1, [&] {
        if (place == 0) place = table_row(p, find_place(p.c, p.a, t), t, &cs) ? 1 : -1;
        return place > 0;
      });
      continue;
    }
    // -------------------------------------------- K and V
    const std::integral_constant<Pairs, P> of_k;
    const T* kn = (const T*)p.k_new + t * p.tok_stride;
    const T* vn = (const T*)p.v_new + t * p.tok_stride;
    const int n = p.c.heads * rs.units, chunks = D / 8, nv = p.c.heads * chunks;
    const int nc = Full ? nv : nv + p.c.heads * rs.plain;  // chunks of V, then those of K
    struct Chunk {
      int h, d;
    };
    const auto chunk = [&](int i) {
      const bool v = Full || i < nv;
      const int h = v ? rs.by_chunks(i) : rs.by_plain(i - nv);
      return v ? Chunk{h, (i - h * chunks) * 8} : Chunk{h, p.rot + (i - nv - h * rs.plain) * 8};
    };
    const auto chunk_from = [&](int i) {
      const Chunk c = chunk(i);
      return (Full || i < nv ? vn : kn) + (long long)c.h * k_head + c.d;
    };
    Cols<T> ka[kKAhead], kb[kKAhead], va[kVAhead];
    Unit u = first;
#pragma unroll
    for (int k = 0; k < kKAhead; ++k) {
      if (lane + 32 * k < n) load(kn + (long long)u.h * k_head, u, ka[k], kb[k], of_k);
      u = next(u, rs.units, rs.step_h, rs.step_j);
    }
#pragma unroll
    for (int k = 0; k < kVAhead; ++k)
      if (lane + 32 * k < nc) va[k].load(chunk_from(lane + 32 * k));
    const RowPlace pl = find_place(p.c, p.a, t);
    if (!table_row(p, pl, t, &cs)) continue;
    const CacheRow at = cache_row<FP4>(p.c, pl);
    // mask: the lanes that have one (both of a group, as their units are in range together).
    const auto put_k = [&](unsigned mask, const Unit& u, Cols<T>& a, Cols<T>& b) {
      angles(u, of_k);
      const int d = 8 * u.j;
      if constexpr (FP4) {
        uint8_t* base = (uint8_t*)p.c.k + (long long)u.h * c_head;
        uint8_t *codes = base + at.codes + d / 2, *scale = base + at.scales + d / 16;
        float x[8], y[8];
        {
          // In fp32, whose error is at most 3 2^-24 of the largest element times the largest of the
          // angles (which a table scaled for long contexts has above 1): mostly no code and no scale
          // hangs on it.
          f32x2 x2[4], y2[4];
          rotate(a, b, x2, y2, of_k);
          float top = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float e0, e1;
            unpack2(a.get(i), e0, e1);
            top = fmaxf(top, fmaxf(fabsf(e0), fabsf(e1)));
            if (!Inter) {
              unpack2(b.get(i), e0, e1);
              top = fmaxf(top, fmaxf(fabsf(e0), fabsf(e1)));
              if (P == kHalves) unpack2(y2[i], y[2 * i], y[2 * i + 1]);
            }
            unpack2(x2[i], x[2 * i], x[2 * i + 1]);
          }
          top *= largest * 2.4e-7f;
          top = fmaxf(top, __shfl_xor_sync(mask, top, 1));
          bool sure = store_fp4_if_sure(mask, x, top, p.k_factor, codes, scale);
          if (P == kHalves) sure = store_fp4_if_sure(mask, y, top, p.k_factor, codes + half / 2, scale + half / 16) && sure;
          if (sure) return;  // (all lanes)
          // (Rows and angles again: kept, they would cost the common path their registers.)
          load(kn + (long long)u.h * k_head, u, a, b, of_k);
          at_j = -1;
          angles(u, of_k);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          unpack2(a.get(i), x[2 * i], x[2 * i + 1]);
          float ci[2], si[2];
          unpack2(c[(Inter ? i / 2 : i) % kAngles], ci[0], ci[1]);
          unpack2(s[(Inter ? i / 2 : i) % kAngles], si[0], si[1]);
          if (Inter) {
            const float e = x[2 * i], o = x[2 * i + 1];
            x[2 * i] = rotated_odd(e, ci[i & 1], o, -si[i & 1]);
            x[2 * i + 1] = rotated_odd(o, ci[i & 1], e, si[i & 1]);
          } else {
            float o[2];
            unpack2(b.get(i), o[0], o[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float e = x[2 * i + k];
              x[2 * i + k] = rotated_odd(e, ci[k], o[k], P == kHalf ? si[k] : -si[k]);
              if (P == kHalves) y[2 * i + k] = rotated_odd(o[k], ci[k], e, si[k]);
            }
          }
        }
        store_fp4(mask, x, p.k_factor, codes, scale);
        if (P == kHalves) store_fp4(mask, y, p.k_factor, codes + half / 2, scale + half / 16);
      } else {
        f32x2 x[4], y[4];
        rotate(a, b, x, y, of_k);
        T* dst = (T*)p.c.k + at.at + (long long)u.h * c_head + d;
        Cols<T> g;
#pragma unroll
        for (int i = 0; i < 4; ++i) g.set(i, x[i]);
        g.store(dst);
        if (P == kHalves) {
#pragma unroll
          for (int i = 0; i < 4; ++i) g.set(i, y[i]);
          g.store(dst + half);
        }
      }
    };
    const auto put = [&](unsigned mask, int i, Cols<T>& g) {
      const Chunk c = chunk(i);
      void* pool = Full || i < nv ? p.c.v : p.c.k;
      if constexpr (FP4) {
        uint8_t* base = (uint8_t*)pool + (long long)c.h * c_head;
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack2(g.get(e), x[2 * e], x[2 * e + 1]);
        store_fp4(mask, x, Full || i < nv ? p.v_factor : p.k_factor, base + at.codes + c.d / 2, base + at.scales + c.d / 16);
      } else {
        g.store((T*)pool + at.at + (long long)c.h * c_head + c.d);
      }
    };
    u = first;
#pragma unroll
    for (int k = 0; k < kKAhead; ++k) {
      const unsigned mask = __ballot_sync(0xffffffffu, lane + 32 * k < n);
      if (lane + 32 * k < n) put_k(mask, u, ka[k], kb[k]);
      u = next(u, rs.units, rs.step_h, rs.step_j);
    }
#pragma unroll 1
    for (int i0 = 32 * kKAhead; i0 < n; i0 += 32) {
      const unsigned mask = __ballot_sync(0xffffffffu, i0 + lane < n);
      if (i0 + lane < n) {
        load(kn + (long long)u.h * k_head, u, ka[0], kb[0], of_k);
        put_k(mask, u, ka[0], kb[0]);
      }
      u = next(u, rs.units, rs.step_h, rs.step_j);
    }
#pragma unroll
    for (int k = 0; k < kVAhead; ++k) {
      const unsigned mask = __ballot_sync(0xffffffffu, lane + 32 * k < nc);
      if (lane + 32 * k < nc) put(mask, lane + 32 * k, va[k]);
    }
#pragma unroll 1
    for (int i0 = 32 * kVAhead; i0 < nc; i0 += 32 * kMore) {
#pragma unroll
      for (int k = 0; k < kMore; ++k)
        if (i0 + lane + 32 * k < nc) va[k].load(chunk_from(i0 + lane + 32 * k));
#pragma unroll
      for (int k = 0; k < kMore; ++k) {
        const unsigned mask = __ballot_sync(0xffffffffu, i0 + lane + 32 * k < nc);
        if (i0 + lane + 32 * k < nc) put(mask, i0 + lane + 32 * k, va[k]);
      }
    }
    if (P == kHalf) at_j = -1;  // (a unit is another one now)
    if (rs.parts == 1) some_queries(0, 1, [] { return true; });
  }
}

// ------------------------------------------------------------------ read
// Rows of the cache as values: a row a warp.  4-bit rows in units of eight elements, whose
// results are whole vectors of neighbouring lanes, several a lane in flight.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) read_fp4_kernel(const CacheReadArgs p, const Divider by_units) {
  constexpr int kAhead = 8;
  const int lane = threadIdx.x & 31, D = p.c.head_dim;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_previous();
  if (blockIdx.x == 0) {
    append_status(p.c, p.a, p.status);
    return;
  }
  const int units = D / 8, n = p.c.heads * units;
  for (int t = (blockIdx.x - 1) * kWarps + (threadIdx.x >> 5); t < p.a.n_tokens; t += (gridDim.x - 1) * kWarps) {
    const RowPlace pl = find_place(p.c, p.a, t);
    if (pl.page < 0) continue;
    const CacheRow at = cache_row<true>(p.c, pl);
    const long long to = (long long)t * p.c.heads * D;
#pragma unroll 1
    for (int i0 = lane; i0 < 2 * n; i0 += 32 * kAhead) {
      uint32_t w[kAhead], sc[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + 32 * k;
        if (i < 2 * n) {
          const int u = i < n ? i : i - n, h = by_units(u), j = u - h * units;
          const uint8_t* src = (const uint8_t*)(i < n ? p.c.k : p.c.v) + h * p.c.head_stride;
          w[k] = *(const uint32_t*)(src + at.codes + j * 4);
          sc[k] = src[at.scales + j / 2];
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + 32 * k;
        if (i < 2 * n) {
          // (code x scale is exact in fp16; the factor rounds once)
          const uint32_t s = e4m3x2_to_half(sc[k] * 0x101u);
          const float f = i < n ? p.k_factor : p.v_factor;
          uint32_t x[4];
          fp4x8_to_half(w[k], x);
          Cols<T> out;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t y = hmul2(x[e], s);
            out.set(e, mul2(pack2(half_lo(y), half_hi(y)), pack2(f, f)));
          }
          out.store(i < n ? (T*)p.k_out + to + i * 8 : (T*)p.v_out + to + (i - n) * 8);
        }
      }
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

int row_ctas(long long jobs) {  // a warp each (the first CTA for the status word: also without any)
  const long long ctas = (jobs + kWarps - 1) / kWarps;
  return (int)(ctas < 1215 ? ctas : 1215) + 1;
}

}  // namespace

// Whether rows are whole groups on 16-byte boundaries, pairs lie in whole eights, and
// strides and the number of jobs fit 32 bits.
static bool whole_groups(const RotaryAppendArgs& p, int esize, bool fp4, int parts) {
  const CacheView& c = p.c;
  const int ve = 16 / esize;
  uintptr_t at = (uintptr_t)p.k_new | (uintptr_t)p.v_new | (uintptr_t)p.cos_sin;
  long long strides = p.tok_stride | p.head_stride;
  if (p.Hq > 0) at |= (uintptr_t)p.q | (uintptr_t)p.q_out, strides |= p.q_tok | p.q_head | p.qo_tok | p.qo_head;
  if (!fp4) at |= (uintptr_t)c.k | (uintptr_t)c.v, strides |= c.page_stride | c.token_stride | c.head_stride;
  const long long most = 0x7fffffff;
  return c.head_dim % 16 == 0 && p.rot % 16 == 0 && strides % ve == 0 && (at & 15u) == 0 &&
         p.head_stride <= most && p.q_head <= most && p.qo_head <= most && c.head_stride <= most &&
         (long long)p.a.n_tokens * parts < 0x40000000;
}

template <typename T, bool FP4>
static cudaError_t launch_append(const RotaryAppendArgs& p, cudaStream_t s) {
  const Pairs pairs = p.interleaved ? kNeighbours : FP4 && p.rot % 32 != 0 ? kHalf : kHalves;
  const int units = p.rot / (pairs == kHalves ? 16 : 8), plain = (p.c.head_dim - p.rot) / 8, some = units > 0 ? units : 1;
  const int step = 32 * (p.interleaved && plain == 0 ? kQUnits<true> : kQUnits<false>);
  const int q_units = p.rot / (p.interleaved ? 8 : 16), q_some = q_units > 0 ? q_units : 1;
  const int split = 1 + (p.Hq * (q_units + plain / (p.interleaved ? 1 : 2)) + step - 1) / step;
  const int at_once = kWarpsAtOnce / (p.a.n_tokens > 0 ? p.a.n_tokens : 1);
  const auto warps = [&](int most) { return at_once < 1 ? 1 : at_once < most ? at_once : most; };  // a token
  const bool vec = whole_groups(p, sizeof(T), FP4, warps(split));
  const int parts = warps(vec ? split : p.c.heads + p.Hq);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg =
      overlapped_launch(dim3(row_ctas((long long)p.a.n_tokens * parts)), kWarps * 32, 0, s, &attr);
  if (!vec) return cudaLaunchKernelEx(&cfg, append_rotary_any_kernel<T, FP4>, p, parts);
  const RowSteps rs{units, 32 / some, 32 % some, q_units, 32 / q_some, 32 % q_some, plain, parts,
                    Divider((unsigned)some), Divider((unsigned)q_some), Divider((unsigned)(plain > 0 ? plain : 1)), Divider((unsigned)p.c.head_dim / 8),
                    Divider((unsigned)parts)};
  if constexpr (FP4) {  // (a whole head is a multiple of 32 there)
    if (pairs == kHalf) return cudaLaunchKernelEx(&cfg, append_rotary_kernel<T, FP4, kHalf, false>, p, rs);
  }
  if (plain == 0)
    return p.interleaved ? cudaLaunchKernelEx(&cfg, append_rotary_kernel<T, FP4, kNeighbours, true>, p, rs)
                         : cudaLaunchKernelEx(&cfg, append_rotary_kernel<T, FP4, kHalves, true>, p, rs);
  return p.interleaved ? cudaLaunchKernelEx(&cfg, append_rotary_kernel<T, FP4, kNeighbours, false>, p, rs)
                       : cudaLaunchKernelEx(&cfg, append_rotary_kernel<T, FP4, kHalves, false>, p, rs);
}

cudaError_t launch_append_rotary(const RotaryAppendArgs& p, int dtype, bool fp4, cudaStream_t s) {
  if (dtype == DSPARK_BF16) return fp4 ? launch_append<__nv_bfloat16, true>(p, s) : launch_append<__nv_bfloat16, false>(p, s);
  return fp4 ? launch_append<float, true>(p, s) : launch_append<float, false>(p, s);
}

cudaError_t launch_cache_read(const CacheReadArgs& p, int esize, bool fp4, cudaStream_t s) {
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = overlapped_launch(dim3(row_ctas(p.a.n_tokens)), kWarps * 32, 0, s, &attr);
  if (fp4)
    return esize == 2 ? cudaLaunchKernelEx(&cfg, read_fp4_kernel<__nv_bfloat16>, p, Divider(p.c.head_dim / 8))
                      : cudaLaunchKernelEx(&cfg, read_fp4_kernel<float>, p, Divider(p.c.head_dim / 8));
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
