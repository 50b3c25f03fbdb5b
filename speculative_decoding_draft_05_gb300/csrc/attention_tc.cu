// attention_tc.cu -- bf16 attention of a chunk over the paged cache on the
// 5th-generation tensor cores (sm_103a).
//
// Per item (up to 256 rows, the G query heads of a K/V head side by side) and
// tile of 128 keys: S = Q K^T (128 x 128 x D), the online softmax
//   m' = max(m, max_j s_j),  p_j = 2^{s_j - m'},  l' = l 2^{m-m'} + sum_j p_j,
//   O' = O 2^{m-m'} + P V
// in units of log2, with S and O in TMEM and P (bf16) written over the lower half of
// S in TMEM as the first operand of P V.  out = O / l is the same whatever reference m the
// two share, and floating-point rounding does not depend on it either, as long
// as nothing leaves the exponent range.  So m starts at 0 and stays until a
// row's maximum lies more than 60 above it (or, in a piece's first tile, below):
// p <= 2^60, sums stay under 2^100, and a term that underflows is under 2^-66 of
// the largest.  The softmax then needs one pass over S, not two.
//
// Structure (one CTA an SM, persistent over its share of the work; a piece is
// the part of an item in it):
//   * warp 11 (producer): TMA of K and V pages into a ring of tiles; each lane
//     owns one (page, 64-column half) box of a tile, so a tile of 16-token
//     pages is 16 boxes issued at once.
//   * warp 9 (MMA): one thread issues tcgen05.mma; S from shared-memory
//     descriptors, P V with P in TMEM and V as stored ([keys, D]: the N-major
//     second operand).
//   * warp 10 (loader): walks the share ahead of the others, loads each piece's
//     Q by TMA (boxes of G heads x tokens: the rows in order) and publishes
//     what the piece is.  Pieces of one row block alternate between the two Q
//     tiles, so the products of a run of such pieces follow one another
//     without a gap.
//   * warps 0..3 and 4..7: two softmax streams, one row a thread.  With two row
//     blocks the streams are the blocks and share each K/V tile; with one they
//     are alternate tiles of the same rows.  While one stream is in its softmax
//     the tensor cores run the other's products, and the product of P's first 96
//     keys begins while the rest of P is in the making.
//   * warps 12..15 (results): merge a piece's streams, scale and write it, while
//     the softmax warps are at the next piece.
//   * Keys at or past an item's end: pages past it are not loaded, S is
//     replaced by -inf, and V's rows are overwritten with zeros, since 0 x NaN of
//     an unused cache slot would reach the sum.  The same for a V that is not
//     finite at a key that some rows of the block see and some do not (positions
//     of the chunk itself): its row is cleared, and the rows that do see it become
//     NaN when the results are written.
//   * P is rounded to bf16, the type of V, as both operands of a product are of
//     one type.  Against 64 bits the output is then off by 2.3e-3 of its norm,
//     with P in 32 bits by 1.7e-3, which is the rounding of the output itself.
//     l sums p before it is rounded and all sums are fp32; an fp32 cache keeps P in
//     32 bits too.
//   * What bounds it: with few rows the read of K and V (verifying, 64 requests
//     of up to 17 tokens over 500 .. 8192 positions, 1.18 GB: 186 us, 6.3 TB/s;
//     4 requests of 17 tokens over 100 k positions, 1.87 GB: 283 us, 6.6 TB/s;
//     decoding, 16 requests of 200 .. 2048 positions, 85 MB: 29 us, of which 6
//     pass before the first scores and 6 after the last); with many rows the
//     chain of a stream, S, softmax, P V, against 1024 cycles of matrix
//     instructions a tile: about 2850 cycles a tile of each of the two streams
//     (prefill of 2901 + 4096 tokens at 5000 .. 8192 positions: 425 us, 1.56
//     PFLOP/s, 83 % of a library product's rate, for the first tenth of a second
//     at 2070 MHz; 458 us, 1.44 PFLOP/s, once the power limit holds the clock at
//     1.75 .. 1.95 GHz).
//   * Over a 4-bit cache (FP4), operands are fp16, in which code x scale is exact:
//     - warps 11 and 8 bring blocks of K's and V's codes (bulk copies, the blocks of a page
//       in one) and warps 16..23 turn them into the ring's tiles, a block of 16 keys each, with
//       the keys past an item's end as zeros and the NaN scales of V dealt with on the way;
//       results' warps load Q, a row times a power of two; the factor of V is in the results.
//     - P is fp16, so m has to stand before P is written: two passes over S (see the softmax).
//     - 768 threads share the registers and the instruction cache, which decides more than
//       the arithmetic does: loops, not unrolled code, 112 / 88 / 56 registers.
//     - What bounds it: the chain of a stream again, about 2500 cycles for a K and V tile of
//       each stream whether a block has 8 rows or 68; 1600 of them are the traffic of shared memory.
//       Verify as above, 349 MB: 177 us; 4 requests over 100 k positions, 569 MB: 259 us; prompts of
//       3556 + 4096 tokens: 607 us, 1.06 PFLOP/s.
//   * Every mbarrier wait is bounded; on expiry the CTA flags
//     DSPARK_DEV_TIMEOUT, drains what it issued, frees TMEM and returns.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <mutex>
#include <type_traits>

#include "attention.cuh"
#include "fp4.cuh"
#include "per_device.h"
#include "ptx.cuh"

namespace dspark {

namespace {

constexpr int kMR = 256;  // rows of an item, at most: two tiles of 128 / G tokens x G heads
constexpr int kTN = 128;  // keys of a tile
constexpr int kEarly = 96;  // of which the first are multiplied while the rest of P is in the making
constexpr int kMaxCtas = 152;  // one an SM of GB300; what the workspace holds pieces of
static_assert(kMaxCtas <= kAttnMaxCtas, "");
// Four warpgroups: two of softmax, the single roles, the results; with a 4-bit
// cache two more that turn codes into the products' operands.
template <bool FP4>
constexpr int kThreads = FP4 ? 768 : 512;
// Registers a thread after the split: 256 x 168 + 128 x 96 + 128 x 80 of the
// launch's 512 x 128; with a 4-bit cache 256 x 112 + 128 x 56 + 128 x 88 + 256 x
// 56 of 768 x 80.
template <bool FP4>
constexpr int kRegsSoftmax = FP4 ? 112 : 168;
template <bool FP4>
constexpr int kRegsOther = FP4 ? 56 : 96;
template <bool FP4>
constexpr int kRegsResult = FP4 ? 88 : 80;
constexpr int kRegsDecode = 56;
template <bool FP4>
constexpr int kRegsLaunch = FP4 ? 80 : 128;
static_assert(256 * kRegsSoftmax<false> + 128 * kRegsOther<false> + 128 * kRegsResult<false> <=
                  kThreads<false> * kRegsLaunch<false>, "a split above the launch's registers waits forever");
static_assert(256 * kRegsSoftmax<true> + 128 * kRegsOther<true> + 128 * kRegsResult<true> + 256 * kRegsDecode <=
                  kThreads<true> * kRegsLaunch<true>, "a split above the launch's registers waits forever");
static_assert(kThreads<true> * kRegsLaunch<true> <= 65536 && kThreads<false> * kRegsLaunch<false> <= 65536, "registers");
constexpr int kFirstRoleWarp = 8;  // (bf16: 8 idles, as warps 0, 4 and 12 share its scheduler, the busiest one for few rows)
constexpr int kMmaWarp = 9, kLoaderWarp = 10, kProducerWarp = 11, kResultWarp = 12;
constexpr int kDecodeWarp = 16, kDecodeWarps = 8;  // (4-bit) an eighth of a tile's keys each
constexpr int kProducerVWarp = 8;  // (4-bit) of V's codes; the other one brings K's
constexpr float kRangeLog2 = 60.0f;
// P in fp16 (4-bit): m is kBelow below the maximum that sets it, and stays until a
// score lies kRise above it: p < 2^15, and what underflows is below 2^-31 of the largest.
constexpr float kRise = 15.0f, kBelow = 8.0f, kLeast = 7.0f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kTmemCols = 512;  // S0, S1, O0, O1: 128 columns each

// Shared memory for head_dim padded to DP (64 or 128), from a 1024-aligned base.
template <int DP, bool FP4>
struct Layout {
  static constexpr int kHalves = DP / 64;
  static constexpr int kHalfBytes = 128 * 128;             // 128 rows of 128 bytes
  static constexpr int kTileBytes = kHalves * kHalfBytes;  // a Q, K or V tile
  static constexpr int kStages = FP4 ? (DP == 128 ? 3 : 6) : DP == 128 ? 5 : 10;
  // (4-bit) tiles as the cache holds them, and the factors of Q's rows
  static constexpr int kRawStages = FP4 ? (DP == 128 ? 6 : 12) : 0;
  static constexpr int kRawBytes = kTN / kFp4Block * fp4_block_bytes(DP);
  static constexpr int kOffQ = 0;  // two row blocks, or this piece's and the next one's rows
  static constexpr int kOffRing = 2 * kTileBytes;
  static constexpr int kOffRaw = kOffRing + kStages * kTileBytes;
  static constexpr int kOffTile = kOffRaw + kRawStages * kRawBytes;   // RawTile [kRawStages]
  static constexpr int kOffScale = kOffTile + kRawStages * 16;        // [2][128]
  static constexpr int kOffMerge = kOffScale + (FP4 ? 2 * 128 * 4 : 0);  // (m, l) [2][128]
  static constexpr int kOffBar = kOffMerge + 2 * 128 * 8;
  static constexpr int kBars = 2 * kStages + 2 * kRawStages + 2 + 2 + 2 + 2 + 2 + 1 + 1 + 2 + 2 + 2 + 1 + (FP4 ? 2 : 0);
  static constexpr int kBadWords = FP4 ? 4 : 2;
  static constexpr int kOffBad = kOffBar + kBars * 8;  // (see bad_v)
  static constexpr int kOffPiece = (kOffBad + kBadWords * 8 + 12 + 15) & ~15;  // PieceInfo [4]
  // The plan has room of its own: the roles read it after the last barrier of
  // all threads, so nothing may be written over it.
  static constexpr int kOffStart = (kOffPiece + 4 * 64 + 15) & ~15;
  static constexpr int kEnd = kOffStart + (int)sizeof(AttnStart<kTN>);
  // Dynamic shared memory starts on a 1024-byte boundary when a kernel has no
  // static shared memory; the slack covers most others, and the kernel checks.
  static constexpr int kBytes = kEnd + 1024 < 232448 ? kEnd + 1024 : 232448;
};
static_assert(Layout<64, false>::kEnd <= 232448 && Layout<128, false>::kEnd <= 232448, "shared memory");
static_assert(Layout<64, true>::kEnd <= 232448 && Layout<128, true>::kEnd <= 232448, "shared memory");
template <int DP, bool FP4>
constexpr bool plan_apart() {  // from all that is written while roles may still read it
  using Lo = Layout<DP, FP4>;
  return Lo::kOffStart >= Lo::kOffMerge + 2 * 128 * 8 && Lo::kOffStart >= Lo::kOffPiece + 4 * 64;
}
static_assert(plan_apart<64, false>() && plan_apart<128, false>(), "the plan's room");
static_assert(plan_apart<64, true>() && plan_apart<128, true>(), "the plan's room");

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// The MMA warp runs as a whole, and its instructions are issued under a
// predicate that one lane holds: operands then are the same for the warp and
// stay in uniform registers, which is where tcgen05.mma wants them.  (One lane
// in a branch of its own took about 130 clocks an instruction to issue.)
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}

__device__ __forceinline__ void tc_commit(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_addr(bar)),
      "r"(lead)
      : "memory");
}

// D[tmem] (+)= A[smem] B[smem], K = 16.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem], K = 16: A is 8 columns of bf16 pairs.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle, version 1.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// Instruction descriptor, kind::f16: fp32 accumulator, bf16 operands (or fp16), A K-major.
__host__ __device__ constexpr uint32_t make_idesc(int M, int N, bool b_n_major, bool half) {
  return (1u << 4) | (half ? 0u : (1u << 7) | (1u << 10)) | ((b_n_major ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 32 lanes x 32 columns of 32 bits: thread i gets row i's.  No wait.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
// Waits for the loads so far; the operands tie the uses of v behind the wait.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
                 "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]),
                 "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]),
                 "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]),
                 "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}
// 32 lanes x 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
      "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max(a, b, c) in one instruction.
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Whether a tile's row maximum (log2 units) is too far from the reference m:
// above it, or, before anything is summed, below it (-inf: no key seen).
template <bool FP4>
__device__ __forceinline__ bool out_of_range(float mx, float m, bool first) {
  if (FP4) return mx > m + kRise || (first && mx < m + kLeast && mx > -INFINITY);
  return mx > m + kRangeLog2 || (first && mx < m - kRangeLog2 && mx > -INFINITY);
}

// Scores of keys at or past the first `n` become -inf.
template <int N>
__device__ __forceinline__ void mask_from(uint32_t* x, int n) {
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (k >= n) x[k] = 0xff800000u;
}

// {hi, lo} rounded to bf16 and packed.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

// Accesses by shared-memory address.
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared2(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}

// A warp's registers from the launch's number to N.
template <int Launch, int N>
__device__ __forceinline__ void set_regs() {
  if constexpr (N > Launch)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

struct TcParams {
  explicit TcParams(const AttnArgs& a) : by_g((unsigned)a.G), by_page((unsigned)a.c.page_size) {}
  AttnParams p;
  int box_tokens;  // tokens of a K/V box: the largest power of two in page_size, up to 128
  int q_tokens;    // tokens of a Q tile (a box): 128 / G
  int tile_rows;   // rows of a Q tile: q_tokens G (128 where G > 128)
  int q_tma;       // q can be loaded by TMA (else by the loader's threads)
  int q_vec;       // (4-bit) q's rows are whole 16-byte vectors
  Divider by_g, by_page;  // (4-bit)
  float sign;      // of the scale; |scale| is in p.scale_log2
  long long wait_budget;
};

// Byte offset of 16-byte chunk c (0..7) of row r in a 128-byte-row swizzled tile.
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
}

// One piece: the part of an item that lies in this CTA's share.  Piece n's is in
// slot n & 3 and stays there while any warp is at it: the loader publishes piece
// n + 4 after all warps have read that piece n + 2 is there, which they do one
// after the other.
struct alignas(16) PieceInfo {
  int t0, nt;       // first tile, tiles (0: no more pieces)
  int rows, row0;   // rows of the block (more than tile_rows: two Q tiles), first row of the chunk
  int h, q0;        // K/V head, the chunk's first token
  int lim;          // keys that the chunk's token 0 sees (L - n + 1; may be <= 0)
  int end;          // keys of the item
  int slot;         // where the result goes (attn_slot)
  int next_joined;  // both this piece and the next one have one Q tile
  int all_see;      // keys that all rows of the block see
  int masked;       // the piece's tiles from this one on have keys that not all rows see
};
static_assert(sizeof(PieceInfo) <= 64, "piece slot");

// What the decoding warps have to know of a tile of codes (its loader writes it).
struct alignas(16) RawTile {
  int key0;     // -1: no more tiles
  int end;      // keys of the item from key0 on
  int all_see;  // of which all rows of the block see this many
  int tag;      // piece + 1, of a tile of V; else 0
};

template <int DP, bool FP4>
__global__ void __launch_bounds__(kThreads<FP4>, 1)
attention_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ TcParams tp) {
  using Lo = Layout<DP, FP4>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const AttnParams& p = tp.p;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (smem + Lo::kEnd > smem_raw + Lo::kBytes) {  // (never: see Layout)
    if (threadIdx.x == 0) p.flags[blockIdx.x] = DSPARK_DEV_TIMEOUT;
    return;
  }
  uint64_t* bars = (uint64_t*)(smem + Lo::kOffBar);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = bars + Lo::kStages;
  uint64_t* s_full = kv_empty + Lo::kStages;  // [2] S of a stream ready
  uint64_t* p_full = s_full + 2;              // [2] P of a stream written (4 warps)
  uint64_t* q_full = p_full + 2;   // [2] piece n (n & 1) published and its Q loaded
  uint64_t* q_empty = q_full + 2;  // [2] its last Q K^T done (1) and its info read (12 warps)
  uint64_t* o_full = q_empty + 2;  // [2] piece n's last product done
  uint64_t* ml_full = o_full + 2;  // piece n's (m, l) written (8 softmax warps)
  uint64_t* ml_empty = ml_full + 1;  // and read (4 result warps)
  uint64_t* o_free = ml_empty + 1;   // [2] a stream's O of piece n read (4 result warps)
  uint64_t* h_full = o_free + 2;   // [2] P's first kEarly keys written (4 warps)
  uint64_t* h_done = h_full + 2;   // [2] and their product done
  uint64_t* drain = h_done + 2;
  uint64_t* raw_full = drain + 1;                // (4-bit) a tile's codes loaded
  uint64_t* raw_empty = raw_full + Lo::kRawStages;  // and read (the decoding warps)
  uint64_t* i_full = raw_empty + Lo::kRawStages;    // (4-bit) [2] piece n (n & 1) published
  // Piece n's first key with a V that is not finite among those that not all of
  // its rows see: word n & 1 (4-bit: n & 3, as codes are decoded ahead of the results of the
  // piece before), (n + 1) << 32 | 2^31 - 1 - key, the largest counts.
  // (Of another piece: none.  The tag spares the clearing between pieces.)
  unsigned long long* bad_v = (unsigned long long*)(smem + Lo::kOffBad);
  uint32_t* tmem_slot = (uint32_t*)(bad_v + Lo::kBadWords);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  int* flags = (int*)(tmem_slot + 2);  // the CTA's status bits
  AttnStart<kTN>* st = (AttnStart<kTN>*)(smem + Lo::kOffStart);
  float2* merge = (float2*)(smem + Lo::kOffMerge);
  PieceInfo* infos = (PieceInfo*)(smem + Lo::kOffPiece);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!FP4 && threadIdx.x == kProducerWarp * 32) {
    prefetch_map(&tmK);
    prefetch_map(&tmV);
  }
  if (!FP4 && threadIdx.x == kLoaderWarp * 32 && tp.q_tma) prefetch_map(&tmQ);
  if (threadIdx.x == 0) {
    for (int i = 0; i < Lo::kStages; ++i) {
      mbar_init(&kv_full[i], FP4 ? kDecodeWarps : 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&h_full[i], 4);
      mbar_init(&h_done[i], 1);
      mbar_init(&q_full[i], FP4 ? 4 : 1);
      if (FP4) mbar_init(&i_full[i], 1);
      mbar_init(&q_empty[i], 13);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(ml_full, 8);
    mbar_init(ml_empty, 4);
    mbar_init(&o_free[0], 4);
    mbar_init(&o_free[1], 4);
    mbar_init(drain, 1);
    for (int i = 0; i < Lo::kRawStages; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], kDecodeWarps);
    }
    for (int i = 0; i < Lo::kBadWords; ++i) bad_v[i] = 0ull;
    *abort_flag = 0;
    *flags = 0;
    fence_barrier_init();
  }
  if (FP4 && p.a.c.head_dim < DP) {  // the columns that no code fills
    for (int i = threadIdx.x; i < Lo::kStages * Lo::kTileBytes / 16; i += kThreads<FP4>)
      ((uint4*)(smem + Lo::kOffRing))[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  wait_for_previous();
  attn_plan<kTN>(p, st, flags);  // ends with a barrier
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  bool ok = true;

  // (The register split stands in each role's own branch: after a join the
  // compiler would hold every role to the smaller number.)
  if (FP4 && warp >= kDecodeWarp) {
    // ------------------------------------------------------------ decoding (4-bit)
    if constexpr (FP4) {
      set_regs<kRegsLaunch<FP4>, kRegsDecode>();
      const int D = p.a.c.head_dim, block = fp4_block_bytes(D);
      constexpr int kKeys = kTN / kDecodeWarps;  // of a warp
      static_assert(kKeys == kFp4Block, "a block a warp");
      const int row0 = (warp - kDecodeWarp) * kKeys;
      const RawTile* tiles = (const RawTile*)(smem + Lo::kOffTile);
      for (uint32_t sl = 0;; ++sl) {
        const int stage = (int)(sl % Lo::kStages), rs = (int)(sl % Lo::kRawStages);
        ok = __all_sync(0xffffffffu, mbar_wait(&raw_full[rs], (sl / Lo::kRawStages) & 1u, abort_flag, tp.wait_budget));
        if (!ok) break;
        const RawTile c = tiles[rs];
        if (c.key0 < 0) break;
        ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[stage], ((sl / Lo::kStages) & 1u) ^ 1u, abort_flag,
                                               tp.wait_budget));
        if (!ok) break;
        const uint32_t raw = smem_addr(smem + Lo::kOffRaw) + rs * Lo::kRawBytes;
        const uint32_t tile = smem_addr(smem + Lo::kOffRing) + stage * Lo::kTileBytes;
        const bool masked = c.all_see < kTN;
        // A unit: 32 elements of a key, 16 bytes x of codes and two scales, to the four 16-byte chunks
        // of the row from `to` on (a row's chunk k at to ^ 16 k).
        auto decode = [&](int row, uint4 x, uint32_t sc, uint32_t to, auto offset) {
          if (masked && row >= c.all_see) {
            // Past the item's end: any bytes.  Where some rows of the block do not see the key, V's
            // scales that are NaN are hidden from them, and make the others NaN in the results.
            if (row >= c.end) {
              sc = 0u;
            } else if (c.tag && ((sc & 0x7fu) == 0x7fu || (sc & 0x7f00u) == 0x7f00u)) {
              sc = 0u;
              atomicMax(&bad_v[(c.tag - 1) & 3], (unsigned long long)c.tag << 32 | (uint32_t)(0x7fffffff - (c.key0 + row)));
            }
          }
          const uint32_t s2 = e4m3x2_to_half(sc), f0 = __byte_perm(s2, 0, 0x1010), f1 = __byte_perm(s2, 0, 0x3232);
          const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t h[4];
            fp4x8_to_half(w4[k], h);
            const uint32_t f = k < 2 ? f0 : f1;
            st_shared16((to ^ (k << 4)) + offset, hmul2(h[0], f), hmul2(h[1], f), hmul2(h[2], f), hmul2(h[3], f));
          }
        };
        if (D == DP) {
          // Eight rows a step (64-element rows: 16).  Eight consecutive lanes have one half's columns,
          // so that their stores do not meet on a bank.
          constexpr int kUnits = DP / 32, kRows = 32 / kUnits, kRun = kKeys / kRows;  // of a key; keys a step; steps
          const int r = DP == 128 ? (lane >> 1) & 7 : lane >> 1, col = (lane & 1) + (DP == 128 ? lane >> 4 << 1 : 0);
          const uint32_t block0 = raw + (row0 >> 4) * fp4_block_bytes(DP);
          const uint32_t to = tile + (col >> 1) * Lo::kHalfBytes + swz(row0 + r, (col & 1) * 4);
          uint4 x[kRun];
          uint32_t sc[kRun];
#pragma unroll
          for (int i = 0; i < kRun; ++i) {
            x[i] = ld_shared16(block0 + (r + i * kRows) * (DP / 2) + col * 16);
            sc[i] = ld_shared2(block0 + 8 * DP + (r + i * kRows) * (DP / 16) + col * 2);
          }
#pragma unroll
          for (int i = 0; i < kRun; ++i) decode(row0 + i * kRows + r, x[i], sc[i], to, i * kRows * 128);
        } else {
          const int units = D / 32;
          for (int u = lane; u < kKeys * units; u += 32) {
            const int r = u / units, col = u - r * units, row = row0 + r;
            const uint32_t b = raw + (row >> 4) * block;
            decode(row, ld_shared16(b + (row & 15) * (D / 2) + col * 16),
                   ld_shared2(b + 8 * D + (row & 15) * (D / 16) + col * 2),
                   tile + (col >> 1) * Lo::kHalfBytes + swz(row, (col & 1) * 4), 0);
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[rs]);
          mbar_arrive(&kv_full[stage]);
        }
      }
    }
  } else if (FP4 && (warp == kProducerWarp || warp == kProducerVWarp)) {
    // ------------------------------------------------------------ producers (4-bit)
    if constexpr (FP4) {
      set_regs<kRegsLaunch<FP4>, kRegsOther<FP4>>();
      const bool is_v = warp == kProducerVWarp;
      if (is_v && lane == 0) attn_write_cut(p, *st);
      constexpr int kBlocks = kTN / kFp4Block;     // of a tile; a lane looks one up
      constexpr int kTiles = 32 / kBlocks;         // looked up at once, the next ones ahead
      const int S = p.a.c.page_size, block = fp4_block_bytes(p.a.c.head_dim);
      const uint8_t* pool = (const uint8_t*)(is_v ? p.a.c.v : p.a.c.k);
      RawTile* tiles = (RawTile*)(smem + Lo::kOffTile);
      const uint32_t raw0 = smem_addr(smem + Lo::kOffRaw) + lane * block;
      uint32_t n = 0, last = 0;  // piece; one past the slot of the last load
      // Order of the operands' ring: with two row blocks K0 V0 K1 V1 ..; over a run of smaller pieces,
      // whose products run a tile ahead, K0 K1 V0 K2 V1 ..
      uint32_t base = 0, run = 0;  // slot of the run's first tile, steps of it before this piece
      AttnWalk<kTN> w = st->walk;
      while (!w.done() && ok) {
        const AttnWalk<kTN> cur = w;
        w.next(p, flags);
        const bool two = cur.block_rows(p) > tp.tile_rows;
        const bool joined = !two && !w.done() && w.block_rows(p) <= tp.tile_rows;
        const int all_see = cur.q.L - cur.q.n + 1 + tp.by_g(cur.m * p.mr);
        const int32_t* table = p.a.a.page_table + (size_t)cur.r * p.a.a.max_pages;
        const long long head = cur.h * p.a.c.head_stride;
        const int t1 = cur.last_tile();
        auto look_up = [&](int t) {
          const int k = t * kTN + lane * kFp4Block;
          return k < cur.end ? table[tp.by_page(k)] : 0;
        };
        int t = cur.first_tile(), left = kTiles;
        int ids = look_up(t), ids_next = look_up(t + kTiles);
        // (a run's K_i is at 2 i - 1, but the first; V_i behind K_{i + 1}, but the last)
        uint32_t slot = two ? base + (is_v ? 1 : 0) : base + 2 * run + (is_v ? 2 : -1);
        if (!joined) base += 2 * (run + (t1 - t));  // (run: 0 where there are two blocks)
        for (; t < t1; ++t, slot += 2) {
          if (left == 0) {
            left = kTiles;
            ids = ids_next, ids_next = look_up(t + kTiles);
          }
          const int key = t * kTN + lane * kFp4Block, keys = cur.end - key;  // from the lane's block on
          const bool has = lane < kBlocks && keys > 0;
          int pg = __shfl_sync(0xffffffffu, ids, (kTiles - left--) * kBlocks + (lane & (kBlocks - 1)));
          if (has && (pg < 0 || pg >= p.a.c.n_pages)) {
            flag_status(flags, DSPARK_DEV_BAD_INPUT);
            pg = pg < 0 ? 0 : p.a.c.n_pages - 1;
          }
          const int in_page = (key - tp.by_page(key) * S) / kFp4Block;
          // Blocks of one page follow one another: the first lane of each page brings them all.
          // (Each copy takes the warp's time to issue.)
          int count = 0;
          if (has && (lane == 0 || in_page == 0))
            count = min(min(S / kFp4Block - in_page, kBlocks - lane), (keys + kFp4Block - 1) / kFp4Block);
          const uint8_t* from = pool + pg * p.a.c.page_stride + head + in_page * block;
          const uint32_t sl = two ? slot : !is_v ? (run == 0 && t == cur.first_tile() ? slot + 1 : slot)
                                         : (!joined && t == t1 - 1 ? slot - 1 : slot);
          const int rs = (int)(sl % Lo::kRawStages);
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&raw_empty[rs], ((sl / Lo::kRawStages) & 1u) ^ 1u, abort_flag,
                                                       tp.wait_budget))))
            break;
          if (lane == 0) {  // (keys: the tile's)
            tiles[rs] = RawTile{key, keys, all_see - key, is_v ? (int)n + 1 : 0};
            const int blocks = keys >= kTN ? kBlocks : (keys + kFp4Block - 1) / kFp4Block;
            mbar_expect_tx(&raw_full[rs], (uint32_t)(keys > 0 ? blocks : 0) * block);
          }
          __syncwarp();
          if (count > 0) bulk_load(raw0 + rs * Lo::kRawBytes, from, count * block, &raw_full[rs]);
          last = sl + 1;
        }
        run = joined ? run + (t1 - cur.first_tile()) : 0;
        ++n;
      }
      if (ok && !is_v) {  // no more, after the slots of the last run
        const int rs = (int)(base % Lo::kRawStages);
        ok = __all_sync(0xffffffffu, mbar_wait(&raw_empty[rs], ((base / Lo::kRawStages) & 1u) ^ 1u, abort_flag,
                                               tp.wait_budget));
        if (ok && lane == 0) {
          tiles[rs].key0 = -1;
          mbar_arrive(&raw_full[rs]);
        }
      }
      if (!ok && lane == 0)  // the loads still in flight, the other warp's among them
        for (uint32_t i = last > Lo::kRawStages ? last - Lo::kRawStages : 0; i < last; ++i)
          mbar_drain(&raw_full[i % Lo::kRawStages], (i / Lo::kRawStages) & 1u, tp.wait_budget);
    }
  } else if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    set_regs<kRegsLaunch<FP4>, kRegsOther<FP4>>();
    AttnWalk<kTN> w = st->walk;
    const int bt = tp.box_tokens, E = kTN / bt;  // boxes along a tile's keys
    const int S = p.a.c.page_size;
    const int e = lane / Lo::kHalves, half = lane % Lo::kHalves;  // this lane's box
    uint32_t slot = 0;  // ring slots used so far
    auto load = [&](const CUtensorMap* map, int t, int h, int pg) {
      const int stage = (int)(slot % Lo::kStages);
      const uint32_t phase = (slot / Lo::kStages) & 1u;
      if (!__all_sync(0xffffffffu,
                      mbar_wait(&kv_empty[stage], phase ^ 1u, abort_flag, tp.wait_budget)))
        return false;
      const unsigned boxes = __ballot_sync(0xffffffffu, pg >= 0);
      if (lane == 0) mbar_expect_tx(&kv_full[stage], (uint32_t)__popc(boxes) * bt * 128);
      __syncwarp();
      if (pg >= 0)
        tma_load_4d(smem + Lo::kOffRing + stage * Lo::kTileBytes + half * Lo::kHalfBytes +
                        e * bt * 128,
                    map, half * 64, (t * kTN + e * bt) % S, h, pg, &kv_full[stage]);
      ++slot;
      return true;
    };
    // Ring order: with two row blocks K0 V0 K1 V1 ..; over a run of smaller
    // pieces, whose products run a tile ahead, K0 K1 V0 K2 V1 ..
    bool pending = false;  // a V that the next K goes before
    int pend_t = 0, pend_h = 0, pend_pg = -1;
    for (; !w.done() && ok; w.next(p, flags)) {
      const int32_t* table = p.a.a.page_table + (size_t)w.r * p.a.a.max_pages;
      // The page of this lane's box of tile t, as the table has it, if the item
      // has keys there.  It is checked when it is used, a tile later.
      auto has_box = [&](int t) { return e < E && t * kTN + e * bt < w.end; };
      auto page_at = [&](int t) { return has_box(t) ? table[(t * kTN + e * bt) / S] : -1; };
      auto checked = [&](int t, int pg) {
        if (!has_box(t)) return -1;
        if (pg < 0 || pg >= p.a.c.n_pages) {
          flag_status(flags, DSPARK_DEV_BAD_INPUT);
          pg = pg < 0 ? 0 : p.a.c.n_pages - 1;
        }
        return pg;
      };
      const int t1 = w.last_tile();
      const bool two = w.block_rows(p) > tp.tile_rows;
      if (two && pending) {
        ok = load(&tmV, pend_t, pend_h, pend_pg);
        pending = false;
      }
      int raw = page_at(w.first_tile());
      for (int t = w.first_tile(); t < t1 && ok; ++t) {
        const int raw_next = t + 1 < t1 ? page_at(t + 1) : -1;  // read a tile ahead
        const int pg = checked(t, raw);
        ok = load(&tmK, t, w.h, pg);
        if (two) {
          ok = ok && load(&tmV, t, w.h, pg);
        } else {
          if (pending) ok = ok && load(&tmV, pend_t, pend_h, pend_pg);
          pending = true;
          pend_t = t, pend_h = w.h, pend_pg = pg;
        }
        raw = raw_next;
      }
    }
    if (ok && pending) ok = load(&tmV, pend_t, pend_h, pend_pg);
    if (!ok && lane == 0) {
      // Drain: wait (bounded) for the loads still in flight before leaving.
      for (uint32_t i = slot > Lo::kStages ? slot - Lo::kStages : 0; i < slot; ++i)
        mbar_drain(&kv_full[i % Lo::kStages], (i / Lo::kStages) & 1u, tp.wait_budget);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    set_regs<kRegsLaunch<FP4>, kRegsOther<FP4>>();
    {
      const uint32_t lead = elect_one();
      const uint32_t id_s = make_idesc(128, kTN, false, FP4), id_o = make_idesc(128, DP, true, FP4);
      const uint32_t q0 = smem_addr(smem + Lo::kOffQ), ring = smem_addr(smem + Lo::kOffRing);
      uint32_t slot = 0;  // next ring slot, in the order of use
      uint32_t n = 0, steps0 = 0, steps1 = 0;  // piece, P tiles of each stream so far
      // A piece's first products overwrite O: the results of the one before are read.
      // Every piece waits for both streams' hand-backs, also where it has products
      // on one alone: a wait tells a phase by its parity, so no phase may be left out.
      auto wait_o_free = [&](int s, uint32_t piece) {
        if (piece == 0) return true;
        const bool r = __all_sync(0xffffffffu, mbar_wait(&o_free[s], (piece - 1) & 1u, abort_flag,
                                                         tp.wait_budget));
        tc_fence_after();
        return r;
      };
      auto wait_full = [&](uint32_t sl) {
        const bool r = __all_sync(0xffffffffu, mbar_wait(&kv_full[sl % Lo::kStages],
                                                         (sl / Lo::kStages) & 1u, abort_flag,
                                                         tp.wait_budget));
        tc_fence_after();
        return r;
      };
      // Descriptors differ in their address field (16-byte units) alone.
      const uint64_t q_desc = smem_desc(q0, 16, 1024), k_desc = smem_desc(ring, 16, 1024),
                     v_desc = smem_desc(ring, Lo::kHalfBytes, 1024);
      auto qk = [&](int s, int block, uint32_t sl) {  // S_s = Q_block K^T
        const uint64_t kt = k_desc + (sl % Lo::kStages) * (Lo::kTileBytes >> 4);
        const uint64_t qt = q_desc + block * (Lo::kTileBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
          const int off = ((kk / 4) * Lo::kHalfBytes + (kk % 4) * 32) >> 4;
          mma_ss(tmem + s * 128, qt + off, kt + off, id_s, kk != 0, lead);
        }
        tc_commit(&s_full[s], lead);
      };
      // O_s (+)= P_s V, the first kEarly keys while the rest of P is in the making.
      auto pv = [&](int s, uint32_t sl, bool first) {
        const uint64_t vt = v_desc + (sl % Lo::kStages) * (Lo::kTileBytes >> 4);
        const uint32_t o = tmem + 256 + s * 128, pt = tmem + s * 128;
#pragma unroll
        for (int kk = 0; kk < kEarly / 16; ++kk)
          mma_ts(o, pt + kk * 8, vt + kk * (2048 >> 4), id_o, !(first && kk == 0), lead);
        if (!FP4) tc_commit(&h_done[s], lead);  // (4-bit: P stands once it is written)
        uint32_t& k = s ? steps1 : steps0;
        const bool r = __all_sync(0xffffffffu, mbar_wait(&p_full[s], k++ & 1u, abort_flag, tp.wait_budget));
        tc_fence_after();
        if (!r) return false;
#pragma unroll
        for (int kk = kEarly / 16; kk < kTN / 16; ++kk)
          mma_ts(o, pt + kk * 8, vt + kk * (2048 >> 4), id_o, 1u, lead);
        return true;
      };
      // A tile's slot is free once its products are done.  (4-bit: K's by the softmax warps, as S is ready.)
      auto release = [&](uint32_t sl) { tc_commit(&kv_empty[sl % Lo::kStages], lead); };
      auto wait_half = [&](int s) {
        const uint32_t k = s ? steps1 : steps0;
        const bool r = __all_sync(0xffffffffu, mbar_wait(&h_full[s], k & 1u, abort_flag, tp.wait_budget));
        tc_fence_after();
        return r;
      };
      auto wait_piece = [&] {  // piece n published
        const bool r = __all_sync(0xffffffffu, mbar_wait(&q_full[n & 1], (n >> 1) & 1u, abort_flag,
                                                         tp.wait_budget));
        tc_fence_after();
        return r;
      };
      while (ok) {
        if (!(ok = wait_piece())) break;
        int nt = infos[n & 3].nt;
        if (nt == 0) break;
        if (infos[n & 3].rows > tp.tile_rows) {
          ok = wait_full(slot);
          if (!ok) break;
          qk(0, 0, slot);
          qk(1, 1, slot);
          if (!FP4) release(slot);
          if (nt == 1) tc_commit(&q_empty[n & 1], lead);
          for (int j = 0; j < nt; ++j) {
            const uint32_t vs = slot + 1, ks = slot + 2;
            const bool more = j + 1 < nt;
            if (!(ok = wait_full(vs) && wait_half(0) && (j > 0 || wait_o_free(0, n)))) break;
            if (!(ok = pv(0, vs, j == 0))) break;
            if (more) {
              if (!(ok = wait_full(ks))) break;
              qk(0, 0, ks);
            }
            if (!(ok = wait_half(1) && (j > 0 || wait_o_free(1, n)))) break;
            if (!(ok = pv(1, vs, j == 0))) break;
            release(vs);
            if (more) {
              qk(1, 1, ks);
              if (!FP4) release(ks);
              if (j + 2 == nt) tc_commit(&q_empty[n & 1], lead);
            }
            slot += 2;
          }
          tc_commit(&o_full[n & 1], lead);
          ++n;
        } else {
          // A run of pieces of up to 128 rows: step i on stream i & 1; the
          // first product of step i + 2 follows the second of step i.
          int jq = 0;
          uint32_t iq = 0;           // steps whose first product is issued
          // Of the step in flight on a stream: 1 the stream's first of its piece, 2 the
          // piece's last, 4 the piece's first.
          uint32_t flags0 = 0, flags1 = 0;
          bool open = true;
          uint32_t np = n;           // the piece of the second products
          auto issue_qk = [&] {
            if (jq == nt) {  // the next piece, if it belongs to the run
              ++n;
              if (!(ok = wait_piece())) return;
              nt = infos[n & 3].nt;
              if (nt == 0 || infos[n & 3].rows > tp.tile_rows) {
                open = false;
                return;
              }
              jq = 0;
            }
            if (!(ok = wait_full(slot))) return;
            const int s = iq & 1;
            qk(s, n & 1, slot);
            if (!FP4) release(slot);
            ++slot;
            const bool last = ++jq == nt;
            (s ? flags1 : flags0) = (jq <= 2 ? 1u : 0u) | (last ? 2u : 0u) | (jq == 1 ? 4u : 0u);
            if (last) tc_commit(&q_empty[n & 1], lead);
            ++iq;
          };
          issue_qk();
          if (ok) issue_qk();
          for (uint32_t i = 0; i < iq && ok; ++i) {
            const int s = i & 1;
            if (!(ok = wait_full(slot) && wait_half(s))) break;
            const uint32_t f = s ? flags1 : flags0;
            if (f & 4u && !(ok = wait_o_free(0, np) && wait_o_free(1, np))) break;
            if (!(ok = pv(s, slot, f & 1u))) break;
            release(slot++);
            if (f & 2u) tc_commit(&o_full[np++ & 1], lead);
            if (open) issue_qk();
          }
        }
      }
      // All products done before TMEM is freed.
      tc_commit(drain, lead);
      mbar_drain(drain, 0, tp.wait_budget);
    }
  } else if (warp < kFirstRoleWarp) {
    // ------------------------------------------------------------ softmax
    set_regs<kRegsLaunch<FP4>, kRegsSoftmax<FP4>>();
    const int s = warp >> 2;               // stream
    const int trow = threadIdx.x & 127;    // row in the 128-row tile (TMEM lane)
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;  // 32 lanes a warp
    const uint32_t tS = tmem + lane_base + s * 128, tO = tmem + lane_base + 256;
    uint32_t base = 0;  // ring slot of the run's (or two-block piece's) first tile
    uint32_t run = 0;   // steps of the run before this piece
    uint32_t n = 0, steps = 0;

    while (true) {
      ok = __all_sync(0xffffffffu, mbar_wait(&q_full[n & 1], (n >> 1) & 1u, abort_flag, tp.wait_budget));
      if (!ok) break;
      const PieceInfo c = infos[n & 3];
      float scale = p.scale_log2;
      if (FP4) scale = ((const float*)(smem + Lo::kOffScale))[(c.rows > tp.tile_rows ? s : (int)(n & 1)) * 128 + trow];
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[n & 1]);
      if (c.nt == 0) break;
      const bool two = c.rows > tp.tile_rows;
      const int a = two ? s * tp.tile_rows + trow : trow;  // row of the block
      const bool live = trow < tp.tile_rows && a < c.rows;
      const bool warp_live = (two ? s * tp.tile_rows : 0) + (warp & 3) * 32 < c.rows;
      // Keys the row sees (rows past the block's: their scores are left as they
      // are, since a mask would slow the whole warp, and they are never read).
      const int lim = live ? c.lim + (c.row0 + a) / p.a.G : 0x7fffffff;
      float m = FP4 ? -kBelow : 0.0f, l = 0.0f;  // the reference in use, and the sum relative to it
      bool first = true;
      // This stream's tiles: all with two row blocks, else those on steps of its parity.
      for (int j = two ? 0 : (int)((s ^ run) & 1u); j < c.nt; j += two ? 1 : 2) {
        const int k0 = (c.t0 + j) * kTN;
        ok = __all_sync(0xffffffffu,
                        mbar_wait(&s_full[s], steps & 1u, abort_flag, tp.wait_budget));
        ++steps;
        if (!ok) break;
        tc_fence_after();
        if (FP4 && (warp & 3) == 0 && lane == 0 && (!two || s == 1)) {  // K's slot
          const uint32_t i = two ? j : run + j;
          mbar_arrive(&kv_empty[(two || i == 0 ? base + 2 * i : base + 2 * i - 1) % Lo::kStages]);
        }
        bool early = false;  // P's first kEarly keys are handed over
        if (warp_live) {
          const int vis = lim - k0;  // keys of the tile that the row sees
          if constexpr (FP4) {
            // Two passes over S, the maximum and the probabilities: m is set before any of P is
            // written, which fp16's range asks for, and the threads get by with few registers.
            // Loops, and masks written into S beforehand: what the roles execute at a time has to
            // fit the SM's instruction cache.  (Unrolled, with the masks in line: verify 355 us for 265.)
            uint32_t xa[16], xb[16];
            if (__any_sync(0xffffffffu, vis < kTN)) {
#pragma unroll 1
              for (int k = 0; k < kTN; k += 16) {
                tmem_ld16(tS + k, xa);
                tmem_wait_ld16(xa);
                mask_from<16>(xa, vis - k);
                tmem_st16(tS + k, xa);
              }
              tmem_wait_st();
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            auto largest = [&](const uint32_t* x) {
#pragma unroll
              for (int i = 0; i < 16; i += 2)
                top[i / 2 & 3] = fmax3(top[i / 2 & 3], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            };
            tmem_ld16(tS, xa);
#pragma unroll 1
            for (int k = 0; k < kTN; k += 32) {
              tmem_wait_ld16(xa);
              tmem_ld16(tS + k + 16, xb);
              largest(xa);
              tmem_wait_ld16(xb);
              tmem_ld16(tS + (k + 32) % kTN, xa);  // (at last the first again)
              largest(xb);
            }
            const float mx = fmax3(fmaxf(top[0], top[1]), top[2], top[3]) * scale;
            const bool grow = live && out_of_range<true>(mx, m, l == 0.0f);
            if (__any_sync(0xffffffffu, grow)) {
              const float mn = grow ? mx - kBelow : m;
              const float f = grow && l != 0.0f ? ex2(m - mn) : 1.0f;
              tmem_wait_ld16(xa);
              if (!first) {  // (before, O is the piece before's, whose products may go on)
#pragma unroll 1
                for (int k = 0; k < DP; k += 16) {
                  tmem_ld16(tO + s * 128 + k, xb);
                  tmem_wait_ld16(xb);
#pragma unroll
                  for (int i = 0; i < 16; ++i) xb[i] = __float_as_uint(__uint_as_float(xb[i]) * f);
                  tmem_st16(tO + s * 128 + k, xb);
                }
              }
              l *= f;
              m = mn;
            }
            const f32x2 sc2 = pack2(scale, scale), ms2 = pack2(-m, -m);
            f32x2 sum2[2] = {0ull, 0ull};
            auto chunk = [&](const uint32_t* x, int k) {
              uint32_t pk[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float y0, y1;
                unpack2(fma2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), sc2, ms2), y0, y1);
                const float e0 = ex2(y0), e1 = ex2(y1);
                sum2[i & 1] = add2(sum2[i & 1], pack2(e0, e1));
                pk[i] = pack_half(e0, e1);
              }
              tmem_st8(tS + k / 2, pk);  // (over scores that are read by then)
            };
#pragma unroll 1
            for (int k = 0; k < kTN; k += 32) {
              tmem_wait_ld16(xa);
              tmem_ld16(tS + k + 16, xb);
              if (k == kEarly) {  // the first keys are written
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&h_full[s]);
              }
              chunk(xa, k);
              tmem_wait_ld16(xb);
              if (k + 32 < kTN) tmem_ld16(tS + k + 32, xa);
              chunk(xb, k + 16);
            }
            early = true;
            float s0, s1;
            unpack2(add2(sum2[0], sum2[1]), s0, s1);
            l += s0 + s1;
          } else {
          // (By the piece's tile as well: V is looked through before any warp hands P
          // over early.  By that alone the compiler spills 100 bytes: verify 196 us.)
          const bool masked = __any_sync(0xffffffffu, vis < kTN || j >= c.masked);
          // One pass: probabilities against the reference in use, and this tile's
          // maximum beside them.  They stand unless a row's maximum is out of range.
          // A tile without a mask hands over its first kEarly keys on the way; if a
          // row's maximum turns out to lie out of range after that, their product
          // is waited for and O rescaled.  Returns whether P stands.
          auto one_pass = [&](auto with_mask) {
            uint32_t pk[64], xa[32], xb[32];
            const f32x2 sc2 = pack2(p.scale_log2, p.scale_log2), ms2 = pack2(-m, -m);
            f32x2 sum2[2] = {0ull, 0ull};
            float mx = -INFINITY;
            auto chunk = [&](const uint32_t* v, uint32_t* out, int k) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float v0 = __uint_as_float(v[2 * i]), v1 = __uint_as_float(v[2 * i + 1]);
                if (with_mask) {
                  v0 = k + 2 * i < vis ? v0 : -INFINITY;
                  v1 = k + 2 * i + 1 < vis ? v1 : -INFINITY;
                }
                mx = fmax3(mx, v0, v1);
                float y0, y1;
                unpack2(fma2(pack2(v0, v1), sc2, ms2), y0, y1);
                const float e0 = ex2(y0), e1 = ex2(y1);
                sum2[i & 1] = add2(sum2[i & 1], pack2(e0, e1));
                out[i] = pack_bf16(e0, e1);
              }
            };
            auto add_sums = [&](f32x2 sums) {
              float s0, s1;
              unpack2(sums, s0, s1);
              l += s0 + s1;
            };
            tmem_ld32(tS, xa);
            tmem_wait_ld32(xa);
            tmem_ld32(tS + 32, xb);
            chunk(xa, pk, 0);
            tmem_wait_ld32(xb);
            tmem_ld32(tS + 64, xa);
            chunk(xb, pk + 16, 32);
            tmem_wait_ld32(xa);
            tmem_ld32(tS + 96, xb);
            chunk(xa, pk + 32, 64);
            if (with_mask) {
              tmem_wait_ld32(xb);
              chunk(xb, pk + 48, 96);
              if (__any_sync(0xffffffffu, live && out_of_range<false>(mx * p.scale_log2, m, first))) return false;
              tmem_st32(tS, pk);
              tmem_st32(tS + 32, pk + 32);
              add_sums(add2(sum2[0], sum2[1]));
              return true;
            }
            const f32x2 early_sum = add2(sum2[0], sum2[1]);
            sum2[0] = sum2[1] = 0ull;
            const bool bad = __any_sync(0xffffffffu, live && out_of_range<false>(mx * p.scale_log2, m, first));
            tmem_wait_ld32(xb);
            if (bad) return false;
            tmem_st32(tS, pk);
            tmem_st16(tS + 32, pk + 32);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&h_full[s]);
            early = true;
            chunk(xb, pk, 96);
            mx *= p.scale_log2;
            if (__any_sync(0xffffffffu, live && out_of_range<false>(mx, m, false))) {
              add_sums(early_sum);
              return false;
            }
            tmem_st16(tS + 48, pk);
            add_sums(add2(early_sum, add2(sum2[0], sum2[1])));
            return true;
          };
          const bool done = masked ? one_pass(std::true_type{}) : one_pass(std::false_type{});
          if (!done) {
            // Two passes over S: the maximum, then the probabilities.  After a first
            // part that stands only the rest is left (its part of S is intact).
            const int from = early ? kEarly : 0;
            if (early) {
              ok = __all_sync(0xffffffffu, mbar_wait(&h_done[s], (steps - 1) & 1u, abort_flag,
                                                     tp.wait_budget));
              if (!ok) break;
              tc_fence_after();
            }
            uint32_t x[32];
            float mx = -INFINITY;
#pragma unroll 1
            for (int k = from; k < kTN; k += 32) {
              tmem_ld32(tS + k, x);
              tmem_wait_ld32(x);
              if (masked) mask_from<32>(x, vis - k);
#pragma unroll
              for (int i = 0; i < 32; i += 2)
                mx = fmax3(mx, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            }
            mx *= p.scale_log2;
            const bool fresh = first && !early;  // nothing is summed yet
            const bool grow = live && out_of_range<false>(mx, m, fresh);
            if (__any_sync(0xffffffffu, grow)) {
              const float mn = grow ? mx : m;
              const float f = grow && !fresh ? ex2(m - mn) : 1.0f;
              if (!fresh) {
#pragma unroll
                for (int k = 0; k < DP; k += 32) {
                  tmem_ld32(tO + s * 128 + k, x);
                  tmem_wait_ld32(x);
#pragma unroll
                  for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                  tmem_st32(tO + s * 128 + k, x);
                }
              }
              l *= f;
              m = mn;
            }
            // (P's columns k / 2 .. lie over scores that are read by then)
#pragma unroll 1
            for (int k = from; k < kTN; k += 32) {
              uint32_t pk[16];
              float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              tmem_ld32(tS + k, x);
              tmem_wait_ld32(x);
              if (masked) mask_from<32>(x, vis - k);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float e0 = ex2(fmaf(__uint_as_float(x[2 * i]), p.scale_log2, -m));
                const float e1 = ex2(fmaf(__uint_as_float(x[2 * i + 1]), p.scale_log2, -m));
                sum[i & 3] += e0 + e1;
                pk[i] = pack_bf16(e0, e1);
              }
              tmem_st16(tS + k / 2, pk);
              l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            }
          }
          }
          first = false;
          tmem_wait_st();
        }
        tc_fence_before();
        // V rows past the item's end, and those that are not finite where not all
        // rows see them, become zeros (by the stream that multiplies first).
        if (!FP4 && j >= c.masked && (!two || s == 0)) {
          const int all_see = infos[n & 3].all_see, end = infos[n & 3].end;
          const uint32_t i = run + j;
          const uint32_t sl = base + (two ? 2 * j + 1 : j + 1 < c.nt || c.next_joined ? 2 * i + 2 : 2 * i + 1);
          const int stage = (int)(sl % Lo::kStages);
          ok = __all_sync(0xffffffffu, mbar_wait(&kv_full[stage], (sl / Lo::kStages) & 1u, abort_flag,
                                                 tp.wait_budget));
          if (!ok) break;
          const int key = k0 + trow;
          // (16-byte chunks in an order of the row's own: free of bank conflicts)
          uint8_t* v = smem + Lo::kOffRing + stage * Lo::kTileBytes + trow * 128;
          auto chunk_of = [&](int i) {
            return (uint4*)(v + (i >> 3) * Lo::kHalfBytes + (((i ^ trow) & 7) << 4));
          };
          bool clear = key >= end;
          if (key >= all_see && !clear) {
            uint32_t bad = 0;  // an exponent of all ones carries into bit 15 or 31
#pragma unroll
            for (int i = 0; i < Lo::kHalves * 8; ++i) {
              const uint4 x = *chunk_of(i);
              bad |= ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
                     ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
            }
            clear = bad & 0x80008000u;
            if (clear)
              atomicMax(&bad_v[n & 1], (unsigned long long)(n + 1) << 32 | (uint32_t)(0x7fffffff - key));
          }
          if (clear) {
#pragma unroll
            for (int i = 0; i < Lo::kHalves * 8; ++i) *chunk_of(i) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) {
          if (!early) mbar_arrive(&h_full[s]);
          mbar_arrive(&p_full[s]);
        }
      }
      if (!ok) break;
      // (m, l) to the result warps, once they have read the piece before's.
      if (n > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(ml_empty, (n - 1) & 1u, abort_flag, tp.wait_budget));
        if (!ok) break;
      }
      merge[s * 128 + trow] = make_float2(l == 0.0f ? -INFINITY : m, l);  // (no key seen: no weight)
      __syncwarp();
      if (lane == 0) mbar_arrive(ml_full);
      if (two) {
        base += 2 * c.nt;
      } else {
        run += c.nt;
        if (!c.next_joined) {
          base += 2 * run;
          run = 0;
        }
      }
      ++n;
    }
  } else if (warp >= kResultWarp) {
    // ------------------------------------------------------------ results
    set_regs<kRegsLaunch<FP4>, kRegsResult<FP4>>();
    const int trow = threadIdx.x & 127;
    const uint32_t tO = tmem + ((uint32_t)(warp & 3) << 21) + 256;
    const int D = p.a.c.head_dim, G = p.a.G;
    uint32_t n = 0, run = 0;
    // (4-bit) Piece q's rows of Q as fp16, a row times the power of two that brings its largest to
    // 2^14 .. 2^15; the scores' factor takes it back.  Four lanes a row.
    auto load_q = [&](uint32_t q) {
      if (!__all_sync(0xffffffffu, mbar_wait_idle(&i_full[q & 1], (q >> 1) & 1u, abort_flag, tp.wait_budget, 64)))
        return false;
      const int rows = infos[q & 3].rows, row0 = infos[q & 3].row0, h = infos[q & 3].h, q0 = infos[q & 3].q0;
      const bool two = rows > tp.tile_rows;
      const uint32_t tile = smem_addr(smem + Lo::kOffQ) + (two ? 0 : (q & 1) * Lo::kTileBytes);
      float* scales = (float*)(smem + Lo::kOffScale) + (two ? 0 : (q & 1) * 128);
      const int part = lane & 3;
      constexpr int kChunks = DP / 32;  // of a lane: columns 8 (part + 4 j) ..
      for (int a0 = (warp & 3) * 8; a0 < rows; a0 += 32) {
        const int a = a0 + (lane >> 2);
        const bool live = a < rows;
        uint4 x[kChunks];
        const int tok = tp.by_g(row0 + (live ? a : 0)), g = row0 + (live ? a : 0) - tok * G;
        const uint16_t* src = (const uint16_t*)p.a.q + (long long)(q0 + tok) * p.a.q_token_stride +
                              (long long)(h * G + g) * p.a.q_head_stride + part * 8;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
          x[j] = make_uint4(0u, 0u, 0u, 0u);
          if (live && 32 * j < D) {
            const uint16_t* e = src + 32 * j;
            x[j] = tp.q_vec ? *(const uint4*)e
                            : make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16,
                                         e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
          }
        }
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
          const uint32_t w4[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) top = max(top, max(w4[i] & 0x7fffu, (w4[i] >> 16) & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int field = (int)(top >> 7), up = field == 255 ? 127 : min(268 - field, 253);
        const float f = __uint_as_float((uint32_t)up << 23) * tp.sign;
        const int blk = a >> 7, t = a & 127;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
          uint32_t w4[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w4[i] = pack_half(__uint_as_float(w4[i] << 16) * f, __uint_as_float(w4[i] & 0xffff0000u) * f);
          const int c = part + 4 * j;
          if (live)
            st_shared16(tile + blk * Lo::kTileBytes + (c >> 3) * Lo::kHalfBytes + swz(t, c & 7), w4[0], w4[1], w4[2], w4[3]);
        }
        // (not 0: a masked score is -inf times this)
        if (live && part == 0)
          scales[a] = fmaxf(__uint_as_float((uint32_t)(254 - up) << 23) * p.scale_log2, 1e-37f);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[q & 1]);
      return true;
    };
    if (FP4) ok = load_q(0);
    while (true) {
      if (!FP4)
        ok = __all_sync(0xffffffffu, mbar_wait_idle(&q_full[n & 1], (n >> 1) & 1u, abort_flag, tp.wait_budget, 64));
      if (!ok) break;
      const PieceInfo c = infos[n & 3];
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[n & 1]);
      if (FP4 && c.nt != 0 && !(ok = load_q(n + 1))) break;
      if (c.nt == 0) break;
      const bool two = c.rows > tp.tile_rows;
      ok = __all_sync(0xffffffffu, mbar_wait_idle(ml_full, n & 1u, abort_flag, tp.wait_budget, 64));
      if (!ok) break;
      const int s0 = two ? 0 : (int)(run & 1u);  // the stream of a one-block piece's first tile
      float2 x0 = merge[s0 * 128 + trow];
      const float2 x1 = merge[(s0 ^ 1) * 128 + trow];
      unsigned long long bad = FP4 ? 0ull : *(volatile unsigned long long*)&bad_v[n & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(ml_empty);
      ok = __all_sync(0xffffffffu,
                      mbar_wait_idle(&o_full[n & 1], (n >> 1) & 1u, abort_flag, tp.wait_budget, 64));
      if (!ok) break;
      tc_fence_after();
      if (FP4) bad = *(volatile unsigned long long*)&bad_v[n & 3];  // (all of the piece's V are decoded)
      const int bad_from = bad >> 32 == n + 1 ? 0x7fffffff - (int)(uint32_t)bad : 0x7fffffff;
      float w0 = 1.0f, w1 = 0.0f;  // weights of the two streams' O
      const bool both = !two && c.nt > 1;
      if (!two) {
        const float m = fmaxf(x0.x, x1.x), ms = m == -INFINITY ? 0.0f : m;
        w0 = ex2(x0.x - ms);
        w1 = ex2(x1.x - ms);
        x0 = make_float2(m, x0.y * w0 + x1.y * w1);
      }
      for (int blk = 0; blk < (two ? 2 : 1); ++blk) {
        if (blk == 1) {  // the first block's O may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_free[0]);
        }
        const float m = blk ? x1.x : x0.x;
        float l = blk ? x1.y : x0.y;
        const int a = blk * tp.tile_rows + trow;
        if (blk * tp.tile_rows + (warp & 3) * 32 >= c.rows) continue;  // (arrives below)
        const bool live = trow < tp.tile_rows && a < c.rows;
        const unsigned row = c.row0 + a, tok = row / (unsigned)G, g = row - tok * G;
        if (c.lim + (int)tok > bad_from) l = __int_as_float(0x7fc00000);
        const size_t orow = (size_t)(c.q0 + tok) * p.a.Hq + c.h * G + g;
        const size_t prow = ((size_t)blockIdx.x * 2 + (c.slot < 0 ? 0 : c.slot)) * kMR + a;
        const float inv = c.slot >= 0 ? 1.0f : l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
        const uint32_t own = tO + (uint32_t)(two ? blk : s0) * 128;
        const float f0 = FP4 ? w0 * inv * p.a.v_factor : w0 * inv, f1 = FP4 ? w1 * inv * p.a.v_factor : w1 * inv;
        // 16 columns at a time from both streams, or 32 from one.
        auto store16 = [&](const uint32_t* o, int k) {
          if (!live) return;
          if (c.slot < 0) {
            uint4* out = (uint4*)((__nv_bfloat16*)p.a.out + orow * D + k);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (k + 8 * i < D) {
                uint32_t v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  v[q] = pack_bf16(__uint_as_float(o[8 * i + 2 * q]), __uint_as_float(o[8 * i + 2 * q + 1]));
                out[i] = make_uint4(v[0], v[1], v[2], v[3]);
              }
            }
          } else {
            uint4* out = (uint4*)(p.part + prow * D + k);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (k + 4 * i < D) out[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        };
        if (both) {
#pragma unroll 1
          for (int k = 0; k < DP; k += 16) {
            uint32_t o[16], o1[16];
            tmem_ld16(own + k, o);
            tmem_ld16((own ^ 128u) + k, o1);  // the other stream's: the base is 256-aligned
            tmem_wait_ld16(o);
            tmem_wait_ld16(o1);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * f0 + __uint_as_float(o1[i]) * f1);
            store16(o, k);
          }
        } else {
#pragma unroll 1
          for (int k = 0; k < DP; k += 32) {
            uint32_t o[32];
            tmem_ld32(own + k, o);
            tmem_wait_ld32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f0);
            store16(o, k);
            store16(o + 16, k + 16);
          }
        }
        if (live) {
          if (c.slot < 0)
            p.a.lse[orow] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
          else
            p.stats[prow] = make_float2(m, l);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (!two) mbar_arrive(&o_free[0]);
        mbar_arrive(&o_free[1]);
      }
      run = two || !c.next_joined ? 0 : run + c.nt;
      ++n;
    }
  } else if (warp == kLoaderWarp) {
    // ------------------------------------------------------------ loader
    set_regs<kRegsLaunch<FP4>, kRegsOther<FP4>>();
    AttnWalk<kTN> w = st->walk;
    const int D = p.a.c.head_dim, G = p.a.G;
    bool prev_two = false;
    uint32_t n = 0;
    for (;; ++n) {
      const bool end = w.done();
      PieceInfo c;
      c.t0 = end ? 0 : w.first_tile();
      c.nt = end ? 0 : w.last_tile() - c.t0;
      c.rows = end ? 0 : w.block_rows(p);
      c.row0 = w.m * p.mr;
      c.h = w.h;
      c.q0 = w.q.q0;
      c.lim = w.q.L - w.q.n + 1;
      c.all_see = c.lim + c.row0 / G;
      c.masked = (c.all_see > 0 ? c.all_see / kTN : 0) - c.t0;
      c.end = w.end;
      c.slot = end ? 0 : attn_slot(w);
      c.next_joined = 0;
      const bool two = c.rows > tp.tile_rows;
      // The Q tile(s) of this piece and its info slot are free again: piece n - 2
      // is done with them, and piece n - 1 where either of the two takes both.
      if (n >= 2)
        ok = __all_sync(0xffffffffu, mbar_wait_idle(&q_empty[n & 1], ((n - 2) >> 1) & 1u, abort_flag,
                                                    tp.wait_budget));
      if (ok && n >= 1 && (two || prev_two))
        ok = __all_sync(0xffffffffu, mbar_wait_idle(&q_empty[(n - 1) & 1], ((n - 1) >> 1) & 1u,
                                                    abort_flag, tp.wait_budget));
      if (!ok) break;
      uint8_t* tile = smem + Lo::kOffQ + (two ? 0 : (int)(n & 1) * Lo::kTileBytes);
      if (!end) {
        w.next(p, flags);
        c.next_joined = !two && !w.done() && w.block_rows(p) <= tp.tile_rows;
      }
      if (lane == 0) infos[n & 3] = c;
      if (end) {
        __syncwarp();
        if (lane == 0) mbar_arrive(FP4 ? &i_full[n & 1] : &q_full[n & 1]);
        break;
      }
      if constexpr (FP4) {  // (the results' warps load the rows)
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_full[n & 1]);
      } else if (tp.q_tma) {
        // One box a tile and half: q_tokens tokens x G heads, the tile's rows in
        // order (tokens past the chunk's bring rows that are not read).
        if (lane == 0) {
          const int boxes = (two ? 2 : 1) * Lo::kHalves;
          const uint32_t bytes = (uint32_t)tp.tile_rows * 128u;
          mbar_expect_tx(&q_full[n & 1], boxes * bytes);
          const int tok = c.q0 + c.row0 / G;
          for (int b = 0; b < boxes; ++b) {
            const int blk = b / Lo::kHalves, half = b % Lo::kHalves;
            tma_load_3d(tile + blk * Lo::kTileBytes + half * Lo::kHalfBytes, &tmQ, half * 64, c.h * G,
                        tok + blk * tp.q_tokens, &q_full[n & 1]);
          }
        }
      } else {
        // Element by element into the swizzled tiles; columns past D are zero
        // (K's are, by the tensor map's fill).
        for (int i = lane; i < c.rows * DP; i += 32) {
          const int a = i / DP, d = i % DP;
          const unsigned row = c.row0 + a, tok = row / (unsigned)G, g = row - tok * G;
          unsigned short x = 0;
          if (d < D) {
            x = __bfloat16_as_ushort(
                ((const __nv_bfloat16*)p.a.q)[(long long)(c.q0 + tok) * p.a.q_token_stride +
                                              (long long)(c.h * G + g) * p.a.q_head_stride + d]);
            if (tp.sign < 0.0f) x ^= 0x8000u;
          }
          const int blk = a >= tp.tile_rows ? 1 : 0, t = a - blk * tp.tile_rows;
          *(unsigned short*)(tile + blk * Lo::kTileBytes + (d >> 6) * Lo::kHalfBytes +
                             swz(t, (d >> 3) & 7) + (d & 7) * 2) = x;
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[n & 1]);
      }
      prev_two = two;
    }
    if (!FP4 && !ok && tp.q_tma && lane == 0)  // the loads that may still be in flight
      for (uint32_t i = n >= 2 ? n - 2 : 0; i < n; ++i)
        mbar_drain(&q_full[i & 1], (i >> 1) & 1u, tp.wait_budget);
  } else {  // (4-bit: none)
    set_regs<kRegsLaunch<FP4>, kRegsOther<FP4>>();
    if (lane == 0) attn_write_cut(p, *st);
  }
  if (*abort_flag && lane == 0) flag_status(flags, DSPARK_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) p.flags[blockIdx.x] = *flags;
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                 : "memory");
  }
}

PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (PFN_cuTensorMapEncodeTiled_v12000)ptr;
  });
  return fn;
}

// K or V as (head_dim, token in page, head, page); boxes of 64 columns and box_tokens tokens.
bool encode_cache(CUtensorMap* map, const void* base, const CacheView& c, int box_tokens) {
  const auto fn = get_encode();
  if (!fn) return false;
  // The stride of a dimension of size 1 is not used: any valid one.
  const cuuint64_t tok = c.page_size == 1 ? 16 : (cuuint64_t)c.token_stride * 2;
  const cuuint64_t head = c.heads == 1 ? 16 : (cuuint64_t)c.head_stride * 2;
  const cuuint64_t page = c.n_pages == 1 ? 16 : (cuuint64_t)c.page_stride * 2;
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.heads,
                              (cuuint64_t)c.n_pages};
  const cuuint64_t strides[3] = {tok, head, page};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_tokens, 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
            one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q as (head_dim, head, token); boxes of 64 columns, G heads and `tokens` tokens.
bool encode_q(CUtensorMap* map, const AttnArgs& a, int tokens) {
  const auto fn = get_encode();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)a.c.head_dim, (cuuint64_t)a.Hq, (cuuint64_t)a.a.n_tokens};
  const cuuint64_t strides[2] = {a.Hq == 1 ? 16 : (cuuint64_t)a.q_head_stride * 2,
                                 a.a.n_tokens == 1 ? 16 : (cuuint64_t)a.q_token_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)tokens};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box,
            one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
  const int n = device_sms();
  return n < kMaxCtas ? n : kMaxCtas;
}

template <int DP, bool FP4>
cudaError_t launch(const TcParams& tp, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q,
                   cudaStream_t s) {
  const cudaError_t attr =
      once_per_device([] { return allow_smem(attention_tc_kernel<DP, FP4>, Layout<DP, FP4>::kBytes); });
  if (attr != cudaSuccess) return attr;
  cudaLaunchAttribute attr_pdl;
  const cudaLaunchConfig_t cfg =
      overlapped_launch(dim3(sm_count()), kThreads<FP4>, Layout<DP, FP4>::kBytes, s, &attr_pdl);
  return cudaLaunchKernelEx(&cfg, attention_tc_kernel<DP, FP4>, k, v, q, tp);
}

}  // namespace

// The tensor-core kernel takes bf16 with head_dim a multiple of 8 up to 128 (two
// 64-column halves of 128-byte rows), pages of any multiple of 8 tokens (whole
// 8-row swizzle groups: a box is the largest power of two in the page size, up to
// the 128 keys of a tile), and what TMA asks of addresses and strides (16 bytes).
// (A call without tokens, which only checks its offsets, needs no map of q.)
bool attention_tc_supported(const AttnArgs& a) {
  const CacheView& c = a.c;
  if (a.a.n_tokens == 0) return false;
  if (a.dtype != DSPARK_BF16 || c.head_dim % 8 != 0 || c.head_dim > 128) return false;
  if (c.page_size % 8 != 0) return false;  // (a tile is at most 16 boxes of 8 tokens, two halves each)
  if (((uintptr_t)c.k | (uintptr_t)c.v) & 15u) return false;
  const long long most = 1ll << 39;  // elements: 2^40 bytes
  if (c.token_stride % 8 != 0 || c.token_stride >= most) return false;
  if (c.heads > 1 && (c.head_stride % 8 != 0 || c.head_stride >= most)) return false;
  if (c.n_pages > 1 && (c.page_stride % 8 != 0 || c.page_stride >= most)) return false;
  return get_encode() != nullptr;
}

// Over a 4-bit cache: head_dim up to 128, bf16 queries.
bool attention_tc_fp4_supported(const AttnArgs& a) {
  return a.fp4 && a.dtype == DSPARK_BF16 && a.c.head_dim <= 128 && a.a.n_tokens > 0;
}

cudaError_t launch_attention_tc_fp4(const AttnArgs& a, char* ws, cudaStream_t s) {
  const AttnWorkspace w = attn_workspace_layout(kMR, a.c.head_dim, kMaxCtas);
  TcParams tp(a);
  tp.p = AttnParams{a, (int*)ws, (int*)(ws + w.flags), (CutItem*)(ws + w.cuts),
                    (float2*)(ws + w.stats), (float*)(ws + w.out), fabsf(a.scale) * 1.4426950408889634f,
                    attn_item_units(a), kMR};
  tp.sign = a.scale < 0 ? -1.0f : 1.0f;
  tp.tile_rows = 128;
  tp.q_vec = ((uintptr_t)a.q & 15u) == 0 && a.q_head_stride % 8 == 0 && a.q_token_stride % 8 == 0;
  tp.wait_budget = kWaitBudget;
  const CUtensorMap none = {};
  const cudaError_t e = a.c.head_dim <= 64 ? launch<64, true>(tp, none, none, none, s)
                                           : launch<128, true>(tp, none, none, none, s);
  return e != cudaSuccess ? e : launch_attn_combine(tp.p, kMR, sm_count(), s);
}

size_t attention_tc_workspace_bytes(int head_dim) { return attn_workspace_layout(kMR, head_dim, kMaxCtas).total; }

cudaError_t launch_attention_tc(const AttnArgs& a, char* ws, cudaStream_t s) {
  const AttnWorkspace w = attn_workspace_layout(kMR, a.c.head_dim, kMaxCtas);
  TcParams tp(a);
  tp.p = AttnParams{a, (int*)ws, (int*)(ws + w.flags), (CutItem*)(ws + w.cuts),
                    (float2*)(ws + w.stats), (float*)(ws + w.out),
                    // (not 0: a masked score is -inf times this)
                    fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-37f),
                    attn_item_units(a), kMR};
  tp.sign = a.scale < 0 ? -1.0f : 1.0f;
  tp.box_tokens = a.c.page_size & -a.c.page_size;
  if (tp.box_tokens > kTN) tp.box_tokens = kTN;
  tp.q_tokens = a.G <= 128 ? 128 / a.G : 1;
  tp.tile_rows = a.G <= 128 ? tp.q_tokens * a.G : 128;
  tp.p.mr = 2 * tp.tile_rows;
  const long long most = 1ll << 39;
  tp.q_tma = a.G <= 128 && a.scale >= 0 && ((uintptr_t)a.q & 15u) == 0 &&
             (a.Hq == 1 || (a.q_head_stride % 8 == 0 && a.q_head_stride > 0 && a.q_head_stride < most)) &&
             (a.a.n_tokens == 1 ||
              (a.q_token_stride % 8 == 0 && a.q_token_stride > 0 && a.q_token_stride < most));
  tp.wait_budget = kWaitBudget;
  CUtensorMap mk, mv, mq = {};
  if (!encode_cache(&mk, a.c.k, a.c, tp.box_tokens) || !encode_cache(&mv, a.c.v, a.c, tp.box_tokens))
    return cudaErrorInvalidValue;
  if (tp.q_tma && !encode_q(&mq, a, tp.q_tokens)) return cudaErrorInvalidValue;
  cudaError_t e = a.c.head_dim <= 64 ? launch<64, false>(tp, mk, mv, mq, s) : launch<128, false>(tp, mk, mv, mq, s);
  if (e != cudaSuccess) return e;
  return launch_attn_combine(tp.p, kMR, sm_count(), s);
}

}  // namespace dspark
