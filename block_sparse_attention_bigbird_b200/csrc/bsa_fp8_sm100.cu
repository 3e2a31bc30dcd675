// Product of 8-bit matrices with a scale for each block of 128, for B200 (sm_100a):
//
//     out[m, n] = sum_kb sa[m, kb] sb[n, kb] ( sum_{k in block kb} a[m, k] b[n, k] ) + bias[n].
//
// The scale of a block multiplies a finished partial sum, so the sum over 128 products stays
// in the tensor cores and the sum over blocks is done in fp32 by threads, each block's
// partial read from TMEM and added with its scale by one fma an element.
//
// bsa_fp8_mma_kernel, for more than 8 rows.  Persistent, one CTA per SM, 384 threads.  A
// unit of work is a tile of 128 rows by kBN columns, over all of K or one of `splits` ranges
// of blocks.
//   warp 0     TMA producer: per block of K (128 bytes: one 128-byte swizzle atom) the A box
//              (128 rows) and the B box (kBN rows) into a ring of shared-memory stages.
//   warps 1-2  MMA issuers, taking blocks in turn: four tcgen05.mma (kind::f8f6f4, M = 128,
//              N = kBN, K = 32) a block into one of 512 / kBN accumulators, from 0 each.
//   warp 3     scales, four blocks at a time, two such batches in shared memory.
//   warps 4-11 keep the tile's sums in registers, read each accumulator with tcgen05.ld as its
//              MMAs complete, hand it back and add it with its scales; at a tile's end they
//              add the bias and write.  With a scale for 128 rows of b a thread owns a row of
//              half the columns and its scale is one number a block (the 32x32b form).  With a
//              scale for each row of b (kBRows) that form would need 128 column scales a thread
//              and block; in the 16x128b form a thread has one column of every four and four
//              rows, so 32 column scales and four row scales.
// Cycles a block of a 128 x 256 tile, measured: its MMAs 512; the eight warps' reads of TMEM 160
// (16x128b 277, 16x256b 521), their additions 340 (kBRows 540: two operations a pair), waits and
// hand-overs about 350.  Reads and additions hardly overlap, as the two warps of a scheduler wait
// for the same accumulator, so the adding warps are what bounds long products: about 1000 cycles,
// kBRows 1300.  Their reads and additions alone would fit under the MMAs (kBRows would not): it is
// the waits in series with them that do not.  65536 x 2304 x 768 takes 141 us (1.65 PFLOP/s; without its loads 128, without
// writing 124), 8192^3 524 us (2.10 PFLOP/s, at the power limit), 2304 x 768 x 65536 with
// kBRows 159 us (1.46 PFLOP/s).
// What follows from it.  An issuer whose loop is uniform over the warp and elects a lane for the
// MMAs alone takes half the time of a single thread's loop, whose descriptors have to be moved to
// uniform registers after every wait (513 cycles a block, 711 to 851); two of them hide the waits.
// Registers may hardly spill: with the shared memory taken, L1 is too small to hold them (256
// columns with kBRows spill 16 bytes, the other forms none).  Both halves
// of the columns run the same code (a copy for each took 147 us instead of 141).  Halves with
// MMAs of N = 128 and accumulators of their own took 155 us: at that width shared memory cannot
// feed the tensor cores.
//
// bsa_fp8_rows_kernel, for up to 8 rows (tokens).  There the time is that of reading b once.
// A block of threads takes 16 rows of b at a time, its warps an equal share of K's blocks each;
// every warp brings its part of b with cp.async, kRowsAhead blocks of K ahead and over the end
// of one 16-row tile into the next, so that the loads in flight do not depend on registers.
// Codes are widened to fp16, which holds every e4m3 and e5m2 value, and multiplied by mma.sync
// m16n8k16 with b as the 16-row side and the tokens as the 8 columns (a tcgen05 tile of 128 rows
// would be 15/16 empty).  The products of a block of 128 are summed in fp32 before their scale;
// the warps' sums meet in shared memory in a fixed order.
// 4 x 8192 x 8192 (67 MB of b) takes 16.9 us in a graph, a loop that only reads b 11 us: its 512
// tiles are three rounds of 148 SMs and one of 68, so that the SMs stand still for 13 % of the
// time, and a short kernel's start and end do the rest.  Where
// the kernels meet, 8 and 9 rows of N = K = 8192 take 17.2 and 19.4 us, of 2304 x 768 2.6 and 4.9:
// eight tokens are what one mma.sync has columns for.
//
// Every wait is bounded; on expiry the CTA records BSA_ERR_DEVICE_TIMEOUT, drains its copies
// and MMAs, frees TMEM and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "sm100_ptx.cuh"
#include "bsa_wait.cuh"
#include "bsa_elem.cuh"
#include "bsa_host_cuda.h"

namespace bsa {
namespace {

constexpr int kMThreads = 384;
constexpr int kMB = 128;   // tile rows (TMEM lanes)
constexpr int kKB = 128;   // block of K: bytes, products and scales
constexpr int kIssueWarp0 = 1, kIssuers = 2, kScaleWarp = 3, kPromoteWarp0 = 4, kPromoteWarps = 8;
constexpr int kBatch = 4;  // blocks whose scales come together
constexpr uint32_t kTmem = 512;

template <int kBN, bool kBRows>
struct MmaCfg {
  // With kBRows results leave from registers; else a warp's 32 rows of bf16 results have room
  // in shared memory and leave by TMA while the next tile is added, for which a stage is given
  // up (K is short where results are most of the bytes).
  static constexpr int kStages = kBN == 256 ? (kBRows ? 4 : 3) : 5;
  static constexpr uint32_t kStgBytes = kBRows ? 0 : 32 * (kBN / 2) * 2;  // a promoting warp's
  static constexpr int kAcc = static_cast<int>(kTmem) / kBN;  // accumulators
  static constexpr uint32_t kABytes = kMB * kKB, kBBytes = kBN * kKB, kStageBytes = kABytes + kBBytes;
  static constexpr uint32_t kStg = kStages * kStageBytes;
  // a block's scales: of 128 rows of a and kBN rows of b, or their products for two halves
  // (kBRows: 128 of a, then of each half of b's rows n the four n % 4, a bank's width apart)
  static constexpr int kColGap = kBN / 8 + 4;
  static constexpr int kScales = kBRows ? kMB + 8 * kColGap : 2 * kMB;
  static constexpr uint32_t kScale = kStg + kPromoteWarps * kStgBytes;  // [2][kBatch][kScales] fp32
  // The bias of a unit's columns, brought with its first batch.  Batches run at most two ahead,
  // so at most two units ahead of the one whose bias is read.
  static constexpr uint32_t kBias = kScale + 2 * kBatch * kScales * 4;  // [4][kBN] fp32
  static constexpr uint32_t kBar = kBias + (kBRows ? 0 : 4 * kBN * 4);
  // barriers: stage full, stage empty, accumulator full, accumulator empty, scales full, scales empty, final
  static constexpr int kFull = 0, kEmpty = kStages, kAccFull = 2 * kStages, kAccEmpty = kAccFull + kAcc,
                       kScFull = kAccEmpty + kAcc, kScEmpty = kScFull + 2, kFinal = kScEmpty + 2,
                       kBars = kFinal + 1;
  static constexpr uint32_t kMisc = kBar + 8 * kBars;
  static constexpr uint32_t kAlloc = kMisc + 16 + 1024;  // + slack for 1024-byte alignment
  static_assert(kAlloc <= 227 * 1024, "shared memory budget");
  static_assert(kIssuers <= kAcc, "an issuer's wait is never a phase behind");
  static_assert(kStageBytes % 1024 == 0 && kStgBytes % 1024 == 0, "swizzle atoms must stay 1024-byte aligned");
};

struct MmaParams {
  CUtensorMap tm_a, tm_b;
  CUtensorMap tm_out;  // boxes of 128 bytes by 32 rows; unused where rows are not multiples of 16 bytes
  int tma_out;
  const float *sa, *sb;
  const void* bias;
  void* out;
  int M, N, kb;         // kb: blocks of K
  int a_shift, b_rows;  // row of sa = m >> a_shift; b_rows: a scale for each row of b
  int bias_f32, out_f32;
  int wide;             // a batch's scales of a row lie in 16 aligned bytes
  int idesc_formats;    // A and B format bits of the instruction descriptor
  int n_tiles, splits, kb_split, units;
  int64_t split_stride;  // elements of one split's partial result (splits > 1: out is fp32 partials)
  uint64_t timeout_ns;
};

__device__ __forceinline__ uint32_t bar_at(uint32_t bars, int i) { return bars + 8u * static_cast<uint32_t>(i); }

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, 8-bit floating point in, fp32 accumulate.
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Waits that poll the barrier a while (a poll lets the thread sleep in hardware for a short
// time) before they take the timed path, whose clock read and call cost more than a block's
// MMAs.
constexpr int kPolls = 64;
__device__ __forceinline__ bool ready(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t timeout_ns) {
  for (int i = 0; i < kPolls; ++i)
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
  return wait_warp(bar, parity, abort_flag, timeout_ns);
}

__device__ __forceinline__ void tma_store_3d(const void* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// 16 lanes of 32 TMEM columns (16x128b, eight times): of column 4 i + lane % 4 the words 2 i in
// row lane / 4 and 2 i + 1 in row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x128b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Ties registers to the preceding tcgen05.wait::ld so their uses stay below it.
__device__ __forceinline__ void reg_fence16(uint32_t (&r)[16]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
               "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// A unit of work: tile (m0, n0) over the blocks [k0, k1) of K.  Column tiles go fastest, so
// that the CTAs of one moment share a few row tiles of A and all of B stays in L2.
struct Unit {
  int m0, n0, k0, k1, split;
};
template <int kBN>
__device__ __forceinline__ Unit unit_of(const MmaParams& p, int u) {
  const int tile = u / p.splits, split = u % p.splits;
  Unit t;
  t.m0 = (tile / p.n_tiles) * kMB;
  t.n0 = (tile % p.n_tiles) * kBN;
  t.k0 = split * p.kb_split;
  t.k1 = min(t.k0 + p.kb_split, p.kb);
  t.split = split;
  return t;
}

// The roles below are run by whole warps (one loop, uniform over the warp); an elected lane
// issues.
template <int kBN, bool kBRows>
__device__ void mma_producer(const MmaParams& p, uint32_t smem, uint32_t bars, volatile int* abort_flag) {
  using C = MmaCfg<kBN, kBRows>;
  const uint64_t pol_a = ptx::policy_evict_first(), pol_b = ptx::policy_evict_last();
  uint32_t it = 0;
  bool alive = true;
  for (int u = blockIdx.x; alive && u < p.units; u += gridDim.x) {
    const Unit t = unit_of<kBN>(p, u);
    for (int kb = t.k0; kb < t.k1; ++kb, ++it) {
      const uint32_t s = it % C::kStages;
      if (it >= C::kStages &&
          !ready(bar_at(bars, C::kEmpty + s), ((it / C::kStages) - 1u) & 1u, abort_flag, p.timeout_ns)) {
        alive = false;
        break;
      }
      const uint32_t full = bar_at(bars, C::kFull + s), dst = smem + s * C::kStageBytes;
      if (elected()) {
        ptx::mbar_arrive_expect_tx(full, C::kStageBytes);
        ptx::tma_load_2d(dst, &p.tm_a, full, kb * kKB, t.m0, pol_a);
        ptx::tma_load_2d(dst + C::kABytes, &p.tm_b, full, kb * kKB, t.n0, pol_b);
      }
      __syncwarp();
    }
  }
  // the last load of each stage has landed before the CTA may exit
  for (uint32_t j = it > C::kStages ? it - C::kStages : 0u; j < it; ++j)
    wait_force(bar_at(bars, C::kFull + static_cast<int>(j % C::kStages)), (j / C::kStages) & 1u, abort_flag,
               p.timeout_ns);
}

template <int kBN, bool kBRows>
__device__ void mma_issuer(const MmaParams& p, uint32_t smem, uint32_t bars, uint32_t tmem, uint32_t which,
                           volatile int* abort_flag) {
  using C = MmaCfg<kBN, kBRows>;
  // bits 4-5 D format (1 = fp32), 7-9 and 10-12 A and B formats, 17-22 N >> 3, 24-28 M >> 4
  const uint32_t idesc = (1u << 4) | static_cast<uint32_t>(p.idesc_formats) | (static_cast<uint32_t>(kBN >> 3) << 17) |
                         (static_cast<uint32_t>(kMB >> 4) << 24);
  uint32_t it = 0;
  bool alive = true;
  for (int u = blockIdx.x; alive && u < p.units; u += gridDim.x) {
    const Unit t = unit_of<kBN>(p, u);
    for (int kb = t.k0; kb < t.k1; ++kb, ++it) {
      if (it % kIssuers != which) continue;
      const uint32_t s = it % C::kStages, as = it % C::kAcc;
      if ((it >= C::kAcc &&
           !ready(bar_at(bars, C::kAccEmpty + as), ((it / C::kAcc) - 1u) & 1u, abort_flag, p.timeout_ns)) ||
          !ready(bar_at(bars, C::kFull + s), (it / C::kStages) & 1u, abort_flag, p.timeout_ns)) {
        alive = false;
        break;
      }
      ptx::tc_fence_after();
      const uint32_t sa = smem + s * C::kStageBytes;
      const uint64_t da = ptx::smem_desc_sw128(sa, 16), db = ptx::smem_desc_sw128(sa + C::kABytes, 16);
      if (elected()) {
#pragma unroll
        for (int j = 0; j < kKB / 32; ++j) mma_f8(tmem + as * kBN, da + 2u * j, db + 2u * j, idesc, j > 0 ? 1u : 0u);
        ptx::mma_commit(bar_at(bars, C::kEmpty + s));
        ptx::mma_commit(bar_at(bars, C::kAccFull + as));
      }
      __syncwarp();
    }
  }
  // every MMA of this warp is done before TMEM is released (the elected lane is always the same)
  if (elected()) ptx::mma_commit(bar_at(bars, C::kFinal));
  __syncwarp();
  wait_force(bar_at(bars, C::kFinal), 0u, abort_flag, p.timeout_ns);
}

// The scales of a row's n <= kBatch blocks from `from` on, 0 after them.  A load of a column of
// rows touches a line for each lane, whatever it takes of it.
static_assert(kBatch == 4, "a float4 of scales");
__device__ __forceinline__ void batch_of(const float* from, int n, bool wide, float (&v)[kBatch]) {
  if (wide) {
    const float4 q = __ldg(reinterpret_cast<const float4*>(from));
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
#pragma unroll
    for (int e = 0; e < kBatch; ++e) v[e] = e < n ? __ldg(from + e) : 0.f;
  }
}

// Brings the scales of kBatch blocks at a time: with a scale for 128 rows of b the products
// with the 128 scales of a for both halves of the columns, else a's and then b's own.
template <int kBN, bool kBRows>
__device__ void scale_loader(const MmaParams& p, uint8_t* smem_gen, uint32_t bars, int lane, volatile int* abort_flag) {
  using C = MmaCfg<kBN, kBRows>;
  constexpr int kHalf = kBN / 2, kNB = kBRows ? kBN / 32 : 2;
  uint32_t bt = 0, un = 0;
  for (int u = blockIdx.x; u < p.units; u += gridDim.x, ++un) {
    const Unit t = unit_of<kBN>(p, u);
    for (int k = t.k0; k < t.k1; k += kBatch, ++bt) {
      const int n = min(kBatch, t.k1 - k);
      float* dst = reinterpret_cast<float*>(smem_gen + C::kScale) + (bt & 1u) * (kBatch * C::kScales);
      float a[kMB / 32][kBatch], b[kBRows ? 1 : kNB][kBatch];
#pragma unroll
      for (int i = 0; i < kMB / 32; ++i) {
        const float* from = p.sa + static_cast<int64_t>(min(t.m0 + 32 * i + lane, p.M - 1) >> p.a_shift) * p.kb + k;
        batch_of(from, n, p.wide, a[i]);
      }
      if constexpr (!kBRows) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float* from = p.sb + static_cast<int64_t>(min(t.n0 + h * kHalf, p.N - 1) >> 7) * p.kb + k;
          batch_of(from, n, p.wide, b[h]);
        }
      }
      float v[kBRows ? kNB : 1][kBatch];  // b's own scales
      if constexpr (kBRows) {
#pragma unroll
        for (int i = 0; i < kNB; ++i)
          batch_of(p.sb + static_cast<int64_t>(min(t.n0 + 32 * i + lane, p.N - 1)) * p.kb + k, n, p.wide, v[i]);
      }
      float bias[kBRows ? 1 : kBN / 32];
      const bool first = !kBRows && k == t.k0 && p.bias != nullptr;
      if (first)
#pragma unroll
        for (int i = 0; i < (kBRows ? 0 : kBN / 32); ++i) {
          const int c = t.n0 + 32 * i + lane;
          bias[i] = c >= p.N       ? 0.f
                    : p.bias_f32 ? __ldg(static_cast<const float*>(p.bias) + c)
                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[c]);
        }
      if (bt >= 2 && !ready(bar_at(bars, C::kScEmpty + (bt & 1u)), ((bt >> 1) - 1u) & 1u, abort_flag, p.timeout_ns))
        return;
      if (first)
#pragma unroll
        for (int i = 0; i < (kBRows ? 0 : kBN / 32); ++i)
          reinterpret_cast<float*>(smem_gen + C::kBias)[(un & 3u) * kBN + 32 * i + lane] = bias[i];
      if constexpr (kBRows) {
#pragma unroll
        for (int i = 0; i < kNB; ++i)
#pragma unroll
          for (int e = 0; e < kBatch; ++e) {
            const int c = 32 * i + lane, half = c / kHalf, in = c % kHalf;
            dst[e * C::kScales + kMB + (4 * half + in % 4) * C::kColGap + in / 4] = v[i][e];
          }
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
#pragma unroll
        for (int i = 0; i < kMB / 32; ++i) {
          float* to = dst + e * C::kScales + 32 * i + lane;
          if constexpr (kBRows) {
            to[0] = a[i][e];
          } else {
            to[0] = a[i][e] * b[0][e];
            to[kMB] = a[i][e] * b[1][e];
          }
        }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar_at(bars, C::kScFull + (bt & 1u)));
    }
  }
}

// Adds the blocks of this thread's row and half of the columns, and writes them.
template <int kBN>
__device__ void promoter(const MmaParams& p, uint32_t smem, uint8_t* smem_gen, uint32_t bars, uint32_t tmem, int warp,
                         int lane, volatile int* abort_flag) {
  constexpr bool kBRows = false;
  using C = MmaCfg<kBN, kBRows>;
  constexpr int kCols = kBN / 2, kGroups = kCols / 32;
  const int half = (warp - kPromoteWarp0) >> 2, quad = warp & 3;
  const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * kCols;
  const uint32_t stg = C::kStg + (warp - kPromoteWarp0) * C::kStgBytes;
  const float* scales = reinterpret_cast<const float*>(smem_gen + C::kScale) + half * kMB + quad * 32 + lane;
  const float* bias = reinterpret_cast<const float*>(smem_gen + C::kBias) + half * kCols;
  uint32_t it = 0, bt = 0, un = 0;
  auto give_up = [&] {  // this warp's stores are done with their shared memory
    if (lane == 0) ptx::bulk_wait_all();
  };
  for (int u = blockIdx.x; u < p.units; u += gridDim.x, ++un) {
    const Unit t = unit_of<kBN>(p, u);
    const int n = t.k1 - t.k0, col0 = t.n0 + half * kCols;
    // the sums start from the bias, which came with the first scales
    if (!ready(bar_at(bars, C::kScFull + (bt & 1u)), (bt >> 1) & 1u, abort_flag, p.timeout_ns)) return give_up();
    uint64_t acc[kCols / 2];
    if (p.bias != nullptr) {
      const float4* from = reinterpret_cast<const float4*>(bias + (un & 3u) * kBN);
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) {
        const float4 b = from[i];
        acc[2 * i] = ptx::pack2(b.x, b.y);
        acc[2 * i + 1] = ptx::pack2(b.z, b.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = 0ull;
    }
    for (int k = 0; k < n; ++k, ++it) {
      const uint32_t as = it % C::kAcc;
      if (k > 0 && k % kBatch == 0 && !ready(bar_at(bars, C::kScFull + (bt & 1u)), (bt >> 1) & 1u, abort_flag, p.timeout_ns))
        return give_up();
      const float s = scales[((bt & 1u) * kBatch + k % kBatch) * C::kScales];
      const uint64_t s2 = ptx::pack2(s, s);
      if (!ready(bar_at(bars, C::kAccFull + as), (it / C::kAcc) & 1u, abort_flag, p.timeout_ns)) return give_up();
      ptx::tc_fence_after();
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        uint32_t r[32];
        ptx::tmem_ld32(taddr + as * kBN + 32u * g, r);
        ptx::tmem_wait_ld();
        ptx::reg_fence(r);
        if (g + 1 == kGroups) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar_at(bars, C::kAccEmpty + as));
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
          acc[g * 16 + j] =
              ptx::ffma2(ptx::pack2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), s2, acc[g * 16 + j]);
      }
      if (k % kBatch == kBatch - 1 || k + 1 == n) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_at(bars, C::kScEmpty + (bt & 1u)));
        ++bt;
      }
    }
    // ---- the warp's 32 rows go through its shared memory, a bf16 row (or half an fp32 row) at
    // a time, in boxes of 128 bytes a row: 16-byte chunk j of a box's row r at chunk j ^ (r % 8)
    // (the 128-byte swizzle of the TMA store, and free of bank conflicts)
    const int esize = p.out_f32 ? 4 : 2;
    const int row0 = t.m0 + quad * 32;
    // writes the staged boxes of `cols` columns each from column c0 on, and hands them over
    auto leave = [&](int c0, int boxes, int cols) {
      if (p.tma_out) {
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          for (int b = 0; b < boxes; ++b)
            if (c0 + b * cols < p.N && row0 < p.M)
              tma_store_3d(&p.tm_out, smem + stg + b * 4096u, c0 + b * cols, row0, t.split);
          ptx::bulk_commit_group();
        }
        return;
      }
      __syncwarp();
      // a lane writes the same four bytes of each row: an fp32 column or two bf16 ones
      uint8_t* out = static_cast<uint8_t*>(p.out) + t.split * p.split_stride * esize;
      const int col = c0 + (p.out_f32 ? lane : 2 * lane);
      const bool words = p.out_f32 || ((p.N & 1) == 0 && (reinterpret_cast<uintptr_t>(p.out) & 3u) == 0);
      for (int b = 0; b < boxes; ++b) {
        const int c = col + b * cols;
        if (c >= p.N) break;
        uint8_t* to = out + (static_cast<int64_t>(row0) * p.N + c) * esize;
        const int64_t pitch = static_cast<int64_t>(p.N) * esize;
#pragma unroll 8
        for (int r = 0; r < 32; ++r, to += pitch) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(smem_gen + stg + b * 4096u + r * 128 +
                                                                (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
          if (row0 + r >= p.M) continue;
          if (words) {
            *reinterpret_cast<uint32_t*>(to) = w;
          } else {
            reinterpret_cast<uint16_t*>(to)[0] = static_cast<uint16_t>(w);
            if (c + 1 < p.N) reinterpret_cast<uint16_t*>(to)[1] = static_cast<uint16_t>(w >> 16);
          }
        }
      }
      __syncwarp();
    };
    uint8_t* mine = smem_gen + stg + lane * 128;
    if (lane == 0) ptx::bulk_wait_read_all();  // the last tile's stores have read the room
    __syncwarp();
    if (p.out_f32) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // the room holds half the columns
        if (h == 1) {
          if (lane == 0) ptx::bulk_wait_read_all();
          __syncwarp();
        }
#pragma unroll
        for (int q = 0; q < kCols / 8; ++q) {
          const int e = (h * kCols / 8 + q) * 2;
          float4 v;
          ptx::unpack2(acc[e], v.x, v.y);
          ptx::unpack2(acc[e + 1], v.z, v.w);
          *reinterpret_cast<float4*>(mine + (q / 8) * 4096 + (((q % 8) ^ (lane & 7)) << 4)) = v;
        }
        leave(col0 + h * (kCols / 2), kCols / 64, 32);
      }
    } else {
#pragma unroll
      for (int q = 0; q < kCols / 8; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo, hi;
          ptx::unpack2(acc[4 * q + e], lo, hi);
          w[e] = pack_bf16x2(lo, hi);
        }
        *reinterpret_cast<uint4*>(mine + (q / 8) * 4096 + (((q % 8) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      leave(col0, kCols / 64, 64);
    }
  }
  give_up();
}

// Four lanes (lane % 4) hold one row's columns 4 m + lane % 4 in v[m]; after it lane % 4 = m holds
// the columns 4 m .. 4 m + 3.
__device__ __forceinline__ void turn4(float (&v)[4], int lane) {
  const bool odd = lane & 1, upper = lane & 2;
#pragma unroll
  for (int p = 0; p < 4; p += 2) {
    const float got = __shfl_xor_sync(0xffffffffu, odd ? v[p] : v[p + 1], 1);
    v[p] = odd ? got : v[p];
    v[p + 1] = odd ? v[p + 1] : got;
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const float got = __shfl_xor_sync(0xffffffffu, upper ? v[p] : v[p + 2], 2);
    v[p] = upper ? got : v[p];
    v[p + 2] = upper ? v[p + 2] : got;
  }
}

// The same with a scale for each row of b: of every four columns a thread has one, of rows
// lane / 4, + 8, + 16 and + 24 of its warp's 32.
template <int kBN>
__device__ void promoter_rows(const MmaParams& p, uint8_t* smem_gen, uint32_t bars, uint32_t tmem, int warp, int lane,
                              volatile int* abort_flag) {
  constexpr bool kBRows = true;
  using C = MmaCfg<kBN, kBRows>;
  constexpr int kCols = kBN / 2, kGroups = kCols / 32;
  const int half = (warp - kPromoteWarp0) >> 2, quad = warp & 3;
  const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * kCols;
  const float* scales = reinterpret_cast<const float*>(smem_gen + C::kScale);
  uint32_t it = 0, bt = 0;
  for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
    const Unit t = unit_of<kBN>(p, u);
    const int n = t.k1 - t.k0;
    // [32-column group][4-column group][upper or lower 16 rows], each of rows row, row + 8
    uint64_t acc[kGroups][8][2];
#pragma unroll
    for (int i = 0; i < kGroups * 16; ++i) (&acc[0][0][0])[i] = 0ull;
    for (int k = 0; k < n; ++k, ++it) {
      const uint32_t as = it % C::kAcc;
      if (k % kBatch == 0 && !ready(bar_at(bars, C::kScFull + (bt & 1u)), (bt >> 1) & 1u, abort_flag, p.timeout_ns))
        return;
      const float* sc = scales + ((bt & 1u) * kBatch + k % kBatch) * C::kScales;
      uint64_t sa2[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* at = sc + quad * 32 + 16 * h + (lane >> 2);
        sa2[h] = ptx::pack2(at[0], at[8]);
      }
      const float4* sb = reinterpret_cast<const float4*>(sc + kMB + (4 * half + (lane & 3)) * C::kColGap);
      if (!ready(bar_at(bars, C::kAccFull + as), (it / C::kAcc) & 1u, abort_flag, p.timeout_ns)) return;
      ptx::tc_fence_after();
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        uint32_t r[2][16];
        tmem_ld_frag(taddr + as * kBN + 32u * g, r[0]);
        tmem_ld_frag(taddr + as * kBN + 32u * g + (16u << 16), r[1]);
        const float4 b0 = sb[2 * g], b1 = sb[2 * g + 1];
        const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
        ptx::tmem_wait_ld();
        reg_fence16(r[0]);
        reg_fence16(r[1]);
        if (g + 1 == kGroups) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar_at(bars, C::kAccEmpty + as));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t b2 = ptx::pack2(b[i], b[i]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint64_t x = ptx::pack2(__uint_as_float(r[h][2 * i]), __uint_as_float(r[h][2 * i + 1]));
            acc[g][i][h] = ptx::ffma2(ptx::fmul2(x, sa2[h]), b2, acc[g][i][h]);
          }
        }
      }
      if (k % kBatch == kBatch - 1 || k + 1 == n) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_at(bars, C::kScEmpty + (bt & 1u)));
        ++bt;
      }
    }
    // four lanes turn their columns so that each has four neighbours: together 16 of a row
    const int esize = p.out_f32 ? 4 : 2;
    uint8_t* out = static_cast<uint8_t*>(p.out) + t.split * p.split_stride * esize;
    const bool fours = (p.N & 3) == 0 && (reinterpret_cast<uintptr_t>(p.out) & 15u) == 0;
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int col = t.n0 + half * kCols + 32 * g + 16 * q + 4 * (lane & 3);
        float bias[4] = {};
        if (p.bias != nullptr)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (col + i < p.N)
              bias[i] = p.bias_f32 ? __ldg(static_cast<const float*>(p.bias) + col + i)
                                   : __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[col + i]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[2][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) ptx::unpack2(acc[g][4 * q + i][h], v[0][i], v[1][i]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            turn4(v[e], lane);
            const int row = t.m0 + quad * 32 + 16 * h + 8 * e + (lane >> 2);
            if (row >= p.M || col >= p.N) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[e][i] += bias[i];
            const int64_t at = static_cast<int64_t>(row) * p.N + col;
            if (p.out_f32) {
              float* to = reinterpret_cast<float*>(out) + at;
              if (fours) *reinterpret_cast<float4*>(to) = make_float4(v[e][0], v[e][1], v[e][2], v[e][3]);
              else
                for (int i = 0; i < 4; ++i)
                  if (col + i < p.N) to[i] = v[e][i];
            } else {
              __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(out) + at;
              if (fours)
                *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(v[e][0], v[e][1]), pack_bf16x2(v[e][2], v[e][3]));
              else
                for (int i = 0; i < 4; ++i)
                  if (col + i < p.N) to[i] = __float2bfloat16_rn(v[e][i]);
            }
          }
        }
      }
  }
}

template <int kBN, bool kBRows>
__global__ void __launch_bounds__(kMThreads, 1) bsa_fp8_mma_kernel(const __grid_constant__ MmaParams p) {
  using C = MmaCfg<kBN, kBRows>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);
  const uint32_t bars = base + C::kBar;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kBars; ++i) {
      const bool acc_empty = i >= C::kAccEmpty && i < C::kAccEmpty + C::kAcc;
      const bool sc_empty = i >= C::kScEmpty && i < C::kScEmpty + 2;
      ptx::mbar_init(bar_at(bars, i), acc_empty || sc_empty ? kPromoteWarps : i == C::kFinal ? kIssuers : 1u);
    }
    *abort_flag = 0;
    ptx::fence_barrier_init();
    ptx::prefetch_tensormap(&p.tm_a);
    ptx::prefetch_tensormap(&p.tm_b);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(const_cast<uint32_t*>(&misc[0])), kTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];
  // 384 threads have 168 registers each, which the adding warps use nearly in full
  if (warp < kPromoteWarp0) {
    if (warp == 0) mma_producer<kBN, kBRows>(p, base, bars, abort_flag);
    else if (warp == kScaleWarp) scale_loader<kBN, kBRows>(p, smem, bars, lane, abort_flag);
    else mma_issuer<kBN, kBRows>(p, base, bars, tmem, static_cast<uint32_t>(warp - kIssueWarp0), abort_flag);
    __syncwarp();
  } else {
    if constexpr (kBRows) promoter_rows<kBN>(p, smem, bars, tmem, warp, lane, abort_flag);
    else promoter<kBN>(p, base, smem, bars, tmem, warp, lane, abort_flag);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, kTmem);
}

// A barrier that nothing arrives at: exercises the product's bounded wait and its status word.
__global__ void bsa_fp8_debug_wait_kernel(unsigned long long timeout_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    ptx::mbar_init(ptx::smem_addr(&bar), 1);
    abort_flag = 0;
    ptx::fence_barrier_init();
  }
  __syncthreads();
  ready(ptx::smem_addr(&bar), 0, &abort_flag, timeout_ns);
  __syncthreads();
}

// Sums the splits' partial results in order, adds the bias and rounds once; kVec elements a
// thread (4 where rows of the result are multiples of 4).  Launched as the product's
// programmatic dependent.  The product triggers nothing early, so that its blocks come when the
// product's have ended: what is saved is a launch's own time (2304 x 768 x 65536: 190 us a pass,
// 192 as an ordinary launch).
template <int kVec>
__global__ void __launch_bounds__(256) bsa_fp8_sum_kernel(const float* part, int splits, int64_t stride, int64_t n,
                                                          int N, const void* bias, int bias_f32, void* out,
                                                          int out_f32) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * kVec;
  if (i >= n) return;
  float v[kVec] = {};
  for (int s0 = 0; s0 < splits; s0 += 8) {
    float x[8][kVec];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const float* from = part + (s0 + s) * stride + i;
      if constexpr (kVec == 4) {
        const float4 q = s0 + s < splits ? *reinterpret_cast<const float4*>(from) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[s][0] = q.x, x[s][1] = q.y, x[s][2] = q.z, x[s][3] = q.w;
      } else {
        x[s][0] = s0 + s < splits ? *from : 0.f;
      }
    }
#pragma unroll
    for (int s = 0; s < 8; ++s)
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[e] += x[s][e];
  }
  if (bias != nullptr) {
    const int c = static_cast<int>(i % N);
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      v[e] += bias_f32 ? static_cast<const float*>(bias)[c + e]
                       : __bfloat162float(static_cast<const __nv_bfloat16*>(bias)[c + e]);
  }
  if constexpr (kVec == 4) {
    if (out_f32) *reinterpret_cast<float4*>(static_cast<float*>(out) + i) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + i) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else {
    if (out_f32) static_cast<float*>(out)[i] = v[0];
    else static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v[0]);
  }
}

// ------------------------------------------------------------ a few rows
struct RowsParams {
  const uint8_t *a, *b;
  int64_t lda, ldb;
  const float *sa, *sb;
  const void* bias;
  void* out;
  int M, N, K, kb;
  int a_shift, b_shift;
  int bias_f32, out_f32;
};

constexpr int kRowsMost = 8;        // rows of a that the kernel takes
constexpr int kRowsWarpsMost = 16;  // warps of a block at most
constexpr int kRowsAhead = 4;       // blocks of K on their way to a warp, the one in use included

template <bool kE5>
__device__ __forceinline__ uint32_t widen(uint32_t two) {  // two codes in the low 16 bits -> two fp16
  uint32_t r;
  const uint16_t h = static_cast<uint16_t>(two);
  if constexpr (kE5) asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(h));
  else asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  return r;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 codes of a row at column k (a multiple of 16); zeros past the row's end, which is not
// read past.  kTail: K may end inside the 16.
template <bool kTail>
__device__ __forceinline__ uint4 codes16(const uint8_t* row, int k, int K) {
  if (k + (kTail ? 16 : 1) <= K) return __ldg(reinterpret_cast<const uint4*>(row + k));
  uint32_t x[4] = {};
  if constexpr (kTail) {
#pragma unroll 1
    for (int i = 0; i < 15; ++i)
      if (k + i < K) {
        const uint32_t c = static_cast<uint32_t>(row[k + i]) << (8 * (i & 3));
#pragma unroll
        for (int w = 0; w < 4; ++w) x[w] |= w == i >> 2 ? c : 0u;
      }
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// Thread (g, t) of a warp (lane / 4, lane % 4) holds, of each 64 codes of K, the 16 at 16 t of
// b's rows g and g + 8 and of token g: any order of K's products gives the same sum, so four
// codes of these serve as the thread's k-slots of one m16n8k16 product.
// kHeld: a warp's blocks of K (1 to 4), whose tokens stay widened in registers from tile to
// tile; 0: more, their tokens are read again for every tile.
template <bool kAE5, bool kBE5, bool kTail, int kHeld>
__global__ void __launch_bounds__(kRowsWarpsMost * 32, 1) bsa_fp8_rows_kernel(const __grid_constant__ RowsParams p) {
  __shared__ float part[2][kRowsWarpsMost][32][4];
  // b's codes of the blocks to come, each warp's own: 16 rows of 128 bytes a slot, fetched as
  // whole lines (8 lanes a row); 16-byte chunk c of row r lies at chunk c ^ 4 (r % 2), which
  // spreads what 8 lanes read of two rows over all banks
  extern __shared__ __align__(16) uint8_t ring[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int warps = blockDim.x >> 5, tiles = (p.N + 15) / 16;
  const int per = kHeld > 0 ? kHeld : (p.kb + warps - 1) / warps;
  const int k0 = min(warp * per, p.kb), k1 = min(k0 + per, p.kb);
  const uint32_t mine = ptx::smem_addr(ring) + warp * (kRowsAhead * 2048u);

  // ---- fetching: lane / 8 + 4 j is its row, lane % 8 its 16 bytes
  const int64_t four = 4 * p.ldb, tile_step = static_cast<int64_t>(gridDim.x) * 16 * p.ldb;
  int fk = k0, fr = blockIdx.x * 16 + (lane >> 3);
  const uint8_t* from = p.b + static_cast<int64_t>(fr) * p.ldb + (lane & 7) * 16;
  uint32_t fdst = mine + (lane >> 3) * 128u + (((lane & 7) ^ ((lane >> 3 & 1) << 2)) << 4);
  uint32_t fslot = 0;
  auto fetch = [&] {
    if (fr - (lane >> 3) < p.N && k0 < k1) {
      const int k = fk * kKB + (lane & 7) * 16;
      const uint8_t* at = from + fk * kKB;
#pragma unroll
      for (int j = 0; j < 4; ++j, at += four) {
        const bool row = fr + 4 * j < p.N;
        const uint32_t dst = fdst + j * 512u;
        if (kTail && k + 16 > p.K) {  // the row's last codes, or none
          const uint4 w = row ? codes16<kTail>(at - k, k, p.K) : make_uint4(0, 0, 0, 0);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
        } else {  // outside the matrix nothing is read and zeros are stored
          const bool in = row && k < p.K;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(in ? at : p.b), "r"(in ? 16 : 0)
                       : "memory");
        }
      }
      if (++fk == k1) {
        fk = k0;
        fr += gridDim.x * 16;
        from += tile_step;
      }
      const bool wrap = ++fslot == kRowsAhead;
      fdst += wrap ? -(kRowsAhead - 1) * 2048u : 2048u;
      fslot = wrap ? 0 : fslot;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i + 1 < kRowsAhead; ++i) fetch();

  // ---- the tokens
  const uint8_t* a = p.a + static_cast<int64_t>(min(g, p.M - 1)) * p.lda;
  const float* sa0 = p.sa + static_cast<int64_t>(min(2 * t, p.M - 1) >> p.a_shift) * p.kb;
  const float* sa1 = p.sa + static_cast<int64_t>(min(2 * t + 1, p.M - 1) >> p.a_shift) * p.kb;
  struct Tokens {  // a block's: four codes of each of two 64s widened, and two tokens' scales
    uint32_t x[2][8];
    float m0, m1;
  };
  auto tokens = [&](int kb) {
    Tokens c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 w = g < p.M ? codes16<kTail>(a, kb * kKB + h * 64 + t * 16, p.K) : make_uint4(0, 0, 0, 0);
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c.x[h][2 * i] = widen<kAE5>(v[i]);
        c.x[h][2 * i + 1] = widen<kAE5>(v[i] >> 16);
      }
    }
    c.m0 = __ldg(sa0 + kb);
    c.m1 = __ldg(sa1 + kb);
    return c;
  };
  Tokens held[kHeld > 0 ? kHeld : 1];
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (k0 + i < k1) held[i] = tokens(k0 + i);

  uint32_t rd = mine + g * 128u, slot = 0;
  const uint32_t c0 = (t ^ ((g & 1) << 2)) << 4, c1 = ((4 + t) ^ ((g & 1) << 2)) << 4;
  // adds the block at hand, of tokens c and of the scales s0 and s1 of b's rows g and g + 8
  auto use = [&](const Tokens& c, float s0, float s1, float (&acc)[4]) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kRowsAhead - 1) : "memory");
    __syncwarp();
    float d[4] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t r[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[e][0]), "=r"(r[e][1]), "=r"(r[e][2]), "=r"(r[e][3])
                     : "r"(rd + e * 1024u + (h ? c1 : c0)));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mma_f16(d, widen<kBE5>(r[0][i]), widen<kBE5>(r[1][i]), widen<kBE5>(r[0][i] >> 16), widen<kBE5>(r[1][i] >> 16),
                c.x[h][2 * i], c.x[h][2 * i + 1]);
    }
    acc[0] = fmaf(d[0], s0 * c.m0, acc[0]);
    acc[1] = fmaf(d[1], s0 * c.m1, acc[1]);
    acc[2] = fmaf(d[2], s1 * c.m0, acc[2]);
    acc[3] = fmaf(d[3], s1 * c.m1, acc[3]);
    const bool wrap = ++slot == kRowsAhead;
    rd += wrap ? -(kRowsAhead - 1) * 2048u : 2048u;
    slot = wrap ? 0 : slot;
    __syncwarp();  // the slot may be fetched into again
  };
  int turn = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, turn ^= 1) {
    float acc[4] = {};
    const float* sb0 = p.sb + static_cast<int64_t>(min(tile * 16 + g, p.N - 1) >> p.b_shift) * p.kb;
    const float* sb1 = p.b_shift ? sb0 : p.sb + static_cast<int64_t>(min(tile * 16 + g + 8, p.N - 1)) * p.kb;
    if constexpr (kHeld > 0) {
      float s0[kHeld], s1[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const bool there = k0 + i < k1;
        s0[i] = there ? __ldg(sb0 + k0 + i) : 0.f;
        s1[i] = p.b_shift ? s0[i] : there ? __ldg(sb1 + k0 + i) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (k0 + i < k1) {
          fetch();
          use(held[i], s0[i], s1[i], acc);
        }
    } else {
      for (int kb = k0; kb < k1; ++kb) {
        fetch();
        const float s0 = __ldg(sb0 + kb), s1 = __ldg(sb1 + kb);
        use(tokens(kb), s0, s1, acc);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) part[turn][warp][lane][i] = acc[i];
    __syncthreads();  // the other half of part is read before the next one
    // output (m, n): 16 neighbouring threads write 16 neighbouring columns of one token
    for (int o = threadIdx.x; o < 8 * 16; o += blockDim.x) {
      const int c = o & 15, m = o >> 4, n = tile * 16 + c;
      if (m >= p.M || n >= p.N) continue;
      const int ln = (c & 7) * 4 + (m >> 1), i = (c >> 3) * 2 + (m & 1);
      float v = 0.f;
      for (int w = 0; w < warps; ++w) v += part[turn][w][ln][i];
      if (p.bias != nullptr)
        v += p.bias_f32 ? static_cast<const float*>(p.bias)[n]
                        : __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[n]);
      const int64_t at = static_cast<int64_t>(m) * p.N + n;
      if (p.out_f32) static_cast<float*>(p.out)[at] = v;
      else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
    }
  }
}

template <bool kAE5, bool kBE5, bool kTail, int kHeld>
int start_rows(const RowsParams& p, int grid, int threads, cudaStream_t s) {
  auto* kernel = bsa_fp8_rows_kernel<kAE5, kBE5, kTail, kHeld>;
  const int smem = kRowsAhead * 2048 * (threads / 32);
  // The limit belongs to the process, and one kernel serves several counts of warps: it is only
  // ever set to the most, so that a call from another thread never finds it below its own size.
  if (smem > 32 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kRowsAhead * 2048 * kRowsWarpsMost) != cudaSuccess)
    return BSA_ERR_CUDA;
  kernel<<<grid, threads, smem, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

// A K that is no multiple of 16 is rare and takes the form that holds nothing.
template <bool kAE5, bool kBE5>
int launch_rows(const RowsParams& p, int grid, int threads, cudaStream_t s) {
  if (p.K % 16 != 0) return start_rows<kAE5, kBE5, true, 0>(p, grid, threads, s);
  switch ((p.kb + threads / 32 - 1) / (threads / 32)) {
    case 1: return start_rows<kAE5, kBE5, false, 1>(p, grid, threads, s);
    case 2: return start_rows<kAE5, kBE5, false, 2>(p, grid, threads, s);
    case 3: return start_rows<kAE5, kBE5, false, 3>(p, grid, threads, s);
    case 4: return start_rows<kAE5, kBE5, false, 4>(p, grid, threads, s);
    default: return start_rows<kAE5, kBE5, false, 0>(p, grid, threads, s);
  }
}

// ------------------------------------------------------------ host
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// 8-bit [rows, cols] of the given pitch, boxes of 128 columns x box_rows, 128-byte swizzle;
// what lies past the matrix reads as zeros.
bool map_codes(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint64_t pitch, uint32_t box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {pitch};
  const cuuint32_t box[2] = {kKB, box_rows}, estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The result [splits, M, N] of esize-byte elements, boxes of 128 bytes by 32 rows.
bool map_result(CUtensorMap* m, void* ptr, uint64_t splits, uint64_t rows, uint64_t cols, int f32) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const uint64_t esize = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {cols, rows, splits}, strides[2] = {cols * esize, rows * cols * esize};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / esize), 32, 1}, estr[3] = {1, 1, 1};
  return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, ptr, dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Per device, once: whether it is an sm_100 part, its SM count, and the kernels' shared-
// memory attributes set.  A failed setup is not cached.
constexpr int kMaxFp8Devices = 64;
int g_fp8_sms[kMaxFp8Devices] = {};
std::mutex g_fp8_mu;

template <int kBN, bool kBRows>
bool allow_smem() {
  return cudaFuncSetAttribute(bsa_fp8_mma_kernel<kBN, kBRows>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(MmaCfg<kBN, kBRows>::kAlloc)) == cudaSuccess;
}

int fp8_device_sms() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
  if (dev < 0 || dev >= kMaxFp8Devices) return BSA_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_fp8_mu);
  if (g_fp8_sms[dev] != 0) return g_fp8_sms[dev];
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return BSA_ERR_CUDA;
  if (major != 10 || minor != 0) {
    g_fp8_sms[dev] = BSA_ERR_UNSUPPORTED;
    return BSA_ERR_UNSUPPORTED;
  }
  if (!allow_smem<256, false>() || !allow_smem<256, true>() || !allow_smem<128, false>() || !allow_smem<128, true>())
    return BSA_ERR_CUDA;
  g_fp8_sms[dev] = sms;
  return sms;
}

// Tile width and split of K for a product on `sms` SMs: the pair with the least estimate of
//     waves of units x (blocks of K a unit x block time + a unit's start and end) + bytes of
// the splits' partial results.  The constants are of one scale, fitted to a sweep of widths and
// splits.  In a graph, chosen and next best: 2304 x 768 x 65536 256 columns by 5 splits 158 us,
// 256 by 8 164, 128 by 4 168; 65536 x 2304 x 768 256 139 us, 128 155; 777 x 2050 x 1104 128
// 8.4 us, 256 12.7; 300 x 1000 x 20000 128 by 6 16.3 us, 256 by 10 19.1; 512 x 512 x 8192
// 128 by 4 11.0 us, though 128 by 10 takes 9.9.
struct MmaPlan {
  int bn, splits, kb_split;
  size_t bytes;
};
MmaPlan mma_plan(int64_t M, int64_t N, int64_t kb, int sms) {
  MmaPlan best{256, 1, static_cast<int>(kb), 0};
  double least = 1e30;
  for (const int bn : {256, 128}) {
    const int64_t tiles = ((M + kMB - 1) / kMB) * ((N + bn - 1) / bn);
    for (int64_t want = 1; want <= 32 && want <= kb; ++want) {
      if (want > 1 && tiles * want > 4 * sms) break;  // more units than that only cost partials
      int64_t per = (kb + want - 1) / want;
      if (want > 1) per = (per + kBatch - 1) / kBatch * kBatch;  // whole batches of scales
      const int64_t splits = (kb + per - 1) / per;
      if (splits != want) continue;
      const int64_t waves = (tiles * splits + sms - 1) / sms;
      double cost = static_cast<double>(waves) * (static_cast<double>(per) * (bn == 256 ? 560 : 330) + 2500.0);
      // partials: written and read once, about 3000 bytes a cycle, and a second launch
      if (splits > 1) cost += 4000.0 + static_cast<double>(splits) * M * N * 8.0 / 3000.0;
      if (cost < least) {
        least = cost;
        best = MmaPlan{bn, static_cast<int>(splits), static_cast<int>(per),
                       splits > 1 ? static_cast<size_t>(splits) * M * N * sizeof(float) : 0};
      }
    }
  }
  return best;
}

int format_bits(int type) { return type == BSA_E5M2 ? 1 : 0; }

template <int kBN>
void launch_mma(const MmaParams& p, int grid, cudaStream_t s) {
  if (p.b_rows) bsa_fp8_mma_kernel<kBN, true><<<grid, kMThreads, MmaCfg<kBN, true>::kAlloc, s>>>(p);
  else bsa_fp8_mma_kernel<kBN, false><<<grid, kMThreads, MmaCfg<kBN, false>::kAlloc, s>>>(p);
}

}  // namespace

int fp8_take_status() {
  int st = 0;
  if (cudaMemcpyFromSymbol(&st, g_bsa_status, sizeof(int)) != cudaSuccess) return BSA_ERR_CUDA;
  if (st != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_bsa_status, &zero, sizeof(int)) != cudaSuccess) return BSA_ERR_CUDA;
  }
  return st;
}

}  // namespace bsa

using namespace bsa;

namespace {
bool sizes_ok(int M, int N, int K) {
  return M >= 0 && N >= 0 && K >= 1 && M <= (1 << 30) && N <= (1 << 30) && K <= (1 << 30);
}
}  // namespace

extern "C" {

int bsa_fp8_matmul_workspace_bytes(int M, int N, int K, size_t* bytes) {
  if (bytes == nullptr || !sizes_ok(M, N, K)) return BSA_ERR_INVALID_ARG;
  *bytes = 0;
  if (M <= kRowsMost || N == 0) return BSA_OK;
  const int sms = fp8_device_sms();
  if (sms < 0) return sms;
  *bytes = (mma_plan(M, N, (static_cast<int64_t>(K) + kKB - 1) / kKB, sms).bytes + 255) / 256 * 256;
  return BSA_OK;
}

int bsa_fp8_matmul(const void* a, int a_type, int64_t lda, const float* a_scale, int a_rows, const void* b,
                   int b_type, int64_t ldb, const float* b_scale, int b_rows, const void* bias, int bias_type,
                   int M, int N, int K, void* out, int out_type, void* workspace, size_t workspace_bytes,
                   void* stream) {
  if (!sizes_ok(M, N, K)) return BSA_ERR_INVALID_ARG;
  if ((a_type != BSA_E4M3 && a_type != BSA_E5M2) || (b_type != BSA_E4M3 && b_type != BSA_E5M2) ||
      (out_type != BSA_BF16 && out_type != BSA_FP32) || (a_rows != 1 && a_rows != 128) ||
      (b_rows != 1 && b_rows != 128) || (bias != nullptr && bias_type != BSA_BF16 && bias_type != BSA_FP32))
    return BSA_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return BSA_OK;
  if (a == nullptr || b == nullptr || a_scale == nullptr || b_scale == nullptr || out == nullptr)
    return BSA_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(b) || lda % 16 != 0 || ldb % 16 != 0 || lda < K || ldb < K)
    return BSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(a_scale) | reinterpret_cast<uintptr_t>(b_scale)) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(out) % type_bytes(out_type) != 0 ||
      (bias != nullptr && reinterpret_cast<uintptr_t>(bias) % type_bytes(bias_type) != 0))
    return BSA_ERR_INVALID_ARG;
  const int sms = fp8_device_sms();
  if (sms < 0) return sms;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int kb = static_cast<int>((static_cast<int64_t>(K) + kKB - 1) / kKB);
  const int bias_f32 = bias_type == BSA_FP32, out_f32 = out_type == BSA_FP32;
  if (M <= kRowsMost) {
    RowsParams p{};
    p.a = static_cast<const uint8_t*>(a), p.b = static_cast<const uint8_t*>(b);
    p.lda = lda, p.ldb = ldb, p.sa = a_scale, p.sb = b_scale, p.bias = bias, p.out = out;
    p.M = M, p.N = N, p.K = K, p.kb = kb;
    p.a_shift = a_rows == 128 ? 7 : 0, p.b_shift = b_rows == 128 ? 7 : 0;
    p.bias_f32 = bias_f32, p.out_f32 = out_f32;
    // one block of up to 16 warps an SM, more of fewer warps where K is short
    const int warps = std::min(kb, kRowsWarpsMost), threads = 32 * warps;
    const int grid = std::min((N + 15) / 16, sms * (kRowsWarpsMost / warps));
    const bool ae5 = a_type == BSA_E5M2, be5 = b_type == BSA_E5M2;
    if (ae5) return be5 ? launch_rows<true, true>(p, grid, threads, s) : launch_rows<true, false>(p, grid, threads, s);
    return be5 ? launch_rows<false, true>(p, grid, threads, s) : launch_rows<false, false>(p, grid, threads, s);
  }
  const MmaPlan plan = mma_plan(M, N, kb, sms);
  if (plan.bytes > 0 && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 ||
                         workspace_bytes < plan.bytes))
    return BSA_ERR_WORKSPACE;
  MmaParams p{};
  if (!map_codes(&p.tm_a, a, M, K, lda, kMB) || !map_codes(&p.tm_b, b, N, K, ldb, plan.bn)) return BSA_ERR_CUDA;
  p.sa = a_scale, p.sb = b_scale;
  p.M = M, p.N = N, p.kb = kb;
  p.a_shift = a_rows == 128 ? 7 : 0, p.b_rows = b_rows == 1;
  p.idesc_formats = (format_bits(a_type) << 7) | (format_bits(b_type) << 10);
  p.n_tiles = (N + plan.bn - 1) / plan.bn;
  p.splits = plan.splits, p.kb_split = plan.kb_split;
  const int64_t units = static_cast<int64_t>((M + kMB - 1) / kMB) * p.n_tiles * p.splits;
  if (units > (1 << 30)) return BSA_ERR_INVALID_ARG;
  p.units = static_cast<int>(units);
  p.wide = kb % kBatch == 0 && aligned16(a_scale) && aligned16(b_scale);
  p.timeout_ns = kDefaultTimeoutNs;
  const bool split = plan.splits > 1;
  const int64_t n = static_cast<int64_t>(M) * N;
  p.split_stride = split ? n : 0;
  p.out = split ? workspace : out;
  p.out_f32 = split || out_f32;
  p.bias = split ? nullptr : bias;
  p.bias_f32 = bias_f32;
  p.tma_out = aligned16(p.out) && static_cast<int64_t>(N) * type_bytes(p.out_f32 ? BSA_FP32 : BSA_BF16) % 16 == 0;
  if (p.tma_out && !map_result(&p.tm_out, p.out, plan.splits, M, N, p.out_f32)) return BSA_ERR_CUDA;
  const int grid = static_cast<int>(std::min<int64_t>(units, sms));
  if (plan.bn == 256) launch_mma<256>(p, grid, s);
  else launch_mma<128>(p, grid, s);
  if (split) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const bool four = N % 4 == 0 && aligned16(out);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(((four ? n / 4 : n) + 255) / 256));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const float* part = static_cast<const float*>(workspace);
    if ((four ? cudaLaunchKernelEx(&cfg, bsa_fp8_sum_kernel<4>, part, plan.splits, n, n, N, bias, bias_f32, out, out_f32)
              : cudaLaunchKernelEx(&cfg, bsa_fp8_sum_kernel<1>, part, plan.splits, n, n, N, bias, bias_f32, out,
                                   out_f32)) != cudaSuccess)
      return BSA_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

int bsa_debug_product_wait_timeout(uint64_t timeout_ns, void* stream) {
  const int sms = fp8_device_sms();
  if (sms < 0) return sms;
  const unsigned long long t = std::min<unsigned long long>(std::max<unsigned long long>(timeout_ns, 1000ull), kDefaultTimeoutNs);
  bsa_fp8_debug_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(t);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // extern "C"
