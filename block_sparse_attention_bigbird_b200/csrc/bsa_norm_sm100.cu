// The norms before and after a block, fused with its gate and residual, for B200 (sm_100a):
//
//     z      = N_post(y) w_post + b_post,   stream = beta x + alpha g z,
//     normed = N_pre(stream) w_pre + b_pre,
//
// and the gradients of both outputs.  N is rms or layer normalisation over a row's C columns.
//
// A row belongs to one team of threads (a warp while a lane's share of it is small, else the
// block), every thread owning fixed columns, so that each array is read and written once and
// means, variances (of the centred values), sums and the residual are fp32 in registers.
// Blocks are persistent.  A thread brings its own pieces of the rows to come into shared
// memory with cp.async, up to three rows ahead, and reads back only what it brought, so that
// no barrier is needed and the loads in flight do not depend on the warps that fit.  What a
// column multiplies by (weights, gate, the scales) stays in registers from row to row (in the
// backward, whose sums need the registers, in shared memory), and the arithmetic is done on
// pairs (fma.rn.f32x2): with both the instructions a row stay well below what the SM issues
// in the time its bytes take.
//
// Backward, with D the gradient of the stream by both its uses:
//     a  = dnormed w_pre,  D = dstream + r (a - mean(a) - xh mean(a xh)),   dx = beta D,
//     c  = alpha g D w_post,  dy = r' (c - mean(c) - yh mean(c yh)),
// with xh, yh the normalised stream and y, r and r' the saved 1/sqrt(..), and the plain
// means only for layer norms.  The sums over rows need four quantities a column:
//     S = sum D yh, T = sum D  (over the rows of one gate row),
//     P = sum dnormed xh, Q = sum dnormed,
// because dgate = alpha (w_post S + b_post T), dw_post = alpha sum_b g_b S_b,
// db_post = alpha sum_b g_b T_b, dw_pre = P, db_pre = Q.  A block (one an SM, so that there are
// few partial sums) keeps them in registers over its contiguous rows, adds its teams' sums in
// shared memory when the gate row changes or its rows end, and writes them to slot
// (block + gate row), which no two (block, gate row) pairs share.  A second kernel adds the
// slots in a fixed order.  This suits gate rows that many rows share (a sequence, a batch): with
// one for each row the teams meet at every row and each row has a slot (16384 bf16 rows of 768:
// one gate row 40 us and 0.9 MB of workspace, four 44 us, 16384 of them 1385 us and 51 MB).
//
// What bounds both: the bytes of the activations; parameters stay in L1 and L2.  Measured with
// 65536 bf16 rows of 768, rms norms on both sides and fp32 parameters: forward (403 MB) 66 us
// alone, 73 in a row (5.5 TB/s, where a copy has 6.55); backward (604 MB) 101 us and 9 for
// the sum of the slots, 120 in a row (5.0 TB/s).  What is left is the row's chain: pieces
// landed, sum over the warp, division and root, second sum; four warps a scheduler (three in
// the backward, whose sums take the registers) hide most of it, issue slots are 51 % and 46 %
// busy.  4113 fp32 rows of 1030, backward: 33 us and 8 for the sum, 39 in a row; its rows have
// no 16-byte starts, so that a thread's pieces are of two elements (8-byte copies) and a row takes
// two barriers of a team, both a matter of this layout and no limit of the card.  Without the ring
// (loads straight to registers) the three took 102, 285 and 136 us.
// Statistics of the stored stream (kStored) cost a bf16 layer norm's training forward 5 to 10 % with
// biases (65536 rows of 768: 128 and 135 us, 8192 of 4096: 173 and 192); taken by two sums of
// their own after the first ones they cost up to 35 % (140 and 189 us without biases, now 159).
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "bsa_elem.cuh"
#include "sm100_ptx.cuh"

namespace bsa {
namespace {

constexpr int kMaxCols = 8192;

struct NormParams {
  const void *x, *y, *post_w, *post_b, *gate, *pre_w, *pre_b;
  void *out, *normed;
  float* stats;
  const void *dstream, *dnormed;  // backward
  const float* saved;
  void *dx, *dy;
  float *part, *part_pre;  // [slots][kN][C]: S (and T); [blocks][kN][C]: P (and Q)
  int64_t rows;
  int64_t per_gate;  // rows that share a gate row
  int C, post, pre;
  int params_f32;    // parameters are fp32 (else the activations' type)
  float alpha, beta, eps, inv_c;
  int64_t rows_per_block;
  int depth;  // slots of the ring, 1 to 3
};

// This thread's elements of a row as pairs: element kVec i + j of piece i, two by two.
template <int kE>
struct Pairs {
  uint64_t v[kE / 2];
  __device__ __forceinline__ void set(const float (&x)[kE]) {
#pragma unroll
    for (int e = 0; e < kE / 2; ++e) v[e] = ptx::pack2(x[2 * e], x[2 * e + 1]);
  }
  __device__ __forceinline__ void get(float (&x)[kE]) const {
#pragma unroll
    for (int e = 0; e < kE / 2; ++e) ptx::unpack2(v[e], x[2 * e], x[2 * e + 1]);
  }
};
__device__ __forceinline__ uint64_t twice(float x) { return ptx::pack2(x, x); }
__device__ __forceinline__ float sum2(uint64_t x) {
  float a, b;
  ptx::unpack2(x, a, b);
  return a + b;
}

// A thread's columns of a row of C: pieces of kVec, kNV of them.
template <int kVec, int kNV, bool kWarp>
struct Cols {
  static constexpr int kE = kVec * kNV;
  int C, team_threads, t;
  bool in[kNV];  // piece i lies in the row
  __device__ __forceinline__ Cols(int C_, int team_, int t_) : C(C_), team_threads(team_), t(t_) {
#pragma unroll
    for (int i = 0; i < kNV; ++i) in[i] = at(i) < C;
  }
  __device__ __forceinline__ int team() const { return kWarp ? 32 : team_threads; }
  __device__ __forceinline__ int at(int i) const { return (i * team() + t) * kVec; }
  __device__ __forceinline__ bool has(int i) const { return in[i]; }
  // a parameter's values at these columns (`dflt` where it is absent), 0 past the row's end
  template <typename T>
  __device__ __forceinline__ void param(const void* p, int64_t row, bool f32, float dflt, float (&v)[kE]) const {
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = at(i);
      float e[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) e[j] = has(i) ? dflt : 0.f;
      if (p != nullptr && has(i)) {
        if (f32) Elems<kVec, float>::load(static_cast<const float*>(p) + row * C + c, e);
        else Elems<kVec, T>::load(static_cast<const T*>(p) + row * C + c, e);
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[i * kVec + j] = e[j];
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* mine, const Pairs<kE>& x) const {  // mine: at column at(0) of the row
    float v[kE];
    x.get(v);
    const int step = team() * kVec;
#pragma unroll
    for (int i = 0; i < kNV; ++i, mine += step) {
      float e[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) e[j] = v[i * kVec + j];
      if (has(i)) Elems<kVec, T>::store(mine, e);
    }
  }
  // x where a piece is inside the row, else 0
  __device__ __forceinline__ uint64_t inside(int e, float x) const {
    const float a = has(2 * e / kVec) ? x : 0.f, b = has((2 * e + 1) / kVec) ? x : 0.f;
    return ptx::pack2(a, b);
  }
};

// Sums of kN values over a team; every thread of the team gets them.  A team of a whole
// block meets in shared memory, in one of two areas taken in turn so that one barrier a
// sum is enough.
template <int kN, bool kWarpTeam>
struct TeamSum {
  float* buf;  // [2][kN][32]
  int team_threads, bar_id, turn = 0;
  __device__ __forceinline__ void operator()(float (&v)[kN]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (!kWarpTeam) {
      const int nw = team_threads >> 5, w = (threadIdx.x % team_threads) >> 5, lane = threadIdx.x & 31;
      float* b = buf + turn * kN * 32;
      turn ^= 1;
      if (lane == 0)
#pragma unroll
        for (int i = 0; i < kN; ++i) b[i * 32 + w] = v[i];
      asm volatile("bar.sync %0, %1;" ::"r"(bar_id), "r"(team_threads) : "memory");
      // lanes read the warps' values, repeated over a power of two of lanes
      int top = 1;
      while (top < nw) top <<= 1;
      const int at = lane & (top - 1);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        float s = at < nw ? b[i * 32 + at] : 0.f;
        for (int o = top >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        v[i] = s;
      }
    }
  }
};

// A float for each column in shared memory, in the order that a team's threads read without
// bank conflicts: thread by thread, at most four floats of a piece at a time.
template <int kVec, int kNV, bool kWarp>
struct ColBuf {
  static constexpr int kE = kVec * kNV, kW = kVec < 4 ? kVec : 4, kS = kVec / kW;
  float* base;
  __device__ __forceinline__ float* at(const Cols<kVec, kNV, kWarp>& cols, int i, int h) const {
    return base + ((i * kS + h) * cols.team() + cols.t) * kW;
  }
  __device__ __forceinline__ void store(const Cols<kVec, kNV, kWarp>& cols, const Pairs<kE>& x) const {
    float v[kE];
    x.get(v);
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int h = 0; h < kS; ++h) {
        const float* f = v + i * kVec + h * kW;
        float* to = at(cols, i, h);
        if constexpr (kW == 4) *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
        else if constexpr (kW == 2) *reinterpret_cast<float2*>(to) = make_float2(f[0], f[1]);
        else to[0] = f[0];
      }
  }
  __device__ __forceinline__ void load(const Cols<kVec, kNV, kWarp>& cols, Pairs<kE>& x) const {
    float v[kE];
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int h = 0; h < kS; ++h) {
        float* f = v + i * kVec + h * kW;
        const float* from = at(cols, i, h);
        if constexpr (kW == 4) {
          const float4 q = *reinterpret_cast<const float4*>(from);
          f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
        } else if constexpr (kW == 2) {
          const float2 q = *reinterpret_cast<const float2*>(from);
          f[0] = q.x, f[1] = q.y;
        } else {
          f[0] = from[0];
        }
      }
    x.set(v);
  }
};

// (mean, 1 / sqrt(mean square of the centred values + eps)) of a row over the team; with a
// layer norm v is centred.  Past the row's end v holds 0 and keeps it.
template <int kVec, int kNV, bool kWarpTeam>
__device__ __forceinline__ float2 statistics(Pairs<kVec * kNV>& v, int kind, const Cols<kVec, kNV, kWarpTeam>& cols,
                                             const NormParams& p, TeamSum<1, kWarpTeam>& sum) {
  constexpr int kP = kVec * kNV / 2;
  float mean = 0.f, s[1];
  if (kind == BSA_NORM_LAYER) {
    uint64_t a = 0ull;
#pragma unroll
    for (int e = 0; e < kP; ++e) a = ptx::fadd2(a, v.v[e]);
    s[0] = sum2(a);
    sum(s);
    mean = s[0] * p.inv_c;
#pragma unroll
    for (int e = 0; e < kP; ++e) v.v[e] = ptx::fadd2(v.v[e], cols.inside(e, -mean));
  }
  uint64_t a = 0ull;
#pragma unroll
  for (int e = 0; e < kP; ++e) a = ptx::ffma2(v.v[e], v.v[e], a);
  s[0] = sum2(a);
  sum(s);
  return make_float2(mean, 1.f / sqrtf(fmaf(s[0], p.inv_c, p.eps)));
}

// The same for a layer norm, and what its backward starts from: mean and 1 / sqrt(..) of the row as it
// is stored, rounded to T (x, y of the result; z, w the ones of v itself).  The backward reads the
// stored row, and the statistics of the unrounded one do not fit a row that rounding moves by a good
// part of its deviation: its normalised values would have a mean, or a square, far from 0 and 1.
// Sums of the stored row are taken from the rounded mean s, near which such a row's values are a few
// steps of T, so that the difference of squares does not cancel (a constant row gives exact zeros);
// they share the second sum's steps over the team.
template <typename T, int kVec, int kNV, bool kWarpTeam>
__device__ __forceinline__ float4 statistics_stored(Pairs<kVec * kNV>& v, const Cols<kVec, kNV, kWarpTeam>& cols,
                                                    const NormParams& p, TeamSum<1, kWarpTeam>& sum,
                                                    TeamSum<3, kWarpTeam>& sum3) {
  constexpr int kP = kVec * kNV / 2;
  uint64_t a = 0ull;
#pragma unroll
  for (int e = 0; e < kP; ++e) a = ptx::fadd2(a, v.v[e]);
  float m[1] = {sum2(a)};
  sum(m);
  const float mean = m[0] * p.inv_c, s = to_f32(from_f32<T>(mean));
  uint64_t squares = 0ull, off = 0ull, off2 = 0ull;
#pragma unroll
  for (int e = 0; e < kP; ++e) {
    float lo, hi;
    ptx::unpack2(v.v[e], lo, hi);
    unpack(pack(lo, hi, T()), T(), lo, hi);
    const uint64_t d = ptx::fadd2(ptx::pack2(lo, hi), cols.inside(e, -s));
    off = ptx::fadd2(off, d);
    off2 = ptx::ffma2(d, d, off2);
    v.v[e] = ptx::fadd2(v.v[e], cols.inside(e, -mean));
    squares = ptx::ffma2(v.v[e], v.v[e], squares);
  }
  float q[3] = {sum2(squares), sum2(off), sum2(off2)};
  sum3(q);
  const float d = q[1] * p.inv_c, var = fmaxf(fmaf(q[2], p.inv_c, -d * d), 0.f);
  return make_float4(s + d, 1.f / sqrtf(var + p.eps), mean, 1.f / sqrtf(fmaf(q[0], p.inv_c, p.eps)));
}

constexpr int kWarpBlock = 128;  // threads of a forward block whose teams are warps
// a forward team's areas for its sums: [2][1][32] floats, and [2][3][32] with kStored
__host__ __device__ constexpr int sum_bytes(bool stored) { return stored ? 1024 : 256; }
// Threads of a backward block at most: where a thread has more than eight elements of a row it
// needs 168 registers, else 128 do.  (Rows of more than 4096 columns take 512 threads whatever
// that costs.)
constexpr int kBackBlock = 512, kBackWideBlock = 384;
// Teams of a block that meet at a barrier of their own: ids 1 to 15 (0 is the block's).
constexpr int kNamedBarriers = 15;

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint16_t lds2(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

// Rows on their way to this thread: kNA arrays, kNV pieces of kVec elements of each, `depth`
// slots.  Rows come in the order of the fetches, `stride` bytes apart.  Pieces of two bytes
// (an odd row of 16-bit elements) are copied at once instead.
template <typename T, int kVec, int kNV, int kNA, bool kWarpTeam, int kBlock>
struct Ring {
  static constexpr int kBytes = kVec * static_cast<int>(sizeof(T));
  static constexpr int kPiece = kBytes > 16 ? 16 : kBytes;
  static constexpr int kSplit = kBytes / kPiece;
  const char* src[kNA];  // this thread's first piece in the next row to fetch, or null
  int64_t stride;
  uint32_t base, slot_bytes, cur, nxt;  // shared-memory addresses of this thread's pieces
  int depth;
  __device__ __forceinline__ uint32_t gap() const {  // between a thread's pieces in shared memory
    return (kBlock > 0 ? kBlock : blockDim.x) * kPiece;
  }
  __device__ __forceinline__ void init(uint32_t smem, const Cols<kVec, kNV, kWarpTeam>& cols, int64_t row, int64_t step,
                                       int slots, const void* const (&from)[kNA]) {
    depth = slots;
    base = smem + threadIdx.x * kPiece;
    slot_bytes = kNA * kNV * kSplit * gap();
    cur = base;
    nxt = base;
    stride = step * cols.C * static_cast<int64_t>(sizeof(T));
#pragma unroll
    for (int a = 0; a < kNA; ++a)
      src[a] = from[a] == nullptr ? nullptr
                                  : static_cast<const char*>(from[a]) + (row * cols.C + cols.at(0)) * static_cast<int64_t>(sizeof(T));
  }
  __device__ __forceinline__ uint32_t after(uint32_t slot) const {
    return slot + slot_bytes == base + depth * slot_bytes ? base : slot + slot_bytes;
  }
  // starts bringing the next row (nothing if it is not `there`) into the next slot, as one group
  __device__ __forceinline__ void fetch(const Cols<kVec, kNV, kWarpTeam>& cols, bool there) {
    const uint32_t g = gap();
    const int step = cols.team() * kBytes;
#pragma unroll
    for (int a = 0; a < kNA; ++a) {
      if (src[a] == nullptr) continue;
      if (there) {
        const char* p = src[a];
        uint32_t dst = nxt + a * kNV * kSplit * g;
#pragma unroll
        for (int i = 0; i < kNV; ++i, p += step, dst += kSplit * g) {
          if (!cols.has(i)) continue;
          if constexpr (kBytes < 4) {
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst), "h"(*reinterpret_cast<const uint16_t*>(p)) : "memory");
          } else {
#pragma unroll
            for (int h = 0; h < kSplit; ++h) {
              if constexpr (kPiece == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + h * g), "l"(p + 16 * h) : "memory");
              else
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(p), "n"(kPiece) : "memory");
            }
          }
        }
      }
      src[a] += stride;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    nxt = after(nxt);
  }
  // the oldest row has landed
  __device__ __forceinline__ void wait() const {
    if (depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  __device__ __forceinline__ void done() { cur = after(cur); }
  // this thread's elements of array a in the oldest row; 0 past the row's end and of an array
  // that is not there
  __device__ __forceinline__ void read(const Cols<kVec, kNV, kWarpTeam>& cols, int a, Pairs<kVec * kNV>& to) const {
    float v[kVec * kNV];
    const uint32_t g = gap();
    uint32_t at = cur + a * kNV * kSplit * g;
#pragma unroll
    for (int i = 0; i < kNV; ++i, at += kSplit * g) {
      float e[kVec] = {};
      if (src[a] != nullptr && cols.has(i)) {
        if constexpr (kBytes == 2) {
          const uint16_t w = lds2(at);
          e[0] = to_f32(*reinterpret_cast<const T*>(&w));
        } else if constexpr (kVec == 1) {
          e[0] = __uint_as_float(lds4(at));
        } else if constexpr (kBytes == 4) {
          unpack(lds4(at), T(), e[0], e[1]);
        } else if constexpr (kBytes == 8) {
          const uint2 w = lds8(at);
          e[0] = __uint_as_float(w.x), e[1] = __uint_as_float(w.y);
        } else if constexpr (kBytes == 16) {
          const uint4 w = lds16(at);
          unpack(w.x, T(), e[0], e[1]);
          unpack(w.y, T(), e[2], e[3]);
          unpack(w.z, T(), e[4], e[5]);
          unpack(w.w, T(), e[6], e[7]);
        } else {
          const uint4 w = lds16(at), z = lds16(at + g);
          e[0] = __uint_as_float(w.x), e[1] = __uint_as_float(w.y), e[2] = __uint_as_float(w.z), e[3] = __uint_as_float(w.w);
          e[4] = __uint_as_float(z.x), e[5] = __uint_as_float(z.y), e[6] = __uint_as_float(z.z), e[7] = __uint_as_float(z.w);
        }
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[i * kVec + j] = e[j];
    }
    to.set(v);
  }
};

// kStored: a 16-bit stream is written, its pre norm is a layer norm and its statistics are kept.
template <typename T, int kVec, int kNV, bool kWarpTeam, bool kBias, bool kStored>
__global__ void __launch_bounds__(kWarpTeam ? 128 : 512, kWarpTeam ? 4 : 1) bsa_block_norm_kernel(const __grid_constant__ NormParams p,
                                                                               int team_threads) {
  constexpr int kE = kVec * kNV, kP = kE / 2;
  extern __shared__ __align__(16) uint8_t smem[];  // the reduction areas, then the ring
  const int teams = blockDim.x / team_threads, team = threadIdx.x / team_threads, t = threadIdx.x % team_threads;
  TeamSum<1, kWarpTeam> sum{reinterpret_cast<float*>(smem) + team * 64, team_threads, 1 + team};
  TeamSum<3, kWarpTeam> sum3{reinterpret_cast<float*>(smem) + teams * 64 + team * 192, team_threads, 1 + team};
  const Cols<kVec, kNV, kWarpTeam> cols(p.C, team_threads, t);
  const int step = gridDim.x * teams, rows = static_cast<int>(p.rows);  // rows and steps fit 31 bits
  int row = blockIdx.x * teams + team;
  Ring<T, kVec, kNV, 2, kWarpTeam, kWarpTeam ? kWarpBlock : 0> ring;
  ring.init(ptx::smem_addr(smem) + teams * sum_bytes(kStored), cols, row, step, p.depth, {p.x, p.y});
  int64_t ahead = row;  // the next row to fetch
  for (int d = 0; d + 1 < p.depth; ++d, ahead += step) ring.fetch(cols, ahead < rows);
  T* out = static_cast<T*>(p.out) + static_cast<int64_t>(row) * p.C + cols.at(0);
  T* normed = static_cast<T*>(p.normed) + static_cast<int64_t>(row) * p.C + cols.at(0);
  const int64_t stride = static_cast<int64_t>(step) * p.C;
  const bool f32 = p.params_f32 != 0;
  Pairs<kE> wpre, coef;  // pre weight; branch_scale gate post_weight of the gate row at hand
  {
    float w[kE];
    cols.template param<T>(p.pre_w, 0, f32, 1.f, w);
    wpre.set(w);
  }
  int64_t gate_end = 0;  // rows from here on have another gate row than coef's
  for (; row < rows; row = step > rows - row ? rows : row + step, out += stride, normed += stride) {
    ring.fetch(cols, ahead < rows);
    ahead += step;
    if (p.y != nullptr && row >= gate_end) {
      const uint32_t gate_row = static_cast<uint32_t>(row) / static_cast<uint32_t>(p.per_gate);
      gate_end = (gate_row + 1) * p.per_gate;
      float w[kE], g[kE];
      cols.template param<T>(p.post_w, 0, f32, 1.f, w);
      cols.template param<T>(p.gate, gate_row, f32, 1.f, g);
#pragma unroll
      for (int e = 0; e < kE; ++e) w[e] *= p.alpha * g[e];
      coef.set(w);
    }
    ring.wait();
    Pairs<kE> st;
    ring.read(cols, 0, st);
    float2 post = make_float2(0.f, 0.f), pre = make_float2(0.f, 0.f);
    if (p.y != nullptr) {
      Pairs<kE> y;
      ring.read(cols, 1, y);
      float r = 1.f;
      if (p.post != BSA_NORM_NONE) {
        post = statistics<kVec, kNV, kWarpTeam>(y, p.post, cols, p, sum);
        r = post.y;
      }
      const uint64_t r2 = twice(r), beta = twice(p.beta);
#pragma unroll
      for (int e = 0; e < kP; ++e)
        st.v[e] = ptx::ffma2(ptx::fmul2(y.v[e], r2), coef.v[e], ptx::fmul2(st.v[e], beta));
      if (kBias && p.post_b != nullptr) {
        float b[kE], g[kE];
        Pairs<kE> add;
        cols.template param<T>(p.post_b, 0, f32, 0.f, b);
        cols.template param<T>(p.gate, static_cast<uint32_t>(row) / static_cast<uint32_t>(p.per_gate), f32, 1.f, g);
#pragma unroll
        for (int e = 0; e < kE; ++e) b[e] *= p.alpha * g[e];
        add.set(b);
#pragma unroll
        for (int e = 0; e < kP; ++e) st.v[e] = ptx::fadd2(st.v[e], add.v[e]);
      }
      cols.store(out, st);
    }
    if (p.pre != BSA_NORM_NONE) {
      float r;
      if constexpr (kStored) {
        const float4 both = statistics_stored<T, kVec, kNV, kWarpTeam>(st, cols, p, sum, sum3);
        pre = make_float2(both.x, both.y);
        r = both.w;
      } else {
        pre = statistics<kVec, kNV, kWarpTeam>(st, p.pre, cols, p, sum);
        r = pre.y;
      }
      const uint64_t r2 = twice(r);
#pragma unroll
      for (int e = 0; e < kP; ++e) st.v[e] = ptx::fmul2(ptx::fmul2(st.v[e], r2), wpre.v[e]);
      if (kBias && p.pre_b != nullptr) {
        float b[kE];
        Pairs<kE> add;
        cols.template param<T>(p.pre_b, 0, f32, 0.f, b);
        add.set(b);
#pragma unroll
        for (int e = 0; e < kP; ++e) st.v[e] = ptx::fadd2(st.v[e], add.v[e]);
      }
      cols.store(normed, st);
    }
    if (p.stats != nullptr && t == 0)
      reinterpret_cast<float4*>(p.stats)[row] = make_float4(post.x, post.y, pre.x, pre.y);
    ring.done();
  }
}

// kMeans: a layer norm takes part or biases have gradients (the plain means, T and Q are kept).
// kBlock: threads of the block at most.
template <typename T, int kVec, int kNV, bool kWarpTeam, bool kMeans, int kBlock>
__global__ void __launch_bounds__(kBlock, 1) bsa_block_norm_back_kernel(const __grid_constant__ NormParams p,
                                                                        int team_threads) {
  constexpr int kE = kVec * kNV, kP = kE / 2;
  constexpr int kN = kMeans ? 2 : 1;
  extern __shared__ __align__(16) uint8_t smem[];  // three column buffers, the reduction areas, the ring
  const int teams = blockDim.x / team_threads, team = threadIdx.x / team_threads, t = threadIdx.x % team_threads;
  const Cols<kVec, kNV, kWarpTeam> cols(p.C, team_threads, t);
  float* buf = reinterpret_cast<float*>(smem);
  const int width = kE * cols.team();
  // the teams' sums; pre weight; branch_scale gate post_weight of the gate row at hand
  const ColBuf<kVec, kNV, kWarpTeam> sums{buf}, wpre{buf + width}, coef{buf + 2 * width};
  TeamSum<kN, kWarpTeam> sum{buf + 3 * width + team * (2 * kN * 32), team_threads, 1 + team};
  // rows fit 31 bits
  const int r0 = static_cast<int>(blockIdx.x * p.rows_per_block);
  const int r1 = static_cast<int>(min(blockIdx.x * p.rows_per_block + p.rows_per_block, p.rows));
  const bool f32 = p.params_f32 != 0;
  const bool pre_layer = p.pre == BSA_NORM_LAYER, post_layer = p.post == BSA_NORM_LAYER;

  // The block's rows go round its teams; a team's rows are one sequence for the ring, cut
  // where the gate row changes.
  int64_t row = r0 + team, ahead = row;
  Ring<T, kVec, kNV, 4, kWarpTeam, 0> ring;
  ring.init(ptx::smem_addr(smem) + (3 * width + teams * 2 * kN * 32) * static_cast<uint32_t>(sizeof(float)), cols, row,
            teams, p.depth, {p.dstream, p.y, p.dnormed == nullptr ? nullptr : p.x, p.dnormed});
  for (int d = 0; d + 1 < p.depth; ++d, ahead += teams) ring.fetch(cols, ahead < r1);
  T* dx = static_cast<T*>(p.dx) + row * p.C + cols.at(0);
  T* dy = static_cast<T*>(p.dy) + row * p.C + cols.at(0);
  const float4* saved = reinterpret_cast<const float4*>(p.saved);
  const int stride = teams * p.C;
  float4 st_next = make_float4(0.f, 0.f, 0.f, 0.f);
  if (row < r1) st_next = __ldg(saved + row);

  Pairs<kE> accP{}, accS{};
  Pairs<kMeans ? kE : 2> accQ{}, accT{};
  if (team == 0) {
    float w[kE];
    Pairs<kE> x;
    cols.template param<T>(p.pre_w, 0, f32, 1.f, w);
    x.set(w);
    wpre.store(cols, x);
  }
  // adds the teams' x in shared memory, in their order; the last writes the columns at `to`
  auto flush = [&](Pairs<kE> x, float* to) {
    for (int k = 0; k < teams; ++k) {
      if (team == k) {
        if (k > 0) {
          Pairs<kE> before;
          sums.load(cols, before);
#pragma unroll
          for (int e = 0; e < kP; ++e) x.v[e] = ptx::fadd2(before.v[e], x.v[e]);
        }
        if (k + 1 < teams) {
          sums.store(cols, x);
        } else {
          float v[kE];
          x.get(v);
#pragma unroll
          for (int i = 0; i < kNV; ++i)
#pragma unroll
            for (int j = 0; j < kVec; ++j)
              if (cols.has(i)) to[cols.at(i) + j] = v[i * kVec + j];
        }
      }
      __syncthreads();
    }
  };
  for (int64_t s0 = r0; s0 < r1;) {
    const int64_t gate_row = s0 / p.per_gate;
    const int64_t s1 = min(static_cast<int64_t>(r1), (gate_row + 1) * p.per_gate);
    __syncthreads();  // all teams are done with the last gate row's
    if (team == 0) {
      float w[kE], g[kE];
      Pairs<kE> x;
      cols.template param<T>(p.post_w, 0, f32, 1.f, w);
      cols.template param<T>(p.gate, gate_row, f32, 1.f, g);
#pragma unroll
      for (int e = 0; e < kE; ++e) w[e] *= p.alpha * g[e];
      x.set(w);
      coef.store(cols, x);
    }
    __syncthreads();
    for (; row < s1; row += teams, dx += stride, dy += stride) {
      ring.fetch(cols, ahead < r1);
      ahead += teams;
      const float4 st = st_next;
      if (row + teams < r1) st_next = __ldg(saved + row + teams);
      ring.wait();
      Pairs<kE> D;
      ring.read(cols, 0, D);
      if (p.dnormed != nullptr) {
        Pairs<kE> a, xh;
        ring.read(cols, 2, xh);
        ring.read(cols, 3, a);
        const uint64_t r2 = twice(st.w);
        uint64_t m0 = 0ull, m1 = 0ull;
        Pairs<kE> w;
        wpre.load(cols, w);
#pragma unroll
        for (int e = 0; e < kP; ++e) {
          if constexpr (kMeans) xh.v[e] = ptx::fadd2(xh.v[e], cols.inside(e, -st.z));
          xh.v[e] = ptx::fmul2(xh.v[e], r2);
          accP.v[e] = ptx::ffma2(a.v[e], xh.v[e], accP.v[e]);
          if constexpr (kMeans) accQ.v[e] = ptx::fadd2(accQ.v[e], a.v[e]);
          a.v[e] = ptx::fmul2(a.v[e], w.v[e]);
          m0 = ptx::ffma2(a.v[e], xh.v[e], m0);
          if constexpr (kMeans) m1 = ptx::fadd2(m1, a.v[e]);
        }
        float m[kN];
        m[0] = sum2(m0);
        if constexpr (kMeans) m[1] = sum2(m1);
        sum(m);
        const uint64_t c1 = twice(-m[0] * p.inv_c);
#pragma unroll
        for (int e = 0; e < kP; ++e) {
          uint64_t x = ptx::ffma2(xh.v[e], c1, a.v[e]);
          if constexpr (kMeans) x = ptx::fadd2(x, cols.inside(e, pre_layer ? -m[1] * p.inv_c : 0.f));
          D.v[e] = ptx::ffma2(x, r2, D.v[e]);
        }
      }
      {
        Pairs<kE> o;
        const uint64_t beta = twice(p.beta);
#pragma unroll
        for (int e = 0; e < kP; ++e) o.v[e] = ptx::fmul2(D.v[e], beta);
        cols.store(dx, o);
      }
      if (p.y != nullptr) {
        Pairs<kE> yh, w;
        ring.read(cols, 1, yh);
        coef.load(cols, w);
        const uint64_t r2 = twice(p.post != BSA_NORM_NONE ? st.y : 1.f);
        uint64_t m0 = 0ull, m1 = 0ull;
#pragma unroll
        for (int e = 0; e < kP; ++e) {
          if constexpr (kMeans) yh.v[e] = ptx::fadd2(yh.v[e], cols.inside(e, post_layer ? -st.x : 0.f));
          yh.v[e] = ptx::fmul2(yh.v[e], r2);
          accS.v[e] = ptx::ffma2(D.v[e], yh.v[e], accS.v[e]);
          if constexpr (kMeans) accT.v[e] = ptx::fadd2(accT.v[e], D.v[e]);
          D.v[e] = ptx::fmul2(D.v[e], w.v[e]);
          m0 = ptx::ffma2(D.v[e], yh.v[e], m0);
          if constexpr (kMeans) m1 = ptx::fadd2(m1, D.v[e]);
        }
        if (p.post != BSA_NORM_NONE) {
          float m[kN];
          m[0] = sum2(m0);
          if constexpr (kMeans) m[1] = sum2(m1);
          sum(m);
          const uint64_t c1 = twice(-m[0] * p.inv_c);
#pragma unroll
          for (int e = 0; e < kP; ++e) {
            D.v[e] = ptx::ffma2(yh.v[e], c1, D.v[e]);
            if constexpr (kMeans) D.v[e] = ptx::fadd2(D.v[e], twice(post_layer ? -m[1] * p.inv_c : 0.f));
            D.v[e] = ptx::fmul2(D.v[e], r2);
          }
        }
        cols.store(dy, D);
      }
      ring.done();
    }
    if (p.part != nullptr && p.y != nullptr) {
      float* to = p.part + (blockIdx.x + gate_row) * kN * p.C;
      flush(accS, to);
      accS = Pairs<kE>{};
      if constexpr (kMeans) {
        flush(accT, to + p.C);
        accT = Pairs<kE>{};
      }
    }
    s0 = s1;
  }
  if (p.part != nullptr && p.dnormed != nullptr && r0 < r1) {
    float* to = p.part_pre + static_cast<int64_t>(blockIdx.x) * kN * p.C;
    flush(accP, to);
    if constexpr (kMeans) flush(accQ, to + p.C);
  }
}

struct SumParams {
  const float *part, *part_pre;
  const void *post_w, *post_b, *gate;
  void *dpost_w, *dpost_b, *dgate, *dpre_w, *dpre_b;
  int64_t rows, per_gate, rows_per_block, blocks;
  int C, gate_rows, has_y, has_pre, param_type;
  int lanes_per_gate;  // of a column's lanes: power of two, lanes / it >= gate rows or 1
  float alpha;
};

__device__ __forceinline__ float param_at(const void* p, int64_t i, int type, float dflt) {
  if (p == nullptr) return dflt;
  if (type == BSA_FP32) return static_cast<const float*>(p)[i];
  if (type == BSA_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
  return to_f32(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void param_put(void* p, int64_t i, int type, float v) {
  if (p == nullptr) return;
  if (type == BSA_FP32) static_cast<float*>(p)[i] = v;
  else if (type == BSA_BF16) static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(v);
  else static_cast<__half*>(p)[i] = from_f32<__half>(v);
}

// Sums of slots first, first + step, .. < n of one column (two quantities C apart each): eight
// slots are on their way at once.
template <bool kMeans>
__device__ __forceinline__ void sum_slots(const float* from, int n, int first, int step, int C, float& a, float& b) {
  const int64_t stride = (kMeans ? 2 : 1) * static_cast<int64_t>(C), far = step * stride;
  from += first * stride;
  for (int k = first; k < n; k += 8 * step) {
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i, from += far) {
      const bool there = k + i * step < n;
      x[i] = there ? __ldg(from) : 0.f;
      y[i] = kMeans && there ? __ldg(from + C) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a += x[i];
      b += y[i];
    }
  }
}

// Adds the slots: 32 columns a block, blockDim.y lanes (warps) a column, the gate's and the post
// norm's sums in blocks with blockIdx.y = 0 and the pre norm's in those with 1.  Launched as the
// backward's programmatic dependent.  The backward triggers nothing early, so that these blocks come
// when its own have ended: what is saved is a launch's own time (65536 bf16 rows of 768: 119.8 us a
// pass, 121.3 as an ordinary launch; 4113 fp32 rows of 1030: 38.4 and 39.8).
template <bool kMeans>
__global__ void __launch_bounds__(1024) bsa_block_norm_sum_kernel(const SumParams p) {
  __shared__ float buf[2][32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x, ty = threadIdx.y, lanes = blockDim.y;
  const int c = blockIdx.x * 32 + lane;
  const bool in = c < p.C, post = blockIdx.y == 0;
  float dw = 0.f, db = 0.f;
  if (!post) {
    if (p.has_pre && in) sum_slots<kMeans>(p.part_pre + c, static_cast<int>(p.blocks), ty, lanes, p.C, dw, db);
  } else if (p.has_y) {
    // lane group `bb` of the lanes / lanes_per_gate takes gate rows bb, bb + groups, ...; its
    // lanes share the slots of one
    const int per = p.lanes_per_gate, sub = ty % per, bb = ty / per, groups = lanes / per;
    const float w = in ? param_at(p.post_w, c, p.param_type, 1.f) : 0.f;
    const float b = in ? param_at(p.post_b, c, p.param_type, 0.f) : 0.f;
    for (int64_t g = bb; g < p.gate_rows; g += groups) {
      // the blocks whose rows reach into this gate row
      const int64_t lo = g * p.per_gate / p.rows_per_block;
      const int64_t hi = p.rows == 0 ? -1 : min((min((g + 1) * p.per_gate, p.rows) - 1) / p.rows_per_block, p.blocks - 1);
      float S = 0.f, T = 0.f;
      if (in)
        sum_slots<kMeans>(p.part + (g + lo) * (kMeans ? 2 : 1) * p.C + c, static_cast<int>(hi - lo + 1), sub, per, p.C, S, T);
      if (per > 1) {
        // groups * per = lanes and one pass: every lane comes here at most once
        buf[0][ty][lane] = S;
        buf[1][ty][lane] = T;
      } else {
        const float gt = in ? param_at(p.gate, g * p.C + c, p.param_type, 1.f) : 0.f;
        if (in) param_put(p.dgate, g * p.C + c, p.param_type, p.alpha * (w * S + b * T));
        dw = fmaf(p.alpha * gt, S, dw);
        db = fmaf(p.alpha * gt, T, db);
      }
    }
    __syncthreads();
    if (per > 1 && sub == 0 && bb < p.gate_rows) {
      float S = 0.f, T = 0.f;
      for (int k = 0; k < per; ++k) {
        S += buf[0][ty + k][lane];
        T += buf[1][ty + k][lane];
      }
      const float gt = in ? param_at(p.gate, static_cast<int64_t>(bb) * p.C + c, p.param_type, 1.f) : 0.f;
      if (in) param_put(p.dgate, static_cast<int64_t>(bb) * p.C + c, p.param_type, p.alpha * (w * S + b * T));
      dw = p.alpha * gt * S;
      db = p.alpha * gt * T;
    }
    __syncthreads();
  }
  buf[0][ty][lane] = dw;
  buf[1][ty][lane] = db;
  __syncthreads();
  if (ty < 2 && in) {
    float s = 0.f;
    for (int k = 0; k < lanes; ++k) s += buf[ty][k][lane];
    param_put(post ? (ty == 0 ? p.dpost_w : p.dpost_b) : (ty == 0 ? p.dpre_w : p.dpre_b), c, p.param_type, s);
  }
}

// ------------------------------------------------------------ host
// How a row is laid over threads and blocks over SMs.
struct Team {
  int vec, nv;           // elements a piece, pieces a thread
  int threads, teams;    // threads a team, teams a block
  int depth, per_sm;     // slots of the ring, blocks on an SM
  size_t smem;
  bool warp;             // a warp a row, without barriers
};

constexpr size_t kSmemMost = 220 * 1024;
constexpr int kSmemBlock = 227 * 1024;  // what a block can have, and no layout of team_of is above

// means: the backward's kMeans, or the forward's kStored.
Team team_of(int C, size_t esize, bool aligned, bool backward, bool means) {
  Team t{};
  t.vec = aligned && C % 8 == 0 ? 8 : aligned && C % 2 == 0 ? 2 : 1;
  const int n = C / t.vec;
  // A warp takes a row while a lane's share fits its registers (the backward keeps two sums
  // a column, four with plain means), else the block, with as many elements a thread as 384
  // threads have registers for: what a team does once a row, its sums, is then shared by
  // fewer warps (4113 fp32 rows of 1030, backward: 4, 6 pieces of two took 46, 38 us).
  const int most = t.vec < 8 ? 0 : backward && means ? 2 : 3;
  if (n <= 32 * most) {
    t.nv = (n + 31) / 32;
    t.threads = 32;
    t.warp = true;
  } else {
    t.nv = t.vec == 8 ? (n <= 512 ? 1 : 2) : t.vec == 2 ? (n <= 2048 ? 6 : 8) : (n <= 4096 ? 12 : 16);
    t.threads = ((n + t.nv - 1) / t.nv + 31) / 32 * 32;
  }
  const auto slot = [&] { return static_cast<size_t>(t.threads * t.teams) * (backward ? 4 : 2) * t.nv * t.vec * esize; };
  if (!backward) {
    // about 128 registers a thread
    t.teams = t.warp ? kWarpBlock / 32 : std::max(1, 256 / t.threads);
    t.per_sm = std::max(1, 512 / (t.threads * t.teams));
    const size_t fixed = t.teams * sum_bytes(means);
    t.depth = 3;
    while (t.depth > 1 && (fixed + t.depth * slot() + 1024) * t.per_sm > kSmemMost) --t.depth;
    while (t.per_sm > 1 && (fixed + t.depth * slot() + 1024) * t.per_sm > kSmemMost) --t.per_sm;
    t.smem = fixed + t.depth * slot();
    return t;
  }
  // one block an SM, of as many teams as leave room for two rows on their way in each
  t.per_sm = 1;
  const auto fixed = [&] {
    return (3 * static_cast<size_t>(t.nv * t.vec) * t.threads + t.teams * 2 * (means ? 2 : 1) * 32) * sizeof(float);
  };
  t.teams = std::max(1, (t.nv * t.vec > 8 ? kBackWideBlock : kBackBlock) / t.threads);
  if (!t.warp) t.teams = std::min(t.teams, kNamedBarriers);
  t.depth = 2;
  while (t.teams > 1 && fixed() + 2 * slot() > kSmemMost) --t.teams;
  if (fixed() + 2 * slot() > kSmemMost) t.depth = 1;
  else if (fixed() + 3 * slot() <= kSmemMost) t.depth = 3;
  t.smem = fixed() + t.depth * slot();
  return t;
}

bool all_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p != nullptr && !aligned16(p)) return false;
  return true;
}

int check_args(const bsa_block_norm_args* a) {
  if (a == nullptr) return BSA_ERR_INVALID_ARG;
  if (a->B < 0 || a->rows_per_batch < 0 || a->C < 1) return BSA_ERR_INVALID_ARG;
  if (!is_float_type(a->type) || (a->param_type != a->type && a->param_type != BSA_FP32) || a->C > kMaxCols)
    return BSA_ERR_UNSUPPORTED;
  if (a->post < BSA_NORM_NONE || a->post > BSA_NORM_LAYER || a->pre < BSA_NORM_NONE || a->pre > BSA_NORM_LAYER)
    return BSA_ERR_INVALID_ARG;
  if (a->post == BSA_NORM_NONE && (a->post_weight != nullptr || a->post_bias != nullptr)) return BSA_ERR_INVALID_ARG;
  if (a->pre == BSA_NORM_NONE && (a->pre_weight != nullptr || a->pre_bias != nullptr)) return BSA_ERR_INVALID_ARG;
  if (a->gate_rows != 1 && a->gate_rows != a->B) return BSA_ERR_INVALID_ARG;
  if (!(a->eps >= 0.f) || a->branch_scale != a->branch_scale || a->stream_scale != a->stream_scale)
    return BSA_ERR_INVALID_ARG;
  const size_t ps = type_bytes(a->param_type);
  for (const void* p : {a->post_weight, a->post_bias, a->gate, a->pre_weight, a->pre_bias})
    if (reinterpret_cast<uintptr_t>(p) % ps != 0) return BSA_ERR_INVALID_ARG;
  return BSA_OK;
}

bool misaligned(int type, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % type_bytes(type) != 0) return true;
  return false;
}

void fill(NormParams& p, const bsa_block_norm_args& a) {
  p.post_w = a.post_weight, p.post_b = a.post_bias, p.gate = a.gate, p.pre_w = a.pre_weight, p.pre_b = a.pre_bias;
  p.rows = static_cast<int64_t>(a.B) * a.rows_per_batch;
  p.per_gate = a.gate_rows == 1 ? std::max<int64_t>(p.rows, 1) : std::max(a.rows_per_batch, 1);
  p.C = a.C, p.post = a.post, p.pre = a.pre;
  p.params_f32 = a.param_type == BSA_FP32;
  p.alpha = a.branch_scale, p.beta = a.stream_scale, p.eps = a.eps;
  p.inv_c = 1.f / static_cast<float>(a.C);
}

// The limit of a kernel's dynamic shared memory belongs to the process, and one kernel serves many
// sizes: it is only ever set to the block's most, so that a call from another thread never finds
// it below its own size.  False where the launch was refused: what reads the kernel's results is
// not launched then.
template <typename F>
bool start(F* kernel, const NormParams& p, const Team& t, int64_t blocks, cudaStream_t s) {
  if (t.smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBlock) != cudaSuccess)
    return false;
  kernel<<<static_cast<unsigned>(blocks), t.threads * t.teams, t.smem, s>>>(p, t.threads);
  return cudaPeekAtLastError() == cudaSuccess;
}

template <typename T, bool kBias, bool kStored>
bool launch_norm(const NormParams& p, const Team& t, int64_t blocks, cudaStream_t s) {
  if (t.warp) {
    if (t.nv == 1) return start(bsa_block_norm_kernel<T, 8, 1, true, kBias, kStored>, p, t, blocks, s);
    if (t.nv == 2) return start(bsa_block_norm_kernel<T, 8, 2, true, kBias, kStored>, p, t, blocks, s);
    return start(bsa_block_norm_kernel<T, 8, 3, true, kBias, kStored>, p, t, blocks, s);
  }
  if (t.vec == 8)
    return t.nv == 1 ? start(bsa_block_norm_kernel<T, 8, 1, false, kBias, kStored>, p, t, blocks, s)
                     : start(bsa_block_norm_kernel<T, 8, 2, false, kBias, kStored>, p, t, blocks, s);
  if (t.vec == 2)
    return t.nv == 6 ? start(bsa_block_norm_kernel<T, 2, 6, false, kBias, kStored>, p, t, blocks, s)
                     : start(bsa_block_norm_kernel<T, 2, 8, false, kBias, kStored>, p, t, blocks, s);
  return t.nv == 12 ? start(bsa_block_norm_kernel<T, 1, 12, false, kBias, kStored>, p, t, blocks, s)
                   : start(bsa_block_norm_kernel<T, 1, 16, false, kBias, kStored>, p, t, blocks, s);
}
template <typename T>
bool launch_norm(NormParams p, const Team& t, bool stored, int sms, cudaStream_t s) {
  p.depth = t.depth;
  const int64_t blocks = std::min<int64_t>((p.rows + t.teams - 1) / t.teams, static_cast<int64_t>(sms) * t.per_sm);
  const bool bias = p.post_b != nullptr || p.pre_b != nullptr;
  if constexpr (sizeof(T) == 2)
    if (stored) return bias ? launch_norm<T, true, true>(p, t, blocks, s) : launch_norm<T, false, true>(p, t, blocks, s);
  return bias ? launch_norm<T, true, false>(p, t, blocks, s) : launch_norm<T, false, false>(p, t, blocks, s);
}

struct BackPlan {
  int64_t blocks, rows_per_block, slots;
  size_t bytes;
};

// Contiguous rows for each block, at least one a team.
BackPlan back_plan(const NormParams& p, const Team& t, int gate_rows, bool means, int sms) {
  BackPlan b;
  const int64_t most = std::max<int64_t>(1, (p.rows + t.teams - 1) / t.teams);
  b.blocks = std::min<int64_t>(static_cast<int64_t>(sms) * t.per_sm, most);
  b.rows_per_block = std::max<int64_t>(1, (p.rows + b.blocks - 1) / b.blocks);
  b.blocks = (p.rows + b.rows_per_block - 1) / b.rows_per_block;
  b.slots = b.blocks + gate_rows;
  b.bytes = static_cast<size_t>(b.slots + b.blocks) * (means ? 2 : 1) * p.C * sizeof(float);
  return b;
}

template <typename T, bool kMeans>
bool launch_back(const NormParams& p, const Team& t, const BackPlan& b, cudaStream_t s) {
  constexpr int kB = kBackBlock, kW = kBackWideBlock;
  if (t.warp) {
    if (t.nv == 1) return start(bsa_block_norm_back_kernel<T, 8, 1, true, kMeans, kB>, p, t, b.blocks, s);
    if constexpr (!kMeans)
      if (t.nv == 3) return start(bsa_block_norm_back_kernel<T, 8, 3, true, kMeans, kW>, p, t, b.blocks, s);
    return start(bsa_block_norm_back_kernel<T, 8, 2, true, kMeans, kW>, p, t, b.blocks, s);
  }
  if (t.vec == 8)
    return t.nv == 1 ? start(bsa_block_norm_back_kernel<T, 8, 1, false, kMeans, kB>, p, t, b.blocks, s)
                     : start(bsa_block_norm_back_kernel<T, 8, 2, false, kMeans, kB>, p, t, b.blocks, s);
  if (t.vec == 2)
    return t.nv == 6 ? start(bsa_block_norm_back_kernel<T, 2, 6, false, kMeans, kW>, p, t, b.blocks, s)
                     : start(bsa_block_norm_back_kernel<T, 2, 8, false, kMeans, kB>, p, t, b.blocks, s);
  return t.nv == 12 ? start(bsa_block_norm_back_kernel<T, 1, 12, false, kMeans, kW>, p, t, b.blocks, s)
                   : start(bsa_block_norm_back_kernel<T, 1, 16, false, kMeans, kB>, p, t, b.blocks, s);
}

bool takes_means(const bsa_block_norm_args& a) { return a.post == BSA_NORM_LAYER || a.pre == BSA_NORM_LAYER; }
// T and Q are also what the gradients of biases are made of.
bool keeps_means(const bsa_block_norm_args& a) {
  return takes_means(a) || a.post_bias != nullptr || a.pre_bias != nullptr;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" {

int bsa_block_norm(const bsa_block_norm_args* args, const void* x, const void* y, void* stream_out, void* normed,
                   float* stats, void* stream) {
  const int st = check_args(args);
  if (st != BSA_OK) return st;
  const bsa_block_norm_args& a = *args;
  NormParams p{};
  fill(p, a);
  if (p.rows == 0) return BSA_OK;
  if (x == nullptr || (y != nullptr && stream_out == nullptr) || (a.pre != BSA_NORM_NONE && normed == nullptr))
    return BSA_ERR_INVALID_ARG;
  if (y == nullptr && (a.post != BSA_NORM_NONE || a.gate != nullptr || a.pre == BSA_NORM_NONE))
    return BSA_ERR_INVALID_ARG;
  if (y != nullptr && a.pre != BSA_NORM_NONE && stream_out == normed) return BSA_ERR_INVALID_ARG;
  if (p.rows > 0x7fffffff || misaligned(a.type, {x, y, stream_out, normed}) ||
      (stats != nullptr && !aligned16(stats)))
    return BSA_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms < 0) return sms;
  const bool aligned = all_aligned({x, y, stream_out, normed, a.post_weight, a.post_bias, a.gate, a.pre_weight,
                                    a.pre_bias});
  p.x = x, p.y = y, p.out = stream_out, p.normed = normed, p.stats = stats;
  // an fp32 stream is stored as it is, and without y there is nothing to round
  const bool stored = y != nullptr && stats != nullptr && a.pre == BSA_NORM_LAYER && a.type != BSA_FP32;
  const Team t = team_of(a.C, type_bytes(a.type), aligned, false, stored);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool ok = a.type == BSA_BF16   ? launch_norm<__nv_bfloat16>(p, t, stored, sms, s)
                  : a.type == BSA_FP16 ? launch_norm<__half>(p, t, stored, sms, s)
                                       : launch_norm<float>(p, t, stored, sms, s);
  return cudaGetLastError() == cudaSuccess && ok ? BSA_OK : BSA_ERR_CUDA;
}

int bsa_block_norm_backward_workspace_bytes(const bsa_block_norm_args* args, size_t* bytes) {
  const int st = check_args(args);
  if (st != BSA_OK) return st;
  if (bytes == nullptr) return BSA_ERR_INVALID_ARG;
  NormParams p{};
  fill(p, *args);
  const int sms = sm_count();
  if (sms < 0) return sms;
  // the larger of both layouts: which one runs depends on the alignment of the call
  const bool means = keeps_means(*args);
  size_t most = 0;
  for (const bool aligned : {false, true})
    most = std::max(most, back_plan(p, team_of(args->C, type_bytes(args->type), aligned, true, means),
                                    args->gate_rows, means, sms).bytes);
  *bytes = (most + 255) / 256 * 256;
  return BSA_OK;
}

int bsa_block_norm_backward(const bsa_block_norm_args* args, const void* dstream, const void* dnormed,
                            const void* x, const void* y, const float* stats, void* dx, void* dy,
                            void* dpost_weight, void* dpost_bias, void* dgate, void* dpre_weight,
                            void* dpre_bias, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_args(args);
  if (st != BSA_OK) return st;
  const bsa_block_norm_args& a = *args;
  NormParams p{};
  fill(p, a);
  const bool sums = dpost_weight != nullptr || dpost_bias != nullptr || dgate != nullptr || dpre_weight != nullptr ||
                    dpre_bias != nullptr;
  // a gradient is of a parameter that the call has
  if ((dpost_weight != nullptr && a.post_weight == nullptr) || (dpost_bias != nullptr && a.post_bias == nullptr) ||
      (dgate != nullptr && a.gate == nullptr) || (dpre_weight != nullptr && a.pre_weight == nullptr) ||
      (dpre_bias != nullptr && a.pre_bias == nullptr))
    return BSA_ERR_INVALID_ARG;
  if (p.rows > 0) {
    if (x == nullptr || dx == nullptr || stats == nullptr || (y != nullptr) != (dy != nullptr))
      return BSA_ERR_INVALID_ARG;
    if (y == nullptr && (a.post != BSA_NORM_NONE || a.gate != nullptr || a.pre == BSA_NORM_NONE))
      return BSA_ERR_INVALID_ARG;
    if ((dnormed != nullptr && a.pre == BSA_NORM_NONE) || dx == dy) return BSA_ERR_INVALID_ARG;
    if (p.rows > 0x7fffffff || misaligned(a.type, {x, y, dstream, dnormed, dx, dy}) || !aligned16(stats))
      return BSA_ERR_INVALID_ARG;
  }
  if (misaligned(a.param_type, {dpost_weight, dpost_bias, dgate, dpre_weight, dpre_bias})) return BSA_ERR_INVALID_ARG;
  const bool means = keeps_means(a);
  const int sms = sm_count();
  if (sms < 0) return sms;
  const bool aligned = all_aligned({x, y, dstream, dnormed, dx, dy, a.post_weight, a.gate, a.pre_weight});
  const Team t = team_of(a.C, type_bytes(a.type), aligned, true, means);
  const BackPlan b = back_plan(p, t, a.gate_rows, means, sms);
  if (sums && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || workspace_bytes < b.bytes))
    return BSA_ERR_WORKSPACE;
  p.x = x, p.y = y, p.dstream = dstream, p.dnormed = dnormed, p.saved = stats, p.dx = dx, p.dy = dy;
  if (y == nullptr) p.beta = 1.f;  // the stream is x itself
  p.part = sums ? static_cast<float*>(workspace) : nullptr;
  p.part_pre = sums ? p.part + b.slots * (means ? 2 : 1) * a.C : nullptr;
  p.rows_per_block = b.rows_per_block;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.depth = t.depth;
  bool ok = true;
  if (p.rows > 0) {
    if (a.type == BSA_BF16)
      ok = means ? launch_back<__nv_bfloat16, true>(p, t, b, s) : launch_back<__nv_bfloat16, false>(p, t, b, s);
    else if (a.type == BSA_FP16)
      ok = means ? launch_back<__half, true>(p, t, b, s) : launch_back<__half, false>(p, t, b, s);
    else
      ok = means ? launch_back<float, true>(p, t, b, s) : launch_back<float, false>(p, t, b, s);
  }
  if (sums) {
    SumParams q{};
    q.part = p.part, q.part_pre = p.part_pre;
    q.post_w = a.post_weight, q.post_b = a.post_bias, q.gate = a.gate;
    q.dpost_w = dpost_weight, q.dpost_b = dpost_bias, q.dgate = dgate, q.dpre_w = dpre_weight, q.dpre_b = dpre_bias;
    q.rows = p.rows, q.per_gate = p.per_gate, q.rows_per_block = b.rows_per_block, q.blocks = b.blocks;
    q.C = a.C, q.gate_rows = a.gate_rows;
    q.has_y = p.rows == 0 || y != nullptr;
    q.has_pre = dnormed != nullptr;
    q.param_type = a.param_type, q.alpha = a.branch_scale;
    // few lanes start and end sooner; more share many gate rows
    const int lanes = a.gate_rows <= 8 ? 8 : 32;
    int per = 1;
    while (per < lanes && lanes / (2 * per) >= a.gate_rows) per *= 2;
    q.lanes_per_gate = per;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((a.C + 31) / 32, 2);
    cfg.blockDim = dim3(32, lanes);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = p.rows > 0 ? 1 : 0;  // the backward comes directly before, unless it had no rows
    ok = ok && (means ? cudaLaunchKernelEx(&cfg, bsa_block_norm_sum_kernel<true>, q)
                      : cudaLaunchKernelEx(&cfg, bsa_block_norm_sum_kernel<false>, q)) == cudaSuccess;
  }
  return cudaGetLastError() == cudaSuccess && ok ? BSA_OK : BSA_ERR_CUDA;
}

}  // extern "C"
