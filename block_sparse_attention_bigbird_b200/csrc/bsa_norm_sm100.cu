// The norms before and after a block, fused with its gate and residual, for B200 (sm_100a):
//
//     z      = N_post(y) w_post + b_post,   stream = beta x + alpha g z,
//     normed = N_pre(stream) w_pre + b_pre,
//
// and the gradients of both outputs.  N is rms or layer normalisation over a row's C columns.
//
// Forward.  A row is held in the registers of one team of threads (a warp up to 1024
// columns, else the block), so that x and y are read once and both outputs written once;
// means, variances (of the centred values) and the residual are fp32 in registers.
//
// Backward, with D the gradient of the stream by both its uses:
//     a  = dnormed w_pre,  D = dstream + r (a - mean(a) - xh mean(a xh)),   dx = beta D,
//     c  = alpha g D w_post,  dy = r' (c - mean(c) - yh mean(c yh)),
// with xh, yh the normalised stream and y, r and r' the saved 1/sqrt(..), and the plain
// means only for layer norms.  The sums over rows need four quantities a column:
//     S = sum D yh, T = sum D  (over the rows of one gate row),
//     P = sum dnormed xh, Q = sum dnormed,
// because dgate = alpha (w_post S + b_post T), dw_post = alpha sum_b g_b S_b,
// db_post = alpha sum_b g_b T_b, dw_pre = P, db_pre = Q.  A block keeps them in registers
// over its contiguous rows (every thread owns fixed columns), adds its teams' sums in shared
// memory when the gate row changes or its rows end, and writes them to slot
// (block + gate row), which no two (block, gate row) pairs share.  A second kernel adds the
// slots in a fixed order.
//
// What bounds both: the bytes of the activations; parameters stay in L1 and L2.
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "bsa_elem.cuh"

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
};

template <typename T, int kVec>
__device__ __forceinline__ void load_param(const void* p, int c, bool f32, float dflt, float (&v)[kVec]) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = dflt;
  } else if (f32) {
    Elems<kVec, float>::load(static_cast<const float*>(p) + c, v);
  } else {
    Elems<kVec, T>::load(static_cast<const T*>(p) + c, v);
  }
}

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
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        float s = lane < nw ? b[i * 32 + lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        v[i] = s;
      }
    }
  }
};

// Normalises v (in place) over the team's row: rms or layer; returns (mean, 1 / sqrt(..)).
template <int kE, bool kWarpTeam>
__device__ __forceinline__ float2 normalise(float (&v)[kE], int kind, int valid, const NormParams& p,
                                            TeamSum<1, kWarpTeam>& sum) {
  float mean = 0.f;
  float s[1];
  if (kind == BSA_NORM_LAYER) {
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < kE; ++i) s[0] += v[i];  // columns past C hold 0
    sum(s);
    mean = s[0] * p.inv_c;
#pragma unroll
    for (int i = 0; i < kE; ++i) v[i] = i < valid ? v[i] - mean : 0.f;
  }
  s[0] = 0.f;
#pragma unroll
  for (int i = 0; i < kE; ++i) s[0] = fmaf(v[i], v[i], s[0]);
  sum(s);
  const float r = 1.f / sqrtf(fmaf(s[0], p.inv_c, p.eps));
#pragma unroll
  for (int i = 0; i < kE; ++i) v[i] *= r;
  return make_float2(mean, r);
}

// Thread t of a team owns the columns (i * team + t) * kVec .. + kVec of its row, i < kNV.
template <typename T, int kVec, int kNV, bool kWarpTeam>
__global__ void __launch_bounds__(kWarpTeam ? 128 : 512) bsa_block_norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int kE = kVec * kNV;
  __shared__ float red[2 * 32];
  const int team_threads = kWarpTeam ? 32 : blockDim.x;
  const int t = threadIdx.x % team_threads;
  TeamSum<1, kWarpTeam> sum{red, team_threads, 1};
  const int64_t row = kWarpTeam ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)
                                : static_cast<int64_t>(blockIdx.x);
  if (row >= p.rows) return;  // whole teams
  const int64_t at = row * p.C;
  int valid = 0;  // elements of this thread inside the row
#pragma unroll
  for (int i = 0; i < kNV; ++i)
    if ((i * team_threads + t) * kVec < p.C) valid = (i + 1) * kVec;
  float st[kE];
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = (i * team_threads + t) * kVec;
    float v[kVec] = {};
    if (c < p.C) Elems<kVec, T>::load(static_cast<const T*>(p.x) + at + c, v);
#pragma unroll
    for (int j = 0; j < kVec; ++j) st[i * kVec + j] = v[j];
  }
  float2 post = make_float2(0.f, 0.f), pre = make_float2(0.f, 0.f);
  if (p.y != nullptr) {
    float y[kE];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * team_threads + t) * kVec;
      float v[kVec] = {};
      if (c < p.C) Elems<kVec, T>::load(static_cast<const T*>(p.y) + at + c, v);
#pragma unroll
      for (int j = 0; j < kVec; ++j) y[i * kVec + j] = v[j];
    }
    if (p.post != BSA_NORM_NONE) post = normalise<kE, kWarpTeam>(y, p.post, valid, p, sum);
    const int64_t g0 = row / p.per_gate * p.C;
    const bool f32 = p.params_f32 != 0;
    const void* gate = p.gate == nullptr ? nullptr
                       : f32             ? static_cast<const void*>(static_cast<const float*>(p.gate) + g0)
                                         : static_cast<const void*>(static_cast<const T*>(p.gate) + g0);
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * team_threads + t) * kVec;
      if (c >= p.C) continue;
      float w[kVec], b[kVec], g[kVec], o[kVec];
      load_param<T, kVec>(p.post_w, c, f32, 1.f, w);
      load_param<T, kVec>(p.post_b, c, f32, 0.f, b);
      load_param<T, kVec>(gate, c, f32, 1.f, g);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float z = fmaf(y[i * kVec + j], w[j], b[j]);
        o[j] = st[i * kVec + j] = fmaf(p.alpha * g[j], z, p.beta * st[i * kVec + j]);
      }
      Elems<kVec, T>::store(static_cast<T*>(p.out) + at + c, o);
    }
  }
  if (p.pre != BSA_NORM_NONE) {
    pre = normalise<kE, kWarpTeam>(st, p.pre, valid, p, sum);
    const bool f32 = p.params_f32 != 0;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * team_threads + t) * kVec;
      if (c >= p.C) continue;
      float w[kVec], b[kVec], o[kVec];
      load_param<T, kVec>(p.pre_w, c, f32, 1.f, w);
      load_param<T, kVec>(p.pre_b, c, f32, 0.f, b);
#pragma unroll
      for (int j = 0; j < kVec; ++j) o[j] = fmaf(st[i * kVec + j], w[j], b[j]);
      Elems<kVec, T>::store(static_cast<T*>(p.normed) + at + c, o);
    }
  }
  if (p.stats != nullptr && t == 0)
    reinterpret_cast<float4*>(p.stats)[row] = make_float4(post.x, post.y, pre.x, pre.y);
}

// kMeans: a layer norm takes part (the plain means, T and Q are kept).
template <typename T, int kVec, int kNV, bool kWarpTeam, bool kMeans>
__global__ void __launch_bounds__(kWarpTeam ? 256 : 512) bsa_block_norm_back_kernel(const __grid_constant__ NormParams p,
                                                                                    int team_threads) {
  constexpr int kE = kVec * kNV;
  constexpr int kN = kMeans ? 2 : 1;
  extern __shared__ float smem[];  // [C] sums of the block's teams, then the teams' reduction areas
  const int team = threadIdx.x / team_threads, teams = blockDim.x / team_threads;
  const int t = threadIdx.x % team_threads;
  TeamSum<kN, kWarpTeam> sum{smem + p.C + team * (2 * kN * 32), team_threads, 1 + team};
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_block;
  const int64_t r1 = min(r0 + p.rows_per_block, p.rows);
  const bool f32 = p.params_f32 != 0;
  const bool pre_layer = p.pre == BSA_NORM_LAYER, post_layer = p.post == BSA_NORM_LAYER;

  float accP[kE] = {}, accQ[kMeans ? kE : 1] = {};
  // adds the teams' v in shared memory and writes it to C floats at `to`
  auto flush = [&](const float* v, float* to) {
    for (int k = 0; k < teams; ++k) {
      if (team == k) {
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
          const int c = (i * team_threads + t) * kVec;
          if (c < p.C)
#pragma unroll
            for (int j = 0; j < kVec; ++j) smem[c + j] = k == 0 ? v[i * kVec + j] : smem[c + j] + v[i * kVec + j];
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < p.C; c += blockDim.x) to[c] = smem[c];
    __syncthreads();
  };

  for (int64_t s0 = r0; s0 < r1;) {
    const int64_t gate_row = s0 / p.per_gate;
    const int64_t s1 = min(r1, (gate_row + 1) * p.per_gate);
    const int64_t g0 = gate_row * p.C;
    const void* gate = p.gate == nullptr ? nullptr
                       : f32             ? static_cast<const void*>(static_cast<const float*>(p.gate) + g0)
                                         : static_cast<const void*>(static_cast<const T*>(p.gate) + g0);
    float accS[kE] = {}, accT[kMeans ? kE : 1] = {};
    for (int64_t row = s0 + team; row < s1; row += teams) {
      const int64_t at = row * p.C;
      const float4 st = reinterpret_cast<const float4*>(p.saved)[row];
      float D[kE];
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * team_threads + t) * kVec;
        float v[kVec] = {};
        if (p.dstream != nullptr && c < p.C) Elems<kVec, T>::load(static_cast<const T*>(p.dstream) + at + c, v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) D[i * kVec + j] = v[j];
      }
      float yh[kE];
      if (p.y != nullptr) {
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
          const int c = (i * team_threads + t) * kVec;
          float v[kVec] = {};
          if (c < p.C) Elems<kVec, T>::load(static_cast<const T*>(p.y) + at + c, v);
#pragma unroll
          for (int j = 0; j < kVec; ++j)
            yh[i * kVec + j] = p.post == BSA_NORM_NONE ? v[j] : c < p.C ? (v[j] - st.x) * st.y : 0.f;
        }
      }
      if (p.dnormed != nullptr) {
        float a[kE], xh[kE], m[kN] = {};
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
          const int c = (i * team_threads + t) * kVec;
          float v[kVec] = {}, d[kVec] = {}, w[kVec] = {};
          if (c < p.C) {
            Elems<kVec, T>::load(static_cast<const T*>(p.x) + at + c, v);
            Elems<kVec, T>::load(static_cast<const T*>(p.dnormed) + at + c, d);
            load_param<T, kVec>(p.pre_w, c, f32, 1.f, w);
          }
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            const int e = i * kVec + j;
            xh[e] = c < p.C ? (v[j] - st.z) * st.w : 0.f;
            accP[e] = fmaf(d[j], xh[e], accP[e]);
            if constexpr (kMeans) accQ[e] += d[j];
            a[e] = d[j] * w[j];
            m[0] = fmaf(a[e], xh[e], m[0]);
            if constexpr (kMeans) m[1] += a[e];
          }
        }
        sum(m);
        const float c1 = m[0] * p.inv_c;
        float c2 = 0.f;
        if constexpr (kMeans) c2 = pre_layer ? m[1] * p.inv_c : 0.f;
#pragma unroll
        for (int e = 0; e < kE; ++e) D[e] = fmaf(st.w, a[e] - c2 - xh[e] * c1, D[e]);
      }
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * team_threads + t) * kVec;
        float o[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) o[j] = p.beta * D[i * kVec + j];
        if (c < p.C) Elems<kVec, T>::store(static_cast<T*>(p.dx) + at + c, o);
      }
      if (p.y == nullptr) continue;
      float m[kN] = {};
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * team_threads + t) * kVec;
        float w[kVec] = {}, g[kVec] = {};
        if (c < p.C) {
          load_param<T, kVec>(p.post_w, c, f32, 1.f, w);
          load_param<T, kVec>(gate, c, f32, 1.f, g);
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const int e = i * kVec + j;
          if (c < p.C) {
            accS[e] = fmaf(D[e], yh[e], accS[e]);
            if constexpr (kMeans) accT[e] += D[e];
          }
          D[e] = c < p.C ? p.alpha * g[j] * w[j] * D[e] : 0.f;
          m[0] = fmaf(D[e], yh[e], m[0]);
          if constexpr (kMeans) m[1] += D[e];
        }
      }
      float c1 = 0.f, c2 = 0.f, r = 1.f;
      if (p.post != BSA_NORM_NONE) {
        sum(m);
        c1 = m[0] * p.inv_c;
        if constexpr (kMeans) c2 = post_layer ? m[1] * p.inv_c : 0.f;
        r = st.y;
      }
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * team_threads + t) * kVec;
        float o[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) o[j] = r * (D[i * kVec + j] - c2 - yh[i * kVec + j] * c1);
        if (c < p.C) Elems<kVec, T>::store(static_cast<T*>(p.dy) + at + c, o);
      }
    }
    if (p.part != nullptr && p.y != nullptr) {
      float* to = p.part + (blockIdx.x + gate_row) * kN * p.C;
      flush(accS, to);
      if constexpr (kMeans) flush(accT, to + p.C);
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
  int C, gate_rows, means, has_y, has_pre, param_type;
  int lanes_per_gate;  // of the 32 lanes a column has: power of two, 32 / it >= gate rows or 1
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

// Adds the slots: 32 columns a block, 32 lanes (warps) a column.
__global__ void __launch_bounds__(1024) bsa_block_norm_sum_kernel(const SumParams p) {
  __shared__ float buf[4][32][33];
  const int lane = threadIdx.x, ty = threadIdx.y;
  const int c = blockIdx.x * 32 + lane;
  const bool in = c < p.C;
  float dw = 0.f, db = 0.f;
  if (p.has_y) {
    // lane group `bb` of the 32 / lanes_per_gate takes gate rows bb, bb + groups, ...; its
    // lanes share the slots of one
    const int per = p.lanes_per_gate, sub = ty % per, bb = ty / per, groups = 32 / per;
    const float w = in ? param_at(p.post_w, c, p.param_type, 1.f) : 0.f;
    const float b = in ? param_at(p.post_b, c, p.param_type, 0.f) : 0.f;
    for (int64_t g = bb; g < p.gate_rows; g += groups) {
      // the blocks whose rows reach into this gate row
      const int64_t lo = g * p.per_gate / p.rows_per_block;
      const int64_t hi = p.rows == 0 ? -1 : min((min((g + 1) * p.per_gate, p.rows) - 1) / p.rows_per_block, p.blocks - 1);
      float S = 0.f, T = 0.f;
      if (in)
#pragma unroll 8
        for (int64_t k = lo + sub; k <= hi; k += per) {
          const float* q = p.part + (k + g) * (1 + p.means) * p.C + c;
          S += q[0];
          if (p.means) T += q[p.C];
        }
      if (per > 1) {
        // groups * per = 32 and one pass: every lane comes here exactly once
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
  float P = 0.f, Q = 0.f;
  if (p.has_pre && in)
#pragma unroll 8
    for (int64_t k = ty; k < p.blocks; k += 32) {
      const float* q = p.part_pre + k * (1 + p.means) * p.C + c;
      P += q[0];
      if (p.means) Q += q[p.C];
    }
  buf[0][ty][lane] = dw;
  buf[1][ty][lane] = db;
  buf[2][ty][lane] = P;
  buf[3][ty][lane] = Q;
  __syncthreads();
  if (ty < 4 && in) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += buf[ty][k][lane];
    void* to[4] = {p.dpost_w, p.dpost_b, p.dpre_w, p.dpre_b};
    param_put(ty == 0 ? to[0] : ty == 1 ? to[1] : ty == 2 ? to[2] : to[3], c, p.param_type, s);
  }
}

// ------------------------------------------------------------ host
// How a row is laid over threads.  Vectors of eight where every row starts at 16 bytes.
struct Team {
  bool vec;
  int nv, threads;  // vectors (or elements) a thread, threads a team
};

Team team_of(int C, bool vec, bool backward, bool means) {
  Team t{vec, 1, 32};
  const int n = vec ? C / 8 : C;
  if (vec) {
    // a warp takes a row while a lane's share fits its registers (the backward with layer
    // norms keeps four sums a column), else the fewest vectors a thread that 512 threads allow
    const int most = backward ? (means ? 1 : 3) : 4;
    if (n <= 32 * most) {
      t.nv = (n + 31) / 32;
      return t;
    }
    t.nv = n <= 512 ? 1 : 2;
  } else {
    t.nv = n <= 4 * 512 ? 4 : 16;
  }
  t.threads = ((n + t.nv - 1) / t.nv + 31) / 32 * 32;
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

template <typename T>
void launch_norm(const NormParams& p, const Team& t, cudaStream_t s) {
  if (t.vec && t.threads == 32) {
    const unsigned grid = static_cast<unsigned>((p.rows + 3) / 4);
    if (t.nv == 1) bsa_block_norm_kernel<T, 8, 1, true><<<grid, 128, 0, s>>>(p);
    else if (t.nv == 2) bsa_block_norm_kernel<T, 8, 2, true><<<grid, 128, 0, s>>>(p);
    else if (t.nv == 3) bsa_block_norm_kernel<T, 8, 3, true><<<grid, 128, 0, s>>>(p);
    else bsa_block_norm_kernel<T, 8, 4, true><<<grid, 128, 0, s>>>(p);
    return;
  }
  const unsigned grid = static_cast<unsigned>(p.rows);
  if (t.vec && t.nv == 1) bsa_block_norm_kernel<T, 8, 1, false><<<grid, t.threads, 0, s>>>(p);
  else if (t.vec) bsa_block_norm_kernel<T, 8, 2, false><<<grid, t.threads, 0, s>>>(p);
  else if (t.nv == 4) bsa_block_norm_kernel<T, 1, 4, false><<<grid, t.threads, 0, s>>>(p);
  else bsa_block_norm_kernel<T, 1, 16, false><<<grid, t.threads, 0, s>>>(p);
}

struct BackPlan {
  int teams;  // a block
  int64_t blocks, rows_per_block, slots;
  size_t bytes;
};

// Blocks of about 256 threads, two for each of 148 SMs' places, at least one row a team.
BackPlan back_plan(const NormParams& p, const Team& t, int gate_rows, bool means) {
  BackPlan b;
  b.teams = std::max(1, 256 / t.threads);
  const int64_t want = t.threads > 256 ? 148 * 1 : 148 * 2;
  const int64_t most = std::max<int64_t>(1, (p.rows + b.teams - 1) / b.teams);
  b.blocks = std::min(want, most);
  b.rows_per_block = std::max<int64_t>(1, (p.rows + b.blocks - 1) / b.blocks);
  b.blocks = (p.rows + b.rows_per_block - 1) / b.rows_per_block;
  b.slots = b.blocks + gate_rows;
  b.bytes = static_cast<size_t>(b.slots + b.blocks) * (means ? 2 : 1) * p.C * sizeof(float);
  return b;
}

template <typename T, bool kMeans>
void launch_back(const NormParams& p, const Team& t, const BackPlan& b, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(b.blocks);
  const int threads = b.teams * t.threads;
  const size_t smem = (p.C + b.teams * 2 * (kMeans ? 2 : 1) * 32) * sizeof(float);
  if (t.vec && t.threads == 32) {
    if (t.nv == 1) bsa_block_norm_back_kernel<T, 8, 1, true, kMeans><<<grid, threads, smem, s>>>(p, 32);
    else if constexpr (!kMeans) {
      if (t.nv == 2) bsa_block_norm_back_kernel<T, 8, 2, true, kMeans><<<grid, threads, smem, s>>>(p, 32);
      else bsa_block_norm_back_kernel<T, 8, 3, true, kMeans><<<grid, threads, smem, s>>>(p, 32);
    }
    return;
  }
  if (t.vec && t.nv == 1) bsa_block_norm_back_kernel<T, 8, 1, false, kMeans><<<grid, threads, smem, s>>>(p, t.threads);
  else if (t.vec) bsa_block_norm_back_kernel<T, 8, 2, false, kMeans><<<grid, threads, smem, s>>>(p, t.threads);
  else if (t.nv == 4) bsa_block_norm_back_kernel<T, 1, 4, false, kMeans><<<grid, threads, smem, s>>>(p, t.threads);
  else bsa_block_norm_back_kernel<T, 1, 16, false, kMeans><<<grid, threads, smem, s>>>(p, t.threads);
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
  if (p.rows > 0x7fffffff || misaligned(a.type, {x, y, stream_out, normed}) ||
      (stats != nullptr && !aligned16(stats)))
    return BSA_ERR_INVALID_ARG;
  const bool vec = a.C % 8 == 0 && all_aligned({x, y, stream_out, normed, a.post_weight, a.post_bias, a.gate,
                                                a.pre_weight, a.pre_bias});
  p.x = x, p.y = y, p.out = stream_out, p.normed = normed, p.stats = stats;
  const Team t = team_of(a.C, vec, false, takes_means(a));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.type == BSA_BF16) launch_norm<__nv_bfloat16>(p, t, s);
  else if (a.type == BSA_FP16) launch_norm<__half>(p, t, s);
  else launch_norm<float>(p, t, s);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

int bsa_block_norm_backward_workspace_bytes(const bsa_block_norm_args* args, size_t* bytes) {
  const int st = check_args(args);
  if (st != BSA_OK) return st;
  if (bytes == nullptr) return BSA_ERR_INVALID_ARG;
  NormParams p{};
  fill(p, *args);
  // the larger of both layouts: which one runs depends on the alignment of the call
  size_t most = 0;
  for (const bool vec : {false, true})
    most = std::max(most, back_plan(p, team_of(args->C, vec && args->C % 8 == 0, true, keeps_means(*args)),
                                    args->gate_rows, keeps_means(*args)).bytes);
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
    if (dnormed != nullptr && a.pre == BSA_NORM_NONE) return BSA_ERR_INVALID_ARG;
    if (p.rows > 0x7fffffff || misaligned(a.type, {x, y, dstream, dnormed, dx, dy}) || !aligned16(stats))
      return BSA_ERR_INVALID_ARG;
  }
  if (misaligned(a.param_type, {dpost_weight, dpost_bias, dgate, dpre_weight, dpre_bias})) return BSA_ERR_INVALID_ARG;
  const bool means = keeps_means(a);
  const bool vec = a.C % 8 == 0 && all_aligned({x, y, dstream, dnormed, dx, dy, a.post_weight, a.gate, a.pre_weight});
  const Team t = team_of(a.C, vec, true, means);
  const BackPlan b = back_plan(p, t, a.gate_rows, means);
  if (sums && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || workspace_bytes < b.bytes))
    return BSA_ERR_WORKSPACE;
  p.x = x, p.y = y, p.dstream = dstream, p.dnormed = dnormed, p.saved = stats, p.dx = dx, p.dy = dy;
  p.part = sums ? static_cast<float*>(workspace) : nullptr;
  p.part_pre = sums ? p.part + b.slots * (means ? 2 : 1) * a.C : nullptr;
  p.rows_per_block = b.rows_per_block;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.rows > 0) {
    if (a.type == BSA_BF16) means ? launch_back<__nv_bfloat16, true>(p, t, b, s) : launch_back<__nv_bfloat16, false>(p, t, b, s);
    else if (a.type == BSA_FP16) means ? launch_back<__half, true>(p, t, b, s) : launch_back<__half, false>(p, t, b, s);
    else means ? launch_back<float, true>(p, t, b, s) : launch_back<float, false>(p, t, b, s);
  }
  if (sums) {
    SumParams q{};
    q.part = p.part, q.part_pre = p.part_pre;
    q.post_w = a.post_weight, q.post_b = a.post_bias, q.gate = a.gate;
    q.dpost_w = dpost_weight, q.dpost_b = dpost_bias, q.dgate = dgate, q.dpre_w = dpre_weight, q.dpre_b = dpre_bias;
    q.rows = p.rows, q.per_gate = p.per_gate, q.rows_per_block = b.rows_per_block, q.blocks = b.blocks;
    q.C = a.C, q.gate_rows = a.gate_rows, q.means = means;
    q.has_y = p.rows == 0 || y != nullptr;
    q.has_pre = dnormed != nullptr;
    q.param_type = a.param_type, q.alpha = a.branch_scale;
    int lanes = 1;
    while (lanes < 32 && 32 / (2 * lanes) >= a.gate_rows) lanes *= 2;
    q.lanes_per_gate = lanes;
    bsa_block_norm_sum_kernel<<<(a.C + 31) / 32, dim3(32, 32), 0, s>>>(q);
  }
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // extern "C"
