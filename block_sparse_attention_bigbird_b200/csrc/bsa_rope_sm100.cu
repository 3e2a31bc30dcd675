// Rotary positions with several axes, for B200 (sm_100a).
//
// Pair j of a head, (u, v), is turned by t = p[axis_j] * freq_j, p being the token's
// position on the pair's axis (time, height, width).  The gradient is the turn by -t, so
// one kernel serves both directions.
//
// Mathematics.  t is needed modulo 2 pi with an absolute error far below fp32's 2^-24 while
// p * freq may be a million radians, so the product is formed in fp64 in units of whole
// turns (freq / 2 pi from the host), its integer part removed, and the remaining fraction
// in [-1/2, 1/2] taken to fp32 for sincospif.
//
// What bounds it: q and k are read and written once; the arithmetic is 3 operations an
// element.  The sines are the costly part (about 60 instructions a pair), so a thread keeps
// the angles of eight pairs of one token and walks over heads with them.  It reads the
// pairs' two halves as two 16-byte vectors.  The heads are cut into equal groups (blockIdx.y),
// of at most twelve unless the tokens alone fill the card several times (kRopeFill), so that
// the last wave is short; with one token a call a thread takes one head.
//
// Measured: B = 4, L = 16384, 12 + 12 heads of 64 in bf16 (403 MB read and written) 66 us
// alone, 70 in a row (5.8 TB/s, where a copy has 6.55); 80 registers, six blocks an SM.  Six
// blocks of batches of 4 heads took 70.0 us; 5 of 4, 7 of 4 and 8 of 3 (which hold fewer loads
// or spill) 72.3, 74.2 and 73.4.  8 tokens of 16 + 4 heads of 128: 16 us with the call from
// Python, whose host side is all but a few of them.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "bsa_elem.cuh"
#include "sm100_ptx.cuh"

struct bsa_rope {
  std::vector<int32_t> axis;
  std::vector<double> freq;
  int n_axes = 0, adjacent = 0;
};

namespace bsa {
namespace {

constexpr int kMaxPairs = 128;
constexpr int kMaxAxes = 8;
constexpr int kRopeThreads = 128;
// Heads a thread has on their way at once: their raw words take 32 registers.
template <typename T, int kVec>
constexpr int kBatchOf = kVec == 1 ? 4 : sizeof(T) == 2 ? 4 : 2;

struct RopeParams {
  double turns[kMaxPairs];  // frequency in turns per position
  uint8_t axis[kMaxPairs];
  const void* in[2];  // q, k
  void* out[2];
  int64_t is[2][3], os[2][3];  // element strides (b, h, l)
  int heads[2];
  const void* pos;
  int64_t ps[3];
  int pos_type;
  int B, L, d, pairs;
  int units;         // units of work of a token: kVec pairs each, then the copied tail
  int pair_units;
  int group;         // heads per blockIdx.y
  float sign;
};

__device__ __forceinline__ double position(const RopeParams& p, int axis, int b, int l) {
  const int64_t i = axis * p.ps[0] + b * p.ps[1] + l * p.ps[2];
  if (p.pos_type == BSA_INT64) return static_cast<double>(static_cast<const int64_t*>(p.pos)[i]);
  if (p.pos_type == BSA_INT32) return static_cast<double>(static_cast<const int32_t*>(p.pos)[i]);
  return static_cast<double>(static_cast<const float*>(p.pos)[i]);
}

template <typename T, int kVec, bool kAdj>
__global__ void __launch_bounds__(kRopeThreads, 6) bsa_rope_kernel(const __grid_constant__ RopeParams p) {
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int64_t tok = idx / p.units;
  const int unit = static_cast<int>(idx - tok * p.units);
  if (tok >= static_cast<int64_t>(p.B) * p.L) return;
  const int b = static_cast<int>(tok / p.L), l = static_cast<int>(tok - static_cast<int64_t>(b) * p.L);
  const int h0 = blockIdx.y * p.group, h1 = min(h0 + p.group, p.heads[0] + p.heads[1]);

  // columns of this unit's two vectors; a tail unit may have one
  int c0, c1;
  bool turn = unit < p.pair_units, second = true;
  if (turn) {
    c0 = kAdj ? unit * 2 * kVec : unit * kVec;
    c1 = kAdj ? c0 + kVec : c0 + p.pairs;
  } else {
    c0 = 2 * p.pairs + (unit - p.pair_units) * 2 * kVec;
    c1 = c0 + kVec;
    second = c1 < p.d;
  }
  float cs[kVec], sn[kVec];
  if (turn) {
    int last = -1;
    double at = 0.0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int j = unit * kVec + i;
      if (p.axis[j] != last) {
        last = p.axis[j];
        at = position(p, last, b, l);
      }
      double x = at * p.turns[j];
      x -= rint(x);
      sincospif(2.0f * static_cast<float>(x), &sn[i], &cs[i]);
      sn[i] *= p.sign;
    }
  }
  constexpr int kBatch = kBatchOf<T, kVec>;
  // kBatch heads' loads are issued before the first store, which the compiler could not move
  // them over (the results may lie where the inputs are)
  for (int first = h0; first < h1; first += kBatch) {
    RawElems<kVec, T> ru[kBatch], rv[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = first + i;
      if (h >= h1) break;
      const int w = h >= p.heads[0], hh = w ? h - p.heads[0] : h;
      const T* in = static_cast<const T*>(p.in[w]) + b * p.is[w][0] + hh * p.is[w][1] + l * p.is[w][2];
      ru[i].load(in + c0);
      if (second) rv[i].load(in + c1);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = first + i;
      if (h >= h1) break;
      const int w = h >= p.heads[0], hh = w ? h - p.heads[0] : h;
      T* out = static_cast<T*>(p.out[w]) + b * p.os[w][0] + hh * p.os[w][1] + l * p.os[w][2];
      float u[kVec], v[kVec];
      ru[i].widen(u);
      rv[i].widen(v);
      if (turn && !kAdj && kVec > 1) {
#pragma unroll
        for (int e = 0; e + 1 < kVec; e += 2) {  // two pairs at a time
          const uint64_t x = ptx::pack2(u[e], u[e + 1]), y = ptx::pack2(v[e], v[e + 1]);
          const uint64_t c2 = ptx::pack2(cs[e], cs[e + 1]), s2 = ptx::pack2(sn[e], sn[e + 1]);
          const uint64_t n2 = ptx::pack2(-sn[e], -sn[e + 1]);
          ptx::unpack2(ptx::ffma2(y, n2, ptx::fmul2(x, c2)), u[e], u[e + 1]);
          ptx::unpack2(ptx::ffma2(y, c2, ptx::fmul2(x, s2)), v[e], v[e + 1]);
        }
      } else if (turn) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          // kAdj: the 2 kVec columns hold kVec pairs side by side
          float& x = !kAdj ? u[e] : 2 * e < kVec ? u[(2 * e) % kVec] : v[(2 * e) % kVec];
          float& y = !kAdj ? v[e] : 2 * e + 1 < kVec ? u[(2 * e + 1) % kVec] : v[(2 * e + 1) % kVec];
          const float a = x * cs[e] - y * sn[e];
          y = x * sn[e] + y * cs[e];
          x = a;
        }
      }
      Elems<kVec, T>::store(out + c0, u);
      if (second) Elems<kVec, T>::store(out + c1, v);
    }
  }
}

template <typename T>
void launch_rope(const RopeParams& p, bool vec, bool adj, dim3 grid, cudaStream_t s) {
  if (vec) {
    if (adj) bsa_rope_kernel<T, 8, true><<<grid, kRopeThreads, 0, s>>>(p);
    else bsa_rope_kernel<T, 8, false><<<grid, kRopeThreads, 0, s>>>(p);
  } else {
    if (adj) bsa_rope_kernel<T, 1, true><<<grid, kRopeThreads, 0, s>>>(p);
    else bsa_rope_kernel<T, 1, false><<<grid, kRopeThreads, 0, s>>>(p);
  }
}

// Threads that fill an SM.  Where a call's fill the card less than once, its heads are cut into as
// many groups as fill it once; else into equal groups of at most twelve, but not into more than
// fill it eight times (B = 4, L = 16384, 12 + 12 heads of 64: groups of 24, 12, 8, 6 and 4 took
// 76, 73, 74, 80 and 82 us).
constexpr int64_t kRopeFill = 2048;
constexpr int64_t kRopeGroup = 12;
constexpr int64_t kGridRows = 65535;  // the most blocks along y

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" {

int bsa_rope_build(const int32_t* sections, int n_axes, double base, int per_axis, int interleave, int adjacent,
                   bsa_rope** out) {
  if (out == nullptr) return BSA_ERR_INVALID_ARG;
  *out = nullptr;
  if (sections == nullptr || n_axes < 1 || n_axes > kMaxAxes || !(base > 0.0) || !std::isfinite(base))
    return BSA_ERR_INVALID_ARG;
  int64_t n = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (sections[a] < 0) return BSA_ERR_INVALID_ARG;
    n += sections[a];
  }
  if (n < 1 || n > kMaxPairs) return BSA_ERR_INVALID_ARG;
  int32_t axis[kMaxPairs], used[kMaxAxes] = {};
  double freq[kMaxPairs];
  int a = 0;
  for (int j = 0; j < n; ++j) {
    if (interleave) {
      if (j > 0) a = (a + 1) % n_axes;
      while (used[a] == sections[a]) a = (a + 1) % n_axes;
    } else {
      while (used[a] == sections[a]) ++a;
    }
    axis[j] = a;
    const double e = per_axis ? static_cast<double>(used[a]) / sections[a] : static_cast<double>(j) / n;
    freq[j] = std::pow(base, -e);
    if (!std::isfinite(freq[j])) return BSA_ERR_INVALID_ARG;
    ++used[a];
  }
  return bsa_rope_from_table(axis, freq, static_cast<int>(n), adjacent, out);
}

int bsa_rope_from_table(const int32_t* axis, const double* freq, int n_pairs, int adjacent, bsa_rope** out) {
  if (out == nullptr) return BSA_ERR_INVALID_ARG;
  *out = nullptr;
  if (axis == nullptr || freq == nullptr || n_pairs < 1 || n_pairs > kMaxPairs) return BSA_ERR_INVALID_ARG;
  int top = 0;
  for (int j = 0; j < n_pairs; ++j) {
    if (axis[j] < 0 || axis[j] >= kMaxAxes || !std::isfinite(freq[j])) return BSA_ERR_INVALID_ARG;
    top = std::max(top, static_cast<int>(axis[j]));
  }
  bsa_rope* r = new (std::nothrow) bsa_rope();
  if (r == nullptr) return BSA_ERR_OOM;
  try {
    r->axis.assign(axis, axis + n_pairs);
    r->freq.assign(freq, freq + n_pairs);
  } catch (...) {
    delete r;
    return BSA_ERR_OOM;
  }
  r->n_axes = top + 1;
  r->adjacent = adjacent != 0;
  *out = r;
  return BSA_OK;
}

int bsa_rope_table(const bsa_rope* rope, const int32_t** axis, const double** freq, int* n_pairs, int* n_axes,
                   int* adjacent) {
  if (rope == nullptr) return BSA_ERR_INVALID_ARG;
  if (axis != nullptr) *axis = rope->axis.data();
  if (freq != nullptr) *freq = rope->freq.data();
  if (n_pairs != nullptr) *n_pairs = static_cast<int>(rope->axis.size());
  if (n_axes != nullptr) *n_axes = rope->n_axes;
  if (adjacent != nullptr) *adjacent = rope->adjacent;
  return BSA_OK;
}

void bsa_rope_free(bsa_rope* rope) { delete rope; }

int bsa_rope_apply(const void* q, void* q_out, int H, const void* k, void* k_out, int Hk, int B, int L, int d,
                   int type, const int64_t* strides, const void* positions, int position_type,
                   const int64_t* p_strides, const bsa_rope* rope, int inverse, void* stream) {
  if (rope == nullptr || strides == nullptr || p_strides == nullptr) return BSA_ERR_INVALID_ARG;
  if (B < 0 || L < 0 || H < 0 || Hk < 0 || d < 1) return BSA_ERR_INVALID_ARG;
  if (!is_float_type(type) || d > 256) return BSA_ERR_UNSUPPORTED;
  if (position_type != BSA_INT32 && position_type != BSA_INT64 && position_type != BSA_FP32)
    return BSA_ERR_UNSUPPORTED;
  const int pairs = static_cast<int>(rope->axis.size());
  if (2 * pairs > d) return BSA_ERR_INVALID_ARG;
  if (k == nullptr) Hk = 0;
  if (B == 0 || L == 0 || H + static_cast<int64_t>(Hk) == 0) return BSA_OK;
  if ((H > 0 && (q == nullptr || q_out == nullptr)) || (Hk > 0 && k_out == nullptr) || positions == nullptr)
    return BSA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(positions) % (position_type == BSA_INT64 ? 8 : 4) != 0) return BSA_ERR_INVALID_ARG;
  // one result may not be the other's, nor the other's input
  if (H > 0 && Hk > 0 && (q_out == k_out || q_out == k || k_out == q)) return BSA_ERR_INVALID_ARG;
  RopeParams p;
  const size_t es = type_bytes(type);
  bool vec = d % 8 == 0 && pairs % 8 == 0;
  bool in_place = true;
  p.in[0] = q, p.in[1] = k, p.out[0] = q_out, p.out[1] = k_out;
  p.heads[0] = H, p.heads[1] = Hk;
  for (int w = 0; w < 2; ++w) {
    for (int i = 0; i < 3; ++i) {
      p.is[w][i] = strides[6 * w + i];
      p.os[w][i] = strides[6 * w + 3 + i];
    }
    if (p.heads[w] == 0) continue;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.in[w]) | reinterpret_cast<uintptr_t>(p.out[w]);
    if (bits % es != 0) return BSA_ERR_INVALID_ARG;
    // a stride counts only where there is a second element along it
    const int n[3] = {B, p.heads[w], L};
    int64_t any = 0;
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1) {
        any |= (p.is[w][i] | p.os[w][i]) * static_cast<int64_t>(es);
        in_place = in_place && p.is[w][i] == p.os[w][i];
      }
    vec = vec && (bits % 16 == 0) && (any % 16 == 0);
    in_place = in_place && p.in[w] == p.out[w];
  }
  const int sms = sm_count();
  if (sms < 0) return sms;
  for (int j = 0; j < pairs; ++j) {
    p.turns[j] = rope->freq[j] / 6.283185307179586476925286766559;
    p.axis[j] = static_cast<uint8_t>(rope->axis[j]);
  }
  p.pos = positions;
  p.pos_type = position_type;
  for (int i = 0; i < 3; ++i) p.ps[i] = p_strides[i];
  p.B = B, p.L = L, p.d = d, p.pairs = pairs;
  const int v = vec ? 8 : 1;
  p.pair_units = pairs / v;
  p.units = p.pair_units + (in_place ? 0 : (d - 2 * pairs + 2 * v - 1) / (2 * v));
  p.sign = inverse ? -1.f : 1.f;
  const int64_t threads = static_cast<int64_t>(B) * L * p.units;
  const int64_t blocks = (threads + kRopeThreads - 1) / kRopeThreads;
  const int64_t heads = H + static_cast<int64_t>(Hk);
  if (blocks > 0x7fffffff || heads > (1 << 30)) return BSA_ERR_INVALID_ARG;
  const int64_t fill = sms * kRopeFill;
  const int64_t once = fill / threads, often = std::min(8 * fill / threads, (heads + kRopeGroup - 1) / kRopeGroup);
  // one group a row of the grid
  const int64_t groups = std::min<int64_t>({heads, kGridRows, std::max<int64_t>({1, once, often})});
  p.group = static_cast<int>((heads + groups - 1) / groups);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + p.group - 1) / p.group));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool adj = rope->adjacent != 0;
  if (type == BSA_BF16) launch_rope<__nv_bfloat16>(p, vec, adj, grid, s);
  else if (type == BSA_FP16) launch_rope<__half>(p, vec, adj, grid, s);
  else launch_rope<float>(p, vec, adj, grid, s);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // extern "C"
