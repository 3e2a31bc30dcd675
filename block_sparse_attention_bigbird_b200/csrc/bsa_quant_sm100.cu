// Block quantiser to 8-bit floating point, for B200 (sm_100a): codes and one fp32 scale for
// each block of 128, for the 8-bit product.
//
//     m = max |x| over the block,  scale = m / top,  code = rn(x (top / m)),
//
// top being the format's largest finite value.  x (top / m) takes two roundings to fp32 (the
// division's, one a block, and the product's), so that a quotient within 2^-23 of a tie between two
// codes may go either way.  Of fp32 elements fewer than one in a million lie there; 16-bit ones fall on
// exact ties far more often (bf16 activations, e4m3: one code in about 4000 is not the one that ties
// to even give).  A code exact at ties was measured for fp32 (28 us against 20).  m is at least 2^-100, so that top / m stays
// finite for a block of zeros.  The maximum passes NaN on.
//
// A block of threads takes one 128 x 128 tile of x, so that rows of 128, columns of 128 and
// square blocks all lie in it and both forms come from one read.  Thread (g, c) of 16 x 16
// keeps the 8 x 8 patch of rows 8 g.., columns 8 c.. as it was loaded.  Magnitudes are
// compared as integers (the bits of |x| order as |x| does, with NaN above infinity, and two
// 16-bit elements to a word); a row's maxima meet over 16 neighbouring lanes by halving the
// rows a lane is left with, columns' in shared memory; one thread a row or column divides.
// The rows form leaves as 8-byte stores (16 lanes: one 128-byte row); the columns form goes
// through shared memory, where the patch's columns are stored as 8-byte words in the order
// word ^ c, which spreads both the writes and the 16-byte reads over all banks.
//
// What bounds it: the bytes (2 or 4 in, 1 or 2 out an element), and with two forms of 16-bit
// elements nearly as much the integer and conversion work (about 7 instructions an element and
// form; issue slots 59 % busy, DRAM 50 %).  Measured: both forms of 65536 x 768 bf16 (201 MB)
// 39 us alone, 42 in a row (4.8 TB/s, where a copy has 6.55); both square forms of 4096 x 4096
// fp32 (101 MB) 19 and 21 us.  Persistent blocks that fetch the next tile with cp.async took 43 and 29 us: the
// second copy through shared memory costs what the overlap gives.  Comparing and dividing
// element by element in fp32 took 113 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "bsa_elem.cuh"

namespace bsa {
namespace {

constexpr int kTile = 128;
constexpr float kLeastMax = 7.888609052210118e-31f;  // 2^-100

struct QuantParams {
  const void* x;
  int R, C, vec;  // vec: rows of x may be read 16 bytes at a time
  uint8_t *codes, *codes_t;
  int64_t ld, ld_t;
  float *scale, *scale_t;
  int kb, kb_t;  // blocks along a row, along a column
};

// The 8 columns of one row of a patch as loaded, W words.
template <typename T>
struct Raw {
  static constexpr int kWords = sizeof(T) == 4 ? 8 : 4;
  static constexpr uint32_t kAbs = sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p, bool vec, int n) {  // n columns are there
    if (vec && n > 0) {
#pragma unroll
      for (int h = 0; h < kWords / 4; ++h) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + h);
        w[4 * h] = a.x, w[4 * h + 1] = a.y, w[4 * h + 2] = a.z, w[4 * h + 3] = a.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kWords; ++k) w[k] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= n) continue;
        if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(to_f32(p[j]));
        else w[j >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[j]) << (16 * (j & 1));
      }
    }
  }
  __device__ __forceinline__ float at(int j) const {  // column j
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[j]);
    } else {
      float lo, hi;
      unpack(w[j >> 1], T(), lo, hi);
      return j & 1 ? hi : lo;
    }
  }
};
// maximum of words of magnitude bits: of both halves, or of the whole word
template <typename T>
__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) {
  if constexpr (sizeof(T) == 4) return max(a, b);
  else return __vmaxu2(a, b);
}
template <typename T>
__device__ __forceinline__ uint32_t both_halves(uint32_t a) {
  if constexpr (sizeof(T) == 4) return a;
  else return __vmaxu2(a, a >> 16) & 0xffffu;
}
template <typename T>
__device__ __forceinline__ float magnitude(uint32_t bits) {  // of the low half, or the word
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(bits);
  } else {
    float lo, hi;
    unpack(bits, T(), lo, hi);
    return lo;
  }
}
// the block's maximum, at least 2^-100, NaN where the block has one
__device__ __forceinline__ float at_least(float m) { return m < kLeastMax ? kLeastMax : m; }

template <bool kE5>
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t r;
  if constexpr (kE5) asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool kE5>
__device__ __forceinline__ uint2 codes8(const float (&v)[8]) {
  return make_uint2(codes2<kE5>(v[0], v[1]) | codes2<kE5>(v[2], v[3]) << 16,
                    codes2<kE5>(v[4], v[5]) | codes2<kE5>(v[6], v[7]) << 16);
}

// Blocks an SM, as many as have registers without many spills (us with one block fewer, this many, one
// more): 16-bit elements, one form of 65536 x 768 (29.1, 27.1, -), both (-, 41.4, 43.6); fp32, columns
// of 8192 x 2304 (20.8, 19.3, -), both forms of it (-, 25.1, 37.3).
template <typename T, bool kSquare, int kForm>
constexpr int kQuantBlocks = sizeof(T) == 2 ? (kForm == 2 ? 3 : 4) : kForm == 2 && !kSquare ? 2 : 3;

// kForm: 0 rows, 1 columns, 2 both
template <typename T, bool kE5, bool kSquare, int kForm>
__global__ void __launch_bounds__(256, (kQuantBlocks<T, kSquare, kForm>))
bsa_fp8_quantize_kernel(const __grid_constant__ QuantParams p) {
  constexpr float kTop = kE5 ? 57344.f : 448.f;
  constexpr bool kRows = kForm != 1, kCols = kForm != 0;
  // maxima of the warps' columns (or of the warps), and the columns' top / m
  __shared__ uint32_t tops[kSquare ? 8 : 8 * 16 * Raw<T>::kWords];
  __shared__ __align__(16) float invs[kTile];
  __shared__ __align__(16) uint8_t tr[kCols ? kTile * kTile : 16];
  const int bx = blockIdx.x % p.kb, by = blockIdx.x / p.kb;  // tile of columns, of rows
  const int tid = threadIdx.x, g = tid >> 4, c = tid & 15, warp = tid >> 5, lane = tid & 31;
  const int col0 = bx * kTile + c * 8, row0 = by * kTile + g * 8;
  using R = Raw<T>;
  R v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = row0 + i;
    v[i].load(static_cast<const T*>(p.x) + static_cast<int64_t>(r) * p.C + col0, p.vec,
              r < p.R ? p.C - col0 : 0);
  }
  uint32_t rowm[8];  // magnitude bits of each row of the patch (square: of all in rowm[0])
  if constexpr (kRows || kSquare) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = v[i].w[0] & R::kAbs;
#pragma unroll
      for (int k = 1; k < R::kWords; ++k) m = max_bits<T>(m, v[i].w[k] & R::kAbs);
      rowm[i] = m;
    }
  }
  float row_inv[8], col_inv[8];
  if constexpr (kSquare) {
    uint32_t m = rowm[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_bits<T>(m, rowm[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_bits<T>(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) tops[warp] = both_halves<T>(m);
    __syncthreads();
    m = tops[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max(m, tops[i]);
    const float top = at_least(magnitude<T>(m));
    const float inv = kTop / top;
#pragma unroll
    for (int i = 0; i < 8; ++i) row_inv[i] = col_inv[i] = inv;
    if (tid == 0) {
      if constexpr (kRows) p.scale[static_cast<int64_t>(by) * p.kb + bx] = top / kTop;
      if constexpr (kCols) p.scale_t[static_cast<int64_t>(bx) * p.kb_t + by] = top / kTop;
    }
  } else {
    if constexpr (kCols) {
      // column maxima of the patch, then over the warp's two g, then over the warps
#pragma unroll
      for (int k = 0; k < R::kWords; ++k) {
        uint32_t m = v[0].w[k] & R::kAbs;
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max_bits<T>(m, v[i].w[k] & R::kAbs);
        m = max_bits<T>(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if (lane < 16) tops[(warp * 16 + c) * R::kWords + k] = m;
      }
    }
    if constexpr (kRows) {
      // 16 lanes hold 8 rows each: half of the rows go to the lane's partner three times
      // over, until lane c keeps the maximum of row c / 2 of the patch (both lanes of a pair)
      uint32_t m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool up = c & 8;
        const uint32_t keep = up ? rowm[i + 4] : rowm[i], give = up ? rowm[i] : rowm[i + 4];
        m[i] = max_bits<T>(keep, __shfl_xor_sync(0xffffffffu, give, 8));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool up = c & 4;
        const uint32_t keep = up ? m[i + 2] : m[i], give = up ? m[i] : m[i + 2];
        m[i] = max_bits<T>(keep, __shfl_xor_sync(0xffffffffu, give, 4));
      }
      {
        const bool up = c & 2;
        const uint32_t keep = up ? m[1] : m[0], give = up ? m[0] : m[1];
        m[0] = max_bits<T>(keep, __shfl_xor_sync(0xffffffffu, give, 2));
      }
      m[0] = max_bits<T>(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
      const float top = at_least(magnitude<T>(both_halves<T>(m[0])));
      const float inv = kTop / top;
      const int r = row0 + (c >> 1);
      if ((c & 1) == 0 && r < p.R) p.scale[static_cast<int64_t>(r) * p.kb + bx] = top / kTop;
#pragma unroll
      for (int i = 0; i < 8; ++i) row_inv[i] = __shfl_sync(0xffffffffu, inv, (lane & 16) + 2 * i);
    }
    if constexpr (kCols) {
      __syncthreads();
      if (tid < kTile) {
        // column tid of the tile: its word, and its half of a word of two
        const int word = sizeof(T) == 4 ? tid : tid >> 1;
        uint32_t m = tops[word];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = max_bits<T>(m, tops[w * 16 * R::kWords + word]);
        if (sizeof(T) == 2) m = tid & 1 ? m >> 16 : m & 0xffffu;
        const float top = at_least(magnitude<T>(m));
        invs[tid] = kTop / top;
        if (bx * kTile + tid < p.C) p.scale_t[static_cast<int64_t>(bx * kTile + tid) * p.kb_t + by] = top / kTop;
      }
      __syncthreads();
      const float4 lo = *reinterpret_cast<const float4*>(invs + c * 8);
      const float4 hi = *reinterpret_cast<const float4*>(invs + c * 8 + 4);
      col_inv[0] = lo.x, col_inv[1] = lo.y, col_inv[2] = lo.z, col_inv[3] = lo.w;
      col_inv[4] = hi.x, col_inv[5] = hi.y, col_inv[6] = hi.z, col_inv[7] = hi.w;
    }
  }
  if constexpr (kRows) {
    const int end = (p.C + 15) / 16 * 16;  // the last 16 bytes of a row are written whole
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = v[i].at(j) * row_inv[i];
      const uint2 w = codes8<kE5>(s);
      if (row0 + i < p.R && col0 < end)
        *reinterpret_cast<uint2*>(p.codes + static_cast<int64_t>(row0 + i) * p.ld + col0) = w;
    }
  }
  if constexpr (kCols) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float s[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = v[i].at(j) * col_inv[j];
      *reinterpret_cast<uint2*>(tr + (c * 8 + j) * kTile + ((g ^ c) << 3)) = codes8<kE5>(s);
    }
    __syncthreads();
    const int end = (p.R + 15) / 16 * 16;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = k * 32 + (tid >> 3), m = tid & 7;  // column of the tile, 16-byte word of it
      const int swap = (n >> 3) & 1, at = ((2 * m) ^ (n >> 3)) & ~1;
      const uint4 w = *reinterpret_cast<const uint4*>(tr + n * kTile + (at << 3));
      const int r = by * kTile + m * 16, cc = bx * kTile + n;
      if (cc < p.C && r < end)
        *reinterpret_cast<uint4*>(p.codes_t + static_cast<int64_t>(cc) * p.ld_t + r) =
            swap ? make_uint4(w.z, w.w, w.x, w.y) : w;
    }
  }
}

template <typename T, bool kE5, bool kSquare>
void launch_quant(const QuantParams& p, dim3 grid, cudaStream_t s) {
  if (p.codes_t == nullptr) bsa_fp8_quantize_kernel<T, kE5, kSquare, 0><<<grid, 256, 0, s>>>(p);
  else if (p.codes == nullptr) bsa_fp8_quantize_kernel<T, kE5, kSquare, 1><<<grid, 256, 0, s>>>(p);
  else bsa_fp8_quantize_kernel<T, kE5, kSquare, 2><<<grid, 256, 0, s>>>(p);
}
template <typename T>
void launch_quant(const QuantParams& p, bool e5, bool square, dim3 grid, cudaStream_t s) {
  if (e5) square ? launch_quant<T, true, true>(p, grid, s) : launch_quant<T, true, false>(p, grid, s);
  else square ? launch_quant<T, false, true>(p, grid, s) : launch_quant<T, false, false>(p, grid, s);
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" int bsa_fp8_quantize(const void* x, int type, int R, int C, int square, int code_type, void* codes,
                                int64_t ld, float* scale, void* codes_t, int64_t ld_t, float* scale_t, void* stream) {
  if (R < 0 || C < 0) return BSA_ERR_INVALID_ARG;
  if (!is_float_type(type) || (code_type != BSA_E4M3 && code_type != BSA_E5M2)) return BSA_ERR_UNSUPPORTED;
  if (R == 0 || C == 0) return BSA_OK;
  if (x == nullptr || (codes == nullptr && codes_t == nullptr) || (codes != nullptr && scale == nullptr) ||
      (codes_t != nullptr && scale_t == nullptr))
    return BSA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(x) % type_bytes(type) != 0 ||
      (codes != nullptr && reinterpret_cast<uintptr_t>(scale) % 4 != 0) ||
      (codes_t != nullptr && reinterpret_cast<uintptr_t>(scale_t) % 4 != 0))
    return BSA_ERR_INVALID_ARG;
  const int64_t r16 = (static_cast<int64_t>(R) + 15) / 16 * 16, c16 = (static_cast<int64_t>(C) + 15) / 16 * 16;
  if (codes != nullptr && (!aligned16(codes) || ld % 16 != 0 || ld < c16)) return BSA_ERR_INVALID_ARG;
  if (codes_t != nullptr && (!aligned16(codes_t) || ld_t % 16 != 0 || ld_t < r16)) return BSA_ERR_INVALID_ARG;
  const int64_t nc = (static_cast<int64_t>(C) + kTile - 1) / kTile, nr = (static_cast<int64_t>(R) + kTile - 1) / kTile;
  if (R > (1 << 30) || C > (1 << 30) || nc * nr > 0x7fffffff) return BSA_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms < 0) return sms;
  QuantParams p{};
  p.x = x, p.R = R, p.C = C;
  p.vec = C % 8 == 0 && aligned16(x);
  p.codes = static_cast<uint8_t*>(codes), p.codes_t = static_cast<uint8_t*>(codes_t);
  p.ld = ld, p.ld_t = ld_t, p.scale = scale, p.scale_t = scale_t;
  p.kb = static_cast<int>(nc), p.kb_t = static_cast<int>(nr);
  const dim3 grid(static_cast<unsigned>(nc * nr));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e5 = code_type == BSA_E5M2;
  if (type == BSA_BF16) launch_quant<__nv_bfloat16>(p, e5, square != 0, grid, s);
  else if (type == BSA_FP16) launch_quant<__half>(p, e5, square != 0, grid, s);
  else launch_quant<float>(p, e5, square != 0, grid, s);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}
