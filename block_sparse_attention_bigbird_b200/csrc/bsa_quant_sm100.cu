// Block quantiser to 8-bit floating point, for B200 (sm_100a): codes and one fp32 scale for
// each block of 128, for the 8-bit product.
//
//     m = max |x| over the block,  scale = m / top,  code = rn(x (top / m)),
//
// top being the format's largest finite value.  m is at least 2^-100, so that top / m stays
// finite for a block of zeros.  The maximum passes NaN on.
//
// A block of threads takes one 128 x 128 tile of x, so that rows of 128, columns of 128 and
// square blocks all lie in it and both forms come from one read.  Thread (g, c) of 16 x 16
// keeps the 8 x 8 patch of rows 8 g.., columns 8 c..: row maxima meet over 16 neighbouring
// lanes, column maxima over the 16 g in shared memory.  The rows form leaves as 8-byte
// stores (16 lanes: one 128-byte row); the columns form goes through shared memory, where
// the patch's columns are stored as 8-byte words in the order word ^ c, which spreads both
// the writes and the 16-byte reads over all banks.
//
// What bounds it: the bytes (2 or 4 in, 1 or 2 out an element).
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

// maximum that passes NaN on
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

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

// kForm: 0 rows, 1 columns, 2 both
template <typename T, bool kE5, bool kSquare, int kForm>
__global__ void __launch_bounds__(256) bsa_fp8_quantize_kernel(const __grid_constant__ QuantParams p) {
  constexpr float kTop = kE5 ? 57344.f : 448.f;
  constexpr bool kRows = kForm != 1, kCols = kForm != 0;
  __shared__ float tops[8][kTile];
  __shared__ __align__(16) uint8_t tr[kCols ? kTile * kTile : 16];
  const int bx = blockIdx.x % p.kb, by = blockIdx.x / p.kb;  // tile of columns, of rows
  const int tid = threadIdx.x, g = tid >> 4, c = tid & 15, warp = tid >> 5, lane = tid & 31;
  const int col0 = bx * kTile + c * 8, row0 = by * kTile + g * 8;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = row0 + i;
    const T* src = static_cast<const T*>(p.x) + static_cast<int64_t>(r) * p.C + col0;
    if (p.vec && r < p.R && col0 < p.C) {
      Elems<8, T>::load(src, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = r < p.R && col0 + j < p.C ? to_f32(src[j]) : 0.f;
    }
  }
  float row_inv[8], col_inv[8];
  if constexpr (kSquare) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[i][j]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) tops[warp][0] = m;
    __syncthreads();
    m = kLeastMax;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_nan(m, tops[i][0]);
    const float inv = kTop / m;
#pragma unroll
    for (int i = 0; i < 8; ++i) row_inv[i] = col_inv[i] = inv;
    if (tid == 0) {
      if constexpr (kRows) p.scale[static_cast<int64_t>(by) * p.kb + bx] = m / kTop;
      if constexpr (kCols) p.scale_t[static_cast<int64_t>(bx) * p.kb_t + by] = m / kTop;
    }
  } else {
    if constexpr (kRows) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float m = kLeastMax;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[i][j]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        row_inv[i] = kTop / m;
        if (c == i && row0 + i < p.R) p.scale[static_cast<int64_t>(row0 + i) * p.kb + bx] = m / kTop;
      }
    }
    if constexpr (kCols) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float m = kLeastMax;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(v[i][j]));
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if (lane < 16) tops[warp][c * 8 + j] = m;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float m = tops[0][c * 8 + j];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = max_nan(m, tops[w][c * 8 + j]);
        col_inv[j] = kTop / m;
        if (g == j && col0 + j < p.C) p.scale_t[static_cast<int64_t>(col0 + j) * p.kb_t + by] = m / kTop;
      }
    }
  }
  if constexpr (kRows) {
    const int end = (p.C + 15) / 16 * 16;  // the last 16 bytes of a row are written whole
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = v[i][j] * row_inv[i];
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
      for (int i = 0; i < 8; ++i) s[i] = v[i][j] * col_inv[j];
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
  if (reinterpret_cast<uintptr_t>(x) % type_bytes(type) != 0) return BSA_ERR_INVALID_ARG;
  const int64_t r16 = (static_cast<int64_t>(R) + 15) / 16 * 16, c16 = (static_cast<int64_t>(C) + 15) / 16 * 16;
  if (codes != nullptr && (!aligned16(codes) || ld % 16 != 0 || ld < c16)) return BSA_ERR_INVALID_ARG;
  if (codes_t != nullptr && (!aligned16(codes_t) || ld_t % 16 != 0 || ld_t < r16)) return BSA_ERR_INVALID_ARG;
  const int64_t nc = (static_cast<int64_t>(C) + kTile - 1) / kTile, nr = (static_cast<int64_t>(R) + kTile - 1) / kTile;
  if (R > (1 << 30) || C > (1 << 30) || nc * nr > 0x7fffffff) return BSA_ERR_INVALID_ARG;
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
