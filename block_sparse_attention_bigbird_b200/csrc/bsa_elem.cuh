// Element access shared by the kernels around the attention (rotary positions, block
// norms, the 8-bit quantiser): eight neighbouring elements by 16-byte accesses, or one.
// Arithmetic is in fp32; storing rounds once, to nearest even.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include <cstdint>

#include "../../include/bsa.h"

namespace bsa {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

__device__ __forceinline__ void unpack(uint32_t w, __nv_bfloat16, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack(uint32_t w, __half, float& lo, float& hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  lo = f.x;
  hi = f.y;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack(float lo, float hi, __half) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// kVec elements as they lie in memory, in words.
template <int kVec, typename T>
struct RawElems {
  static constexpr int kWords = (kVec * static_cast<int>(sizeof(T)) + 3) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kVec == 1) {
      if constexpr (sizeof(T) == 4) w[0] = *reinterpret_cast<const uint32_t*>(p);
      else w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
      static_assert(kWords % 4 == 0, "whole 16-byte words");
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 a = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
      }
    }
  }
  __device__ __forceinline__ void widen(float (&v)[kVec]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = __uint_as_float(w[i]);
    } else if constexpr (kVec == 1) {
      float hi;
      unpack(w[0], T(), v[0], hi);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) unpack(w[i], T(), v[2 * i], v[2 * i + 1]);
    }
  }
};

// kVec consecutive elements; kVec = 8 needs a 16-byte aligned address, 2 one of two elements.
template <int kVec, typename T>
struct Elems {
  static __device__ __forceinline__ void load(const T* p, float (&v)[kVec]) {
    if constexpr (kVec == 1) {
      v[0] = to_f32(*p);
    } else if constexpr (kVec == 2 && sizeof(T) == 4) {
      const float2 a = *reinterpret_cast<const float2*>(p);
      v[0] = a.x, v[1] = a.y;
    } else if constexpr (kVec == 2) {
      unpack(*reinterpret_cast<const uint32_t*>(p), T(), v[0], v[1]);
    } else if constexpr (sizeof(T) == 4) {
      static_assert(kVec == 8, "one, two or eight elements");
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      static_assert(kVec == 8, "one, two or eight elements");
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      unpack(a.x, T(), v[0], v[1]);
      unpack(a.y, T(), v[2], v[3]);
      unpack(a.z, T(), v[4], v[5]);
      unpack(a.w, T(), v[6], v[7]);
    }
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[kVec]) {
    if constexpr (kVec == 1) {
      *p = from_f32<T>(v[0]);
    } else if constexpr (kVec == 2 && sizeof(T) == 4) {
      *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    } else if constexpr (kVec == 2) {
      *reinterpret_cast<uint32_t*>(p) = pack(v[0], v[1], T());
    } else if constexpr (sizeof(T) == 4) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack(v[0], v[1], T()), pack(v[2], v[3], T()),
                                                pack(v[4], v[5], T()), pack(v[6], v[7], T()));
    }
  }
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t type_bytes(int type) { return type == BSA_FP32 ? 4 : 2; }  // of bf16, fp16, fp32
inline bool is_float_type(int type) { return type == BSA_BF16 || type == BSA_FP16 || type == BSA_FP32; }

// SMs of the current device, or a negative bsa_status where it is no sm_100 part.  Asked
// once per device; a failed query is not kept.
inline int sm_count() {
  constexpr int kMost = 64;
  static std::atomic<int> known[kMost];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
  if (dev < 0 || dev >= kMost) return BSA_ERR_UNSUPPORTED;
  const int k = known[dev].load(std::memory_order_relaxed);
  if (k != 0) return k;
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return BSA_ERR_CUDA;
  const int got = major == 10 && minor == 0 ? sms : static_cast<int>(BSA_ERR_UNSUPPORTED);
  known[dev].store(got, std::memory_order_relaxed);
  return got;
}

}  // namespace bsa
