// Row elements of the training operators: bf16, f16 or f32 values moved in vectors of kBytes
// (16 where every row starts on a 16-byte boundary, else 8, 4 or 2) and computed on in fp32.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace moe {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) {
  return __half2float(v);
}
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
  return v;
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}

template <int kBytes>
struct RawVec;
template <>
struct RawVec<16> {
  using type = uint4;
};
template <>
struct RawVec<8> {
  using type = uint2;
};
template <>
struct RawVec<4> {
  using type = uint32_t;
};
template <>
struct RawVec<2> {
  using type = uint16_t;
};

// kBytes of T as fp32 values and back (one rounding to nearest even each).
template <typename T, int kBytes>
struct Vec {
  static constexpr int kN = kBytes / static_cast<int>(sizeof(T));
  using Raw = typename RawVec<kBytes>::type;
  __device__ __forceinline__ static void unpack(Raw r, float (&f)[kN]) {
    const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = to_f32<T>(e[i]);
  }
  __device__ __forceinline__ static Raw pack(const float (&f)[kN]) {
    Raw r;
    T* e = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < kN; ++i) e[i] = from_f32<T>(f[i]);
    return r;
  }
};

}  // namespace moe
