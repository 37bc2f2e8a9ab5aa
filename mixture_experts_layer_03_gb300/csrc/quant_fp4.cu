// Rows to and from microscaled 4-bit floating point, and SwiGLU whose result is held so.
//
//   quantise    v = x [R, K]
//   SwiGLU      v = g sigma(g) u of gu [R, 2K], gate then up; never rounded to 16 bits
//   mx          byte = e + 127, e the least integer >= -127 with amax <= 6 * 2^e
//   nv          byte = e4m3(amax / (6 g)), to nearest even, 448 at most; a block that rounds to 0 is zeros
//   code        e2m1(v / (scale [g])), to nearest even
// A block that holds an infinity or a NaN gets the scale NaN and codes 0.
//
// What is rounded is decided as on exact numbers. In f32 the quotients (mx: exact; nv: a few units)
// and SwiGLU (kNear covers its error) are off by little, so a decision can differ from the exact one
// only where a value lies that near to the border between two codes or two scale bytes: there, a few
// times in a million values, the segment is worked out again in 64 bits.
//
// Every value is read and written once; bound by memory: 4.56 bits out for 16 in, or for 32.
#include <cstdint>

#include <cuda_fp8.h>

#include "fp4.cuh"
#include "launch.cuh"
#include "segments.cuh"

namespace moe {
namespace {

// Relative width around a value in which its f32 form may be: x / unit takes two roundings and the
// unit one (under 2^-22); SwiGLU's sigma 3 units, its products two more (under 2^-21, then the
// quotient's).
constexpr float kNearQuotient = 0x1p-21f;
constexpr float kNearSwiglu = 0x1p-20f;

struct Fp4Out {
  uint8_t* codes;       // [R, K / 2]
  uint8_t* scales;      // [R, pitch]
  const float* g;       // nv: g of each plane of rows_per_plane rows, or NULL (1)
  int64_t rows_per_plane;
};

template <int kLanes>
__device__ __forceinline__ float lanes_max(float v) {
  // Magnitudes order as their bit patterns do, infinities and NaNs on top.
  uint32_t m = __float_as_uint(v);
#pragma unroll
  for (int d = 1; d < kLanes; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return __uint_as_float(m);
}

// The least e >= -127 with amax <= 6 * 2^e = 1.5 * 2^(e + 2), as a byte; finite amax.
__device__ __forceinline__ uint32_t mx_byte(float amax) {
  const int e = static_cast<int>((__float_as_uint(amax) + 0x003fffffu) >> 23) - 2;
  return static_cast<uint32_t>(e > 0 ? e : 0);
}
__device__ __forceinline__ float mx_scale(uint32_t byte) {   // 2^(byte - 127)
  return byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}
__device__ __forceinline__ uint32_t nv_byte(float r) {
  return __nv_cvt_float_to_fp8(r, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float nv_scale(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
  return __half2float(__half(h));
}

// The same decisions on 8 values in 64 bits: the block's byte and the codes.
template <bool kNv>
__device__ __noinline__ uint32_t fp4_exact(const double (&v)[8], float g, uint32_t* byte_out) {
  double top = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmax(top, fabs(v[i]));
#pragma unroll
  for (int d = 1; d < (kNv ? 2 : 4); d *= 2) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, d));
  double unit;
  if (kNv) {
    // e4m3: multiples of 2^(e - 3) from 2^e to 2^(e + 1), of 2^-9 below 2^-6.
    const double r = fmin(top / (6.0 * static_cast<double>(g)), 448.0);
    const int e = r < 0x1p-6 ? -6 : ilogb(r);
    const double m = rint(ldexp(r, 3 - e));     // 0..16; even on a tie
    *byte_out = r < 0x1p-6 ? static_cast<uint32_t>(m)
                           : static_cast<uint32_t>((e + 7) * 8 + static_cast<int>(m) - 8);
    unit = ldexp(m, e - 3) * static_cast<double>(g);
  } else {
    int e = -127;
    if (top > 0x6p-127) {
      e = ilogb(top) - 2;                       // top < 2^(e + 3), top >= 4 * 2^e
      if (top > ldexp(6.0, e)) ++e;
    }
    *byte_out = static_cast<uint32_t>(e + 127);
    unit = ldexp(1.0, e);
  }
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double a = fabs(v[i]);
    uint32_t c = 0;
    if (unit > 0.0)
      c = (a > 0.25 * unit) + (a >= 0.75 * unit) + (a > 1.25 * unit) + (a >= 1.75 * unit) +
          (a > 2.5 * unit) + (a >= 3.5 * unit) + (a > 5.0 * unit);
    codes |= (c | (signbit(v[i]) ? 8u : 0u)) << (4 * i);
  }
  return codes;
}

__device__ __forceinline__ double swiglu_d(float g, float u) {
  const double gd = g;
  return gd / (1.0 + exp(-gd)) * static_cast<double>(u);
}

template <typename T, bool kNv, bool kSwiglu>
__global__ void __launch_bounds__(kSegmentThreads)
quantize_fp4_kernel(const T* __restrict__ x, int64_t R, int K, Fp4Out out) {
  pdl_trigger();
  pdl_wait();
  constexpr int kLanes = kNv ? 2 : 4;           // to a block
  constexpr float kNear = kSwiglu ? kNearSwiglu : kNearQuotient;
  const int lane = threadIdx.x & 31;
  const int pitch = fp4_scale_pitch(K, kNv ? kFp4Nv : kFp4Mx);
  // Segments of 256 channels, over the whole row of scales.
  for (SegmentWalk w(kNv ? pitch / 16 : pitch / 8); w.row < R; w.next()) {
    const int c = w.seg * 256 + lane * kPerLane;
    const bool in = c < K;                      // (K % 32 == 0: the same in all lanes of a block)
    float v[kPerLane] = {}, u[kPerLane] = {};
    if (in) {
      const T* src = x + w.row * (kSwiglu ? 2 : 1) * K + c;
      load8(src, v);
      if (kSwiglu) load8(src + K, u);
    }
    float g = 1.0f;
    if (kNv && out.g)
      g = __ldg(out.g + (out.rows_per_plane < R ? w.row / out.rows_per_plane : 0));
    float h[kPerLane], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      // (f32's form of sigma whatever T is: see kNear.)
      h[i] = kSwiglu ? v[i] * sigmoid_of<float>(v[i]).x * u[i] : v[i];
      amax = __uint_as_float(max(__float_as_uint(amax), __float_as_uint(h[i]) & 0x7fffffffu));
    }
    amax = lanes_max<kLanes>(amax);
    const bool finite = __float_as_uint(amax) < 0x7f800000u;
    uint32_t byte, codes;
    bool near;
    float inv;
    if (kNv) {
      const float r = __fdiv_rn(amax, 6.0f * g);
      byte = nv_byte(r);
      near = nv_byte(r * (1.0f - kNear)) != nv_byte(r * (1.0f + kNear));
      const float unit = nv_scale(byte) * g;
      inv = byte == 0 ? 0.0f : __fdiv_rn(1.0f, unit);
      // Out of f32's normal range, as with a g that is far off: in 64 bits too.
      near |= byte != 0 && !(unit > 0x1p-100f && unit < 0x1p100f);
    } else {
      byte = mx_byte(amax);
      near = kSwiglu && (mx_byte(amax * (1.0f - kNear)) != mx_byte(amax * (1.0f + kNear)));
      // 2^-(byte - 127): finite values give bytes up to 253.
      inv = __uint_as_float((254u - (byte < 254u ? byte : 253u)) << 23);
    }
    float z[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) z[i] = h[i] * inv;
    codes = fp4_codes8(z);
    if (kNv || kSwiglu) {
      float lo[kPerLane], hi[kPerLane];
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) {
        lo[i] = z[i] * (1.0f - kNear);
        hi[i] = z[i] * (1.0f + kNear);
      }
      near |= fp4_codes8(lo) != fp4_codes8(hi);
      if (__any_sync(0xffffffffu, near && finite)) {
        double d[kPerLane];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
          d[i] = kSwiglu ? (in ? swiglu_d(v[i], u[i]) : 0.0) : static_cast<double>(v[i]);
        codes = fp4_exact<kNv>(d, g, &byte);
      }
    }
    if (!finite) {
      byte = kNv ? kNvNan : kMxNan;
      codes = 0;
    }
    if (in) *reinterpret_cast<uint32_t*>(out.codes + w.row * (K / 2) + c / 2) = codes;
    // (What fills a row of scales up is zeros.)
    const int at = c / (kLanes * kPerLane);
    if ((lane & (kLanes - 1)) == 0 && at < pitch)
      out.scales[w.row * pitch + at] = static_cast<uint8_t>(in ? byte : 0u);
  }
}

template <typename T, bool kNv>
__global__ void __launch_bounds__(kSegmentThreads)
dequantize_fp4_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      const float* __restrict__ gs, int64_t rows_per_plane, int64_t R, int K,
                      T* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int pitch = fp4_scale_pitch(K, kNv ? kFp4Nv : kFp4Mx);
  for (SegmentWalk w((K + 255) / 256); w.row < R; w.next()) {
    const int c = w.seg * 256 + lane * kPerLane;
    if (c >= K) continue;
    uint32_t h[4];
    fp4_halves8(__ldg(reinterpret_cast<const uint32_t*>(codes + w.row * (K / 2) + c / 2)), h);
    const uint32_t byte = __ldg(scales + w.row * pitch + c / (kNv ? 16 : 32));
    float scale;
    if (kNv) {
      scale = nv_scale(byte);
    } else {
      scale = byte == kMxNan ? __uint_as_float(0x7fffffffu) : mx_scale(byte);
    }
    // code * scale has 6 significant bits: exact; then g's rounding and that to T.
    const float g = kNv && gs ? __ldg(gs + (rows_per_plane < R ? w.row / rows_per_plane : 0)) : 1.0f;
    float f[kPerLane];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 two = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      f[2 * i] = two.x * scale * g;
      f[2 * i + 1] = two.y * scale * g;
    }
    store8(out + w.row * K + c, f);
  }
}

template <typename T>
cudaError_t quantize_t(const void* x, int64_t R, int K, int fmt, bool swiglu, const Fp4Out& out,
                       cudaStream_t s) {
  const int pitch = fp4_scale_pitch(K, fmt);
  const dim3 grid(segment_grid(R, fmt == kFp4Nv ? pitch / 16 : pitch / 8)), block(kSegmentThreads);
  const T* src = static_cast<const T*>(x);
  if (fmt == kFp4Nv)
    return swiglu ? launch_pdl(quantize_fp4_kernel<T, true, true>, grid, block, 0, s, src, R, K, out)
                  : launch_pdl(quantize_fp4_kernel<T, true, false>, grid, block, 0, s, src, R, K, out);
  return swiglu ? launch_pdl(quantize_fp4_kernel<T, false, true>, grid, block, 0, s, src, R, K, out)
                : launch_pdl(quantize_fp4_kernel<T, false, false>, grid, block, 0, s, src, R, K, out);
}

template <typename T>
cudaError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, const float* g,
                         int64_t rows_per_plane, int64_t R, int K, int fmt, void* out,
                         cudaStream_t s) {
  const dim3 grid(segment_grid(R, (K + 255) / 256)), block(kSegmentThreads);
  return fmt == kFp4Nv ? launch_pdl(dequantize_fp4_kernel<T, true>, grid, block, 0, s, codes, scales, g,
                                    rows_per_plane, R, K, static_cast<T*>(out))
                       : launch_pdl(dequantize_fp4_kernel<T, false>, grid, block, 0, s, codes, scales,
                                    g, rows_per_plane, R, K, static_cast<T*>(out));
}

}  // namespace

moe_status launch_quantize_fp4(const void* x, int64_t planes, int64_t rows, int K, int dtype, int fmt,
                               bool swiglu, const float* g, uint8_t* codes, uint8_t* scales,
                               cudaStream_t s) {
  const int64_t R = planes * rows;
  const Fp4Out out{codes, scales, g, rows};
  const cudaError_t err = dtype == MOE_DTYPE_BF16  ? quantize_t<__nv_bfloat16>(x, R, K, fmt, swiglu, out, s)
                          : dtype == MOE_DTYPE_F16 ? quantize_t<__half>(x, R, K, fmt, swiglu, out, s)
                                                   : quantize_t<float>(x, R, K, fmt, swiglu, out, s);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "quantize_fp4 launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

moe_status launch_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, const float* g,
                                 int64_t planes, int64_t rows, int K, int fmt, int dtype, void* out,
                                 cudaStream_t s) {
  const int64_t R = planes * rows;
  const cudaError_t err =
      dtype == MOE_DTYPE_BF16  ? dequantize_t<__nv_bfloat16>(codes, scales, g, rows, R, K, fmt, out, s)
      : dtype == MOE_DTYPE_F16 ? dequantize_t<__half>(codes, scales, g, rows, R, K, fmt, out, s)
                               : dequantize_t<float>(codes, scales, g, rows, R, K, fmt, out, s);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "dequantize_fp4 launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

}  // namespace moe
