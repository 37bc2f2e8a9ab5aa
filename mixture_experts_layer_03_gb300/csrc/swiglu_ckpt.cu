// SwiGLU whose input is kept for the backward pass in 8 bits.
//
// gu [R, 2I] holds the gate g and the up projection u of each row side by side (the order of
// w13's rows); h = g sigma(g) u. What the backward pass needs of gu is kept as e4m3 values with
// one power of two per 32 neighbouring channels of g or of u (the last block of a row's half may
// be shorter):
//   amax = max |v| over the block;  e = the least integer >= -127 with amax <= 448 * 2^e
//   scale byte = e + 127,  q = e4m3(v * 2^-e) rounded to nearest even
// so no value saturates and, the scale being a power of two, v * 2^-e is exact: the kept value
// differs from v by at most |v| / 16, or 2^(e-10) where it falls below e4m3's normal range.
// A block that holds an infinity or a NaN gets scale byte 255, which reads as NaN.
// Backward, with g and u as kept and s = sigma(g):
//   dg = dh u s (1 + g (1 - s)),  du = dh g s,  and, where wanted, h again = g s u
// (what the gradient of the next weights needs: with it neither gu nor h is held in 16 bits
// between the passes, 2I (1 + 1/32) bytes a row instead of 6I).
// Both directions read and write each value once and are bound by memory; the arithmetic is
// kept to an exponential, a reciprocal and a handful of multiplies a channel so that it stays so.
#include <cstdint>

#include <cuda_fp8.h>

#include "internal.h"
#include "launch.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kCkptThreads = 128;
constexpr int kCkptBlock = 32;     // channels that share a scale
constexpr int kPerLane = 8;        // channels a lane holds in the vector form
constexpr uint32_t kNanScale = 255;

// sigma(g) and 1 - sigma(g). For 16-bit results by the fast exponential and quotient, whose error of 2 +
// 1.17 |g| units of 2^-23 (under 2^-16 where sigma is not 0) is small beside the one rounding of the
// result (2^-9 or 2^-12). For f32 ones from exp(-|g|): a few units at any g, and 1 - sigma without
// cancellation. f32, forward and backward with h, the one way and the other: 8192 x 14336 245 and 325 us,
// 243 and 370; 1941 x 13603, bound by instructions, 67 and 94, 60 and 88.
template <typename T>
__device__ __forceinline__ float2 sigmoid_of(float g) {
  if constexpr (sizeof(T) == 4) {
    const float t = expf(-fabsf(g));
    const float big = 1.0f / (1.0f + t), small = t * big;
    return g < 0.0f ? make_float2(small, big) : make_float2(big, small);
  } else {
    const float s = __fdividef(1.0f, 1.0f + __expf(-g));
    return make_float2(s, 1.0f - s);
  }
}

// The scale byte of a block: the least e >= -127 with amax <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax);
  if (b >= 0x7f800000u) return kNanScale;
  // Exponent field E and mantissa M of amax = (1 + M/2^23) 2^(E - 127): e + 8 = E - 127, one
  // more where 1 + M/2^23 > 1.75. Subnormal amax (E = 0) gives the floor.
  const int e = static_cast<int>((b + 0x001fffffu) >> 23) - 8;
  return static_cast<uint32_t>(e > 0 ? e : 0);
}

// 2^-e (to quantise) and 2^e (to read) of a scale byte e + 127. Byte 0 is 2^-127, a subnormal;
// its inverse 2^127 is normal. Byte 255 reads as NaN.
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  // 127 - e = 254 - byte as an exponent field; finite values give bytes up to 247 (448 * 2^120 is over
  // the largest float), and for 255 the products are not used.
  return __uint_as_float((254u - (byte < 254u ? byte : 253u)) << 23);
}
__device__ __forceinline__ float scale_of(uint32_t byte) {
  if (byte == 0) return __uint_as_float(0x00400000u);
  return byte == kNanScale ? __uint_as_float(0x7fffffffu) : __uint_as_float(byte << 23);
}

__device__ __forceinline__ uint32_t quant2(float lo, float hi) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3));
}

__device__ __forceinline__ float2 dequant2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// 8 values of a lane and the largest magnitude of its block of four lanes; a NaN wins.
__device__ __forceinline__ float block_amax(const float (&f)[kPerLane]) {
  uint32_t m = 0;   // magnitudes order as their bit patterns do, infinities and NaNs on top
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return __uint_as_float(m);
}

__device__ __forceinline__ uint2 quant8(const float (&f)[kPerLane], float inv) {
  uint2 q;
  q.x = quant2(f[0] * inv, f[1] * inv) | quant2(f[2] * inv, f[3] * inv) << 16;
  q.y = quant2(f[4] * inv, f[5] * inv) | quant2(f[6] * inv, f[7] * inv) << 16;
  return q;
}

__device__ __forceinline__ void dequant8(uint2 q, float scale, float (&f)[kPerLane]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = (i < 2 ? q.x : q.y) >> (16 * (i & 1)) & 0xffffu;
    const float2 v = dequant2(two);
    f[2 * i] = v.x * scale;
    f[2 * i + 1] = v.y * scale;
  }
}

// 8 elements of T as one or two 16-byte vectors.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[kPerLane]) {
  constexpr int kN = 16 / static_cast<int>(sizeof(T));
#pragma unroll
  for (int h = 0; h < kPerLane / kN; ++h) {
    float part[kN];
    Vec<T, 16>::unpack(__ldg(reinterpret_cast<const uint4*>(p) + h), part);
#pragma unroll
    for (int i = 0; i < kN; ++i) f[h * kN + i] = part[i];
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[kPerLane]) {
  constexpr int kN = 16 / static_cast<int>(sizeof(T));
#pragma unroll
  for (int h = 0; h < kPerLane / kN; ++h) {
    float part[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) part[i] = f[h * kN + i];
    reinterpret_cast<uint4*>(p)[h] = Vec<T, 16>::pack(part);
  }
}

// The work of a warp, one after the other: (row, segment) pairs, a segment 256 channels, four
// lanes to a block of 32. Stepping (row, segment) by the grid's share keeps divisions out.
struct Walk {
  int64_t row;
  int seg;
  int64_t row_step;
  int seg_step, segs;
  __device__ __forceinline__ Walk(int segs_) : segs(segs_) {
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * kCkptThreads + threadIdx.x) >> 5;
    const int64_t n = static_cast<int64_t>(gridDim.x) * (kCkptThreads / 32);
    row = w / segs_;
    seg = static_cast<int>(w - row * segs_);
    row_step = n / segs_;
    seg_step = static_cast<int>(n - row_step * segs_);
  }
  __device__ __forceinline__ void next() {
    row += row_step;
    seg += seg_step;
    if (seg >= segs) {
      seg -= segs;
      ++row;
    }
  }
};

// Rows whose halves start on 16-byte boundaries (I % 8 == 0): 8 channels a lane.
template <typename T>
__global__ void __launch_bounds__(kCkptThreads)
swiglu_ckpt_kernel(const T* __restrict__ gu, int64_t R, int I, T* __restrict__ h,
                   uint8_t* __restrict__ q, uint8_t* __restrict__ qs) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int nb = (I + kCkptBlock - 1) / kCkptBlock;
  for (Walk w((I + 255) / 256); w.row < R; w.next()) {
    const int c = w.seg * 256 + lane * kPerLane;
    const bool in = c < I;
    float g[kPerLane] = {}, u[kPerLane] = {};
    const T* src = gu + w.row * 2 * I + c;
    if (in) {
      load8(src, g);
      load8(src + I, u);
    }
    const uint32_t sg = scale_byte(block_amax(g));
    const uint32_t su = scale_byte(block_amax(u));
    if (!in) continue;   // the four lanes of a block shuffle above, together with all others
    float y[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) y[i] = g[i] * sigmoid_of<T>(g[i]).x * u[i];
    store8(h + w.row * I + c, y);
    uint8_t* dst = q + w.row * 2 * I + c;
    *reinterpret_cast<uint2*>(dst) = quant8(g, inv_scale(sg));
    *reinterpret_cast<uint2*>(dst + I) = quant8(u, inv_scale(su));
    if ((lane & 3) == 0) {
      uint8_t* sd = qs + w.row * 2 * nb + c / kCkptBlock;
      sd[0] = static_cast<uint8_t>(sg);
      sd[nb] = static_cast<uint8_t>(su);
    }
  }
}

template <typename T>
__device__ __forceinline__ void grad_of(float dh, float g, float u, float* dg, float* du,
                                        float* h) {
  const float2 s = sigmoid_of<T>(g);
  const float gs = g * s.x;
  *h = gs * u;
  *du = dh * gs;
  *dg = dh * u * (s.x + gs * s.y);
}

template <typename T, bool kWantH>
__global__ void __launch_bounds__(kCkptThreads)
swiglu_ckpt_grad_kernel(const T* __restrict__ dh, const uint8_t* __restrict__ q,
                        const uint8_t* __restrict__ qs, int64_t R, int I, T* __restrict__ dgu,
                        T* __restrict__ h) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int nb = (I + kCkptBlock - 1) / kCkptBlock;
  for (Walk w((I + 255) / 256); w.row < R; w.next()) {
    const int c = w.seg * 256 + lane * kPerLane;
    if (c >= I) continue;
    const uint8_t* src = q + w.row * 2 * I + c;
    const uint2 qg = __ldg(reinterpret_cast<const uint2*>(src));
    const uint2 qu = __ldg(reinterpret_cast<const uint2*>(src + I));
    const uint8_t* ss = qs + w.row * 2 * nb + c / kCkptBlock;
    float d[kPerLane], g[kPerLane], u[kPerLane], y[kPerLane];
    load8(dh + w.row * I + c, d);
    dequant8(qg, scale_of(__ldg(ss)), g);
    dequant8(qu, scale_of(__ldg(ss + nb)), u);
    float dg[kPerLane], du[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) grad_of<T>(d[i], g[i], u[i], &dg[i], &du[i], &y[i]);
    T* dst = dgu + w.row * 2 * I + c;
    store8(dst, dg);
    store8(dst + I, du);
    if (kWantH) store8(h + w.row * I + c, y);
  }
}

// Any I: neighbouring channels to neighbouring lanes, a warp to a segment of kBlocks blocks of 32
// channels of g and of u. These kernels are bound by instructions, so lane j looks after the scale of
// block j alone (those of g, then of u) and full segments go without a check: 1941 rows of 13603
// channels bf16, forward and backward with h, 48 and 58 us; with each scale in every lane 73 and 79.
// (Vectors of 16 bytes, shifted into place through shuffles or through shared memory, took 62 to 82
// and 80 to 103.) Eight blocks, or four where these hold a row: 8000 rows of 70 channels 4.4 and 4.8 us
// so, with eight 5.3 and 5.4; 1941 of 13603 with four 50 and 62.

// v[lane % n], for n values that are the same in every lane.
template <int n>
__device__ __forceinline__ uint32_t pick_lane(uint32_t (&v)[n], int lane) {
#pragma unroll
  for (int w = n / 2, bit = n / 2; w >= 1; w /= 2, bit /= 2)
#pragma unroll
    for (int i = 0; i < w; ++i) v[i] = lane & bit ? v[i + w] : v[i];
  return v[0];
}

// A warp's segment: channels from c0 on; kFull: all of them below I.
template <typename T, int kBlocks, bool kFull>
__device__ __forceinline__ void ckpt_segment(const T* src, int I, int c0, T* h, uint8_t* q,
                                             uint8_t* qs) {
  const int lane = threadIdx.x & 31;
  const int nb = (I + kCkptBlock - 1) / kCkptBlock, b0 = c0 / kCkptBlock;
  float g[kBlocks], u[kBlocks];
  const T* in = src + c0 + lane;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    const bool there = kFull || c0 + i * kCkptBlock + lane < I;
    g[i] = there ? to_f32<T>(__ldg(in + i * kCkptBlock)) : 0.0f;
    u[i] = there ? to_f32<T>(__ldg(in + I + i * kCkptBlock)) : 0.0f;
  }
  uint32_t m[2 * kBlocks];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    m[i] = __reduce_max_sync(0xffffffffu, __float_as_uint(g[i]) & 0x7fffffffu);
    m[kBlocks + i] = __reduce_max_sync(0xffffffffu, __float_as_uint(u[i]) & 0x7fffffffu);
  }
  const uint32_t mine = scale_byte(__uint_as_float(pick_lane(m, lane)));
  const float inv = inv_scale(mine);
  const int block = b0 + lane % kBlocks;
  if (lane < 2 * kBlocks && (kFull || block < nb))
    qs[lane < kBlocks ? block : nb + block] = static_cast<uint8_t>(mine);
  T* out_h = h + c0 + lane;
  uint8_t* out_q = q + c0 + lane;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    const float ig = __shfl_sync(0xffffffffu, inv, i);
    const float iu = __shfl_sync(0xffffffffu, inv, kBlocks + i);
    if (!kFull && c0 + i * kCkptBlock + lane >= I) continue;
    out_h[i * kCkptBlock] = from_f32<T>(g[i] * sigmoid_of<T>(g[i]).x * u[i]);
    const uint32_t two = quant2(g[i] * ig, u[i] * iu);
    out_q[i * kCkptBlock] = static_cast<uint8_t>(two);
    out_q[I + i * kCkptBlock] = static_cast<uint8_t>(two >> 8);
  }
}

template <typename T, int kBlocks>
__global__ void __launch_bounds__(kCkptThreads)
swiglu_ckpt_any_kernel(const T* __restrict__ gu, int64_t R, int I, T* __restrict__ h,
                       uint8_t* __restrict__ q, uint8_t* __restrict__ qs) {
  pdl_trigger();
  pdl_wait();
  constexpr int kSegment = kBlocks * kCkptBlock;
  const int nb = (I + kCkptBlock - 1) / kCkptBlock;
  for (Walk w((I + kSegment - 1) / kSegment); w.row < R; w.next()) {
    const int c0 = w.seg * kSegment;
    const int64_t at = w.row * I;
    if (c0 + kSegment <= I)
      ckpt_segment<T, kBlocks, true>(gu + 2 * at, I, c0, h + at, q + 2 * at, qs + w.row * 2 * nb);
    else
      ckpt_segment<T, kBlocks, false>(gu + 2 * at, I, c0, h + at, q + 2 * at, qs + w.row * 2 * nb);
  }
}

template <typename T, int kBlocks, bool kWantH, bool kFull>
__device__ __forceinline__ void ckpt_grad_segment(const T* dh, const uint8_t* q, const uint8_t* qs,
                                                  int I, int c0, T* dgu, T* h) {
  const int lane = threadIdx.x & 31;
  const int nb = (I + kCkptBlock - 1) / kCkptBlock, b0 = c0 / kCkptBlock;
  float d[kBlocks];
  uint32_t two[kBlocks];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    // Lanes past the row's end read its last channel, and write nothing.
    const int c = kFull ? c0 + i * kCkptBlock + lane : min(c0 + i * kCkptBlock + lane, I - 1);
    d[i] = to_f32<T>(__ldg(dh + c));
    two[i] = __ldg(q + c) | __ldg(q + I + c) << 8;
  }
  const int block = kFull ? b0 + lane % kBlocks : min(b0 + lane % kBlocks, nb - 1);
  const float scale = scale_of(__ldg(qs + (lane & kBlocks ? nb + block : block)));
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    const float2 v = dequant2(two[i]);
    const float g = v.x * __shfl_sync(0xffffffffu, scale, i);
    const float u = v.y * __shfl_sync(0xffffffffu, scale, kBlocks + i);
    const int c = c0 + i * kCkptBlock + lane;
    if (!kFull && c >= I) continue;
    float dg, du, y;
    grad_of<T>(d[i], g, u, &dg, &du, &y);
    dgu[c] = from_f32<T>(dg);
    dgu[I + c] = from_f32<T>(du);
    if (kWantH) h[c] = from_f32<T>(y);
  }
}

template <typename T, int kBlocks, bool kWantH>
__global__ void __launch_bounds__(kCkptThreads)
swiglu_ckpt_grad_any_kernel(const T* __restrict__ dh, const uint8_t* __restrict__ q,
                            const uint8_t* __restrict__ qs, int64_t R, int I, T* __restrict__ dgu,
                            T* __restrict__ h) {
  pdl_trigger();
  pdl_wait();
  constexpr int kSegment = kBlocks * kCkptBlock;
  const int nb = (I + kCkptBlock - 1) / kCkptBlock;
  for (Walk w((I + kSegment - 1) / kSegment); w.row < R; w.next()) {
    const int c0 = w.seg * kSegment;
    const int64_t at = w.row * I;
    if (c0 + kSegment <= I)
      ckpt_grad_segment<T, kBlocks, kWantH, true>(dh + at, q + 2 * at, qs + w.row * 2 * nb, I, c0,
                                         dgu + 2 * at, h + at);
    else
      ckpt_grad_segment<T, kBlocks, kWantH, false>(dh + at, q + 2 * at, qs + w.row * 2 * nb, I, c0,
                                          dgu + 2 * at, h + at);
  }
}

// Small blocks, four times as many as are resident: a block's warps then end, and their successors'
// loads begin, at different times. At 8192 x 14336 bf16, forward and backward with h: 149 and 175
// us (950 MB at 6.36 TB/s, 1.18 GB at 6.75); blocks of 256 threads 162 and 175; eight of those an
// SM, all resident, 169 and 197.
unsigned ckpt_grid(int64_t R, int segs) {
  const int64_t blocks = (R * segs + kCkptThreads / 32 - 1) / (kCkptThreads / 32);
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 64;
  return static_cast<unsigned>(blocks < cap ? blocks : cap);
}

template <typename T>
cudaError_t forward_t(const void* gu, int64_t R, int I, void* h, uint8_t* q, uint8_t* qs,
                      cudaStream_t s) {
  if (I % kPerLane == 0)
    return launch_pdl(swiglu_ckpt_kernel<T>, dim3(ckpt_grid(R, (I + 255) / 256)),
                      dim3(kCkptThreads), 0, s, static_cast<const T*>(gu), R, I,
                      static_cast<T*>(h), q, qs);
  if (I <= 128)
    return launch_pdl(swiglu_ckpt_any_kernel<T, 4>, dim3(ckpt_grid(R, 1)), dim3(kCkptThreads), 0, s,
                      static_cast<const T*>(gu), R, I, static_cast<T*>(h), q, qs);
  return launch_pdl(swiglu_ckpt_any_kernel<T, 8>, dim3(ckpt_grid(R, (I + 255) / 256)),
                    dim3(kCkptThreads), 0, s, static_cast<const T*>(gu), R, I, static_cast<T*>(h), q,
                    qs);
}

template <typename T, bool kWantH>
cudaError_t backward_t(const void* dh, const uint8_t* q, const uint8_t* qs, int64_t R, int I,
                       void* dgu, void* h, cudaStream_t s) {
  if (I % kPerLane == 0)
    return launch_pdl(swiglu_ckpt_grad_kernel<T, kWantH>, dim3(ckpt_grid(R, (I + 255) / 256)),
                      dim3(kCkptThreads), 0, s, static_cast<const T*>(dh), q, qs, R, I,
                      static_cast<T*>(dgu), static_cast<T*>(h));
  if (I <= 128)
    return launch_pdl(swiglu_ckpt_grad_any_kernel<T, 4, kWantH>, dim3(ckpt_grid(R, 1)),
                      dim3(kCkptThreads), 0, s, static_cast<const T*>(dh), q, qs, R, I,
                      static_cast<T*>(dgu), static_cast<T*>(h));
  return launch_pdl(swiglu_ckpt_grad_any_kernel<T, 8, kWantH>, dim3(ckpt_grid(R, (I + 255) / 256)),
                    dim3(kCkptThreads), 0, s, static_cast<const T*>(dh), q, qs, R, I,
                    static_cast<T*>(dgu), static_cast<T*>(h));
}

}  // namespace

moe_status launch_swiglu_ckpt(const void* gu, int64_t R, int I, int dtype, void* h, uint8_t* q,
                              uint8_t* qs, cudaStream_t s) {
  const cudaError_t err =
      dtype == MOE_DTYPE_BF16  ? forward_t<__nv_bfloat16>(gu, R, I, h, q, qs, s)
      : dtype == MOE_DTYPE_F16 ? forward_t<__half>(gu, R, I, h, q, qs, s)
                               : forward_t<float>(gu, R, I, h, q, qs, s);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "swiglu_ckpt launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

moe_status launch_swiglu_ckpt_backward(const void* dh, const uint8_t* q, const uint8_t* qs,
                                       int64_t R, int I, int dtype, void* dgu, void* h,
                                       cudaStream_t s) {
  cudaError_t err;
  if (dtype == MOE_DTYPE_BF16)
    err = h ? backward_t<__nv_bfloat16, true>(dh, q, qs, R, I, dgu, h, s)
            : backward_t<__nv_bfloat16, false>(dh, q, qs, R, I, dgu, h, s);
  else if (dtype == MOE_DTYPE_F16)
    err = h ? backward_t<__half, true>(dh, q, qs, R, I, dgu, h, s)
            : backward_t<__half, false>(dh, q, qs, R, I, dgu, h, s);
  else
    err = h ? backward_t<float, true>(dh, q, qs, R, I, dgu, h, s)
            : backward_t<float, false>(dh, q, qs, R, I, dgu, h, s);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "swiglu_ckpt_backward launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

}  // namespace moe
