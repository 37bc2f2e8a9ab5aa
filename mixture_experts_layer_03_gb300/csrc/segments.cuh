// Rows walked a warp to a segment, as the operators between the experts' products do: SwiGLU with its checkpoint
// (segments of 256 channels, 8 a lane; of rows that do not start on 16 bytes 4 or 8 blocks of 32) and the
// conversions to 4 bits (256 or 512, 8 or 16 a lane) and back (1024, four times 8 a lane).
#pragma once

#include <cstdint>

#include "internal.h"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kSegmentThreads = 128;
constexpr int kPerLane = 8;        // channels of a vector load or store of a lane

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

// The work of a warp, one after the other: (row, segment) pairs. Stepping (row,
// segment) by the grid's share keeps divisions out.
struct SegmentWalk {
  int64_t row;
  int seg;
  int64_t row_step;
  int seg_step, segs;
  __device__ __forceinline__ SegmentWalk(int segs_) : segs(segs_) {
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * kSegmentThreads + threadIdx.x) >> 5;
    const int64_t n = static_cast<int64_t>(gridDim.x) * (kSegmentThreads / 32);
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

// Small blocks, four times as many as are resident: a block's warps then end, and their successors'
// loads begin, at different times. At 8192 x 14336 bf16, SwiGLU's checkpoint forward and backward with h:
// 149 and 175 us (950 MB at 6.36 TB/s, 1.18 GB at 6.75); blocks of 256 threads 162 and 175; eight of
// those an SM, all resident, 169 and 197.
inline unsigned segment_grid(int64_t R, int segs) {
  const int64_t blocks = (R * segs + kSegmentThreads / 32 - 1) / (kSegmentThreads / 32);
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 64;
  return static_cast<unsigned>(blocks < cap ? blocks : cap);
}

}  // namespace
}  // namespace moe
