// Microscaled 4-bit floating point. A code is e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), two to a
// byte, the lower channel in the low half; a block of neighbouring channels shares a scale byte:
//   mx  32 channels, byte b stands for 2^(b - 127), 255 for NaN
//   nv  16 channels, an e4m3 number, times an f32 g of the whole tensor or of each expert
// A row of scales starts on 16 bytes: its K / block bytes are filled up to a multiple of 16, and what
// fills it is not looked at.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

#include "internal.h"

namespace moe {

constexpr int kFp4Mx = MOE_FP4_MX;
constexpr int kFp4Nv = MOE_FP4_NV;
constexpr uint32_t kMxNan = 255, kNvNan = 0x7f;

__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == kFp4Mx ? 32 : 16; }
__host__ __device__ constexpr int fp4_scale_pitch(int K, int fmt) {
  return (K / fp4_block(fmt) + 15) / 16 * 16;
}

// 8 values rounded to e2m1 (to nearest, ties to even, 6 at most), the first in the lowest 4 bits.
__device__ __forceinline__ uint32_t fp4_codes8(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// The values of 8 codes, in pairs.
__device__ __forceinline__ void fp4_halves8(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

}  // namespace moe
