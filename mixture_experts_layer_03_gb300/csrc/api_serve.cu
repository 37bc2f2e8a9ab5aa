// C ABI entry points of the serving operators on 4-bit operands: argument validation on the host, then
// the launch. Nothing here allocates device memory or synchronises.
#include <cuda_runtime.h>

#include "internal.h"

using namespace moe;

namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// NULL or not on a 16-byte boundary.
bool bad(const void* p) { return !p || !aligned(p, 16); }

moe_status check_format(int format, const float* g) {
  if (format != MOE_FP4_MX && format != MOE_FP4_NV)
    return set_error(MOE_ERR_UNSUPPORTED, "4-bit format %d is not known", format);
  if (g && format != MOE_FP4_NV) return set_error(MOE_ERR_INVALID_ARG, "only NV tensors have a g");
  if (!aligned(g, 4)) return set_error(MOE_ERR_INVALID_ARG, "g misaligned");
  return MOE_OK;
}

moe_status check_fp4(int64_t planes, int64_t rows, int32_t K, int dtype, int format, const float* g) {
  if (planes < 0 || rows < 0 || planes > (int64_t{1} << 31) || rows > (int64_t{1} << 31) ||
      (rows > 0 && planes > (int64_t{1} << 31) / rows))
    return set_error(MOE_ERR_UNSUPPORTED, "%lld planes of %lld rows outside [0, 2^31] rows",
                     static_cast<long long>(planes), static_cast<long long>(rows));
  if (K < 32 || K % 32 != 0 || K > 65536)
    return set_error(MOE_ERR_UNSUPPORTED, "%d channels: must be a multiple of 32 in [32, 65536]", K);
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16 && dtype != MOE_DTYPE_F32)
    return set_error(MOE_ERR_UNSUPPORTED, "dtype %d is not taken here", dtype);
  return check_format(format, g);
}

moe_status quantize(const void* x, int64_t planes, int64_t rows, int32_t K, int dtype, int format,
                    bool swiglu, const float* g, uint8_t* codes, uint8_t* scales, void* stream) {
  const moe_status st = check_fp4(planes, rows, K, dtype, format, g);
  if (st != MOE_OK || planes * rows == 0) return st;
  if (bad(x) || bad(codes) || bad(scales))
    return set_error(MOE_ERR_INVALID_ARG, "4-bit tensors NULL or not 16-byte aligned");
  return launch_quantize_fp4(x, planes, rows, K, dtype, format, swiglu, g, codes, scales,
                             static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

moe_status moe_quantize_fp4(const void* x, int64_t planes, int64_t rows, int32_t K, moe_dtype dtype,
                            moe_fp4_format format, const float* g, uint8_t* codes, uint8_t* scales,
                            void* stream) {
  return quantize(x, planes, rows, K, dtype, format, false, g, codes, scales, stream);
}

moe_status moe_swiglu_fp4(const void* gu, int64_t rows, int32_t I, moe_dtype dtype,
                          moe_fp4_format format, const float* g, uint8_t* codes, uint8_t* scales,
                          void* stream) {
  return quantize(gu, 1, rows, I, dtype, format, true, g, codes, scales, stream);
}

moe_status moe_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, const float* g,
                              int64_t planes, int64_t rows, int32_t K, moe_fp4_format format,
                              moe_dtype dtype, void* out, void* stream) {
  const moe_status st = check_fp4(planes, rows, K, dtype, format, g);
  if (st != MOE_OK || planes * rows == 0) return st;
  if (bad(codes) || bad(scales) || bad(out))
    return set_error(MOE_ERR_INVALID_ARG, "4-bit tensors NULL or not 16-byte aligned");
  return launch_dequantize_fp4(codes, scales, g, planes, rows, K, format, dtype, out,
                               static_cast<cudaStream_t>(stream));
}

moe_status moe_experts_matmul_fp4(const uint8_t* x_codes, const uint8_t* x_scales, const float* x_g,
                                  const uint8_t* w_codes, const uint8_t* w_scales, const float* w_g,
                                  const int32_t* offsets, int64_t R, int32_t E, int32_t N, int32_t K,
                                  moe_fp4_format format, moe_dtype dtype, void* y, void* stream) {
  if (R < 0 || R > (int64_t{1} << 23))
    return set_error(MOE_ERR_UNSUPPORTED, "R %lld outside [0, 2^23]", static_cast<long long>(R));
  if (E < 1 || E > 256) return set_error(MOE_ERR_UNSUPPORTED, "E %d outside [1, 256]", E);
  if (N < 8 || N % 8 != 0 || N > 65536 || K < 32 || K % 32 != 0 || K > 65536)
    return set_error(MOE_ERR_UNSUPPORTED, "N %d must be a multiple of 8, K %d of 32, up to 65536", N, K);
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
    return set_error(MOE_ERR_UNSUPPORTED, "dtype %d is not taken here", dtype);
  moe_status st = check_format(format, x_g);
  if (st == MOE_OK) st = check_format(format, w_g);
  if (st != MOE_OK || R == 0) return st;
  if (bad(x_codes) || bad(x_scales) || bad(w_codes) || bad(w_scales) || bad(y) || !offsets ||
      !aligned(offsets, 4))
    return set_error(MOE_ERR_INVALID_ARG, "rows, weights or offsets NULL or misaligned");
  return launch_experts_fp4(Fp4Operand{x_codes, x_scales, x_g}, Fp4Operand{w_codes, w_scales, w_g},
                            offsets, R, E, N, K, format, dtype, y, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
