// C ABI entry points of the serving operators (4-bit operands, the layer for a few tokens): argument
// validation on the host, then the launch. Nothing here allocates device memory or synchronises.
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

// Limits of moe_layer_few.
bool few_fits(const moe_problem& p) {
  auto by32 = [](int32_t n, int32_t most) { return n >= 32 && n % 32 == 0 && n <= most; };
  return p.T >= 0 && p.T <= MOE_FEW_TOKENS && by32(p.H, 32768) && by32(p.I, 65536) &&
         (p.shared_I == 0 || by32(p.shared_I, 65536)) && p.E >= 1 && p.E <= 256 && p.k >= 1 && p.k <= 8 &&
         p.k <= p.E;
}

moe_status check_weights(const moe_weights* m, int weights, const char* name) {
  const bool four = weights != MOE_WEIGHTS_16BIT;
  if (!m || bad(m->w) || (four && bad(m->scales)))
    return set_error(MOE_ERR_INVALID_ARG, "%s NULL or not 16-byte aligned", name);
  if (!aligned(m->g, 4) || (m->g && weights != MOE_FP4_NV))
    return set_error(MOE_ERR_INVALID_ARG, "%s: g misaligned, or not of NV weights", name);
  return MOE_OK;
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

moe_status moe_selftest_fp4_wait(void* stream) {
  return launch_fp4_wait_selftest(static_cast<cudaStream_t>(stream));
}

moe_status moe_selftest_few_wait(void* stream) {
  return launch_few_wait_selftest(static_cast<cudaStream_t>(stream));
}

size_t moe_layer_few_workspace_bytes(const moe_problem* p) {
  return p && few_fits(*p) ? few_workspace_bytes(*p) : 0;
}

moe_status moe_layer_few(const moe_problem* p, const moe_route_params* route, const void* x,
                         const void* wg, int32_t shared_gate, const float* bias, const moe_weights* w13,
                         const moe_weights* w2, const moe_weights* w13_s, const moe_weights* w2_s,
                         int32_t weights, moe_dtype dtype, int32_t* ids, float* scales, void* y,
                         void* workspace, size_t ws_bytes, void* stream) {
  if (!p || !route) return set_error(MOE_ERR_INVALID_ARG, "problem or route params are NULL");
  if (!few_fits(*p))
    return set_error(MOE_ERR_UNSUPPORTED, "outside the limits for a few tokens (T %lld, H %d, I %d, "
                     "shared_I %d, E %d, k %d)", static_cast<long long>(p->T), p->H, p->I, p->shared_I,
                     p->E, p->k);
  if (weights != MOE_WEIGHTS_16BIT && weights != MOE_FP4_MX && weights != MOE_FP4_NV)
    return set_error(MOE_ERR_UNSUPPORTED, "weights %d are not taken here", weights);
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
    return set_error(MOE_ERR_UNSUPPORTED, "dtype %d is not taken here", dtype);
  if (route->num_experts != p->E || route->top_k != p->k)
    return set_error(MOE_ERR_INVALID_ARG, "route params of %d experts, %d slots for a layer of %d, %d",
                     route->num_experts, route->top_k, p->E, p->k);
  const int32_t reason = route_reason(p->T, *route, 256);
  if (reason == MOE_REASON_DEGENERATE)
    return set_error(MOE_ERR_UNSUPPORTED, "grouped top-k with softmax scoring: every group's score "
                     "is 1, so the group choice would rest on tie-breaking alone");
  if (reason != MOE_REASON_OK)
    return set_error(MOE_ERR_UNSUPPORTED, "routing outside the envelope (reason %d)", reason);
  if (shared_gate < 0 || shared_gate > 1 || (shared_gate == 1 && p->shared_I == 0))
    return set_error(MOE_ERR_INVALID_ARG, "a shared expert's gate without a shared expert");
  if (bias && route->method == MOE_ROUTE_GROUPED_TOPK)
    return set_error(MOE_ERR_INVALID_ARG, "the grouped top-k routing takes no bias");
  if (p->T == 0) return MOE_OK;
  if (bad(x) || bad(wg) || bad(ids) || bad(scales) || bad(y) || !aligned(bias, 16))
    return set_error(MOE_ERR_INVALID_ARG, "layer tensors NULL or not 16-byte aligned");
  moe_status st = check_weights(w13, weights, "w13");
  if (st == MOE_OK) st = check_weights(w2, weights, "w2");
  if (st == MOE_OK && p->shared_I > 0) st = check_weights(w13_s, weights, "w13_s");
  if (st == MOE_OK && p->shared_I > 0) st = check_weights(w2_s, weights, "w2_s");
  if (st != MOE_OK) return st;
  if (!workspace || !aligned(workspace, 256))
    return set_error(MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (ws_bytes < few_workspace_bytes(*p))
    return set_error(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", ws_bytes,
                     few_workspace_bytes(*p));
  FewLayer f = {};
  f.x = x;
  f.wg = wg;
  f.bias = bias;
  f.w13 = w13;
  f.w2 = w2;
  f.w13_s = p->shared_I > 0 ? w13_s : nullptr;
  f.w2_s = p->shared_I > 0 ? w2_s : nullptr;
  f.weights = weights;
  f.dtype = dtype;
  f.shared_gate = shared_gate;
  f.route = *route;
  f.ids = ids;
  f.scales = scales;
  f.y = y;
  return launch_few(*p, f, static_cast<char*>(workspace), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
