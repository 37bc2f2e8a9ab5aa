// C ABI entry points of the training operators: argument validation on the host, then the
// launch. Nothing here allocates device memory or synchronises.
#include <cuda_runtime.h>

#include "internal.h"

using namespace moe;

namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// NULL or not on a 16-byte boundary.
bool bad(const void* p) { return !p || !aligned(p, 16); }

// The status word of a call that launches nothing, where it has a workspace.
cudaError_t clear_status(void* ws, size_t ws_bytes, uintptr_t align, void* stream) {
  if (!ws || !aligned(ws, align) || ws_bytes < 16) return cudaSuccess;
  return cudaMemsetAsync(ws, 0, 16, static_cast<cudaStream_t>(stream));
}

moe_status check_dtype(int dtype, bool with_f32) {
  if (dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F16 || (with_f32 && dtype == MOE_DTYPE_F32))
    return MOE_OK;
  return set_error(MOE_ERR_UNSUPPORTED, "dtype %d is not taken here", dtype);
}

// T tokens, k slots, rows of H elements.
moe_status check_rows(int64_t T, int32_t H, int32_t k, int dtype) {
  if (T < 0 || T > (int64_t{1} << 24))
    return set_error(MOE_ERR_UNSUPPORTED, "T %lld outside [0, 2^24]", static_cast<long long>(T));
  if (k < 1 || k > 8) return set_error(MOE_ERR_UNSUPPORTED, "k %d outside [1, 8]", k);
  if (H < 1 || H > 65536) return set_error(MOE_ERR_UNSUPPORTED, "H %d outside [1, 65536]", H);
  return check_dtype(dtype, true);
}

moe_status check_experts(int64_t R, int32_t E, int32_t N, int32_t K, int dtype) {
  if (R < 0 || R > (int64_t{1} << 23))
    return set_error(MOE_ERR_UNSUPPORTED, "R %lld outside [0, 2^23]", static_cast<long long>(R));
  if (E < 1 || E > 256) return set_error(MOE_ERR_UNSUPPORTED, "E %d outside [1, 256]", E);
  if (N < 8 || N % 8 != 0 || N > 65536 || K < 8 || K % 8 != 0 || K > 65536)
    return set_error(MOE_ERR_UNSUPPORTED, "N %d and K %d must be multiples of 8 in [8, 65536]", N, K);
  return check_dtype(dtype, false);
}

moe_status experts_rows(bool dx, const void* in, const void* w, const int32_t* offsets, int64_t R,
                        int32_t E, int32_t N, int32_t K, int dtype, void* out, void* workspace,
                        size_t ws_bytes, void* stream) {
  const moe_status st = check_experts(R, E, N, K, dtype);
  if (st != MOE_OK) return st;
  if (workspace && (!aligned(workspace, 128) || ws_bytes < 16))
    return set_error(MOE_ERR_INVALID_ARG, "workspace must be 128-byte aligned and hold 16 bytes");
  if (R == 0) return MOE_OK;
  if (bad(in) || bad(w) || bad(out) || !offsets || !aligned(offsets, 4))
    return set_error(MOE_ERR_INVALID_ARG, "rows, weights or offsets NULL or misaligned");
  if (!dx && experts_few(R, E))
    return launch_experts_few(in, w, offsets, R, E, N, K, dtype, out,
                              static_cast<cudaStream_t>(stream));
  return launch_experts_rows(dx, in, w, offsets, R, E, N, K, dtype, out,
                             static_cast<char*>(workspace), ws_bytes,
                             static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

size_t moe_dispatch_workspace_bytes(int64_t T, int32_t E, int32_t k) {
  if (check_rows(T, 1, k, MOE_DTYPE_BF16) != MOE_OK || E < 1 || E > 256) return 0;
  return dispatch_workspace_bytes(T, E);
}

moe_status moe_dispatch(const void* x, const int32_t* ids, int64_t T, int32_t H, int32_t E,
                        int32_t k, moe_dtype dtype, void* x_perm, int32_t* inv, int32_t* offsets,
                        void* workspace, size_t ws_bytes, void* stream) {
  const moe_status st = check_rows(T, H, k, dtype);
  if (st != MOE_OK) return st;
  if (E < 1 || E > 256) return set_error(MOE_ERR_UNSUPPORTED, "E %d outside [1, 256]", E);
  if (T == 0) {
    // No slots: every expert's rows are empty.
    if (!offsets || !aligned(offsets, 4)) return set_error(MOE_ERR_INVALID_ARG, "offsets NULL or misaligned");
    cudaError_t e = cudaMemsetAsync(offsets, 0, 4 * (static_cast<size_t>(E) + 1),
                                    static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) e = clear_status(workspace, ws_bytes, 16, stream);
    return e == cudaSuccess ? MOE_OK
                            : set_error(MOE_ERR_CUDA, "offsets clear: %s", cudaGetErrorString(e));
  }
  if (bad(x) || bad(ids) || bad(x_perm) || bad(inv) || !offsets || !aligned(offsets, 4))
    return set_error(MOE_ERR_INVALID_ARG, "dispatch tensors NULL or not 16-byte aligned");
  if (!aligned(workspace, 16) || (!workspace && T * k > MOE_DISPATCH_SMALL_SLOTS))
    return set_error(MOE_ERR_INVALID_ARG, "workspace NULL or not 16-byte aligned");
  const size_t need = workspace ? dispatch_workspace_bytes(T, E) : 0;
  if (ws_bytes < need)
    return set_error(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", ws_bytes, need);
  return launch_dispatch(x, ids, T, H, E, k, dtype, x_perm, inv, offsets,
                         static_cast<char*>(workspace), static_cast<cudaStream_t>(stream));
}

moe_status moe_dispatch_rows(const void* x, const int32_t* inv, int64_t T, int32_t H, int32_t k,
                             moe_dtype dtype, void* x_perm, void* stream) {
  const moe_status st = check_rows(T, H, k, dtype);
  if (st != MOE_OK || T == 0) return st;
  if (bad(x) || bad(inv) || bad(x_perm))
    return set_error(MOE_ERR_INVALID_ARG, "dispatch tensors NULL or not 16-byte aligned");
  return launch_dispatch_rows(x, inv, T, H, k, dtype, x_perm, static_cast<cudaStream_t>(stream));
}

moe_status moe_combine(const void* rows, const int32_t* inv, const float* scales, int64_t T,
                       int32_t H, int32_t k, moe_dtype dtype, void* y, void* stream) {
  const moe_status st = check_rows(T, H, k, dtype);
  if (st != MOE_OK || T == 0) return st;
  if (bad(rows) || bad(inv) || bad(y) || !aligned(scales, 16))
    return set_error(MOE_ERR_INVALID_ARG, "combine tensors NULL or not 16-byte aligned");
  return launch_combine(rows, inv, scales, T, H, k, dtype, y, static_cast<cudaStream_t>(stream));
}

moe_status moe_combine_backward(const void* dy, const void* rows, const int32_t* inv,
                                const float* scales, int64_t T, int32_t H, int32_t k,
                                moe_dtype dtype, void* drows, float* dscales, void* stream) {
  const moe_status st = check_rows(T, H, k, dtype);
  if (st != MOE_OK || T == 0) return st;
  if (bad(dy) || bad(rows) || bad(inv) || !aligned(scales, 16) || bad(drows) || bad(dscales))
    return set_error(MOE_ERR_INVALID_ARG, "combine_backward tensors NULL or not 16-byte aligned");
  return launch_combine_backward(dy, rows, inv, scales, T, H, k, dtype, drows, dscales,
                                 static_cast<cudaStream_t>(stream));
}

moe_status moe_dispatch_backward(const void* dx_perm, const int32_t* inv, int64_t T, int32_t H,
                                 int32_t k, moe_dtype dtype, void* dx, void* stream) {
  return moe_combine(dx_perm, inv, nullptr, T, H, k, dtype, dx, stream);
}

moe_status moe_swiglu_ckpt(const void* gu, int64_t R, int32_t I, moe_dtype dtype, void* h,
                           uint8_t* q, uint8_t* q_scales, void* stream) {
  if (R < 0 || R > (int64_t{1} << 31) || I < 1 || I > 65536)
    return set_error(MOE_ERR_UNSUPPORTED, "R %lld outside [0, 2^31] or I %d outside [1, 65536]",
                     static_cast<long long>(R), I);
  const moe_status st = check_dtype(dtype, true);
  if (st != MOE_OK || R == 0) return st;
  if (bad(gu) || bad(h) || bad(q) || bad(q_scales))
    return set_error(MOE_ERR_INVALID_ARG, "swiglu_ckpt tensors NULL or not 16-byte aligned");
  return launch_swiglu_ckpt(gu, R, I, dtype, h, q, q_scales, static_cast<cudaStream_t>(stream));
}

moe_status moe_swiglu_ckpt_backward(const void* dh, const uint8_t* q, const uint8_t* q_scales,
                                    int64_t R, int32_t I, moe_dtype dtype, void* dgu, void* h,
                                    void* stream) {
  if (R < 0 || R > (int64_t{1} << 31) || I < 1 || I > 65536)
    return set_error(MOE_ERR_UNSUPPORTED, "R %lld outside [0, 2^31] or I %d outside [1, 65536]",
                     static_cast<long long>(R), I);
  const moe_status st = check_dtype(dtype, true);
  if (st != MOE_OK || R == 0) return st;
  if (bad(dh) || bad(q) || bad(q_scales) || bad(dgu) || !aligned(h, 16))
    return set_error(MOE_ERR_INVALID_ARG, "swiglu_ckpt_backward tensors NULL or not 16-byte aligned");
  return launch_swiglu_ckpt_backward(dh, q, q_scales, R, I, dtype, dgu, h,
                                     static_cast<cudaStream_t>(stream));
}

size_t moe_experts_workspace_bytes(int32_t E) {
  return E < 1 || E > 256 ? 0 : experts_workspace_bytes(E);
}

size_t moe_experts_split_bytes(int32_t product, int64_t R, int32_t E, int32_t N, int32_t K) {
  if (product < 0 || product > 2 || check_experts(R, E, N, K, MOE_DTYPE_BF16) != MOE_OK || R == 0)
    return 0;
  if (product == 0 && experts_few(R, E)) return 0;
  return experts_split_bytes(product, R, E, N, K);
}

moe_status moe_experts_matmul(const void* x, const void* w, const int32_t* offsets, int64_t R,
                              int32_t E, int32_t N, int32_t K, moe_dtype dtype, void* y,
                              void* workspace, size_t ws_bytes, void* stream) {
  return experts_rows(false, x, w, offsets, R, E, N, K, dtype, y, workspace, ws_bytes, stream);
}

moe_status moe_experts_matmul_dx(const void* dy, const void* w, const int32_t* offsets, int64_t R,
                                 int32_t E, int32_t N, int32_t K, moe_dtype dtype, void* dx,
                                 void* workspace, size_t ws_bytes, void* stream) {
  return experts_rows(true, dy, w, offsets, R, E, N, K, dtype, dx, workspace, ws_bytes, stream);
}

moe_status moe_experts_matmul_dw(const void* dy, const void* x, const int32_t* offsets, int64_t R,
                                 int32_t E, int32_t N, int32_t K, moe_dtype dtype,
                                 moe_dtype dw_dtype, int32_t accumulate, void* dw, void* workspace,
                                 size_t ws_bytes, void* stream) {
  const moe_status st = check_experts(R, E, N, K, dtype);
  if (st != MOE_OK) return st;
  if (dw_dtype != dtype && dw_dtype != MOE_DTYPE_F32)
    return set_error(MOE_ERR_UNSUPPORTED, "dw is of the inputs' type or f32");
  if (accumulate && dw_dtype != MOE_DTYPE_F32)
    return set_error(MOE_ERR_UNSUPPORTED, "only an f32 dw is added to");
  if (bad(dw)) return set_error(MOE_ERR_INVALID_ARG, "dw NULL or not 16-byte aligned");
  if (R == 0) {
    const size_t n = static_cast<size_t>(E) * N * K * (dw_dtype == MOE_DTYPE_F32 ? 4 : 2);
    cudaError_t e = clear_status(workspace, ws_bytes, 128, stream);
    if (e == cudaSuccess && !accumulate)
      e = cudaMemsetAsync(dw, 0, n, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : set_error(MOE_ERR_CUDA, "dw clear: %s", cudaGetErrorString(e));
  }
  if (bad(dy) || bad(x) || !offsets || !aligned(offsets, 4))
    return set_error(MOE_ERR_INVALID_ARG, "rows or offsets NULL or misaligned");
  if (!workspace || !aligned(workspace, 128))
    return set_error(MOE_ERR_INVALID_ARG, "workspace must be 128-byte aligned");
  if (ws_bytes < experts_workspace_bytes(E))
    return set_error(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", ws_bytes,
                     experts_workspace_bytes(E));
  return launch_experts_dw(dy, x, offsets, R, E, N, K, dtype, dw_dtype, accumulate != 0, dw,
                           static_cast<char*>(workspace), ws_bytes,
                           static_cast<cudaStream_t>(stream));
}

moe_status moe_read_timeouts(void* stream, int32_t* flags) {
  void* word[2] = {nullptr, nullptr};
  moe_status st = experts_timeout_word(&word[0]);
  if (st == MOE_OK) st = gate_timeout_word(&word[1]);
  if (st != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t v[2] = {0, 0};
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 2 && e == cudaSuccess; ++i)
    e = cudaMemcpyAsync(&v[i], word[i], sizeof(v[i]), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  // Only what was read is cleared: another stream's call may set a word meanwhile.
  for (int i = 0; i < 2 && e == cudaSuccess; ++i)
    if (v[i]) e = cudaMemsetAsync(word[i], 0, sizeof(v[i]), s);
  if (e == cudaSuccess && (v[0] | v[1])) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "timeouts read: %s", cudaGetErrorString(e));
  if (flags) *flags = v[0] | v[1];
  return v[0] | v[1] ? MOE_ERR_DEVICE_TIMEOUT : MOE_OK;
}

moe_status moe_selftest_experts_wait(void* stream) {
  return launch_experts_wait_selftest(static_cast<cudaStream_t>(stream));
}

moe_status moe_route_backward(const float* logits, const int32_t* ids, const float* dscales,
                              int64_t T, const moe_route_params* p, float* dlogits, void* stream) {
  if (!p) return set_error(MOE_ERR_INVALID_ARG, "route params are NULL");
  if (T < 0 || T > (int64_t{1} << 31) / 8 || p->num_experts < 1 || p->num_experts > 256 ||
      p->top_k < 1 || p->top_k > 8 || p->top_k > p->num_experts)
    return set_error(MOE_ERR_UNSUPPORTED, "routing outside the envelope (T %lld, E %d, k %d)",
                     static_cast<long long>(T), p->num_experts, p->top_k);
  // The gradient does not depend on how the experts were chosen, so the group parameters are
  // not looked at; the method has to be one that moe_route runs.
  switch (p->method) {
    case MOE_ROUTE_DEFAULT:
    case MOE_ROUTE_RENORMALIZE:
    case MOE_ROUTE_DEEPSEEKV3:
    case MOE_ROUTE_LLAMA4:
    case MOE_ROUTE_RENORMALIZE_NAIVE:
    case MOE_ROUTE_MINIMAX2:
    case MOE_ROUTE_SIGMOID_RENORM:
    case MOE_ROUTE_GROUPED_TOPK:
      break;
    default:
      return set_error(MOE_ERR_UNSUPPORTED, "no gradient for routing method %d", p->method);
  }
  if (T == 0) return MOE_OK;
  if (bad(logits) || bad(ids) || bad(dscales) || bad(dlogits))
    return set_error(MOE_ERR_INVALID_ARG, "route_backward tensors NULL or not 16-byte aligned");
  return launch_route_backward(logits, ids, dscales, T, *p, dlogits,
                               static_cast<cudaStream_t>(stream));
}

}  // extern "C"
