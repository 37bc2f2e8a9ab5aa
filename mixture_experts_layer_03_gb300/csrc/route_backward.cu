// Gradient of the routing weights to the router's logits, for every method of moe_route.
//
// With C the chosen slots of a token (ids in [0, E); others take no part), ds their gradients:
//   softmax over all E (Default)     p = softmax(l):       dl_e = p_e (sum_{j: id_j = e} ds_j - sum_j ds_j p_{id_j})
//   softmax over the chosen          a = softmax(l_C):     dl_j = a_j (ds_j - sum_i ds_i a_i)
//   sigmoid over the chosen's sum    a = sigma(l_C), D = sum a + eps:
//                                    dl_j = c (ds_j - sum_i ds_i a_i / D) / D * a_j (1 - a_j)
//   sigmoid                          dl_j = ds_j a_j (1 - a_j)
// and 0 for every expert that is not chosen (but under Default). The selection itself has no
// gradient, so the selection bias takes no part. Non-finite logits count as -inf, as in
// moe_route: their weight and their gradient are 0.
//
// One warp per token: lanes 0..k-1 hold a slot each, then every lane writes its experts' entries
// (the slots' values passed round by shuffles). The [T, E] result is most of the traffic: 8192
// tokens, 256 experts, k = 8 (9.2 MB) take 4.6 us, of which about two are a launch's.
#include <cstdint>

#include "internal.h"
#include "launch.cuh"

namespace moe {
namespace {

constexpr int kGradThreads = 256;
constexpr int kSlots = 8;
constexpr float kFarBelow = -20.0f;

enum : int { kSoftmaxAll, kSoftmaxChosen, kSigmoidSum, kSigmoidEach };

__device__ __forceinline__ float sum_warp(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float max_warp(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

__device__ __forceinline__ float finite_or_low(float l) { return isfinite(l) ? l : -INFINITY; }

template <int kForm>
__global__ void __launch_bounds__(kGradThreads)
route_grad_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                  const float* __restrict__ ds, int64_t T, int E, int k, float c, float eps,
                  float* __restrict__ dl) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kGradThreads / 32);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kGradThreads / 32) + (threadIdx.x >> 5);
       t < T; t += warps) {
    const float* row = logits + t * E;
    int id = -1;
    float d = 0.0f, l = -INFINITY;
    if (lane < k) {
      id = __ldg(ids + t * k + lane);
      if (id < 0 || id >= E) id = -1;
      if (id >= 0) {
        d = __ldg(ds + t * k + lane);
        l = finite_or_low(__ldg(row + id));
        if (l == -INFINITY) d = 0.0f;   // its weight is 0 whatever the logit
      }
    }
    float p[kSlots], common = 0.0f;   // Default: this lane's probabilities and sum_j ds_j p_j
    if (kForm == kSoftmaxAll) {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const int e = lane + 32 * i;
        p[i] = e < E ? finite_or_low(__ldg(row + e)) : -INFINITY;
        m = fmaxf(m, p[i]);
      }
      m = max_warp(m);
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        p[i] = p[i] == -INFINITY ? 0.0f : expf(p[i] - m);
        z += p[i];
      }
      z = sum_warp(z);
      const float inv = z > 0.0f ? 1.0f / z : 0.0f;   // no finite logit: every gradient is 0
#pragma unroll
      for (int i = 0; i < kSlots; ++i) p[i] *= inv;
      common = sum_warp(id >= 0 && l != -INFINITY ? d * (expf(l - m) * inv) : 0.0f);
    } else {
      const bool live = id >= 0 && l != -INFINITY;
      if (kForm == kSoftmaxChosen) {
        const float m = max_warp(l);
        const float ex = live ? expf(l - m) : 0.0f;
        const float z = sum_warp(ex);
        const float a = z > 0.0f ? ex / z : 0.0f;
        d = a * (d - sum_warp(d * a));
      } else {
        // sigma(l) (1 - sigma(l)) from exp(-|l|): no cancellation at either end
        const float ex = live ? expf(-fabsf(l)) : 0.0f;
        const float r = 1.0f / (1.0f + ex);
        float slope = ex * r * r;
        if (kForm == kSigmoidSum) {
          if (__any_sync(0xffffffffu, live && l > kFarBelow)) {
            // Where one weight is nearly the sum, d less its share cancels: sigma and the share are rounded
            // as few times as can be (far below, where exp(-l) ends, sigma is exp(l)).
            const float a = !live ? 0.0f : l > -80.0f ? 1.0f / (1.0f + expf(-l)) : ex * r;
            const float sum = sum_warp(a) + eps;
            d = sum > 0.0f ? c * (d - sum_warp(d * a) / sum) / sum : 0.0f;
          } else {
            // Every chosen logit far below zero: sigma(l) = exp(l) and 1 - sigma(l) = 1 to 2^-28. The
            // sigmoids and 1 / sum leave the range of 32 bits (from -88 on), the weights do not: they
            // are taken from exp(l - max), eps by exp(-max) in two factors.
            const float m = max_warp(l);
            const float e = live ? expf(l - m) : 0.0f;
            const float half = expf(-0.5f * m);
            const float w = e / (sum_warp(e) + (eps > 0.0f ? eps * half * half : 0.0f));
            d = c * (d - sum_warp(d * w));
            slope = w;
          }
        }
        d *= slope;
      }
      if (!live) d = 0.0f;
    }
    float out[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) out[i] = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int ej = __shfl_sync(0xffffffffu, id, j);
      const float dj = __shfl_sync(0xffffffffu, d, j);
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        if (ej == lane + 32 * i) out[i] += dj;
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int e = lane + 32 * i;
      if (e < E) dl[t * E + e] = kForm == kSoftmaxAll ? p[i] * (out[i] - common) : out[i];
    }
  }
}

}  // namespace

moe_status launch_route_backward(const float* logits, const int32_t* ids, const float* ds,
                                 int64_t T, const moe_route_params& p, float* dl,
                                 cudaStream_t s) {
  const int64_t blocks = (T + kGradThreads / 32 - 1) / (kGradThreads / 32);
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 8;
  const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap)), block(kGradThreads);
  const int E = p.num_experts, k = p.top_k;
  cudaError_t err;
  switch (p.method) {
    case MOE_ROUTE_DEFAULT:
      err = launch_pdl(route_grad_kernel<kSoftmaxAll>, grid, block, 0, s, logits, ids, ds, T, E, k,
                       1.0f, 0.0f, dl);
      break;
    case MOE_ROUTE_RENORMALIZE:
    case MOE_ROUTE_RENORMALIZE_NAIVE:
      err = launch_pdl(route_grad_kernel<kSoftmaxChosen>, grid, block, 0, s, logits, ids, ds, T, E,
                       k, 1.0f, 0.0f, dl);
      break;
    case MOE_ROUTE_LLAMA4:
      err = launch_pdl(route_grad_kernel<kSigmoidEach>, grid, block, 0, s, logits, ids, ds, T, E,
                       k, 1.0f, 0.0f, dl);
      break;
    default: {
      // The factor and the 1e-20 as moe_route applies them.
      const bool factor = p.method == MOE_ROUTE_DEEPSEEKV3 || p.method == MOE_ROUTE_GROUPED_TOPK;
      err = launch_pdl(route_grad_kernel<kSigmoidSum>, grid, block, 0, s, logits, ids, ds, T, E, k,
                       factor ? p.routed_scaling_factor : 1.0f,
                       p.method == MOE_ROUTE_DEEPSEEKV3 ? 1e-20f : 0.0f, dl);
      break;
    }
  }
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "route_backward launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

}  // namespace moe
