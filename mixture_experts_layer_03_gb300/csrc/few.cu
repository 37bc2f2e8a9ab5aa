// The whole layer for a few tokens (T <= 16) in two kernels:
//   few_gate_kernel   logits = x wg^T, fp32
//   few_layer_kernel  routing, both products of the chosen experts and of the shared one, the weighted
//                     sum:  y[t] = sum over slots j of s[t, j] w2[e] (silu(g) u),  g, u = w13[e] x[t]
// For a few tokens the layer reads each chosen expert's weights once and little else: the floor is
// their bytes at the memory's rate, and what is added to it is latency, between kernels and between the
// two products. So one block an SM stays for the whole layer, and four warps of it (the weights'
// producers) keep its ring full from the moment the experts are known, on into the second products'
// weights while the first products' results are still awaited.
//
// Work. The first tickets are slices of the first products: the chosen experts' I channels one after the
// other (a channel is its gate and its up row), and the shared expert's, each cut into equal parts to
// a channel, one a block. The others are slices of the H rows of the second products, over all experts,
// one a block. A block takes tickets in order until none is left; a slice of the second products waits for
// the first ones' results, which are in blocks that run already, so that blocks that are not resident yet
// are waited for by nobody.
// Every element of h and of y is summed by one block in one order: the same result on every run.
//
// Products by mma.sync m16n8k16: 16 rows of weights by 8 tokens, so that one pass over a weight serves all
// tokens. (tcgen05's least M, 64 rows of 16-bit operands in one CTA and 128 of 4-bit ones, does not fit slices of
// some dozen rows. mma.sync takes 8 cycles an instruction on an SM quarter; a block's share of the bandwidth
// brings 16 x 16 weights of 16 bits every 84 cycles, of 4 bits every 25: it is used for a third of the time or
// less with one column tile, for a fifth with two of 16 bits and for two thirds with two of 4 bits, which is what
// nv weights and 16 tokens would need at full bandwidth and, bound by the conversions, do not reach.) All T tokens are
// columns for every expert, which keeps lists of tokens out of the loops: in the first products the others'
// results are dropped, in the second an expert's sums are added to those of its tokens only (a weight
// that is not finite reaches nobody else); the routing weight is multiplied into h.
// Four teams of two consumer warps: a team takes every fourth stage, its warps half of the stage's
// channels each, and they add up at the end of a part. (One team of eight or sixteen warps for every
// stage: a warp has more instructions beside its work than for it. More warps, fewer registers: what is
// spilled does not fit what the ring leaves of L1, and each access is one to L2.)
//
// Numbers. 16-bit weights: operands of x's type, h rounded to it once (with the routing weight; f16 after
// a power of two for each token, see below). 4-bit weights: codes to f16 exactly; nv scales
// multiplied in f16, exactly (6 significant bits, 2^-10 to 2688); mx scales, which f16 does not reach,
// by an FMA a block of 32 on its fp32 sum. x and h go to f16 times a power of two for each token
// that brings the largest to [2^14, 2^15): x of 8 or 11 significant bits is exact but for what is less
// than 2^-29 of the token's largest, h is rounded to 11 bits. The power comes off the parts' sums; so that no mx
// scale takes such a sum out of range that its result is in, scales are multiplied by the least of the
// tokens' inverse powers (see scale_unit). Sums, SwiGLU and the sum over experts: fp32.
#include <atomic>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "internal.h"
#include "launch.cuh"
#include "pairs.cuh"
#include "ptx.cuh"
#include "route_device.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kFewTokens = MOE_FEW_TOKENS;
static_assert(kFewTokens == 16, "two column tiles");
constexpr int kFewExperts = 128 + 1;             // T * k at most, and the shared one
constexpr int kMmaWarps = 8;                     // consumers
constexpr int kXWarps = 4;                       // producers of the tokens' side, a chunk each in turn
constexpr int kWWarps = 4;                       // producers of the weights' side, a stage each in turn
constexpr int kWarpW = kMmaWarps, kWarpX = kWarpW + kWWarps;
constexpr int kFewThreads = 32 * (kWarpX + kXWarps);
constexpr int kTeams = 4, kTeamWarps = kMmaWarps / kTeams;   // of consumers
constexpr int kXSlots = kXWarps;                 // chunks of the tokens' side, one a producer
static_assert(kXSlots == kTeams, "a slot belongs to the same teams throughout a part");
constexpr int kFewRows = 32;                     // rows of weights a stage
constexpr int kFewMaxBlocks = 192;
constexpr int kFewTickets = 2 * kFewMaxBlocks + 2;
constexpr int kFewSmem = 232448 - 10240;         // of a block, without the static part

enum : int { kW16b = 0, kW16h = 1, kW4mx = 2, kW4nv = 3 };   // bf16, f16, mx, nv

template <int kW>
struct FewW {
  static constexpr bool k4 = kW >= kW4mx;
  static constexpr int kChunk = k4 ? 512 : 256;                  // channels of the contraction a stage
  static constexpr int kGroups = kChunk / 32 / kTeamWarps;       // of 32 channels, a warp's part
  static constexpr int kRowBytes = k4 ? kChunk / 2 : 2 * kChunk;
  static constexpr int kPitch = k4 ? kRowBytes + 16 : kRowBytes + 64;   // (rows' parts on different banks)
  static constexpr int kScaleBytes = kW == kW4nv ? kChunk / 16 : kW == kW4mx ? kChunk / 32 : 0;
  static constexpr int kScalePitch = k4 ? 48 : 0;
  static constexpr int kStage = kFewRows * (kPitch + kScalePitch);
  static constexpr int kXPitch = 2 * kChunk + 64;
};

template <int kW, int kNt>
constexpr int few_x_bytes() { return kXSlots * 8 * kNt * FewW<kW>::kXPitch; }
template <int kNt>
constexpr int few_red_bytes() { return kMmaWarps * 2 * kNt * 512; }
// A multiple of the teams: a stage's place in the ring then belongs to one team throughout a part, which
// waits for each of its uses in turn.
template <int kW, int kNt>
constexpr int few_stages() {
  constexpr int n = (kFewSmem - 128 - few_x_bytes<kW, kNt>() - few_red_bytes<kNt>()) / FewW<kW>::kStage;
  return (n < 16 ? n : 16) / kTeams * kTeams;
}
template <int kW, int kNt>
constexpr int few_smem_bytes() {
  return 128 + few_x_bytes<kW, kNt>() + few_red_bytes<kNt>() + few_stages<kW, kNt>() * FewW<kW>::kStage;
}

struct FewMatrix {
  const uint8_t* w;        // 16-bit elements or codes
  const uint8_t* scales;
  const float* g;          // nv: of each expert, or NULL
};

struct FewArgs {
  const void* x;           // [T, H]
  FewMatrix w13, w2, w13_s, w2_s;
  const float* bias;
  moe_route_params route;
  int32_t* ids;            // [T, k]
  float* scales;
  void* y;                 // [T, H]
  int T, H, I, E, k, shared_I, shared_gate;
  int bf16;                // x, y: bf16, else f16
  // workspace
  int32_t* ticket;         // next slice; then how many channels of the first products are done
  uint32_t* tmax;          // [16] the largest |h| of each token, as bits
  float* amax;             // [16] the largest |x|
  float* logits;           // [T, E]
  float* shared_logits;    // [T]
  float* h;                // [T, k + 1, h_ld]
  int h_ld;
};

__device__ int32_t g_few_timeouts;

__device__ __forceinline__ void few_timeout(volatile int* abort) {
  *abort = 1;
  atomicOr(&g_few_timeouts, MOE_DEVICE_FLAG_TIMEOUT);
}

// ------------------------------------------------------------------ gate

constexpr int kGateThreads = 256;

template <typename T>
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  Vec<T, 16>::unpack(v, f);
}

// A block computes the logits of kPer rows of wg for kT tokens (of blockIdx.y), its warps each an eighth of H;
// blocks past those find the largest |x| of a token each.
template <typename T, int kT, int kPer>
__global__ void __launch_bounds__(kGateThreads)
few_gate_kernel(const T* __restrict__ x, const T* __restrict__ wg, int n_tok, int H, int E, int rows,
                int gate_blocks, float* __restrict__ logits, float* __restrict__ shared_logits,
                int32_t* ticket, uint32_t* tmax, float* amax) {
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nv = H / 8;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (tid < 2) ticket[tid] = 0;
    if (tid < kFewTokens) tmax[tid] = 0;
  }
  if (static_cast<int>(blockIdx.x) >= gate_blocks) {
    if (blockIdx.y != 0) return;
    __shared__ uint32_t s_max[kGateThreads / 32];
    const int t = blockIdx.x - gate_blocks;
    const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(t) * H);
    uint32_t m = 0;
    for (int v = tid; v < nv; v += kGateThreads) {
      float f[8];
      unpack8<T>(__ldg(src + v), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int i = 1; i < kGateThreads / 32; ++i) m = max(m, s_max[i]);
      amax[t] = __uint_as_float(m);
    }
    return;
  }
  __shared__ float s_sum[kGateThreads / 32][kPer][kT];
  const int e0 = blockIdx.x * kPer, t0 = blockIdx.y * kT;
  float acc[kPer][kT] = {};
#pragma unroll 2
  for (int v = tid; v < nv; v += kGateThreads) {
    float w[kPer][8];
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int e = min(e0 + p, rows - 1);
      unpack8<T>(__ldg(reinterpret_cast<const uint4*>(wg + static_cast<int64_t>(e) * H) + v), w[p]);
    }
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      float f[8];
      unpack8<T>(__ldg(reinterpret_cast<const uint4*>(x + static_cast<int64_t>(min(t0 + t, n_tok - 1)) * H) + v), f);
#pragma unroll
      for (int p = 0; p < kPer; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[p][t] = fmaf(w[p][i], f[i], acc[p][t]);
    }
  }
#pragma unroll
  for (int p = 0; p < kPer; ++p)
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      float s = acc[p][t];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      if (lane == 0) s_sum[warp][p][t] = s;
    }
  __syncthreads();
  if (tid < kPer * kT) {
    const int p = tid / kT, t = t0 + tid % kT, e = e0 + p;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kGateThreads / 32; ++i) s += s_sum[i][p][tid % kT];
    if (t < n_tok && e < rows) {
      if (e < E) logits[t * E + e] = s;
      else shared_logits[t] = s;
    }
  }
}

// ------------------------------------------------------------------ layer

// d = a (16 rows of weights, 16 channels) b (16 channels, 8 tokens) + c.
template <bool kBf16>
__device__ __forceinline__ void mma_16bit(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                          const float (&c)[4]) {
  if constexpr (kBf16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
          "f"(c[3]));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
          "f"(c[3]));
}

// 16 bytes to shared memory, the first `bytes` of them from global memory, past L1, without a register on the
// way, the others zeros.
__device__ __forceinline__ void async_load_16(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
               : "memory");
}
// One of the arrivals that `bar` counts, once this thread's copies so far are there.
__device__ __forceinline__ void async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void mbar_arrive_many(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

// mbar_wait (ptx.cuh) that leaves the polling to the hardware for up to 20 us at a time: of a block's 16 warps
// those that wait would, polling by themselves, keep the shared-memory pipe from the few that work.
__device__ __forceinline__ bool few_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  auto poll = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
  };
  if (poll()) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!poll())
    if (*abort || globaltimer_ns() - t0 > kWaitLimitNs) return false;
  return true;
}

// 2^(14 - e) for a largest value of [2^e, 2^(e + 1)), 1 for none or one that is not finite; bounded so
// that the inverse is a normal number too.
__device__ __forceinline__ float to_f16_range(float amax) {
  const uint32_t b = __float_as_uint(amax) >> 23;
  if (b == 0 || b >= 255) return 1.0f;
  const uint32_t e = 268u - b;
  return __uint_as_float((e > 253u ? 253u : e) << 23);
}
__device__ __forceinline__ float inverse_power(float p) {
  return __uint_as_float((254u << 23) - __float_as_uint(p));
}

// What mx scales are multiplied by, of the tokens' inverse powers of two (a lane each, positive): the least, so
// that a token's sums are at most what they stand for; within [2^-33, 1]. (From 2^-33 down no sum overflows: x or
// h below 2^15, codes to 6, scales to 2^127, 2^16 channels. Less would cost small scales.) The unit takes an
// instruction a row and block, which FMAs of two sums each give back but for 2 to 4% (1 token, 256 experts of
// 7168 x 2048 93.4 us without it and 95.5, 16 tokens 627 and 655; every block's sums by their token's inverse 718).
__device__ __forceinline__ float scale_unit(float inv) {
  const float least = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(inv)));
  return fminf(fmaxf(least, 0x1p-33f), 1.0f);
}

// Everything about the chosen experts that the block's warps share.
struct FewShared {
  int32_t ids[kFewTokens * kMaxTopK];
  float scales[kFewTokens * kMaxTopK];
  int sel[kFewTokens * kMaxTopK];
  float sel_l[kFewTokens * kMaxTopK];
  double e[kFewTokens * kMaxTopK];
  Pair sel_e[kFewTokens * kMaxTopK];
  float ek[kFewTokens * kMaxTopK];
  double z[kFewTokens];
  uint32_t mask[8];
  uint8_t list[kFewExperts];               // the chosen experts, ascending
  int8_t slot[kFewExperts][kFewTokens];    // of a token at a chosen expert, -1: none; last: the shared one
  uint16_t tokens[kFewExperts];            // of a chosen expert, a bit each
  float weight_s[kFewTokens];              // of the shared expert
  float x_mul[kFewTokens], x_inv[kFewTokens];
  float x_unit, h_unit[kXSlots];           // mx: of x, and of h as each producer of the tokens' side has it
  uint32_t tmax[kFewTokens];
  int n;                                   // chosen experts
};

// One token by one warp.
template <int EPL>
__device__ __noinline__ void few_select(const float* row, const FewArgs& a, int t, float* s_key,
                                        uint8_t* s_exact, uint8_t* s_list, FewShared* sh) {
  const int lane = threadIdx.x & 31;
  const PairSlots ps{sh->sel, sh->sel_l, sh->e, sh->ek, sh->z};
  const moe_route_params& r = a.route;
  int sel[kMaxTopK];
  double z = 0.0;
  if (r.method == MOE_ROUTE_GROUPED_TOPK) {
    grouped_topk_select_token<EPL>(row, a.E, a.k, r.n_group, r.topk_group, lane, s_key, sel);
  } else if (r.method == MOE_ROUTE_DEEPSEEKV3 || r.method == MOE_ROUTE_MINIMAX2) {
    const bool grouped = r.method == MOE_ROUTE_DEEPSEEKV3;
    select_token<EPL, true>(row, a.E, a.bias, r.method, a.k, grouped ? r.n_group : 1,
                            grouped ? r.topk_group : 1, lane, s_key, s_exact, s_list, sel, &z);
  } else {
    select_token<EPL, false>(row, a.E, nullptr, r.method, a.k, 1, 1, lane, s_key, s_exact, s_list, sel, &z);
    if (lane == 0) sh->z[t] = z;
  }
  record_selection(row, sel, a.k, lane, ps, t);
}

// The weights of block_pair_weights (route_device.cuh) for the methods whose slots are in order already, in
// pairs, for one rounding at the end; by one thread a slot. (In fp64, which runs at 1/64 of fp32's rate,
// the exponentials and divisions of 128 slots took every block 10 us.) False, in every thread: a logit is
// so far off that fp32's range may not do.
__device__ __forceinline__ bool few_weights(const FewArgs& a, FewShared* sh) {
  const int p = threadIdx.x, pairs = a.T * a.k, method = a.route.method;
  const bool sigmoid = method != MOE_ROUTE_DEFAULT && method != MOE_ROUTE_RENORMALIZE &&
                       method != MOE_ROUTE_RENORMALIZE_NAIVE;
  const int t = p / a.k, j = p - t * a.k;
  bool fits = method != MOE_ROUTE_GROUPED_TOPK;
  Pair e = {};
  if (p < pairs && fits) {
    const float* l = sh->sel_l + t * kMaxTopK;
    const float v = l[j];
    if (sigmoid) {
      fits = fabsf(v) <= 60.0f;
      const Pair x = pair_exp(Pair{fits ? -fabsf(v) : 0.0f, 0.0f});
      e = pair_div(v < 0.0f ? x : Pair{1.0f, 0.0f}, pair_add(Pair{1.0f, 0.0f}, x));
    } else {
      const Pair d = pair_sum(v, -l[0]);      // slot 0 has the largest logit
      fits = d.hi >= -60.0f;
      e = pair_exp(fits ? d : Pair{});
    }
    sh->sel_e[p] = e;
  }
  if (!__syncthreads_and(fits)) return false;
  if (p < pairs) {
    Pair w = e;
    if (method == MOE_ROUTE_DEFAULT) {
      const double z = sh->z[t];
      const float hi = static_cast<float>(z);
      w = pair_div(e, Pair{hi, static_cast<float>(z - static_cast<double>(hi))});
    } else if (method != MOE_ROUTE_LLAMA4) {
      Pair sum = {};
      for (int i = 0; i < a.k; ++i) sum = pair_add(sum, sh->sel_e[t * a.k + i]);
      if (method == MOE_ROUTE_DEEPSEEKV3) sum = pair_add(sum, Pair{1e-20f, 0.0f});
      w = pair_div(e, sum);
    }
    const float rsf = method == MOE_ROUTE_DEEPSEEKV3 ? a.route.routed_scaling_factor : 1.0f;
    const float product = w.hi * rsf;
    sh->ids[p] = sh->sel[t * kMaxTopK + j];
    sh->scales[p] = product + (fmaf(w.hi, rsf, -product) + w.lo * rsf);
  }
  __syncthreads();
  return true;
}

constexpr int kFewRouteBytes = 36 * 1024;        // scratch

// Routing of all tokens by the whole block, and the tables of the chosen experts.
__device__ __noinline__ void few_route(const FewArgs& a, FewShared* sh, uint8_t* scratch) {
  const int tid = threadIdx.x, warp = tid >> 5;
  constexpr int kWarps = kFewThreads / 32;
  static_assert(kWarps * (1024 + 512) <= kFewRouteBytes, "scratch");
  float* s_key = reinterpret_cast<float*>(scratch) + warp * 256;
  uint8_t* s_exact = scratch + kWarps * 1024 + warp * 512;
  for (int i = tid; i < kFewExperts * kFewTokens; i += kFewThreads) (&sh->slot[0][0])[i] = -1;
  if (tid < 8) sh->mask[tid] = 0;
  if (tid < kFewTokens) sh->tmax[tid] = 0;
  for (int t = warp; t < a.T; t += kWarps) {
    const float* row = a.logits + t * a.E;
    if (a.E <= 128) few_select<4>(row, a, t, s_key, s_exact, s_exact + 256, sh);
    else few_select<8>(row, a, t, s_key, s_exact, s_exact + 256, sh);
    __syncwarp();
  }
  __syncthreads();
  if (!few_weights(a, sh)) {
    const PairSlots ps{sh->sel, sh->sel_l, sh->e, sh->ek, sh->z};
    const int method = a.route.method;
    const float rsf = a.route.routed_scaling_factor;
    if (method == MOE_ROUTE_GROUPED_TOPK)
      block_pair_weights<2>(a.T, 0, a.T, a.k, method, rsf, ps, sh->ids, sh->scales);
    else if (method == MOE_ROUTE_DEEPSEEKV3 || method == MOE_ROUTE_MINIMAX2)
      block_pair_weights<1>(a.T, 0, a.T, a.k, method, method == MOE_ROUTE_DEEPSEEKV3 ? rsf : 1.0f, ps,
                            sh->ids, sh->scales);
    else
      block_pair_weights<0>(a.T, 0, a.T, a.k, method, 1.0f, ps, sh->ids, sh->scales);
  }
  const int pairs = a.T * a.k;
  if (tid < pairs) {
    const int e = sh->ids[tid];
    atomicOr(&sh->mask[e >> 5], 1u << (e & 31));
    if (blockIdx.x == 0) {
      a.ids[tid] = e;
      a.scales[tid] = sh->scales[tid];
    }
  }
  __syncthreads();
  if (tid < pairs) {
    // The place of expert e among the chosen ones.
    const int e = sh->ids[tid];
    int at = __popc(sh->mask[e >> 5] & ((1u << (e & 31)) - 1u));
    for (int i = 0; i < (e >> 5); ++i) at += __popc(sh->mask[i]);
    sh->list[at] = static_cast<uint8_t>(e);
    sh->slot[at][tid / a.k] = static_cast<int8_t>(tid % a.k);
  }
  if (tid == kFewThreads - 1) {
    int n = 0;
    for (int i = 0; i < 8; ++i) n += __popc(sh->mask[i]);
    sh->n = n;
  }
  __syncthreads();
  if (tid < a.T && a.shared_I > 0) {
    sh->slot[sh->n][tid] = static_cast<int8_t>(a.k);
    sh->weight_s[tid] = a.shared_gate ? 1.0f / (1.0f + expf(-a.shared_logits[tid])) : 1.0f;
  }
  __syncthreads();
  if (tid < kFewExperts) {
    uint32_t bits = 0;
    for (int t = 0; t < kFewTokens; ++t) bits |= static_cast<uint32_t>(sh->slot[tid][t] >= 0) << t;
    sh->tokens[tid] = static_cast<uint16_t>(bits);
  }
  __syncthreads();
}

// A part of a slice, as all roles walk them: its rows in 1, 2 or 4 equal subs, a stage each for every chunk
// of the contraction. Stage i of a part (chunk i / subs, sub i % subs) is team i % 4's, so that a team
// has one sub throughout a part: its sums are 8 registers a column tile, and with few rows the teams
// share out the chunks.
struct FewPart {
  int a;       // first products: place among the chosen experts (n: the shared one)
  int at;      // its first channel, or first row of y
  int n;       // channels or rows
  int subs, per;
  __device__ __forceinline__ FewPart(int a_, int at_, int n_, int most) : a(a_), at(at_), n(n_) {
    subs = n <= most ? 1 : n <= 2 * most ? 2 : 4;
    per = (n + subs - 1) / subs;
  }
  __device__ __forceinline__ int of(int sub) const { return min(per, n - sub * per); }
};

template <int kW, int kNt>
__global__ void __launch_bounds__(kFewThreads, 1) few_layer_kernel(const __grid_constant__ FewArgs a) {
  using W = FewW<kW>;
  constexpr bool kBf16 = kW == kW16b;            // the products' operands
  constexpr int kStages = few_stages<kW, kNt>();
  static_assert(kStages >= kTeams && kStages % kTeams == 0, "ring");
  static_assert(kFewRouteBytes <= kStages * W::kStage, "routing scratch");
  extern __shared__ uint8_t smem_raw[];
  __shared__ FewShared sh;
  __shared__ uint64_t w_full[kStages], w_empty[kStages], x_full[kXSlots], x_empty[kXSlots];
  __shared__ int s_ticket[kFewTickets];
  __shared__ int s_abort, s_current;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* sW = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  uint8_t* sX = sW + kStages * W::kStage;
  float* sRed = reinterpret_cast<float*>(sX + few_x_bytes<kW, kNt>());
  volatile int* abort = &s_abort;

  pdl_trigger();
  for (int i = tid; i < kFewTickets; i += kFewThreads) s_ticket[i] = -1;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&w_full[s], 32);           // a producer warp's lanes
      mbar_init(&w_empty[s], kTeamWarps);
    }
    for (int s = 0; s < kXSlots; ++s) {
      mbar_init(&x_full[s], 1);
      mbar_init(&x_empty[s], kMmaWarps);   // 4 / subs from each warp that reads it
    }
    s_abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  const int n_blocks = gridDim.x;
  // (under way while the tokens are routed)
  if (tid == 32 * kWarpW) s_ticket[0] = atomicAdd(a.ticket, 1);
  if (tid < a.T) {
    const float p = W::k4 ? to_f16_range(__ldcg(a.amax + tid)) : 1.0f;
    sh.x_mul[tid] = p;
    sh.x_inv[tid] = inverse_power(p);
  }
  if constexpr (kW == kW4mx) {
    __syncwarp();
    if (warp == 0) {
      const float unit = scale_unit(lane < a.T ? sh.x_inv[lane] : 1.0f);
      if (lane == 0) sh.x_unit = unit;
    }
  }
  few_route(a, &sh, sW);

  const int n_exp = sh.n, T = a.T, H = a.H;
  const int n_all = n_exp + (a.shared_I > 0);
  const int routed = n_exp * a.I, total = routed + a.shared_I;   // channels of the first products
  // A slice of each of the two products a block. (Four of the first a block, for experts with more tokens,
  // which take more time, to even out: 602 us became 665 for 16 tokens over 256 experts of 7168 x 2048.)
  const int n_first = n_blocks;
  const int n_tickets = n_first + n_blocks;
  // Slice `i` of the first products: channels [s0, s0 + ns) of the shared expert, then [r0, r0 + nr) of the
  // chosen ones', one after the other. Every slice has its share of the shared expert, which has all the
  // tokens and takes more time for its bytes (16 tokens, all of it in the last slices: they ended 1.7
  // times as late as the others). The second products' slice starts at row cut2(i).
  struct Slice {
    int s0, ns, r0, nr;
    __device__ __forceinline__ int size() const { return ns + nr; }
  };
  auto cut = [](int n, int i, int of) { return static_cast<int>(static_cast<int64_t>(n) * i / of); };
  auto slice1 = [&](int i) {
    const int s0 = cut(a.shared_I, i, n_first), r0 = cut(routed, i, n_first);
    return Slice{s0, cut(a.shared_I, i + 1, n_first) - s0, r0, cut(routed, i + 1, n_first) - r0};
  };
  auto cut2 = [&](int i) { return cut(H, i, n_blocks); };
  constexpr int kMost1 = kTeams * 16;
  // The part at channel z of a slice.
  auto part1 = [&](const Slice& sl, int z) {
    if (z < sl.ns) return FewPart(n_exp, sl.s0 + z, min(kMost1, sl.ns - z), 16);
    const int q = sl.r0 + z - sl.ns, at = q / a.I, ch = q - at * a.I;
    return FewPart(at, ch, min(kMost1, min(sl.size() - z, a.I - ch)), 16);
  };
  // Of the rows left, equal parts.
  auto part2 = [&](int r, int end) {
    const int left = end - r, parts = (left + kTeams * kFewRows - 1) / (kTeams * kFewRows);
    return FewPart(0, r, (left + parts - 1) / parts, kFewRows);
  };
  auto inner = [&](int at) { return at < n_exp ? a.I : a.shared_I; };   // channels of a chosen expert
  // Ticket i of this block, when it is there; n_tickets (no work) if it does not come.
  auto ticket_at = [&](int i, bool& ok) {
    const volatile int* at = &s_ticket[i];
    int v = *at;
    if (v >= 0) return v;
    const uint64_t t0 = globaltimer_ns();
    while ((v = *at) < 0) {
      if (*abort || globaltimer_ns() - t0 > kWaitLimitNs) {
        ok = false;
        return n_tickets;
      }
      __nanosleep(64);
    }
    return v;
  };

  if (warp >= kWarpW && warp < kWarpX) {
    // ------------------------------------------------------------ weights
    // Rows as they lie in memory, by 16-byte asynchronous copies of whole warps. (Bulk copies of a row each
    // are issued one lane after the other, at 30 to 60 cycles: 511 us for 4 tokens through 8 experts of
    // 4096 x 14336 in bf16, so 336.)
    const int mine = warp - kWarpW;
    int stage = 0, turn = 0;
    uint32_t phase = 0;
    bool ok = true;
    // n rows of len channels, from `row` of m and channel k0 of K on, to rows from `at` on of the stage;
    // zeros up to the chunk's end (which the products then need not know).
    auto rows = [&](const FewMatrix& m, int64_t row, int n, int at, int K, int k0, int len) {
      constexpr int kLanes = W::kRowBytes / 16, kStep = 32 / kLanes;   // lanes to a row, rows at once
      const int part = lane % kLanes, first = lane / kLanes;
      const int bytes = W::k4 ? len / 2 : len * 2;
      const int64_t pitch = W::k4 ? K / 2 : 2 * static_cast<int64_t>(K);
      const bool in = part * 16 < bytes;
      uint8_t* dst = sW + stage * W::kStage + (at + first) * W::kPitch + part * 16;
      const uint8_t* src = m.w + (row + first) * pitch + (W::k4 ? k0 / 2 : 2 * k0) + (in ? part * 16 : 0);
#pragma unroll 4
      for (int i = first; i < n; i += kStep) {
        async_load_16(dst, src, in ? 16u : 0u);
        dst += kStep * W::kPitch;
        src += kStep * pitch;
      }
      if constexpr (W::k4) {
        constexpr int kBlock = kW == kW4nv ? 16 : 32;
        constexpr int kLanesS = W::kScaleBytes / 16;   // to a row of scales
        const int sp = fp4_scale_pitch(K, kW == kW4nv ? kFp4Nv : kFp4Mx);
        const int ps = lane % kLanesS, i = lane / kLanesS;
        static_assert(32 / kLanesS >= 16, "a row each");
        uint8_t* to = sW + stage * W::kStage + kFewRows * W::kPitch + (at + i) * W::kScalePitch + ps * 16;
        // (of the row's own scales: what fills it up may be anything)
        const int left = (K - k0) / kBlock - ps * 16;
        const uint32_t there = left <= 0 ? 0u : left < 16 ? left : 16u;
        const uint8_t* from = m.scales + (row + i) * sp + k0 / kBlock + (there ? ps * 16 : 0);
        if (i < n) async_load_16(to, from, there);
        if (32 / kLanesS < kFewRows && i + 32 / kLanesS < n)
          async_load_16(to + 32 / kLanesS * W::kScalePitch, from + 32 / kLanesS * sp, there);
      }
    };
    // A stage is this warp's or another one's.
    auto begin = [&] {
      const bool is = turn == mine;
      turn = turn + 1 == kWWarps ? 0 : turn + 1;
      if (is) ok = __all_sync(0xffffffffu, few_wait(&w_empty[stage], phase ^ 1u, abort));
      return is && ok;
    };
    auto end_stage = [&](bool is) {
      if (is) async_arrive(&w_full[stage]);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    };
    for (int i = 0; ok; ++i) {
      int ticket = 0;
      if (mine == 0) {
        if (lane == 0) {
          ticket = i == 0 ? s_ticket[0] : atomicAdd(a.ticket, 1);
          *const_cast<volatile int*>(&s_ticket[i]) = ticket;
        }
      } else {
        ticket = ticket_at(i, ok);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      ticket = __shfl_sync(0xffffffffu, ticket, 0);
      if (ticket >= n_tickets) break;
      if (ticket < n_first) {
        const Slice slice = slice1(ticket);
        for (int z = 0; z < slice.size() && ok;) {
          const FewPart p = part1(slice, z);
          z += p.n;
          const bool own = p.a < n_exp;
          const FewMatrix& m = own ? a.w13 : a.w13_s;
          const int width = inner(p.a);
          const int64_t base = (own ? static_cast<int64_t>(sh.list[p.a]) * 2 * width : 0) + p.at;
          for (int k0 = 0; k0 < H && ok; k0 += W::kChunk) {
            const int len = min(W::kChunk, H - k0);
            for (int s = 0; s < p.subs && ok; ++s) {
              const bool is = begin();
              if (is) {
                rows(m, base + s * p.per, p.of(s), 0, H, k0, len);
                rows(m, base + width + s * p.per, p.of(s), 16, H, k0, len);
              }
              end_stage(is);
            }
          }
        }
      } else {
        for (int r = cut2(ticket - n_first), end = cut2(ticket - n_first + 1); r < end && ok;) {
          const FewPart p = part2(r, end);
          r += p.n;
          for (int e = 0; e < n_all && ok; ++e) {
            const bool own = e < n_exp;
            const FewMatrix& m = own ? a.w2 : a.w2_s;
            const int K = inner(e);
            const int64_t base = (own ? static_cast<int64_t>(sh.list[e]) * H : 0) + p.at;
            for (int k0 = 0; k0 < K && ok; k0 += W::kChunk)
              for (int s = 0; s < p.subs && ok; ++s) {
                const bool is = begin();
                if (is) rows(m, base + s * p.per, p.of(s), 0, K, k0, min(W::kChunk, K - k0));
                end_stage(is);
              }
          }
        }
      }
    }
    if (!ok) few_timeout(abort);
    async_wait_all();   // (nothing is under way into the memory of a block that has ended)
  } else if (warp >= kWarpX) {
    // ------------------------------------------------------------ tokens
    // Chunk after chunk goes round the four warps and their slots. Only the rows of an expert's tokens are
    // written: what the others' hold reaches columns that nobody looks at. Rows are loaded two batches
    // ahead, the first ones (mostly all) before the slot is waited for.
    const int mine = warp - kWarpX;
    uint32_t phase = 0;
    int before = 0;                         // chunks of the tickets so far, mod kXWarps
    bool ok = true, waited = false;
    float t_mul = 1.0f;                     // lane t: token t's power of two for h
    constexpr int kVecs = W::kChunk / 8, kPer = kVecs / 32;   // of 8 channels: of a row of a slot, a lane's
    uint8_t* dst = sX + mine * 8 * kNt * W::kXPitch;
    for (int i = 0; ok; ++i) {
      const int ticket = __shfl_sync(0xffffffffu, ticket_at(i, ok), 0);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok || ticket >= n_tickets) break;
      const bool fc1 = ticket < n_first;
      if (!fc1 && !waited) {
        // All of h, and each token's largest.
        ok = __all_sync(0xffffffffu, wait_count(a.ticket + 1, total, abort));
        if (!ok) break;
        waited = true;
        if (!kBf16 && lane < T) t_mul = to_f16_range(__uint_as_float(__ldcg(a.tmax + lane)));
        if (kW == kW4mx) {
          const float unit = scale_unit(inverse_power(t_mul));
          if (lane == 0) sh.h_unit[mine] = unit;
        }
      }
      // Where in the slice: the next part (from `at` on), the expert, the chunk of its contraction.
      const Slice slice = slice1(fc1 ? ticket : 0);
      const int end = fc1 ? slice.size() : cut2(ticket - n_first + 1);
      int at = fc1 ? 0 : cut2(ticket - n_first);
      int e = 0, chunk = 0, count = 0;
      bool there = at < end;
      auto enter = [&] {                    // the part at `at`
        if (fc1) {
          const FewPart p = part1(slice, at);
          at += p.n;
          e = p.a;
        } else {
          at += part2(at, end).n;
          e = 0;
        }
      };
      auto width = [&] { return fc1 ? H : inner(e); };
      auto step = [&](int by) {
        chunk += by;
        count += by;
        for (int n; there && chunk >= (n = (width() + W::kChunk - 1) / W::kChunk);) {
          chunk -= n;
          if (!fc1 && ++e < n_all) continue;
          there = at < end;
          if (there) enter();
        }
        if (!there) count -= chunk;         // (chunks past the slice's end)
      };
      if (there) {
        enter();
        step((mine - before + kXWarps) % kXWarps);
      }
      // A batch: rows of x of 4 tokens as they are, or of h in f32 of 2.
      struct Batch {
        uint4 u[4][kPer];
        uint32_t tokens;
      };
      uint32_t rest = 0;                    // tokens to load yet
      auto load = [&](Batch& b) {
        const int k0 = chunk * W::kChunk, nv = min(W::kChunk, width() - k0) / 8;
        b.tokens = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!rest || (!fc1 && j >= 2)) break;
          const int t = __ffs(rest) - 1;
          rest &= rest - 1;
          b.tokens |= 1u << t;
          if (fc1) {
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) +
                                                              static_cast<int64_t>(t) * H + k0);
#pragma unroll
            for (int h = 0; h < kPer; ++h)
              if (lane + 32 * h < nv) b.u[j][h] = __ldg(src + lane + 32 * h);
          } else {
            const uint4* src = reinterpret_cast<const uint4*>(
                a.h + (static_cast<int64_t>(t) * (a.k + 1) + sh.slot[e][t]) * a.h_ld + k0);
#pragma unroll
            for (int h = 0; h < kPer; ++h)
              if (lane + 32 * h < nv) {
                b.u[2 * (j & 1)][h] = __ldcg(src + 2 * (lane + 32 * h));
                b.u[2 * (j & 1) + 1][h] = __ldcg(src + 2 * (lane + 32 * h) + 1);
              }
          }
        }
      };
      auto store = [&](const Batch& b) {
        const int nv = min(W::kChunk, width() - chunk * W::kChunk) / 8;
        uint32_t left = b.tokens;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!left) break;
          const int t = __ffs(left) - 1;
          left &= left - 1;
          const float h_mul = __shfl_sync(0xffffffffu, t_mul, t);
          const float mul = fc1 ? sh.x_mul[t] : h_mul;
#pragma unroll
          for (int h = 0; h < kPer; ++h) {
            if (lane + 32 * h >= nv) {      // zeros up to the chunk's end
              *reinterpret_cast<uint4*>(dst + t * W::kXPitch + (lane + 32 * h) * 16) = make_uint4(0, 0, 0, 0);
              continue;
            }
            uint4 v = b.u[j][h];
            if (!fc1 || W::k4) {
              float f[8];
              if (!fc1) {
                const uint4 lo = b.u[2 * (j & 1)][h], hi = b.u[2 * (j & 1) + 1][h];
                f[0] = __uint_as_float(lo.x);
                f[1] = __uint_as_float(lo.y);
                f[2] = __uint_as_float(lo.z);
                f[3] = __uint_as_float(lo.w);
                f[4] = __uint_as_float(hi.x);
                f[5] = __uint_as_float(hi.y);
                f[6] = __uint_as_float(hi.z);
                f[7] = __uint_as_float(hi.w);
              } else if (a.bf16) {
                unpack8<__nv_bfloat16>(v, f);
              } else {
                unpack8<__half>(v, f);
              }
#pragma unroll
              for (int k = 0; k < 8; ++k) f[k] *= mul;
              if constexpr (kBf16) v = Vec<__nv_bfloat16, 16>::pack(f);
              else v = Vec<__half, 16>::pack(f);
            }
            *reinterpret_cast<uint4*>(dst + t * W::kXPitch + (lane + 32 * h) * 16) = v;
          }
        }
      };
      while (there && ok) {
        Batch one, two;
        rest = sh.tokens[e];
        load(one);
        load(two);
        ok = __all_sync(0xffffffffu, few_wait(&x_empty[mine], phase ^ 1u, abort));
        phase ^= 1u;
        if (!ok) break;
        while (one.tokens) {
          store(one);
          load(one);
          store(two);
          load(two);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&x_full[mine]);
        step(kXWarps);
      }
      before = (before + count) % kXWarps;
    }
    if (!ok) few_timeout(abort);
  } else {
    // ------------------------------------------------------------ products
    // A wait that runs out leaves the loops' course as it is (the warps meet at barriers), without further
    // waits: what is computed after it is garbage that the host hears of.
    bool ok = true;
    const int g = lane >> 2, c = lane & 3;         // of the fragments
    const int team = warp / kTeamWarps, member = warp % kTeamWarps;
    int chunks = 0;                                // of the parts before this one: the tokens' slots so far
    int first = 0;                                 // place in the ring of the part's first stage
    uint32_t first_phase = 0;

    // Stage i of the part, by its team: products of chunk `xc` (of all so far) with kTiles
    // column tiles from `tile` on, of all their columns, whoever's token is in them. kM: are there rows
    // past the first 16? (No branch inside a group: the compiler moves loads and conversions over
    // products only within one.)
    auto multiply = [&](auto m_tiles, auto n_tiles, float (&acc)[2][kNt][4], int tile, int i, int xc, int subs,
                        bool fc1) {
      constexpr int kM = decltype(m_tiles)::value, kTiles = decltype(n_tiles)::value;
      const int place = first + i, lap = place / kStages;
      const int stage = place - lap * kStages, xs = xc % kXSlots;
      const uint32_t phase = first_phase ^ (lap & 1), x_phase = xc / kXSlots & 1;
      const uint8_t* x = sX + ((xs * kNt + tile) * 8 + g) * W::kXPitch + member * W::kGroups * 64 + c * 16;
      const uint8_t* w = sW + stage * W::kStage + g * W::kPitch + member * W::kGroups * (W::k4 ? 16 : 64) +
                         c * (W::k4 ? 4 : 16);
      const uint8_t* sc = sW + stage * W::kStage + kFewRows * W::kPitch + g * W::kScalePitch +
                          member * W::kGroups * (kW == kW4nv ? 2 : 1);
      ok = ok && few_wait(&x_full[xs], x_phase, abort) && few_wait(&w_full[stage], phase, abort);
      const float unit = kW != kW4mx ? 1.0f : fc1 ? sh.x_unit : sh.h_unit[xs];
      // Rows g, g + 8, g + 16, g + 24: scales of four groups, nv as f16 pairs, mx as bytes.
      uint32_t scale[2 * kM][2] = {}, nan[2 * kM] = {};
      auto scales = [&](int k0) {
#pragma unroll
        for (int r = 0; r < 2 * kM; ++r) {
          if constexpr (kW == kW4nv) {
            const uint2 v = *reinterpret_cast<const uint2*>(sc + r * 8 * W::kScalePitch + k0 * 2);
            // this lane's block of each group
            const uint32_t of_lane = __byte_perm(v.x, v.y, c >> 1 ? 0x7531u : 0x6420u);
            asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
                "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
                : "=r"(scale[r][0]), "=r"(scale[r][1])
                : "r"(of_lane));
          } else if constexpr (kW == kW4mx) {
            const uint32_t four = *reinterpret_cast<const uint32_t*>(sc + r * 8 * W::kScalePitch + k0);
            scale[r][0] = four;
            // a byte of 255: the highest bit of a byte whose other bits carry into it
            nan[r] |= ((four & 0x7f7f7f7fu) + 0x01010101u) & four & 0x80808080u;
          }
        }
      };
      auto group = [&](int k, int of) {   // `of` the four that scales() read
        uint4 b[kTiles];
#pragma unroll
        for (int n = 0; n < kTiles; ++n) b[n] = *reinterpret_cast<const uint4*>(x + n * 8 * W::kXPitch + k * 64);
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          uint32_t p[2][4];   // rows g and g + 8 of the tile: four pairs of neighbouring channels
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint8_t* src = w + (m * 16 + r * 8) * W::kPitch;
            if constexpr (W::k4) {
              fp4_halves8(*reinterpret_cast<const uint32_t*>(src + k * 16), p[r]);
              if constexpr (kW == kW4nv) {
                const uint32_t both = of & 2 ? scale[2 * m + r][1] : scale[2 * m + r][0];
                const uint32_t twice = __byte_perm(both, 0, of & 1 ? 0x3232u : 0x1010u);
                const __half2 one = *reinterpret_cast<const __half2*>(&twice);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&p[r][j]), one);
                  p[r][j] = *reinterpret_cast<const uint32_t*>(&v);
                }
              }
            } else {
              const uint4 u = *reinterpret_cast<const uint4*>(src + k * 64);
              p[r][0] = u.x;
              p[r][1] = u.y;
              p[r][2] = u.z;
              p[r][3] = u.w;
            }
          }
          const uint32_t a0[4] = {p[0][0], p[1][0], p[0][1], p[1][1]};
          const uint32_t a1[4] = {p[0][2], p[1][2], p[0][3], p[1][3]};
          if constexpr (kW == kW4mx) {
            float f[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              // 2^(byte - 127); 2^-127, which is no normal number, as 0
              const uint32_t word = scale[2 * m + r][0];
              f[r] = __uint_as_float((of == 3 ? word >> 1 : word << (23 - 8 * of)) & 0x7f800000u) * unit;
            }
            const uint64_t by[2] = {two(f[0], f[0]), two(f[1], f[1])};
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
              const float zero[4] = {};
              float d[4], d2[4];
              // (one after the other in the same sum: a third more time)
              mma_16bit<kBf16>(d, a0, b[n].x, b[n].y, zero);
              mma_16bit<kBf16>(d2, a1, b[n].z, b[n].w, zero);
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                uint64_t sum = two(acc[m][n][2 * r], acc[m][n][2 * r + 1]);
                sum = times_plus(two(d[2 * r], d[2 * r + 1]), by[r], sum);
                sum = times_plus(two(d2[2 * r], d2[2 * r + 1]), by[r], sum);
                acc[m][n][2 * r] = moe::first(sum);
                acc[m][n][2 * r + 1] = moe::second(sum);
              }
            }
          } else {
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
              mma_16bit<kBf16>(acc[m][n], a0, b[n].x, b[n].y, acc[m][n]);
              mma_16bit<kBf16>(acc[m][n], a1, b[n].z, b[n].w, acc[m][n]);
            }
          }
        }
      };
      static_assert(W::kGroups % 4 == 0, "groups by fours");
      // (Not all unrolled, and few forms of it: the instruction cache holds the producers' code as well.)
#pragma unroll 1
      for (int k = 0; k < W::kGroups; k += 4) {
        if (W::k4) scales(k);
#pragma unroll
        for (int j = 0; j < 4; ++j) group(k + j, j);
      }
      if constexpr (kW == kW4mx) {
#pragma unroll
        for (int r = 0; r < 2 * kM; ++r)
          if (nan[r]) {
#pragma unroll
            for (int n = 0; n < kTiles; ++n)
              acc[r >> 1][n][2 * (r & 1)] = acc[r >> 1][n][2 * (r & 1) + 1] = __uint_as_float(0x7fffffffu);
          }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&w_empty[stage]);
        mbar_arrive_many(&x_empty[xs], kTeams / subs);
      }
    };
    // The warps' sums of a part meet in shared memory; then the part's stages are behind everybody.
    auto gather = [&](const float (&v)[2][kNt][4], int stages, int n_chunks) {
      named_barrier_sync(1, 32 * kMmaWarps);      // what was there has been read
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < kNt; ++n)
          *reinterpret_cast<float4*>(sRed + ((warp * 2 + m) * kNt + n) * 128 + lane * 4) =
              make_float4(v[m][n][0], v[m][n][1], v[m][n][2], v[m][n][3]);
      named_barrier_sync(1, 32 * kMmaWarps);
      chunks += n_chunks;
      const int place = first + stages, lap = place / kStages;
      first = place - lap * kStages;
      first_phase ^= lap & 1;
    };
    // Sub `s`, value (m, n, at) over the teams that had it.
    auto sum_at = [&](int subs, int s, int m, int n, int at) {
      float v = 0.0f;
      for (int t = s; t < kTeams; t += subs)
#pragma unroll
        for (int w = 0; w < kTeamWarps; ++w) v += sRed[(((t * kTeamWarps + w) * 2 + m) * kNt + n) * 128 + at];
      return v;
    };
    auto clear = [](float (&v)[2][kNt][4]) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[m][n][j] = 0.0f;
    };

    bool waited = false;
    float y_inv = 1.0f;       // lane t: inverse of token t's power of two; mx: lane 31 of the scales' unit
    for (int i = 0;; ++i) {
      if (tid == 0) s_current = ticket_at(i, ok);
      named_barrier_sync(1, 32 * kMmaWarps);
      const int ticket = s_current;
      named_barrier_sync(1, 32 * kMmaWarps);      // read by all before it is written again
      if (ticket >= n_tickets) break;
      const bool fc1 = ticket < n_first;
      const Slice slice = slice1(fc1 ? ticket : 0);
      const int from = fc1 ? 0 : cut2(ticket - n_first);
      const int end = fc1 ? slice.size() : cut2(ticket - n_first + 1);
      for (int at = from; at < end;) {
        const FewPart p = fc1 ? part1(slice, at) : part2(at, end);
        at += p.n;
        // The team's stages: sub `sub` of every 4 / subs-th chunk, over all experts in the second products.
        const int sub = team % p.subs;
        const bool second = fc1 || p.of(sub) > 16;
        float all[2][kNt][4];
        clear(all);
        int ck = 0;
        for (int e = fc1 ? p.a : 0, last = fc1 ? p.a + 1 : n_all; e < last; ++e) {
          const int K = fc1 ? H : inner(e);
          const uint32_t tokens = sh.tokens[e];
          // The column tiles that hold tokens of the expert.
          const bool both = kNt == 2 && (tokens & 0xffu) && tokens > 0xffu;
          const int tile = kNt == 2 && !(tokens & 0xffu) ? 1 : 0;
          float acc[2][kNt][4];
          clear(acc);
#pragma unroll 1
          for (int k0 = 0; k0 < K; k0 += W::kChunk, ++ck) {
            if ((ck * p.subs + sub) % kTeams != team) continue;
            const int i2 = ck * p.subs + sub, xc = chunks + ck;
            using One = std::integral_constant<int, 1>;
            using Two = std::integral_constant<int, 2>;
            if constexpr (kNt == 2) {
              if (both) {
                multiply(Two{}, Two{}, acc, 0, i2, xc, p.subs, fc1);
                continue;
              }
            }
            if (second) multiply(Two{}, One{}, acc, tile, i2, xc, p.subs, fc1);
            else multiply(One{}, One{}, acc, tile, i2, xc, p.subs, fc1);
          }
          // Sums of the expert's tokens only (in the first products, all: the rest is dropped below).
#pragma unroll
          for (int n = 0; n < kNt; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (!(tokens >> (n * 8 + 2 * c + j) & 1u)) continue;
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                const float* v = kNt == 2 && both ? acc[m][n] : acc[m][0];
                all[m][n][j] += v[j];
                all[m][n][j + 2] += v[j + 2];
              }
            }
        }
        gather(all, ck * p.subs, ck);
        if (fc1) {
          const bool own = p.a < n_exp;
          float g13 = 1.0f, g2 = 1.0f;
          if (kW == kW4nv) {
            const int e = own ? sh.list[p.a] : 0;
            const float* p13 = own ? a.w13.g : a.w13_s.g;
            const float* p2 = own ? a.w2.g : a.w2_s.g;
            if (p13) g13 = __ldg(p13 + e);
            if (p2) g2 = __ldg(p2 + e);
          }
          for (int pos = tid; pos < p.subs * kNt * 128; pos += 32 * kMmaWarps) {
            const int s = pos / (kNt * 128), n = pos / 128 % kNt, at_ = pos & 127, l = at_ >> 2, j = at_ & 3;
            const int row = (l >> 2) + 8 * (j >> 1), t = n * 8 + (l & 3) * 2 + (j & 1);
            const int sl = t < T ? sh.slot[p.a][t] : -1;
            if (sl < 0 || row >= p.of(s)) continue;
            // (one after the other: their product may be past f32's range where the sums are 0)
            const float f = sh.x_inv[t], f2 = kW == kW4mx ? 1.0f / sh.x_unit : g13;
            float gate = sum_at(p.subs, s, 0, n, at_) * f, up = sum_at(p.subs, s, 1, n, at_) * f;
            if constexpr (W::k4) {
              gate *= f2;
              up *= f2;
            }
            const float wt = own ? sh.scales[t * a.k + sl] : sh.weight_s[t];
            const float ex = expf(-fabsf(gate));
            const float sig = (gate < 0.0f ? ex : 1.0f) / (1.0f + ex);
            const float h = gate * sig * up * (wt * g2);
            a.h[(static_cast<int64_t>(t) * (a.k + 1) + sl) * a.h_ld + p.at + s * p.per + row] = h;
            if (!kBf16) atomicMax(&sh.tmax[t], __float_as_uint(h) & 0x7fffffffu);
          }
        } else {
          if (!waited) {
            // (h came through the tokens' warps, which waited for all of it)
            waited = true;
            if (!kBf16 && lane < T) y_inv = inverse_power(to_f16_range(__uint_as_float(__ldcg(a.tmax + lane))));
            if constexpr (kW == kW4mx) {
              const float unit = scale_unit(y_inv);
              if (lane == 31) y_inv = 1.0f / unit;
            }
          }
          for (int pos = tid; pos < p.subs * 2 * kNt * 128; pos += 32 * kMmaWarps) {
            const int s = pos / (2 * kNt * 128), m = pos / (kNt * 128) % 2, n = pos / 128 % kNt;
            const int at_ = pos & 127, l = at_ >> 2, j = at_ & 3;
            const int row = m * 16 + (l >> 2) + 8 * (j >> 1), t = n * 8 + (l & 3) * 2 + (j & 1);
            const float inv = __shfl_sync(0xffffffffu, y_inv, t);   // (a warp's positions come and go together)
            const float unit_inv = kW == kW4mx ? __shfl_sync(0xffffffffu, y_inv, 31) : 1.0f;
            if (t >= T || row >= p.of(s)) continue;
            float v = sum_at(p.subs, s, m, n, at_) * inv;
            if constexpr (kW == kW4mx) v *= unit_inv;
            const int64_t to = static_cast<int64_t>(t) * H + p.at + s * p.per + row;
            if (a.bf16) static_cast<__nv_bfloat16*>(a.y)[to] = __float2bfloat16_rn(v);
            else static_cast<__half*>(a.y)[to] = __float2half_rn(v);
          }
        }
      }
      if (fc1) {
        // This slice's h, and the largest so far, before the count (a release covers what the block's other
        // threads wrote before the barrier).
        named_barrier_sync(1, 32 * kMmaWarps);
        if (warp == 0 && end > from) {
          if (!kBf16 && lane < T) atomicMax(a.tmax + lane, sh.tmax[lane]);
          __syncwarp();
          if (lane == 0) red_release_gpu_add(a.ticket + 1, end - from);
        }
      }
    }
    if (!ok) few_timeout(abort);
  }
  __syncthreads();
}

// The waits of the kernel above, for a barrier that nothing arrives on and for a count that does not come: the
// first to run out ends the other.
__global__ void __launch_bounds__(64) few_wait_selftest_kernel() {
  __shared__ uint64_t bar;
  __shared__ int s_abort;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  volatile int* abort = &s_abort;
  if (threadIdx.x < 32) {
    if (!__all_sync(0xffffffffu, few_wait(&bar, 0, abort))) few_timeout(abort);
  } else {
    // Half a limit later, so that the abort flag ends it before its own limit does.
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kWaitLimitNs / 2) __nanosleep(1000000);
    if (!__all_sync(0xffffffffu, wait_count(&g_few_timeouts, INT32_MAX, abort))) few_timeout(abort);
  }
}

template <int kW, int kNt>
moe_status launch_layer(const FewArgs& a, cudaStream_t s) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return set_error(MOE_ERR_CUDA, "cudaGetDevice failed");
  constexpr int kSmem = few_smem_bytes<kW, kNt>();
  if (!ready[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(few_layer_kernel<kW, kNt>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess)
      return set_error(MOE_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    ready[dev].store(true, std::memory_order_release);
  }
  const int sms = device_sm_count();
  const cudaError_t err =
      launch_pdl(few_layer_kernel<kW, kNt>, dim3(static_cast<unsigned>(sms < kFewMaxBlocks ? sms : kFewMaxBlocks)),
                 dim3(kFewThreads), kSmem, s, a);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "few_layer launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

template <typename T, int kT, int kPer>
cudaError_t launch_gate_t(const FewArgs& a, const void* wg, bool want_amax, cudaStream_t s) {
  const int rows = a.E + a.shared_gate, blocks = (rows + kPer - 1) / kPer;
  return launch_pdl(few_gate_kernel<T, kT, kPer>,
                    dim3(static_cast<unsigned>(blocks + (want_amax ? a.T : 0)), (a.T + kT - 1) / kT),
                    dim3(kGateThreads), 0, s, static_cast<const T*>(a.x), static_cast<const T*>(wg), a.T, a.H,
                    a.E, rows, blocks, a.logits, a.shared_logits, a.ticket, a.tmax, a.amax);
}

// Blocks for about one wave, each of few rows and tokens: x and wg come from L2 again for every block, and a
// block that has all 16 tokens waits for them one after the other (16 tokens, 256 x 7168: 14 us with two
// rows by all tokens, 7 with four by four).
template <typename T>
cudaError_t launch_gate_tokens(const FewArgs& a, const void* wg, bool want_amax, cudaStream_t s) {
  const bool many = a.E + a.shared_gate > device_sm_count();
  if (a.T == 1)
    return many ? launch_gate_t<T, 1, 2>(a, wg, want_amax, s) : launch_gate_t<T, 1, 1>(a, wg, want_amax, s);
  if (a.T <= 4)
    return many ? launch_gate_t<T, 4, 2>(a, wg, want_amax, s) : launch_gate_t<T, 4, 1>(a, wg, want_amax, s);
  return launch_gate_t<T, 4, 4>(a, wg, want_amax, s);
}

size_t to_256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

moe_status few_timeout_word(void** word) {
  const cudaError_t e = cudaGetSymbolAddress(word, g_few_timeouts);
  return e == cudaSuccess ? MOE_OK
                          : set_error(MOE_ERR_CUDA, "cudaGetSymbolAddress: %s", cudaGetErrorString(e));
}

moe_status launch_few_wait_selftest(cudaStream_t s) {
  few_wait_selftest_kernel<<<1, 64, 0, s>>>();
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MOE_OK
                          : set_error(MOE_ERR_CUDA, "self-test launch: %s", cudaGetErrorString(e));
}

size_t few_workspace_bytes(const moe_problem& p) {
  const size_t h_ld = p.I > p.shared_I ? p.I : p.shared_I;
  return 256 + to_256(4 * static_cast<size_t>(p.T) * p.E) + 256 + 4 * static_cast<size_t>(p.T) * (p.k + 1) * h_ld;
}

moe_status launch_few(const moe_problem& p, const FewLayer& f, char* ws, cudaStream_t s) {
  auto matrix = [](const moe_weights* w) {
    return w ? FewMatrix{static_cast<const uint8_t*>(w->w), w->scales, w->g} : FewMatrix{};
  };
  FewArgs a = {};
  a.x = f.x;
  a.w13 = matrix(f.w13);
  a.w2 = matrix(f.w2);
  a.w13_s = matrix(f.w13_s);
  a.w2_s = matrix(f.w2_s);
  a.bias = f.bias;
  a.route = f.route;
  a.ids = f.ids;
  a.scales = f.scales;
  a.y = f.y;
  a.T = static_cast<int>(p.T);
  a.H = p.H;
  a.I = p.I;
  a.E = p.E;
  a.k = p.k;
  a.shared_I = p.shared_I;
  a.shared_gate = f.shared_gate;
  a.bf16 = f.dtype == MOE_DTYPE_BF16;
  a.ticket = reinterpret_cast<int32_t*>(ws);
  a.tmax = reinterpret_cast<uint32_t*>(ws + 64);
  a.amax = reinterpret_cast<float*>(ws + 128);
  a.logits = reinterpret_cast<float*>(ws + 256);
  char* after = ws + 256 + to_256(4 * static_cast<size_t>(p.T) * p.E);
  a.shared_logits = reinterpret_cast<float*>(after);
  a.h = reinterpret_cast<float*>(after + 256);
  a.h_ld = p.I > p.shared_I ? p.I : p.shared_I;
  const bool four = f.weights != MOE_WEIGHTS_16BIT;
  const cudaError_t err = a.bf16 ? launch_gate_tokens<__nv_bfloat16>(a, f.wg, four, s)
                                 : launch_gate_tokens<__half>(a, f.wg, four, s);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "few_gate launch: %s", cudaGetErrorString(err));
  const bool wide = p.T > 8;
  switch (f.weights) {
    case MOE_FP4_MX:
      return wide ? launch_layer<kW4mx, 2>(a, s) : launch_layer<kW4mx, 1>(a, s);
    case MOE_FP4_NV:
      return wide ? launch_layer<kW4nv, 2>(a, s) : launch_layer<kW4nv, 1>(a, s);
    default:
      if (a.bf16) return wide ? launch_layer<kW16b, 2>(a, s) : launch_layer<kW16b, 1>(a, s);
      return wide ? launch_layer<kW16h, 2>(a, s) : launch_layer<kW16h, 1>(a, s);
  }
}

}  // namespace moe
