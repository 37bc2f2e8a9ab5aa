// The experts' forward product for a handful of rows (a decode step of one or two tokens): y[r] =
// x[r] . w[e]^T, as in experts_matmul.cu.
//
// What is to be done is reading the weights of the few experts that have rows, once, with all of the
// SMs. The tensor-core kernel gives a CTA pair 256 channels and the whole contraction (or an eighth
// of it): with few experts that is a few tiles, each streamed by one pair at what its stages keep in
// flight. Here the plain FMA units, which a weight's use by at most four rows keeps well inside their
// rate, let the work be cut as finely as is wanted: up to eight warps share 8 channels, each an
// interleaved part of K, 8 elements a lane and 8 loads of 16 bytes in flight. (dx, whose weights lie
// across the contraction, gained nothing from such a kernel over the tensor-core one in parts: 1 row,
// N = 14336, K = 4096, 27 us against 24.)
// Sums are in fp32, in a fixed order: the same result on every run. An expert with more than four rows
// is taken four rows at a time.
#include <cstdint>

#include "internal.h"
#include "launch.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewRows = 4;          // of an item
constexpr int kFwdChannels = 8;      // of a unit
constexpr int kMaxFew = 32;          // rows of a call

// Up to four neighbouring rows of one expert, or one row of none (e < 0).
struct Item {
  int32_t e, r0, rows;
};

// The items of the call, by the first warp: a lane looks its row's expert up (offsets kept inside
// [0, R] and in order), and the first of every four rows of an expert starts an item.
__device__ __forceinline__ void find_items(const int32_t* offsets, int E, int R, int32_t* s_start,
                                           Item* s_item, int* s_count) {
  const int lane = threadIdx.x & 31;
  constexpr int kPer = 9;   // 32 * 9 > 257 offsets
  int start[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = lane * kPer + i;
    start[i] = g <= E ? min(max(offsets[g], 0), R) : R;
    if (i > 0) start[i] = max(start[i], start[i - 1]);
  }
  int most = start[kPer - 1];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, most, off);
    if (lane >= off) most = max(most, o);
  }
  most = __shfl_up_sync(0xffffffffu, most, 1);
  if (lane == 0) most = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = lane * kPer + i;
    if (g <= E) s_start[g] = max(start[i], most);
  }
  __syncwarp();
  // The last offset that is not past this row.
  int lo = -1, hi = E + 1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_start[mid] <= lane) lo = mid;
    else hi = mid;
  }
  const bool mine = lane < R;
  const int e = lo >= 0 && lo < E ? lo : -1;
  const int first = e >= 0 ? s_start[e] : lane;
  const bool head = mine && (lane - first) % kFewRows == 0;
  const uint32_t heads = __ballot_sync(0xffffffffu, head);
  if (head) {
    const int end = e >= 0 ? s_start[e + 1] : lane + 1;
    s_item[__popc(heads & ((1u << lane) - 1u))] = Item{e, lane, min(kFewRows, end - lane)};
  }
  if (lane == 0) *s_count = __popc(heads);
}

// A weight vector is read once: past L1.
__device__ __forceinline__ uint4 load_weights(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The sums of 8 channels over this warp's part of K: every `share`-th 256 elements from the sub-th on.
// Lane l < 8 gets channel l's.
template <typename T, int kRows>
__device__ __forceinline__ void forward_partial(const T* __restrict__ x, const T* __restrict__ wp,
                                                const Item& it, int K, int sub, int share,
                                                float (&sum)[kFewRows]) {
  using V = Vec<T, 16>;
  const int lane = threadIdx.x & 31;
  float acc[kRows][kFwdChannels] = {};
  for (int k = (sub * 32 + lane) * 8; k < K; k += share * 256) {
    uint4 raw[kFwdChannels];
#pragma unroll
    for (int c = 0; c < kFwdChannels; ++c) raw[c] = load_weights(wp + static_cast<int64_t>(c) * K + k);
    float xf[kRows][8];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      V::unpack(__ldg(reinterpret_cast<const uint4*>(
                    x + static_cast<int64_t>(it.r0 + (r < it.rows ? r : 0)) * K + k)), xf[r]);
#pragma unroll
    for (int c = 0; c < kFwdChannels; ++c) {
      float wf[8];
      V::unpack(raw[c], wf);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[r][c] = fmaf(xf[r][i], wf[i], acc[r][c]);
    }
  }
  // Over the lanes: at each of three steps a lane keeps half of the channels, and in the last two
  // all lanes that hold the same channel add up.
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = acc[r][c];
#pragma unroll
    for (int n = 4; n >= 1; n >>= 1) {
      const bool up = lane & n;
#pragma unroll
      for (int c = 0; c < n; ++c) {
        const float give = up ? v[c] : v[c + n];
        const float keep = up ? v[c + n] : v[c];
        v[c] = keep + __shfl_xor_sync(0xffffffffu, give, n);
      }
    }
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 8);
    sum[r] = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
  }
}

// `share` warps (1, 2, 4 or 8) to a unit of 8 channels of an item, 8 / share units to a block.
template <typename T>
__global__ void __launch_bounds__(kFewThreads, 2)
experts_few_forward_kernel(const T* __restrict__ x, const T* __restrict__ w,
                           const int32_t* __restrict__ offsets, int R, int E, int N, int K,
                           int share, T* __restrict__ y) {
  __shared__ int32_t s_start[257];
  __shared__ Item s_item[kMaxFew];
  __shared__ int s_count;
  __shared__ float s_sum[2][kFewWarps][kFewRows][kFwdChannels];
  pdl_trigger();
  pdl_wait();
  if (threadIdx.x < 32) find_items(offsets, E, R, s_start, s_item, &s_count);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int at_once = kFewWarps / share, mine = warp / share, sub = warp - mine * share;
  const int blocks = N / kFwdChannels;   // N is a multiple of 8
  const int units = s_count * blocks;
  int turn = 0;
  for (int u0 = blockIdx.x * at_once; u0 < units; u0 += gridDim.x * at_once) {
    const int u = u0 + mine;
    const bool live = u < units;
    const int i = live ? u / blocks : 0, c0 = live ? (u - i * blocks) * kFwdChannels : 0;
    const Item it = s_item[i];
    float sum[kFewRows] = {};
    if (live && it.e >= 0) {
      const T* wp = w + (static_cast<int64_t>(it.e) * N + c0) * K;
      if (it.rows == 1) forward_partial<T, 1>(x, wp, it, K, sub, share, sum);
      else if (it.rows == 2) forward_partial<T, 2>(x, wp, it, K, sub, share, sum);
      else forward_partial<T, 4>(x, wp, it, K, sub, share, sum);
    }
    // Lane l of a unit's first warp then has row l / 8, channel l % 8. Two sets of sums in turn: who
    // writes one has passed the barrier that its readers reach after reading.
    if (lane < 8)
#pragma unroll
      for (int r = 0; r < kFewRows; ++r)
        if (r < it.rows) s_sum[turn][warp][r][lane] = sum[r];
    if (share > 1) __syncthreads();
    else __syncwarp();
    const int r = lane >> 3, c = lane & 7;
    if (live && sub == 0 && r < it.rows) {
      float total = 0.0f;
      for (int q = 0; q < share; ++q) total += s_sum[turn][warp + q][r][c];
      y[static_cast<int64_t>(it.r0 + r) * N + c0 + c] = from_f32<T>(total);
    }
    turn ^= 1;
  }
}

template <typename T>
cudaError_t launch_few(const void* x, const void* w, const int32_t* offsets, int R, int E, int N,
                       int K, void* y, cudaStream_t s) {
  // The most warps to a unit whose shares of K, in steps of 256, leave few lanes without work: K = 2280
  // over eight warps would take two steps for 1.1 (R = 2, N = 8792: 22.6 us, over two warps 16.5).
  const int64_t units = static_cast<int64_t>(R) * (N / kFwdChannels);
  auto steps = [&](int share) { return (K + 256 * share - 1) / (256 * share) * share; };
  int share = kFewWarps;
  while (share > 1 && 17 * steps(share) > 20 * steps(1)) share /= 2;
  const int64_t blocks = (units * share + kFewWarps - 1) / kFewWarps;
  const int64_t cap = 2 * device_sm_count();
  return launch_pdl(experts_few_forward_kernel<T>,
                    dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)), dim3(kFewThreads), 0, s,
                    static_cast<const T*>(x), static_cast<const T*>(w), offsets, R, E, N, K, share,
                    static_cast<T*>(y));
}

}  // namespace

// A rule on the rows and experts, which is what the host knows: where the rows are, it does not. Against
// the tensor-core kernel, us:
//                                       9 rows         12 rows        16 rows
//   of 128 experts, 1536 x 2048, spread 14.0 | 13.9    16.6 | 15.9    21.8 | 24.6
//                           all of one  6.7 | 11.7     6.9 | 11.7     8.9 | 11.7
//   of 8 experts, 4096 x 4096, spread   35 | 44        39 | 42        47 | 45
//                           all of one  20.4 | 19.9    22.5 | 19.9    28.5 | 19.9
//   of 8 experts, 14336 x 4096, spread  110 | 107      126 | 114      152 | 130
//                           all of one  69 | 25        76 | 25        99 | 25
// and 2 rows over those 14336 x 4096 40 | 45, of one 22.9 | 24.2, 8 rows 106 | 104 and 52 | 24. Rows of one
// expert of large weights, which are read once for every four rows, are what it decides wrongly. Few
// experts: 5 rows of one (N = 136, K = 14336) 8.5 | 12.5, 12 of one (4096 x 4096) 22 | 13; 32 rows of 8
// (14336 x 4096) 234 | 145.
bool experts_few(int64_t R, int E) { return R <= 16 && R <= 8 * E; }

moe_status launch_experts_few(const void* x, const void* w, const int32_t* offsets, int64_t R, int E,
                              int N, int K, int dtype, void* y, cudaStream_t s) {
  const cudaError_t err =
      dtype == MOE_DTYPE_F16
          ? launch_few<__half>(x, w, offsets, static_cast<int>(R), E, N, K, y, s)
          : launch_few<__nv_bfloat16>(x, w, offsets, static_cast<int>(R), E, N, K, y, s);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "experts_few launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

}  // namespace moe
