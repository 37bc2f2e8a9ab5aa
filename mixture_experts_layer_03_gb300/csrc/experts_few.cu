// The experts' forward product and its dx for a handful of rows (a decode step of one or two
// tokens): y[r] = x[r] . w[e]^T and dx[r] = dy[r] . w[e], as in experts_matmul.cu.
//
// What is to be done is reading the weights of the few experts that have rows, once, with all of the
// SMs. The tensor-core kernel gives a CTA pair 256 channels and the whole contraction: with few
// experts that is a few tiles, each streamed by one pair at what its stages keep in flight. Here
// the plain FMA units, which a weight's use by at most four rows keeps well inside their rate, let
// the work be cut as finely as is wanted:
//   forward  up to eight warps share 8 channels, each an interleaved part of K, 8 elements a lane and 8
//            loads of 16 bytes in flight
//   dx       a block has 64 channels (a 128-byte line of every row of w[e]); its warps and the eight
//            blocks of its cluster share N; the blocks' sums meet through the cluster's shared memory
// Sums are in fp32, in a fixed order: the same result on every run. An expert with more than four
// rows is taken four rows at a time.
#include <cstdint>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewRows = 4;          // of an item
constexpr int kFwdChannels = 8;      // of a block
constexpr int kDxChannels = 64;
constexpr int kDxCluster = 8;
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

// Lane l of a warp has channels 8 (l % 8) .. + 7 of the block's 64 and rows n of w[e] with n = l / 8
// modulo 4 of the warp's.
template <typename T, int kRows>
__device__ __forceinline__ void dx_partial(const T* __restrict__ dy, const T* __restrict__ w,
                                           const Item& it, int c0, int n_lo, int n_hi, int N,
                                           int K, float (&acc)[kRows][8]) {
  using V = Vec<T, 16>;
  constexpr int kU = 8;                   // loads in flight a lane
  constexpr int kStep = kFewWarps * 4;    // rows of w[e] a step of the block
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = c0 + (lane & 7) * 8;
  if (c >= K) return;   // K is a multiple of 8
  const T* wp = w + static_cast<int64_t>(it.e) * N * K + c;
  for (int n0 = n_lo + warp * 4 + (lane >> 3); n0 < n_hi; n0 += kU * kStep) {
    // Rows past the end read the last one and count as zeros: a branch in here would put each
    // row's loads behind the one before.
    uint4 raw[kU];
    float d[kU][kRows];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int n = min(n0 + i * kStep, n_hi - 1);
      raw[i] = load_weights(wp + static_cast<int64_t>(n) * K);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        d[i][r] = to_f32<T>(__ldg(dy + static_cast<int64_t>(it.r0 + (r < it.rows ? r : 0)) * N + n));
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const bool in = n0 + i * kStep < n_hi;
      if (i > 0) raw[i] = in ? raw[i] : make_uint4(0, 0, 0, 0);
      float wf[8];
      V::unpack(raw[i], wf);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float f = in ? d[i][r] : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[r][j] = fmaf(f, wf[j], acc[r][j]);
      }
    }
  }
}

template <typename T, int kRows>
__device__ __forceinline__ void dx_unit(const T* __restrict__ dy, const T* __restrict__ w,
                                        const Item& it, int c0, int N, int K, int rank, int split,
                                        float* s_warp, float* s_part, T* __restrict__ dx) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float acc[kRows][8] = {};
  const int slice = (N + split - 1) / split;
  dx_partial<T, kRows>(dy, w, it, c0, rank * slice, min(N, (rank + 1) * slice), N, K, acc);
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc[r][j] += __shfl_xor_sync(0xffffffffu, acc[r][j], 8);
      acc[r][j] += __shfl_xor_sync(0xffffffffu, acc[r][j], 16);
      if (lane < 8) s_warp[(warp * kRows + r) * kDxChannels + lane * 8 + j] = acc[r][j];
    }
  __syncthreads();
  if (threadIdx.x < kRows * kDxChannels) {
    const int r = threadIdx.x / kDxChannels, ch = threadIdx.x % kDxChannels;
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < kFewWarps; ++q) sum += s_warp[q * kRows * kDxChannels + threadIdx.x];
    if (split == 1) {
      if (r < it.rows && c0 + ch < K)
        dx[static_cast<int64_t>(it.r0 + r) * K + c0 + ch] = from_f32<T>(sum);
    } else {
      s_part[threadIdx.x] = sum;
    }
  }
  if (split == 1) {
    __syncthreads();   // s_warp is read
    return;
  }
  cluster_sync();   // every block's part is there
  // Each block adds up its share of the channels over the blocks.
  const int per = kDxChannels / split;
  if (static_cast<int>(threadIdx.x) < kRows * per) {
    const int r = threadIdx.x / per, ch = rank * per + threadIdx.x % per;
    float sum = 0.0f;
    for (int b = 0; b < split; ++b)
      sum += ld_shared_cluster_f32(mapa_shared(smem_u32(s_part + r * kDxChannels + ch), b));
    if (r < it.rows && c0 + ch < K) dx[static_cast<int64_t>(it.r0 + r) * K + c0 + ch] = from_f32<T>(sum);
  }
  cluster_sync();   // s_part is read
}

// Launched in clusters of `split` blocks (1, 2, 4 or 8), which share N.
template <typename T>
__global__ void __launch_bounds__(kFewThreads, 2)
experts_few_dx_kernel(const T* __restrict__ dy, const T* __restrict__ w,
                      const int32_t* __restrict__ offsets, int R, int E, int N, int K, int split,
                      T* __restrict__ dx) {
  __shared__ int32_t s_start[257];
  __shared__ Item s_item[kMaxFew];
  __shared__ int s_count;
  __shared__ float s_warp[kFewWarps * kFewRows * kDxChannels];
  __shared__ float s_part[kFewRows * kDxChannels];
  const int rank = static_cast<int>(cluster_ctarank());
  pdl_trigger();
  pdl_wait();
  if (threadIdx.x < 32) find_items(offsets, E, R, s_start, s_item, &s_count);
  __syncthreads();
  const int blocks = (K + kDxChannels - 1) / kDxChannels;
  const int units = s_count * blocks;
  for (int u = blockIdx.x / split; u < units; u += gridDim.x / split) {
    const int i = u / blocks, c0 = (u - i * blocks) * kDxChannels;
    const Item it = s_item[i];
    if (it.e < 0) {
      const int ch = c0 + threadIdx.x;
      if (rank == 0 && threadIdx.x < kDxChannels && ch < K)
        dx[static_cast<int64_t>(it.r0) * K + ch] = from_f32<T>(0.0f);
      continue;
    }
    if (it.rows == 1) dx_unit<T, 1>(dy, w, it, c0, N, K, rank, split, s_warp, s_part, dx);
    else if (it.rows == 2) dx_unit<T, 2>(dy, w, it, c0, N, K, rank, split, s_warp, s_part, dx);
    else dx_unit<T, 4>(dy, w, it, c0, N, K, rank, split, s_warp, s_part, dx);
  }
}

template <typename T>
cudaError_t launch_few(bool dx, const void* in, const void* w, const int32_t* offsets, int R, int E,
                       int N, int K, void* out, cudaStream_t s) {
  const int sms = device_sm_count();
  if (dx) {
    const int64_t units = static_cast<int64_t>(R) * ((K + kDxChannels - 1) / kDxChannels);
    int split = 1;
    while (split < kDxCluster && units * split < 2 * sms && N >= 256 * split) split *= 2;
    const int64_t cap = 2 * sms / split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((units < cap ? units : cap) * split));
    cfg.blockDim = dim3(kFewThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, experts_few_dx_kernel<T>, static_cast<const T*>(in),
                              static_cast<const T*>(w), offsets, R, E, N, K, split,
                              static_cast<T*>(out));
  }
  // The most warps to a unit whose shares of K, in steps of 256, leave few lanes without work: K = 2280
  // over eight warps would take two steps for 1.1 (R = 2, N = 8792: 22.6 us, over two warps 16.5).
  const int64_t units = static_cast<int64_t>(R) * (N / kFwdChannels);
  auto steps = [&](int share) { return (K + 256 * share - 1) / (256 * share) * share; };
  int share = kFewWarps;
  while (share > 1 && 17 * steps(share) > 20 * steps(1)) share /= 2;
  const int64_t blocks = (units * share + kFewWarps - 1) / kFewWarps;
  const int64_t cap = 2 * sms;
  return launch_pdl(experts_few_forward_kernel<T>,
                    dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)), dim3(kFewThreads), 0, s,
                    static_cast<const T*>(in), static_cast<const T*>(w), offsets, R, E, N, K, share,
                    static_cast<T*>(out));
}

}  // namespace

// Measured against the tensor-core kernel. Forward: 8 rows over 128 experts (N = 1536, K = 2048, 50 MB
// of weights) 12.1 us against 14.3, 8 rows over 256 (N = 4096, K = 7168) 75.7 against 78.9, 5 rows of
// one (N = 136, K = 14336) 8.4 against 17; 32 rows of 8 (14336 x 4096) 234 against 142. dx is behind as soon as that kernel has a tile for most CTA pairs: 1 row
// (N = 14336, K = 4096, 16 tiles) 27 us against 59, 8 rows of 8 experts (N = 7168, K = 2048, 64
// tiles) 46 against 39; nor does it take an expert's rows twice (12 rows of one: 37 against 21).
bool experts_few(bool dx, int64_t R, int E, int K) {
  if (!dx) return R <= 16;
  return R <= kFewRows && (R < E ? R : E) * ((K + 255) / 256) < 48;
}

moe_status launch_experts_few(bool dx, const void* in, const void* w, const int32_t* offsets,
                              int64_t R, int E, int N, int K, int dtype, void* out,
                              cudaStream_t s) {
  const cudaError_t err =
      dtype == MOE_DTYPE_F16
          ? launch_few<__half>(dx, in, w, offsets, static_cast<int>(R), E, N, K, out, s)
          : launch_few<__nv_bfloat16>(dx, in, w, offsets, static_cast<int>(R), E, N, K, out, s);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "experts_few launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

}  // namespace moe
