// Rows sorted by expert and back, with the routing weights applied, and the gradients.
//
// With f = t*k + j the flat (token, slot) index, the rows of the sorted order are the slots
// sorted stably by expert, dropped slots (id -1, or out of range) last:
//   place(f)        the row of slot f;  inv[f] = place(f), or ~place(f) for a dropped slot
//   dispatch        x_perm[place(f)] = x[f / k], zero for a dropped slot
//   combine         y[t] = sum_j s[t,j] rows[inv[t,j]] over the kept slots
//   combine grad    drows[place(f)] = s[f] dy[t] (zero when dropped), ds[f] = <dy[t], rows[inv[f]]>
//   dispatch grad   dx[t] = sum_j dx_perm[inv[t,j]] over the kept slots
// Every row of a [T*k, H] result is written exactly once, so nothing needs clearing first. All
// four are bound by memory: each row is read and written once, token-major, so that the one
// token row a dispatch reads (or a combine writes) crosses HBM once and not k times. Sums run
// in fp32 in slot order, by one thread: no atomics, the same result on every run.
// Measured (bf16): dispatch and combine of 8192 x 4096, k = 4, 61 and 53 us (5.5 and 6.4 TB/s); the
// gradients of 8192 x 7168, k = 8, 291 and 162 us (6.9 and 6.5 TB/s, as fast as a copy). A decode
// batch (64 x 2048, k = 8) takes 3.3 and 2.8 us, which is a launch's.
#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "launch.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
// The most blocks that the tokens are cut into, and the scan's threads, one a block. Four are resident on
// an SM: a second wave fills in where the first ones' copies end, which pays where the copies are long
// (8192 x 4096 bf16 to four rows each 61.5 us, with one wave 64.9), while those of up to kOneWaveBytes
// are cut for one wave (1000 x 101 bf16 to eight rows each 8.0 us, with 1000 blocks 11.4; 8192 x 64 10.8
// and 12.1).
constexpr int64_t kOneWaveBytes = 16 << 20;
constexpr int kBlocksPerSm = 4;
constexpr int kMaxBlocks = 1024;
constexpr int kScanThreads = kMaxBlocks;
constexpr int kMaxBins = 257;        // up to 256 experts, then the dropped slots

// The expert bin of an id: [0, E), or E for a dropped slot.
__device__ __forceinline__ int bin_of(int id, int E) { return id >= 0 && id < E ? id : E; }

struct SortArgs {
  const int32_t* ids;
  int64_t T;
  int64_t P;
  int E;
  int k;
  int nb;               // blocks; block b sorts and copies the tokens [b * chunk, +chunk)
  int64_t chunk;
  int32_t* hist;        // [E + 2][nb]: per bin and block; then the blocks' bad-id flags
  int32_t* totals;      // [E]
  int32_t* inv;
  int32_t* offsets;
  int32_t* status;      // NULL (one launch only): no flag
};

// Slots per bin of each block's tokens, and whether an id is neither -1 nor in [0, E).
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a) {
  __shared__ int32_t h[kMaxBins];
  __shared__ int s_bad;
  pdl_trigger();
  for (int e = threadIdx.x; e <= a.E; e += kSortThreads) h[e] = 0;
  if (threadIdx.x == 0) s_bad = 0;
  pdl_wait();
  __syncthreads();
  const int64_t f0 = a.chunk * blockIdx.x * a.k;
  const int64_t f1 = min(a.P, f0 + a.chunk * a.k);
  for (int64_t f = f0 + threadIdx.x; f < f1; f += kSortThreads) {
    const int id = a.ids[f];
    if (id < -1 || id >= a.E) s_bad = 1;
    atomicAdd(&h[bin_of(id, a.E)], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= a.E; e += kSortThreads)
    a.hist[static_cast<int64_t>(e) * a.nb + blockIdx.x] = h[e];
  if (threadIdx.x == 0) a.hist[static_cast<int64_t>(a.E + 1) * a.nb + blockIdx.x] = s_bad;
}

// Block-wide exclusive scan of one value a thread; *total receives the sum.
template <int kWarps>
__device__ int scan_block(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  *total = all;
  return before + incl - v;
}

// One block per bin, one thread per block of tokens: the exclusive scan of the bin's counts, in
// place, and its total. The last block turns the blocks' flags into the status word. (A warp per
// bin, 32 counts after the other, took 8 us of a dispatch of 32768 slots.)
__global__ void __launch_bounds__(kScanThreads) sort_scan_kernel(SortArgs a) {
  __shared__ int s_warp[kScanThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int e = blockIdx.x;
  int32_t* row = a.hist + static_cast<int64_t>(e) * a.nb;
  const bool mine = static_cast<int>(threadIdx.x) < a.nb;
  int total;
  const int before = scan_block<kScanThreads / 32>(mine ? row[threadIdx.x] : 0, s_warp, &total);
  if (e <= a.E) {
    if (mine) row[threadIdx.x] = before;
    if (e < a.E && threadIdx.x == 0) a.totals[e] = total;
  } else if (threadIdx.x < 4) {
    a.status[threadIdx.x] = threadIdx.x == 0 && total ? MOE_DEVICE_FLAG_BAD_ID : 0;
  }
}

// How a block copies token rows: a group of 32..256 threads takes a token, each thread up to kQ vectors
// of it at a time, a group apart.
__device__ __forceinline__ int group_of(int n) {
  return n > 128 ? 256 : n > 64 ? 128 : n > 32 ? 64 : 32;
}

template <int kBytes>
struct RowCopy {
  using Raw = uint4;
  static_assert(kBytes == 16);
  static constexpr int kQ = 4;
  __device__ __forceinline__ static int group(int nvec) { return group_of(nvec); }
  __device__ __forceinline__ static int first(int in_group) { return in_group; }
  __device__ __forceinline__ static void load(Raw (&val)[kQ], const char* row, int v, int g, int nvec) {
    const Raw* src = reinterpret_cast<const Raw*>(row);
#pragma unroll
    for (int q = 0; q < kQ; ++q)
      if (v + q * g < nvec) val[q] = __ldg(src + v + q * g);
  }
  // The same vectors to row p of x_perm, or zeros to row ~p (a dropped slot).
  __device__ __forceinline__ static void store(const Raw (&val)[kQ], char* x_perm, int32_t p, int v,
                                               int g, int nvec) {
    Raw* d = reinterpret_cast<Raw*>(x_perm + static_cast<int64_t>(p < 0 ? ~p : p) * nvec * kBytes);
    const Raw zero{};
#pragma unroll
    for (int q = 0; q < kQ; ++q)
      if (v + q * g < nvec) __stcs(d + v + q * g, p < 0 ? zero : val[q]);
  }
};

// Narrower vectors, whose copies have instructions to save: a thread's lie 32 apart, so that one address
// and constants reach them, and are not checked one by one where all exist. (4096 tokens to six rows
// each of 7167 bf16 97 us, of 7164 81; in the form above 156 and 85. What is left at 7167 is neither
// instructions, 27% of the issue slots, nor bandwidth, 51% of the DRAM's: waiting, with 16 bytes a thread
// under way at a time.)
template <int kBytes>
struct NarrowCopy {
  using Raw = typename RawVec<kBytes>::type;
  static constexpr int kQ = 8;
  __device__ __forceinline__ static int group(int nvec) { return group_of((nvec + kQ - 1) / kQ); }
  __device__ __forceinline__ static int first(int in_group) {
    return (in_group & ~31) * kQ + (in_group & 31);
  }
  __device__ __forceinline__ static void load(Raw (&val)[kQ], const char* row, int v, int, int nvec) {
    const Raw* src = reinterpret_cast<const Raw*>(row) + v;
    if (v + (kQ - 1) * 32 < nvec) {
#pragma unroll
      for (int q = 0; q < kQ; ++q) val[q] = __ldg(src + q * 32);
    } else {
#pragma unroll
      for (int q = 0; q < kQ; ++q)
        if (v + q * 32 < nvec) val[q] = __ldg(src + q * 32);
    }
  }
  __device__ __forceinline__ static void store(const Raw (&val)[kQ], char* x_perm, int32_t p, int v,
                                               int, int nvec) {
    Raw* d = reinterpret_cast<Raw*>(x_perm) + static_cast<int64_t>(p < 0 ? ~p : p) * nvec + v;
    const Raw zero{};
    if (p >= 0 && v + (kQ - 1) * 32 < nvec) {
#pragma unroll
      for (int q = 0; q < kQ; ++q) __stcs(d + q * 32, val[q]);
    } else {
#pragma unroll
      for (int q = 0; q < kQ; ++q)
        if (v + q * 32 < nvec) __stcs(d + q * 32, p < 0 ? zero : val[q]);
    }
  }
};
template <>
struct RowCopy<8> : NarrowCopy<8> {};
template <>
struct RowCopy<4> : NarrowCopy<4> {};
template <>
struct RowCopy<2> : NarrowCopy<2> {};

// Places of a block's slots and the copy of their rows. kSelfCount: every block counts all
// ids itself, and nothing ran before it; else the scan kernel left each block its first place
// in every bin. A sub-chunk of whole tokens (at most one slot a thread) is ranked, published
// and copied at a time; what each thread copies first is on its way while the places are found.
template <int kBytes, bool kSelfCount>
__global__ void __launch_bounds__(kSortThreads)
sort_place_kernel(SortArgs a, const char* __restrict__ x, char* __restrict__ x_perm, int nvec) {
  __shared__ int32_t s_run[kMaxBins];                       // next free place per bin
  __shared__ int32_t s_cnt[kSelfCount ? 2 : 1][kMaxBins];   // slots before this block, and from it on
  __shared__ int32_t s_wcnt[kSortWarps][kMaxBins];          // slots per (warp, bin) of a sub-chunk
  __shared__ int32_t s_dst[kSortThreads];
  __shared__ int s_warp[kSortWarps];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t_first = a.chunk * blockIdx.x;
  const int64_t t_last = min(a.T, t_first + a.chunk);
  const int64_t row_bytes = static_cast<int64_t>(nvec) * kBytes;
  using Copy = RowCopy<kBytes>;
  const int g = Copy::group(nvec), first = Copy::first(tid & (g - 1)), my_token = tid / g;
  pdl_trigger();
  for (int i = tid; i < kSortWarps * kMaxBins; i += kSortThreads) (&s_wcnt[0][0])[i] = 0;
  if (kSelfCount) {
    for (int e = tid; e <= a.E; e += kSortThreads) s_cnt[0][e] = s_cnt[1][e] = 0;
    if (tid == 0) s_bad = 0;
    __syncthreads();
  }
  pdl_wait();
  typename Copy::Raw val[Copy::kQ];
  if (t_first + my_token < t_last)
    Copy::load(val, x + (t_first + my_token) * row_bytes, first, g, nvec);
  int total;
  if (kSelfCount) {
    const int P = static_cast<int>(a.P), f_first = static_cast<int>(t_first) * a.k;
    auto count = [&](int f, int id) {
      if (id < -1 || id >= a.E) s_bad = 1;
      atomicAdd(&s_cnt[f >= f_first][bin_of(id, a.E)], 1);
    };
    const int4* ids4 = reinterpret_cast<const int4*>(a.ids);   // 16-byte aligned
#pragma unroll 4
    for (int i = tid; i < P / 4; i += kSortThreads) {
      const int4 v = __ldg(ids4 + i);
      count(4 * i, v.x);
      count(4 * i + 1, v.y);
      count(4 * i + 2, v.z);
      count(4 * i + 3, v.w);
    }
    if (tid < (P & 3)) count((P & ~3) + tid, __ldg(a.ids + (P & ~3) + tid));
    __syncthreads();
    const int before = tid < a.E ? s_cnt[0][tid] : 0;
    const int off = scan_block<kSortWarps>(tid < a.E ? before + s_cnt[1][tid] : 0, s_warp, &total);
    if (tid < a.E) s_run[tid] = off + before;
    if (tid == 0) s_run[a.E] = total + s_cnt[0][a.E];
    if (blockIdx.x == 0) {
      if (tid < a.E) a.offsets[tid] = off;
      if (tid == 0) a.offsets[a.E] = total;
      if (a.status && tid < 4) a.status[tid] = tid == 0 && s_bad ? MOE_DEVICE_FLAG_BAD_ID : 0;
    }
  } else {
    const int count = tid < a.E ? a.totals[tid] : 0;
    const int before = tid < a.E ? a.hist[static_cast<int64_t>(tid) * a.nb + blockIdx.x] : 0;
    const int dropped = tid == 0 ? a.hist[static_cast<int64_t>(a.E) * a.nb + blockIdx.x] : 0;
    const int off = scan_block<kSortWarps>(count, s_warp, &total);
    if (tid < a.E) s_run[tid] = off + before;
    if (tid == 0) s_run[a.E] = total + dropped;
    if (blockIdx.x == 0) {
      if (tid < a.E) a.offsets[tid] = off;
      if (tid == 0) a.offsets[a.E] = total;
    }
  }
  const int per = kSortThreads / a.k;   // tokens of a sub-chunk
  for (int64_t t0 = t_first; t0 < t_last; t0 += per) {
    const int n = static_cast<int>(min(static_cast<int64_t>(per), t_last - t0));
    const bool mine = tid < n * a.k;
    const int64_t f = t0 * a.k + tid;
    const int e = mine ? bin_of(a.ids[f], a.E) : -1;
    __syncthreads();   // s_run is set; the copy before has read s_dst
    const uint32_t peers = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    if (mine && rank == 0) s_wcnt[warp][e] = __popc(peers);
    __syncthreads();
    if (mine) {
      int p = s_run[e] + rank;
      for (int w = 0; w < warp; ++w) p += s_wcnt[w][e];
      if (e == a.E) p = ~p;
      s_dst[tid] = p;
      a.inv[f] = p;
    }
    __syncthreads();
    if (t0 + per < t_last) {
      for (int b = tid; b <= a.E; b += kSortThreads) {
        int add = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
          add += s_wcnt[w][b];
          s_wcnt[w][b] = 0;
        }
        s_run[b] += add;
      }
    }
    for (int i = my_token; i < n; i += kSortThreads / g) {
      const char* row = x + (t0 + i) * row_bytes;
      for (int v = first; v < nvec; v += Copy::kQ * g) {
        if (t0 > t_first || i > my_token || v > first) Copy::load(val, row, v, g, nvec);
        for (int j = 0; j < a.k; ++j)
          Copy::store(val, x_perm, s_dst[i * a.k + j], v, g, nvec);
      }
    }
  }
}

// The same copy by a map that is there already (inv). Places outside [0, T*k) write nothing.
template <int kBytes>
__global__ void __launch_bounds__(kSortThreads)
dispatch_rows_kernel(const char* __restrict__ x, const int32_t* __restrict__ inv, int64_t T, int k,
                     int nvec, char* __restrict__ x_perm) {
  pdl_trigger();
  pdl_wait();
  const int64_t P = T * k;
  using Copy = RowCopy<kBytes>;
  const int g = Copy::group(nvec), first = Copy::first(threadIdx.x & (g - 1));
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (kSortThreads / g);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kSortThreads / g) + threadIdx.x / g; t < T;
       t += groups) {
    const char* row = x + t * nvec * kBytes;
    for (int v = first; v < nvec; v += Copy::kQ * g) {
      typename Copy::Raw val[Copy::kQ];
      Copy::load(val, row, v, g, nvec);
      for (int j = 0; j < k; ++j) {
        const int32_t p = __ldg(inv + t * k + j);
        if ((p < 0 ? ~p : p) < P) Copy::store(val, x_perm, p, v, g, nvec);
      }
    }
  }
}

// A thread takes a vector of a token's row: the row loads of its slots are issued together and summed
// in slot order. scales NULL: every weight is 1.
template <typename T, int kSlots>
__global__ void __launch_bounds__(kSortThreads)
combine_kernel(const T* __restrict__ rows, const int32_t* __restrict__ inv,
               const float* __restrict__ scales, int64_t n_tok, int k, int nvec,
               T* __restrict__ y) {
  using V = Vec<T, 16>;
  pdl_trigger();
  pdl_wait();
  const int64_t P = n_tok * k;
  const int64_t total = n_tok * nvec;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kSortThreads;
  const uint4* in = reinterpret_cast<const uint4*>(rows);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x; i < total;
       i += stride) {
    const int64_t t = total <= UINT32_MAX
                          ? static_cast<uint32_t>(i) / static_cast<uint32_t>(nvec) : i / nvec;
    const int v = static_cast<int>(i - t * nvec);
    int32_t row[kSlots];
    float s[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      row[j] = -1;
      s[j] = 1.0f;
      if (j < k) {
        row[j] = __ldg(inv + t * k + j);
        if (row[j] >= P) row[j] = -1;
        if (scales) s[j] = __ldg(scales + t * k + j);
      }
    }
    float acc[V::kN] = {};
    uint4 val[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (row[j] >= 0) val[j] = __ldg(in + static_cast<int64_t>(row[j]) * nvec + v);
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      if (row[j] < 0) continue;
      float f[V::kN];
      V::unpack(val[j], f);
#pragma unroll
      for (int c = 0; c < V::kN; ++c) acc[c] = fmaf(s[j], f[c], acc[c]);
    }
    reinterpret_cast<uint4*>(y)[t * nvec + v] = V::pack(acc);
  }
}

// Rows that do not start on 16 bytes: vectors of kBytes. These kernels have instructions to save, so a
// warp takes kU times 32 neighbouring vectors, which one address a row reaches, unchecked where all of
// them exist (kFull), kJ slots at a time. (4096 tokens, k = 6, bf16: H = 7167 94 us, H = 7164 75; a
// thread for every four vectors, each with its own addresses, took 154 for either. Reading rows in
// aligned 16-byte vectors and shifting these into place took 125, and 1001 f32 69 instead of 23.)
template <typename T, int kBytes, int kU, int kJ, bool kFull>
__device__ __forceinline__ void combine_segment(const T* rows, int32_t place, float scale, int64_t P,
                                                int k, int nvec, int v, T* y) {
  using V = Vec<T, kBytes>;
  using Raw = typename V::Raw;
  float acc[kU][V::kN] = {};
  for (int j = 0; j < k; j += kJ) {
    Raw val[kJ][kU];
    float s[kJ];
#pragma unroll
    for (int h = 0; h < kJ; ++h) {
      const int32_t p = __shfl_sync(0xffffffffu, place, j + h);   // (-1 in the lanes past k)
      s[h] = __shfl_sync(0xffffffffu, scale, j + h);
      const bool kept = p >= 0 && p < P;
      const Raw* src = reinterpret_cast<const Raw*>(rows) + static_cast<int64_t>(p) * nvec + v;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        val[h][u] = Raw{};
        if (kept && (kFull || v + u * 32 < nvec)) val[h][u] = __ldg(src + u * 32);
      }
      if (!kept) s[h] = 0.0f;
    }
#pragma unroll
    for (int h = 0; h < kJ; ++h)
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float f[V::kN];
        V::unpack(val[h][u], f);
#pragma unroll
        for (int c = 0; c < V::kN; ++c) acc[u][c] = fmaf(s[h], f[c], acc[u][c]);
      }
  }
#pragma unroll
  for (int u = 0; u < kU; ++u)
    if (kFull || v + u * 32 < nvec) reinterpret_cast<Raw*>(y)[v + u * 32] = V::pack(acc[u]);
}

template <typename T, int kBytes, int kU, int kJ>
__global__ void __launch_bounds__(kSortThreads)
combine_narrow_kernel(const T* __restrict__ rows, const int32_t* __restrict__ inv,
                      const float* __restrict__ scales, int64_t n_tok, int k, int nvec,
                      T* __restrict__ y) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t P = n_tok * k;
  const int segs = (nvec + 32 * kU - 1) / (32 * kU);
  const int64_t total = n_tok * segs, stride = static_cast<int64_t>(gridDim.x) * kSortWarps;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kSortWarps + (threadIdx.x >> 5); i < total;
       i += stride) {
    const int64_t t = total <= UINT32_MAX
                          ? static_cast<uint32_t>(i) / static_cast<uint32_t>(segs) : i / segs;
    const int v = static_cast<int>(i - t * segs) * 32 * kU;
    int32_t place = -1;
    float scale = 1.0f;
    if (lane < k) {
      place = __ldg(inv + t * k + lane);
      if (scales) scale = __ldg(scales + t * k + lane);
    }
    T* to = y + t * nvec * Vec<T, kBytes>::kN;
    if (v + 32 * kU <= nvec)
      combine_segment<T, kBytes, kU, kJ, true>(rows, place, scale, P, k, nvec, v + lane, to);
    else
      combine_segment<T, kBytes, kU, kJ, false>(rows, place, scale, P, k, nvec, v + lane, to);
  }
}

// kWarps warps to a slot (dy[t] comes from L1 or L2 to the second and later ones of its token), a warp kU
// times 32 neighbouring vectors of kBytes at a time, unchecked where all of them exist (kFull). The dot
// product is summed in a thread, over the lanes and over the warps, in that order. bf16: 8192 tokens of
// 7168, k = 8, 291 us, of 2048 83, of 256 17; 4096 of 7167, k = 6, 176, of 7164 129. (A token's slots
// together, dy read once, its dot products side by side: 306, 113, 24, 212 and 212, as fewer loads were
// in flight and more instructions spent on addresses.)
template <typename T, int kBytes, int kU, bool kFull>
__device__ __forceinline__ float combine_grad_segment(const T* dy, const T* rows, float s, int nvec,
                                                      int v, T* drows) {
  using V = Vec<T, kBytes>;
  using Raw = typename V::Raw;
  Raw d[kU], val[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    d[u] = val[u] = Raw{};
    if (kFull || v + u * 32 < nvec) {
      d[u] = __ldg(reinterpret_cast<const Raw*>(dy) + v + u * 32);
      val[u] = __ldg(reinterpret_cast<const Raw*>(rows) + v + u * 32);
    }
  }
  float dot = 0.0f;
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    float df[V::kN], f[V::kN], o[V::kN];
    V::unpack(d[u], df);
    V::unpack(val[u], f);
#pragma unroll
    for (int c = 0; c < V::kN; ++c) {
      dot = fmaf(df[c], f[c], dot);
      o[c] = s * df[c];
    }
    if (kFull || v + u * 32 < nvec) __stcs(reinterpret_cast<Raw*>(drows) + v + u * 32, V::pack(o));
  }
  return dot;
}

template <typename T, int kBytes, int kU, int kWarps>
__global__ void __launch_bounds__(kSortThreads)
combine_grad_kernel(const T* __restrict__ dy, const T* __restrict__ rows,
                           const int32_t* __restrict__ inv, const float* __restrict__ scales,
                           int64_t n_tok, int k, int nvec, T* __restrict__ drows,
                           float* __restrict__ dscales) {
  using V = Vec<T, kBytes>;
  using Raw = typename V::Raw;
  constexpr int kAtOnce = kSortWarps / kWarps;   // slots of a block
  __shared__ float s_dot[kSortWarps];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % kWarps;
  const int64_t P = n_tok * k;
  for (int64_t f0 = static_cast<int64_t>(blockIdx.x) * kAtOnce; f0 < P;
       f0 += static_cast<int64_t>(gridDim.x) * kAtOnce) {
    const int64_t f = f0 + warp / kWarps;
    float dot = 0.0f;
    if (f < P) {
      const int32_t p = __ldg(inv + f);
      const float s = scales ? __ldg(scales + f) : 1.0f;
      const int64_t t = P <= UINT32_MAX ? static_cast<uint32_t>(f) / static_cast<uint32_t>(k) : f / k;
      const int64_t r = p < 0 ? ~p : p;
      const T* from = dy + t * nvec * V::kN;
      const T* with = rows + r * nvec * V::kN;
      T* to = drows + r * nvec * V::kN;
      if (p >= 0 && r < P) {
        for (int v = sub * 32 * kU; v < nvec; v += kWarps * 32 * kU)
          dot += v + 32 * kU <= nvec
                     ? combine_grad_segment<T, kBytes, kU, true>(from, with, s, nvec, v + lane, to)
                     : combine_grad_segment<T, kBytes, kU, false>(from, with, s, nvec, v + lane, to);
      } else if (r < P) {
        for (int v = sub * 32 + lane; v < nvec; v += kWarps * 32)
          __stcs(reinterpret_cast<Raw*>(to) + v, Raw{});
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    if (kWarps == 1) {
      if (f < P && lane == 0) dscales[f] = dot;
    } else {
      if (lane == 0) s_dot[warp] = dot;
      __syncthreads();
      if (f < P && sub == 0 && lane == 0) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s_dot[warp + w];
        dscales[f] = sum;
      }
      __syncthreads();
    }
  }
}

// The widest of 16, 8, 4 and 2 bytes that divides a row.
int copy_bytes(int64_t row_bytes) {
  return row_bytes % 16 == 0 ? 16 : row_bytes % 8 == 0 ? 8 : row_bytes % 4 == 0 ? 4 : 2;
}

unsigned grid_of(int64_t blocks, int per_sm) {
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * per_sm;
  return static_cast<unsigned>(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
}

template <int kBytes>
cudaError_t launch_place(const SortArgs& a, bool self, const void* x, void* x_perm, int nvec,
                         cudaStream_t s) {
  if (self)
    return launch_pdl(sort_place_kernel<kBytes, true>, dim3(a.nb), dim3(kSortThreads), 0, s, a,
                      static_cast<const char*>(x), static_cast<char*>(x_perm), nvec);
  return launch_pdl(sort_place_kernel<kBytes, false>, dim3(a.nb), dim3(kSortThreads), 0, s, a,
                    static_cast<const char*>(x), static_cast<char*>(x_perm), nvec);
}

template <typename T, int kSlots>
cudaError_t combine_t(const void* rows, const int32_t* inv, const float* scales, int64_t n_tok,
                      int H, int k, void* y, cudaStream_t s) {
  const int nvec = H / Vec<T, 16>::kN;
  const int64_t blocks = (n_tok * nvec + kSortThreads - 1) / kSortThreads;
  return launch_pdl(combine_kernel<T, kSlots>, dim3(grid_of(blocks, 32)), dim3(kSortThreads), 0, s,
                    static_cast<const T*>(rows), inv, scales, n_tok, k, nvec, static_cast<T*>(y));
}

template <typename T, int kBytes, int kU, int kJ>
cudaError_t combine_narrow_u(const void* rows, const int32_t* inv, const float* scales,
                             int64_t n_tok, int nvec, int k, void* y, cudaStream_t s) {
  const int64_t warps = n_tok * ((nvec + 32 * kU - 1) / (32 * kU));
  return launch_pdl(combine_narrow_kernel<T, kBytes, kU, kJ>,
                    dim3(grid_of((warps + kSortWarps - 1) / kSortWarps, 32)), dim3(kSortThreads), 0,
                    s, static_cast<const T*>(rows), inv, scales, n_tok, k, nvec,
                    static_cast<T*>(y));
}

template <typename T, int kBytes>
cudaError_t combine_narrow_t(const void* rows, const int32_t* inv, const float* scales,
                             int64_t n_tok, int H, int k, void* y, cudaStream_t s) {
  const int nvec = H / Vec<T, kBytes>::kN;
  // 256 vectors a warp, two slots at a time, or, for short rows and where that leaves few warps, 128 and
  // four: 4096 tokens, k = 6, H = 7167 bf16 94 us the one way and 116 the other; 500 tokens, k = 8, H =
  // 2050 5.2 and 4.6, 8192 tokens, k = 8, H = 65 f16 10.0 and 7.0.
  if (nvec <= 128 || n_tok * ((nvec + 255) / 256) <= 4096)
    return combine_narrow_u<T, kBytes, 4, 4>(rows, inv, scales, n_tok, nvec, k, y, s);
  return combine_narrow_u<T, kBytes, 8, 2>(rows, inv, scales, n_tok, nvec, k, y, s);
}

template <typename T, int kBytes, int kU>
cudaError_t combine_grad_u(const void* dy, const void* rows, const int32_t* inv,
                           const float* scales, int64_t n_tok, int k, int nvec, void* drows,
                           float* dscales, cudaStream_t s) {
  const int64_t P = n_tok * k;
  auto run = [&](auto* kernel, int64_t blocks) {
    return launch_pdl(kernel, dim3(grid_of(blocks, 32)), dim3(kSortThreads), 0, s,
                      static_cast<const T*>(dy), static_cast<const T*>(rows), inv, scales, n_tok, k,
                      nvec, static_cast<T*>(drows), dscales);
  };
  // A warp to a slot where it holds a row, where the slots alone fill the GPU, or nearly so with rows that
  // are not long, else a block: k = 8 bf16, 512 tokens of 7167 45 us a warp each and 33 a block each, of
  // 7168 22 and 24, 256 tokens of 1001 4.2 and 4.6, 8192 of 2048 84 and 138; 4000 of 333 (k = 4) 7 and 18.
  if constexpr (kU == 4) {
    if (nvec > 32 * kU && P < (nvec <= 1024 ? 2048 : 8192))
      return run(combine_grad_kernel<T, kBytes, kU, kSortWarps>, P);
  }
  return run(combine_grad_kernel<T, kBytes, kU, 1>, (P + kSortWarps - 1) / kSortWarps);
}

template <typename T, int kBytes>
cudaError_t combine_grad_t(const void* dy, const void* rows, const int32_t* inv,
                           const float* scales, int64_t n_tok, int H, int k, void* drows,
                           float* dscales, cudaStream_t s) {
  const int nvec = H / Vec<T, kBytes>::kN;
  // As many vectors as a row has for a warp, up to four: 8192 tokens bf16, H = 256, k = 8 17.0 us with
  // one, 29.6 with four; H = 512, k = 4 15.1 with two, 15.9 and 19.4; H = 2048, k = 8 83 with four, 88
  // with one.
  if (nvec <= 32)
    return combine_grad_u<T, kBytes, 1>(dy, rows, inv, scales, n_tok, k, nvec, drows, dscales, s);
  if (nvec <= 64)
    return combine_grad_u<T, kBytes, 2>(dy, rows, inv, scales, n_tok, k, nvec, drows, dscales, s);
  return combine_grad_u<T, kBytes, 4>(dy, rows, inv, scales, n_tok, k, nvec, drows, dscales, s);
}

// Calls f<T, bytes>() for the type and the vectors of its rows: 16 bytes where all rows start on them,
// 4 where they start on these, else an element.
template <typename F>
cudaError_t by_width(int dtype, int H, const F& f) {
  auto width = [&](auto t) {
    using T = decltype(t);
    const int64_t row = static_cast<int64_t>(H) * sizeof(T);
    if (row % 16 == 0) return f.template operator()<T, 16>();
    if (row % 4 == 0) return f.template operator()<T, 4>();
    return f.template operator()<T, static_cast<int>(sizeof(T))>();
  };
  if (dtype == MOE_DTYPE_BF16) return width(__nv_bfloat16());
  if (dtype == MOE_DTYPE_F16) return width(__half());
  return width(float());
}

struct CombineCall {
  const void* rows;
  const int32_t* inv;
  const float* scales;
  int64_t T;
  int H, k;
  void* y;
  cudaStream_t s;
  template <typename E, int kBytes>
  cudaError_t operator()() const {
    if constexpr (kBytes < 16) {
      return combine_narrow_t<E, kBytes>(rows, inv, scales, T, H, k, y, s);
    } else {
      return k == 1   ? combine_t<E, 1>(rows, inv, scales, T, H, k, y, s)
             : k == 2 ? combine_t<E, 2>(rows, inv, scales, T, H, k, y, s)
             : k <= 4 ? combine_t<E, 4>(rows, inv, scales, T, H, k, y, s)
                      : combine_t<E, 8>(rows, inv, scales, T, H, k, y, s);
    }
  }
};

struct CombineGradCall {
  const void* dy;
  const void* rows;
  const int32_t* inv;
  const float* scales;
  int64_t T;
  int H, k;
  void* drows;
  float* dscales;
  cudaStream_t s;
  template <typename E, int kBytes>
  cudaError_t operator()() const {
    return combine_grad_t<E, kBytes>(dy, rows, inv, scales, T, H, k, drows, dscales, s);
  }
};

int elem_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

// Problems of at most this many slots are sorted and copied in one launch, every block counting all
// ids (9222 slots, rows of 1001 f32: 12.3 us, in three launches 14.2; 32768 slots of 4096 bf16:
// 69 us, in three launches 64).
constexpr int64_t kSelfCountMax = MOE_DISPATCH_SMALL_SLOTS;

void chunk_plan(int64_t T, int64_t out_bytes, int64_t* chunk, int* nb) {
  int most = kMaxBlocks;
  if (out_bytes <= kOneWaveBytes) most = std::min(most, kBlocksPerSm * device_sm_count());
  *chunk = (T + most - 1) / most;
  *nb = static_cast<int>((T + *chunk - 1) / *chunk);
}

}  // namespace

size_t dispatch_workspace_bytes(int64_t T, int E) {
  int64_t chunk = 1;
  int nb = 1;
  if (T > 0) chunk_plan(T, kOneWaveBytes + 1, &chunk, &nb);   // (the more blocks of the two)
  return 16 + 4 * (static_cast<size_t>(E) + static_cast<size_t>(E + 2) * nb);
}

moe_status launch_dispatch(const void* x, const int32_t* ids, int64_t T, int H, int E, int k,
                           int dtype, void* x_perm, int32_t* inv, int32_t* offsets, char* ws,
                           cudaStream_t s) {
  SortArgs a;
  a.ids = ids;
  a.T = T;
  a.P = T * k;
  a.E = E;
  a.k = k;
  chunk_plan(T, a.P * H * elem_bytes(dtype), &a.chunk, &a.nb);
  a.status = reinterpret_cast<int32_t*>(ws);
  a.totals = ws ? a.status + 4 : nullptr;
  a.hist = ws ? a.totals + E : nullptr;
  a.inv = inv;
  a.offsets = offsets;
  const bool self = a.P <= kSelfCountMax;
  cudaError_t err = cudaSuccess;
  if (!self) {
    err = launch_pdl(sort_count_kernel, dim3(a.nb), dim3(kSortThreads), 0, s, a);
    if (err == cudaSuccess)
      err = launch_pdl(sort_scan_kernel, dim3(E + 2), dim3(kScanThreads), 0, s, a);
  }
  if (err == cudaSuccess) {
    const int64_t row = static_cast<int64_t>(H) * elem_bytes(dtype);
    const int cb = copy_bytes(row);
    const int nvec = static_cast<int>(row / cb);
    err = cb == 16  ? launch_place<16>(a, self, x, x_perm, nvec, s)
          : cb == 8 ? launch_place<8>(a, self, x, x_perm, nvec, s)
          : cb == 4 ? launch_place<4>(a, self, x, x_perm, nvec, s)
                    : launch_place<2>(a, self, x, x_perm, nvec, s);
  }
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "dispatch launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

moe_status launch_dispatch_rows(const void* x, const int32_t* inv, int64_t T, int H, int k,
                                int dtype, void* x_perm, cudaStream_t s) {
  const int64_t row = static_cast<int64_t>(H) * elem_bytes(dtype);
  const int cb = copy_bytes(row);
  const int nvec = static_cast<int>(row / cb);
  const dim3 grid(grid_of(T, 16)), block(kSortThreads);
  const char* in = static_cast<const char*>(x);
  char* out = static_cast<char*>(x_perm);
  const cudaError_t err =
      cb == 16  ? launch_pdl(dispatch_rows_kernel<16>, grid, block, 0, s, in, inv, T, k, nvec, out)
      : cb == 8 ? launch_pdl(dispatch_rows_kernel<8>, grid, block, 0, s, in, inv, T, k, nvec, out)
      : cb == 4 ? launch_pdl(dispatch_rows_kernel<4>, grid, block, 0, s, in, inv, T, k, nvec, out)
                : launch_pdl(dispatch_rows_kernel<2>, grid, block, 0, s, in, inv, T, k, nvec, out);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "dispatch_rows launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

moe_status launch_combine(const void* rows, const int32_t* inv, const float* scales, int64_t T,
                          int H, int k, int dtype, void* y, cudaStream_t s) {
  const cudaError_t err = by_width(dtype, H, CombineCall{rows, inv, scales, T, H, k, y, s});
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "combine launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

moe_status launch_combine_backward(const void* dy, const void* rows, const int32_t* inv,
                                   const float* scales, int64_t T, int H, int k, int dtype,
                                   void* drows, float* dscales, cudaStream_t s) {
  const cudaError_t err =
      by_width(dtype, H, CombineGradCall{dy, rows, inv, scales, T, H, k, drows, dscales, s});
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "combine_backward launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

}  // namespace moe
