// Tiles of the experts' products over ragged groups of rows: which rows and channels a tile index stands
// for, shared by the kernels on 16-bit and on 4-bit operands.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace moe {
namespace {

enum : int { kFwd = 0, kDx = 1, kDw = 2 };

constexpr int kXBK = 64;                      // contraction elements a block, of 16 bits
constexpr int kXGroups = 258;                 // up to 256 experts, and the rows before and after them
constexpr int kXRowBlocks = 8;                // row blocks that are walked together

struct ExpertsArgs {
  const int32_t* offsets;   // [E + 1]
  int32_t E;
  int32_t R;                // rows of x, dy, y, dx
  int32_t m_ext;            // forward, dx: columns of the result (M); dw: rows of a dw[e] (M)
  int32_t n_ext;            // dw: columns of a dw[e] (N)
  int32_t k_ext;            // forward, dx: the contraction
  int32_t f16;              // 16-bit type: 0 bf16, 1 f16
  int32_t add;              // dw, f32: add to what is there
  int32_t split;            // log2 of the parts that the contraction is cut into
  void* out;                // forward, dx: the result rows (masked stores); dw: dw (rows of odd
                            // multiples of 16 bytes)
  float* part;              // forward, dx with f32 results: [parts][R][m_ext] sums of the parts
  const CUtensorMap* maps;  // dw: [2][E] maps of dy and of x, cut off at each expert's end
  int32_t* status;          // or NULL
};

struct Tile {
  int g;        // the expert
  int m0;       // this CTA's first index along M: a channel of the result, or a row of dw[g]
  int m_here;   // how many of its 128 exist
  int m_peer;   // the same of the other CTA
  int n0;       // the pair's first index along N: a row, or a column of dw[g]
  int n_here;   // how many exist, 1..256
  int n;        // the instruction's N: n_here rounded up to 16
  int k0;       // first element of the contraction (dw: a row)
  int part;     // of the contraction's parts
  int nkb;      // contraction blocks; 0: the tile is zeros
  int nks;      // contraction steps of 16 elements, the last one filled up with zeros
};

__device__ __forceinline__ int clamp_int(int v, int lo, int hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

// n / d by a rounded 1 / d: exact for 0 <= n < 2^24 (the quotient is off by one at most, which the
// remainder shows). The divisions of a tile's index are on the epilogue's path between two tiles.
struct Div {
  int d;
  float inv;
  __device__ __forceinline__ explicit Div(int d_) : d(d_), inv(1.0f / static_cast<float>(d_)) {}
  __device__ __forceinline__ int operator()(int n) const {
    const int q = static_cast<int>(static_cast<float>(n) * inv);
    const int r = n - q * d;
    return r < 0 ? q - 1 : r >= d ? q + 1 : q;
  }
};

// n / d for 0 <= n < 2^12 and small d, by an approximate reciprocal: (n + 1/2) / d is at least 1 / 2d
// from a whole number, far more than its error.
__device__ __forceinline__ int small_div(int n, int d) {
  return static_cast<int>(__fdividef(static_cast<float>(n) + 0.5f, static_cast<float>(d)));
}

// Divisors of a tile's index. "Outer" tiles are those of the rows in forward and dx and of M in dw,
// "inner" ones those of M and of N: kXRowBlocks outer tiles by all inner ones make a set, walked
// outer tile first.
struct Walk {
  Div inner, set, outer;
  template <int kMode>
  __device__ __forceinline__ static Walk of(const ExpertsArgs& a) {
    const int inner = ((kMode == kDw ? a.n_ext : a.m_ext) + 255) >> 8;
    return Walk{Div(inner), Div(inner * kXRowBlocks), Div(kMode == kDw ? (a.m_ext + 255) >> 8 : 1)};
  }
};

// The tile of an index, by a whole warp whose indices only grow (`from`: the group of its last
// one, 0 to begin with). s_blk[g] (forward, dx): row tiles of the groups before g. s_start[g]: the first row of g;
// s_start[G] the last one's end. dw's groups are the experts; forward and dx have the rows before
// the first expert's as group 0, expert e as group e + 1 and the rows past the last one's as
// group E + 1.
// f32 results: neighbouring indices are the parts of a tile's contraction, whole blocks each.
// kMost: rows of a tile (forward, dx), a multiple of 16.
template <int kMode, bool kF32, int kMost = 256>
__device__ __forceinline__ Tile decode_tile(int idx, const uint16_t* s_blk, const int32_t* s_start,
                                            int G, const ExpertsArgs& a, const Walk& w,
                                            int rank, int lane, int& from) {
  const int part = kF32 ? idx & ((1 << a.split) - 1) : 0;
  if (kF32) idx >>= a.split;
  const int blk = w.inner(idx);
  int g, outer, before;
  if (kMode == kDw) {
    (void)lane, (void)from, (void)s_blk, (void)G;
    outer = w.outer.d;
    g = w.outer(blk);
    before = g * outer;
  } else {
    // On from the last tile's group, 32 groups a step: s_blk[g] <= blk < s_blk[g + 1].
    g = from;
    for (int more = 32; more == 32; g += more)
      more = __popc(__ballot_sync(0xffffffffu, s_blk[min(g + 1 + lane, G)] <= blk));
    from = g;
    before = s_blk[g];
    outer = s_blk[g + 1] - before;
  }
  const int start = s_start[g], rows = s_start[g + 1] - start;
  const int local = idx - before * w.inner.d;
  const int set = w.set(local);
  const int rest = local - set * w.set.d;
  const int here = min(kXRowBlocks, outer - set * kXRowBlocks);
  const int i = small_div(rest, here);              // inner tile (rest < 8 * 256)
  const int o = set * kXRowBlocks + rest - i * here;   // outer tile
  Tile t;
  t.g = g;
  int n_end;
  if (kMode == kDw) {
    t.m0 = o * 256;
    t.n0 = i * 256;
    n_end = min(a.n_ext, t.n0 + 256);
    t.k0 = start;
  } else {
    // Of the group's equal tiles: u = rows / 16 (rounded up) over `outer` = u / (kMost / 16) (rounded
    // up), rounded up, that is kMost / 16 - (kMost / 16 * outer - u) / outer, the difference under kMost / 16.
    const int spare = kMost / 16 * outer - ((rows + 15) >> 4);
    const int size = kMost - 16 * small_div(spare, outer);
    t.m0 = i * 256;
    t.n0 = start + o * size;
    n_end = min(start + rows, t.n0 + size);
    t.k0 = 0;
  }
  t.n_here = n_end - t.n0;
  t.n = (t.n_here + 15) & ~15;
  t.m_peer = clamp_int(a.m_ext - (t.m0 + 128 * (rank ^ 1)), 0, 128);
  t.m0 += 128 * rank;
  t.m_here = clamp_int(a.m_ext - t.m0, 0, 128);
  if (kMode != kDw) t.g = g - 1;
  const int len = kMode == kDw ? rows : g > 0 && g <= a.E ? a.k_ext : 0;
  t.part = part;
  t.nkb = (len + kXBK - 1) / kXBK;
  t.nks = (len + 15) / 16;
  if (kF32) {
    const int b0 = t.nkb * part >> a.split, b1 = t.nkb * (part + 1) >> a.split;
    t.k0 += b0 * kXBK;
    t.nks = min(t.nks, b1 * (kXBK / 16)) - b0 * (kXBK / 16);
    t.nkb = b1 - b0;
  }
  return t;
}

// The groups, by one warp: their first rows, kept inside [0, R] and in order here, so that no offset
// can lead a load or a store out of range, and the scan of their row blocks.
template <int kMode, int kMost = 256>
__device__ __forceinline__ void scan_groups(const ExpertsArgs& a, int lane, uint16_t* s_blk,
                                            int32_t* s_start) {
  const int G = kMode == kDw ? a.E : a.E + 2;
  constexpr int kHead = kMode == kDw ? 0 : 1;
  constexpr int kPer = kXGroups / 32 + 1;   // 32 * kPer > kXGroups: a lane reaches entry G
  int start[kPer + 1], most = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = lane * kPer + i;
    start[i] = g < kHead ? 0 : g - kHead <= a.E ? clamp_int(a.offsets[g - kHead], 0, a.R) : a.R;
    if (i > 0) start[i] = max(start[i], start[i - 1]);
  }
  most = start[kPer - 1];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) most = max(most, __shfl_up_sync(0xffffffffu, most, off));
  most = __shfl_up_sync(0xffffffffu, most, 1);
  if (lane == 0) most = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) start[i] = max(start[i], most);
  start[kPer] = __shfl_down_sync(0xffffffffu, start[0], 1);
  if (lane == 31) start[kPer] = a.R;
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) sum += (start[i + 1] - start[i] + kMost - 1) / kMost;
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  int at = incl - sum;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = lane * kPer + i;
    if (g <= G) {
      s_start[g] = start[i];
      s_blk[g] = static_cast<uint16_t>(at);
    }
    at += (start[i + 1] - start[i] + kMost - 1) / kMost;
  }
}

__device__ __forceinline__ uint32_t pack_16bit(float lo, float hi, bool f16) {
  if (f16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace
}  // namespace moe
