// The experts' matrix products over ragged groups of rows, with their gradients:
//   forward   y[r]  = x[r] . w[e]^T           rows r of expert e, w [E, N, K]
//   dx        dx[r] = dy[r] . w[e]
//   dw        dw[e] = sum_{r of e} dy[r]^T . x[r]
// Rows of expert e are [offsets[e], offsets[e+1]), offsets on the device. Rows of no expert, before
// offsets[0] and from offsets[E] on, are 0 in y and dx; an expert without rows has dw = 0.
//
// One persistent kernel over all groups, CTA pairs (tcgen05.mma.cta_group::2, M = 256, N up to 256,
// fp32 accumulators in TMEM, 64 elements of the contraction a block). The tensor cores take an
// operand from shared memory along the contraction (K-major) or across it (M- or N-major), so that
// nothing is transposed on the way in:
//            A, M = 256                          B, N <= 256             contraction
//   forward  channels of w[e] (rows), K-major    x rows, K-major         K
//   dx       channels of w[e] (columns), M-major dy rows, K-major        N
//   dw       columns of dy, M-major              columns of x, N-major   the expert's rows
//
// Ragged rows. In forward and dx they are N, which the instruction takes in steps of 16: an expert's
// rows are cut into equal tiles of at most 256, rounded up to 16, and little is multiplied that is
// not wanted (with the rows as M = 256 the tiles of 512-row experts held a quarter of waste, which
// the power limit turns into time). The result then lies channels by rows in TMEM and is turned over
// in the epilogue's boxes. What a tile reads past its rows stays in columns that are not stored.
// In dw the rows are the contraction, where another expert's must not enter: every expert gets
// its own pair of tensor maps whose row count ends at its last row, so that TMA fills what is
// beyond with zeros (a small kernel writes the maps; 0 * NaN cannot reach a neighbour's gradient),
// and steps of 16 rows with nothing in them are not issued.
//
// Where the tiles are few and the contraction long (experts_split), it is cut into 2, 4 or 8 parts, tiles
// of their own whose f32 sums go to the workspace and are added up, in order, by a second kernel.
//
// Measured (one GB300, calls of one product back to back): forward of 8192 x 14336 x 4096 over 8 experts
// 541 us, 0.92 of cuBLAS's burst rate (0.92 of its sustained one too, 625 us, where the power limit
// holds for a second and more); the tensor pipe is active for 92% of the cycles. dx and dw of 32768 x
// 1536 x 4096 over 64 experts 259 and 270 us with 512 rows each, 273 and 280 with uneven ones: the power
// limit (1.56 and 1.69 of 2.07 GHz under ncu), the tensor pipe active for 83% and 76% of the cycles, L2 at
// 54%. Of dx's rest the last round is the most, 10.1 rounds of tiles done as 11. A tile of dw has 8 blocks
// of 0.385 us and 0.26 us beside them (from 512 and 1024 rows each: 270 and 520 us in 81 rounds). dx and dw
// over 256 experts (32768 x 2048 x 7168) 1.16 and 1.27 ms, bound by memory. An f32 dw has twice the bytes
// to write: over those 64 experts 372 to 394 us, added to what is there 670, over 256 with 128 rows each
// 2.99 and 5.90 ms (in 16 bits 1.37 to 1.43), 0.75 to 0.8 of the copy rate.
//
// Tiles go to the CTA pairs in order, pair i taking tiles i, i + pairs, ...: neighbouring tiles
// (eight row tiles by the channels) share operands in L2. No counter hands them out: whole tiles of one
// product cost the same, but the last round is rarely full (above), and with uneven groups some tiles
// have few rows, which costs 2 to 5% above. Every result element is written by one CTA from one
// accumulator: the same result on every run.
//
// Warp roles (352 threads per CTA): warps 0 and 10 TMA producers of A and of B, warp 1 TMEM allocator
// and, in the first CTA, MMA issuer, warps 2-9 epilogue (TMEM lanes 32 * (warp % 4) .. + 31), four
// to each of two accumulators, so that the epilogue of a tile overlaps the next one's mainloop.
#include <atomic>
#include <cstdint>

#include <cuda.h>

#include "experts_tiles.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "rows.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

constexpr int kXSlotBytes = 128 * kXBK * 2;   // one operand of one block in one CTA
constexpr int kXAccCols = 256;
constexpr int kXTmemCols = 512;
constexpr int kXEpiWarps = 8;                 // two sets of four, one set to an accumulator
constexpr int kXWarpB = 2 + kXEpiWarps;       // the producer of B
constexpr int kXThreads = 32 * (kXWarpB + 1);
constexpr int kXStages = 6;                   // a block of both operands each
constexpr int kXBoxBytes = 4096;              // epilogue staging of a warp
constexpr int kXSmemBytes = 1024 + 2 * kXStages * kXSlotBytes + kXEpiWarps * kXBoxBytes;
constexpr uint16_t kXPairMask = 0x3;

// Set by every wait that runs out, whoever holds the call's workspace, if there is one.
__device__ int32_t g_experts_timeouts;

__device__ __forceinline__ void x_timeout(int32_t* status, volatile int* abort) {
  *abort = 1;
  if (status) atomicOr(status, MOE_DEVICE_FLAG_TIMEOUT);
  atomicOr(&g_experts_timeouts, MOE_DEVICE_FLAG_TIMEOUT);
}

// Loads are issued by the whole warp, one thread of it taking effect: descriptors, addresses and
// coordinates are then the same in all lanes and stay in uniform registers, where the TMA unit takes
// them from. Issued from a branch of one lane, their way there cost 100 cycles and more an
// instruction, and the producer, not the tensor cores, set the pace (dw at 8192 x 14336 x 4096
// over 8 experts, four boxes a block: 768 us, so 604; dx there, three boxes: 691 us, so 571). A and
// B have a warp each: one warp for both took 5% more for dw.
//
// The loads of one tile in this CTA. A: its 128 indices along M (left out where none exists: what
// the stage holds then only reaches accumulator lanes that are not stored). B: its half of the
// tile's N, in one box of 128 rows, or of 32 rows each where at most 64 are wanted (mb32); in dw
// in boxes of 64 columns. An operand across the contraction comes in boxes of 64 (its swizzle's
// width) by the 64 of the block.
template <int kMode>
__device__ __forceinline__ bool produce_a(const Tile& t, const CUtensorMap* ma, int rank, int& stage,
                                          uint32_t& phase, uint8_t* sA, uint32_t lead_full,
                                          uint64_t* full_bar, uint64_t* empty_bar,
                                          volatile int* abort) {
  const uint32_t tx = kXSlotBytes * ((t.m_here > 0) + (t.m_peer > 0));
  for (int kb = 0; kb < t.nkb; ++kb) {
    if (!__all_sync(0xffffffffu, mbar_wait<true>(&empty_bar[stage], phase ^ 1u, abort))) return false;
    if (elect_one()) {
      if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], tx);
      const uint32_t fb = lead_full + 8u * stage;
      uint8_t* as = sA + stage * kXSlotBytes;
      const int kc = t.k0 + kb * kXBK;
      if (t.m_here > 0) {
        if (kMode == kFwd) {
          tma_load_3d_pair(as, ma, fb, kc, t.m0, t.g);
        } else if (kMode == kDx) {
          tma_load_3d_pair(as, ma, fb, t.m0, kc, t.g);
          tma_load_3d_pair(as + kXSlotBytes / 2, ma, fb, t.m0 + 64, kc, t.g);
        } else {
          tma_load_2d_pair(as, ma, fb, t.m0, kc);
          tma_load_2d_pair(as + kXSlotBytes / 2, ma, fb, t.m0 + 64, kc);
        }
      }
    }
    __syncwarp();
    if (++stage == kXStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  return true;
}

template <int kMode>
__device__ __forceinline__ bool produce_b(const Tile& t, const CUtensorMap* mb,
                                          const CUtensorMap* mb32, int rank, int& stage,
                                          uint32_t& phase, uint8_t* sB, uint32_t lead_full,
                                          uint64_t* full_bar, uint64_t* empty_bar,
                                          volatile int* abort) {
  const int half = t.n >> 1;
  const bool narrow = kMode != kDw && half <= 64;
  const int box = kMode == kDw ? 64 : narrow ? 32 : 128;   // along N; 128 bytes each
  const bool two = half > box;
  const CUtensorMap* mbx = narrow ? mb32 : mb;
  const uint32_t tx = 2 * (two ? 2 : 1) * box * 128;
  const int n0 = t.n0 + rank * half;
  for (int kb = 0; kb < t.nkb; ++kb) {
    if (!__all_sync(0xffffffffu, mbar_wait<true>(&empty_bar[stage], phase ^ 1u, abort))) return false;
    if (elect_one()) {
      if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], tx);
      const uint32_t fb = lead_full + 8u * stage;
      uint8_t* bs = sB + stage * kXSlotBytes;
      const int kc = t.k0 + kb * kXBK;
      if (kMode == kDw) {
        tma_load_2d_pair(bs, mbx, fb, n0, kc);
        if (two) tma_load_2d_pair(bs + kXSlotBytes / 2, mbx, fb, n0 + 64, kc);
      } else {
        tma_load_2d_pair(bs, mbx, fb, kc, n0);
        if (two) tma_load_2d_pair(bs + 32 * 128, mbx, fb, kc, n0 + 32);
      }
    }
    __syncwarp();
    if (++stage == kXStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  return true;
}

// The MMAs of one tile, issued the same way (2% faster there than from one lane's branch).
template <int kMode>
__device__ __forceinline__ bool multiply_tile(uint32_t d, uint32_t idesc, int nks, int& stage,
                                              uint32_t& phase, uint64_t da0, uint64_t db0,
                                              uint64_t* full_bar, uint64_t* empty_bar,
                                              volatile int* abort) {
  // 16 elements of the contraction further on: 32 bytes inside the rows, or 16 rows of 128 bytes.
  constexpr uint32_t kStepA = (kMode == kFwd ? 32u : 2048u) >> 4;
  constexpr uint32_t kStepB = (kMode == kDw ? 2048u : 32u) >> 4;
  constexpr int kPer = kXBK / 16;   // instructions a block
  for (int ks = 0; ks < nks; ks += kPer) {
    if (!__all_sync(0xffffffffu, mbar_wait<true>(&full_bar[stage], phase, abort))) return false;
    tc_fence_after();
    const uint64_t da = da0 + ((stage * kXSlotBytes) >> 4), db = db0 + ((stage * kXSlotBytes) >> 4);
    if (elect_one()) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (ks + i >= nks) break;
        umma_bf16_pair(d, da + i * kStepA, db + i * kStepB, idesc, (ks | i) != 0);
      }
      umma_commit_pair(&empty_bar[stage], kXPairMask);
    }
    __syncwarp();
    if (++stage == kXStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  return true;
}

// dw in 16 bits where its rows are an odd number of 16 bytes long, so that every other one starts in the
// middle of a sector (32 bytes): parts of sectors are what costs L2, and each box below would have two
// a row. So in those rows a step's 64 columns are those from 8 on, the last 8 being the next step's
// first, and the tile's first 8 are stored by themselves; steps go out through shared memory by
// plain stores. 54 experts of 2048 x 4104, 128 rows each: 172 us, by boxes 266 (of 2048 x 4096:
// 160); 16 rows each 193 and 247.
template <typename Done>
__device__ __forceinline__ void store_dw_odd(uint32_t tb, const Tile& t, int q, int lane, uint8_t* buf,
                                             const ExpertsArgs& a, Done&& done) {
  const int cols = t.n_here, rows = t.m_here - 32 * q;   // (cols % 8 == 0)
  if (rows <= 0) {
    done();
    return;
  }
  const bool f16 = a.f16 != 0;
  uint16_t* dst = static_cast<uint16_t*>(a.out) +
                  (static_cast<int64_t>(t.g) * a.m_ext + t.m0 + 32 * q) * a.n_ext + t.n0;
  const int odd0 = static_cast<int>(reinterpret_cast<uintptr_t>(dst) >> 4 & 1);   // of the first row
  const bool odd = ((odd0 ^ lane) & 1) != 0;
  uint4* mine = reinterpret_cast<uint4*>(buf + lane * 128);
#pragma unroll 1
  for (int c0 = 0; c0 < cols; c0 += 64) {
    uint32_t v[2][32], next[8] = {};
    tmem_issue(tb + c0, v[0]);
    tmem_issue(tb + c0 + 32, v[1]);
    if (c0 + 64 < cols) tmem_issue(tb + c0 + 64, next);
    tmem_wait();
    tmem_ready(v[0]);
    tmem_ready(v[1]);
    tmem_ready(next);
    if (c0 + 64 >= cols) done();
    uint32_t w[36];
#pragma unroll
    for (int i = 0; i < 32; ++i)
      w[i] = pack_16bit(__uint_as_float(v[i / 16][2 * i % 32]),
                        __uint_as_float(v[i / 16][2 * i % 32 + 1]), f16);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[32 + i] = pack_16bit(__uint_as_float(next[2 * i]), __uint_as_float(next[2 * i + 1]), f16);
    if (c0 == 0 && odd && lane < rows)
      *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(lane) * a.n_ext) =
          make_uint4(w[0], w[1], w[2], w[3]);
    __syncwarp();   // the step before has been read out
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint4 o;
      o.x = odd ? w[4 * i + 4] : w[4 * i];
      o.y = odd ? w[4 * i + 5] : w[4 * i + 1];
      o.z = odd ? w[4 * i + 6] : w[4 * i + 2];
      o.w = odd ? w[4 * i + 7] : w[4 * i + 3];
      mine[i ^ (lane & 7)] = o;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      const int c = c0 + 8 * ((lane & 7) + ((odd0 ^ r) & 1));
      if (r < rows && c < cols)
        *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(r) * a.n_ext + c) =
            *reinterpret_cast<const uint4*>(buf + r * 128 + (((lane ^ r) & 7) << 4));
    }
  }
}

// The zeros of an expert without rows for such a dw, by rows: all of dw[g] is zeros, so that the pieces of
// rows that start in the middle of a sector are moved on by 8 columns, into the next tile's. 54 experts
// of 2048 x 4104 bf16, four rows in all: 160 us, by rows alone 199, by boxes 239 (of 2048 x 4096: 144).
__device__ __forceinline__ void store_dw_zeros(const Tile& t, int q, int lane, const ExpertsArgs& a) {
  const int rows = min(32, t.m_here - 32 * q);
  uint16_t* dst = static_cast<uint16_t*>(a.out) +
                  (static_cast<int64_t>(t.g) * a.m_ext + t.m0 + 32 * q) * a.n_ext;
  for (int r = 0; r < rows; ++r, dst += a.n_ext) {
    const int on = static_cast<int>(reinterpret_cast<uintptr_t>(dst) >> 4 & 1) * 8;   // (n_ext % 8 == 0)
    const int c = t.n0 + on + 8 * lane;
    if (8 * lane < t.n_here && c < a.n_ext) *reinterpret_cast<uint4*>(dst + c) = uint4{};
    if (c == 8 && on) *reinterpret_cast<uint4*>(dst) = uint4{};
  }
}

// dw: one warp's part of a tile, 32 rows of dw[g] (TMEM lane quarter q) by its columns, in boxes of
// 128 bytes of columns (64 16-bit or 32 f32 values) through shared memory and out by TMA, which
// leaves out what lies beyond dw[g]. `done` runs once the accumulator has been read.
// A box costs its warp about 700 cycles of latency (TMEM load, fence, the store's read of the box
// before), and with a short contraction the epilogue is the longer part of a tile. 256 experts of 128
// rows, N = 7168, K = 2048 (8.1 GB): 2.50 ms with one set of four warps, 1.87 with eight that each had
// half of a tile's columns, 1.55 with a set to each accumulator, 1.25 once the accumulators went back
// without a release of these stores; 6.5 TB/s, bound by memory.
template <bool kF32, typename Done>
__device__ __forceinline__ void store_dw(uint32_t tb, const Tile& t, int q, int lane,
                                         uint8_t* buf, const CUtensorMap* map,
                                         const ExpertsArgs& a, Done&& done) {
  const int cols = t.n_here;
  if (32 * q >= t.m_here) {
    done();
    return;
  }
  constexpr int kCols = kF32 ? 32 : 64;   // of a box
  const bool f16 = a.f16 != 0;
  const int row = t.m0 + 32 * q, col = t.n0;
  uint4* mine = reinterpret_cast<uint4*>(buf + lane * 128);
#pragma unroll 1
  for (int c0 = 0; c0 < cols; c0 += 64) {
    uint32_t v[2][32];
    if (t.nkb > 0) {
      tmem_issue(tb + c0, v[0]);
      tmem_issue(tb + c0 + 32, v[1]);
      tmem_wait();
      tmem_ready(v[0]);
      tmem_ready(v[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[0][i] = v[1][i] = 0;
    }
    if (c0 + 64 >= cols) done();
#pragma unroll
    for (int c = 0; c < 64; c += kCols) {
      if (c0 + c >= cols) break;
      uint4 o[8];
      uint32_t* w = reinterpret_cast<uint32_t*>(o);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if constexpr (kF32)
          w[i] = v[c / 32][i];
        else
          w[i] = pack_16bit(__uint_as_float(v[i / 16][2 * i % 32]),
                            __uint_as_float(v[i / 16][2 * i % 32 + 1]), f16);
      }
      if (lane == 0) bulk_wait_group_read<0>();   // the box before has been read out
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) mine[i ^ (lane & 7)] = o[i];
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        // Parts of a split contraction are planes of their own.
        const int plane = kF32 ? t.part * a.E + t.g : t.g;
        if (kF32 && a.add) tma_add_3d(map, buf, col + c0 + c, row, plane);
        else tma_store_3d(map, buf, col + c0 + c, row, plane);
        bulk_commit_group();
      }
    }
  }
}

// Forward and dx: one warp's part of a tile, 32 channels (its TMEM lane quarter) by the tile's rows, 32
// at a time. The accumulator, channels by rows, is read in matrix fragments, two rows of a
// channel packed together, and transposed by the matrix store into a box of 32 rows of 64 bytes
// (64-byte swizzle). Whole boxes go out by TMA, which leaves out channels past the last; of the
// box with a group's last rows, the rows that exist.
template <typename Done>
__device__ __forceinline__ void store_rows(uint32_t tb, const Tile& t, int q, int lane,
                                           uint8_t* buf, int& sbuf, const CUtensorMap* map,
                                           const ExpertsArgs& a, Done&& done) {
  if (32 * q >= t.m_here) {
    done();
    return;
  }
  const bool f16 = a.f16 != 0;
  const int ch = t.m0 + 32 * q;
#pragma unroll 1
  for (int r2 = 0; r2 < t.n_here; r2 += 64) {
    // Two of them at once: a load takes 400 cycles beside the others.
    uint32_t v[2][2][16];   // [block of 32 rows][lanes 0-15, 16-31]
    const bool both = r2 + 32 < t.n_here;
    if (t.nkb > 0) {
      tmem_issue_fragments(tb + r2, v[0][0]);
      tmem_issue_fragments(tb + r2 + (16u << 16), v[0][1]);
      if (both) {
        tmem_issue_fragments(tb + r2 + 32, v[1][0]);
        tmem_issue_fragments(tb + r2 + 32 + (16u << 16), v[1][1]);
      }
      tmem_wait();
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ready(v[i >> 1][i & 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i >> 5][(i >> 4) & 1][i & 15] = 0;
    }
    if (r2 + 64 >= t.n_here) done();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k == 1 && !both) break;
      const int r0 = r2 + 32 * k;
      uint32_t p[16];   // [channels 8 b .. + 7][rows 8 i .. + 7]: p[4 i + b]
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          p[4 * i + b] = pack_16bit(__uint_as_float(v[k][b >> 1][4 * i + 2 * (b & 1)]),
                                    __uint_as_float(v[k][b >> 1][4 * i + 2 * (b & 1) + 1]), f16);
      uint8_t* box = buf + sbuf * (kXBoxBytes / 2);
      if (lane == 0) bulk_wait_group_read<1>();   // what was stored from this box before is out
      __syncwarp();
      // Row 8 i + lane % 8, chunk of 8 channels lane / 8.
      const uint32_t at = smem_u32(box) + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        stmatrix_trans(at + i * 512, p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
      const int rows = t.n_here - r0;
      if (rows < 32) {
        __syncwarp();
        const int c = lane & 3;   // chunk of 8 channels; m_ext is a multiple of 8
        if (32 * q + 8 * c < t.m_here) {
          uint16_t* dst = static_cast<uint16_t*>(a.out) +
                          static_cast<int64_t>(t.n0 + r0) * a.m_ext + ch + 8 * c;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + (lane >> 2);
            if (row < rows)
              *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(row) * a.m_ext) =
                  *reinterpret_cast<const uint4*>(box + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
          }
        }
        break;   // a tile's last box
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(map, box, ch, t.n0 + r0);
        bulk_commit_group();
      }
      sbuf ^= 1;
    }
  }
}

// The same for one part of a split contraction: f32 sums, a lane to a channel, row by row.
template <typename Done>
__device__ __forceinline__ void store_part(uint32_t tb, const Tile& t, int q, int lane,
                                           const ExpertsArgs& a, Done&& done) {
  if (32 * q >= t.m_here) {
    done();
    return;
  }
  const bool mine = 32 * q + lane < t.m_here;
  float* dst = a.part + (static_cast<int64_t>(t.part) * a.R + t.n0) * a.m_ext + t.m0 + 32 * q + lane;
#pragma unroll 1
  for (int r0 = 0; r0 < t.n_here; r0 += 32) {
    uint32_t v[32];
    if (t.nkb > 0) {
      tmem_issue(tb + r0, v);
      tmem_wait();
      tmem_ready(v);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0;
    }
    if (r0 + 32 >= t.n_here) done();
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (mine && r0 + i < t.n_here)
        dst[static_cast<int64_t>(r0 + i) * a.m_ext] = __uint_as_float(v[i]);
  }
}

template <int kMode, bool kF32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kXThreads, 1)
experts_matmul_kernel(const __grid_constant__ CUtensorMap map_a,
                      const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ CUtensorMap map_b32,
                      const __grid_constant__ CUtensorMap map_out, ExpertsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[kXStages], empty_bar[kXStages];
  __shared__ uint64_t tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;
  __shared__ uint16_t s_blk[kXGroups + 1];
  __shared__ int32_t s_start[kXGroups + 1];

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool lead = rank == 0;
  // 1024-byte aligned stages, at the same offsets in both CTAs.
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sA = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  uint8_t* sB = sA + kXStages * kXSlotBytes;
  uint8_t* sOut = sB + kXStages * kXSlotBytes;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kXStages; ++s) {
      mbar_init(&full_bar[s], 2);    // first CTA: its two producers, and both CTAs' bytes
      mbar_init(&empty_bar[s], 1);   // the pair commit, delivered to both CTAs
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull_bar[s], 1);
      mbar_init(&tempty_bar[s], kXEpiWarps);  // first CTA: four epilogue warps of each CTA
    }
    mbar_init(&drain_bar, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
    tma_prefetch_map(&map_b32);
    tma_prefetch_map(&map_out);
  }
  if (warp == 1) {
    tmem_alloc_pair(&s_tmem_base, kXTmemCols);   // collective with the other CTA's warp 1
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any remote arrival or copy
  tc_fence_after();
  // Everything above overlaps the kernel before.
  pdl_wait();
  const int G = kMode == kDw ? a.E : a.E + 2;
  if (warp == 2) scan_groups<kMode>(a, lane, s_blk, s_start);
  __syncthreads();
  const uint32_t tmem_base = s_tmem_base;
  volatile int* abort = &s_abort;
  const Walk walk = Walk::of<kMode>(a);
  const int total = walk.inner.d * (kMode == kDw ? a.E * walk.outer.d : s_blk[G])
                    << (kF32 ? a.split : 0);
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const uint32_t lead_full = mapa_shared(smem_u32(&full_bar[0]), 0);
  const uint32_t lead_tempty = mapa_shared(smem_u32(&tempty_bar[0]), 0);

  int group = 0;   // of this warp's last tile
  if (warp == 0 || warp == kXWarpB) {
    // ------------------------------------------------------------ TMA producers of A and of B
    int stage = 0, last_g = -1;
    uint32_t phase = 0;
    for (int idx = first; idx < total; idx += step) {
      const Tile t = decode_tile<kMode, kF32>(idx, s_blk, s_start, G, a, walk, rank, lane, group);
      if (t.nkb == 0) continue;
      const CUtensorMap* map = warp == 0 ? &map_a : &map_b;
      if (kMode == kDw) {
        map = a.maps + (warp == 0 ? 0 : a.E) + t.g;
        if (t.g != last_g) tmap_acquire(map);
        last_g = t.g;
      }
      const bool ok = warp == 0 ? produce_a<kMode>(t, map, rank, stage, phase, sA, lead_full,
                                                   full_bar, empty_bar, abort)
                                : produce_b<kMode>(t, map, &map_b32, rank, stage, phase, sB,
                                                   lead_full, full_bar, empty_bar, abort);
      if (!ok) {
        x_timeout(a.status, abort);
        break;
      }
    }
    // Every commit of a stage that was filled arrives in this CTA's barriers before it may leave
    // (a stage never filled passes at once).
    volatile int never = 0;
    for (int i = 0; i < kXStages; ++i) {
      mbar_wait<true>(&empty_bar[stage], phase ^ 1u, &never);
      if (++stage == kXStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 1) {
    if (lead) {
      // ------------------------------------------------------------ MMA issuer (first CTA)
      // The whole warp walks the tiles; one thread issues.
      int stage = 0, acc = 1;
      uint32_t phase = 0, acc_phase = 0;   // bit `acc`: of that accumulator's barriers
      bool ok = true;
      const uint64_t da0 = kMode == kFwd ? sdesc_k_major(smem_u32(sA), 128)
                                         : sdesc_mn_major(smem_u32(sA), kXSlotBytes / 2);
      const uint64_t db0 = kMode == kDw ? sdesc_mn_major(smem_u32(sB), kXSlotBytes / 2)
                                        : sdesc_k_major(smem_u32(sB), 128);
      for (int idx = first; idx < total; idx += step) {
        const Tile t = decode_tile<kMode, kF32>(idx, s_blk, s_start, G, a, walk, 0, lane, group);
        acc ^= 1;
        if (t.nkb == 0) continue;
        ok = __all_sync(0xffffffffu, mbar_wait<true>(&tempty_bar[acc], ~(acc_phase >> acc) & 1u, abort));
        if (ok) {
          tc_fence_after();
          const uint32_t idesc = idesc_16bit_f32(256, t.n, a.f16 != 0, kMode != kFwd, kMode == kDw);
          ok = multiply_tile<kMode>(tmem_base + acc * kXAccCols, idesc, t.nks, stage, phase, da0,
                                    db0, full_bar, empty_bar, abort);
        }
        if (!ok) {
          x_timeout(a.status, abort);
          break;
        }
        if (elect_one()) umma_commit_pair(&tfull_bar[acc], kXPairMask);
        __syncwarp();
        acc_phase ^= 1u << acc;
      }
      if (!ok) {
        // Every MMA issued so far ends (bounded wait) before TMEM is released.
        if (elect_one()) umma_commit_pair(&drain_bar, 0x1);
        volatile int never = 0;
        mbar_wait(&drain_bar, 0, &never);
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue (both CTAs)
    // Tile i of the pair has accumulator i % 2, which one set of four warps reads: a set's latency
    // from one tile to its next has two tiles' time.
    const int q = warp & 3;   // TMEM lane quarter of this warp
    const int acc = (warp - 2) >> 2;
    uint8_t* my_box = sOut + (warp - 2) * kXBoxBytes;
    const uint32_t tb = tmem_base + acc * kXAccCols + (static_cast<uint32_t>(q * 32) << 16);
    int sbuf = 0;
    uint32_t acc_phase = 0;
    for (int idx = first + acc * step; idx < total; idx += 2 * step) {
      const Tile t = decode_tile<kMode, kF32>(idx, s_blk, s_start, G, a, walk, rank, lane, group);
      const bool zeros = t.nkb == 0;   // nothing was multiplied
      if (zeros && kMode == kDw && kF32 && a.add) continue;
      if (!zeros) {
        const bool got = mbar_wait<true>(&tfull_bar[acc], acc_phase, abort);
        // Lanes may leave the poll at different times; tcgen05.ld is warp-collective.
        if (!__all_sync(0xffffffffu, got)) {
          x_timeout(a.status, abort);
          break;
        }
        tc_fence_after();
        acc_phase ^= 1u;
      }
      auto done = [&] {
        if (zeros) return;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (lead) mbar_arrive(&tempty_bar[acc]);
          else mbar_arrive_relaxed(lead_tempty + 8u * acc);
        }
      };
      if constexpr (kMode == kDw && !kF32) {
        if (!(a.n_ext & 8)) store_dw<false>(tb, t, q, lane, my_box, &map_out, a, done);
        else if (zeros) store_dw_zeros(t, q, lane, a);
        else store_dw_odd(tb, t, q, lane, my_box, a, done);
      } else if constexpr (kMode == kDw)
        store_dw<true>(tb, t, q, lane, my_box, &map_out, a, done);
      else if constexpr (kF32)
        store_part(tb, t, q, lane, a, done);
      else
        store_rows(tb, t, q, lane, my_box, sbuf, &map_out, a, done);
    }
    // Every TMA store of this warp has written its box before the CTA ends.
    if (lane == 0) bulk_wait_group<0>();
  }

  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kXTmemCols);   // collective with the other CTA's warp 1
  }
  // No CTA leaves while the other may still write into it or arrive on its barriers.
  cluster_sync();
}

// A wait of the kernel above for a barrier that nothing arrives on, in a call without a workspace.
__global__ void __launch_bounds__(32) experts_wait_selftest_kernel() {
  __shared__ uint64_t bar;
  __shared__ int s_abort;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  __syncwarp();
  volatile int* abort = &s_abort;
  if (!__all_sync(0xffffffffu, mbar_wait(&bar, 0, abort))) x_timeout(nullptr, abort);
}

// The maps of dw: for each expert, dy's and x's map with the row count cut off at the expert's
// last row. One warp a map. Also clears the status word.
__global__ void __launch_bounds__(256)
experts_maps_kernel(const __grid_constant__ CUtensorMap map_dy,
                    const __grid_constant__ CUtensorMap map_x, const int32_t* __restrict__ offsets,
                    int E, int R, CUtensorMap* maps, int32_t* status) {
  __shared__ __align__(128) CUtensorMap s_map[8];
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + warp;   // [0, E): dy's, [E, 2E): x's
  const uint32_t* src = reinterpret_cast<const uint32_t*>(i < E ? &map_dy : &map_x);
  reinterpret_cast<uint32_t*>(&s_map[warp])[lane] = src[lane];
  __syncwarp();
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x < 4) status[threadIdx.x] = 0;
  if (i >= 2 * E) return;
  const int g = i < E ? i : i - E;
  // The expert's end as the product's kernel has it: no less than any offset before it.
  int end = 0;
  for (int j = lane; j <= g + 1; j += 32) end = max(end, clamp_int(offsets[j], 0, R));
  end = max(__reduce_max_sync(0xffffffffu, end), 1);   // (an extent of 0 is none; no rows, no load)
  if (lane == 0) tmap_set_extent<1>(&s_map[warp], static_cast<uint32_t>(end));
  __syncwarp();
  tmap_publish(maps + i, &s_map[warp]);
}

// A tensor map of a 16-bit or f32 tensor [planes, rows, cols] (cols contiguous; planes 0: a
// matrix), boxes of box_cols x box_rows, swizzled by `swizzle`.
bool encode_any(CUtensorMap* m, const void* base, uint64_t planes, uint64_t rows, uint64_t cols,
                CUtensorMapDataType type, uint32_t box_cols, uint32_t box_rows,
                CUtensorMapSwizzle swizzle) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const uint64_t eb = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
  cuuint64_t dims[3] = {cols, rows, planes};
  cuuint64_t strides[2] = {cols * eb, rows * cols * eb};
  cuuint32_t box[3] = {box_cols, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, type, planes ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The shared-memory opt-in of a kernel form and how many of its clusters can be resident, found
// once a device (published after the attribute is set; a second thread does the same again).
template <int kMode, bool kF32>
moe_status prepare_form(int* max_clusters) {
  static std::atomic<int> clusters_dev[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return set_error(MOE_ERR_CUDA, "cudaGetDevice failed");
  int have = clusters_dev[dev].load(std::memory_order_acquire);
  if (!have) {
    const cudaError_t e =
        cudaFuncSetAttribute(experts_matmul_kernel<kMode, kF32>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kXSmemBytes);
    if (e != cudaSuccess)
      return set_error(MOE_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    const int sms = device_sm_count();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (sms / 2), 1, 1);
    cfg.blockDim = dim3(kXThreads, 1, 1);
    cfg.dynamicSmemBytes = kXSmemBytes;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, experts_matmul_kernel<kMode, kF32>, &cfg) != cudaSuccess ||
        n < 1) {
      cudaGetLastError();   // clear the failed query; fall back to one cluster per SM pair
      n = sms / 2;
    }
    clusters_dev[dev].store(n, std::memory_order_release);
    have = n;
  }
  *max_clusters = have;
  return MOE_OK;
}

template <int kMode, bool kF32>
moe_status launch_form(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mb32,
                       const CUtensorMap& mo, const ExpertsArgs& a, int64_t tiles, cudaStream_t s) {
  int clusters = 1;
  const moe_status st = prepare_form<kMode, kF32>(&clusters);
  if (st != MOE_OK) return st;
  if (clusters > tiles) clusters = static_cast<int>(tiles);
  const cudaError_t err =
      launch_pdl(experts_matmul_kernel<kMode, kF32>, dim3(2 * static_cast<unsigned>(clusters)),
                 dim3(kXThreads), kXSmemBytes, s, ma, mb, mb32, mo, a);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "experts_matmul launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

CUtensorMapDataType map_type(int dtype) {
  return dtype == MOE_DTYPE_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
         : dtype == MOE_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// out[i] (+)= the sum of the parts' i-th values, in order; 8 values a thread.
template <typename T>
__global__ void __launch_bounds__(256)
sum_parts_kernel(const float* __restrict__ part, int parts, int64_t n, T* __restrict__ out,
                 bool add) {
  pdl_trigger();
  pdl_wait();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256 * 8;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8; i < n; i += stride) {
    float sum[8] = {};
    for (int p = 0; p < parts; ++p) {
      const float4* src = reinterpret_cast<const float4*>(part + p * n + i);
      const float4 a = __ldg(src), b = __ldg(src + 1);
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += v[j];
    }
    constexpr int kN = 16 / static_cast<int>(sizeof(T));
    uint4* dst = reinterpret_cast<uint4*>(out + i);
#pragma unroll
    for (int h = 0; h < 8 / kN; ++h) {
      float f[kN], old[kN] = {};
      if (add) Vec<T, 16>::unpack(dst[h], old);
#pragma unroll
      for (int j = 0; j < kN; ++j) f[j] = old[j] + sum[h * kN + j];
      dst[h] = Vec<T, 16>::pack(f);
    }
  }
}

moe_status launch_sum_parts(const float* part, int parts, int64_t n, int dtype, bool add, void* out,
                            cudaStream_t s) {
  const int64_t blocks = (n / 8 + 255) / 256, cap = static_cast<int64_t>(device_sm_count()) * 8;
  const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap)), block(256);
  const cudaError_t err =
      dtype == MOE_DTYPE_F32 ? launch_pdl(sum_parts_kernel<float>, grid, block, 0, s, part, parts, n,
                                          static_cast<float*>(out), add)
      : dtype == MOE_DTYPE_F16 ? launch_pdl(sum_parts_kernel<__half>, grid, block, 0, s, part, parts,
                                            n, static_cast<__half*>(out), add)
                               : launch_pdl(sum_parts_kernel<__nv_bfloat16>, grid, block, 0, s, part,
                                            parts, n, static_cast<__nv_bfloat16*>(out), add);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "sum_parts launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

size_t to_128(size_t n) { return (n + 127) / 128 * 128; }

}  // namespace

moe_status experts_timeout_word(void** word) {
  const cudaError_t e = cudaGetSymbolAddress(word, g_experts_timeouts);
  return e == cudaSuccess ? MOE_OK
                          : set_error(MOE_ERR_CUDA, "cudaGetSymbolAddress: %s", cudaGetErrorString(e));
}

moe_status launch_experts_wait_selftest(cudaStream_t s) {
  experts_wait_selftest_kernel<<<1, 32, 0, s>>>();
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MOE_OK
                          : set_error(MOE_ERR_CUDA, "self-test launch: %s", cudaGetErrorString(e));
}

int experts_split(int product, int64_t R, int E, int N, int K) {
  const int64_t pairs = device_sm_count() / 2;
  int64_t tiles, blocks;
  if (product == kDw) {
    tiles = static_cast<int64_t>(E) * ((N + 255) / 256) * ((K + 255) / 256);
    blocks = R / E / kXBK;
  } else {
    const int cols = product == kDx ? K : N;
    tiles = (R / 256 + (R < E ? R : E)) * ((cols + 255) / 256);
    blocks = (product == kDx ? N : K) / kXBK;
  }
  // Cut only where that takes more off the blocks' 0.28 us each than the 5 us of adding up: 100 rows of
  // one expert (N = 136, K = 14336) 58 us, in eight parts 17; dw of 8192 rows (256 x 4096) 42 us, in
  // four 26; but 2000 rows (256 x 1024, 16 blocks) 11 us, in four 18.
  int split = 0;
  while (split < 3 && (tiles << (split + 1)) <= pairs &&
         blocks >> (split + 1) >= (split == 0 ? 24 : 12))
    ++split;
  return split;
}

size_t experts_workspace_bytes(int E) { return 128 + 2 * static_cast<size_t>(E) * sizeof(CUtensorMap); }

size_t experts_split_bytes(int product, int64_t R, int E, int N, int K) {
  const int split = experts_split(product, R, E, N, K);
  if (split == 0) return 0;
  const int64_t n = product == kDw ? static_cast<int64_t>(E) * N * K
                                   : R * static_cast<int64_t>(product == kDx ? K : N);
  return to_128(experts_workspace_bytes(E)) + (sizeof(float) * n << split);
}

moe_status launch_experts_rows(bool dx, const void* in, const void* w, const int32_t* offsets,
                               int64_t R, int E, int N, int K, int dtype, void* out,
                               char* ws, size_t ws_bytes, cudaStream_t s) {
  const CUtensorMapDataType t = map_type(dtype);
  const int kc = dx ? N : K, nc = dx ? K : N;   // contraction, columns of the result
  CUtensorMap ma, mb, mb32, mo;
  // A, w [E, N, K]: boxes of 64 K x 128 channels (rows of w[e]), or of 64 channels x 64 N. B: boxes
  // of 64 x 128 and 64 x 32 rows.
  const bool ok =
      encode_any(&ma, w, E, N, K, t, 64, dx ? kXBK : 128, CU_TENSOR_MAP_SWIZZLE_128B) &&
      encode_any(&mb, in, 0, R, kc, t, kXBK, 128, CU_TENSOR_MAP_SWIZZLE_128B) &&
      encode_any(&mb32, in, 0, R, kc, t, kXBK, 32, CU_TENSOR_MAP_SWIZZLE_128B) &&
      encode_any(&mo, out, 0, R, nc, t, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (!ok) return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  ExpertsArgs a = {};
  a.offsets = offsets;
  a.E = E;
  a.R = static_cast<int32_t>(R);
  a.m_ext = nc;
  a.k_ext = kc;
  a.f16 = dtype == MOE_DTYPE_F16;
  a.out = out;
  a.status = reinterpret_cast<int32_t*>(ws);
  const int64_t tiles = (R / 256 + E + 2) * ((nc + 255) / 256);
  const size_t need = ws ? experts_split_bytes(dx ? kDx : kFwd, R, E, N, K) : 0;
  if (need > 0 && ws_bytes >= need) {
    a.split = experts_split(dx ? kDx : kFwd, R, E, N, K);
    a.part = reinterpret_cast<float*>(ws + to_128(experts_workspace_bytes(E)));
    const moe_status st = dx ? launch_form<kDx, true>(ma, mb, mb32, mo, a, tiles << a.split, s)
                             : launch_form<kFwd, true>(ma, mb, mb32, mo, a, tiles << a.split, s);
    if (st != MOE_OK) return st;
    return launch_sum_parts(a.part, 1 << a.split, R * nc, dtype, false, out, s);
  }
  return dx ? launch_form<kDx, false>(ma, mb, mb32, mo, a, tiles, s)
            : launch_form<kFwd, false>(ma, mb, mb32, mo, a, tiles, s);
}

moe_status launch_experts_dw(const void* dy, const void* x, const int32_t* offsets, int64_t R,
                             int E, int N, int K, int dtype, int out_dtype, bool add, void* dw,
                             char* ws, size_t ws_bytes, cudaStream_t s) {
  const CUtensorMapDataType t = map_type(dtype);
  const size_t need = experts_split_bytes(kDw, R, E, N, K);
  const int split = need > 0 && ws_bytes >= need ? experts_split(kDw, R, E, N, K) : 0;
  float* part = reinterpret_cast<float*>(ws + to_128(experts_workspace_bytes(E)));
  const bool f32 = split > 0 || out_dtype == MOE_DTYPE_F32;   // what the product's kernel writes
  CUtensorMap ma, mb, mo;
  const bool ok =
      encode_any(&ma, dy, 0, R, N, t, 64, kXBK, CU_TENSOR_MAP_SWIZZLE_128B) &&
      encode_any(&mb, x, 0, R, K, t, 64, kXBK, CU_TENSOR_MAP_SWIZZLE_128B) &&
      (split > 0 ? encode_any(&mo, part, static_cast<uint64_t>(E) << split, N, K,
                              CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B)
                 : encode_any(&mo, dw, E, N, K, map_type(out_dtype), f32 ? 32 : 64, 32,
                              CU_TENSOR_MAP_SWIZZLE_128B));
  if (!ok) return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  ExpertsArgs a = {};
  a.offsets = offsets;
  a.E = E;
  a.R = static_cast<int32_t>(R);
  a.m_ext = N;
  a.n_ext = K;
  a.f16 = dtype == MOE_DTYPE_F16;
  a.out = dw;
  a.add = add && split == 0;
  a.split = split;
  a.status = reinterpret_cast<int32_t*>(ws);
  CUtensorMap* maps = reinterpret_cast<CUtensorMap*>(ws + 128);
  a.maps = maps;
  const cudaError_t err =
      launch_pdl(experts_maps_kernel, dim3((2 * E + 7) / 8), dim3(256), 0, s, ma, mb, offsets, E,
                 a.R, maps, a.status);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "experts_maps launch: %s", cudaGetErrorString(err));
  const int64_t tiles = static_cast<int64_t>(E) * ((N + 255) / 256) * ((K + 255) / 256);
  const moe_status st = f32 ? launch_form<kDw, true>(ma, mb, mb, mo, a, tiles << split, s)
                            : launch_form<kDw, false>(ma, mb, mb, mo, a, tiles, s);
  if (st != MOE_OK || split == 0) return st;
  return launch_sum_parts(part, 1 << split, static_cast<int64_t>(E) * N * K, out_dtype, add, dw, s);
}

}  // namespace moe
