// The experts' forward products over ragged groups of rows with both operands in microscaled 4 bits:
//   y[r, n] = g_x g_w[e] sum over blocks b of sx[r, b] sw[e, n, b] sum over k of b of x[r, k] w[e, n, k]
// for the rows r of expert e, x [R, K] and w [E, N, K] as codes with block scales (fp4.cuh).
//
// tcgen05.mma of block-scaled e2m1 operands takes the scales from TMEM and multiplies 64 elements of the
// contraction an instruction, so that codes go from memory to the tensor cores as they are. One
// persistent kernel over all groups, CTA pairs (M = 256 channels of w, N up to 208 or 224 rows of x, the
// tiles and their order those of the 16-bit products); a block is 256 elements of the contraction, 128
// bytes a row, by TMA with the 128-byte swizzle.
//
// Scales. The instruction wants those of 128 rows by 4 bytes of the contraction as 32 lanes by 4 columns
// (row 32 i + l in lane l, column i), the same in each quarter of TMEM's lanes. A row's scales lie along the
// contraction in memory: they come by TMA as they lie, 16 bytes a row (mx: for two blocks), and four warps, one
// a quarter, read rows l, l + 32, ... and store them to TMEM. Each CTA needs the scales of its 128 channels and of
// all of the tile's rows (the pair shares the rows' codes, but each tensor core scales its own half of D). Bytes
// past the row's K / block are zeros, whatever fills the row up; codes past K are TMA's zeros.
// (Scales written to shared memory for tcgen05.cp, which the first CTA's thread issues for both, would take a
// release by the second's writers to the other SM, 1700 cycles a block: 8192 x 28672 x 4096 over 8 experts
// 815 us, and 425 without it, which PTX does not order. TMEM is handed over by tcgen05.fence instead: 442.)
// TMEM: two accumulators (nv: of 208 columns, mx: 224) and two sets of scales, each written when the products
// of the block two before are done (that a copy into columns that a product before it still reads would wait for
// that is not promised either).
//
// Measured (one GB300, back to back): 8192 rows over 8 experts, N = 28672, K = 4096, nv, 442 us, 4.35
// PFLOP/s, 2.3 times cuBLAS's bf16 rate: 910 cycles a block of 256 x 208 x 256, of which the products take 380;
// what feeds the tensor pipe bounds it (with a quarter of the products 469 us, so 487 then).
// 512 rows over 128 experts, N = 1536, K = 2048, nv, 44 us and 4096 rows over 256 experts, N = 7168,
// K = 2048, mx, 364 us: 5.1 and 5.7 TB/s, bound by memory. A fifth and a seventh block under way, for which
// scales in shared memory left no room, are 3% of the first (452 us with four) and 2% of the last (370 with six).
//
// Warp roles (608 threads per CTA): warps 0 and 18 TMA producers of the weights and of the rows, warp 1 TMEM
// allocator and, in the first CTA, MMA issuer, warps 2-9 scales, in two teams that take a block each in
// turn, warps 10-17 epilogue, four to each accumulator.
#include <atomic>
#include <cstdint>

#include <cuda.h>

#include "experts_tiles.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

constexpr int kQBK = 256;                      // contraction elements a block: 128 bytes
constexpr int kQSlotA = 128 * 128;             // codes of the weights of one block in one CTA

// Wide tiles: as many rows as TMEM has room for. Narrow ones, for launches of few rows an expert: up to 64, with
// more blocks of weights under way instead.
template <bool kNv, bool kWide>
struct QTile {
  static constexpr int kMost = !kWide ? 64 : kNv ? 208 : 224;    // rows of a tile
  static constexpr int kStages = kWide ? 5 : 7;
  static constexpr int kSlotB = (kWide ? 128 : 32) * 128;        // codes of half of the rows
  static constexpr int kRawBytes = (kWide ? 3 : 2) * 128 * 16;   // scales as they lie: A's 128 rows, B's
  static constexpr int kStage = kQSlotA + kSlotB + kRawBytes;
  static constexpr int kWords = kNv ? 4 : 2;                     // of scales, of a row in a block
  static constexpr int kPitchB = kWide ? 8 : 4;                  // columns a word of up to 256 or 128 rows
  static constexpr int kColsA = 4 * kWords, kColsB = kPitchB * kWords;
  static constexpr int kScales = 2 * kMost, kSet = kColsA + kColsB;   // first TMEM column, of a set
  static_assert(kScales + 2 * kSet <= 512, "TMEM");
};
constexpr int kQScaleWarp = 2, kQScaleWarps = 4, kQScaleTeams = 2;   // a stage each in turn
constexpr int kQEpiWarp = kQScaleWarp + kQScaleWarps * kQScaleTeams, kQEpiWarps = 8;
constexpr int kQWarpX = kQEpiWarp + kQEpiWarps;   // the producer of the rows
constexpr int kQThreads = 32 * (kQWarpX + 1);
constexpr int kQBoxBytes = 4096;               // epilogue staging of a warp
template <bool kNv, bool kWide>
constexpr int kQSmemBytes = 1024 + QTile<kNv, kWide>::kStages * QTile<kNv, kWide>::kStage + kQEpiWarps * kQBoxBytes;
static_assert(kQSmemBytes<false, true> <= 232448 - 2048 && kQSmemBytes<false, false> <= 232448 - 2048, "shared memory");
constexpr int kQTmemCols = 512;
static_assert(kQScaleTeams == 2 && kQScaleWarps == 4, "a team a set of scales, a warp a quarter of TMEM");
constexpr uint16_t kQPairMask = 0x3;
constexpr int kQNarrowRows = 16;

struct Fp4Args {
  ExpertsArgs e;
  const float* x_g;          // or NULL
  const float* w_g;          // [E] or NULL
  int blocks;                // scale bytes of a row
};

__device__ int32_t g_fp4_timeouts;

__device__ __forceinline__ void q_timeout(volatile int* abort) {
  *abort = 1;
  atomicOr(&g_fp4_timeouts, MOE_DEVICE_FLAG_TIMEOUT);
}

// Two factors whose product is a b, where f32 does not hold that: each with half of the exponent. (A sum is 0 or
// between 2^-20 and 2^39, so that from 2^250 or 2^-250 on the result is past f32's range either way.)
__device__ __noinline__ void split_gain(float a, float b, float& gain, float& rest) {
  int ea, eb;
  const float m = frexpf(a, &ea) * frexpf(b, &eb);
  const int e = max(-250, min(250, ea + eb)), half = e / 2;
  gain = ldexpf(m, half);
  rest = ldexpf(1.0f, e - half);
}

// D (+)= A B^T of the pair, 64 elements of the contraction of e2m1 with scales in TMEM.
template <bool kNv>
__device__ __forceinline__ void umma_fp4_pair(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc,
                                              uint32_t sa, uint32_t sb, uint32_t accumulate) {
  if constexpr (kNv)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}\n" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], "
        "p;\n\t}\n" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}

// kind::mxf4 and mxf4nvf4: A and B e2m1 (1 at bits 7-9 and 10-11), K-major, N >> 3 at bits 17-22, the
// scales' type at bit 23 (0 e4m3, 1 powers of two), M >> 4 at bits 24-28; which of a word's two halves
// holds the scales of a step of two blocks: bits 29-30 (A) and 4-5 (B).
template <bool kNv>
__device__ __forceinline__ uint32_t idesc_fp4(int N) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | ((kNv ? 0u : 1u) << 23) |
         (static_cast<uint32_t>(256 >> 4) << 24);
}

template <bool kNv, bool kWide>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kQThreads, 1)
experts_fp4_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                   const __grid_constant__ CUtensorMap map_x32,
                   const __grid_constant__ CUtensorMap map_ws, const __grid_constant__ CUtensorMap map_xs,
                   const __grid_constant__ CUtensorMap map_out, Fp4Args q) {
  using Q = QTile<kNv, kWide>;
  constexpr int kQStages = Q::kStages, kQMost = Q::kMost;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[kQStages], raw_bar[kQStages], read_bar[kQStages], scale_bar[kQStages];
  __shared__ uint64_t empty_bar[kQStages];
  __shared__ uint64_t tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;
  __shared__ uint16_t s_blk[kXGroups + 1];
  __shared__ int32_t s_start[kXGroups + 1];

  const ExpertsArgs& a = q.e;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool lead = rank == 0;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sA = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  uint8_t* sB = sA + kQStages * kQSlotA;
  uint8_t* sRaw = sB + kQStages * Q::kSlotB;
  uint8_t* sOut = sRaw + kQStages * Q::kRawBytes;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kQStages; ++s) {
      mbar_init(&full_bar[s], 2);                    // first CTA: its two producers, and both CTAs' bytes
      mbar_init(&raw_bar[s], 2);                     // this CTA's scales, as they lie
      mbar_init(&read_bar[s], kQScaleWarps);         // they have been read
      mbar_init(&scale_bar[s], 2 * kQScaleWarps);    // first CTA: both CTAs' scale warps
      mbar_init(&empty_bar[s], 1);                   // the pair commit, delivered to both CTAs
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull_bar[s], 1);
      mbar_init(&tempty_bar[s], kQEpiWarps);         // first CTA: four epilogue warps of each CTA
    }
    mbar_init(&drain_bar, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&map_w);
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_x32);
    tma_prefetch_map(&map_ws);
    tma_prefetch_map(&map_xs);
    tma_prefetch_map(&map_out);
  }
  if (warp == 1) {
    tmem_alloc_pair(&s_tmem_base, kQTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any remote arrival or copy
  tc_fence_after();
  pdl_wait();
  const int G = a.E + 2;
  if (warp == 2) scan_groups<kFwd, kQMost>(a, lane, s_blk, s_start);
  __syncthreads();
  const uint32_t tmem_base = s_tmem_base;
  volatile int* abort = &s_abort;
  const Walk walk = Walk::of<kFwd>(a);
  const int total = walk.inner.d * s_blk[G];
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const uint32_t lead_full = mapa_shared(smem_u32(&full_bar[0]), 0);
  const uint32_t lead_scale = mapa_shared(smem_u32(&scale_bar[0]), 0);
  const uint32_t lead_tempty = mapa_shared(smem_u32(&tempty_bar[0]), 0);
  const int nkb = (a.k_ext + kQBK - 1) / kQBK;       // blocks and instructions of a tile
  const int nks = (a.k_ext + 63) / 64;

  int group = 0;   // of this warp's last tile
  auto tile = [&](int idx) {
    return decode_tile<kFwd, false, kQMost>(idx, s_blk, s_start, G, a, walk, rank, lane, group);
  };
  if (warp == 0 || warp == kQWarpX) {
    // ------------------------------------------------------------ TMA producers of the weights and of the rows
    // (One warp for both took 410 cycles a block, as much as the products of 208 rows.)
    const bool weights = warp == 0;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int idx = first; idx < total && ok; idx += step) {
      const Tile t = tile(idx);
      if (t.nkb == 0) continue;
      const int half = t.n >> 1;
      // (narrow tiles: half is 32 at most)
      const bool narrow = !kWide || half <= 64;
      const int box = narrow ? 32 : 128;
      const bool two = kWide && half > box;
      const CUtensorMap* mx = narrow ? &map_x32 : &map_x;
      const uint32_t tx = weights ? kQSlotA * ((t.m_here > 0) + (t.m_peer > 0)) : 2 * (two ? 2 : 1) * box * 128;
      const int n0 = t.n0 + rank * half;
      for (int kb = 0; kb < nkb; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait<true>(&empty_bar[stage], phase ^ 1u, abort) &&
                                         mbar_wait(&read_bar[stage], phase ^ 1u, abort));
        if (!ok) break;
        if (elect_one()) {
          if (lead) mbar_arrive_expect_tx(&full_bar[stage], tx);
          const uint32_t fb = lead_full + 8u * stage;
          uint8_t* bs = sB + stage * Q::kSlotB;
          uint8_t* raw_s = sRaw + stage * Q::kRawBytes;
          const int at = kNv ? kb * 16 : (kb >> 1) * 16;   // (mx: this block's half of it is kb's lowest bit)
          if (weights) {
            mbar_arrive_expect_tx(&raw_bar[stage], 128 * 16);
            tma_load_3d(raw_s, &map_ws, &raw_bar[stage], at, t.m0, t.g);
            if (t.m_here > 0)
              tma_load_3d_pair(sA + stage * kQSlotA, &map_w, fb, kb * 128, t.m0, t.g);
          } else {
            mbar_arrive_expect_tx(&raw_bar[stage], (kWide && t.n > 128 ? 2 : 1) * 128 * 16);
            tma_load_2d(raw_s + 128 * 16, &map_xs, &raw_bar[stage], at, t.n0);
            if (kWide && t.n > 128) tma_load_2d(raw_s + 256 * 16, &map_xs, &raw_bar[stage], at, t.n0 + 128);
            tma_load_2d_pair(bs, mx, fb, kb * 128, n0);
            if (two) tma_load_2d_pair(bs + 32 * 128, mx, fb, kb * 128, n0 + 32);
          }
        }
        __syncwarp();
        if (++stage == kQStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) q_timeout(abort);
    // Every commit of a stage that was filled arrives in this CTA's barriers before it may leave.
    volatile int never = 0;
    for (int i = 0; i < kQStages; ++i) {
      mbar_wait<true>(&empty_bar[stage], phase ^ 1u, &never);
      if (++stage == kQStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 1) {
    if (lead) {
      // ------------------------------------------------------------ MMA issuer (first CTA)
      int stage = 0, acc = 1, set = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      const uint64_t da0 = sdesc_k_major(smem_u32(sA), 128), db0 = sdesc_k_major(smem_u32(sB), 128);
      for (int idx = first; idx < total; idx += step) {
        const Tile t = tile(idx);
        acc ^= 1;
        if (t.nkb == 0) continue;
        ok = __all_sync(0xffffffffu, mbar_wait<true>(&tempty_bar[acc], ~(acc_phase >> acc) & 1u, abort));
        if (ok) tc_fence_after();
        const uint32_t idesc = idesc_fp4<kNv>(t.n), d = tmem_base + acc * kQMost;
        for (int ks = 0; ok && ks < nks; ks += 4) {
          ok = __all_sync(0xffffffffu, mbar_wait<true>(&full_bar[stage], phase, abort) &&
                                           mbar_wait<true>(&scale_bar[stage], phase, abort));
          if (!ok) break;
          tc_fence_after();
          const uint64_t da = da0 + ((stage * kQSlotA) >> 4), db = db0 + ((stage * Q::kSlotB) >> 4);
          const uint32_t sfa = tmem_base + Q::kScales + set * Q::kSet, sfb = sfa + Q::kColsA;
          set ^= 1;
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (ks + i >= nks) break;
              const int j = kNv ? i : i / 2;
              const uint32_t part = kNv ? 0u : static_cast<uint32_t>(i & 1) * 2u;
              umma_fp4_pair<kNv>(d, da + i * 2, db + i * 2, idesc | part << 29 | part << 4, sfa + 4 * j,
                                 sfb + Q::kPitchB * j, (ks | i) != 0);
            }
            umma_commit_pair(&empty_bar[stage], kQPairMask);
          }
          __syncwarp();
          if (++stage == kQStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) {
          q_timeout(abort);
          break;
        }
        if (elect_one()) umma_commit_pair(&tfull_bar[acc], kQPairMask);
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
  } else if (warp < kQEpiWarp) {
    // ------------------------------------------------------------ scales (both CTAs)
    // Block by block in turn, a team's always with the same set of columns.
    constexpr int kWords = Q::kWords;
    const int team = (warp - kQScaleWarp) / kQScaleWarps;
    const uint32_t ts = tmem_base + Q::kScales + team * Q::kSet + (static_cast<uint32_t>(warp & 3) << 21);
    // Word j of rows lane, lane + 32, ... to registers j * pitch + i, what is past the rows' ends as zeros.
    auto words = [&](const uint8_t* rows, int n, int pitch, int kb, uint32_t* out) {
      const int left = q.blocks - kb * 4 * kWords;   // bytes that are scales
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const uint8_t* src = rows + (32 * i + lane) * 16;
        uint32_t w[kWords];
        if constexpr (kNv) {
          const uint4 v = *reinterpret_cast<const uint4*>(src);
          w[0] = v.x;
          w[1] = v.y;
          w[2] = v.z;
          w[3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(src + (kb & 1) * 8);
          w[0] = v.x;
          w[1] = v.y;
        }
        if (left < 4 * kWords) {
#pragma unroll
          for (int j = 0; j < kWords; ++j) {
            const int m = left - 4 * j;
            if (m < 4) w[j] = m <= 0 ? 0u : w[j] & ((1u << (8 * m)) - 1u);
          }
        }
#pragma unroll
        for (int j = 0; j < kWords; ++j) out[j * pitch + i] = w[j];
      }
    };
    int stage = 0, set = 0, before = -1;             // before: the team's stage before this one
    uint32_t phase = 0, before_phase = 0;
    bool ok = true;
    for (int idx = first; idx < total && ok; idx += step) {
      const Tile t = tile(idx);
      if (t.nkb == 0) continue;
      const bool wide = kWide && t.n > 128;
      for (int kb = 0; kb < nkb; ++kb) {
        if (set == team) {
          ok = __all_sync(0xffffffffu, mbar_wait(&raw_bar[stage], phase, abort));
          if (!ok) break;
          const uint8_t* raw_s = sRaw + stage * Q::kRawBytes;
          uint32_t sa[Q::kColsA], sb[Q::kColsB] = {};
          words(raw_s + 128 * 16, 4, Q::kPitchB, kb, sb);
          if (wide) words(raw_s + 256 * 16, 4, Q::kPitchB, kb, sb + 4);
          // The products that had this set of columns before are done.
          if (before >= 0) {
            ok = __all_sync(0xffffffffu, mbar_wait<true>(&empty_bar[before], before_phase, abort));
            if (!ok) break;
          }
          tc_fence_after();
          tmem_store(ts + Q::kColsA, sb);
          words(raw_s, 4, 4, kb, sa);                // (now: both at once would not fit the registers)
          tmem_store(ts, sa);
          __syncwarp();
          if (lane == 0) mbar_arrive(&read_bar[stage]);
          tmem_store_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_relaxed(lead_scale + 8u * stage);
          before = stage;
          before_phase = phase;
        }
        set ^= 1;
        if (++stage == kQStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) q_timeout(abort);
  } else {
    // -------------------------------------------------------------- epilogue (both CTAs)
    const int quarter = warp & 3;   // TMEM lane quarter of this warp
    const int acc = (warp - kQEpiWarp) >> 2;
    uint8_t* buf = sOut + (warp - kQEpiWarp) * kQBoxBytes;
    const uint32_t tb = tmem_base + acc * kQMost + (static_cast<uint32_t>(quarter * 32) << 16);
    int sbuf = 0;
    uint32_t acc_phase = 0;
    const bool f16 = a.f16 != 0;
    const float gx = q.x_g ? __ldg(q.x_g) : 1.0f;
    for (int idx = first + acc * step; idx < total; idx += 2 * step) {
      const Tile t = tile(idx);
      const bool zeros = t.nkb == 0;
      if (!zeros) {
        const bool got = mbar_wait<true>(&tfull_bar[acc], acc_phase, abort);
        if (!__all_sync(0xffffffffu, got)) {
          q_timeout(abort);
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
      if (32 * quarter >= t.m_here) {
        done();
        continue;
      }
      const float gw = q.w_g && !zeros ? __ldg(q.w_g + t.g) : 1.0f;
      float gain = gx * gw, rest = 1.0f;
      if (!(gain >= 0x1p-126f && gain < INFINITY)) split_gain(gx, gw, gain, rest);
      const int ch = t.m0 + 32 * quarter;
      // 32 channels by 32 rows at a time, as the 16-bit products' epilogue: read in matrix fragments,
      // turned over by the matrix store into a box of 32 rows of 64 bytes, out by TMA.
#pragma unroll 1
      for (int r0 = 0; r0 < t.n_here; r0 += 32) {
        uint32_t v[2][16];
        if (!zeros) {
          tmem_issue_fragments(tb + r0, v[0]);
          tmem_issue_fragments(tb + r0 + (16u << 16), v[1]);
          tmem_wait();
          tmem_ready(v[0]);
          tmem_ready(v[1]);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j >> 4][j & 15] = 0;
        }
        if (r0 + 32 >= t.n_here) done();
        if (rest != 1.0f) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            v[j >> 4][j & 15] = __float_as_uint(rest * __uint_as_float(v[j >> 4][j & 15]));
        }
        uint32_t p[16];   // [channels 8 b .. + 7][rows 8 i .. + 7]: p[4 i + b]
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int b = 0; b < 4; ++b)
            p[4 * i + b] = pack_16bit(gain * __uint_as_float(v[b >> 1][4 * i + 2 * (b & 1)]),
                                      gain * __uint_as_float(v[b >> 1][4 * i + 2 * (b & 1) + 1]), f16);
        uint8_t* box = buf + sbuf * (kQBoxBytes / 2);
        if (lane == 0) bulk_wait_group_read<1>();   // what was stored from this box before is out
        __syncwarp();
        const uint32_t at = smem_u32(box) + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          stmatrix_trans(at + i * 512, p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
        const int rows = t.n_here - r0;
        if (rows < 32) {
          __syncwarp();
          const int c = lane & 3;   // chunk of 8 channels; m_ext is a multiple of 8
          if (32 * quarter + 8 * c < t.m_here) {
            uint16_t* dst = static_cast<uint16_t*>(a.out) +
                            static_cast<int64_t>(t.n0 + r0) * a.m_ext + ch + 8 * c;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 8 * i + (lane >> 2);
              if (r < rows)
                *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(r) * a.m_ext) =
                    *reinterpret_cast<const uint4*>(box + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
            }
          }
          break;   // a tile's last box
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&map_out, box, ch, t.n0 + r0);
          bulk_commit_group();
        }
        sbuf ^= 1;
      }
    }
    if (lane == 0) bulk_wait_group<0>();
  }

  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kQTmemCols);
  }
  // No CTA leaves while the other may still write into it or arrive on its barriers.
  cluster_sync();
}

// A wait of the kernel above for a barrier that nothing arrives on.
__global__ void __launch_bounds__(32) fp4_wait_selftest_kernel() {
  __shared__ uint64_t bar;
  __shared__ int s_abort;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  __syncwarp();
  volatile int* abort = &s_abort;
  if (!__all_sync(0xffffffffu, mbar_wait<true>(&bar, 0, abort))) q_timeout(abort);
}

// Bytes [planes, rows, cols] (planes 0: a matrix), boxes of 128 (with the 128-byte swizzle) or 16 by box_rows.
bool encode_bytes(CUtensorMap* m, const void* base, uint64_t planes, uint64_t rows, uint64_t cols,
                  uint32_t box_cols, uint32_t box_rows) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {cols, rows, planes};
  cuuint64_t strides[2] = {cols, rows * cols};
  cuuint32_t box[3] = {box_cols, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, planes ? 3 : 2, const_cast<void*>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_cols == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kNv, bool kWide>
moe_status launch_fp4(const CUtensorMap& mw, const CUtensorMap& mx, const CUtensorMap& mx32,
                      const CUtensorMap& mws, const CUtensorMap& mxs, const CUtensorMap& mo,
                      const Fp4Args& q, int64_t tiles, cudaStream_t s) {
  static std::atomic<int> clusters_dev[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return set_error(MOE_ERR_CUDA, "cudaGetDevice failed");
  int have = clusters_dev[dev].load(std::memory_order_acquire);
  if (!have) {
    const cudaError_t e = cudaFuncSetAttribute(
        experts_fp4_kernel<kNv, kWide>, cudaFuncAttributeMaxDynamicSharedMemorySize, kQSmemBytes<kNv, kWide>);
    if (e != cudaSuccess)
      return set_error(MOE_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    const int sms = device_sm_count();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (sms / 2), 1, 1);
    cfg.blockDim = dim3(kQThreads, 1, 1);
    cfg.dynamicSmemBytes = kQSmemBytes<kNv, kWide>;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, experts_fp4_kernel<kNv, kWide>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();   // clear the failed query; fall back to one cluster per SM pair
      n = sms / 2;
    }
    clusters_dev[dev].store(n, std::memory_order_release);
    have = n;
  }
  const unsigned pairs = static_cast<unsigned>(have < tiles ? have : tiles);
  const cudaError_t err = launch_pdl(experts_fp4_kernel<kNv, kWide>, dim3(2 * pairs), dim3(kQThreads),
                                     kQSmemBytes<kNv, kWide>, s, mw, mx, mx32, mws, mxs, mo, q);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "experts_fp4 launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

}  // namespace

moe_status fp4_timeout_word(void** word) {
  const cudaError_t e = cudaGetSymbolAddress(word, g_fp4_timeouts);
  return e == cudaSuccess ? MOE_OK
                          : set_error(MOE_ERR_CUDA, "cudaGetSymbolAddress: %s", cudaGetErrorString(e));
}

moe_status launch_fp4_wait_selftest(cudaStream_t s) {
  fp4_wait_selftest_kernel<<<1, 32, 0, s>>>();
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MOE_OK
                          : set_error(MOE_ERR_CUDA, "self-test launch: %s", cudaGetErrorString(e));
}

moe_status launch_experts_fp4(const Fp4Operand& x, const Fp4Operand& w, const int32_t* offsets, int64_t R,
                              int E, int N, int K, int fmt, int dtype, void* y, cudaStream_t s) {
  CUtensorMap mw, mx, mx32, mws, mxs, mo;
  const int pitch = fp4_scale_pitch(K, fmt);
  EncodeTiledFn enc = get_encode_fn();
  bool ok = enc && encode_bytes(&mw, w.codes, E, N, K / 2, 128, 128) &&
            encode_bytes(&mx, x.codes, 0, R, K / 2, 128, 128) &&
            encode_bytes(&mx32, x.codes, 0, R, K / 2, 128, 32) &&
            encode_bytes(&mws, w.scales, E, N, pitch, 16, 128) && encode_bytes(&mxs, x.scales, 0, R, pitch, 16, 128);
  if (ok) {
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(R)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(N) * 2};
    cuuint32_t box[2] = {32, 32}, estr[2] = {1, 1};
    ok = enc(&mo, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, y, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  if (!ok) return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  Fp4Args q = {};
  q.e.offsets = offsets;
  q.e.E = E;
  q.e.R = static_cast<int32_t>(R);
  q.e.m_ext = N;
  q.e.k_ext = K;
  q.e.f16 = dtype == MOE_DTYPE_F16;
  q.e.out = y;
  q.x_g = x.g;
  q.w_g = w.g;
  q.blocks = K / fp4_block(fmt);
  // Wide tiles where the experts have more than 16 rows on average (an expert of more than 64 rows reads its
  // weights again for every narrow tile). N = 7168, K = 2048, mx, 256 experts of 8, 16, 32, 48 rows on average,
  // all alike: narrow 411, 370, 343, 342 us, wide 435, 387, 356, 355; spread log-normally, sigma 1: narrow 398, 389,
  // 397, 437, wide 415, 401, 377, 378; as 1 / rank, an expert having a row of each token at most, eight a token:
  // narrow 464, 443, 441, 482, wide 474, 436, 416, 421. N = 1536, nv, 128 experts of 4, 16, 32: all alike narrow
  // 45, 42, 43, wide 47, 44, 45; log-normally 38, 42, 46 and 40, 43, 46.
  const bool wide = R > static_cast<int64_t>(kQNarrowRows) * E;
  const int most = !wide ? QTile<true, false>::kMost : fmt == kFp4Nv ? QTile<true, true>::kMost : QTile<false, true>::kMost;
  const int64_t tiles = (R / most + E + 2) * ((N + 255) / 256);
  if (wide)
    return fmt == kFp4Nv ? launch_fp4<true, true>(mw, mx, mx32, mws, mxs, mo, q, tiles, s)
                         : launch_fp4<false, true>(mw, mx, mx32, mws, mxs, mo, q, tiles, s);
  return fmt == kFp4Nv ? launch_fp4<true, false>(mw, mx, mx32, mws, mxs, mo, q, tiles, s)
                       : launch_fp4<false, false>(mw, mx, mx32, mws, mxs, mo, q, tiles, s);
}

}  // namespace moe
