// Rows to and from microscaled 4-bit floating point, and SwiGLU whose result is held so.
//
//   quantise    v = x [R, K]
//   SwiGLU      v = g sigma(g) u of gu [R, 2K], gate then up; never rounded to 16 bits
//   mx          byte = e + 127, e the least integer >= -127 with amax <= 6 * 2^e
//   nv          byte = e4m3(amax / (6 g)), to nearest even, 448 at most; a block that rounds to 0 is zeros
//   code        e2m1(v / (scale [g])), to nearest even
// A block that holds an infinity or a NaN gets the scale NaN and codes 0.
//
// What is rounded is decided as on exact numbers. In f32 the quotients (mx: exact; nv: a few units off) and
// SwiGLU decide otherwise only where a value lies within its error of the border between two codes or
// two scale bytes. So codes and bytes are made of the value a little less and a little more; where
// the two differ, the border itself is compared: for values that are given, with the products of the
// border, the scale and g in two f32 numbers, which is exact (such cases are common: the quotient of two
// 8-bit mantissas is often a tie but for g's rounding); for SwiGLU, a few times in a million, the
// segment is worked out again in pairs of f32 (2^-26), and where that does not do either, in 64 bits.
//
// Every value is read and written once, 4.25 or 4.5 bits out for 16 in, or for 32 (SwiGLU). Bound by
// instructions, hence lanes of 16 channels, two products an instruction, and a border only looked at where
// two codes differ. Measured, bf16: SwiGLU of 8192 x 14336 to mx 91 us (532 MB at 5.8 TB/s; lanes of 8 109,
// and with one product an instruction 120), to nv 106; 8192 x 7168 to mx 26, to nv 37 (lanes of 8: 32 and 51);
// back, 8192 x 14336, 56. (At the registers of that many blocks an SM to nv spills 60 bytes a thread, SwiGLU by 16
// 68 and 128.) All in 64 bits where f32 is in doubt: 8192 x 7168 to nv 1.06 ms (ties are common
// there), SwiGLU of 512 x 768 to nv 15 us, so 3.
#include <cstdint>

#include <cuda_fp8.h>

#include "fp4.cuh"
#include "launch.cuh"
#include "pairs.cuh"
#include "segments.cuh"

namespace moe {
namespace {

// Relative widths around a value in which its f32 form may be. A quotient: the divisor's rounding and the
// reciprocal's (2), the product's and that of the factor 1 -+ kNear, 3.5 units of 2^-23. SwiGLU (16-bit and
// f32 rows alike): 2 + 0.75 |gate| units of the exponential (its argument's rounding and log2 e's), 1.5 of
// the sum and its reciprocal, 1 of the products, then the quotient's. SwiGLU in pairs: under 2^-27.
constexpr float kNearQuotient = 0x1p-21f;
constexpr float kNearSwiglu = 1e-6f, kNearGate = 1.5e-7f;
constexpr float kNearPairs = 0x1p-26f;
// SwiGLU of fewer values goes by lanes of 8: a segment that has to be worked out again takes a lane of 16
// twice as long, which shows where a warp has few segments. bf16, K = 2048, mx, 512, 2048, 4096, 8192 rows:
// lanes of 8 4.3, 8.2, 13.4, 20.6 us, of 16 5.5, 9.1, 13.0, 20.9; 8192 x 14336 109 and 93, nv 136 and 106.
// (f32, whose values fill the registers, always by 8: 152 us, by 16 163.)
constexpr int64_t kFewValues = int64_t{1} << 23;
// These hold where no product on the way leaves f32's normal numbers by much: for gates from kLeastGate on
// (or 0) and results from kLeastValue on, as blocks' largest. (bf16's 8 bits survive sigma of a smaller gate.)
constexpr float kLeastGate = 0x1p-100f, kLeastValue = 0x1p-90f;

struct Fp4Out {
  uint8_t* codes;       // [R, K / 2]
  uint8_t* scales;      // [R, pitch]
  const float* g;       // nv: g of each plane of rows_per_plane rows, or NULL (1)
  int64_t rows_per_plane;
};

template <int kLanes>
__device__ __forceinline__ float lanes_max(float v) {
  // Magnitudes order as their bit patterns do, infinities and NaNs on top.
  uint32_t m = __float_as_uint(v);
#pragma unroll
  for (int d = 1; d < kLanes; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return __uint_as_float(m);
}

// 1 / x to 2^-23, 0 past f32's normal numbers.
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^x to 2^-22, 0 below f32's normal numbers.
__device__ __forceinline__ float power_of_2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// N values times f.
template <int N>
__device__ __forceinline__ void times_all(const float (&v)[N], float f, float (&out)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const uint64_t r = times(two(v[i], v[i + 1]), two(f, f));
    out[i] = first(r);
    out[i + 1] = second(r);
  }
}

// N channels as they lie in memory.
template <int N, typename T>
__device__ __forceinline__ void load_all(const T* p, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    float part[8];
    load8(p + i, part);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i + j] = part[j];
  }
}
template <int N>
struct alignas(N / 2) Fp4Codes {
  uint32_t word[N / 8];
};
template <int N>
__device__ __forceinline__ Fp4Codes<N> codes_of(const float (&f)[N]) {
  Fp4Codes<N> r;
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    float part[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) part[j] = f[i + j];
    r.word[i / 8] = fp4_codes8(part);
  }
  return r;
}

// The least e >= -127 with amax <= 6 * 2^e = 1.5 * 2^(e + 2), as a byte; finite amax.
__device__ __forceinline__ uint32_t mx_byte(float amax) {
  const int e = static_cast<int>((__float_as_uint(amax) + 0x003fffffu) >> 23) - 2;
  return static_cast<uint32_t>(e > 0 ? e : 0);
}
__device__ __forceinline__ float mx_scale(uint32_t byte) {   // 2^(byte - 127)
  return byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}
__device__ __forceinline__ uint32_t nv_byte(float r) {
  return __nv_cvt_float_to_fp8(r, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float nv_scale(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
  return __half2float(__half(h));
}

// Is v above a b, or just there and `tie`? a has few bits, so that a b is hi + lo with hi = a b rounded.
// Where v is known to kTol of itself only and lies that near, `near` is set.
template <bool kPairs>
__device__ __forceinline__ bool above(Pair v, float a, float b, bool tie, bool& near) {
  const float hi = a * b, lo = fmaf(a, b, -hi);
  if constexpr (kPairs) {
    const float d = (v.hi - hi) + (v.lo - lo);
    near |= fabsf(d) <= kNearPairs * hi;
    return d > 0.0f;
  } else {
    return v.hi > hi || (v.hi == hi && (lo < 0.0f || (lo == 0.0f && tie)));
  }
}

// The byte of a block, its largest |value| and the codes of a lane's N values h (+ l, in pairs) of it.
// `near`: f32 does not decide.
template <bool kNv, bool kPairs, int N>
__device__ __forceinline__ Fp4Codes<N> decide(const float (&h)[N], const float (&l)[N], float g, uint32_t& byte,
                                              float& amax, bool& near) {
  constexpr int kLanes = (kNv ? 16 : 32) / N;   // to a block
  Pair top{0.0f, 0.0f};
  if constexpr (kPairs) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float a = fabsf(h[i]), b = signbit(h[i]) ? -l[i] : l[i];
      if (!(a < top.hi) && !(a == top.hi && b <= top.lo)) top = Pair{a, b};
    }
#pragma unroll
    for (int d = 1; d < kLanes; d *= 2) {
      const float a = __shfl_xor_sync(0xffffffffu, top.hi, d), b = __shfl_xor_sync(0xffffffffu, top.lo, d);
      if (!(a < top.hi) && !(a == top.hi && b <= top.lo)) top = Pair{a, b};
    }
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(h[i]) & 0x7fffffffu);
    top.hi = lanes_max<kLanes>(__uint_as_float(m));
  }
  amax = top.hi;
  float inv, scale;
  if constexpr (kNv) {
    const float r = __fdividef(amax, 6.0f * g);
    byte = nv_byte(r * (1.0f - kNearQuotient));
    // the border between two neighbouring numbers of e4m3, times 6: 7 bits
    if (byte != nv_byte(r * (1.0f + kNearQuotient)) && byte < 126)
      byte += above<kPairs>(top, 3.0f * (nv_scale(byte) + nv_scale(byte + 1)), g, byte & 1, near);
    scale = nv_scale(byte);
    inv = byte == 0 ? 0.0f : __fdividef(1.0f, scale * g);
    // Products of g that f32 does not hold in two parts, and quotients that it does not hold at all.
    near |= !(6.0f * g > 0x1p-90f && 6.0f * g < 0x1p90f) ||
            (amax > 0.0f && !(amax > 0x1p-90f && amax < 0x1p90f));
  } else {
    byte = mx_byte(amax);
    if (kPairs) {   // on either side of 6 * 2^e
      const float border = 6.0f * mx_scale(byte), d = (amax - border) + top.lo;
      const float under = 0.5f * border, d2 = (amax - under) + top.lo;
      near |= fabsf(d) <= kNearPairs * border || fabsf(d2) <= kNearPairs * under || amax < 0x1p-90f;
      if (d > 0.0f) ++byte;
      else if (byte > 0 && d2 <= 0.0f) --byte;
    }
    scale = mx_scale(byte);
    // 2^-(byte - 127): finite values give bytes up to 253.
    inv = __uint_as_float((254u - (byte < 254u ? byte : 253u)) << 23);
  }
  if constexpr (!kNv && !kPairs) {
    float z[N];
    times_all(h, inv, z);   // exact
    return codes_of(z);
  } else {
    float lo[N], hi[N];
    times_all(h, inv * (1.0f - kNearQuotient), lo);
    times_all(h, inv * (1.0f + kNearQuotient), hi);
    Fp4Codes<N> codes = codes_of(lo);
    const Fp4Codes<N> more = codes_of(hi);
#pragma unroll
    for (int w = 0; w < N / 8; ++w) {
      uint32_t differ = codes.word[w] ^ more.word[w];
      // hi's code is the next one up: its border, in quarters, is looked up.
      while (differ) {
        const int at = (__ffs(differ) - 1) & ~3;
        const uint32_t c = codes.word[w] >> at & 7u;
        const float border = 0.25f * static_cast<float>(0x00140e0a07050301ull >> (8 * c) & 0xffu);
        Pair v{};
#pragma unroll
        for (int i = 8 * w; i < 8 * w + 8; ++i)
          if (at == 4 * (i - 8 * w)) v = Pair{fabsf(h[i]), kPairs ? (signbit(h[i]) ? -l[i] : l[i]) : 0.0f};
        codes.word[w] +=
            static_cast<uint32_t>(above<kPairs>(v, border * scale, kNv ? g : 1.0f, c & 1, near)) << at;
        differ &= ~(0xfu << at);
      }
    }
    return codes;
  }
}

// SwiGLU in pairs, and what it decides. `near`: a value that pairs do not hold or decide.
template <bool kNv, int N>
__device__ __forceinline__ Fp4Codes<N> fp4_swiglu_pairs(const float (&v)[N], const float (&u)[N], float g,
                                                        uint32_t* byte, bool* near) {
  float h[N], l[N];
  bool doubt = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float a = fabsf(v[i]);
    const Pair x = pair_exp(Pair{a <= 80.0f ? -a : 0.0f, 0.0f});
    const Pair s = pair_div(v[i] < 0.0f ? x : Pair{1.0f, 0.0f}, pair_add(Pair{1.0f, 0.0f}, x));
    const Pair y = pair_mul(pair_mul(s, v[i]), u[i]);
    // (pairs' sums lose the sign of a zero)
    h[i] = y.hi != 0.0f ? y.hi : __uint_as_float((__float_as_uint(v[i]) ^ __float_as_uint(u[i])) & 0x80000000u);
    l[i] = y.lo;
    doubt |= !(a <= 80.0f) || (a > 0.0f && a < kLeastGate) || !(fabsf(y.hi) < 0x1p90f) ||
             (y.hi != 0.0f && fabsf(y.hi) < kLeastValue);
  }
  float amax;
  const Fp4Codes<N> codes = decide<kNv, true, N>(h, l, g, *byte, amax, doubt);
  *near = doubt;
  return codes;
}

// The same decisions on N values in 64 bits: the block's byte and the codes.
template <bool kNv, int N>
__device__ __forceinline__ Fp4Codes<N> fp4_exact(const double (&v)[N], float g, uint32_t* byte_out) {
  double top = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmax(top, fabs(v[i]));
#pragma unroll
  for (int d = 1; d < (kNv ? 16 : 32) / N; d *= 2) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, d));
  double unit;
  if (kNv) {
    // e4m3: multiples of 2^(e - 3) from 2^e to 2^(e + 1), of 2^-9 below 2^-6.
    const double r = fmin(top / (6.0 * static_cast<double>(g)), 448.0);
    const int e = r < 0x1p-6 ? -6 : ilogb(r);
    const double m = rint(ldexp(r, 3 - e));     // 0..16; even on a tie
    *byte_out = r < 0x1p-6 ? static_cast<uint32_t>(m)
                           : static_cast<uint32_t>((e + 7) * 8 + static_cast<int>(m) - 8);
    unit = ldexp(m, e - 3) * static_cast<double>(g);
  } else {
    int e = -127;
    if (top > 0x6p-127) {
      e = ilogb(top) - 2;                       // top < 2^(e + 3), top >= 4 * 2^e
      if (top > ldexp(6.0, e)) ++e;
    }
    *byte_out = static_cast<uint32_t>(e + 127);
    unit = ldexp(1.0, e);
  }
  Fp4Codes<N> codes = {};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const double a = fabs(v[i]);
    uint32_t c = 0;
    if (unit > 0.0)
      c = (a > 0.25 * unit) + (a >= 0.75 * unit) + (a > 1.25 * unit) + (a >= 1.75 * unit) +
          (a > 2.5 * unit) + (a >= 3.5 * unit) + (a > 5.0 * unit);
    codes.word[i / 8] |= (c | (signbit(v[i]) ? 8u : 0u)) << (4 * (i % 8));
  }
  return codes;
}

__device__ __forceinline__ double swiglu_d(float g, float u) {
  const double gd = g;
  return gd / (1.0 + exp(-gd)) * static_cast<double>(u);
}

// What f32 does not decide, by a whole warp: its lanes' values are read again (a call that takes them in
// arrays would keep them in memory in every segment). Codes and the block's byte.
template <int N>
struct Fp4Again {
  Fp4Codes<N> codes;
  uint32_t byte;
};
template <typename T, bool kNv, bool kSwiglu, int N>
__device__ __noinline__ Fp4Again<N> fp4_again(const T* src, int K, bool in, bool finite, float g) {
  float v[N] = {}, u[N] = {};
  if (in) {
    load_all(src, v);
    if (kSwiglu) load_all(src + K, u);
  }
  Fp4Again<N> r;
  if (kSwiglu) {
    bool near;
    r.codes = fp4_swiglu_pairs<kNv>(v, u, g, &r.byte, &near);
    if (!__any_sync(0xffffffffu, near && finite)) return r;
  }
  double d[N];
#pragma unroll
  for (int i = 0; i < N; ++i) d[i] = !kSwiglu ? static_cast<double>(v[i]) : in ? swiglu_d(v[i], u[i]) : 0.0;
  r.codes = fp4_exact<kNv>(d, g, &r.byte);
  return r;
}

// Segments of 32 lanes of `per` channels that reach a row's scales, with what fills them up.
__host__ __device__ constexpr int quant_segments(int pitch, bool nv, int per) {
  return (pitch * (nv ? 16 : 32) + 32 * per - 1) / (32 * per);
}

// By lanes of N channels. (Of 16: what a lane does once is shared by more, and a block of nv is one lane's.)
template <typename T, bool kNv, bool kSwiglu, int N>
__global__ void __launch_bounds__(kSegmentThreads, N == 8 ? 12 : kSwiglu && kNv ? 9 : 10)
quantize_fp4_kernel(const T* __restrict__ x, int64_t R, int K, Fp4Out out) {
  pdl_trigger();
  pdl_wait();
  constexpr int kLanes = (kNv ? 16 : 32) / N;   // to a block
  const int lane = threadIdx.x & 31;
  const int pitch = fp4_scale_pitch(K, kNv ? kFp4Nv : kFp4Mx);
  // Segments of 32 N channels, over the whole row of scales.
  for (SegmentWalk w(quant_segments(pitch, kNv, N)); w.row < R; w.next()) {
    const int c = w.seg * 32 * N + lane * N;
    const bool in = c < K;                      // (K % 32 == 0: the same in all lanes of a block)
    float v[N] = {}, u[N] = {};
    const T* src = x + w.row * (kSwiglu ? 2 : 1) * K + c;
    if (in) {
      load_all(src, v);
      if (kSwiglu) load_all(src + K, u);
    }
    float g = 1.0f;
    if (kNv && out.g)
      g = __ldg(out.g + (out.rows_per_plane < R ? w.row / out.rows_per_plane : 0));
    uint32_t byte;
    Fp4Codes<N> codes;
    bool finite;
    if constexpr (!kSwiglu) {
      bool near = false;
      float amax;
      codes = decide<kNv, false, N>(v, v, g, byte, amax, near);
      finite = amax < INFINITY;
      if (kNv && __any_sync(0xffffffffu, near && finite)) {
        const Fp4Again<N> r = fp4_again<T, kNv, false, N>(src, K, in, finite, g);
        codes = r.codes;
        byte = r.byte;
      }
    } else {
      float h[N], amax = 0.0f, gates = 0.0f;
      constexpr float kMinusLog2E = -1.44269504f;
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const uint64_t gate = two(v[i], v[i + 1]), x = times(gate, two(kMinusLog2E, kMinusLog2E));
        const uint64_t d = plus(two(power_of_2(first(x)), power_of_2(second(x))), two(1.0f, 1.0f));
        const uint64_t y = times(times(gate, two(reciprocal(first(d)), reciprocal(second(d)))), two(u[i], u[i + 1]));
        h[i] = first(y);
        h[i + 1] = second(y);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        gates = fmaxf(gates, fabsf(v[i]));
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(amax) : "f"(fabsf(h[i])));   // (a NaN stays)
      }
      amax = lanes_max<kLanes>(amax);
      gates = lanes_max<kLanes>(gates);
      finite = amax < INFINITY;
      // A gate below -80: sigma leaves f32's range.
      bool near = gates > 80.0f || (kNv && !(6.0f * g > 0x1p-90f && 6.0f * g < 0x1p90f)) ||
                  (amax > 0.0f && amax < kLeastValue);
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) near |= v[i] != 0.0f && fabsf(v[i]) < kLeastGate;
      }
      const float by = fmaf(gates, kNearGate, kNearSwiglu);
      float inv;
      if constexpr (kNv) {
        const float r = __fdividef(amax, 6.0f * g);
        byte = nv_byte(r * (1.0f - by));
        near |= byte != nv_byte(r * (1.0f + by)) || amax >= 0x1p90f;
        inv = byte == 0 ? 0.0f : __fdividef(1.0f, nv_scale(byte) * g);
      } else {
        byte = mx_byte(amax * (1.0f - by));
        near |= byte != mx_byte(amax * (1.0f + by));
        inv = __uint_as_float((254u - (byte < 254u ? byte : 253u)) << 23);
      }
      float lo[N], hi[N];
      times_all(h, inv * (1.0f - by), lo);
      times_all(h, inv * (1.0f + by), hi);
      codes = codes_of(lo);
      const Fp4Codes<N> up = codes_of(hi);
#pragma unroll
      for (int i = 0; i < N / 8; ++i) near |= codes.word[i] != up.word[i];
      if (__any_sync(0xffffffffu, near && finite)) {
        const Fp4Again<N> r = fp4_again<T, kNv, true, N>(src, K, in, finite, g);
        codes = r.codes;
        byte = r.byte;
      }
    }
    if (!finite) {
      byte = kNv ? kNvNan : kMxNan;
      codes = {};
    }
    if (in) *reinterpret_cast<Fp4Codes<N>*>(out.codes + w.row * (K / 2) + c / 2) = codes;
    // (What fills a row of scales up is zeros.)
    const int at = c / (kLanes * N);
    if ((lane & (kLanes - 1)) == 0 && at < pitch)
      out.scales[w.row * pitch + at] = static_cast<uint8_t>(in ? byte : 0u);
  }
}

// Four times 8 channels a lane, loaded before the first is worked on: 4 bytes of codes a lane are little to
// have under way. (8192 x 14336, mx to bf16: 56 us; with one load
// a lane 64; with 16 channels side by side a lane, whose stores leave half of their sectors to the next, 73.)
template <typename T, bool kNv>
__global__ void __launch_bounds__(kSegmentThreads)
dequantize_fp4_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      const float* __restrict__ gs, int64_t rows_per_plane, int64_t R, int K,
                      T* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int pitch = fp4_scale_pitch(K, kNv ? kFp4Nv : kFp4Mx);
  for (SegmentWalk w((K + 1023) / 1024); w.row < R; w.next()) {
    const int c0 = w.seg * 1024 + lane * kPerLane;
    const uint8_t* src = codes + w.row * (K / 2) + c0 / 2;
    const uint8_t* sc = scales + w.row * pitch + c0 / (kNv ? 16 : 32);
    uint32_t code[4], byte[4];
#pragma unroll
    for (int p = 0; p < 4; ++p)
      if (c0 + 256 * p < K) {
        code[p] = __ldg(reinterpret_cast<const uint32_t*>(src + 128 * p));
        byte[p] = __ldg(sc + (kNv ? 16 : 8) * p);
      }
    // code * scale has 6 significant bits: exact; then g's rounding and that to T.
    const float g = kNv && gs ? __ldg(gs + (rows_per_plane < R ? w.row / rows_per_plane : 0)) : 1.0f;
    T* dst = out + w.row * K + c0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      if (c0 + 256 * p >= K) break;
      float scale;
      if (kNv) {
        scale = nv_scale(byte[p]);
      } else {
        scale = byte[p] == kMxNan ? __uint_as_float(0x7fffffffu) : mx_scale(byte[p]);
      }
      uint32_t h[4];
      fp4_halves8(code[p], h);
      float f[kPerLane];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 two = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        f[2 * i] = two.x * scale * g;
        f[2 * i + 1] = two.y * scale * g;
      }
      store8(dst + 256 * p, f);
    }
  }
}

template <typename T, bool kNv, bool kSwiglu, int N>
cudaError_t quantize_lanes(const T* x, int64_t R, int K, const Fp4Out& out, cudaStream_t s) {
  const dim3 grid(segment_grid(R, quant_segments(fp4_scale_pitch(K, kNv ? kFp4Nv : kFp4Mx), kNv, N)));
  return launch_pdl(quantize_fp4_kernel<T, kNv, kSwiglu, N>, grid, dim3(kSegmentThreads), 0, s, x, R, K, out);
}

template <typename T, bool kNv, bool kSwiglu>
cudaError_t quantize_one(const T* x, int64_t R, int K, const Fp4Out& out, cudaStream_t s) {
  if constexpr (kSwiglu) {
    if (sizeof(T) == 4 || R * K < kFewValues) return quantize_lanes<T, kNv, true, 8>(x, R, K, out, s);
  }
  if constexpr (!kSwiglu || sizeof(T) == 2) return quantize_lanes<T, kNv, kSwiglu, 16>(x, R, K, out, s);
  else return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t quantize_t(const void* x, int64_t R, int K, int fmt, bool swiglu, const Fp4Out& out,
                       cudaStream_t s) {
  const T* src = static_cast<const T*>(x);
  if (fmt == kFp4Nv)
    return swiglu ? quantize_one<T, true, true>(src, R, K, out, s)
                  : quantize_one<T, true, false>(src, R, K, out, s);
  return swiglu ? quantize_one<T, false, true>(src, R, K, out, s)
                : quantize_one<T, false, false>(src, R, K, out, s);
}

template <typename T>
cudaError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, const float* g,
                         int64_t rows_per_plane, int64_t R, int K, int fmt, void* out,
                         cudaStream_t s) {
  const dim3 grid(segment_grid(R, (K + 1023) / 1024)), block(kSegmentThreads);
  return fmt == kFp4Nv ? launch_pdl(dequantize_fp4_kernel<T, true>, grid, block, 0, s, codes, scales, g,
                                    rows_per_plane, R, K, static_cast<T*>(out))
                       : launch_pdl(dequantize_fp4_kernel<T, false>, grid, block, 0, s, codes, scales,
                                    g, rows_per_plane, R, K, static_cast<T*>(out));
}

}  // namespace

moe_status launch_quantize_fp4(const void* x, int64_t planes, int64_t rows, int K, int dtype, int fmt,
                               bool swiglu, const float* g, uint8_t* codes, uint8_t* scales,
                               cudaStream_t s) {
  const int64_t R = planes * rows;
  const Fp4Out out{codes, scales, g, rows};
  const cudaError_t err = dtype == MOE_DTYPE_BF16  ? quantize_t<__nv_bfloat16>(x, R, K, fmt, swiglu, out, s)
                          : dtype == MOE_DTYPE_F16 ? quantize_t<__half>(x, R, K, fmt, swiglu, out, s)
                                                   : quantize_t<float>(x, R, K, fmt, swiglu, out, s);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "quantize_fp4 launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

moe_status launch_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, const float* g,
                                 int64_t planes, int64_t rows, int K, int fmt, int dtype, void* out,
                                 cudaStream_t s) {
  const int64_t R = planes * rows;
  const cudaError_t err =
      dtype == MOE_DTYPE_BF16  ? dequantize_t<__nv_bfloat16>(codes, scales, g, rows, R, K, fmt, out, s)
      : dtype == MOE_DTYPE_F16 ? dequantize_t<__half>(codes, scales, g, rows, R, K, fmt, out, s)
                               : dequantize_t<float>(codes, scales, g, rows, R, K, fmt, out, s);
  if (err != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "dequantize_fp4 launch: %s", cudaGetErrorString(err));
  return MOE_OK;
}

}  // namespace moe
