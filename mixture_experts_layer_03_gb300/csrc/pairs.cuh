// Numbers hi + lo of two f32, lo half a unit of hi or less: sums, products, quotients and exponentials to some
// 2^-28 of the value, where fp64, at 1/64 of fp32's rate, would be waited for. And two f32 as one operand.
#pragma once

#include <cstdint>

namespace moe {
namespace {

// Two products or sums an instruction.
__device__ __forceinline__ uint64_t two(float a, float b) {
  return static_cast<uint64_t>(__float_as_uint(b)) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ float first(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float second(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint64_t times(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t plus(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t times_plus(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair pair_of(float a, float b) {      // a + b, |a| >= |b| or a = 0
  const float s = a + b;
  return Pair{s, b - (s - a)};
}
__device__ __forceinline__ Pair pair_sum(float a, float b) {     // any a, b (Knuth)
  const float s = a + b, t = s - a;
  return Pair{s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  const Pair s = pair_sum(a.hi, b.hi);
  return pair_of(s.hi, s.lo + (a.lo + b.lo));
}
__device__ __forceinline__ Pair pair_div(Pair a, Pair b) {
  const float q = __fdiv_rn(a.hi, b.hi);
  const float rest = fmaf(-q, b.hi, a.hi) + (a.lo - q * b.lo);
  return pair_of(q, __fdividef(rest, b.hi));
}
// exp(a), -80 <= a <= 0: a = n ln 2 + r with ln 2 in two parts, the first of 16 bits (Cody and Waite), so
// that n times it is exact; then 1 + r + r^2 / 2 + ..., |r| <= 0.35, its first terms in pairs.
__device__ __forceinline__ Pair pair_exp(Pair a) {
  constexpr float kLn2Hi = 0x1.62e4p-1f, kLn2Lo = static_cast<float>(0.693147180559945309417 - 0x1.62e4p-1);
  const float n = rintf(a.hi * 1.44269504f);
  const Pair r = pair_sum(fmaf(-n, kLn2Hi, a.hi), fmaf(-n, kLn2Lo, a.lo));
  const float sq = r.hi * r.hi, sq_lo = fmaf(r.hi, r.hi, -sq);
  float q = 1.0f / 40320;
  q = fmaf(q, r.hi, 1.0f / 5040);
  q = fmaf(q, r.hi, 1.0f / 720);
  q = fmaf(q, r.hi, 1.0f / 120);
  q = fmaf(q, r.hi, 1.0f / 24);
  q = fmaf(q, r.hi, 1.0f / 6);
  // r.lo (1 + r): the slope of exp at r.hi
  const float small = fmaf(r.lo, r.hi, r.lo) + fmaf(0.5f, sq_lo, r.hi * sq * q);
  const Pair one = pair_of(1.0f, r.hi);
  const Pair two = pair_sum(one.hi, 0.5f * sq);
  const Pair e = pair_of(two.hi, (one.lo + two.lo) + small);
  const float scale = __uint_as_float(static_cast<uint32_t>(static_cast<int>(n) + 127) << 23);
  return Pair{e.hi * scale, e.lo * scale};
}
__device__ __forceinline__ Pair pair_mul(Pair a, float b) {
  const float p = a.hi * b;
  return pair_of(p, fmaf(a.hi, b, -p) + a.lo * b);
}

}  // namespace
}  // namespace moe
