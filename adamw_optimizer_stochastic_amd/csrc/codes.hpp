// 8-bit codes of a group of values that share a scale: a row or column of a
// product's operand, or a block of columns of a stored activation.
//   s = f32(max|x| / 127),  q = sign(x) * min(127, Q(|x| / s)),
// Q rounding the EXACT quotient: to nearest, ties to even, or stochastically,
// floor(|x|/s + r16/65536). The decision needs no division: with r = r16/65536
// (1/2 to nearest) and m the whole number nearest to |x| * (1/s) + r, the code is
// m or m - 1. m - r has at most 24 bits, so it is exact in binary32, and
// |x|/s + r reaches m exactly when fma(-(m - r), s, |x|) >= 0: one rounding
// keeps a sign. To nearest, 0 there is a tie: m - 1 if m is odd.
#pragma once

#include "device.hpp"

#pragma clang fp contract(off)

namespace asr_i8 {

struct __align__(16) GroupScale {
  float s;        // the scale the group's codes are divided by, times k
  float inv;      // 1 / s
  float k;        // power of two that keeps every product with s a normal number
  uint32_t live;  // all ones, or 0: every code is 0 (no element, only tiny ones, Inf or NaN)
};

// The scale to store for a group whose largest |x| has these bits, and what
// the codes need. Below 127 * 2**-126 the scale would be subnormal: such a
// group is stored as zeros. Inf or NaN anywhere makes the scale NaN, which
// every product with the group then shows.
__device__ __forceinline__ float group_scale(uint32_t max_bits, GroupScale& g) {
  // (top / 127 rounded to nearest, without a division: an estimate by the rounded
  // 1/127 and one correction, equal for every 24-bit top)
  const float top = __uint_as_float(max_bits), guess = top * (1.0f / 127.0f);
  const float s = __builtin_fmaf(__builtin_fmaf(-127.0f, guess, top), 1.0f / 127.0f, guess);
  const bool finite = max_bits < 0x7F800000u;
  const bool live = finite && s >= 0x1p-126f;
  g.live = live ? 0xFFFFFFFFu : 0u;
  g.k = s < 0x1p-60f ? 0x1p64f : 1.0f;
  g.s = live ? s * g.k : 1.0f;
  g.inv = __builtin_amdgcn_rcpf(g.s);   // off by 2**-23 of itself at most
  return finite ? (live ? s : 0.0f) : __uint_as_float(0x7FC00000u);
}

// The exact code of any element (of a live group).
template <bool SR>
__device__ __forceinline__ int32_t exact_code(float x, const GroupScale& g, uint32_t r16) {
  const float ax = __builtin_fabsf(x) * g.k;
  const float r = SR ? static_cast<float>(r16) * 0x1p-16f : 0.5f;
  const float m = __builtin_rintf(__builtin_fmaf(ax, g.inv, r));
  const float rest = __builtin_fmaf(-(m - r), g.s, ax);
  const int32_t i = static_cast<int32_t>(m);
  const bool down = rest < 0.0f || (!SR && rest == 0.0f && (i & 1));
  const int32_t q = min(i - (down ? 1 : 0), 127);
  return x < 0.0f ? -q : q;
}

// Byte 0 of four words. (As asm: the compiler takes the permutes apart into
// 16-bit shifts and merges, three times as many instructions.)
__device__ __forceinline__ uint32_t pack_bytes(uint32_t u0, uint32_t u1, uint32_t u2, uint32_t u3) {
  uint32_t lo, hi, all;
  asm("v_perm_b32 %0, %1, %2, %3" : "=v"(lo) : "v"(u1), "v"(u0), "s"(0x0C0C0400u));
  asm("v_perm_b32 %0, %1, %2, %3" : "=v"(hi) : "v"(u3), "v"(u2), "s"(0x0C0C0400u));
  asm("v_perm_b32 %0, %1, %2, %3" : "=v"(all) : "v"(hi), "v"(lo), "s"(0x05040100u));
  return all;
}

// Codes of 4 elements of one group, packed. With the exact decision for every
// element its arithmetic is what bounds the kernels, so the usual case is short: |x| * (1/s) is off by less than
// 2.4e-5 here (the reciprocal's 2**-23 and the sum's 2**-24, of 129 at most), so a value
// further than that from a border has its code from one multiply-add (to nearest:
// onto 1.5 * 2**23, whose low byte is then the code; stochastic: floor of the
// quotient plus 1 + r16/65536). A wave that has an element nearer (3e-5) than that
// decides this one of its lanes' elements exactly, 11 instructions instead of 4. (bf16
// values equal to half the group's largest are ties but for the rounding of s, so
// a quarter of the blocks of 128 have such an element: one test for all four
// elements together cost a third of the instructions of a kernel of codes.)
template <bool SR>
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], const GroupScale& g,
                                           const uint32_t (&r16)[4]) {
  constexpr float kByte = 12582912.0f;  // 1.5 * 2**23
  // (a scaled group, k != 1, takes the exact way: its inv is that of the scaled s)
  const float near = g.k != 1.0f ? -1.0f : 0.49997f;
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float off;  // from the middle between two borders
    if constexpr (SR) {
      const float one_r = __uint_as_float(0x3F800000u | (r16[e] << 7));  // 1 + r16 / 65536
      const float v = __builtin_fmaf(__builtin_fabsf(x[e]), g.inv, one_r);
      const float f = __builtin_floorf(v);
      off = (v - f) - 0.5f;
      u[e] = __float_as_uint(__builtin_copysignf(__builtin_fminf(f - 1.0f, 127.0f), x[e]) + kByte);
    } else {
      const float t = __builtin_fmaf(x[e], g.inv, kByte);
      off = __builtin_fmaf(x[e], g.inv, -(t - kByte));
      u[e] = __float_as_uint(t);
    }
    if (__builtin_amdgcn_ballot_w64(__builtin_fabsf(off) > near) != 0)
      u[e] = static_cast<uint32_t>(exact_code<SR>(g.live ? x[e] : 0.0f, g, r16[e]));
  }
  return pack_bytes(u[0], u[1], u[2], u[3]) & g.live;
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// 8 consecutive elements from column j of a row (j a multiple of 8); past
// `cols` they are zero.
template <typename S>
__device__ __forceinline__ void load8(const S* row, int64_t j, int64_t cols, bool vec,
                                      float (&x)[8]) {
  if (vec && j + 8 <= cols) {
    asr::load_vec<false, 8>(row + j, x);
  } else {
    asr::load_range<8>(row, j, 0, static_cast<int>(max(int64_t{0}, min(int64_t{8}, cols - j))), x);
  }
}

// 8 elements as they lie in memory.
template <typename S>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  asr::u32x4 w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = *reinterpret_cast<const asr::u32x4*>(p); }
  __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = (__float_as_uint(x[2 * k]) >> 16) | (__float_as_uint(x[2 * k + 1]) & 0xFFFF0000u);
  }
  __device__ __forceinline__ float get(int e) const {
    return __uint_as_float(e % 2 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
  }
};
template <>
struct Raw8<float> {
  asr::f32x4 w[2];
  __device__ __forceinline__ void load(const float* p) {
    w[0] = reinterpret_cast<const asr::f32x4*>(p)[0];
    w[1] = reinterpret_cast<const asr::f32x4*>(p)[1];
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    w[0] = asr::f32x4{x[0], x[1], x[2], x[3]};
    w[1] = asr::f32x4{x[4], x[5], x[6], x[7]};
  }
  __device__ __forceinline__ float get(int e) const { return w[e / 4][e % 4]; }
};

}  // namespace asr_i8
