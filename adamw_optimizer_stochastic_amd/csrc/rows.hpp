// Pieces of the kernels that walk rows of a matrix: 8 columns a lane, loads and
// stores of 16 bytes from any element's address, and reductions over lanes.
#pragma once

#include "codes.hpp"

#pragma clang fp contract(off)

namespace asr_rows {

// Element-aligned vectors: global accesses of 16 bytes need no more than that,
// so rows of any width and views from any element keep the wide form.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Streams are read and written past the caches (non-temporal): what a pass reads
// once need not push out what others will read again. Outputs always, large inputs that
// nothing reads soon again (gated SiLU of 8192 x 14336 bf16: 110 us, 122 with ordinary
// loads, its gradient 185 and 205); not the rows of a layer norm, of a table and
// of its gradient, which are often in the caches and read again (8192 x 4096 bf16:
// norm 24 us, 29 past the caches; lookup 22 and 25, gradient 182 and 190). (f32 outputs, 32
// bytes a lane, are half lines of two stores: by ordinary ones 8192 x 4096 norms take 45 us
// instead of 59 and 8192 x 14336 unpacked 110 instead of 184, but a norm's gradient 81
// instead of 77 and gated SiLU of 1000 x 4096 10.7 instead of 9.8.)
// (Functions of their own for each type: a template would drop the alignment.)
__device__ __forceinline__ asr::u32x4 load_stream(const u32x4_any* p) { return __builtin_nontemporal_load(p); }
__device__ __forceinline__ asr::f32x4 load_stream(const f32x4_any* p) { return __builtin_nontemporal_load(p); }
__device__ __forceinline__ asr::u32x2 load_stream(const asr::u32x2* p) { return __builtin_nontemporal_load(p); }
__device__ __forceinline__ void store_stream(u32x4_any* p, asr::u32x4 v) { __builtin_nontemporal_store(v, p); }
__device__ __forceinline__ void store_stream(f32x4_any* p, asr::f32x4 v) { __builtin_nontemporal_store(v, p); }
__device__ __forceinline__ void store_stream(asr::u32x2* p, asr::u32x2 v) { __builtin_nontemporal_store(v, p); }

// 8 columns of a row as they lie in memory. count: how many of them there are
// (8 or more: all; the others read as 0). At a row's end the elements are loaded
// one by one, but all at once: places past the end load the last element again,
// as a branch for each would wait for every load by itself (5 us for 7 of them).
// load_repeated leaves that element there instead of 0.
template <typename S>
struct Run;
template <>
struct Run<uint16_t> {
  asr::u32x4 w;
  template <bool ONCE, bool REPEAT = false>
  __device__ __forceinline__ void load_as(const uint16_t* p, int64_t count) {
    if (count >= 8) {
      const u32x4_any* from = reinterpret_cast<const u32x4_any*>(p);
      w = ONCE ? load_stream(from) : *from;
    } else {
      w = asr::u32x4{0, 0, 0, 0};
      if (count > 0) {
        uint32_t t[7];
#pragma unroll
        for (int e = 0; e < 7; ++e) t[e] = p[min(static_cast<int>(count) - 1, e)];
#pragma unroll
        for (int e = 0; e < 7; ++e) w[e / 2] |= (REPEAT || e < count ? t[e] : 0u) << (e % 2 * 16);
        if (REPEAT) w[3] |= t[6] << 16;
      }
    }
  }
  __device__ __forceinline__ void load(const uint16_t* p, int64_t count) { load_as<false>(p, count); }
  __device__ __forceinline__ void load_once(const uint16_t* p, int64_t count) { load_as<true>(p, count); }
  __device__ __forceinline__ void load_repeated(const uint16_t* p, int64_t count) { load_as<false, true>(p, count); }
  __device__ __forceinline__ float get(int e) const {
    return __uint_as_float(e % 2 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
  }
};
template <>
struct Run<float> {
  asr::f32x4 w[2];
  template <bool ONCE, bool REPEAT = false>
  __device__ __forceinline__ void load_as(const float* p, int64_t count) {
    if (count >= 8) {
      const f32x4_any* from = reinterpret_cast<const f32x4_any*>(p);
      w[0] = ONCE ? load_stream(from) : from[0];
      w[1] = ONCE ? load_stream(from + 1) : from[1];
    } else {
      w[0] = w[1] = asr::f32x4{0, 0, 0, 0};
      if (count > 0) {
        float t[7];
#pragma unroll
        for (int e = 0; e < 7; ++e) t[e] = p[min(static_cast<int>(count) - 1, e)];
#pragma unroll
        for (int e = 0; e < 7; ++e) w[e / 4][e % 4] = REPEAT || e < count ? t[e] : 0.0f;
        if (REPEAT) w[1][3] = t[6];
      }
    }
  }
  __device__ __forceinline__ void load(const float* p, int64_t count) { load_as<false>(p, count); }
  __device__ __forceinline__ void load_once(const float* p, int64_t count) { load_as<true>(p, count); }
  __device__ __forceinline__ void load_repeated(const float* p, int64_t count) { load_as<false, true>(p, count); }
  __device__ __forceinline__ float get(int e) const { return w[e / 4][e % 4]; }
};

// Two f32 to two bf16 (low half first), to nearest, ties to even.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, asr::bf16x2));
}

__device__ __forceinline__ void store8(uint16_t* p, int64_t count, const float (&x)[8]) {
  const asr::u32x4 w = {bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7])};
  if (count >= 8) {
    store_stream(reinterpret_cast<u32x4_any*>(p), w);
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < count) p[e] = static_cast<uint16_t>(w[e / 2] >> (e % 2 * 16));
  }
}

__device__ __forceinline__ void store8(float* p, int64_t count, const float (&x)[8]) {
  if (count >= 8) {
    store_stream(reinterpret_cast<f32x4_any*>(p), asr::f32x4{x[0], x[1], x[2], x[3]});
    store_stream(reinterpret_cast<f32x4_any*>(p) + 1, asr::f32x4{x[4], x[5], x[6], x[7]});
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < count) p[e] = x[e];
  }
}

// 8 parameters (a norm's weight or bias) of either type.
__device__ __forceinline__ void load_params(const void* p, bool bf16, int64_t col, int64_t count, float (&x)[8]) {
  if (bf16) {
    Run<uint16_t> r;
    r.load(static_cast<const uint16_t*>(p) + col, count);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = r.get(e);
  } else {
    Run<float> r;
    r.load(static_cast<const float*>(p) + col, count);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = r.get(e);
  }
}

// A value from the lane N places round the 16 lanes of a row (every lane of
// the wave active).
template <int N>
__device__ __forceinline__ uint32_t turned(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x120 + N, 0xF, 0xF, true));
}
template <int N>
__device__ __forceinline__ float turned(float v) {
  return __uint_as_float(turned<N>(__float_as_uint(v)));
}
template <int N>
__device__ __forceinline__ double turned(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, static_cast<uint64_t>(turned<N>(static_cast<uint32_t>(u))) |
                                        static_cast<uint64_t>(turned<N>(static_cast<uint32_t>(u >> 32))) << 32);
}

// Over 16 lanes, the result in each of them (the same bits: every step adds
// the two halves of one set).
template <typename V, typename F>
__device__ __forceinline__ V reduce16(V v, F f) {
  v = f(v, turned<8>(v));
  v = f(v, turned<4>(v));
  v = f(v, turned<2>(v));
  return f(v, turned<1>(v));
}

template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
  v = reduce16(v, [](V a, V b) { return a + b; });
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// How many terms of a long f32 sum are added before the sum so far goes into a second
// one: an addition is off by half a step of the sum, so n of them in one chain by up to n
// half steps, in two levels by 2 sqrt(n) to 3 sqrt(n). Up to 256 terms stay one chain.
inline int32_t fold_of(int64_t terms) {
  int64_t f = 256;
  while (f * f < terms) f *= 2;
  return static_cast<int32_t>(f);
}

}  // namespace asr_rows
