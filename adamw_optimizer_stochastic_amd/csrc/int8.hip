// 8-bit integer products with a scale for each row of both operands, and the
// quantiser that makes their operands.
//
// quantise: a group (a row of x, or a column of x for the transposed form) has
//   s = f32(max|x| / 127),  q = sign(x) * min(127, Q(|x| / s)),
// where Q rounds the EXACT quotient: to nearest, ties to even, or
// stochastically, floor(|x|/s + r16/65536) with the 16 bits of the element's
// stream position. The decision is exact and needs no division: with c =
// (k + 1) - r16/65536 (at most 24 bits, so exact in binary32), |x|/s + r16/65536
// reaches k + 1 exactly when fma(-c, s, |x|) >= 0, and one rounding keeps a
// sign. k comes from |x| * (1/s), off by at most one, and two such tests
// settle it; to nearest is the same with r16 = 32768 and a step back from an
// odd tie.
//
// product: C[m][n] = round((f32(sum_k A[m][k] B[n][k]) * sa[m]) * sb[n]), the
// sum exact in 32-bit integers (K < 2**17), so it does not depend on how K
// is split or ordered.
#include "mfma_loop.hpp"
#include "status.hpp"

#include <adamw_sr.h>

#include <algorithm>
#include <string>

#pragma clang fp contract(off)

namespace asr_i8 {

using asr_mfma::static_for;

// ------------------------------------------------------------- quantiser
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
  const float s = __uint_as_float(max_bits) / 127.0f;
  const bool finite = max_bits < 0x7F800000u;
  const bool live = finite && s >= 0x1p-126f;
  g.live = live ? 0xFFFFFFFFu : 0u;
  g.k = s < 0x1p-60f ? 0x1p64f : 1.0f;
  g.s = live ? s * g.k : 1.0f;
  g.inv = 1.0f / g.s;
  return finite ? (live ? s : 0.0f) : __uint_as_float(0x7FC00000u);
}

// The exact code of any element (of a live group).
template <bool SR>
__device__ __forceinline__ int32_t exact_code(float x, const GroupScale& g, uint32_t r16) {
  const float ax = __builtin_fabsf(x) * g.k;
  const float r = SR ? static_cast<float>(r16) * 0x1p-16f : 0.5f;
  float q = __builtin_floorf(__builtin_fmaf(ax, g.inv, r));
  if (__builtin_fmaf(-((q + 1.0f) - r), g.s, ax) >= 0.0f) {
    q += 1.0f;
  } else if (__builtin_fmaf(-(q - r), g.s, ax) < 0.0f) {
    q -= 1.0f;
  }
  int32_t i = static_cast<int32_t>(q);
  if constexpr (!SR) {
    if ((i & 1) && __builtin_fmaf(-(q - 0.5f), g.s, ax) == 0.0f) i -= 1;
  }
  i = min(i, 127);
  return x < 0.0f ? -i : i;
}

// Codes of 4 elements of one group, packed. With the exact decision for every
// element its arithmetic is what bounds the kernels, so the usual case is short: |x| * (1/s) is off by less than
// 2**-16 here, so a value further than that from a border has its code from
// one multiply-add (to nearest: onto 1.5 * 2**23, whose low byte is then the
// code; stochastic: floor of the quotient plus 1 + r16/65536). A wave that
// has an element nearer (1e-4) than that decides these exactly: 40 instructions an
// element instead of 6. (58.7e6 bf16 values, rows, RN: 43 us, 58 us with the
// exact decision for all.)

// Byte 0 of four words. (As asm: the compiler takes the permutes apart into
// 16-bit shifts and merges, three times as many instructions.)
__device__ __forceinline__ uint32_t pack_bytes(uint32_t u0, uint32_t u1, uint32_t u2, uint32_t u3) {
  uint32_t lo, hi, all;
  asm("v_perm_b32 %0, %1, %2, %3" : "=v"(lo) : "v"(u1), "v"(u0), "s"(0x0C0C0400u));
  asm("v_perm_b32 %0, %1, %2, %3" : "=v"(hi) : "v"(u3), "v"(u2), "s"(0x0C0C0400u));
  asm("v_perm_b32 %0, %1, %2, %3" : "=v"(all) : "v"(hi), "v"(lo), "s"(0x05040100u));
  return all;
}

template <bool SR>
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], const GroupScale& g,
                                           const uint32_t (&r16)[4]) {
  constexpr float kByte = 12582912.0f;  // 1.5 * 2**23
  uint32_t u[4];
  float off[4];  // distance from the middle between two borders
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (SR) {
      const float one_r = __uint_as_float(0x3F800000u | (r16[e] << 7));  // 1 + r16 / 65536
      const float v = __builtin_fmaf(__builtin_fabsf(x[e]), g.inv, one_r);
      const float f = __builtin_floorf(v);
      off[e] = (v - f) - 0.5f;
      u[e] = __float_as_uint(__builtin_copysignf(__builtin_fminf(f - 1.0f, 127.0f), x[e]) + kByte);
    } else {
      const float t = __builtin_fmaf(x[e], g.inv, kByte);
      off[e] = __builtin_fmaf(x[e], g.inv, -(t - kByte));
      u[e] = __float_as_uint(t);
    }
  }
  float most = __builtin_fmaxf(__builtin_fmaxf(__builtin_fabsf(off[0]), __builtin_fabsf(off[1])),
                               __builtin_fmaxf(__builtin_fabsf(off[2]), __builtin_fabsf(off[3])));
  // (a scaled group, k != 1, takes the exact way: its inv is that of the scaled s)
  if (__builtin_amdgcn_ballot_w64(most > 0.4999f || g.k != 1.0f) != 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
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

// A matrix of a launch, and the codes wanted of it: of its rows, of its
// columns, or both.
struct QuantJob {
  const void* x;
  int8_t* q_row;        // NULL: not wanted
  int8_t* q_col;
  float* s_row;
  float* s_col;
  uint32_t* part_row;   // row maxima of each strip of 256 columns
  uint32_t* part_col;   // column maxima of each chunk of rows
  int64_t ldx, ld_row, ld_col;
  uint64_t base;
  int32_t rows, cols, chunk, strips, tiles;
  int32_t chunks;       // 0: one tile of rows, without partial maxima
  uint32_t first, blocks;  // its workgroups in this launch
  uint32_t vec;         // every 8-element run of a row starts on a 16-byte address
  uint32_t sr;
};

constexpr int kMaxJobs = 3;

struct QuantArgs {
  QuantJob j[kMaxJobs];
  int32_t count;
  uint32_t seed, step;
};

__device__ __forceinline__ const QuantJob& job_of(const QuantArgs& a) {
  int k = 0;
  if (a.count > 1 && blockIdx.x >= a.j[1].first) k = 1;
  if (a.count > 2 && blockIdx.x >= a.j[2].first) k = 2;
  return a.j[k];
}

// One row by LANES lanes (64: four rows a workgroup, 256: one). The first
// KEEP runs of 8 a lane holds stay in registers between the pass for the
// maximum and the pass for the codes; a longer row's others are read again.
// x and w of a linear layer, 4096 and 14336 rows of 4096 bf16 (226 MB with the
// codes), take 49-57 us, 4.0-4.6 TB/s, 1.35 to 1.55 times a copy's time: a workgroup
// holds one row from its load through two reductions to its store, with no other
// in flight. 14336 rows alone: 37-41 us to nearest, 53-58 stochastic (the random
// bits). One row of 4096 takes 3 us, its latency.
template <typename S, bool SR, int LANES>
__global__ __launch_bounds__(256) void quantize_rows(QuantArgs args) {
  constexpr int KEEP = 4;
  constexpr int kRowsHere = 256 / LANES;
  const QuantJob& a = job_of(args);
  const int lane = threadIdx.x % LANES;
  const int64_t row = static_cast<int64_t>(blockIdx.x - a.first) * kRowsHere + threadIdx.x / LANES;
  if (LANES == 64 && row >= a.rows) return;  // (whole waves; no barrier follows for LANES == 64)
  const S* x = static_cast<const S*>(a.x) + row * a.ldx;
  const int32_t runs = static_cast<int32_t>((static_cast<int64_t>(a.cols) + 15) / 16 * 2);  // padding included
  float keep[KEEP][8];
  uint32_t top = 0;
#pragma unroll
  for (int v = 0; v < KEEP; ++v) {
    const int32_t run = lane + v * LANES;
    if (run < runs) {
      load8<S>(x, static_cast<int64_t>(run) * 8, a.cols, a.vec, keep[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, abs_bits(keep[v][e]));
    }
  }
  for (int32_t run = lane + KEEP * LANES; run < runs; run += LANES) {
    float t[8];
    load8<S>(x, static_cast<int64_t>(run) * 8, a.cols, a.vec, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, abs_bits(t[e]));
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1)
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
  if constexpr (LANES == 256) {
    __shared__ uint32_t tops[4];
    if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = top;
    __syncthreads();
    top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  }
  GroupScale g;
  const float s = group_scale(top, g);
  if (lane == 0) a.s_row[row] = s;
  int8_t* q = a.q_row + row * a.ld_row;
  auto codes = [&](int32_t run, const float (&t)[8]) {
    uint32_t bits[8] = {};
    if constexpr (SR) {
      const uint64_t p = a.base + static_cast<uint64_t>(row) * static_cast<uint64_t>(a.cols) +
                         static_cast<uint64_t>(run) * 8;
      asr_mfma::random_run<8>(p, (p & 3u) == 0, args.seed, args.step, bits);
    }
    const uint32_t r0[4] = {bits[0], bits[1], bits[2], bits[3]}, r1[4] = {bits[4], bits[5], bits[6], bits[7]};
    const float t0[4] = {t[0], t[1], t[2], t[3]}, t1[4] = {t[4], t[5], t[6], t[7]};
    *reinterpret_cast<asr::u32x2*>(q + static_cast<int64_t>(run) * 8) =
        asr::u32x2{codes4<SR>(t0, g, r0), codes4<SR>(t1, g, r1)};
  };
#pragma unroll
  for (int v = 0; v < KEEP; ++v) {
    const int32_t run = lane + v * LANES;
    if (run < runs) codes(run, keep[v]);
  }
  for (int32_t run = lane + KEEP * LANES; run < runs; run += LANES) {
    float t[8];
    load8<S>(x, static_cast<int64_t>(run) * 8, a.cols, a.vec, t);
    codes(run, t);
  }
}

// Column maxima of one chunk of rows, and if wanted the row maxima of one
// strip: a workgroup takes 256 columns (512 bytes of a bf16 row), 8 rows at a
// time. Few chunks, so that the second kernel reads few of them. Bound by
// memory: 8192 x 4096 bf16 (67 MB) in 11.5-12.5 us, 5.4-5.8 TB/s.
template <typename S>
__global__ __launch_bounds__(256) void maxima(QuantArgs args) {
  __shared__ uint32_t tops[8][256 + 4];
  const QuantJob& a = job_of(args);
  const int32_t block = static_cast<int32_t>(asr_mfma::xcd_order(blockIdx.x - a.first, a.blocks));
  const int32_t strip = block % a.strips, chunk = block / a.strips;
  const int cg = threadIdx.x % 32, rr = threadIdx.x / 32;
  const int64_t c0 = static_cast<int64_t>(strip) * 256, col = c0 + cg * 8;
  const int32_t r0 = chunk * a.chunk;
  const int32_t r1 = static_cast<int32_t>(min(static_cast<int64_t>(a.rows), static_cast<int64_t>(r0) + a.chunk));
  uint32_t top[8] = {};
  for (int32_t r = r0 + rr; r < r1; r += 32) {  // 4 rows' loads in flight
    float t[4][8] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r + 8 * i < r1) load8<S>(static_cast<const S*>(a.x) + (r + 8 * i) * a.ldx, col, a.cols, a.vec, t[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t across = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t v = abs_bits(t[i][e]);
        top[e] = max(top[e], v);
        across = max(across, v);
      }
      if (a.part_row) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
          across = max(across, static_cast<uint32_t>(__shfl_xor(static_cast<int>(across), d)));
        if (cg == 0 && r + 8 * i < r1) a.part_row[static_cast<int64_t>(strip) * a.rows + r + 8 * i] = across;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) tops[rr][cg * 8 + e] = top[e];
  __syncthreads();
  if (c0 + threadIdx.x < a.cols) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, tops[i][threadIdx.x]);
    a.part_col[static_cast<int64_t>(chunk) * a.cols + c0 + threadIdx.x] = m;
  }
}

// Row maxima of many strips, down to one (a tile of the next kernel would
// otherwise read more of them than of the matrix).
__global__ __launch_bounds__(256) void join_strips(uint32_t* part, int32_t rows, int32_t strips) {
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (r >= rows) return;
  uint32_t m = 0;
#pragma unroll 8
  for (int32_t s = 0; s < strips; ++s) m = max(m, part[static_cast<int64_t>(s) * rows + r]);
  part[r] = m;
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

// Codes of 64 columns x `tiles` times 128 rows, tile by tile: of the columns,
// written as 64 rows of the transposed result, and if wanted of the rows (which
// share the random bits, most of the stochastic form's work). A thread takes
// 4 consecutive rows of 8 columns, so 4 codes of one column make one LDS word,
// and the next tile's loads are in flight while it works on this one. The
// stochastic form is bound by the random bits and the codes: 8192 x 4096 bf16
// columns, 101 MB in and out, in 38 us (2.6 TB/s), of which the 8.4e6 Philox
// calls, 20 quarter-rate 64-bit multiply-adds each, come to about 25. A
// linear layer's backward (dy 4096 x 14336 both ways, x 4096 x 4096 and w 14336 x
// 4096 by columns; 460 MB) takes 153-178 us.
struct TileLds {
  uint32_t tile[64 * 33];  // 33 words a column: 32 and one against bank conflicts
  uint32_t tops[256];
  GroupScale col_scale[64];
  GroupScale row_scale[128];
};

template <typename S, bool SR>
__device__ __forceinline__ void quantize_strip(const QuantArgs& args, const QuantJob& a, TileLds& lds) {
  constexpr int kWords = 33;
  const int32_t across = (a.cols + 63) / 64;
  // (neighbouring tiles on one XCD: the row codes of two of them share a line)
  const int32_t block = static_cast<int32_t>(asr_mfma::xcd_order(blockIdx.x - a.first, a.blocks));
  const int32_t tc = block % across, tr0 = block / across * a.tiles;
  const int32_t tr1 = min(tr0 + a.tiles, (a.rows + 127) / 128);
  const int64_t c0 = static_cast<int64_t>(tc) * 64;
  const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3;  // 8 columns, rows rg * 4 .. + 3
  const int64_t col = c0 + cg * 8;
  const bool whole = a.vec && col + 8 <= a.cols;
  Raw8<S> raw[4];
  auto fetch = [&](int32_t tr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = static_cast<int64_t>(tr) * 128 + rg * 4 + i;
      const S* row = static_cast<const S*>(a.x) + r * a.ldx;
      if (whole && r < a.rows) {
        raw[i].load(row + col);
      } else {
        float x[8] = {};
        if (r < a.rows) load8<S>(row, col, a.cols, false, x);
        raw[i].set(x);
      }
    }
  };
  fetch(tr0);
  if (a.chunks == 0) {  // this tile is all of its columns
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, abs_bits(raw[i].get(e)));
#pragma unroll
      for (int d = 8; d < 64; d <<= 1)
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
      if (rg % 8 == 0) lds.tops[threadIdx.x / 64 * 64 + cg * 8 + e] = top;
    }
  } else {
    const int c = threadIdx.x % 64, quarter = threadIdx.x / 64;
    uint32_t top = 0;
    if (c0 + c < a.cols) {
#pragma unroll 8
      for (int32_t p = quarter; p < a.chunks; p += 4)
        top = max(top, a.part_col[static_cast<int64_t>(p) * a.cols + c0 + c]);
    }
    lds.tops[threadIdx.x] = top;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    GroupScale g;
    const float s = group_scale(max(max(lds.tops[threadIdx.x], lds.tops[64 + threadIdx.x]),
                                    max(lds.tops[128 + threadIdx.x], lds.tops[192 + threadIdx.x])), g);
    lds.col_scale[threadIdx.x] = g;
    if (tr0 == 0 && c0 + threadIdx.x < a.cols) a.s_col[c0 + threadIdx.x] = s;
  }
  for (int32_t tr = tr0; tr < tr1; ++tr) {
    const int64_t r0 = static_cast<int64_t>(tr) * 128;
    if (a.q_row && threadIdx.x >= 128) {
      const int64_t r = r0 + threadIdx.x - 128;
      uint32_t top = 0;
      if (r < a.rows) {
#pragma unroll 8
        for (int32_t p = 0; p < a.strips; ++p) top = max(top, a.part_row[static_cast<int64_t>(p) * a.rows + r]);
      }
      GroupScale g;
      const float s = group_scale(top, g);
      lds.row_scale[threadIdx.x - 128] = g;
      if (tc == 0 && r < a.rows) a.s_row[r] = s;
    }
    float x[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = raw[i].get(e);
    if (tr + 1 < tr1) fetch(tr + 1);
    uint32_t bits[4][8] = {};
    if constexpr (SR) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t p = a.base + static_cast<uint64_t>(r0 + rg * 4 + i) * static_cast<uint64_t>(a.cols) +
                           static_cast<uint64_t>(col);
        asr_mfma::random_run<8>(p, (p & 3u) == 0, args.seed, args.step, bits[i]);
      }
    }
    __syncthreads();  // the scales are there, the last tile's codes are read
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const GroupScale g = lds.col_scale[cg * 8 + e];
      const float v[4] = {x[0][e], x[1][e], x[2][e], x[3][e]};
      const uint32_t r[4] = {bits[0][e], bits[1][e], bits[2][e], bits[3][e]};
      lds.tile[(cg * 8 + e) * kWords + rg] = codes4<SR>(v, g, r);
    }
    if (a.q_row) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + rg * 4 + i;
        const GroupScale g = lds.row_scale[rg * 4 + i];
        const float v0[4] = {x[i][0], x[i][1], x[i][2], x[i][3]};
        const float v1[4] = {x[i][4], x[i][5], x[i][6], x[i][7]};
        const uint32_t b0[4] = {bits[i][0], bits[i][1], bits[i][2], bits[i][3]};
        const uint32_t b1[4] = {bits[i][4], bits[i][5], bits[i][6], bits[i][7]};
        const asr::u32x2 w = {codes4<SR>(v0, g, b0), codes4<SR>(v1, g, b1)};
        if (r < a.rows && col < (static_cast<int64_t>(a.cols) + 15) / 16 * 16)
          *reinterpret_cast<asr::u32x2*>(a.q_row + r * a.ld_row + col) = w;
      }
    }
    __syncthreads();
    for (int t = threadIdx.x; t < 64 * 8; t += 256) {
      const int cc = t / 8, part = t % 8;
      const int64_t r = r0 + part * 16;
      if (c0 + cc < a.cols && r < a.rows) {
        const uint32_t* w = lds.tile + cc * kWords + part * 4;
        *reinterpret_cast<asr::u32x4*>(a.q_col + (c0 + cc) * a.ld_col + r) = asr::u32x4{w[0], w[1], w[2], w[3]};
      }
    }
  }
}

template <typename S>
__global__ __launch_bounds__(256) void quantize_tiles(QuantArgs args) {
  __shared__ TileLds lds;
  const QuantJob& a = job_of(args);
  if (a.sr) quantize_strip<S, true>(args, a, lds);
  else quantize_strip<S, false>(args, a, lds);
}

// --------------------------------------------------------------- product
struct GemmArgs {
  const int8_t* a;
  const int8_t* b;
  const float* sa;
  const float* sb;
  uint16_t* c;
  float* c32;
  int64_t lda, ldb, ldc;
  uint64_t base_index;
  int32_t m, n, k;
  uint32_t tiles_m, tiles_n;
  uint32_t seed, step;
  uint32_t vec4;   // runs of 4 outputs start on 8-byte (f32: 16-byte) addresses
  uint32_t vec16;  // runs of 8 outputs start on 16-byte addresses, also f32 ones
  uint32_t pos4;   // runs of 4 outputs start on stream positions divisible by 4
};

template <int ROUND>
__device__ __forceinline__ uint32_t round_one(float x, uint32_t r16) {
  return ROUND == ASR_ROUND_SR ? asr::round_sr(__float_as_uint(x), r16)
                               : asr::round_rn(__float_as_uint(x));
}

using Big = asr_mfma::Tile<256, 256, 128, 64, 2>;
using Half = asr_mfma::Tile<256, 128, 64, 64, 2>;
using Small = asr_mfma::Tile<128, 128, 64, 64, 2>;
using Small8 = asr_mfma::Tile<128, 128, 64, 32, 3>;
using Tiny = asr_mfma::Tile<64, 64, 32, 32, 4>;

// `count` (4, or fewer at a row's end) outputs from C's element `at`.
__device__ __forceinline__ void store4(const GemmArgs& args, int64_t at, int count, const uint32_t (&h)[4],
                                       const float (&x)[4]) {
  if (args.vec4 && count == 4) {
    asr::store_vec_bf16<false, 4>(args.c + at, h);
    if (args.c32) asr::store_vec<false, 4>(args.c32 + at, x);
  } else {
    asr::store_range_bf16<4>(args.c, at, 0, count, h);
    if (args.c32) asr::store_range<4>(args.c32, at, 0, count, x);
  }
}

// The tile of C from (m0, n0). Bound by the matrix instructions and what keeps
// them fed (58% of the cycles busy at 8192 x 14336 x 4096: 433-472 us by box, 2.0-2.2 POP/s;
// 450 with stochastic rounding);
// the epilogue is the part no other work covers, so its stores go in whole
// lines. REST: K is not a multiple of 16 (a variant of
// its own: its byte loads cost the largest tile registers that it has not
// got). SPLIT: groups of T's waves that walk a share of K each (the integer sums
// are the same in any order), joined in LDS, and share the epilogue. smem: SPLIT
// times T's kLoopLds bytes.
template <typename T, int ROUND, bool REST, int SPLIT = 1>
__device__ __forceinline__ void gemm_tile(const GemmArgs& args, int64_t m0, int64_t n0, unsigned char* smem) {
  using E = asr_mfma::ElemI8;
  static_assert(asr_mfma::Rows<T>::kBytes <= T::kLoopLds, "the slices lie in the ring");
  E::acc acc[T::kFragM][T::kFragN] = {};
  asr_mfma::Operands op;
  op.a = reinterpret_cast<const char*>(args.a + m0 * args.lda);
  op.b = reinterpret_cast<const char*>(args.b + n0 * args.ldb);
  op.ld_a = static_cast<uint32_t>(args.lda);
  op.ld_b = static_cast<uint32_t>(args.ldb);
  op.last_a = args.m - 1 - static_cast<int32_t>(m0);
  op.last_b = args.n - 1 - static_cast<int32_t>(n0);
  op.kbytes = args.k & ~15;
  op.ktiles = asr_mfma::ktiles_of(op.kbytes);
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t wave = all_waves % T::kWaves;
  [[maybe_unused]] const uint32_t group = SPLIT > 1 ? all_waves / T::kWaves : 0;
  if constexpr (SPLIT > 1) {
    op.ktiles = (op.ktiles + SPLIT - 1) / SPLIT;
    const int32_t from = static_cast<int32_t>(group) * op.ktiles * asr_mfma::kRowBytes;
    op.kbytes = max(0, min(op.kbytes - from, op.ktiles * asr_mfma::kRowBytes));
    // (a group past K reads nothing; its pointers stay inside the rows)
    op.a += op.kbytes > 0 ? from : 0;
    op.b += op.kbytes > 0 ? from : 0;
    asr_mfma::mfma_loop<T, E>(op, smem + group * T::kLoopLds, acc);
  } else {
    asr_mfma::mfma_loop<T, E>(op, smem, acc);
  }

  const uint32_t wm = wave / T::kWavesN, wn = wave % T::kWavesN;
  [[maybe_unused]] const uint32_t row = lane & 31u, half = lane >> 5;

  // The last K % 16 codes of every row, byte by byte (what lies behind a
  // row's end is not read); lanes of the upper half hold zeros.
  if constexpr (REST) if (group == 0) {
    const int rest = args.k & 15;
    auto last_codes = [&](const int8_t* base, int64_t ld, int64_t r) {
      const int8_t* p = base + r * ld + (args.k - rest);
      uint32_t w[4] = {};
#pragma unroll
      for (int e = 0; e < 15; ++e)
        if (e < rest && half == 0) w[e / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(p[e])) << (8 * (e % 4));
      return E::frag{static_cast<int32_t>(w[0]), static_cast<int32_t>(w[1]),
                     static_cast<int32_t>(w[2]), static_cast<int32_t>(w[3])};
    };
    E::frag fb[T::kFragN];
#pragma unroll
    for (int j = 0; j < T::kFragN; ++j)
      fb[j] = last_codes(args.b, args.ldb,
                         min(n0 + wn * T::WN + j * 32 + row, static_cast<int64_t>(args.n - 1)));
#pragma unroll
    for (int i = 0; i < T::kFragM; ++i) {
      const E::frag fa = last_codes(
          args.a, args.lda, min(m0 + wm * T::WM + i * 32 + row, static_cast<int64_t>(args.m - 1)));
#pragma unroll
      for (int j = 0; j < T::kFragN; ++j) acc[i][j] = E::mfma(fb[j], fa, acc[i][j]);
    }
  }

  // Scaled, rounded and stored in runs of 8 columns, whole lines at a time.
  using Rows = asr_mfma::Rows<T>;
  static_assert(32 % Rows::kGroups == 0, "a lane's columns are those of every pass");
  __syncthreads();  // the last K tile is read
  static_assert(SPLIT == 1 || (T::kFragM == 1 && Rows::kPasses % SPLIT == 0), "passes shared evenly");
  uint32_t* first = reinterpret_cast<uint32_t*>(smem) + wave * (Rows::kSliceBytes / 4);
  uint32_t* slice = first + group * (Rows::kBytes / 4);
  uint32_t row0, col;
  Rows::place(0, lane, row0, col);
  const int64_t n = n0 + wn * T::WN + col;
  const int count = static_cast<int>(max(int64_t{0}, min(int64_t{8}, args.n - n)));
  float sb[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sb[e] = args.sb[min(n + e, static_cast<int64_t>(args.n - 1))];
  static_for<T::kFragM>([&](auto ic) {
    constexpr int i = decltype(ic)::value;
    Rows::put(slice, acc[i], lane);
    if constexpr (SPLIT > 1) __syncthreads();
    static_for<Rows::kPasses / SPLIT>([&](auto pc) {
      uint32_t r, same_col, raw[8];
      Rows::place(decltype(pc)::value * SPLIT + static_cast<int>(group), lane, r, same_col);
      Rows::get(first, r, col, raw);
#pragma unroll
      for (int g = 1; g < SPLIT; ++g) {
        uint32_t more[8];
        Rows::get(first + g * (Rows::kBytes / 4), r, col, more);
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[e] += more[e];
      }
      const int64_t m = m0 + wm * T::WM + i * 32 + r;
      if (m >= args.m || count == 0) return;
      const float sa = args.sa[m];
      uint32_t bits[8] = {}, h[8];
      if constexpr (ROUND == ASR_ROUND_SR) {
        const uint64_t pos = args.base_index + static_cast<uint64_t>(m) * static_cast<uint64_t>(args.n) +
                             static_cast<uint64_t>(n);
        asr_mfma::random_run<8>(pos, args.pos4 != 0, args.seed, args.step, bits);
      }
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = (static_cast<float>(static_cast<int32_t>(raw[e])) * sa) * sb[e];
        h[e] = round_one<ROUND>(x[e], bits[e]);
      }
      const int64_t at = m * args.ldc + n;
      if (args.vec16 && count == 8) {
        asr::store_vec_bf16<false, 8>(args.c + at, h);
        if (args.c32) asr::store_vec<false, 8>(args.c32 + at, x);
      } else {
        const uint32_t h0[4] = {h[0], h[1], h[2], h[3]}, h1[4] = {h[4], h[5], h[6], h[7]};
        const float x0[4] = {x[0], x[1], x[2], x[3]}, x1[4] = {x[4], x[5], x[6], x[7]};
        store4(args, at, min(count, 4), h0, x0);
        store4(args, at + 4, count - 4, h1, x1);
      }
    });
  });
}

template <typename T, int ROUND, bool REST, int SPLIT>
__global__ __launch_bounds__(SPLIT * T::kThreads, T::kMinWaves) void gemm_i8(GemmArgs args) {
  __shared__ __align__(1024) unsigned char smem[SPLIT * T::kLoopLds];
  uint32_t tm, tn;
  asr_mfma::grouped_tile(asr_mfma::xcd_order(blockIdx.x, args.tiles_m * args.tiles_n),
                         args.tiles_m, args.tiles_n, tm, tn);
  gemm_tile<T, ROUND, REST, SPLIT>(args, static_cast<int64_t>(tm) * T::BM, static_cast<int64_t>(tn) * T::BN, smem);
}

// Big tiles for as many whole rounds of the chip as there are, and what is left
// over, up to half a round, in twice as many half tiles: 4096 x 14336 x 4096,
// 3.5 rounds, takes 247 us instead of 250, 4200 x 4300 x 1000, 289 tiles, 53
// instead of 63.
template <int ROUND, bool REST>
__global__ __launch_bounds__(Big::kThreads, Big::kMinWaves) void gemm_i8_halves(GemmArgs args, uint32_t whole) {
  static_assert(Half::kThreads == Big::kThreads && Half::kLoopLds <= Big::kLoopLds && 2 * Half::BN == Big::BN);
  __shared__ __align__(1024) unsigned char smem[Big::kLoopLds];
  const uint32_t tiles = args.tiles_m * args.tiles_n;
  uint32_t tm, tn;
  if (blockIdx.x < whole) {
    asr_mfma::grouped_tile(asr_mfma::xcd_order(blockIdx.x, whole), args.tiles_m, args.tiles_n, tm, tn);
    gemm_tile<Big, ROUND, REST>(args, static_cast<int64_t>(tm) * Big::BM, static_cast<int64_t>(tn) * Big::BN, smem);
  } else {
    const uint32_t half = asr_mfma::xcd_order(blockIdx.x - whole, 2 * (tiles - whole));
    asr_mfma::grouped_tile(whole + half / 2, args.tiles_m, args.tiles_n, tm, tn);
    const int64_t n0 = static_cast<int64_t>(tn) * Big::BN + half % 2 * Half::BN;
    if (n0 < args.n) gemm_tile<Half, ROUND, REST>(args, static_cast<int64_t>(tm) * Half::BM, n0, smem);
  }
}

// A few rows of A (decoding): bound by reading B once (1 x 28672 x 8192, 235 MB:
// 41.8 us, 5.6 TB/s). A workgroup takes 16
// rows of B against MB blocks of 16 rows of A; its 8 waves split K in units of
// 128 bytes, with every load straight into the operand registers of a 16x16x64
// instruction (B on its row side, so a lane ends with 4 consecutive columns of
// one row of C). The waves' integer sums meet in LDS: no order to care for.
template <int MB, int ROUND>
__global__ __launch_bounds__(512) void gemm_i8_few(GemmArgs args) {
  using asr_mfma::i32x4;
  constexpr int kWaves = 8;
  __shared__ i32x4 sums[kWaves][MB][64];
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  // rows past the end are clamped: they only feed outputs that are not stored
  const int8_t* pb = args.b + min(n0 + (lane & 15u), static_cast<int64_t>(args.n - 1)) * args.ldb;
  const int8_t* pa[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
    pa[i] = args.a + min(static_cast<int64_t>(16 * i + (lane & 15u)), static_cast<int64_t>(args.m - 1)) * args.lda;
  const int32_t k_lane = static_cast<int32_t>(lane >> 4) * 32;
  i32x4 acc[MB] = {};
  const int32_t whole = args.k / 128;
  auto step = [&](int32_t unit, auto count) {
    constexpr int U = decltype(count)::value;
    i32x4 b[U][2], a[U][MB][2];
#pragma unroll
    for (int v = 0; v < U; ++v)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int32_t k = (unit + v * kWaves) * 128 + k_lane + 16 * h;
        b[v][h] = *reinterpret_cast<const i32x4*>(pb + k);
#pragma unroll
        for (int i = 0; i < MB; ++i) a[v][i][h] = *reinterpret_cast<const i32x4*>(pa[i] + k);
      }
#pragma unroll
    for (int v = 0; v < U; ++v)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MB; ++i)
          acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[v][h], a[v][i][h], acc[i], 0, 0, 0);
  };
  // 4 units a turn, all their loads first
  constexpr int kUnits = 4;
  int32_t u = static_cast<int32_t>(wave);
  for (; u + (kUnits - 1) * kWaves < whole; u += kUnits * kWaves) step(u, std::integral_constant<int, kUnits>{});
  for (; u < whole; u += kWaves) step(u, std::integral_constant<int, 1>{});
  if (args.k % 128 != 0 && whole % kWaves == static_cast<int32_t>(wave)) {
    // the last codes: whole 16-byte chunks by one load, the rest byte by byte
    auto tail = [&](const int8_t* row, int32_t k) {
      if (k + 16 <= args.k) return *reinterpret_cast<const i32x4*>(row + k);
      uint32_t w[4] = {};
#pragma unroll
      for (int e = 0; e < 15; ++e)
        if (k + e < args.k) w[e / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k + e])) << (8 * (e % 4));
      return i32x4{static_cast<int32_t>(w[0]), static_cast<int32_t>(w[1]),
                   static_cast<int32_t>(w[2]), static_cast<int32_t>(w[3])};
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int32_t k = whole * 128 + k_lane + 16 * h;
      const i32x4 b = tail(pb, k);
#pragma unroll
      for (int i = 0; i < MB; ++i)
        acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b, tail(pa[i], k), acc[i], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) sums[wave][i][lane] = acc[i];
  __syncthreads();
  if (wave >= MB) return;
  i32x4 t = sums[0][wave][lane];
#pragma unroll
  for (int v = 1; v < kWaves; ++v) t += sums[v][wave][lane];
  const int64_t m = 16 * wave + (lane & 15u), n = n0 + 4 * (lane >> 4);
  if (m >= args.m || n >= args.n) return;
  const float sa = args.sa[m];
  uint32_t r16[4] = {}, h[4];
  float x[4];
  if constexpr (ROUND == ASR_ROUND_SR)
    asr_mfma::random_run<4>(args.base_index + static_cast<uint64_t>(m) * static_cast<uint64_t>(args.n) +
                          static_cast<uint64_t>(n), args.pos4 != 0, args.seed, args.step, r16);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float sb = args.sb[min(n + e, static_cast<int64_t>(args.n - 1))];
    x[e] = (static_cast<float>(t[e]) * sa) * sb;
    h[e] = round_one<ROUND>(x[e], r16[e]);
  }
  store4(args, m * args.ldc + n, static_cast<int>(min(int64_t{4}, args.n - n)), h, x);
}

// C = 0 (a linear layer's sums over nothing).
__global__ __launch_bounds__(256) void clear(GemmArgs args) {
  const int64_t total = static_cast<int64_t>(args.m) * args.n;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256)
    args.c[i / args.n * args.ldc + i % args.n] = 0;
}

}  // namespace asr_i8

// =========================================================== host side
namespace {

using asr_host::fail;
using asr_host::hip_fail;
using asr_host::ok;

bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

constexpr int64_t kMaxDim = int64_t{1} << 31;

template <typename F>
hipError_t launch(F* f, int64_t grid, int threads, void* args, hipStream_t s) {
  void* argv[] = {args};
  return hipLaunchKernel(reinterpret_cast<const void*>(f), dim3(static_cast<uint32_t>(grid)), dim3(threads),
                         argv, 0, s);
}

// How the maxima of a rows x cols matrix are cut: strips of 256 columns, and
// chunks of rows (a multiple of 64), enough for about 1024 workgroups, 64 at most.
struct Cut {
  int32_t strips, chunk, chunks;
  Cut(int64_t rows, int64_t cols) {
    strips = static_cast<int32_t>((cols + 255) / 256);
    const int64_t want = std::clamp<int64_t>(1024 / strips, 1, 64);
    const int64_t c = ((rows + want - 1) / want + 63) / 64 * 64;
    chunk = static_cast<int32_t>(std::min<int64_t>(c, 0x7FFFFFC0));
    chunks = static_cast<int32_t>((rows + chunk - 1) / chunk);
  }
};

// Row codes of every job (which share their width), one launch.
template <typename S, bool SR>
hipError_t launch_rows(asr_i8::QuantArgs& a, hipStream_t s) {
  // 64 lanes hold a row of up to 2048 elements in registers
  const bool narrow = a.j[0].cols <= 2048;
  int64_t total = 0;
  for (int k = 0; k < a.count; ++k) {
    a.j[k].first = static_cast<uint32_t>(total);
    total += narrow ? (static_cast<int64_t>(a.j[k].rows) + 3) / 4 : a.j[k].rows;
  }
  return narrow ? launch(&asr_i8::quantize_rows<S, SR, 64>, total, 256, &a, s)
                : launch(&asr_i8::quantize_rows<S, SR, 256>, total, 256, &a, s);
}

// Column codes of every job, and row codes of those that want them too.
template <typename S>
hipError_t launch_tiles(asr_i8::QuantArgs& a, hipStream_t s) {
  constexpr int32_t kJoin = 16;  // strips a tile reads itself: half a matrix row's bytes at most
  int64_t total = 0;
  // One tile of rows finds its columns' maxima itself, in one launch: 128 x 64 to
  // 8192 6.5 to 8.0 us instead of 10.0 to 11.9. (A strip of two tiles, walked twice
  // by its workgroup: 10.1 to 12.3 against 10.6 to 11.9.)
  const bool alone = a.count == 1 && !a.j[0].q_row && a.j[0].rows <= 128;
  for (int k = 0; k < a.count; ++k) {
    asr_i8::QuantJob& j = a.j[k];
    const Cut cut(j.rows, j.cols);
    j.strips = cut.strips;
    j.chunk = cut.chunk;
    j.chunks = alone ? 0 : cut.chunks;
    j.first = static_cast<uint32_t>(total);
    j.blocks = static_cast<uint32_t>(cut.strips * cut.chunks);
    total += j.blocks;
  }
  hipError_t e = alone ? hipSuccess : launch(&asr_i8::maxima<S>, total, 256, &a, s);
  total = 0;
  for (int k = 0; k < a.count && e == hipSuccess; ++k) {
    asr_i8::QuantJob& j = a.j[k];
    if (j.q_row && j.strips > kJoin) {
      void* argv[] = {&j.part_row, &j.rows, &j.strips};
      e = hipLaunchKernel(reinterpret_cast<const void*>(&asr_i8::join_strips),
                          dim3(static_cast<uint32_t>((static_cast<int64_t>(j.rows) + 255) / 256)), dim3(256),
                          argv, 0, s);
      j.strips = 1;
    }
    j.first = static_cast<uint32_t>(total);
    // up to 4 tiles a workgroup, as long as there are about 2048 workgroups
    const int64_t across = (static_cast<int64_t>(j.cols) + 63) / 64, down = (static_cast<int64_t>(j.rows) + 127) / 128;
    j.tiles = static_cast<int32_t>(std::clamp<int64_t>(across * down / 2048, 1, 4));
    j.blocks = static_cast<uint32_t>(across * ((down + j.tiles - 1) / j.tiles));
    total += j.blocks;
  }
  return e == hipSuccess ? launch(&asr_i8::quantize_tiles<S>, total, 256, &a, s) : e;
}

// A launch has fewer than 2**32 threads: of 256-thread workgroups, this many.
constexpr int64_t kMaxBlocks = 0xFFFFFF;

bool too_many_blocks(int64_t rows, int64_t cols, bool transpose) {
  // (the kernels count rows in 32 bits, 32 at a time past the last one)
  if (transpose) return ((cols + 63) / 64) * ((rows + 127) / 128) > kMaxBlocks || rows > kMaxDim - 64;
  return (cols <= 2048 ? (rows + 3) / 4 : rows) > kMaxBlocks;
}

int64_t padded16(int64_t x) { return (x + 15) / 16 * 16; }

// Consecutive parts of a workspace, each on a 256-byte boundary.
struct Parts {
  char* base;
  int64_t at = 0;
  explicit Parts(void* p) : base(static_cast<char*>(p)) {}
  template <typename P>
  P* take(int64_t count) {
    P* p = reinterpret_cast<P*>(base + at);
    at += (count * static_cast<int64_t>(sizeof(P)) + 255) / 256 * 256;
    return p;
  }
};

template <typename T, int SPLIT = 1>
hipError_t launch_gemm(asr_i8::GemmArgs args, int32_t rounding, hipStream_t s) {
  using namespace asr_i8;
  args.tiles_m = static_cast<uint32_t>((args.m + T::BM - 1) / T::BM);
  args.tiles_n = static_cast<uint32_t>((args.n + T::BN - 1) / T::BN);
  const int64_t grid = static_cast<int64_t>(args.tiles_m) * args.tiles_n;
  const bool rest = args.k % 16 != 0;
  if (rounding == ASR_ROUND_SR)
    return rest ? launch(&gemm_i8<T, ASR_ROUND_SR, true, SPLIT>, grid, SPLIT * T::kThreads, &args, s)
               : launch(&gemm_i8<T, ASR_ROUND_SR, false, SPLIT>, grid, SPLIT * T::kThreads, &args, s);
  return rest ? launch(&gemm_i8<T, ASR_ROUND_RN, true, SPLIT>, grid, SPLIT * T::kThreads, &args, s)
             : launch(&gemm_i8<T, ASR_ROUND_RN, false, SPLIT>, grid, SPLIT * T::kThreads, &args, s);
}

constexpr int64_t kCus = 256;  // compute units of an MI355X, one big tile each

hipError_t launch_halves(asr_i8::GemmArgs args, int32_t rounding, hipStream_t s) {
  using namespace asr_i8;
  args.tiles_m = static_cast<uint32_t>((args.m + Big::BM - 1) / Big::BM);
  args.tiles_n = static_cast<uint32_t>((args.n + Big::BN - 1) / Big::BN);
  const uint32_t tiles = args.tiles_m * args.tiles_n;
  uint32_t whole = tiles / kCus * kCus;
  void* argv[] = {&args, &whole};
  const bool rest = args.k % 16 != 0;
  const void* f = rounding == ASR_ROUND_SR
                      ? (rest ? reinterpret_cast<const void*>(&gemm_i8_halves<ASR_ROUND_SR, true>)
                              : reinterpret_cast<const void*>(&gemm_i8_halves<ASR_ROUND_SR, false>))
                      : (rest ? reinterpret_cast<const void*>(&gemm_i8_halves<ASR_ROUND_RN, true>)
                              : reinterpret_cast<const void*>(&gemm_i8_halves<ASR_ROUND_RN, false>));
  return hipLaunchKernel(f, dim3(whole + 2 * (tiles - whole)), dim3(Big::kThreads), argv, 0, s);
}

template <int MB>
hipError_t launch_few(asr_i8::GemmArgs args, int32_t rounding, hipStream_t s) {
  using namespace asr_i8;
  const int64_t grid = (static_cast<int64_t>(args.n) + 15) / 16;
  return rounding == ASR_ROUND_SR ? launch(&gemm_i8_few<MB, ASR_ROUND_SR>, grid, 512, &args, s)
                                  : launch(&gemm_i8_few<MB, ASR_ROUND_RN>, grid, 512, &args, s);
}

// The product after its arguments were checked.
hipError_t product(const asr_i8::GemmArgs& g, int32_t rounding, hipStream_t s) {
  const int64_t m = g.m, n = g.n;
  auto tiles = [&](int64_t t) { return ((m + t - 1) / t) * ((n + t - 1) / t); };
  // Few rows: reading B is all there is, and the kernel for them keeps more of
  // it in flight than tiles do, with one workgroup for 16 columns on every
  // compute unit (16 x 4096 x 4096: 7.2 us against 9.0 in 64 x 64 tiles; 16 x
  // 256 x 14336: 14.8 against 21.9; 32 x 5120 x 5120, more of them than
  // compute units: 16.0 against 10.8), or for any N up to 4 rows (1 x 28672 x
  // 8192: 41.7 against 53.2; 1 x 16384 x 8192: 25.8 against 33.6; 1 x 14336 x 7168
  // in rows of 7184 bytes: 23.7 against 24.2), unless K is too short to split (1 x
  // 100000 x 64: 21.0 against 11.3). Rows a multiple of 4096 bytes apart meet in the
  // same memory channels, which costs this kernel, whose workgroup reads 16 rows at
  // one place, more than the tile (1 x 14336 x 4096: 15.8 against 13.6, in rows of
  // 4224 bytes 13.4 against 13.7; 4 x 10240 x 3584 in rows of 4096: 11.9 against
  // 11.0), as long as most compute units get one tile (1 x 8192 x 4096: 10.4
  // against 11.0; 1 x 16400 x 4096: 17.6 against 20.3) of a K up to 4096 (2048: 10.1
  // against 10.4; 8192: 24.9 against 29.6). (Not followed: 4 rows of 14336 columns
  // with a longer K, 7168: 23.8 against 20.9.) All with B from memory.
  // (n below 2**26: a launch's threads)
  const bool one_each = n > 64 * (kCus / 2) && n <= 64 * kCus && g.k >= 2560 && g.k <= 4096 && g.ldb % 4096 == 0;
  if ((m <= 32 && n <= 16 * kCus) || (m <= 4 && g.k >= 512 && n < (int64_t{1} << 26) && !one_each))
    return m <= 16 ? launch_few<1>(g, rounding, s) : launch_few<2>(g, rounding, s);
  // (1000 x 14336 x 4096, 224 tiles of 256: 63 us, 80 us in 128 x 128 tiles;
  // 512 x 14336 x 4096, 112 of them: 55 and 44 us)
  if (const int64_t left = tiles(256) % kCus; tiles(256) > kCus && left > 0 && left <= kCus / 2)
    return launch_halves(g, rounding, s);
  if (tiles(256) >= 192) return launch_gemm<asr_i8::Big>(g, rounding, s);
  if (tiles(128) > 256) return launch_gemm<asr_i8::Small>(g, rounding, s);
  if (tiles(128) > 128) return launch_gemm<asr_i8::Small8>(g, rounding, s);
  // one tile or none a compute unit: two K ranges in it (333 x 1009 x 1111: 8.6 ->
  // 8.1 us, 256 x 4096 x 4096: 12.2 -> 10.2, 100 x 200 x 8192: 19.4 -> 14.6)
  if (tiles(64) <= kCus) return launch_gemm<asr_i8::Tiny, 2>(g, rounding, s);
  return launch_gemm<asr_i8::Tiny>(g, rounding, s);
}

asr_i8::GemmArgs gemm_args(const int8_t* a, int64_t lda, const int8_t* b, int64_t ldb, const float* sa,
                           const float* sb, uint16_t* c, int64_t ldc, float* c_f32, int64_t m, int64_t n,
                           int64_t k) {
  asr_i8::GemmArgs g{};
  g.a = a;
  g.b = b;
  g.sa = sa;
  g.sb = sb;
  g.c = c;
  g.c32 = c_f32;
  g.lda = lda;
  g.ldb = ldb;
  g.ldc = ldc;
  g.m = static_cast<int32_t>(m);
  g.n = static_cast<int32_t>(n);
  g.k = static_cast<int32_t>(k);
  g.vec4 = ldc % 4 == 0 && aligned_to(c, 8) && (!c_f32 || aligned_to(c_f32, 16));
  g.vec16 = ldc % 8 == 0 && aligned_to(c, 16) && (!c_f32 || aligned_to(c_f32, 16));
  return g;
}

asr_i8::QuantJob matrix_job(const void* x, int64_t ldx, int64_t size, int64_t rows, int64_t cols) {
  asr_i8::QuantJob j{};
  j.x = x;
  j.ldx = ldx;
  j.rows = static_cast<int32_t>(rows);
  j.cols = static_cast<int32_t>(cols);
  j.vec = aligned_to(x, 16) && (rows == 1 || ldx * size % 16 == 0);
  return j;
}

// The buffers of the linear layer's two calls in their workspace.
struct LinearForward {
  int8_t *qx, *qw;
  float *sx, *sw;
  int64_t bytes;
  LinearForward(void* ws, int64_t t, int64_t n, int64_t k) {
    Parts p(ws);
    qx = p.take<int8_t>(t * padded16(k));
    qw = p.take<int8_t>(n * padded16(k));
    sx = p.take<float>(t);
    sw = p.take<float>(n);
    bytes = p.at;
  }
};

struct LinearBackward {
  int8_t *qd, *qdt, *qwt, *qxt;
  float *sd, *sdt, *swt, *sxt;
  uint32_t *pd_row, *pd, *pw, *px;
  int64_t bytes;
  LinearBackward(void* ws, int64_t t, int64_t n, int64_t k) {
    Parts p(ws);
    qd = p.take<int8_t>(t * padded16(n));
    qdt = p.take<int8_t>(n * padded16(t));
    qwt = p.take<int8_t>(k * padded16(n));
    qxt = p.take<int8_t>(k * padded16(t));
    sd = p.take<float>(t);
    sdt = p.take<float>(n);
    swt = p.take<float>(k);
    sxt = p.take<float>(k);
    pd_row = p.take<uint32_t>(t * Cut(t, n).strips);
    pd = p.take<uint32_t>(n * Cut(t, n).chunks);
    pw = p.take<uint32_t>(k * Cut(n, k).chunks);
    px = p.take<uint32_t>(k * Cut(t, k).chunks);
    bytes = p.at;
  }
};

constexpr int64_t kMaxSum = int64_t{1} << 17;  // int8 products summed in 32 bits

int check_linear(int64_t t, int64_t n, int64_t k) {
  if (t < 0 || n < 0 || k < 0 || t >= kMaxSum || n >= kMaxSum || k >= kMaxSum)
    return fail(ASR_EINVAL, "linear_i8: tokens, n and k must be in [0, 2**17)");
  return ASR_OK;
}

// An operand of rows x cols bf16 values with row stride ld.
int check_operand(const void* p, int64_t ld, int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return ASR_OK;
  if (!p) return fail(ASR_EINVAL, "linear_i8: null matrix pointer");
  if (ld < cols) return fail(ASR_EINVAL, "linear_i8: a row stride is below the row's length");
  if (!aligned_to(p, 2)) return fail(ASR_EALIGN, "linear_i8: matrices must be aligned to 2 bytes");
  return ASR_OK;
}

}  // namespace

extern "C" {

size_t asr_quantize_i8_workspace_bytes(int64_t rows, int64_t cols, int32_t transpose) {
  if (!transpose || rows <= 0 || cols <= 0 || rows >= kMaxDim || cols >= kMaxDim) return 0;
  return static_cast<size_t>((Cut(rows, cols).chunks * cols * 4 + 255) / 256 * 256);
}

int asr_quantize_i8(const void* x, int32_t dtype, int64_t ldx, int64_t rows, int64_t cols,
                    int32_t transpose, int8_t* q, int64_t ldq, float* scale, int32_t rounding,
                    uint32_t seed, uint32_t step, uint64_t base_index, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (rows < 0 || cols < 0 || rows >= kMaxDim || cols >= kMaxDim)
    return fail(ASR_EINVAL, "quantize_i8: rows and cols must be in [0, 2**31)");
  if (dtype != ASR_F32 && dtype != ASR_BF16) return fail(ASR_EDTYPE, "quantize_i8: unknown dtype");
  if (rounding != ASR_ROUND_SR && rounding != ASR_ROUND_RN)
    return fail(ASR_EINVAL, "quantize_i8: rounding must be ASR_ROUND_SR or ASR_ROUND_RN");
  const int64_t groups = transpose ? cols : rows, length = transpose ? rows : cols;
  if (groups == 0) return ok();
  if (!scale || (length > 0 && (!x || !q))) return fail(ASR_EINVAL, "quantize_i8: null pointer");
  if (ldx < cols) return fail(ASR_EINVAL, "quantize_i8: ldx >= cols");
  if (ldq < padded16(length) || ldq % 16 != 0)
    return fail(ASR_EINVAL, "quantize_i8: ldq must be a multiple of 16 and hold a group's codes "
                            "up to a multiple of 16");
  const int64_t size = dtype == ASR_F32 ? 4 : 2;
  if (!aligned_to(x, size) || !aligned_to(scale, 4) || !aligned_to(q, 16))
    return fail(ASR_EALIGN, "quantize_i8: x and scale aligned to their elements, q to 16 bytes");
  if (length > 0 && static_cast<uint64_t>(rows) * static_cast<uint64_t>(cols) - 1 > ~base_index)
    return fail(ASR_EINVAL, "quantize_i8: base_index + rows*cols exceeds 2**64");
  if (too_many_blocks(length == 0 ? groups : rows, length == 0 ? 0 : cols, transpose && length > 0))
    return fail(ASR_EINVAL, "quantize_i8: the matrix is too large for one call");
  if (transpose && length > 0) {
    if (!workspace || !aligned_to(workspace, 16) ||
        workspace_bytes < asr_quantize_i8_workspace_bytes(rows, cols, transpose))
      return fail(ASR_EWORKSPACE, "quantize_i8: workspace NULL, too small or not 16-byte aligned");
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool sr = rounding == ASR_ROUND_SR;
  asr_i8::QuantArgs a{};
  a.count = 1;
  a.seed = seed;
  a.step = step;
  asr_i8::QuantJob& j = a.j[0];
  // (a group without elements still gets its scale, 0: as a row of none)
  const bool rows_form = !transpose || length == 0;
  j = matrix_job(x, ldx, size, transpose && length == 0 ? cols : rows, transpose && length == 0 ? 0 : cols);
  j.base = base_index;
  j.sr = sr;
  hipError_t e;
  if (rows_form) {
    j.q_row = q;
    j.ld_row = ldq;
    j.s_row = scale;
    if (dtype == ASR_F32) e = sr ? launch_rows<float, true>(a, s) : launch_rows<float, false>(a, s);
    else e = sr ? launch_rows<uint16_t, true>(a, s) : launch_rows<uint16_t, false>(a, s);
  } else {
    j.q_col = q;
    j.ld_col = ldq;
    j.s_col = scale;
    j.part_col = static_cast<uint32_t*>(workspace);
    e = dtype == ASR_F32 ? launch_tiles<float>(a, s) : launch_tiles<uint16_t>(a, s);
  }
  return e == hipSuccess ? ok() : hip_fail(e, "quantize_i8 launch");
}

int asr_gemm_i8(const int8_t* a, int64_t lda, const int8_t* b, int64_t ldb, const float* scale_a,
                const float* scale_b, uint16_t* c, int64_t ldc, float* c_f32, int64_t m, int64_t n,
                int64_t k, int32_t rounding, uint32_t seed, uint32_t step, uint64_t base_index,
                void* stream) {
  if (m < 0 || n < 0 || m >= kMaxDim || n >= kMaxDim)
    return fail(ASR_EINVAL, "gemm_i8: m and n must be in [0, 2**31)");
  if (k < 0 || k >= (int64_t{1} << 17))
    return fail(ASR_EINVAL, "gemm_i8: k must be in [0, 2**17) (the sums are 32-bit integers)");
  if (rounding != ASR_ROUND_SR && rounding != ASR_ROUND_RN)
    return fail(ASR_EINVAL, "gemm_i8: rounding must be ASR_ROUND_SR or ASR_ROUND_RN");
  if (m == 0 || n == 0) return ok();
  if (!c || !scale_a || !scale_b || (k > 0 && (!a || !b)))
    return fail(ASR_EINVAL, "gemm_i8: null pointer");
  if (lda < k || ldb < k || ldc < n) return fail(ASR_EINVAL, "gemm_i8: lda, ldb >= k and ldc >= n");
  if (lda >= asr_mfma::kMaxLdBytes || ldb >= asr_mfma::kMaxLdBytes)
    return fail(ASR_EINVAL, "gemm_i8: lda and ldb must be below 2**23");
  if (lda % 16 != 0 || ldb % 16 != 0)
    return fail(ASR_EALIGN, "gemm_i8: lda and ldb must be multiples of 16");
  if (!aligned_to(a, 16) || !aligned_to(b, 16))
    return fail(ASR_EALIGN, "gemm_i8: A and B must be 16-byte aligned");
  if (!aligned_to(scale_a, 4) || !aligned_to(scale_b, 4) || !aligned_to(c, 2) ||
      (c_f32 && !aligned_to(c_f32, 4)))
    return fail(ASR_EALIGN, "gemm_i8: scales and outputs must be aligned to their element size");
  if (static_cast<uint64_t>(m) * static_cast<uint64_t>(n) - 1 > ~base_index)
    return fail(ASR_EINVAL, "gemm_i8: base_index + m*n exceeds 2**64");
  // (launches of fewer than 2**32 threads, with room for a last round of halves)
  if (((m + 255) / 256) * ((n + 255) / 256) > (int64_t{1} << 23) - kCus)
    return fail(ASR_EINVAL, "gemm_i8: too many tiles");
  asr_i8::GemmArgs g = gemm_args(a, lda, b, ldb, scale_a, scale_b, c, ldc, c_f32, m, n, k);
  g.base_index = base_index;
  g.seed = seed;
  g.step = step;
  g.pos4 = base_index % 4 == 0 && n % 4 == 0;
  const hipError_t e = product(g, rounding, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "gemm_i8 launch");
}

size_t asr_linear_i8_workspace_bytes(int64_t tokens, int64_t n, int64_t k, int32_t backward) {
  if (tokens < 0 || n < 0 || k < 0 || tokens >= kMaxSum || n >= kMaxSum || k >= kMaxSum) return 0;
  if (tokens == 0 || n == 0 || k == 0) return 0;
  return static_cast<size_t>(backward ? LinearBackward(nullptr, tokens, n, k).bytes
                                      : LinearForward(nullptr, tokens, n, k).bytes);
}

int asr_linear_i8_forward(const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw, uint16_t* y,
                          int64_t ldy, int64_t tokens, int64_t n, int64_t k, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (int rc = check_linear(tokens, n, k)) return rc;
  if (int rc = check_operand(x, ldx, tokens, k)) return rc;
  if (int rc = check_operand(w, ldw, n, k)) return rc;
  if (int rc = check_operand(y, ldy, tokens, n)) return rc;
  if (tokens == 0 || n == 0) return ok();
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (k == 0) {  // the empty sum
    const float* none = nullptr;
    asr_i8::GemmArgs g = gemm_args(nullptr, 16, nullptr, 16, none, none, y, ldy, nullptr, tokens, n, 0);
    const hipError_t e = launch(&asr_i8::clear, std::min<int64_t>((tokens * n + 255) / 256, 65536), 256, &g, s);
    return e == hipSuccess ? ok() : hip_fail(e, "linear_i8 launch");
  }
  if (!workspace || !aligned_to(workspace, 256) ||
      workspace_bytes < asr_linear_i8_workspace_bytes(tokens, n, k, 0))
    return fail(ASR_EWORKSPACE, "linear_i8: workspace NULL, too small or not 256-byte aligned");
  const LinearForward f(workspace, tokens, n, k);
  asr_i8::QuantArgs a{};
  a.count = 2;
  a.j[0] = matrix_job(x, ldx, 2, tokens, k);
  a.j[0].q_row = f.qx;
  a.j[0].s_row = f.sx;
  a.j[1] = matrix_job(w, ldw, 2, n, k);
  a.j[1].q_row = f.qw;
  a.j[1].s_row = f.sw;
  a.j[0].ld_row = a.j[1].ld_row = padded16(k);
  hipError_t e = launch_rows<uint16_t, false>(a, s);
  if (e == hipSuccess)
    e = product(gemm_args(f.qx, padded16(k), f.qw, padded16(k), f.sx, f.sw, y, ldy, nullptr, tokens, n, k),
                ASR_ROUND_RN, s);
  return e == hipSuccess ? ok() : hip_fail(e, "linear_i8 launch");
}

int asr_linear_i8_backward(const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw,
                           const uint16_t* dy, int64_t lddy, uint16_t* dx, int64_t lddx, uint16_t* dw,
                           int64_t lddw, int64_t tokens, int64_t n, int64_t k, int32_t rounding,
                           uint32_t seed, uint32_t step, uint64_t base_index, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (int rc = check_linear(tokens, n, k)) return rc;
  if (rounding != ASR_ROUND_SR && rounding != ASR_ROUND_RN)
    return fail(ASR_EINVAL, "linear_i8: rounding must be ASR_ROUND_SR or ASR_ROUND_RN");
  if (dw)
    if (int rc = check_operand(x, ldx, tokens, k)) return rc;
  if (dx)
    if (int rc = check_operand(w, ldw, n, k)) return rc;
  if (dx || dw)
    if (int rc = check_operand(dy, lddy, tokens, n)) return rc;
  if (dx)
    if (int rc = check_operand(dx, lddx, tokens, k)) return rc;
  if (dw)
    if (int rc = check_operand(dw, lddw, n, k)) return rc;
  if (tokens > 0 && n > 0 && static_cast<uint64_t>(tokens) * static_cast<uint64_t>(n) - 1 > ~base_index)
    return fail(ASR_EINVAL, "linear_i8: base_index + tokens*n exceeds 2**64");
  if ((!dx && !dw) || k == 0) return ok();
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (tokens == 0 || n == 0) {  // empty sums
    asr_i8::GemmArgs g = tokens == 0 ? gemm_args(nullptr, 16, nullptr, 16, nullptr, nullptr, dw, lddw, nullptr, n, k, 0)
                                     : gemm_args(nullptr, 16, nullptr, 16, nullptr, nullptr, dx, lddx, nullptr, tokens, k, 0);
    if (g.c && g.m > 0) e = launch(&asr_i8::clear, std::min<int64_t>((static_cast<int64_t>(g.m) * g.n + 255) / 256, 65536), 256, &g, s);
    return e == hipSuccess ? ok() : hip_fail(e, "linear_i8 launch");
  }
  if (!workspace || !aligned_to(workspace, 256) ||
      workspace_bytes < asr_linear_i8_workspace_bytes(tokens, n, k, 1))
    return fail(ASR_EWORKSPACE, "linear_i8: workspace NULL, too small or not 256-byte aligned");
  const LinearBackward f(workspace, tokens, n, k);
  asr_i8::QuantArgs a{};
  a.seed = seed;
  a.step = step;
  asr_i8::QuantJob d = matrix_job(dy, lddy, 2, tokens, n);
  d.base = base_index;
  d.sr = rounding == ASR_ROUND_SR;
  if (dx) {
    d.q_row = f.qd;
    d.s_row = f.sd;
    d.part_row = f.pd_row;
    d.ld_row = padded16(n);
  }
  if (dw) {
    d.q_col = f.qdt;
    d.s_col = f.sdt;
    d.part_col = f.pd;
    d.ld_col = padded16(tokens);
    a.j[a.count++] = d;
    asr_i8::QuantJob& j = a.j[a.count++];
    j = matrix_job(x, ldx, 2, tokens, k);
    j.q_col = f.qxt;
    j.s_col = f.sxt;
    j.part_col = f.px;
    j.ld_col = padded16(tokens);
  } else {  // only the rows of dy
    a.count = 1;
    a.j[0] = d;
    e = d.sr ? launch_rows<uint16_t, true>(a, s) : launch_rows<uint16_t, false>(a, s);
    a.count = 0;
  }
  if (dx) {
    asr_i8::QuantJob& j = a.j[a.count++];
    j = matrix_job(w, ldw, 2, n, k);
    j.q_col = f.qwt;
    j.s_col = f.swt;
    j.part_col = f.pw;
    j.ld_col = padded16(n);
  }
  if (e == hipSuccess) e = launch_tiles<uint16_t>(a, s);
  if (e == hipSuccess && dx)
    e = product(gemm_args(f.qd, padded16(n), f.qwt, padded16(n), f.sd, f.swt, dx, lddx, nullptr, tokens, k, n),
                ASR_ROUND_RN, s);
  if (e == hipSuccess && dw)
    e = product(gemm_args(f.qdt, padded16(tokens), f.qxt, padded16(tokens), f.sdt, f.sxt, dw, lddw, nullptr, n, k,
                          tokens), ASR_ROUND_RN, s);
  return e == hipSuccess ? ok() : hip_fail(e, "linear_i8 launch");
}

}  // extern "C"
