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
struct GroupScale {
  float s;     // the scale the group's codes are divided by, times k
  float inv;   // 1 / s
  float k;     // power of two that keeps every product with s a normal number
  uint32_t live;  // 0: every code is 0 (no element, only tiny ones, Inf or NaN)
};

// The scale to store for a group whose largest |x| has these bits, and what
// the codes need. Below 127 * 2**-126 the scale would be subnormal: such a
// group is stored as zeros. Inf or NaN anywhere makes the scale NaN, which
// every product with the group then shows.
__device__ __forceinline__ float group_scale(uint32_t max_bits, GroupScale& g) {
  const float s = __uint_as_float(max_bits) / 127.0f;
  const bool finite = max_bits < 0x7F800000u;
  g.live = finite && s >= 0x1p-126f;
  g.k = s < 0x1p-60f ? 0x1p64f : 1.0f;
  g.s = g.live ? s * g.k : 1.0f;
  g.inv = 1.0f / g.s;
  return finite ? (g.live ? s : 0.0f) : __uint_as_float(0x7FC00000u);
}

template <bool SR>
__device__ __forceinline__ int32_t quantize(float x, const GroupScale& g, uint32_t r16) {
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
  i = x < 0.0f ? -i : i;
  return g.live ? i : 0;
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

__device__ __forceinline__ uint32_t pack4(const int32_t (&q)[4]) {
  return (q[0] & 0xFF) | ((q[1] & 0xFF) << 8) | ((q[2] & 0xFF) << 16) |
         (static_cast<uint32_t>(q[3]) << 24);
}

__device__ __forceinline__ void random8(uint64_t p, uint32_t seed, uint32_t step,
                                        uint32_t (&r)[8]) {
  const bool aligned = (p & 3u) == 0;
  uint32_t lo[4], hi[4];
  asr_mfma::random4(p, aligned, seed, step, lo);
  asr_mfma::random4(p + 4, aligned, seed, step, hi);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    r[e] = lo[e];
    r[4 + e] = hi[e];
  }
}

struct QuantArgs {
  const void* x;
  int8_t* q;
  float* scale;
  uint32_t* part;  // transposed form: column maxima of each chunk of rows
  int64_t ldx, rows, cols, ldq;
  uint64_t base_index;
  uint32_t seed, step;
  uint32_t vec;       // every 8-element run of a row starts on a 16-byte address
  int32_t chunk, chunks;
};

// One row by LANES lanes (64: four rows a workgroup, 256: one). The first
// KEEP runs of 8 a lane holds stay in registers between the pass for the
// maximum and the pass for the codes; a longer row's others are read again.
template <typename S, bool SR, int LANES>
__global__ __launch_bounds__(256) void quantize_rows(QuantArgs a) {
  constexpr int KEEP = 4;
  constexpr int kRowsHere = 256 / LANES;
  const int lane = threadIdx.x % LANES;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsHere + threadIdx.x / LANES;
  if (LANES == 64 && row >= a.rows) return;  // (whole waves; no barrier follows for LANES == 64)
  const S* x = static_cast<const S*>(a.x) + row * a.ldx;
  const int64_t runs = (a.cols + 15) / 16 * 2;  // codes are written up to a multiple of 16
  float keep[KEEP][8];
  uint32_t top = 0;
#pragma unroll
  for (int v = 0; v < KEEP; ++v) {
    const int64_t run = lane + static_cast<int64_t>(v) * LANES;
    if (run < runs) {
      load8<S>(x, run * 8, a.cols, a.vec, keep[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, abs_bits(keep[v][e]));
    }
  }
  for (int64_t run = lane + static_cast<int64_t>(KEEP) * LANES; run < runs; run += LANES) {
    float t[8];
    load8<S>(x, run * 8, a.cols, a.vec, t);
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
  if (lane == 0) a.scale[row] = s;
  int8_t* q = a.q + row * a.ldq;
  auto codes = [&](int64_t run, const float (&t)[8]) {
    uint32_t r[8] = {};
    if constexpr (SR)
      random8(a.base_index + static_cast<uint64_t>(row) * static_cast<uint64_t>(a.cols) +
                  static_cast<uint64_t>(run) * 8, a.seed, a.step, r);
    int32_t lo[4], hi[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[e] = quantize<SR>(t[e], g, r[e]);
      hi[e] = quantize<SR>(t[4 + e], g, r[4 + e]);
    }
    *reinterpret_cast<asr::u32x2*>(q + run * 8) = asr::u32x2{pack4(lo), pack4(hi)};
  };
#pragma unroll
  for (int v = 0; v < KEEP; ++v) {
    const int64_t run = lane + static_cast<int64_t>(v) * LANES;
    if (run < runs) codes(run, keep[v]);
  }
  for (int64_t run = lane + static_cast<int64_t>(KEEP) * LANES; run < runs; run += LANES) {
    float t[8];
    load8<S>(x, run * 8, a.cols, a.vec, t);
    codes(run, t);
  }
}

// Column maxima of one chunk of rows: a workgroup takes 128 columns (256
// bytes of a bf16 row) and 16 rows at a time. Few chunks, so that the second
// kernel reads few of them; narrow strips, so that few chunks fill the chip.
template <typename S>
__global__ __launch_bounds__(256) void column_maxima(QuantArgs a) {
  __shared__ uint32_t tops[16][128 + 4];
  const int cg = threadIdx.x % 16, rr = threadIdx.x / 16;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * 128, col = c0 + cg * 8;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * a.chunk;
  const int64_t r1 = min(a.rows, r0 + a.chunk);
  uint32_t top[8] = {};
  if (col < a.cols) {
#pragma unroll 4
    for (int64_t r = r0 + rr; r < r1; r += 16) {
      float t[8];
      load8<S>(static_cast<const S*>(a.x) + r * a.ldx, col, a.cols, a.vec, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) top[e] = max(top[e], abs_bits(t[e]));
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) tops[rr][cg * 8 + e] = top[e];
  __syncthreads();
  if (threadIdx.x < 128 && c0 + threadIdx.x < a.cols) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, tops[i][threadIdx.x]);
    a.part[static_cast<int64_t>(blockIdx.y) * a.cols + c0 + threadIdx.x] = m;
  }
}

// Codes of a tile of 128 rows x 64 columns of x, written as 64 rows of 128
// codes of the transposed result. A thread takes 4 consecutive rows of 8
// columns, so 4 codes of one column make one LDS word.
template <typename S, bool SR>
__global__ __launch_bounds__(256) void quantize_columns(QuantArgs a) {
  constexpr int kWords = 33;  // LDS words a column: 32 and one against bank conflicts
  __shared__ uint32_t tile[64 * kWords];
  __shared__ uint32_t tops[4][64];
  __shared__ __align__(16) GroupScale scales[64];
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * 64;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 128;
  const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3;  // 8 columns, rows rg * 4 .. + 3
  const int64_t col = c0 + cg * 8;
  float x[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + rg * 4 + i;
    if (r < a.rows && col < a.cols) {
      load8<S>(static_cast<const S*>(a.x) + r * a.ldx, col, a.cols, a.vec, x[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
    }
  }
  const int c = threadIdx.x % 64, quarter = threadIdx.x / 64;
  uint32_t top = 0;
  if (c0 + c < a.cols) {
#pragma unroll 8
    for (int p = quarter; p < a.chunks; p += 4)
      top = max(top, a.part[static_cast<int64_t>(p) * a.cols + c0 + c]);
  }
  tops[quarter][c] = top;
  uint32_t bits[4][8] = {};
  if constexpr (SR) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      random8(a.base_index + static_cast<uint64_t>(r0 + rg * 4 + i) * static_cast<uint64_t>(a.cols) +
                  static_cast<uint64_t>(col), a.seed, a.step, bits[i]);
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    GroupScale g;
    const float s = group_scale(max(max(tops[0][c], tops[1][c]), max(tops[2][c], tops[3][c])), g);
    scales[c] = g;
    if (blockIdx.y == 0 && c0 + c < a.cols) a.scale[c0 + c] = s;
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const GroupScale g = scales[cg * 8 + e];
    int32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = quantize<SR>(x[i][e], g, bits[i][e]);
    tile[(cg * 8 + e) * kWords + rg] = pack4(q);
  }
  __syncthreads();
  for (int t = threadIdx.x; t < 64 * 8; t += 256) {
    const int cc = t / 8, part = t % 8;
    const int64_t r = r0 + part * 16;
    if (c0 + cc < a.cols && r < a.rows) {
      const uint32_t* w = tile + cc * kWords + part * 4;
      *reinterpret_cast<asr::u32x4*>(a.q + (c0 + cc) * a.ldq + r) = asr::u32x4{w[0], w[1], w[2], w[3]};
    }
  }
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
  uint32_t vec16;  // runs of 8 outputs start on 16-byte addresses
  uint32_t pos4;   // runs of 4 outputs start on stream positions divisible by 4
};

template <int ROUND>
__device__ __forceinline__ uint32_t round_one(float x, uint32_t r16) {
  return ROUND == ASR_ROUND_SR ? asr::round_sr(__float_as_uint(x), r16)
                               : asr::round_rn(__float_as_uint(x));
}

using Big = asr_mfma::Tile<256, 256, 128, 64, 2>;
using Small = asr_mfma::Tile<128, 128, 64, 64, 2>;
using Small8 = asr_mfma::Tile<128, 128, 64, 32, 3>;
using Tiny = asr_mfma::Tile<64, 64, 32, 32, 4>;

// REST: K is not a multiple of 16 (a variant of its own: its byte loads cost
// the largest tile registers that it has not got).
template <typename T, int ROUND, bool REST>
__global__ __launch_bounds__(T::kThreads, T::kMinWaves) void gemm_i8(GemmArgs args) {
  using E = asr_mfma::ElemI8;
  __shared__ __align__(1024) unsigned char smem[T::kLoopLds];
  uint32_t tm, tn;
  asr_mfma::grouped_tile(asr_mfma::xcd_order(blockIdx.x, args.tiles_m * args.tiles_n),
                         args.tiles_m, args.tiles_n, tm, tn);
  const int64_t m0 = static_cast<int64_t>(tm) * T::BM, n0 = static_cast<int64_t>(tn) * T::BN;
  E::acc acc[T::kFragM][T::kFragN] = {};
  asr_mfma::Operands op;
  op.a = reinterpret_cast<const char*>(args.a + m0 * args.lda);
  op.b = reinterpret_cast<const char*>(args.b + n0 * args.ldb);
  op.ld_a = static_cast<uint32_t>(args.lda);
  op.ld_b = static_cast<uint32_t>(args.ldb);
  op.last_a = args.m - 1 - static_cast<int32_t>(m0);
  op.last_b = args.n - 1 - static_cast<int32_t>(n0);
  op.kbytes = args.k & ~15;
  asr_mfma::mfma_loop<T, E>(op, smem, acc);

  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t wm = wave / T::kWavesN, wn = wave % T::kWavesN;
  const uint32_t row = lane & 31u, half = lane >> 5;

  // The last K % 16 codes of every row, byte by byte (what lies behind a
  // row's end is not read); lanes of the upper half hold zeros.
  if constexpr (REST) {
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

  // Each lane scales and rounds its own runs of 4 columns (one Philox call a
  // run, as the keying lays them out); v_permlane32_swap then pairs lanes l
  // and l + 32 into runs of 8 for one 16-byte store. Both lanes of a pair
  // take that store only when all 16 columns of the pair lie in the row.
  static_for<T::kFragN>([&](auto jc) {
    constexpr int j = decltype(jc)::value;
    const int64_t nj = n0 + wn * T::WN + j * 32;
    float sb[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sb[q][e] = args.sb[min(nj + 8 * q + 4 * half + e, static_cast<int64_t>(args.n - 1))];
    static_for<T::kFragM>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      const int64_t m = m0 + wm * T::WM + i * 32 + row;
      const float sa = args.sa[min(m, static_cast<int64_t>(args.m - 1))];
      static_for<2>([&](auto pc) {
        constexpr int p = decltype(pc)::value;
        uint32_t w[2][2];
        float xs[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t n = nj + 16 * p + 8 * h + 4 * half;
          uint32_t r16[4] = {};
          if constexpr (ROUND == ASR_ROUND_SR)
            asr_mfma::random4(args.base_index + static_cast<uint64_t>(m) * static_cast<uint64_t>(args.n) +
                                  static_cast<uint64_t>(n),
                              args.pos4 != 0, args.seed, args.step, r16);
          uint32_t u[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            xs[h][e] = (static_cast<float>(acc[i][j][8 * p + 4 * h + e]) * sa) * sb[2 * p + h][e];
            u[e] = round_one<ROUND>(xs[h][e], r16[e]);
          }
          w[h][0] = u[0] | (u[1] << 16);
          w[h][1] = u[2] | (u[3] << 16);
        }
        const auto s0 = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
        const auto s1 = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
        const int64_t n16 = nj + 16 * p;
        if (m < args.m) {
          if (args.vec16 && n16 + 16 <= args.n) {
            *reinterpret_cast<asr::u32x4*>(args.c + m * args.ldc + n16 + 8 * half) =
                asr::u32x4{s0[0], s1[0], s0[1], s1[1]};
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int64_t n = n16 + 8 * h + 4 * half;
              uint16_t* d = args.c + m * args.ldc + n;
              if (args.vec4 && n + 4 <= args.n) {
                *reinterpret_cast<asr::u32x2*>(d) = asr::u32x2{w[h][0], w[h][1]};
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (n + e < args.n) d[e] = static_cast<uint16_t>(w[h][e / 2] >> (16 * (e % 2)));
              }
            }
          }
          if (args.c32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int64_t n = n16 + 8 * h + 4 * half;
              float* d = args.c32 + m * args.ldc + n;
              if (args.vec4 && n + 4 <= args.n) {
                *reinterpret_cast<asr::f32x4*>(d) = asr::f32x4{xs[h][0], xs[h][1], xs[h][2], xs[h][3]};
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (n + e < args.n) d[e] = xs[h][e];
              }
            }
          }
        }
      });
    });
  });
}

// A few rows of A (decoding): bound by reading B once. A workgroup takes 16
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
  auto step = [&](int32_t k) {
    i32x4 b[2], a[MB][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      b[h] = *reinterpret_cast<const i32x4*>(pb + k + k_lane + 16 * h);
#pragma unroll
      for (int i = 0; i < MB; ++i) a[i][h] = *reinterpret_cast<const i32x4*>(pa[i] + k + k_lane + 16 * h);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MB; ++i)
        acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[h], a[i][h], acc[i], 0, 0, 0);
  };
  int32_t u = static_cast<int32_t>(wave);
#pragma unroll 4
  for (; u < whole; u += kWaves) step(u * 128);
  if (args.k % 128 != 0 && u == whole) {
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
    asr_mfma::random4(args.base_index + static_cast<uint64_t>(m) * static_cast<uint64_t>(args.n) +
                          static_cast<uint64_t>(n), args.pos4 != 0, args.seed, args.step, r16);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float sb = args.sb[min(n + e, static_cast<int64_t>(args.n - 1))];
    x[e] = (static_cast<float>(t[e]) * sa) * sb;
    h[e] = round_one<ROUND>(x[e], r16[e]);
  }
  const int64_t at = m * args.ldc + n;
  const int count = static_cast<int>(min(int64_t{4}, args.n - n));
  if (args.vec4 && count == 4) {
    asr::store_vec_bf16<false, 4>(args.c + at, h);
    if (args.c32) asr::store_vec<false, 4>(args.c32 + at, x);
  } else {
    asr::store_range_bf16<4>(args.c, at, 0, count, h);
    if (args.c32) asr::store_range<4>(args.c32, at, 0, count, x);
  }
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

// Rows a workgroup of column_maxima takes (a multiple of 64): enough chunks for
// about 1024 workgroups, no more than 64 of them.
int64_t chunk_rows(int64_t rows, int64_t cols) {
  const int64_t strips = (cols + 127) / 128;
  const int64_t chunks = std::clamp<int64_t>(1024 / strips, 1, 64);
  return ((rows + chunks - 1) / chunks + 63) / 64 * 64;
}

template <typename F>
hipError_t launch(F* f, dim3 grid, int threads, void* args, hipStream_t s) {
  void* argv[] = {args};
  return hipLaunchKernel(reinterpret_cast<const void*>(f), grid, dim3(threads), argv, 0, s);
}

template <typename S, bool SR>
hipError_t launch_quantize(asr_i8::QuantArgs& a, bool transpose, hipStream_t s) {
  using namespace asr_i8;
  if (!transpose) {
    // 64 lanes hold a row of up to 2048 elements in registers
    if (a.cols <= 2048)
      return launch(&quantize_rows<S, SR, 64>, dim3(static_cast<uint32_t>((a.rows + 3) / 4)), 256, &a, s);
    return launch(&quantize_rows<S, SR, 256>, dim3(static_cast<uint32_t>(a.rows)), 256, &a, s);
  }
  const hipError_t e =
      launch(&column_maxima<S>, dim3(static_cast<uint32_t>((a.cols + 127) / 128),
                                     static_cast<uint32_t>(a.chunks)), 256, &a, s);
  if (e != hipSuccess) return e;
  return launch(&quantize_columns<S, SR>, dim3(static_cast<uint32_t>((a.cols + 63) / 64),
                                               static_cast<uint32_t>((a.rows + 127) / 128)),
                256, &a, s);
}

template <typename T>
hipError_t launch_gemm(asr_i8::GemmArgs args, int32_t rounding, hipStream_t s) {
  using namespace asr_i8;
  args.tiles_m = static_cast<uint32_t>((args.m + T::BM - 1) / T::BM);
  args.tiles_n = static_cast<uint32_t>((args.n + T::BN - 1) / T::BN);
  const dim3 grid(args.tiles_m * args.tiles_n);
  const bool rest = args.k % 16 != 0;
  if (rounding == ASR_ROUND_SR)
    return rest ? launch(&gemm_i8<T, ASR_ROUND_SR, true>, grid, T::kThreads, &args, s)
               : launch(&gemm_i8<T, ASR_ROUND_SR, false>, grid, T::kThreads, &args, s);
  return rest ? launch(&gemm_i8<T, ASR_ROUND_RN, true>, grid, T::kThreads, &args, s)
             : launch(&gemm_i8<T, ASR_ROUND_RN, false>, grid, T::kThreads, &args, s);
}

template <int MB>
hipError_t launch_few(asr_i8::GemmArgs args, int32_t rounding, hipStream_t s) {
  using namespace asr_i8;
  const dim3 grid(static_cast<uint32_t>((args.n + 15) / 16));
  return rounding == ASR_ROUND_SR ? launch(&gemm_i8_few<MB, ASR_ROUND_SR>, grid, 512, &args, s)
                                  : launch(&gemm_i8_few<MB, ASR_ROUND_RN>, grid, 512, &args, s);
}

}  // namespace

extern "C" {

size_t asr_quantize_i8_workspace_bytes(int64_t rows, int64_t cols, int32_t transpose) {
  if (!transpose || rows <= 0 || cols <= 0 || rows >= kMaxDim || cols >= kMaxDim) return 0;
  const int64_t chunk = chunk_rows(rows, cols), chunks = (rows + chunk - 1) / chunk;
  return static_cast<size_t>((chunks * cols * 4 + 255) / 256 * 256);
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
  if (ldq < (length + 15) / 16 * 16 || ldq % 16 != 0)
    return fail(ASR_EINVAL, "quantize_i8: ldq must be a multiple of 16 and hold a group's codes "
                            "up to a multiple of 16");
  const int64_t size = dtype == ASR_F32 ? 4 : 2;
  if (!aligned_to(x, size) || !aligned_to(scale, 4) || !aligned_to(q, 16))
    return fail(ASR_EALIGN, "quantize_i8: x and scale aligned to their elements, q to 16 bytes");
  if (length > 0 && static_cast<uint64_t>(rows) * static_cast<uint64_t>(cols) - 1 > ~base_index)
    return fail(ASR_EINVAL, "quantize_i8: base_index + rows*cols exceeds 2**64");
  if (transpose && (rows + 127) / 128 > 65535)
    return fail(ASR_EINVAL, "quantize_i8: at most 128 * 65535 rows in the transposed form");
  if (transpose && length > 0) {
    if (!workspace || !aligned_to(workspace, 16) ||
        workspace_bytes < asr_quantize_i8_workspace_bytes(rows, cols, transpose))
      return fail(ASR_EWORKSPACE, "quantize_i8: workspace NULL, too small or not 16-byte aligned");
  }
  asr_i8::QuantArgs a{};
  a.x = x;
  a.q = q;
  a.scale = scale;
  a.part = static_cast<uint32_t*>(workspace);
  a.ldx = ldx;
  a.rows = rows;
  a.cols = cols;
  a.ldq = ldq;
  a.base_index = base_index;
  a.seed = seed;
  a.step = step;
  a.vec = aligned_to(x, 16) && (rows == 1 || ldx * size % 16 == 0);
  a.chunk = static_cast<int32_t>(length > 0 ? chunk_rows(rows > 0 ? rows : 1, cols) : 1);
  a.chunks = static_cast<int32_t>((rows + a.chunk - 1) / a.chunk);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool sr = rounding == ASR_ROUND_SR;
  // (a group without elements still gets its scale, 0)
  if (transpose && length == 0) {
    a.chunks = 0;
    const dim3 grid(static_cast<uint32_t>((cols + 63) / 64), 1);
    const hipError_t e = launch(&asr_i8::quantize_columns<uint16_t, false>, grid, 256, &a, s);
    return e == hipSuccess ? ok() : hip_fail(e, "quantize_i8 launch");
  }
  hipError_t e;
  if (dtype == ASR_F32)
    e = sr ? launch_quantize<float, true>(a, transpose, s) : launch_quantize<float, false>(a, transpose, s);
  else
    e = sr ? launch_quantize<uint16_t, true>(a, transpose, s)
           : launch_quantize<uint16_t, false>(a, transpose, s);
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
  asr_i8::GemmArgs g{};
  g.a = a;
  g.b = b;
  g.sa = scale_a;
  g.sb = scale_b;
  g.c = c;
  g.c32 = c_f32;
  g.lda = lda;
  g.ldb = ldb;
  g.ldc = ldc;
  g.base_index = base_index;
  g.m = static_cast<int32_t>(m);
  g.n = static_cast<int32_t>(n);
  g.k = static_cast<int32_t>(k);
  g.seed = seed;
  g.step = step;
  g.vec4 = ldc % 4 == 0 && aligned_to(c, 8) && (!c_f32 || aligned_to(c_f32, 16));
  g.vec16 = ldc % 8 == 0 && aligned_to(c, 16);
  g.pos4 = base_index % 4 == 0 && n % 4 == 0;
  auto tiles = [&](int64_t t) { return static_cast<uint64_t>((m + t - 1) / t) * ((n + t - 1) / t); };
  if (tiles(64) > 0x7FFFFFFFull) return fail(ASR_EINVAL, "gemm_i8: too many tiles");
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
#ifndef ASR_I8_FEW
#define ASR_I8_FEW 64
#endif
  if (m <= std::min(ASR_I8_FEW, 16)) e = launch_few<1>(g, rounding, s);
  else if (m <= std::min(ASR_I8_FEW, 32)) e = launch_few<2>(g, rounding, s);
  else if (m <= std::min(ASR_I8_FEW, 64)) e = launch_few<4>(g, rounding, s);
  else if (tiles(256) >= 256) e = launch_gemm<asr_i8::Big>(g, rounding, s);
  else if (tiles(128) > 256) e = launch_gemm<asr_i8::Small>(g, rounding, s);
  else if (tiles(128) > 128) e = launch_gemm<asr_i8::Small8>(g, rounding, s);
  else e = launch_gemm<asr_i8::Tiny>(g, rounding, s);
  return e == hipSuccess ? ok() : hip_fail(e, "gemm_i8 launch");
}

}  // extern "C"
