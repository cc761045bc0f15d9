// Orthogonalisation of a matrix by Newton-Schulz products, and the Muon step
// around it: momentum, orthogonalisation, decoupled weight decay and the
// (stochastically rounded) write-back of the weights.
//
//   X0 = U / (|U|_F + eps),  S <= T its sides, X taken with S rows
//   A = X X^T,  B = b A + c A A,  X <- a X + B X       (a number of times)
//
// Every product is C = P * Q^T with K contiguous in both operands: A = X X^T
// and A A = A A^T (A is symmetric) as they stand, and B X as B * Y^T with Y =
// X^T kept beside X. The last product's epilogue writes its result both ways,
// the turned copy through the LDS the K loop has left; A and B need one half
// of their tiles, mirrored by the same means.
//
// Precision: the matrix instructions take 16-bit operands. In bf16 the
// result is 1e-2 (Gaussian) to 2e-1 (low rank) from the 64-bit one. Here the
// operands are f16, held in powers of two that keep them near 1 (|X| <= 1, so
// |X| * 2**14 fits), and X is kept as hi + lo, two f16 numbers: the products
// use hi, the term a X uses both. What rounding hi costs then only enters
// through B X, so directions with small singular values, which a
// multiplies by hundreds over the steps, are not drowned in the rounding of the large
// ones: 3e-4 to 2e-3 on the same matrices, about a bf16 rounding.
#include "mfma_loop.hpp"
#include "status.hpp"

#include <adamw_sr.h>

#include <algorithm>
#include <cmath>
#include <string>

#pragma clang fp contract(off)

namespace asr_muon {

using asr_mfma::static_for;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxBatch = 16;   // matrices of one launch
constexpr int kMaxParts = 1024; // partial sums of one matrix's squared norm

struct Matrices {
  const void* g[kMaxBatch];
  float* m[kMaxBatch];      // momentum (NULL without)
  void* p[kMaxBatch];       // weights, or the result
  uint64_t base[kMaxBatch];
};

struct PrepareArgs {
  Matrices mat;
  int64_t rows, cols, numel, chunk;
  char* ws;
  int64_t stride;                  // workspace bytes a matrix
  int64_t parts, direct, turned, lo;  // offsets in it
  int64_t ld_direct, ld_turned;    // elements
  double eps, scale;
  float momentum;
  int32_t nesterov, parts_n;
  uint32_t vec;
};

// U of 8 consecutive elements: the gradient, or the momentum step's update.
template <typename G, bool MUON>
__device__ __forceinline__ void momentum_update(const float (&g)[8], float (&m)[8], float mu,
                                                bool nesterov, bool fresh, float (&u)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (MUON) {
      if (fresh) m[e] = mu * m[e] + g[e];
      u[e] = nesterov ? g[e] + mu * m[e] : m[e];
    } else {
      u[e] = g[e];
    }
  }
}

// Sum of squares of one chunk of U, in 64 bits; the momentum is updated on
// the way. Memory bound: 2 (bf16 gradient) + 8 bytes an element.
template <typename G, bool MUON>
__global__ __launch_bounds__(256) void sum_squares(PrepareArgs a) {
  const int k = blockIdx.y;
  const G* g = static_cast<const G*>(a.mat.g[k]);
  float* m = a.mat.m[k];
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
  const int64_t i1 = min(a.numel, i0 + a.chunk);
  double sum = 0.0;
  for (int64_t i = i0 + threadIdx.x * 8; i < i1; i += 256 * 8) {
    const int n = static_cast<int>(min(int64_t{8}, i1 - i));
    const bool whole = a.vec && n == 8;
    float gx[8], mx[8], u[8];
    if (whole) {
      asr::load_vec<false, 8>(g + i, gx);
      if constexpr (MUON) asr::load_vec<false, 8>(m + i, mx);
    } else {
      asr::load_range<8>(g, i, 0, n, gx);
      if constexpr (MUON) asr::load_range<8>(m, i, 0, n, mx);
    }
    momentum_update<G, MUON>(gx, mx, a.momentum, a.nesterov, true, u);
    if constexpr (MUON) {
      if (whole) asr::store_vec<false, 8>(m + i, mx);
      else asr::store_range<8>(m, i, 0, n, mx);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) sum += static_cast<double>(u[e]) * static_cast<double>(u[e]);
  }
  __shared__ double sums[4];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = sum;
  __syncthreads();
  if (threadIdx.x == 0)
    reinterpret_cast<double*>(a.ws + k * a.stride + a.parts)[blockIdx.x] =
        (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// X0 as hi + lo, and hi turned, for one 64 x 64 tile, with zeros up to the
// leading dimensions (the K loops read whole 128-byte lines).
template <typename G, bool MUON>
__global__ __launch_bounds__(256) void scale_matrix(PrepareArgs a) {
  constexpr int kLd = 72;  // f16 a row of the turned tile
  __shared__ __align__(16) _Float16 tile[64 * kLd];
  __shared__ double sums[4];
  const int k = blockIdx.z;
  char* ws = a.ws + k * a.stride;
  const double* parts = reinterpret_cast<const double*>(ws + a.parts);
  double sum = 0.0;
  for (int i = threadIdx.x; i < a.parts_n; i += 256) sum += parts[i];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = sum;
  __syncthreads();
  const double norm = __builtin_sqrt((sums[0] + sums[1]) + (sums[2] + sums[3]));
  const double factor = a.scale / (norm + a.eps);

  const G* g = static_cast<const G*>(a.mat.g[k]);
  const float* m = a.mat.m[k];
  _Float16* hi_out = reinterpret_cast<_Float16*>(ws + a.direct);
  _Float16* lo_out = reinterpret_cast<_Float16*>(ws + a.lo);
  _Float16* turned = reinterpret_cast<_Float16*>(ws + a.turned);
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 64, c0 = static_cast<int64_t>(blockIdx.x) * 64;
  const int cg = threadIdx.x & 7;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int rr = (threadIdx.x >> 3) + 32 * pass;
    const int64_t r = r0 + rr, c = c0 + cg * 8;
    float gx[8] = {}, mx[8] = {}, u[8];
    if (r < a.rows) {
      const int n = static_cast<int>(max(int64_t{0}, min(int64_t{8}, a.cols - c)));
      const int64_t i = r * a.cols + c;
      if (a.vec && n == 8 && a.cols % 8 == 0) {
        asr::load_vec<false, 8>(g + i, gx);
        if constexpr (MUON) asr::load_vec<false, 8>(m + i, mx);
      } else {
        asr::load_range<8>(g, i, 0, n, gx);
        if constexpr (MUON) asr::load_range<8>(m, i, 0, n, mx);
      }
    }
    momentum_update<G, MUON>(gx, mx, a.momentum, a.nesterov, false, u);
    asr_mfma::f16x8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = static_cast<float>(static_cast<double>(u[e]) * factor);
      // (elements past the matrix stay zero whatever the factor is)
      const float y = r < a.rows && c + e < a.cols ? x : 0.0f;
      hi[e] = static_cast<_Float16>(y);
      lo[e] = static_cast<_Float16>(y - static_cast<float>(hi[e]));
      tile[(cg * 8 + e) * kLd + rr] = hi[e];
    }
    if (r < a.rows) {
      *reinterpret_cast<asr_mfma::f16x8*>(hi_out + r * a.ld_direct + c) = hi;
      *reinterpret_cast<asr_mfma::f16x8*>(lo_out + r * a.ld_direct + c) = lo;
    }
  }
  __syncthreads();
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int cc = (threadIdx.x >> 3) + 32 * pass;
    const int64_t c = c0 + cc, r = r0 + cg * 8;
    if (c < a.cols)
      *reinterpret_cast<asr_mfma::f16x8*>(turned + c * a.ld_turned + r) =
          *reinterpret_cast<const asr_mfma::f16x8*>(tile + cc * kLd + cg * 8);
  }
}

// ---------------------------------------------------------------- products
enum Mode {
  kGram,    // D = alpha * acc, symmetric
  kSquare,  // D = beta * C + alpha * acc, symmetric
  kUpdate,  // v = beta * (C + lo) + alpha * acc; D, lo = v in two parts; D turned
  kFinal    // o = (beta * (C + lo) + alpha * acc) * out_scale: the result, or the weights' step
};

struct ProductArgs {
  Matrices mat;            // kFinal
  char* ws;
  int64_t stride;
  int64_t a, b, c, lo, d, turned;  // offsets of a matrix's buffers
  uint32_t ld_a, ld_b;             // bytes
  int64_t ld_d, ld_turned;         // elements (C and lo have D's)
  int32_t m, n, kbytes;
  uint32_t tiles_m, tiles_n, tiles, batch;
  float alpha, beta;
  // kFinal
  float out_scale, decay, eta;
  int64_t ld_out;
  uint32_t seed, step, vec4, pos4;
};

// What kFinal does with o: the result in bf16, or p <- round(p * decay - eta * o).
enum Out { kOutBf16, kOutWeightBf16Sr, kOutWeightBf16Rn, kOutWeightF32 };

// Tile t of the lower triangle, rows in order.
__device__ __forceinline__ void triangle_tile(uint32_t t, uint32_t& tm, uint32_t& tn) {
  uint32_t r = static_cast<uint32_t>((__builtin_sqrtf(8.0f * static_cast<float>(t) + 1.0f) - 1.0f) * 0.5f);
  while ((r + 1) * (r + 2) / 2 <= t) ++r;
  while (r * (r + 1) / 2 > t) --r;
  tm = r;
  tn = t - r * (r + 1) / 2;
}

template <typename T>
constexpr int lds_bytes() {
  const int turned = T::BN * (T::BM + 8) * 2;
  return turned > T::kLoopLds ? turned : T::kLoopLds;
}

template <int OUT>
__device__ __forceinline__ void store_out(const ProductArgs& args, int k, int64_t m, int64_t n,
                                          const float (&v)[4]) {
  // runs of 4 that are whole and aligned move as vectors
  const bool full = args.vec4 && n + 4 <= args.n;
  const int count = static_cast<int>(min(int64_t{4}, static_cast<int64_t>(args.n) - n));
  const int64_t at = m * args.ld_out + n;
  if constexpr (OUT == kOutBf16) {
    uint16_t* d = static_cast<uint16_t*>(args.mat.p[k]);
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = asr::round_rn(__float_as_uint(v[e] * args.out_scale));
    if (full) asr::store_vec_bf16<false, 4>(d + at, h);
    else asr::store_range_bf16<4>(d, at, 0, count, h);
  } else if constexpr (OUT == kOutWeightF32) {
    float* p = static_cast<float*>(args.mat.p[k]);
    float x[4];
    if (full) asr::load_vec<false, 4>(p + at, x);
    else asr::load_range<4>(p, at, 0, count, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = x[e] * args.decay - args.eta * (v[e] * args.out_scale);
    if (full) asr::store_vec<false, 4>(p + at, x);
    else asr::store_range<4>(p, at, 0, count, x);
  } else {
    uint16_t* p = static_cast<uint16_t*>(args.mat.p[k]);
    float x[4];
    if (full) asr::load_vec<false, 4>(p + at, x);
    else asr::load_range<4>(p, at, 0, count, x);
    uint32_t r16[4] = {}, h[4];
    if constexpr (OUT == kOutWeightBf16Sr)
      asr_mfma::random4(args.mat.base[k] + static_cast<uint64_t>(at),
                        args.pos4 && (args.mat.base[k] & 3u) == 0, args.seed, args.step, r16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float y = x[e] * args.decay - args.eta * (v[e] * args.out_scale);
      h[e] = OUT == kOutWeightBf16Sr ? asr::round_sr(__float_as_uint(y), r16[e])
                                     : asr::round_rn(__float_as_uint(y));
    }
    if (full) asr::store_vec_bf16<false, 4>(p + at, h);
    else asr::store_range_bf16<4>(p, at, 0, count, h);
  }
}

template <typename T, int MODE, int OUT>
__global__ __launch_bounds__(T::kThreads) void product(ProductArgs args) {
  using E = asr_mfma::ElemF16;
  constexpr bool kSymmetric = MODE == kGram || MODE == kSquare;
  __shared__ __align__(1024) unsigned char smem[lds_bytes<T>()];
  const uint32_t t = asr_mfma::xcd_order(blockIdx.x, args.tiles * args.batch);
  const uint32_t k = t / args.tiles;
  uint32_t tm, tn;
  if constexpr (kSymmetric) triangle_tile(t % args.tiles, tm, tn);
  else asr_mfma::grouped_tile(t % args.tiles, args.tiles_m, args.tiles_n, tm, tn);
  const int64_t m0 = static_cast<int64_t>(tm) * T::BM, n0 = static_cast<int64_t>(tn) * T::BN;
  char* ws = args.ws + static_cast<int64_t>(k) * args.stride;
  E::acc acc[T::kFragM][T::kFragN] = {};
  asr_mfma::Operands op;
  op.a = ws + args.a + m0 * args.ld_a;
  op.b = ws + args.b + n0 * args.ld_b;
  op.ld_a = args.ld_a;
  op.ld_b = args.ld_b;
  op.last_a = args.m - 1 - static_cast<int32_t>(m0);
  op.last_b = args.n - 1 - static_cast<int32_t>(n0);
  op.kbytes = args.kbytes;
  asr_mfma::mfma_loop<T, E>(op, smem, acc);

  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t wm = wave / T::kWavesN, wn = wave % T::kWavesN;
  const uint32_t row = lane & 31u, half = lane >> 5;
  const _Float16* c_in = reinterpret_cast<const _Float16*>(ws + args.c);
  _Float16* lo_io = reinterpret_cast<_Float16*>(ws + args.lo);
  _Float16* d_out = reinterpret_cast<_Float16*>(ws + args.d);

  if constexpr (MODE == kFinal) {
    static_for<T::kFragM>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      const int64_t m = m0 + wm * T::WM + i * 32 + row;
      if (m >= args.m) return;
      static_for<T::kFragN>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        static_for<4>([&](auto qc) {
          constexpr int q = decltype(qc)::value;
          const int64_t n = n0 + wn * T::WN + j * 32 + 8 * q + 4 * half;
          if (n >= args.n) return;
          const f16x4 hi = *reinterpret_cast<const f16x4*>(c_in + m * args.ld_d + n);
          const f16x4 lo = *reinterpret_cast<const f16x4*>(lo_io + m * args.ld_d + n);
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = args.beta * (static_cast<float>(hi[e]) + static_cast<float>(lo[e])) +
                   args.alpha * acc[i][j][4 * q + e];
          store_out<OUT>(args, k, m, n, v);
        });
      });
    });
    return;
  }

  // The turned copy goes through LDS: element (m, n) of the tile at n * kLd + m.
  constexpr int kLd = T::BM + 8;
  _Float16* tile = reinterpret_cast<_Float16*>(smem);
  const bool turn = !kSymmetric || tm != tn;
  __syncthreads();  // every wave has read the last K tile
  static_for<T::kFragM>([&](auto ic) {
    constexpr int i = decltype(ic)::value;
    const uint32_t mt = wm * T::WM + i * 32 + row;
    const int64_t m = m0 + mt;
    const bool live = m < args.m;
    static_for<T::kFragN>([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      static_for<2>([&](auto pc) {
        constexpr int p = decltype(pc)::value;
        uint32_t w[2][2], wl[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t nt = wn * T::WN + j * 32 + 16 * p + 8 * h + 4 * half;
          const int64_t n = n0 + nt;
          f16x4 hi = {}, lo = {};
          if constexpr (MODE != kGram) {
            if (live && n < args.ld_d) {
              hi = *reinterpret_cast<const f16x4*>(c_in + m * args.ld_d + n);
              if constexpr (MODE == kUpdate)
                lo = *reinterpret_cast<const f16x4*>(lo_io + m * args.ld_d + n);
            }
          }
          f16x4 vh, vl;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = args.alpha * acc[i][j][8 * p + 4 * h + e];
            if constexpr (MODE == kSquare) v = args.beta * static_cast<float>(hi[e]) + v;
            if constexpr (MODE == kUpdate)
              v = args.beta * (static_cast<float>(hi[e]) + static_cast<float>(lo[e])) + v;
            if (!live || n + e >= args.n) v = 0.0f;  // the padding reads as zeros
            vh[e] = static_cast<_Float16>(v);
            vl[e] = static_cast<_Float16>(v - static_cast<float>(vh[e]));
            if (turn) tile[(nt + e) * kLd + mt] = vh[e];
          }
          w[h][0] = __builtin_bit_cast(uint32_t, f16x2{vh[0], vh[1]});
          w[h][1] = __builtin_bit_cast(uint32_t, f16x2{vh[2], vh[3]});
          wl[h][0] = __builtin_bit_cast(uint32_t, f16x2{vl[0], vl[1]});
          wl[h][1] = __builtin_bit_cast(uint32_t, f16x2{vl[2], vl[3]});
        }
        // lanes l and l + 32 pair their runs of 4 into one 16-byte store each
        const int64_t n16 = n0 + wn * T::WN + j * 32 + 16 * p;
        auto put = [&](_Float16* d, const uint32_t (&x)[2][2]) {
          const auto s0 = __builtin_amdgcn_permlane32_swap(x[0][0], x[1][0], false, false);
          const auto s1 = __builtin_amdgcn_permlane32_swap(x[0][1], x[1][1], false, false);
          if (live && n16 < args.ld_d)
            *reinterpret_cast<asr::u32x4*>(d + m * args.ld_d + n16 + 8 * half) =
                asr::u32x4{s0[0], s1[0], s0[1], s1[1]};
        };
        put(d_out, w);
        if constexpr (MODE == kUpdate) put(lo_io, wl);
      });
    });
  });
  if (!turn) return;
  __syncthreads();
  _Float16* t_out = reinterpret_cast<_Float16*>(ws + args.turned);
  for (int q = threadIdx.x; q < T::BN * (T::BM / 8); q += T::kThreads) {
    const int nt = q / (T::BM / 8), c8 = q % (T::BM / 8) * 8;
    if (n0 + nt < args.n && m0 + c8 < args.ld_turned)
      *reinterpret_cast<asr_mfma::f16x8*>(t_out + (n0 + nt) * args.ld_turned + m0 + c8) =
          *reinterpret_cast<const asr_mfma::f16x8*>(tile + nt * kLd + c8);
  }
}

using Big = asr_mfma::Tile<256, 256, 128, 64, 2>;
using Small = asr_mfma::Tile<128, 128, 64, 64, 2>;
using Small8 = asr_mfma::Tile<128, 128, 64, 32, 3>;
using Tiny = asr_mfma::Tile<64, 64, 32, 32, 4>;

}  // namespace asr_muon

// =========================================================== host side
namespace {

using asr_host::fail;
using asr_host::hip_fail;
using asr_host::ok;
using namespace asr_muon;

bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

constexpr int64_t kMaxSide = int64_t{1} << 20;
constexpr int64_t kWorkspaceAim = int64_t{4} << 30;

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// A matrix's part of the workspace: X and Y = X^T (f16, rows padded to 128
// bytes; Y twice, since the product that makes the next X reads all of the
// last Y), the low parts, A, B and the norm's partial sums.
struct Layout {
  int64_t s, t, ld_s, ld_t;
  bool wide;  // the matrix itself has its short side first
  int64_t x, y[2], lo, a, b, parts, stride;
  Layout(int64_t rows, int64_t cols) {
    wide = rows <= cols;
    s = std::min(rows, cols);
    t = std::max(rows, cols);
    ld_s = up(s, 64);
    ld_t = up(t, 64);
    const int64_t across = s * ld_t * 2, down = t * ld_s * 2, square = s * ld_s * 2;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
      const int64_t here = at;
      at += up(bytes, 1024);
      return here;
    };
    x = take(across);
    y[0] = take(down);
    y[1] = take(down);
    lo = take(wide ? across : down);
    a = take(square);
    b = take(square);
    parts = take(kMaxParts * 8);
    stride = at;
  }
};

int32_t chunk_of(int32_t n, int64_t rows, int64_t cols) {
  const int64_t stride = Layout(rows, cols).stride;
  return static_cast<int32_t>(
      std::min<int64_t>({n, kMaxBatch, std::max<int64_t>(1, kWorkspaceAim / stride)}));
}

template <typename F>
hipError_t launch(F* f, dim3 grid, int threads, void* args, hipStream_t s) {
  void* argv[] = {args};
  return hipLaunchKernel(reinterpret_cast<const void*>(f), grid, dim3(threads), argv, 0, s);
}

template <typename T, int MODE, int OUT>
hipError_t launch_tile(ProductArgs& a, hipStream_t s) {
  a.tiles_m = static_cast<uint32_t>((a.m + T::BM - 1) / T::BM);
  a.tiles_n = static_cast<uint32_t>((a.n + T::BN - 1) / T::BN);
  a.tiles = MODE == kGram || MODE == kSquare ? a.tiles_m * (a.tiles_m + 1) / 2
                                             : a.tiles_m * a.tiles_n;
  return launch(&product<T, MODE, OUT>, dim3(a.tiles * a.batch), T::kThreads, &a, s);
}

// The tile by how many of them there are for the chip's 256 compute units.
template <int MODE, int OUT = kOutBf16>
hipError_t launch_product(ProductArgs& a, hipStream_t s) {
  auto tiles = [&](int64_t t) {
    const int64_t tm = (a.m + t - 1) / t, tn = (a.n + t - 1) / t;
    return (MODE == kGram || MODE == kSquare ? tm * (tm + 1) / 2 : tm * tn) * a.batch;
  };
  if (tiles(256) >= 256) return launch_tile<Big, MODE, OUT>(a, s);
  if (tiles(128) > 256) return launch_tile<Small, MODE, OUT>(a, s);
  if (tiles(128) > 128) return launch_tile<Small8, MODE, OUT>(a, s);
  return launch_tile<Tiny, MODE, OUT>(a, s);
}

struct Settings {
  int64_t rows, cols;
  int32_t g_dtype, steps;
  double a, b, c, eps;
  char* ws;
  hipStream_t stream;
};

// Largest singular value the polynomial lets any of [0, 1] reach in `steps`
// steps, and the largest |b l + c l^2| it meets: what the f16 operands' scales
// (2**14 at most) have to hold.
bool coefficients_ok(double a, double b, double c, int steps) {
  if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
  double top = 1.0;
  for (int k = 0; k < steps; ++k) {
    double next = 0.0;
    for (int i = 0; i <= 256; ++i) {
      const double x = top * i / 256, l = x * x;
      if (std::fabs(b * l + c * l * l) > 3.75) return false;
      next = std::max(next, std::fabs(x * (a + b * l + c * l * l)));
    }
    if (next > 1.4) return false;
    if (next <= top) return true;  // the later steps stay inside what was looked at
    top = next;
  }
  return true;
}

template <int OUT, bool MUON>
hipError_t run(const Settings& st, const Matrices& mat, int32_t batch, ProductArgs last,
               float momentum, bool nesterov) {
  const Layout l(st.rows, st.cols);
  auto power = [](double x) { return std::ldexp(1.0, std::min(14, static_cast<int>(std::lround(std::log2(x))))); };
  const double sx = power(std::sqrt(static_cast<double>(l.s) * static_cast<double>(l.t)));
  const double sa = power(static_cast<double>(l.s));

  PrepareArgs pa{};
  pa.mat = mat;
  pa.rows = st.rows;
  pa.cols = st.cols;
  pa.numel = st.rows * st.cols;
  const int64_t parts = std::clamp<int64_t>((pa.numel + 8191) / 8192, 1, kMaxParts);
  pa.chunk = up((pa.numel + parts - 1) / parts, 2048);
  pa.parts_n = static_cast<int32_t>((pa.numel + pa.chunk - 1) / pa.chunk);
  pa.ws = st.ws;
  pa.stride = l.stride;
  pa.parts = l.parts;
  pa.direct = l.wide ? l.x : l.y[0];
  pa.turned = l.wide ? l.y[0] : l.x;
  pa.lo = l.lo;
  pa.ld_direct = l.wide ? l.ld_t : l.ld_s;
  pa.ld_turned = l.wide ? l.ld_s : l.ld_t;
  pa.eps = st.eps;
  pa.scale = sx;
  pa.momentum = momentum;
  pa.nesterov = nesterov;
  pa.vec = 1;
  for (int32_t k = 0; k < batch; ++k)
    pa.vec = pa.vec && aligned_to(mat.g[k], 16) && (!MUON || aligned_to(mat.m[k], 16));
  const dim3 grid1(static_cast<uint32_t>(pa.parts_n), static_cast<uint32_t>(batch));
  const dim3 grid2(static_cast<uint32_t>((st.cols + 63) / 64), static_cast<uint32_t>((st.rows + 63) / 64),
                   static_cast<uint32_t>(batch));
  hipError_t e;
  if (st.g_dtype == ASR_F32) {
    e = launch(&sum_squares<float, MUON>, grid1, 256, &pa, st.stream);
    if (e == hipSuccess) e = launch(&scale_matrix<float, MUON>, grid2, 256, &pa, st.stream);
  } else {
    e = launch(&sum_squares<uint16_t, MUON>, grid1, 256, &pa, st.stream);
    if (e == hipSuccess) e = launch(&scale_matrix<uint16_t, MUON>, grid2, 256, &pa, st.stream);
  }

  ProductArgs gram{};
  gram.ws = st.ws;
  gram.stride = l.stride;
  gram.batch = static_cast<uint32_t>(batch);
  gram.a = gram.b = l.x;
  gram.ld_a = gram.ld_b = static_cast<uint32_t>(l.ld_t * 2);
  gram.kbytes = static_cast<int32_t>(l.ld_t * 2);
  gram.m = gram.n = static_cast<int32_t>(l.s);
  gram.d = gram.turned = l.a;
  gram.ld_d = gram.ld_turned = l.ld_s;
  gram.alpha = static_cast<float>(sa / (sx * sx));
  ProductArgs square = gram;
  square.a = square.b = square.c = l.a;
  square.ld_a = square.ld_b = static_cast<uint32_t>(l.ld_s * 2);
  square.kbytes = static_cast<int32_t>(l.ld_s * 2);
  square.d = square.turned = l.b;
  square.alpha = static_cast<float>(st.c / sa);
  square.beta = static_cast<float>(st.b);
  for (int32_t i = 0; i < st.steps && e == hipSuccess; ++i) {
    e = launch_product<kGram>(gram, st.stream);
    if (e == hipSuccess) e = launch_product<kSquare>(square, st.stream);
    if (e != hipSuccess) break;
    // B X in the matrix's own orientation: rows of B (or Y) by rows of Y (or B)
    const int64_t y = l.y[i & 1], y_next = l.y[(i & 1) ^ 1];
    ProductArgs u = i + 1 < st.steps ? square : last;
    u.ws = st.ws;
    u.stride = l.stride;
    u.batch = gram.batch;
    u.a = l.wide ? l.b : y;
    u.b = l.wide ? y : l.b;
    u.ld_a = u.ld_b = static_cast<uint32_t>(l.ld_s * 2);
    u.kbytes = static_cast<int32_t>(l.ld_s * 2);
    u.m = static_cast<int32_t>(st.rows);
    u.n = static_cast<int32_t>(st.cols);
    u.c = l.wide ? l.x : y;
    u.lo = l.lo;
    u.d = l.wide ? l.x : y_next;
    u.turned = l.wide ? y_next : l.x;
    u.ld_d = pa.ld_direct;
    u.ld_turned = pa.ld_turned;
    u.alpha = static_cast<float>(1.0 / sa);
    u.beta = static_cast<float>(st.a);
    u.out_scale = static_cast<float>(1.0 / sx);
    if (i + 1 < st.steps) {
      e = launch_product<kUpdate>(u, st.stream);
    } else {
      u.mat = mat;
      e = launch_product<kFinal, OUT>(u, st.stream);
    }
  }
  return e;
}

int check(const char* who, int32_t n, int64_t rows, int64_t cols, int32_t g_dtype, int32_t steps,
          double a, double b, double c, double eps) {
  const std::string w(who);
  if (n < 0) return fail(ASR_EINVAL, w + ": a negative number of matrices");
  if (rows < 0 || cols < 0 || rows > kMaxSide || cols > kMaxSide)
    return fail(ASR_EINVAL, w + ": rows and cols must be in [0, 2**20]");
  if (g_dtype != ASR_F32 && g_dtype != ASR_BF16) return fail(ASR_EDTYPE, w + ": unknown dtype");
  if (steps < 1 || steps > 64) return fail(ASR_EINVAL, w + ": steps must be in [1, 64]");
  if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(ASR_EINVAL, w + ": eps must be finite, >= 0");
  if (!coefficients_ok(a, b, c, steps))
    return fail(ASR_EINVAL, w + ": the coefficients let singular values in [0, 1] grow past 1.4 "
                                "(or |b x^2 + c x^4| past 3.75)");
  return ASR_OK;
}

int check_workspace(const char* who, void* ws, size_t bytes, size_t need) {
  if (!ws || !aligned_to(ws, 256) || bytes < need)
    return fail(ASR_EWORKSPACE, std::string(who) + ": workspace NULL, too small or not 256-byte aligned");
  return ASR_OK;
}

}  // namespace

extern "C" {

size_t asr_newton_schulz_workspace_bytes(int32_t n, int64_t rows, int64_t cols) {
  if (n <= 0 || rows <= 0 || cols <= 0 || rows > kMaxSide || cols > kMaxSide) return 0;
  return static_cast<size_t>(chunk_of(n, rows, cols) * Layout(rows, cols).stride);
}

int asr_newton_schulz(const void* const* g, uint16_t* const* out, int32_t n, int64_t rows,
                      int64_t cols, int32_t g_dtype, int32_t steps, double a, double b, double c,
                      double eps, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "newton_schulz";
  if (int rc = check(who, n, rows, cols, g_dtype, steps, a, b, c, eps)) return rc;
  if (n == 0 || rows == 0 || cols == 0) return ok();
  if (!g || !out) return fail(ASR_EINVAL, "newton_schulz: null array");
  for (int32_t k = 0; k < n; ++k) {
    if (!g[k] || !out[k]) return fail(ASR_EINVAL, "newton_schulz: null matrix");
    if (!aligned_to(g[k], g_dtype == ASR_F32 ? 4 : 2) || !aligned_to(out[k], 2))
      return fail(ASR_EALIGN, "newton_schulz: matrices must be aligned to their element size");
  }
  if (int rc = check_workspace(who, workspace, workspace_bytes,
                               asr_newton_schulz_workspace_bytes(n, rows, cols)))
    return rc;
  const Settings st{rows, cols, g_dtype, steps, a, b, c, eps, static_cast<char*>(workspace),
                    static_cast<hipStream_t>(stream)};
  const int32_t chunk = chunk_of(n, rows, cols);
  for (int32_t k0 = 0; k0 < n; k0 += chunk) {
    const int32_t batch = std::min(chunk, n - k0);
    Matrices mat{};
    ProductArgs last{};
    last.ld_out = cols;
    last.vec4 = cols % 4 == 0;
    for (int32_t k = 0; k < batch; ++k) {
      mat.g[k] = g[k0 + k];
      mat.p[k] = out[k0 + k];
      last.vec4 = last.vec4 && aligned_to(mat.p[k], 8);
    }
    const hipError_t e = run<kOutBf16, false>(st, mat, batch, last, 0.0f, false);
    if (e != hipSuccess) return hip_fail(e, "newton_schulz launch");
  }
  return ok();
}

int asr_muon_step(const asr_muon_tensor* tensors, int32_t n, int64_t rows, int64_t cols,
                  int32_t param_dtype, int32_t grad_dtype, double lr, double momentum,
                  int32_t nesterov, double weight_decay, double lr_factor, int32_t ns_steps,
                  double ns_a, double ns_b, double ns_c, double eps, int64_t step, uint32_t seed,
                  int32_t rounding, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "muon";
  if (int rc = check(who, n, rows, cols, grad_dtype, ns_steps, ns_a, ns_b, ns_c, eps)) return rc;
  if (param_dtype != ASR_F32 && param_dtype != ASR_BF16)
    return fail(ASR_EDTYPE, "muon: unknown param dtype");
  if (rounding != ASR_ROUND_SR && rounding != ASR_ROUND_RN)
    return fail(ASR_EINVAL, "muon: rounding must be ASR_ROUND_SR or ASR_ROUND_RN");
  if (!(lr >= 0.0) || !std::isfinite(lr) || !(weight_decay >= 0.0) || !std::isfinite(weight_decay) ||
      !(lr_factor >= 0.0) || !std::isfinite(lr_factor) || !(momentum >= 0.0 && momentum < 1.0))
    return fail(ASR_EINVAL, "muon: lr, weight_decay and lr_factor finite and >= 0, momentum in [0, 1)");
  if (step < 1 || step >= (int64_t{1} << 32))
    return fail(ASR_EINVAL, "muon: step must be in [1, 2**32 - 1]");
  if (n == 0 || rows == 0 || cols == 0) return ok();
  if (!tensors) return fail(ASR_EINVAL, "muon: null list");
  for (int32_t k = 0; k < n; ++k) {
    const asr_muon_tensor& t = tensors[k];
    if (!t.param || !t.grad || !t.momentum) return fail(ASR_EINVAL, "muon: null buffer");
    if (!aligned_to(t.param, param_dtype == ASR_F32 ? 4 : 2) ||
        !aligned_to(t.grad, grad_dtype == ASR_F32 ? 4 : 2) || !aligned_to(t.momentum, 4))
      return fail(ASR_EALIGN, "muon: buffers must be aligned to their element size");
  }
  if (int rc = check_workspace(who, workspace, workspace_bytes,
                               asr_newton_schulz_workspace_bytes(n, rows, cols)))
    return rc;
  const Settings st{rows, cols, grad_dtype, ns_steps, ns_a, ns_b, ns_c, eps,
                    static_cast<char*>(workspace), static_cast<hipStream_t>(stream)};
  const int32_t chunk = chunk_of(n, rows, cols);
  for (int32_t k0 = 0; k0 < n; k0 += chunk) {
    const int32_t batch = std::min(chunk, n - k0);
    Matrices mat{};
    ProductArgs last{};
    last.ld_out = cols;
    last.vec4 = cols % 4 == 0;
    last.pos4 = cols % 4 == 0;
    last.decay = static_cast<float>(1.0 - lr * weight_decay);
    last.eta = static_cast<float>(lr * lr_factor);
    last.seed = seed;
    last.step = static_cast<uint32_t>(step);
    for (int32_t k = 0; k < batch; ++k) {
      const asr_muon_tensor& t = tensors[k0 + k];
      mat.g[k] = t.grad;
      mat.m[k] = t.momentum;
      mat.p[k] = t.param;
      mat.base[k] = t.base_index;
      last.vec4 = last.vec4 && aligned_to(t.param, param_dtype == ASR_F32 ? 16 : 8);
    }
    const float mu = static_cast<float>(momentum);
    hipError_t e;
    if (param_dtype == ASR_F32)
      e = run<kOutWeightF32, true>(st, mat, batch, last, mu, nesterov != 0);
    else if (rounding == ASR_ROUND_SR)
      e = run<kOutWeightBf16Sr, true>(st, mat, batch, last, mu, nesterov != 0);
    else
      e = run<kOutWeightBf16Rn, true>(st, mat, batch, last, mu, nesterov != 0);
    if (e != hipSuccess) return hip_fail(e, "muon launch");
  }
  return ok();
}

}  // extern "C"
