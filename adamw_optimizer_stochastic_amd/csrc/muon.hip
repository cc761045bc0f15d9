// Orthogonalisation of a matrix by Newton-Schulz products, and the Muon step
// around it: momentum, orthogonalisation, decoupled weight decay and the
// (stochastically rounded) write-back of the weights.
//
//   X0 = U / (|U|_F + eps),  S <= T its sides, X taken with S rows
//   A = X X^T,  B = b A + c A A,  X <- a X + B X       (a number of times)
//
// Every product is C = P * Q^T with K contiguous in both operands: A = X X^T
// and A A = A A^T (A is symmetric) as they stand, and B X as B * Y^T with Y =
// X^T kept beside X. That product's epilogue writes its result both ways, the
// turned copy through the LDS the K loop has left; A and B need one half of
// their tiles, mirrored by the same means. One launch does one product for all
// matrices of a list, whatever their shapes: what is left over of the chip's
// last round of tiles is paid once a list, not once a matrix. A matrix
// small enough for one workgroup's LDS goes through all steps in one launch.
//
// Precision: the matrix instructions take 16-bit operands. In bf16 the
// result is 1e-2 (Gaussian) to 2e-1 (low rank) from the 64-bit one. Here the
// operands are f16, held in powers of two that keep them near 1 (|X| <= 1, so
// |X| * 2**14 fits), and X is kept as hi + lo, two f16 numbers: the products
// use hi, the term a X uses both. What rounding hi costs then only enters
// through B X, so directions with small singular values, which a
// multiplies by hundreds over the steps, are not drowned in the rounding of the large
// ones: 3e-4 to 2e-3 on the same matrices, about a bf16 rounding. That is an
// average of many roundings: short sides below 16, equal entries and orthogonal
// rows leave few or equal ones, up to 1.4e-2 on some 40,000 simulated matrices.
#include "mfma_loop.hpp"
#include "status.hpp"

#include <adamw_sr.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>
#include <string>
#include <utility>

#pragma clang fp contract(off)

namespace asr_muon {

using asr_mfma::f16x8;
using asr_mfma::static_for;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxBatch = 32;    // matrices of one launch
constexpr int kMaxParts = 1024;  // partial sums of one matrix's squared norm

// One matrix of a launch.
struct Desc {
  const void* g;
  float* m;        // momentum (NULL without)
  void* p;         // weights, or the result
  uint64_t base;   // stream position of the weights' element 0
  int64_t ws;      // its part of the workspace
  int32_t rows, cols;
  float eta;       // p <- p * decay - eta * O
  uint32_t first;  // its first workgroup in this launch
};

__host__ __device__ constexpr int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// A matrix's part of the workspace: X and Y = X^T (f16, rows padded to 128
// bytes; Y twice, since the product that makes the next X reads all of the
// last Y), the low parts, A, B and the norm's partial sums. X, A and B are
// held times sx and sa, powers of two that keep their entries near 1 and
// |X| <= 1.4, |A|, |B| <= 3.75 inside f16.
struct Layout {
  bool wide;  // the matrix itself has its short side first
  int32_t s, t, ld_s, ld_t;
  int64_t x, y, y_stride, lo, a, b, parts, bytes;
  float sx, sa;
  __host__ __device__ Layout(int32_t rows, int32_t cols) {
    wide = rows <= cols;
    s = wide ? rows : cols;
    t = wide ? cols : rows;
    ld_s = static_cast<int32_t>(up(s, 64));
    ld_t = static_cast<int32_t>(up(t, 64));
    const int64_t across = up(static_cast<int64_t>(s) * ld_t * 2, 1024);
    const int64_t down = up(static_cast<int64_t>(t) * ld_s * 2, 1024);
    const int64_t square = up(static_cast<int64_t>(s) * ld_s * 2, 1024);
    x = 0;
    y = across;
    y_stride = down;
    lo = y + 2 * down;
    a = lo + (wide ? across : down);
    b = a + square;
    parts = b + square;
    bytes = parts + kMaxParts * 8;
    // floor(log2(s t) / 2) and floor(log2 s)
    const int32_t half = (63 - __builtin_clzll(static_cast<uint64_t>(s) * static_cast<uint64_t>(t))) / 2;
    const int32_t whole = 31 - __builtin_clz(static_cast<uint32_t>(s));
    sx = static_cast<float>(1 << (half < 14 ? half : 14));
    sa = static_cast<float>(1 << (whole < 14 ? whole : 14));
  }
};

// Workgroups of sum_squares for a matrix, and the elements each takes.
__host__ __device__ inline int64_t part_size(int64_t numel) {
  int64_t parts = (numel + 8191) / 8192;
  if (parts > kMaxParts) parts = kMaxParts;
  return up((numel + parts - 1) / parts, 2048);
}

struct PrepareArgs {
  Desc d[kMaxBatch];
  char* ws;
  double eps;
  float momentum;
  int32_t nesterov, count;
  uint32_t vec;
};

// The matrix that workgroup b belongs to.
__device__ __forceinline__ int matrix_of(const Desc* d, int count, uint32_t b) {
  if (count == 1) return 0;
  const int lane = threadIdx.x & 63;
  const bool reached = lane < count && d[lane < count ? lane : 0].first <= b;
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(reached)) - 1);
}

// U of V consecutive elements: the gradient, or the momentum step's update;
// `fresh` does the momentum's own step, otherwise m has it already.
template <bool MUON, int V>
__device__ __forceinline__ void momentum_update(const float (&g)[V], float (&m)[V], float mu,
                                                bool nesterov, bool fresh, float (&u)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if constexpr (MUON) {
      if (fresh) m[e] = mu * m[e] + g[e];
      u[e] = nesterov ? g[e] + mu * m[e] : m[e];
    } else {
      u[e] = g[e];
    }
  }
}

// Sum of a workgroup's values in a fixed order; every thread gets it.
template <int THREADS>
__device__ __forceinline__ double group_sum(double x, double* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
  __syncthreads();
  double sum = 0.0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) sum += lds[w];
  return sum;
}

// Sum of squares of one chunk of U, in 64 bits; the momentum is updated on
// the way. Memory bound: 2 (bf16 gradient) + 8 bytes an element; 138e6 elements
// in 250 us, 5.5 TB/s.
template <typename G, bool MUON>
__global__ __launch_bounds__(256) void sum_squares(PrepareArgs a) {
  __shared__ double lds[4];
  const int k = matrix_of(a.d, a.count, blockIdx.x);
  const Desc& d = a.d[k];
  const G* g = static_cast<const G*>(d.g);
  float* m = d.m;
  const int64_t numel = static_cast<int64_t>(d.rows) * d.cols, chunk = part_size(numel);
  const uint32_t part = blockIdx.x - d.first;
  const int64_t i0 = part * chunk, i1 = min(numel, i0 + chunk);
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
    momentum_update<MUON>(gx, mx, a.momentum, a.nesterov, true, u);
    if constexpr (MUON) {
      if (whole) asr::store_vec<false, 8>(m + i, mx);
      else asr::store_range<8>(m, i, 0, n, mx);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) sum += static_cast<double>(u[e]) * static_cast<double>(u[e]);
  }
  sum = group_sum<256>(sum, lds);
  if (threadIdx.x == 0)
    reinterpret_cast<double*>(a.ws + d.ws + Layout(d.rows, d.cols).parts)[part] = sum;
}

// X0 as hi + lo, and hi turned, for one 64 x 64 tile, with zeros up to the
// leading dimensions (the K loops read whole 128-byte lines). Memory bound: 6
// bytes an element read (2 without momentum) and 6 written; 138e6 in 342 us,
// 4.8 TB/s.
template <typename G, bool MUON>
__global__ __launch_bounds__(256) void scale_matrix(PrepareArgs a) {
  constexpr int kLd = 72;  // f16 a row of the turned tile
  __shared__ __align__(16) _Float16 tile[64 * kLd];
  __shared__ double lds[4];
  const int k = matrix_of(a.d, a.count, blockIdx.x);
  const Desc& d = a.d[k];
  const int32_t rows = d.rows, cols = d.cols;
  const Layout l(rows, cols);
  char* ws = a.ws + d.ws;
  const int64_t numel = static_cast<int64_t>(rows) * cols, chunk = part_size(numel);
  const double* parts = reinterpret_cast<const double*>(ws + l.parts);
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i * chunk < numel; i += 256) sum += parts[i];
  const double norm = __builtin_sqrt(group_sum<256>(sum, lds));
  const double factor = static_cast<double>(l.sx) / (norm + a.eps);

  const G* g = static_cast<const G*>(d.g);
  const float* m = d.m;
  const int64_t ld_direct = l.wide ? l.ld_t : l.ld_s, ld_turned = l.wide ? l.ld_s : l.ld_t;
  _Float16* hi_out = reinterpret_cast<_Float16*>(ws + (l.wide ? l.x : l.y));
  _Float16* lo_out = reinterpret_cast<_Float16*>(ws + l.lo);
  _Float16* turned = reinterpret_cast<_Float16*>(ws + (l.wide ? l.y : l.x));
  const uint32_t t = blockIdx.x - d.first, across = static_cast<uint32_t>((cols + 63) / 64);
  const int64_t r0 = static_cast<int64_t>(t / across) * 64, c0 = static_cast<int64_t>(t % across) * 64;
  const int cg = threadIdx.x & 7;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int rr = (threadIdx.x >> 3) + 32 * pass;
    const int64_t r = r0 + rr, c = c0 + cg * 8;
    float gx[8] = {}, mx[8] = {}, u[8];
    if (r < rows) {
      const int n = static_cast<int>(max(int64_t{0}, min(int64_t{8}, cols - c)));
      const int64_t i = r * cols + c;
      if (a.vec && n == 8 && cols % 8 == 0) {
        asr::load_vec<false, 8>(g + i, gx);
        if constexpr (MUON) asr::load_vec<false, 8>(m + i, mx);
      } else {
        asr::load_range<8>(g, i, 0, n, gx);
        if constexpr (MUON) asr::load_range<8>(m, i, 0, n, mx);
      }
    }
    momentum_update<MUON>(gx, mx, a.momentum, a.nesterov, false, u);
    f16x8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = static_cast<float>(static_cast<double>(u[e]) * factor);
      // (elements past the matrix stay zero whatever the factor is)
      const float y = r < rows && c + e < cols ? x : 0.0f;
      hi[e] = static_cast<_Float16>(y);
      lo[e] = static_cast<_Float16>(y - static_cast<float>(hi[e]));
      tile[(cg * 8 + e) * kLd + rr] = hi[e];
    }
    if (r < rows) {
      *reinterpret_cast<f16x8*>(hi_out + r * ld_direct + c) = hi;
      *reinterpret_cast<f16x8*>(lo_out + r * ld_direct + c) = lo;
    }
  }
  __syncthreads();
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int cc = (threadIdx.x >> 3) + 32 * pass;
    const int64_t c = c0 + cc, r = r0 + cg * 8;
    if (c < cols)
      *reinterpret_cast<f16x8*>(turned + c * ld_turned + r) =
          *reinterpret_cast<const f16x8*>(tile + cc * kLd + cg * 8);
  }
}

// ---------------------------------------------------------------- products
enum Mode {
  kGram,    // A = X X^T
  kSquare,  // B = b A + c A A
  kUpdate,  // X <- a X + B X, in two parts, and the high one turned
  kFinal    // the same, into the result or the weights
};

// What becomes of O: the result in bf16, or p <- round(p * decay - eta * O).
enum Out { kOutBf16, kOutWeightBf16Sr, kOutWeightBf16Rn, kOutWeightF32 };

struct OutArgs {
  float decay;
  uint32_t seed, step;
  uint32_t vec8;  // runs of 8 of every matrix's rows start on 16-byte addresses
  uint32_t vec4;  // runs of 4 on 8-byte ones (f32: 16)
};

struct ProductArgs {
  Desc d[kMaxBatch];
  char* ws;
  float a, b, c;
  int32_t count, y;  // which Y holds the current X^T
  OutArgs out;
};

// Of a lane's two f16 values v0, v1 of one row m in neighbouring columns n, n +
// 1, and its neighbour lane's (row m ^ 1): an even lane gets column n of rows m,
// m + 1, an odd one column n + 1 of rows m - 1, m -- a whole LDS word of the
// turned tile instead of two halves.
__device__ __forceinline__ uint32_t turn_pair(float v0, float v1, uint32_t sel) {
  const uint32_t mine = __builtin_bit_cast(uint32_t, f16x2{static_cast<_Float16>(v0), static_cast<_Float16>(v1)});
  const uint32_t other = static_cast<uint32_t>(
      __builtin_amdgcn_mov_dpp(static_cast<int>(mine), 0xB1, 0xF, 0xF, true));  // quad_perm 1 0 3 2
  return __builtin_amdgcn_perm(other, mine, sel);
}
__device__ __forceinline__ uint32_t turn_selector(uint32_t lane) {
  return lane & 1u ? 0x03020706u : 0x05040100u;
}

// Tile t of the lower triangle, rows in order.
__device__ __forceinline__ void triangle_tile(uint32_t t, uint32_t& tm, uint32_t& tn) {
  uint32_t r = static_cast<uint32_t>((__builtin_sqrtf(8.0f * static_cast<float>(t) + 1.0f) - 1.0f) * 0.5f);
  while ((r + 1) * (r + 2) / 2 <= t) ++r;
  while (r * (r + 1) / 2 > t) --r;
  tm = r;
  tn = t - r * (r + 1) / 2;
}

__host__ __device__ inline int64_t tiles_of(int mode, int32_t rows, int32_t cols, int tile) {
  const int64_t tm = (rows + tile - 1) / tile, tn = (cols + tile - 1) / tile;
  if (mode != kGram && mode != kSquare) return tm * tn;
  const int64_t ts = tm < tn ? tm : tn;
  return ts * (ts + 1) / 2;
}

// The turned copy's stage in LDS, beside the waves' slices: element (m, n) of
// the tile at row n, rows taken a phase at a time (half of the 256 tile's, for
// room). Its 16-byte chunks are XOR-swizzled by n / 8, which is what differs
// between the lanes that write at once.
template <typename T>
struct Turn {
  static constexpr int kPhases = T::BM == 256 ? 2 : 1;
  static constexpr int kBlocks = T::kFragM / kPhases;      // blocks of 32 rows a wave, a phase
  static constexpr int kRows = T::BM / kPhases;
  static constexpr int kBytes = T::BN * kRows * 2;
  static constexpr int kLds = asr_mfma::Rows<T>::kBytes + kBytes;
  static_assert(kRows % 64 == 0, "whole groups of 8 chunks");
  static __device__ __forceinline__ uint32_t at(uint32_t n, uint32_t chunk) {
    return n * kRows + ((chunk ^ ((n >> 3) & 7u)) << 3);
  }
};

template <typename T>
constexpr int lds_bytes() {
  return Turn<T>::kLds > T::kLoopLds ? Turn<T>::kLds : T::kLoopLds;
}

// V consecutive elements (V = 4 or 8) of O from element `at` of a matrix, `n`
// of them inside it; vec: they are whole and aligned.
template <int OUT, int V>
__device__ __forceinline__ void store_out(const OutArgs& out, const Desc& d, int64_t at, int n,
                                          bool vec, const float (&o)[V]) {
  if constexpr (OUT == kOutWeightF32) {
    float* p = static_cast<float*>(d.p);
    float x[V];
    if (vec) asr::load_vec<false, V>(p + at, x);
    else asr::load_range<V>(p, at, 0, n, x);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = x[e] * out.decay - d.eta * o[e];
    if (vec) asr::store_vec<false, V>(p + at, x);
    else asr::store_range<V>(p, at, 0, n, x);
    return;
  }
  uint16_t* p = static_cast<uint16_t*>(d.p);
  uint32_t h[V];
  if constexpr (OUT == kOutBf16) {
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = asr::round_rn(__float_as_uint(o[e]));
  } else {
    float x[V];
    if (vec) asr::load_vec<false, V>(p + at, x);
    else asr::load_range<V>(p, at, 0, n, x);
    const uint64_t pos = d.base + static_cast<uint64_t>(at);
    uint32_t r16[V] = {};
    if constexpr (OUT == kOutWeightBf16Sr)
      asr_mfma::random_run<V>(pos, (pos & 3u) == 0, out.seed, out.step, r16);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float y = x[e] * out.decay - d.eta * o[e];
      h[e] = OUT == kOutWeightBf16Sr ? asr::round_sr(__float_as_uint(y), r16[e])
                                     : asr::round_rn(__float_as_uint(y));
    }
  }
  if (vec) asr::store_vec_bf16<false, V>(p + at, h);
  else asr::store_range_bf16<V>(p, at, 0, n, h);
}

// One product for all matrices of the launch. The K loop alone runs at 1288
// TFLOP/s on large matrices (f16 products of the library: 1481 for 8192^3);
// what it leaves is the epilogue, which nothing else covers: a tile that
// updates X reads 4 and writes 6 bytes an element, all tiles of a round at
// once. 4096 x 4096, 1024 x 4096, 14336 x 4096 and 4096 x 14336 together: A 620
// to 680 us, B 210-230, the new X 1040-1100, the weights 1085-1110 (in 256
// tiles, A in 192). 8 x 1024 x 4096: A 62-70, B 23-27, X 111-122, where the 52 us of K
// loops are less than the traffic. X and what the last product adds to
// are fetched a block ahead of their use (4096 x 14336: 4132 against 4168 us for all
// five steps).
template <typename T, int MODE, int OUT>
__global__ __launch_bounds__(T::kThreads, T::kMinWaves) void product(ProductArgs args) {
  using E = asr_mfma::ElemF16;
  constexpr bool kSymmetric = MODE == kGram || MODE == kSquare;
  __shared__ __align__(1024) unsigned char smem[lds_bytes<T>()];
  const int k = matrix_of(args.d, args.count, blockIdx.x);
  const Desc& d = args.d[k];
  const Layout l(d.rows, d.cols);
  char* ws = args.ws + d.ws;
  // operands, output size and strides of this product
  const int32_t m_all = kSymmetric ? l.s : d.rows, n_all = kSymmetric ? l.s : d.cols;
  const int64_t y_now = l.y + args.y * l.y_stride, y_next = l.y + (args.y ^ 1) * l.y_stride;
  const int64_t direct = l.wide ? l.x : y_now;
  const int64_t ld_d = kSymmetric ? l.ld_s : l.wide ? l.ld_t : l.ld_s;
  const int64_t ld_turned = kSymmetric ? l.ld_s : l.wide ? l.ld_s : l.ld_t;

  const uint32_t tiles = static_cast<uint32_t>(tiles_of(MODE, d.rows, d.cols, T::BM));
  const uint32_t t = asr_mfma::xcd_order(blockIdx.x - d.first, tiles);
  uint32_t tm, tn;
  if constexpr (kSymmetric)
    triangle_tile(t, tm, tn);
  else
    asr_mfma::grouped_tile(t, static_cast<uint32_t>((m_all + T::BM - 1) / T::BM),
                           static_cast<uint32_t>((n_all + T::BN - 1) / T::BN), tm, tn);
  const int64_t m0 = static_cast<int64_t>(tm) * T::BM, n0 = static_cast<int64_t>(tn) * T::BN;
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t wm = wave / T::kWavesN, wn = wave % T::kWavesN;
  const _Float16* c_in = reinterpret_cast<const _Float16*>(ws + (MODE == kSquare ? l.a : direct));
  _Float16* lo_io = reinterpret_cast<_Float16*>(ws + l.lo);

  // What C adds, for the 32 rows of block i: 16 bytes a lane and pass.
  using Rows = asr_mfma::Rows<T>;
  constexpr int P = Rows::kPasses;
  auto fetch = [&](int i, f16x8 (&hi)[P], f16x8 (&lo)[P]) {
    static_for<P>([&](auto pc) {
      constexpr int p = decltype(pc)::value;
      uint32_t row, col;
      Rows::place(p, lane, row, col);
      const int64_t m = m0 + wm * T::WM + i * 32 + row, n = n0 + wn * T::WN + col;
      hi[p] = f16x8{};
      lo[p] = f16x8{};
      if (m < m_all && n < ld_d) {  // (ld_d is a multiple of 64)
        hi[p] = *reinterpret_cast<const f16x8*>(c_in + m * ld_d + n);
        if constexpr (MODE != kSquare) lo[p] = *reinterpret_cast<const f16x8*>(lo_io + m * ld_d + n);
      }
    });
  };
  // The smallest tile fetches it before the K loop: a latency of its own at
  // the end of a short loop otherwise.
  constexpr bool kEarly = MODE != kGram && T::WM == 32;
  [[maybe_unused]] f16x8 hi_in[2][P], lo_in[2][P];  // of this block and the next
  if constexpr (kEarly) fetch(0, hi_in[0], lo_in[0]);

  E::acc acc[T::kFragM][T::kFragN] = {};
  {
    asr_mfma::Operands op;
    op.ld_a = op.ld_b = static_cast<uint32_t>((MODE == kGram ? l.ld_t : l.ld_s) * 2);
    op.kbytes = static_cast<int32_t>(op.ld_a);
    op.ktiles = asr_mfma::ktiles_of(op.kbytes);
    op.a = ws + (MODE == kGram ? l.x : MODE == kSquare ? l.a : l.wide ? l.b : y_now) + m0 * op.ld_a;
    op.b = ws + (MODE == kGram ? l.x : MODE == kSquare ? l.a : l.wide ? y_now : l.b) + n0 * op.ld_b;
    op.last_a = m_all - 1 - static_cast<int32_t>(m0);
    op.last_b = n_all - 1 - static_cast<int32_t>(n0);
    asr_mfma::mfma_loop<T, E>(op, smem, acc);
  }

  _Float16* d_out = reinterpret_cast<_Float16*>(
      ws + (MODE == kGram ? l.a : MODE == kSquare ? l.b : l.wide ? l.x : y_next));
  const float inv_sa = 1.0f / l.sa;
  const float alpha = MODE == kGram ? l.sa / (l.sx * l.sx) : MODE == kSquare ? args.c * inv_sa : inv_sa;
  const float beta = MODE == kSquare ? args.b : args.a;
  const float inv_sx = 1.0f / l.sx;

  uint32_t* slice = reinterpret_cast<uint32_t*>(smem) + wave * (Rows::kSliceBytes / 4);
  _Float16* tile = reinterpret_cast<_Float16*>(smem + Rows::kBytes);
  const bool turn = MODE == kUpdate || (kSymmetric && tm != tn);
  const uint32_t turn_sel = turn_selector(lane);
  if constexpr (MODE != kGram && !kEarly) fetch(0, hi_in[0], lo_in[0]);
  static_for<Turn<T>::kPhases>([&](auto phase_c) {
    constexpr int phase = decltype(phase_c)::value;
    // the last K tile is read, or the last phase's turned rows
    if (phase == 0 || turn) __syncthreads();
    static_for<Turn<T>::kBlocks>([&](auto bc) {
      constexpr int block = decltype(bc)::value, i = phase * Turn<T>::kBlocks + block;
      if constexpr (MODE != kGram && i + 1 < T::kFragM) fetch(i + 1, hi_in[(i + 1) & 1], lo_in[(i + 1) & 1]);
      Rows::put(slice, acc[i], lane);
      static_for<P>([&](auto pc) {
        constexpr int p = decltype(pc)::value;
        uint32_t row, col, raw[8];
        Rows::place(p, lane, row, col);
        Rows::get(slice, row, col, raw);
        const uint32_t nt = wn * T::WN + col;
        const int64_t m = m0 + wm * T::WM + i * 32 + row, n = n0 + nt;
        const bool live = m < m_all;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = alpha * __uint_as_float(raw[e]);
        if constexpr (MODE != kGram) {
          const f16x8 hi = hi_in[i & 1][p], lo = lo_in[i & 1][p];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = MODE == kSquare ? static_cast<float>(hi[e])
                                            : static_cast<float>(hi[e]) + static_cast<float>(lo[e]);
            v[e] = beta * x + v[e];
          }
        }
        if constexpr (MODE == kFinal) {
          if (live && n < n_all) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= inv_sx;
            const int count = static_cast<int>(min(int64_t{8}, n_all - n));
            const int64_t at = m * n_all + n;
            if (args.out.vec8 && count == 8) {
              store_out<OUT, 8>(args.out, d, at, 8, true, v);
            } else {
              const float v0[4] = {v[0], v[1], v[2], v[3]}, v1[4] = {v[4], v[5], v[6], v[7]};
              store_out<OUT, 4>(args.out, d, at, min(count, 4), args.out.vec4 && count >= 4, v0);
              store_out<OUT, 4>(args.out, d, at + 4, count - 4, args.out.vec4 && count == 8, v1);
            }
          }
        } else {
          f16x8 hi, lo;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] = live && n + e < n_all ? v[e] : 0.0f;  // the padding reads as zeros
            hi[e] = static_cast<_Float16>(v[e]);
            lo[e] = static_cast<_Float16>(v[e] - static_cast<float>(hi[e]));
          }
          if (turn) {
            const uint32_t mt = wm * (Turn<T>::kBlocks * 32) + block * 32 + row;
#pragma unroll
            for (int e = 0; e < 8; e += 2)
              *reinterpret_cast<uint32_t*>(tile + Turn<T>::at(nt + e + (lane & 1u), mt >> 3) + (mt & 6u)) =
                  turn_pair(v[e], v[e + 1], turn_sel);
          }
          if (live && n < ld_d) {
            *reinterpret_cast<f16x8*>(d_out + m * ld_d + n) = hi;
            if constexpr (MODE == kUpdate) *reinterpret_cast<f16x8*>(lo_io + m * ld_d + n) = lo;
          }
        }
      });
    });
    if constexpr (MODE != kFinal) {
      if (turn) {
        __syncthreads();
        _Float16* t_out = reinterpret_cast<_Float16*>(
            ws + (MODE == kGram ? l.a : MODE == kSquare ? l.b : l.wide ? y_next : l.x));
        constexpr int kChunks = Turn<T>::kRows / 8, kWaveChunks = Turn<T>::kBlocks * 4;
        for (uint32_t q = threadIdx.x; q < T::BN * kChunks; q += T::kThreads) {
          const uint32_t nt = q / kChunks, chunk = q % kChunks;
          const int64_t m = m0 + chunk / kWaveChunks * T::WM + phase * (Turn<T>::kBlocks * 32) +
                            chunk % kWaveChunks * 8;
          if (n0 + nt < n_all && m < ld_turned)
            *reinterpret_cast<f16x8*>(t_out + (n0 + nt) * ld_turned + m) =
                *reinterpret_cast<const f16x8*>(tile + Turn<T>::at(nt, chunk));
        }
      }
    }
  });
}

using Big = asr_mfma::Tile<256, 256, 128, 64, 2>;
using Mid = asr_mfma::Tile<192, 192, 96, 96, 3>;
using Small = asr_mfma::Tile<128, 128, 64, 64, 2>;
using Small8 = asr_mfma::Tile<128, 128, 64, 32, 3>;
using Tiny = asr_mfma::Tile<64, 64, 32, 32, 3>;

// ------------------------------------------------------- one workgroup
// All steps of a small matrix in one workgroup of 16 waves: X stays in f32 in
// the accumulator registers (32 x 32 blocks, kSmallBlocks of them a wave), its
// f16 copy lies in LDS both ways, and a X + B X accumulates onto a X. Three
// launches a step become four barriers. Bound by the latency of dependent
// products and LDS accesses on one compute unit: 128 x 128 takes 25 us, where
// the 17 launches of the other way took 78.
constexpr int kSmallWaves = 16;
constexpr int kSmallBlocks = 3;
constexpr int kSmallLds = 159 * 1024;

__host__ __device__ inline bool is_small(int32_t rows, int32_t cols) {
  const int64_t s = up(rows < cols ? rows : cols, 32), t = up(rows < cols ? cols : rows, 32);
  return s <= 128 && (s / 32) * (t / 32) <= kSmallWaves * kSmallBlocks &&
         2 * (s * (t + 8) + t * (s + 8) + 2 * s * (s + 8)) <= kSmallLds && 4 * s * (t + 4) <= kSmallLds;
}

struct SmallArgs {
  Desc d[kMaxBatch];
  double eps;
  float a, b, c, momentum;
  int32_t nesterov, steps;
  uint32_t vec;  // gradient and momentum start on 16-byte addresses
  OutArgs out;
};

// A value the compiler has to take as new: what is computed from it is not
// kept in registers from one part of the kernel to the next (the index
// arithmetic of all parts together would not fit beside X).
__device__ __forceinline__ int32_t fresh(int32_t x) {
  asm volatile("" : "+s"(x));
  return x;
}

template <typename G, bool MUON, int OUT>
__global__ __launch_bounds__(kSmallWaves * 64) void small_matrix(SmallArgs args) {
  using E = asr_mfma::ElemF16;
  __shared__ __align__(16) unsigned char smem[kSmallLds];
  __shared__ double lds[kSmallWaves];
  const Desc& d = args.d[blockIdx.x];
  const Layout l(d.rows, d.cols);
  const int32_t s = l.s, t = l.t;
  const int32_t sb = (s + 31) / 32, tb = (t + 31) / 32;  // blocks a side
  const int32_t ld_x = tb * 32 + 8, ld_y = sb * 32 + 8;  // (8: against bank conflicts)
  _Float16* x = reinterpret_cast<_Float16*>(smem);
  _Float16* y = x + sb * 32 * ld_x;
  _Float16* gram = y + tb * 32 * ld_y;
  _Float16* poly = gram + sb * 32 * ld_y;
  const int32_t lane = threadIdx.x & 63, row = lane & 31, half = lane >> 5;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const G* g = static_cast<const G*>(d.g);

  // Block b of this wave is block (i, j) of X; register r of it is row
  // i * 32 + lane % 32, column j * 32 + 8 (r / 4) + 4 (lane / 32) + r % 4.
  E::acc xr[kSmallBlocks];
  auto each_block = [&](auto&& f) {
    static_for<kSmallBlocks>([&](auto bc) {
      const int32_t at = fresh(wave) + decltype(bc)::value * kSmallWaves;
      if (at < sb * tb) f(xr[decltype(bc)::value], at / tb, at % tb);
    });
  };
  // U comes in, and O goes out, 8 elements of a thread at a time in memory's
  // order, through an f32 copy of X in the LDS (that the f16 ones then take).
  float* stage = reinterpret_cast<float*>(smem);
  const int32_t ld_f = tb * 32 + 4;
  const int32_t cols = d.cols, numel = d.rows * cols;
  const bool vec = args.vec && cols % 8 == 0;
  // f(first element, how many, row and column of element e of the run)
  auto each_run = [&](auto&& f) {
    for (int32_t i = static_cast<int32_t>(threadIdx.x) * 8; i < numel; i += kSmallWaves * 64 * 8) f(i, min(8, numel - i));
  };
  auto stage_at = [&](int32_t i) {
    const int32_t r = i / cols, c = i - r * cols;
    return l.wide ? r * ld_f + c : c * ld_f + r;
  };
  double sum = 0.0;
  each_run([&](int32_t i, int32_t n) {
    float gx[8], mx[8] = {}, u[8];
    if (vec) {
      asr::load_vec<false, 8>(g + i, gx);
      if constexpr (MUON) asr::load_vec<false, 8>(d.m + i, mx);
    } else {
      asr::load_range<8>(g, i, 0, n, gx);
      if constexpr (MUON) asr::load_range<8>(d.m, i, 0, n, mx);
    }
    momentum_update<MUON>(gx, mx, args.momentum, args.nesterov, true, u);
    if constexpr (MUON) {
      if (vec) asr::store_vec<false, 8>(d.m + i, mx);
      else asr::store_range<8>(d.m, i, 0, n, mx);
    }
    const int32_t at = stage_at(i);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (e < n) {
        sum += static_cast<double>(u[e]) * static_cast<double>(u[e]);
        stage[vec ? (l.wide ? at + e : at + e * ld_f) : stage_at(i + e)] = u[e];
      }
    }
  });
  const double norm = __builtin_sqrt(group_sum<kSmallWaves * 64>(sum, lds));
  const double factor = static_cast<double>(l.sx) / (norm + args.eps);
  each_block([&](E::acc& xb, int32_t i, int32_t j) {
    const int32_t m = i * 32 + row, n = j * 32 + 4 * half;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      // (what lies past the matrix is zero whatever the factor is)
      const bool in = m < s && n + 8 * (r / 4) + r % 4 < t;
      const float u = in ? stage[m * ld_f + n + 8 * (r / 4) + r % 4] : 0.0f;
      xb[r] = in ? static_cast<float>(static_cast<double>(u) * factor) : 0.0f;
    }
  });
  __syncthreads();  // the f16 copies take the LDS over

  const uint32_t turn_sel = turn_selector(static_cast<uint32_t>(lane));
  const float gram_scale = l.sa / (l.sx * l.sx), inv_sa = 1.0f / l.sa;
  // this wave's block of A and B, in the lower triangle: the LDS reads of the
  // operands are what bounds a step
  const bool squares = wave < sb * (sb + 1) / 2;
  const int32_t si = wave < 1 ? 0 : wave < 3 ? 1 : wave < 6 ? 2 : 3, sj = wave - si * (si + 1) / 2;
  auto frag = [&](const _Float16* base, int32_t ld, int32_t block, int32_t kk) {
    return *reinterpret_cast<const f16x8*>(base + (block * 32 + row) * ld + 16 * kk + 8 * half);
  };
  // c += the block of rows pa of p times rows qa of q, over `blocks` * 32 of K
  auto dot = [&](E::acc& c, const _Float16* q, int32_t ld_q, int32_t qa, const _Float16* p,
                 int32_t ld_p, int32_t pa, int32_t blocks) {
    for (int32_t kk = 0; kk < blocks; ++kk) {
      const f16x8 q0 = frag(q, ld_q, qa, 2 * kk), p0 = frag(p, ld_p, pa, 2 * kk);
      const f16x8 q1 = frag(q, ld_q, qa, 2 * kk + 1), p1 = frag(p, ld_p, pa, 2 * kk + 1);
      c = E::mfma(q0, p0, c);
      c = E::mfma(q1, p1, c);
    }
  };
  auto put4 = [&](_Float16* at, float v0, float v1, float v2, float v3) {
    *reinterpret_cast<f16x4*>(at) = f16x4{static_cast<_Float16>(v0), static_cast<_Float16>(v1),
                                          static_cast<_Float16>(v2), static_cast<_Float16>(v3)};
  };
  // block (si, sj) of a symmetric matrix, and its mirror
  auto put_square = [&](_Float16* base, const E::acc& v) {
    _Float16* to = base + (si * 32 + row) * ld_y + sj * 32 + 4 * half;
    _Float16* mirror = base + (sj * 32 + 4 * half + (lane & 1)) * ld_y + si * 32 + (row & ~1);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      put4(to + 8 * q, v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      if (si != sj) {
#pragma unroll
        for (int e = 0; e < 4; e += 2)
          *reinterpret_cast<uint32_t*>(mirror + (8 * q + e) * ld_y) = turn_pair(v[4 * q + e], v[4 * q + e + 1], turn_sel);
      }
    }
  };
  for (int step = 0; step < args.steps; ++step) {
    each_block([&](E::acc& xb, int32_t i, int32_t j) {
      _Float16* to_x = x + (i * 32 + row) * ld_x + j * 32 + 4 * half;
      _Float16* to_y = y + (j * 32 + 4 * half + (lane & 1)) * ld_y + i * 32 + (row & ~1);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        put4(to_x + 8 * q, xb[4 * q], xb[4 * q + 1], xb[4 * q + 2], xb[4 * q + 3]);
#pragma unroll
        for (int e = 0; e < 4; e += 2)
          *reinterpret_cast<uint32_t*>(to_y + (8 * q + e) * ld_y) = turn_pair(xb[4 * q + e], xb[4 * q + e + 1], turn_sel);
      }
    });
    __syncthreads();
    E::acc aa = {};
    if (squares) {
      dot(aa, x, ld_x, sj, x, ld_x, si, tb);
      // (b A takes the same rounded A as c A A: near singular values of 1 the two
      // terms' slopes, -4.8 and 4.1, all but cancel what the rounding costs)
#pragma unroll
      for (int r = 0; r < 16; ++r) aa[r] = static_cast<float>(static_cast<_Float16>(aa[r] * gram_scale));
      put_square(gram, aa);
    }
    __syncthreads();
    if (squares) {
      E::acc bb = {};
      dot(bb, gram, ld_y, sj, gram, ld_y, si, sb);
#pragma unroll
      for (int r = 0; r < 16; ++r) bb[r] = args.b * aa[r] + args.c * inv_sa * bb[r];
      put_square(poly, bb);
    }
    __syncthreads();
    each_block([&](E::acc& xb, int32_t i, int32_t j) {
#pragma unroll
      for (int r = 0; r < 16; ++r) xb[r] *= args.a * l.sa;
      dot(xb, y, ld_y, j, poly, ld_y, i, sb);
#pragma unroll
      for (int r = 0; r < 16; ++r) xb[r] *= inv_sa;
    });
    __syncthreads();  // every wave has read X^T and B
  }

  const float inv_sx = 1.0f / l.sx;
  each_block([&](E::acc& xb, int32_t i, int32_t j) {
    float* to = stage + (i * 32 + row) * ld_f + j * 32 + 4 * half;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<asr::f32x4*>(to + 8 * q) = asr::f32x4{xb[4 * q] * inv_sx, xb[4 * q + 1] * inv_sx,
                                                              xb[4 * q + 2] * inv_sx, xb[4 * q + 3] * inv_sx};
  });
  __syncthreads();
  each_run([&](int32_t i, int32_t n) {
    float o[8] = {};
    const int32_t at = stage_at(i);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) o[e] = stage[vec ? (l.wide ? at + e : at + e * ld_f) : stage_at(i + e)];
    store_out<OUT, 8>(args.out, d, i, n, args.out.vec8 && n == 8, o);
  });
}

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

template <typename F>
hipError_t launch(F* f, uint32_t grid, int threads, void* args, hipStream_t s) {
  void* argv[] = {args};
  return hipLaunchKernel(reinterpret_cast<const void*>(f), dim3(grid), dim3(threads), argv, 0, s);
}

template <typename T, int MODE, int OUT>
hipError_t launch_tile(ProductArgs& a, hipStream_t s) {
  uint32_t total = 0;
  for (int k = 0; k < a.count; ++k) {
    a.d[k].first = total;
    total += static_cast<uint32_t>(tiles_of(MODE, a.d[k].rows, a.d[k].cols, T::BM));
  }
  return launch(&product<T, MODE, OUT>, total, T::kThreads, &a, s);
}

// A tile size: `slots` of them run at once; one costs `fixed` microseconds
// (`store` more where it updates X and the chip is full: the traffic of the
// epilogues) and for every 64 of K `alone` to `full`, by how many of the slots
// are taken. Fitted to one-round launches of 1024^2 to 4096^2 and 8 x 1024 x 4096
// (microseconds a product, 256 / 192 / 128 / 128 in 8 waves / 64 tile):
//   A of 1024^2 28/24/16/13/8.5, of 2048^2 44/37/26/22/28, of 4096^2
//   92/82/109/118/160; X of 1024^2 34/30/18/15/10, of 4096^2
//   135/173/150/178/230, of 8 x 1024 x 4096 116/174/134/154/191.
struct Choice {
  int tile, slots;
  double fixed, store, alone, full;
};
constexpr Choice kChoices[] = {{256, 256, 14.0, 16.0, 1.35, 1.6},
                               {192, 256, 10.0, 8.0, 0.9, 1.1},
                               {128, 512, 8.0, 8.0, 0.62, 1.05},
                               {128, 256, 5.0, 4.0, 0.57, 0.6},
                               {64, 768, 4.0, 3.0, 0.3, 0.65}};

// Time of a launch in one tile size: its matrices' tiles, in order, go to the
// next free slot.
double launch_time(int mode, const ProductArgs& a, const Choice& c) {
  const int slots = c.slots;
  int64_t tiles = 0;
  for (int k = 0; k < a.count; ++k) tiles += tiles_of(mode, a.d[k].rows, a.d[k].cols, c.tile);
  const double taken = std::clamp((static_cast<double>(tiles) - 128.0) / (slots - 128.0), 0.0, 1.0);
  const double fixed = c.fixed + (mode == kGram || mode == kSquare ? 0.0 : c.store * taken);
  const double per_k = c.alone + (c.full - c.alone) * taken;
  // free[i] slots are free at when[i]; few different times ever coexist
  double when[kMaxBatch + 2] = {0.0};
  int free[kMaxBatch + 2] = {slots};
  int levels = 1;
  double end = 0.0;
  for (int k = 0; k < a.count; ++k) {
    const Layout l(a.d[k].rows, a.d[k].cols);
    const double cost = fixed + per_k * ((mode == kGram ? l.ld_t : l.ld_s) / 64);
    int64_t n = tiles_of(mode, a.d[k].rows, a.d[k].cols, c.tile);
    if (n > 4 * slots) {  // whole rounds at once
      const int64_t rounds = n / slots - 2;
      for (int i = 0; i < levels; ++i) when[i] += rounds * cost;
      n -= rounds * slots;
    }
    while (n > 0) {
      int first = 0;
      for (int i = 1; i < levels; ++i)
        if (when[i] < when[first]) first = i;
      const int take = static_cast<int>(std::min<int64_t>(n, free[first]));
      const double done = when[first] + cost;
      end = std::max(end, done);
      n -= take;
      free[first] -= take;
      int same = -1;
      for (int i = 0; i < levels; ++i)
        if (when[i] == done) same = i;
      if (same >= 0) free[same] += take;
      else if (free[first] == 0) when[first] = done, free[first] = take;
      else if (levels < kMaxBatch + 2) when[levels] = done, free[levels++] = take;
      else when[first] = done, free[first] += take;  // (no room: a little late)
      if (free[first] == 0) {
        --levels;
        when[first] = when[levels];
        free[first] = free[levels];
      }
    }
  }
  for (int i = 0; i < levels; ++i) end = std::max(end, when[i]);
  return end;
}

template <int MODE, int OUT = kOutBf16>
hipError_t launch_product(ProductArgs& a, hipStream_t s) {
  int best = 0;
  double least = launch_time(MODE, a, kChoices[0]);
  for (int i = 1; i < 5; ++i) {
    const double t = launch_time(MODE, a, kChoices[i]);
    if (t < least) best = i, least = t;
  }
  switch (best) {
    case 0: return launch_tile<Big, MODE, OUT>(a, s);
    case 1: return launch_tile<Mid, MODE, OUT>(a, s);
    case 2: return launch_tile<Small, MODE, OUT>(a, s);
    case 3: return launch_tile<Small8, MODE, OUT>(a, s);
    default: return launch_tile<Tiny, MODE, OUT>(a, s);
  }
}

// What a call does with every matrix of its list.
struct Settings {
  int32_t steps;
  double a, b, c, eps;
  float momentum;
  bool nesterov;
  OutArgs out;
  char* ws;
  hipStream_t stream;
};

// Largest singular value the polynomial lets any of [0, 1] reach in `steps`
// steps, and the largest |b x^2 + c x^4| it meets: what the f16 operands'
// scales (2**14 at most) have to hold.
bool coefficients_ok(double a, double b, double c, int steps) {
  if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
  double top = 1.0;
  for (int k = 0; k < steps; ++k) {
    double next = 0.0;
    for (int i = 0; i <= 256; ++i) {
      const double x = top * i / 256, q = x * x;
      if (std::fabs(b * q + c * q * q) > 3.75) return false;
      next = std::max(next, std::fabs(x * (a + b * q + c * q * q)));
    }
    if (next > 1.4) return false;
    if (next <= top) return true;  // the later steps stay inside what was looked at
    top = next;
  }
  return true;
}

template <typename G, bool MUON, int OUT>
hipError_t run_small(const Settings& st, const Desc* const* list, int32_t n) {
  SmallArgs a{};
  a.eps = st.eps;
  a.a = static_cast<float>(st.a);
  a.b = static_cast<float>(st.b);
  a.c = static_cast<float>(st.c);
  a.momentum = st.momentum;
  a.nesterov = st.nesterov;
  a.steps = st.steps;
  a.out = st.out;
  for (int32_t k0 = 0; k0 < n; k0 += kMaxBatch) {
    const int32_t count = std::min(kMaxBatch, n - k0);
    a.vec = 1;
    for (int32_t k = 0; k < count; ++k) {
      a.d[k] = *list[k0 + k];
      a.vec = a.vec && aligned_to(a.d[k].g, 16) && (!MUON || aligned_to(a.d[k].m, 16));
    }
    const hipError_t e = launch(&small_matrix<G, MUON, OUT>, static_cast<uint32_t>(count),
                                kSmallWaves * 64, &a, st.stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// One group of matrices that share a workspace, the longest K first.
template <typename G, bool MUON, int OUT>
hipError_t run_group(const Settings& st, const Desc* const* list, int32_t count) {
  PrepareArgs pa{};
  pa.ws = st.ws;
  pa.eps = st.eps;
  pa.momentum = st.momentum;
  pa.nesterov = st.nesterov;
  pa.count = count;
  pa.vec = 1;
  int64_t at = 0;
  uint32_t total = 0;
  for (int32_t k = 0; k < count; ++k) {
    Desc& d = pa.d[k];
    d = *list[k];
    d.ws = at;
    at += Layout(d.rows, d.cols).bytes;
    pa.vec = pa.vec && aligned_to(d.g, 16) && (!MUON || aligned_to(d.m, 16));
    const int64_t numel = static_cast<int64_t>(d.rows) * d.cols;
    d.first = total;
    total += static_cast<uint32_t>((numel + part_size(numel) - 1) / part_size(numel));
  }
  hipError_t e = launch(&sum_squares<G, MUON>, total, 256, &pa, st.stream);
  if (e != hipSuccess) return e;
  total = 0;
  for (int32_t k = 0; k < count; ++k) {
    pa.d[k].first = total;
    total += static_cast<uint32_t>(((pa.d[k].rows + 63) / 64) * ((pa.d[k].cols + 63) / 64));
  }
  e = launch(&scale_matrix<G, MUON>, total, 256, &pa, st.stream);
  if (e != hipSuccess) return e;

  ProductArgs a{};
  std::copy(pa.d, pa.d + count, a.d);
  a.ws = st.ws;
  a.a = static_cast<float>(st.a);
  a.b = static_cast<float>(st.b);
  a.c = static_cast<float>(st.c);
  a.count = count;
  a.out = st.out;
  for (int32_t i = 0; i < st.steps; ++i) {
    a.y = i & 1;
    if ((e = launch_product<kGram>(a, st.stream)) != hipSuccess) return e;
    if ((e = launch_product<kSquare>(a, st.stream)) != hipSuccess) return e;
    if (i + 1 < st.steps) e = launch_product<kUpdate>(a, st.stream);
    else e = launch_product<kFinal, OUT>(a, st.stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The list's order: matrices for one workgroup first, then the others by
// falling long side, cut into groups of at most kMaxBatch whose workspace stays
// near kWorkspaceAim (one matrix, if it alone needs more).
bool goes_before(int32_t r0, int32_t c0, int32_t r1, int32_t c1) {
  const bool s0 = is_small(r0, c0), s1 = is_small(r1, c1);
  if (s0 != s1) return s0;
  return std::max(r0, c0) > std::max(r1, c1);
}

template <typename Shape>
int32_t group_end(int32_t k0, int32_t n, Shape shape, int64_t& bytes) {
  bytes = 0;
  int32_t k = k0;
  for (; k < n && k - k0 < kMaxBatch; ++k) {
    const auto [r, c] = shape(k);
    const int64_t b = Layout(r, c).bytes;
    if (k > k0 && bytes + b > kWorkspaceAim) break;
    bytes += b;
  }
  return k;
}

template <typename G, bool MUON, int OUT>
hipError_t run(const Settings& st, const Desc* const* list, int32_t n) {
  int32_t small = 0;
  while (small < n && is_small(list[small]->rows, list[small]->cols)) ++small;
  hipError_t e = run_small<G, MUON, OUT>(st, list, small);
  for (int32_t k0 = small; k0 < n && e == hipSuccess;) {
    int64_t bytes;
    const int32_t k1 = group_end(k0, n, [&](int32_t k) { return std::pair(list[k]->rows, list[k]->cols); }, bytes);
    e = run_group<G, MUON, OUT>(st, list + k0, k1 - k0);
    k0 = k1;
  }
  return e;
}

int check(const char* who, int32_t n, int32_t g_dtype, int32_t steps, double a, double b, double c,
          double eps) {
  const std::string w(who);
  if (n < 0) return fail(ASR_EINVAL, w + ": a negative number of matrices");
  if (g_dtype != ASR_F32 && g_dtype != ASR_BF16) return fail(ASR_EDTYPE, w + ": unknown dtype");
  if (steps < 1 || steps > 64) return fail(ASR_EINVAL, w + ": steps must be in [1, 64]");
  if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(ASR_EINVAL, w + ": eps must be finite, >= 0");
  if (!coefficients_ok(a, b, c, steps))
    return fail(ASR_EINVAL, w + ": the coefficients let singular values in [0, 1] grow past 1.4 "
                                "(or |b x^2 + c x^4| past 3.75)");
  return ASR_OK;
}

bool sides_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && rows <= kMaxSide && cols <= kMaxSide;
}

int check_workspace(const char* who, void* ws, size_t bytes, size_t need) {
  if (need > 0 && (!ws || !aligned_to(ws, 256) || bytes < need))
    return fail(ASR_EWORKSPACE, std::string(who) + ": workspace NULL, too small or not 256-byte aligned");
  return ASR_OK;
}

struct Shape { int32_t rows, cols; };

// Workspace of n matrices in list order (see goes_before).
template <typename F>
size_t list_bytes(int32_t n, F shape) {
  int32_t k0 = 0;
  while (k0 < n && is_small(shape(k0).first, shape(k0).second)) ++k0;
  int64_t most = 0;
  while (k0 < n) {
    int64_t bytes;
    k0 = group_end(k0, n, shape, bytes);
    most = std::max(most, bytes);
  }
  return static_cast<size_t>(most);
}

}  // namespace

extern "C" {

size_t asr_newton_schulz_workspace_bytes(int32_t n, int64_t rows, int64_t cols) {
  if (n <= 0 || rows <= 0 || cols <= 0 || !sides_ok(rows, cols) ||
      is_small(static_cast<int32_t>(rows), static_cast<int32_t>(cols)))
    return 0;
  int64_t bytes;
  group_end(0, n, [&](int32_t) { return std::pair(static_cast<int32_t>(rows), static_cast<int32_t>(cols)); }, bytes);
  return static_cast<size_t>(bytes);
}

int asr_newton_schulz(const void* const* g, uint16_t* const* out, int32_t n, int64_t rows,
                      int64_t cols, int32_t g_dtype, int32_t steps, double a, double b, double c,
                      double eps, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "newton_schulz";
  if (int rc = check(who, n, g_dtype, steps, a, b, c, eps)) return rc;
  if (!sides_ok(rows, cols)) return fail(ASR_EINVAL, "newton_schulz: rows and cols must be in [0, 2**20]");
  if (n == 0 || rows == 0 || cols == 0) return ok();
  if (!g || !out) return fail(ASR_EINVAL, "newton_schulz: null array");
  Settings st{steps, a, b, c, eps, 0.0f, false, {}, static_cast<char*>(workspace),
              static_cast<hipStream_t>(stream)};
  st.out.vec8 = cols % 8 == 0;
  st.out.vec4 = cols % 4 == 0;
  for (int32_t k = 0; k < n; ++k) {
    if (!g[k] || !out[k]) return fail(ASR_EINVAL, "newton_schulz: null matrix");
    if (!aligned_to(g[k], g_dtype == ASR_F32 ? 4 : 2) || !aligned_to(out[k], 2))
      return fail(ASR_EALIGN, "newton_schulz: matrices must be aligned to their element size");
    st.out.vec8 = st.out.vec8 && aligned_to(out[k], 16);
    st.out.vec4 = st.out.vec4 && aligned_to(out[k], 8);
  }
  if (int rc = check_workspace(who, workspace, workspace_bytes,
                               asr_newton_schulz_workspace_bytes(n, rows, cols)))
    return rc;
  std::unique_ptr<Desc[]> descs(new (std::nothrow) Desc[n]);
  std::unique_ptr<const Desc*[]> list(new (std::nothrow) const Desc*[n]);
  if (!descs || !list) return fail(ASR_EINVAL, "newton_schulz: out of host memory");
  for (int32_t k = 0; k < n; ++k) {
    descs[k] = Desc{g[k], nullptr, out[k], 0, 0, static_cast<int32_t>(rows), static_cast<int32_t>(cols), 0.0f, 0};
    list[k] = &descs[k];
  }
  const hipError_t e = g_dtype == ASR_F32 ? run<float, false, kOutBf16>(st, list.get(), n)
                                          : run<uint16_t, false, kOutBf16>(st, list.get(), n);
  return e == hipSuccess ? ok() : hip_fail(e, "newton_schulz launch");
}

size_t asr_muon_workspace_bytes(const asr_muon_tensor* tensors, int32_t n) {
  if (!tensors || n <= 0) return 0;
  std::unique_ptr<Shape[]> shapes(new (std::nothrow) Shape[n]);
  if (!shapes) return 0;
  int32_t live = 0;
  for (int32_t k = 0; k < n; ++k) {
    const asr_muon_tensor& t = tensors[k];
    if (!sides_ok(t.rows, t.cols)) return 0;
    if (t.rows > 0 && t.cols > 0)
      shapes[live++] = Shape{static_cast<int32_t>(t.rows), static_cast<int32_t>(t.cols)};
  }
  std::sort(shapes.get(), shapes.get() + live, [](const Shape& x, const Shape& y) {
    return goes_before(x.rows, x.cols, y.rows, y.cols);
  });
  return list_bytes(live, [&](int32_t k) { return std::pair(shapes[k].rows, shapes[k].cols); });
}

int asr_muon_step(const asr_muon_tensor* tensors, int32_t n, int32_t param_dtype, int32_t grad_dtype,
                  double lr, double momentum, int32_t nesterov, double weight_decay,
                  int32_t ns_steps, double ns_a, double ns_b, double ns_c, double eps, int64_t step,
                  uint32_t seed, int32_t rounding, void* workspace, size_t workspace_bytes,
                  void* stream) {
  const char* who = "muon";
  if (int rc = check(who, n, grad_dtype, ns_steps, ns_a, ns_b, ns_c, eps)) return rc;
  if (param_dtype != ASR_F32 && param_dtype != ASR_BF16)
    return fail(ASR_EDTYPE, "muon: unknown param dtype");
  if (rounding != ASR_ROUND_SR && rounding != ASR_ROUND_RN)
    return fail(ASR_EINVAL, "muon: rounding must be ASR_ROUND_SR or ASR_ROUND_RN");
  if (!(lr >= 0.0) || !std::isfinite(lr) || !(weight_decay >= 0.0) || !std::isfinite(weight_decay) ||
      !(momentum >= 0.0 && momentum < 1.0))
    return fail(ASR_EINVAL, "muon: lr and weight_decay finite and >= 0, momentum in [0, 1)");
  if (step < 1 || step >= (int64_t{1} << 32))
    return fail(ASR_EINVAL, "muon: step must be in [1, 2**32 - 1]");
  if (n == 0) return ok();
  if (!tensors) return fail(ASR_EINVAL, "muon: null list");
  std::unique_ptr<Desc[]> descs(new (std::nothrow) Desc[n]);
  std::unique_ptr<const Desc*[]> list(new (std::nothrow) const Desc*[n]);
  if (!descs || !list) return fail(ASR_EINVAL, "muon: out of host memory");
  Settings st{ns_steps, ns_a, ns_b, ns_c, eps, static_cast<float>(momentum),
              nesterov != 0, {}, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)};
  st.out.decay = static_cast<float>(1.0 - lr * weight_decay);
  st.out.seed = seed;
  st.out.step = static_cast<uint32_t>(step);
  st.out.vec8 = st.out.vec4 = 1;
  int32_t live = 0;
  for (int32_t k = 0; k < n; ++k) {
    const asr_muon_tensor& t = tensors[k];
    if (!sides_ok(t.rows, t.cols)) return fail(ASR_EINVAL, "muon: rows and cols must be in [0, 2**20]");
    if (!(t.lr_factor >= 0.0) || !std::isfinite(t.lr_factor))
      return fail(ASR_EINVAL, "muon: lr_factor must be finite and >= 0");
    if (t.rows == 0 || t.cols == 0) continue;
    if (!t.param || !t.grad || !t.momentum) return fail(ASR_EINVAL, "muon: null buffer");
    if (!aligned_to(t.param, param_dtype == ASR_F32 ? 4 : 2) ||
        !aligned_to(t.grad, grad_dtype == ASR_F32 ? 4 : 2) || !aligned_to(t.momentum, 4))
      return fail(ASR_EALIGN, "muon: buffers must be aligned to their element size");
    st.out.vec8 = st.out.vec8 && t.cols % 8 == 0 && aligned_to(t.param, 16);
    st.out.vec4 = st.out.vec4 && t.cols % 4 == 0 && aligned_to(t.param, param_dtype == ASR_F32 ? 16 : 8);
    descs[live] = Desc{t.grad, t.momentum, t.param, t.base_index, 0, static_cast<int32_t>(t.rows),
                       static_cast<int32_t>(t.cols), static_cast<float>(lr * t.lr_factor), 0};
    list[live] = &descs[live];
    ++live;
  }
  if (live == 0) return ok();
  std::sort(list.get(), list.get() + live, [](const Desc* x, const Desc* y) {
    return goes_before(x->rows, x->cols, y->rows, y->cols);
  });
  const size_t need = list_bytes(live, [&](int32_t k) { return std::pair(list[k]->rows, list[k]->cols); });
  if (int rc = check_workspace(who, workspace, workspace_bytes, need)) return rc;
  hipError_t e;
  auto go = [&](auto g) {
    using G = decltype(g);
    if (param_dtype == ASR_F32) return run<G, true, kOutWeightF32>(st, list.get(), live);
    if (rounding == ASR_ROUND_SR) return run<G, true, kOutWeightBf16Sr>(st, list.get(), live);
    return run<G, true, kOutWeightBf16Rn>(st, list.get(), live);
  };
  if (grad_dtype == ASR_F32) e = go(float{});
  else e = go(uint16_t{});
  return e == hipSuccess ? ok() : hip_fail(e, "muon launch");
}

}  // extern "C"
