// The layers between a model's products, and activations kept in 8 bits for
// the backward pass.
//
// 8-bit activations: a block is 128 consecutive columns of a row (the last one
// shorter) and has one scale: codes and scale as in codes.hpp. What they stand
// for is f32(q * s). 1.03 bytes an element.
//
// layer norm of a row x of C columns:
//   mean = sum x / C, var = sum (x - mean)^2 / C, rstd = 1 / sqrt(var + eps),
//   xh = (x - mean) rstd, y = xh w + b;
//   with g = dy w: dx = rstd (g - sum g / C - xh sum(g xh) / C),
//   dw = sum over rows of dy xh, db = sum over rows of dy.
// mean and var are summed in 64 bits (so that one pass over the row gives both) and
// kept for the backward pass as two f32 numbers for the mean and one for rstd. Or the
// pass keeps the 8-bit codes of xh instead of x: their definition is the codes of the
// 64-bit xh, so that no rounding on the way decides one, and gradients use what the
// codes stand for.
//
// gated SiLU: y = g sig(g) u, du = dy g sig(g), dg = dy u sig(g) (1 + g (1 - sig(g))),
// from g and u themselves or from their 8-bit codes.
//
// Large calls are bound by memory; the kernels read their inputs once and hold them in
// registers, but for a norm's rows of more than 8192 columns, which are read twice forward
// and three times backward. 8 columns a lane, so 16 lanes hold a block of codes.
#include "mfma_loop.hpp"
#include "rows.hpp"
#include "status.hpp"

#include <adamw_sr.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#pragma clang fp contract(off)

namespace asr_layers {

using namespace asr_rows;

constexpr int kBlockCols = 128;  // columns that share a scale

// ------------------------------------------------ elementwise over rows
// A workgroup of 256 lanes is 16 groups of 16 lanes, a block of 128 columns each: 2**side
// blocks of a row side by side, and 16 >> side rows; U times that many rows an item of
// work, loaded together. Items are numbered row groups first, chunks of a row within.
struct Grid {
  int64_t rows;
  int32_t cols, blocks;   // blocks of 128 columns in a row
  int32_t side, chunks;   // log2 of blocks side by side; chunks of them in a row
  uint32_t items;
};

// A lane's place in its item, the same in every item, and an item's own, which is
// the same for the whole workgroup: addresses are one add of a lane's offset.
struct Spot {
  int32_t row, col, block;
};

__device__ __forceinline__ Spot spot_of(const Grid& g) {
  const int32_t group = threadIdx.x / 16, block = group & ((1 << g.side) - 1);
  return Spot{group >> g.side, block * kBlockCols + static_cast<int32_t>(threadIdx.x % 16) * 8, block};
}

struct Item {
  int64_t row;          // of the first of the U row groups
  int32_t col, block;
  int32_t left, padded; // columns from col to the row's end, and to the next multiple of 16
};

template <int U>
__device__ __forceinline__ Item item_of(const Grid& g, uint32_t item) {
  const uint32_t chunks = static_cast<uint32_t>(g.chunks);
  const uint32_t up = item / chunks, chunk = item - up * chunks;
  Item i;
  i.row = static_cast<int64_t>(up) * (U * (16 >> g.side));
  i.block = static_cast<int32_t>(chunk << g.side);
  i.col = i.block * kBlockCols;
  i.left = g.cols - i.col;
  i.padded = (i.left + 15) / 16 * 16;
  return i;
}

// Row group u of an item: its first row, and how many of a lane's columns there are (0
// or less: none).
struct Place {
  int64_t row;
  int32_t count, padded;
};

__device__ __forceinline__ Place place_of(const Grid& g, const Item& i, const Spot& s, int u) {
  Place p;
  p.row = i.row + u * (16 >> g.side);
  const bool there = s.row < static_cast<int32_t>(min(g.rows - p.row, int64_t{16}));
  p.count = there ? i.left - s.col : 0;
  p.padded = there ? i.padded - s.col : 0;
  return p;
}

// A matrix with row stride ld, and a lane's offset in any item.
template <typename T>
struct Lanes {
  T* base;
  int64_t ld, lane;
  __device__ __forceinline__ Lanes(T* p, int64_t ld_, const Spot& s) : base(p), ld(ld_), lane(s.row * ld_ + s.col) {}
  __device__ __forceinline__ T* at(const Item& i, const Place& p) const { return base + (p.row * ld + i.col) + lane; }
};

// Codes of 8 columns in a block that 16 lanes hold, and the block's scale.
template <bool SR>
__device__ __forceinline__ asr::u32x2 block_codes(const float (&x)[8], const uint32_t (&r)[8], float& scale) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, asr_i8::abs_bits(x[e]));
  top = reduce16(top, [](uint32_t a, uint32_t b) { return max(a, b); });
  asr_i8::GroupScale g;
  scale = asr_i8::group_scale(top, g);
  const float x0[4] = {x[0], x[1], x[2], x[3]}, x1[4] = {x[4], x[5], x[6], x[7]};
  const uint32_t r0[4] = {r[0], r[1], r[2], r[3]}, r1[4] = {r[4], r[5], r[6], r[7]};
  return asr::u32x2{asr_i8::codes4<SR>(x0, g, r0), asr_i8::codes4<SR>(x1, g, r1)};
}

struct Codes {
  int8_t* q;
  float* s;       // rows x blocks
  int64_t ld;     // of q, a multiple of 16
};

// 8 codes and their block's scale as loaded; q's rows are padded to 16 bytes.
struct Stored {
  asr::u32x2 w;
  float s;
  __device__ __forceinline__ void load(const int8_t* q, const float* s_, bool there) {
    w = there ? load_stream(reinterpret_cast<const asr::u32x2*>(q)) : asr::u32x2{0, 0};
    s = there ? *s_ : 0.0f;
  }
  __device__ __forceinline__ float get(int e) const {
    return static_cast<float>(static_cast<int32_t>(w[e / 4] << (24 - e % 4 * 8)) >> 24) * s;
  }
};

struct CodeLanes {
  Lanes<int8_t> q;
  Lanes<float> s;
  __device__ __forceinline__ CodeLanes(const Codes& c, const Grid& g, const Spot& spot)
      : q(c.q, c.ld, spot), s(c.s, g.blocks, Spot{spot.row, spot.block, 0}) {}
  __device__ __forceinline__ float* scale(const Item& i, const Place& p) const {
    return s.base + (p.row * s.ld + i.block) + s.lane;
  }
  __device__ __forceinline__ void store(const Item& i, const Place& p, asr::u32x2 w, float value) const {
    if (p.padded > 0) store_stream(reinterpret_cast<asr::u32x2*>(q.at(i, p)), w);
    if (threadIdx.x % 16 == 0 && p.count > 0) *scale(i, p) = value;
  }
  __device__ __forceinline__ Stored load(const Item& i, const Place& p) const {
    Stored c;
    c.load(q.at(i, p), scale(i, p), p.count > 0);
    return c;
  }
};

struct Pack {
  Grid g;
  void* x;       // read by pack, written by unpack
  int64_t ldx;
  Codes c;
  uint64_t base;
  uint32_t seed, step;
};

// Bound by memory to nearest: 8192 x 14336 bf16, 352 MB in and out, in 59 us, 5.9 TB/s.
// Stochastic 96 us: the random bits, 2 Philox calls of 10 rounds for 8 columns. The
// scale is the 16 lanes' maximum by 4 register moves, no LDS and no second read.
template <typename S, bool SR, int U>
__global__ __launch_bounds__(256) void pack(Pack a) {
  const Spot spot = spot_of(a.g);
  const Lanes<const S> x(static_cast<const S*>(a.x), a.ldx, spot);
  const CodeLanes c(a.c, a.g, spot);
  for (uint32_t item = blockIdx.x; item < a.g.items; item += gridDim.x) {
    const Item i = item_of<U>(a.g, item);
    Run<S> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Place p = place_of(a.g, i, spot, u);
      raw[u].load_once(x.at(i, p), p.count);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Place p = place_of(a.g, i, spot, u);
      uint32_t bits[8] = {};
      if constexpr (SR) {
        const uint64_t at = a.base + static_cast<uint64_t>(p.row + spot.row) * static_cast<uint64_t>(a.g.cols) +
                            static_cast<uint64_t>(i.col + spot.col);
        asr_mfma::random_run<8>(at, (at & 3u) == 0, a.seed, a.step, bits);
      }
      float v[8], scale;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = raw[u].get(e);
      const asr::u32x2 w = block_codes<SR>(v, bits, scale);
      c.store(i, p, w, scale);
    }
  }
}

// The same bytes the other way: 57 us, 6.2 TB/s.
template <typename S, int U>
__global__ __launch_bounds__(256) void unpack(Pack a) {
  const Spot spot = spot_of(a.g);
  const Lanes<S> x(static_cast<S*>(a.x), a.ldx, spot);
  const CodeLanes c(a.c, a.g, spot);
  for (uint32_t item = blockIdx.x; item < a.g.items; item += gridDim.x) {
    const Item i = item_of<U>(a.g, item);
    Stored in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) in[u] = c.load(i, place_of(a.g, i, spot, u));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Place p = place_of(a.g, i, spot, u);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = in[u].get(e);
      store8(x.at(i, p), p.count, v);
    }
  }
}

// --------------------------------------------------------- gated SiLU
struct Silu {
  Grid g;
  const void* gate;
  const void* up;
  const void* dy;
  void* y;
  void* dgate;
  void* dup;
  Codes cg, cu;
  int64_t ld_gate, ld_up, ld_dy, ld_y, ld_dgate, ld_dup;
};

// 1 / (1 + exp(-x)). For bf16 values the exponential and reciprocal instructions: the
// argument's two roundings come to |x| 0.9 * 2**-23 of the value, the instructions to a step
// each, so it is off by (|x| + 3) 2**-23 of itself at most, far below the output's 2**-9. A
// value below 2**-126 is 0 there. f32 values take the accurate functions (0 from where
// exp(-x) overflows, x < -88.7).
template <typename S>
__device__ __forceinline__ float sigmoid(float x) {
  if constexpr (std::is_same_v<S, float>) return 1.0f / (1.0f + expf(-x));
  else return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

// Bound by memory: 8192 x 14336 bf16, 705 MB, in 110 us, 6.4 TB/s; with both inputs'
// codes, 943 MB, in 155 us, 6.1 TB/s (codes and memory take about as long here, so
// what the codes cost shows).
template <typename S, bool SAVE, int U>
__global__ __launch_bounds__(256) void silu_forward(Silu a) {
  const Spot spot = spot_of(a.g);
  const Lanes<const S> gate(static_cast<const S*>(a.gate), a.ld_gate, spot), up(static_cast<const S*>(a.up), a.ld_up, spot);
  const Lanes<S> out(static_cast<S*>(a.y), a.ld_y, spot);
  const CodeLanes cg(a.cg, a.g, spot), cu(a.cu, a.g, spot);
  for (uint32_t item = blockIdx.x; item < a.g.items; item += gridDim.x) {
    const Item i = item_of<U>(a.g, item);
    Run<S> rg[U], ru[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const Place p = place_of(a.g, i, spot, k);
      rg[k].load_once(gate.at(i, p), p.count);
      ru[k].load_once(up.at(i, p), p.count);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const Place p = place_of(a.g, i, spot, k);
      float g[8], u[8], y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        g[e] = rg[k].get(e);
        u[e] = ru[k].get(e);
        y[e] = g[e] * sigmoid<S>(g[e]) * u[e];
      }
      store8(out.at(i, p), p.count, y);
      if constexpr (SAVE) {
        const uint32_t none[8] = {};
        float scale;
        asr::u32x2 w = block_codes<false>(g, none, scale);
        cg.store(i, p, w, scale);
        w = block_codes<false>(u, none, scale);
        cu.store(i, p, w, scale);
      }
    }
  }
}

// Bound by memory: 1174 MB in 185 us, 6.4 TB/s; from codes 943 MB in 147 us, 6.4 TB/s.
template <typename S, bool SAVED, int U>
__global__ __launch_bounds__(256) void silu_backward(Silu a) {
  const Spot spot = spot_of(a.g);
  const Lanes<const S> gate(static_cast<const S*>(a.gate), a.ld_gate, spot), up(static_cast<const S*>(a.up), a.ld_up, spot),
      dy(static_cast<const S*>(a.dy), a.ld_dy, spot);
  const Lanes<S> dgate(static_cast<S*>(a.dgate), a.ld_dgate, spot), dup(static_cast<S*>(a.dup), a.ld_dup, spot);
  const CodeLanes cg(a.cg, a.g, spot), cu(a.cu, a.g, spot);
  for (uint32_t item = blockIdx.x; item < a.g.items; item += gridDim.x) {
    const Item i = item_of<U>(a.g, item);
    Run<S> rd[U];
    std::conditional_t<SAVED, Stored, Run<S>> rg[U], ru[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const Place p = place_of(a.g, i, spot, k);
      rd[k].load_once(dy.at(i, p), p.count);
      if constexpr (SAVED) {
        rg[k] = cg.load(i, p);
        ru[k] = cu.load(i, p);
      } else {
        rg[k].load_once(gate.at(i, p), p.count);
        ru[k].load_once(up.at(i, p), p.count);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const Place p = place_of(a.g, i, spot, k);
      float dg[8], du[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = rg[k].get(e), d = rd[k].get(e), sig = sigmoid<S>(g);
        du[e] = d * (g * sig);
        dg[e] = d * (ru[k].get(e) * (sig * (1.0f + g * (1.0f - sig))));   // (d u may overflow where this does not)
      }
      store8(dgate.at(i, p), p.count, dg);
      store8(dup.at(i, p), p.count, du);
    }
  }
}

// ---------------------------------------------------------- layer norm
// What the backward pass needs of a row.
struct __align__(16) RowStat {
  float mean, rest;   // their sum is the mean
  float rstd, none;
};

struct Norm {
  const void* x;
  const void* w;
  const void* b;
  const void* dy;
  void* y;
  void* dx;
  RowStat* stat;
  float* part;        // backward: sums of a workgroup's rows, [workgroup][dw, db][cols]
  void* dw;
  void* db;
  Codes c;
  int64_t rows, ldx, ld_dy;
  int32_t cols, blocks;
  double eps, inv_cols;
  float inv_cols32;
  uint32_t w_bf16, alone;   // alone: one workgroup, whose sums are the result
  uint32_t more;            // the workgroups' sums go on top of an earlier launch's
  int32_t fold;             // rows of a lane's first sum
};

// Two sums over the lanes of a row, in every lane.
struct Pair {
  double a, b;
};

template <int LANES>
__device__ __forceinline__ Pair row_sum(Pair v, Pair* lds) {
  v.a = wave_sum(v.a);
  v.b = wave_sum(v.b);
  if constexpr (LANES > 64) {
    constexpr int kWaves = LANES / 64;
    if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
    __syncthreads();
    v = Pair{0.0, 0.0};
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      v.a += lds[threadIdx.x / LANES * kWaves + i].a;
      v.b += lds[threadIdx.x / LANES * kWaves + i].b;
    }
  }
  return v;
}

__device__ __forceinline__ RowStat stat_of(double mean, double rstd) {
  RowStat s;
  s.mean = static_cast<float>(mean);
  s.rest = static_cast<float>(mean - static_cast<double>(s.mean));
  s.rstd = static_cast<float>(rstd);
  s.none = 0.0f;
  return s;
}

// (x - mean) rstd, the mean in two parts: x - mean's first is exact or off by half a
// step of itself, so a mean far larger than the spread costs nothing.
struct Normal {
  float mean, rstd, off;
  __device__ __forceinline__ explicit Normal(const RowStat& s) : mean(s.mean), rstd(s.rstd), off(-s.rest * s.rstd) {}
  __device__ __forceinline__ float operator()(float x) const { return __builtin_fmaf(x - mean, rstd, off); }
};

// mean and var from one pass: sums of d = x - pivot and of d^2 in 64 bits, the pivot
// being the row's first element. var = sum d^2 / C - (sum d / C)^2 loses little there:
// (pivot - mean)^2 <= C var, as the pivot is itself a term of the variance, so its
// relative error is below about C 2**-52 (and a constant row has d = 0). One
// reduction over the lanes instead of two.
__device__ __forceinline__ void add8(const float (&x)[8], int64_t count, double pivot, Pair& t) {
  if (count >= 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double d = static_cast<double>(x[e]) - pivot;
      t.a += d;
      t.b = __builtin_fma(d, d, t.b);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e) {
      const double d = static_cast<double>(x[e]) - pivot;
      if (e < count) {
        t.a += d;
        t.b = __builtin_fma(d, d, t.b);
      }
    }
  }
}

__device__ __forceinline__ void moments(const Norm& a, Pair t, double pivot, double& mean, double& rstd) {
  const double off = t.a * a.inv_cols, var = t.b * a.inv_cols - off * off;
  mean = pivot + off;
  // 1 / sqrt(v): the instruction's 2**-26 and one Newton step, a quarter of the
  // instructions of a root and a division (v = 0, Inf and NaN give NaN, and 0
  // times an Inf is NaN too)
  const double v = (var < 0.0 ? 0.0 : var) + a.eps, r = __builtin_amdgcn_rsq(v);
  rstd = __builtin_fma(r * 0.5, __builtin_fma(-v * r, r, 1.0), r);
}

// Codes of the normalised values of 8 columns, as 64 bits decide them: scale from the
// largest |x - mean| of the block, which is that of its largest or smallest x (16
// lanes). A code is the nearest whole number to (x - mean) (rstd / s); in 32 bits
// that is off by less than 5e-5 (five roundings of 2**-24 of at most 127, the sum's one
// of 2**-24 of 128), so only a wave with an element nearer than 6e-5 to a border
// decides in 64.
__device__ __forceinline__ asr::u32x2 norm_codes(const float (&x)[8], int64_t count, double mean, double rstd,
                                                 const Normal& normal, float& scale) {
  constexpr float kByte = 12582912.0f;  // 1.5 * 2**23: a sum's low byte is its whole part
  float hi = -__builtin_inff(), lo = __builtin_inff();
  if (count >= 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      hi = __builtin_fmaxf(hi, x[e]);
      lo = __builtin_fminf(lo, x[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e) {
      hi = e < count ? __builtin_fmaxf(hi, x[e]) : hi;
      lo = e < count ? __builtin_fminf(lo, x[e]) : lo;
    }
  }
  hi = reduce16(hi, [](float a, float b) { return __builtin_fmaxf(a, b); });
  lo = reduce16(lo, [](float a, float b) { return __builtin_fminf(a, b); });
  // (a NaN or Inf in the row has made the mean one)
  const double most = __builtin_fmax(__builtin_fabs(static_cast<double>(hi) - mean),
                                     __builtin_fabs(static_cast<double>(lo) - mean));
  const float s = static_cast<float>(most * rstd * (1.0 / 127.0));
  const bool finite = s < __builtin_inff();    // (false for NaN)
  const bool live = finite && s >= 0x1p-126f;
  scale = finite ? (live ? s : 0.0f) : __uint_as_float(0x7FC00000u);
  float inv = __builtin_amdgcn_rcpf(live ? s : 1.0f);
  inv = __builtin_fmaf(__builtin_fmaf(-s, inv, 1.0f), inv, inv);
  const float turn32 = live ? normal.rstd * inv : 0.0f, off = normal.off * inv;
  uint32_t u[8];
  float far = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = __builtin_fmaf(x[e] - normal.mean, turn32, off), v = t + kByte;
    far = __builtin_fmaxf(far, __builtin_fabsf(t - (v - kByte)));
    u[e] = __float_as_uint(v);
  }
  // (turn32 is 127 over the block's largest difference: from 2**-119 on that one is held by
  // 32 bits, and far, which says nothing about a NaN, sees none; rstd below its normal
  // numbers has too few bits)
  const bool held = turn32 > 0x1p-119f && turn32 < 0x1p100f && normal.rstd >= 0x1p-126f && off == off;
  if (__builtin_amdgcn_ballot_w64(live && !(far < 0.49994f && held)) != 0) {
    const double turn = live ? rstd / static_cast<double>(s) : 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double t = __builtin_rint((static_cast<double>(x[e]) - mean) * turn);
      u[e] = static_cast<uint32_t>(static_cast<int32_t>(__builtin_fmin(__builtin_fmax(t, -127.0), 127.0)));
    }
  }
  asr::u32x2 w = {asr_i8::pack_bytes(u[0], u[1], u[2], u[3]), asr_i8::pack_bytes(u[4], u[5], u[6], u[7])};
  if (count < 8) {   // zeros behind the row's end
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e >= count) w[e / 4] &= ~(0xFFu << (e % 4 * 8));
  }
  return live ? w : asr::u32x2{0, 0};
}

// weight and bias of a lane's columns (1 and 0 where there is none)
struct Affine {
  float w[8], b[8];
  __device__ __forceinline__ void load(const Norm& a, int64_t col) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e] = 1.0f;
      b[e] = 0.0f;
    }
    if (a.w) load_params(a.w, a.w_bf16, col, a.cols - col, w);
    if (a.b) load_params(a.b, a.w_bf16, col, a.cols - col, b);
  }
};

// y, and if wanted the codes, of 8 columns.
template <typename S, bool SAVE>
__device__ __forceinline__ void finish8(const Norm& a, int64_t row, int64_t col, int64_t count, bool live,
                                        const float (&x)[8], double mean, double rstd, const RowStat& stat,
                                        const Affine& p) {
  const Normal normal(stat);
  if constexpr (SAVE) {
    float scale;
    const asr::u32x2 codes = norm_codes(x, count, mean, rstd, normal, scale);
    if (live && col < (static_cast<int64_t>(a.cols) + 15) / 16 * 16) {
      store_stream(reinterpret_cast<asr::u32x2*>(a.c.q + row * a.c.ld + col), codes);
      if (threadIdx.x % 16 == 0 && count > 0) a.c.s[row * a.blocks + col / kBlockCols] = scale;
    }
  }
  float out[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = __builtin_fmaf(normal(x[e]), p.w[e], p.b[e]);
  store8(static_cast<S*>(a.y) + row * static_cast<int64_t>(a.cols) + col, count, out);
}

// Rows of up to LANES * KEEP * 8 columns, held in registers by LANES lanes; a group of
// lanes takes several rows, the workgroups' number apart, with its weights and biases
// in registers, and loads the next row before it joins the sums of this one.
// 8192 x 4096 bf16, 134 MB: 24-25 us, 5.5 TB/s, where a copy of it takes 22-24: a row's
// chain of load, sum over its lanes and store is what a workgroup waits for. (Past the
// caches 29 us, by 512 lanes 37, by a wave a row, without a barrier but with 64
// columns a lane, 40.) With codes 36-39 us, 4.5 TB/s: beside the chain, the arithmetic
// (64-bit sums and maxima of blocks: 14 us of it). f32, 268 MB: 60 us, 4.5 TB/s.

// Waves that the registers of a SIMD hold.
constexpr int norm_waves(int keep, bool save) { return keep == 1 ? (save ? 5 : 7) : (save ? 3 : 4); }

template <typename S, int LANES, int KEEP, bool SAVE>
__global__ __launch_bounds__(LANES > 256 ? LANES : 256, norm_waves(KEEP, SAVE)) void norm_rows(Norm a) {
  constexpr int kThreads = LANES > 256 ? LANES : 256, kGroups = kThreads / LANES;
  __shared__ Pair lds[2][kThreads / 64];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  Affine params[KEEP];
#pragma unroll
  for (int v = 0; v < KEEP; ++v) params[v].load(a, (lane + v * LANES) * 8);
  Run<S> next[KEEP], first_next;
  auto fetch = [&](int64_t row) {
    const bool live = row < a.rows;
    const S* x = static_cast<const S*>(a.x) + row * a.ldx;
    first_next.load(x, live ? 1 : 0);
#pragma unroll
    for (int v = 0; v < KEEP; ++v) {
      const int64_t col = (lane + v * LANES) * 8;
      next[v].load(x + col, live ? a.cols - col : 0);
    }
  };
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGroups;
  int64_t first = static_cast<int64_t>(blockIdx.x) * kGroups;
  fetch(first + group);
  for (int turn = 0; first < a.rows; first += stride, turn ^= 1) {
    const int64_t row = first + group;
    const bool live = row < a.rows;
    const double pivot = static_cast<double>(first_next.get(0));
    float x[KEEP][8];
    Pair t = {0.0, 0.0};
#pragma unroll
    for (int v = 0; v < KEEP; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] = next[v].get(e);
      add8(x[v], a.cols - (lane + v * LANES) * 8, pivot, t);
    }
    if (first + stride < a.rows) fetch(row + stride);
    double mean, rstd;
    moments(a, row_sum<LANES>(t, lds[turn]), pivot, mean, rstd);
    const RowStat stat = stat_of(mean, rstd);
    if (a.stat && live && lane == 0) a.stat[row] = stat;
#pragma unroll
    for (int v = 0; v < KEEP; ++v) {
      const int64_t col = (lane + v * LANES) * 8;
      finish8<S, SAVE>(a, row, col, live ? a.cols - col : 0, live, x[v], mean, rstd, stat, params[v]);
    }
  }
}

// Longer rows: a workgroup each, read twice (the second time mostly from the caches), two
// runs of a lane at once. Bound by the chain of a row's loads, sums and stores: 2048 x
// 16384 bf16, 134 MB, in 30 us, 4.4 TB/s.
template <typename S, bool SAVE, int LANES>
__global__ __launch_bounds__(LANES) void norm_long_rows(Norm a) {
  constexpr int kCols = LANES * 8;
  __shared__ Pair lds[LANES / 64];
  const int64_t row = blockIdx.x;
  const S* x = static_cast<const S*>(a.x) + row * a.ldx;
  Run<S> raw[2];
  auto fetch = [&](int64_t col) {
#pragma unroll
    for (int u = 0; u < 2; ++u) raw[u].load(x + col + u * kCols, a.cols - col - u * kCols);
  };
  raw[0].load(x, 1);
  const double pivot = static_cast<double>(raw[0].get(0));
  Pair t = {0.0, 0.0};
  for (int64_t col = threadIdx.x * 8; col < a.cols; col += 2 * kCols) {
    fetch(col);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = raw[u].get(e);
      add8(v, a.cols - col - u * kCols, pivot, t);
    }
  }
  double mean, rstd;
  moments(a, row_sum<LANES>(t, lds), pivot, mean, rstd);
  const RowStat stat = stat_of(mean, rstd);
  if (a.stat && threadIdx.x == 0) a.stat[row] = stat;
  // (all lanes in every turn: the codes' reduction wants them active)
  for (int64_t start = 0; start < a.cols; start += 2 * kCols) {
    const int64_t col = start + threadIdx.x * 8;
    fetch(col);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t c = col + u * kCols;
      float v[8];
      Affine p;
      p.load(a, c);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = raw[u].get(e);
      finish8<S, SAVE>(a, row, c, a.cols - c, true, v, mean, rstd, stat, p);
    }
  }
}

// Normalised values of 8 columns for the backward pass: from x, or from the codes. Places
// past a row's end repeat its last one (lanes with none of it add nothing): dy is 0
// there, and 0 times what a 0 in x would give is NaN where the mean times rstd overflows.
template <typename S, bool SAVED>
struct Normalised {
  std::conditional_t<SAVED, Stored, Run<S>> v;
  __device__ __forceinline__ void load(const Norm& a, int64_t row, int64_t col, int64_t count) {
    if constexpr (SAVED) {
      v.load(a.c.q + row * a.c.ld + col, a.c.s + row * a.blocks + col / kBlockCols, count > 0);
    } else {
      v.load_repeated(static_cast<const S*>(a.x) + row * a.ldx + col, count);
    }
  }
  __device__ __forceinline__ float get(int e, const Normal& normal) const {
    if constexpr (SAVED) return v.get(e);
    else return normal(v.get(e));
  }
};

__device__ __forceinline__ void store_param(void* p, bool bf16, int64_t i, float x) {
  if (bf16) static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(bf16_pair(x, 0.0f));
  else static_cast<float*>(p)[i] = x;
}

// dx, and the sums over rows for dw and db. A row of up to LANES * 8 columns takes
// LANES lanes of a workgroup of 1024, its next row `gridDim` times 1024 / LANES
// further. A lane keeps its columns' sums over all of its rows in registers, the
// next row is loaded while this one is worked on, and one barrier a row joins
// the waves' sums (two sets of them in turn). In the end the groups' sums meet
// in LDS. (16 columns a lane would take more registers than 16 waves have.)
// 8192 x 4096 bf16, 201 MB: 37-40 us, 5.0-5.4 TB/s, with the join below; from codes, 168 MB,
// 35 us. Bound by memory and, every row, the barrier's wait. Rows of odd width 49 us (8192
// x 4091): loads from odd addresses take the vector memory twice as long. f32: 78 us.
template <typename S, bool SAVED, int LANES>
__global__ __launch_bounds__(1024) void norm_backward(Norm a) {
  constexpr int kGroups = 1024 / LANES, kWaves = LANES / 64, kCols = LANES * 8;
  // Lanes with none of the row skip its sums, or have zeros for its statistics: 4096 x
  // 8192 f32 83 and 105 us (by the registers of the 1024 lanes), 32 x 1024 bf16 6.9 and 6.6.
  constexpr bool kSkip = LANES == 1024;
  __shared__ float sums[kGroups * kCols];
  __shared__ f32x2 joint[2][16];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int64_t col = lane * 8;
  float w[8], dw[8] = {}, db[8] = {};
  if (a.w) {
    load_params(a.w, a.w_bf16, col, a.cols - col, w);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.0f;
  }
  Run<S> dy, dy_next;
  Normalised<S, SAVED> xh, xh_next;
  RowStat stat, stat_next;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGroups;
  auto fetch = [&](int64_t row) {
    const bool live = row < a.rows;
    const int64_t count = live ? a.cols - col : 0;
    stat_next = (kSkip ? live : count > 0) ? a.stat[row] : RowStat{0.0f, 0.0f, 0.0f, 0.0f};
    dy_next.load(static_cast<const S*>(a.dy) + row * a.ld_dy + col, count);
    xh_next.load(a, row, col, count);
  };
  int64_t first = static_cast<int64_t>(blockIdx.x) * kGroups;
  fetch(first + group);
  for (int turn = 0; first < a.rows; first += stride, turn ^= 1) {
    const int64_t row = first + group;
    stat = stat_next;
    dy = dy_next;
    xh = xh_next;
    if (first + stride < a.rows) fetch(row + stride);
    const Normal normal(stat);
    f32x2 c = {0.0f, 0.0f};
    if (!kSkip || col < a.cols) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = dy.get(e), h = xh.get(e, normal), g = d * w[e];
        c.x += g;
        c.y = __builtin_fmaf(g, h, c.y);
        dw[e] = __builtin_fmaf(d, h, dw[e]);
        db[e] += d;
      }
    }
    c.x = wave_sum(c.x);
    c.y = wave_sum(c.y);
    if constexpr (kWaves > 1) {
      if (threadIdx.x % 64 == 0) joint[turn][threadIdx.x / 64] = c;
      __syncthreads();
      c = f32x2{0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        c.x += joint[turn][group * kWaves + i].x;
        c.y += joint[turn][group * kWaves + i].y;
      }
    }
    if (a.dx) {
      // rstd (g - m - h k) as g rstd - m rstd - h (k rstd)
      const float m = -c.x * a.inv_cols32 * stat.rstd, k = -c.y * a.inv_cols32 * stat.rstd;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = __builtin_fmaf(xh.get(e, normal), k, __builtin_fmaf(dy.get(e) * w[e], stat.rstd, m));
      store8(static_cast<S*>(a.dx) + row * static_cast<int64_t>(a.cols) + col, row < a.rows ? a.cols - col : 0, x);
    }
  }
  auto finish = [&](const float (&mine)[8], void* result, int which) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[group * kCols + col + e] = mine[e];
    __syncthreads();
    for (int i = threadIdx.x; i < a.cols; i += 1024) {
      float t = 0.0f;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) t += sums[k * kCols + i];
      float* part = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + which) * a.cols + i;
      if (a.alone) store_param(result, a.w_bf16, i, t);
      else *part = a.more ? *part + t : t;
    }
  };
  if (a.dw) finish(dw, a.dw, 0);
  if (a.db) finish(db, a.db, 1);
}

// Longer rows: dx by a workgroup a row, in two passes over it, two runs of a lane at once:
// 2048 x 16384 bf16 with the sums below and their join in 85 us. Dx and sums each read all of dy and
// x, where a shorter row's are read once: three times the floor, for widths that are rare.
template <typename S, bool SAVED, int LANES>
__global__ __launch_bounds__(LANES) void norm_backward_long(Norm a) {
  constexpr int kCols = LANES * 8;
  __shared__ Pair lds[LANES / 64];
  const int64_t row = blockIdx.x;
  const RowStat stat = a.stat[row];
  const Normal normal(stat);
  Run<S> dy[2];
  Normalised<S, SAVED> xh[2];
  float w[2][8];
  auto fetch = [&](int64_t col) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t c = col + u * kCols, count = a.cols - c;
      dy[u].load(static_cast<const S*>(a.dy) + row * a.ld_dy + c, count);
      xh[u].load(a, row, c, count);
      if (a.w) load_params(a.w, a.w_bf16, c, count, w[u]);
    }
  };
  if (!a.w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[0][e] = w[1][e] = 1.0f;
  }
  Pair t = {0.0, 0.0};
  for (int64_t col = threadIdx.x * 8; col < a.cols; col += 2 * kCols) {
    fetch(col);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (col + u * kCols >= a.cols) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) {   // (past the row's end dy is 0)
        const float g = dy[u].get(e) * w[u][e], h = xh[u].get(e, normal);
        t.a += static_cast<double>(g);
        t.b = __builtin_fma(static_cast<double>(g), static_cast<double>(h), t.b);
      }
    }
  }
  t = row_sum<LANES>(t, lds);
  const float m = static_cast<float>(t.a * a.inv_cols), k = static_cast<float>(t.b * a.inv_cols);
  S* out = static_cast<S*>(a.dx) + row * static_cast<int64_t>(a.cols);
  for (int64_t col = threadIdx.x * 8; col < a.cols; col += 2 * kCols) {
    fetch(col);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (dy[u].get(e) * w[u][e] - m - xh[u].get(e, normal) * k) * stat.rstd;
      store8(out + col + u * kCols, a.cols - col - u * kCols, x);
    }
  }
}

// And their sums over rows: a workgroup takes 2048 columns of a share of the rows, four
// rows at once.
template <typename S, bool SAVED>
__global__ __launch_bounds__(256) void norm_columns_long(Norm a, int32_t share, int32_t strips) {
  constexpr int kAhead = 4;
  const int32_t strip = blockIdx.x % strips, part = blockIdx.x / strips;
  const int64_t col = (static_cast<int64_t>(strip) * 256 + threadIdx.x) * 8, count = a.cols - col;
  if (count <= 0) return;
  const int64_t r0 = static_cast<int64_t>(part) * share, r1 = min(a.rows, r0 + share);
  float dw[8] = {}, db[8] = {}, all_dw[8] = {}, all_db[8] = {};
  int32_t held = 0;
  for (int64_t row = r0; row < r1; row += kAhead) {
    Run<S> dy[kAhead];
    Normalised<S, SAVED> xh[kAhead];
    RowStat stat[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const bool in = row + u < r1;
      stat[u] = in ? a.stat[row + u] : RowStat{0.0f, 0.0f, 0.0f, 0.0f};
      dy[u].load(static_cast<const S*>(a.dy) + (row + u) * a.ld_dy + col, in ? count : 0);
      xh[u].load(a, row + u, col, in ? count : 0);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const Normal normal(stat[u]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[e] = __builtin_fmaf(dy[u].get(e), xh[u].get(e, normal), dw[e]);
        db[e] += dy[u].get(e);
      }
    }
    held += kAhead;
    if (held == a.fold || row + kAhead >= r1) {
      held = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        all_dw[e] += dw[e];
        all_db[e] += db[e];
        dw[e] = db[e] = 0.0f;
      }
    }
  }
  float* out = a.part + static_cast<int64_t>(part) * 2 * a.cols + col;
  store8(out, count, all_dw);
  store8(out + a.cols, count, all_db);
}

// dw and db from the workgroups' sums: 64 columns a workgroup, 4 a lane, 64
// shares of the workgroups side by side (4 sums each, loaded at once), joined in
// LDS in their order.
__global__ __launch_bounds__(1024) void norm_params(Norm a, int32_t parts) {
  __shared__ asr::f32x4 lds[1024];
  const int which = blockIdx.y, share = threadIdx.x / 16;
  void* result = which ? a.db : a.dw;
  if (!result) return;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x % 16 * 4;
  asr::f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
  const int32_t each = (parts + 63) / 64, p1 = min(parts, (share + 1) * each);
  const int left = static_cast<int>(min(int64_t{4}, a.cols - col));
  if (left == 4) {
#pragma unroll 4
    for (int32_t p = share * each; p < p1; ++p)
      t += *reinterpret_cast<const f32x4_any*>(a.part + (static_cast<int64_t>(p) * 2 + which) * a.cols + col);
  } else {
#pragma unroll 4
    for (int32_t p = share * each; p < (left > 0 ? p1 : 0); ++p)
#pragma unroll
      for (int e = 0; e < 3; ++e)   // (past the row's end its last one again, which no one stores)
        t[e] += a.part[(static_cast<int64_t>(p) * 2 + which) * a.cols + col + min(e, left - 1)];
  }
  lds[threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.x < 16) {
#pragma unroll 16
    for (int i = 1; i < 64; ++i) t += lds[i * 16 + threadIdx.x];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) store_param(result, a.w_bf16, col + e, t[e]);
  }
}

}  // namespace asr_layers

// =========================================================== host side
namespace {

using asr_host::fail;
using asr_host::hip_fail;
using asr_host::ok;
using namespace asr_layers;

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxDim = int64_t{1} << 31;
constexpr int64_t kMaxItems = int64_t{1} << 31;
constexpr int64_t kMaxGrid = int64_t{1} << 22;   // workgroups of the kernels that loop over items
constexpr int64_t kMaxBlocks = 0xFFFFFF;         // of 256 threads in a launch of fewer than 2**32

template <typename... A>
hipError_t launch(void (*f)(A...), dim3 grid, int threads, hipStream_t s, std::common_type_t<A>... args) {
  void* argv[] = {&args...};
  return hipLaunchKernel(reinterpret_cast<const void*>(f), grid, dim3(threads), argv, 0, s);
}

template <int V>
using Const = std::integral_constant<int, V>;

int64_t blocks_of(int64_t cols) { return (cols + kBlockCols - 1) / kBlockCols; }

// An item has 16 groups of 128 columns, or kMany times as many where that leaves enough
// workgroups for the chip. At 8192 x 14336 bf16 with 1, 2 and 4: packed in 71, 59 and
// 58 us, unpacked in 61, 57 and 58, gated SiLU with codes 153, 155 and 161 (more
// registers, fewer waves), its gradient 185, 185 and 189. 4096 x 4096 (with 1 and 2)
// packed in 12.4 and 10.2; below 2048 items nothing gains (1024 x 4096 4.3 and 4.4).
constexpr int64_t kEnough = 2048;
constexpr int kMany = 2;

// 0: more work than one call takes; else the rows' factor of an item
int make_grid(Grid& g, int64_t rows, int64_t cols, int many) {
  g.rows = rows;
  g.cols = static_cast<int32_t>(cols);
  g.blocks = static_cast<int32_t>(blocks_of(cols));
  g.side = 0;
  while (g.side < 4 && (1 << g.side) < g.blocks) ++g.side;
  g.chunks = (g.blocks + (1 << g.side) - 1) >> g.side;
  const auto up = [&](int64_t each) { return (rows + each - 1) / each; };
  if (up(16 >> g.side) > kMaxItems / g.chunks - 1) return 0;
  const int each = up(many * (16 >> g.side)) * g.chunks >= kEnough ? many : 1;
  g.items = static_cast<uint32_t>(up(each * (16 >> g.side)) * g.chunks);
  return each;
}

uint32_t grid_of(const Grid& g) { return static_cast<uint32_t>(std::min<int64_t>(g.items, kMaxGrid)); }

int check_size(const char* what, int64_t rows, int64_t cols, int32_t dtype) {
  if (rows < 0 || cols < 0 || rows >= kMaxDim || cols >= kMaxDim - 4096)
    return fail(ASR_EINVAL, std::string(what) + ": rows must be in [0, 2**31), columns in [0, 2**31 - 4096)");
  if (dtype != ASR_F32 && dtype != ASR_BF16) return fail(ASR_EDTYPE, std::string(what) + ": unknown dtype");
  return ASR_OK;
}

// A matrix of the call with row stride ld (in elements).
int check_matrix(const char* what, const void* p, int64_t ld, int64_t cols, int32_t dtype) {
  if (!p) return fail(ASR_EINVAL, std::string(what) + ": null pointer");
  if (ld < cols) return fail(ASR_EINVAL, std::string(what) + ": a row stride is below the row's length");
  if (!aligned_to(p, dtype == ASR_F32 ? 4 : 2))
    return fail(ASR_EALIGN, std::string(what) + ": a pointer is not aligned to its elements");
  return ASR_OK;
}

int check_codes(const char* what, const int8_t* q, int64_t ldq, const float* s, int64_t cols) {
  if (!q || !s) return fail(ASR_EINVAL, std::string(what) + ": null pointer");
  if (ldq % 16 != 0 || ldq < (cols + 15) / 16 * 16)
    return fail(ASR_EINVAL, std::string(what) + ": rows of codes must lie a multiple of 16 bytes apart that holds "
                                                "the columns up to a multiple of 16");
  if (!aligned_to(q, 16) || !aligned_to(s, 4))
    return fail(ASR_EALIGN, std::string(what) + ": codes aligned to 16 bytes, scales to 4");
  return ASR_OK;
}

int done(hipError_t e, const char* what) { return e == hipSuccess ? ok() : hip_fail(e, what); }

// The largest number of workgroups whose sums the norm's backward pass joins.
constexpr int64_t kNormGrid = 256;
constexpr int64_t kMaxNorm = int64_t{1} << 24;   // columns of a row
constexpr int64_t kCus = 256;                    // compute units of an MI355X
// Rows of more than 8192 columns from which a workgroup has 256 lanes, not 1024, as several
// of these share a compute unit (us, bf16 forward, 256 lanes and 1024): 1024 x 9000 9.6 and
// 13, 4096 x 8200 31 and 49, with codes 45 and 81; below it the row's own time counts: 64 x
// 131072 49 and 19, 512 x 16384 9.5 and 7.9. (2048 x 16384: 30 and 28.)
constexpr int64_t kManyLong = 1024;

// Workgroups' sums in the norm's backward pass: of rows of more than 8192 columns, which
// workgroups share in strips of 2048, as many as make 8 workgroups a compute unit.
constexpr int64_t kNormStrip = 2048;
int64_t norm_parts(int64_t rows, int64_t cols) {
  const int64_t strips = cols > 8192 ? (cols + kNormStrip - 1) / kNormStrip : 1;
  return std::min({rows, kNormGrid, (8 * kCus + strips - 1) / strips});
}

int check_norm(int64_t rows, int64_t cols, int32_t dtype, int32_t param_dtype) {
  if (int rc = check_size("layer_norm", rows, cols, dtype)) return rc;
  if (param_dtype != ASR_F32 && param_dtype != ASR_BF16) return fail(ASR_EDTYPE, "layer_norm: unknown param_dtype");
  if (cols > kMaxNorm) return fail(ASR_EINVAL, "layer_norm: at most 2**24 columns");
  if (rows > kMaxBlocks) return fail(ASR_EINVAL, "layer_norm: rows must be below 2**24");
  return ASR_OK;
}

template <typename S, bool SAVE>
hipError_t norm_forward(const Norm& a, hipStream_t s) {
  const auto one = [&](auto* f, int lanes, int keep) {
    // As many workgroups as the chip holds at once, each with the same number of rows
    // or one fewer: 8192 x 4096 bf16 in 25 us by 1024, 25 by 2048, 28 by 1280, 29 by 512 and
    // 31 by 8192; with codes 37 by 768, 37 by 2048 and 41 by 512; 4096 x 8192 23 us by 512, 26
    // by 2048 and 32 by 4096. (f32 rows go the other way: 8192 x 4096 60 us by 1024, 47 by 8192.)
    const int threads = std::max(256, lanes);
    const int64_t groups = threads / lanes, rows = (a.rows + groups - 1) / groups;
    const int64_t held = kCus * (4 * norm_waves(keep, SAVE) / (threads / 64)), turns = (rows + held - 1) / held;
    return launch(f, dim3(static_cast<uint32_t>((rows + turns - 1) / turns)), threads, s, a);
  };
  if (a.cols <= 512) return one(&norm_rows<S, 64, 1, SAVE>, 64, 1);
  if (a.cols <= 1024) return one(&norm_rows<S, 128, 1, SAVE>, 128, 1);
  if (a.cols <= 2048) return one(&norm_rows<S, 256, 1, SAVE>, 256, 1);
  if (a.cols <= 4096) return one(&norm_rows<S, 256, 2, SAVE>, 256, 2);
  if constexpr (SAVE) {   // (4096 x 8192 f32 55 us, 63 by 512 lanes; bf16 46-49 and 46, 4096 x 5000 45 and 46)
    if (a.cols <= 8192) return one(&norm_rows<S, 1024, 1, SAVE>, 1024, 1);
  } else {
    if (a.cols <= 8192) return one(&norm_rows<S, 512, 2, SAVE>, 512, 2);
  }
  const dim3 grid(static_cast<uint32_t>(a.rows));
  return a.rows < kManyLong ? launch(&norm_long_rows<S, SAVE, 1024>, grid, 1024, s, a)
                            : launch(&norm_long_rows<S, SAVE, 256>, grid, 256, s, a);
}

template <typename S, bool SAVED>
hipError_t norm_back(Norm a, hipStream_t s) {
  const bool sums = a.dw || a.db;
  int64_t parts = 0;
  hipError_t e = hipSuccess;
  const auto one = [&](auto* f, int groups) {
    // Up to four turns of one workgroup cost less than the launch that joins several
    // ones' sums: 32 rows of 1024 columns 6.7 us alone, 8.1 joined; 8 x 4096 7.6 and
    // 8.7; 64 x 1024 (8 turns) 10.3 and 8.2.
    parts = sums && a.rows <= 4 * groups ? 1 : std::min<int64_t>((a.rows + groups - 1) / groups, kNormGrid);
    a.alone = sums && parts == 1;
    // A lane's sum takes up to `fold` rows (fold_of); more of them are as many launches,
    // each adding its workgroups' sums to the last one's.
    const int64_t turn = parts * groups, slice = turn * fold_of((a.rows + turn - 1) / turn);
    Norm part = a;
    for (int64_t r = 0; r < a.rows && e == hipSuccess; r += slice) {
      part.rows = std::min(slice, a.rows - r);
      part.more = r > 0;
      e = launch(f, dim3(static_cast<uint32_t>(std::min(parts, (part.rows + groups - 1) / groups))), 1024, s, part);
      part.dy = static_cast<const S*>(part.dy) + slice * a.ld_dy;
      if (a.x) part.x = static_cast<const S*>(part.x) + slice * a.ldx;
      if (a.dx) part.dx = static_cast<S*>(part.dx) + slice * a.cols;
      if (a.c.q) part.c = Codes{part.c.q + slice * a.c.ld, part.c.s + slice * a.blocks, a.c.ld};
      part.stat += slice;
    }
  };
  if (a.cols <= 512) one(&norm_backward<S, SAVED, 64>, 16);
  else if (a.cols <= 1024) one(&norm_backward<S, SAVED, 128>, 8);
  else if (a.cols <= 2048) one(&norm_backward<S, SAVED, 256>, 4);
  else if (a.cols <= 4096) one(&norm_backward<S, SAVED, 512>, 2);
  else if (a.cols <= 8192) one(&norm_backward<S, SAVED, 1024>, 1);
  else {
    const dim3 grid(static_cast<uint32_t>(a.rows));
    if (a.dx)
      e = a.rows < kManyLong ? launch(&norm_backward_long<S, SAVED, 1024>, grid, 1024, s, a)
                             : launch(&norm_backward_long<S, SAVED, 256>, grid, 256, s, a);
    if (e == hipSuccess && sums) {
      parts = norm_parts(a.rows, a.cols);
      const int32_t share = static_cast<int32_t>((a.rows + parts - 1) / parts);
      parts = (a.rows + share - 1) / share;
      a.fold = fold_of(share);
      const int32_t strips = static_cast<int32_t>((a.cols + kNormStrip - 1) / kNormStrip);
      e = launch(&norm_columns_long<S, SAVED>, dim3(static_cast<uint32_t>(parts * strips)), 256, s, a, share, strips);
    }
  }
  if (e == hipSuccess && sums && !a.alone)
    e = launch(&norm_params, dim3(static_cast<uint32_t>((static_cast<int64_t>(a.cols) + 63) / 64), 2), 1024, s, a,
               static_cast<int32_t>(parts));
  return e;
}

}  // namespace

extern "C" {

int asr_pack_i8(const void* x, int32_t dtype, int64_t ldx, int64_t rows, int64_t cols, int8_t* q, int64_t ldq,
                float* scale, int32_t rounding, uint32_t seed, uint32_t step, uint64_t base_index, void* stream) {
  if (int rc = check_size("pack_i8", rows, cols, dtype)) return rc;
  if (rounding != ASR_ROUND_SR && rounding != ASR_ROUND_RN)
    return fail(ASR_EINVAL, "pack_i8: rounding must be ASR_ROUND_SR or ASR_ROUND_RN");
  if (rows == 0 || cols == 0) return ok();
  if (int rc = check_matrix("pack_i8", x, ldx, cols, dtype)) return rc;
  if (int rc = check_codes("pack_i8", q, ldq, scale, cols)) return rc;
  if (static_cast<uint64_t>(rows) * static_cast<uint64_t>(cols) - 1 > ~base_index)
    return fail(ASR_EINVAL, "pack_i8: base_index + rows*cols exceeds 2**64");
  Pack a{};
  const int many = make_grid(a.g, rows, cols, kMany);
  if (!many) return fail(ASR_EINVAL, "pack_i8: the matrix is too large for one call");
  a.x = const_cast<void*>(x);
  a.ldx = ldx;
  a.c = Codes{q, scale, ldq};
  a.base = base_index;
  a.seed = seed;
  a.step = step;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool sr = rounding == ASR_ROUND_SR;
  const auto pick = [&](auto u) {
    return dtype == ASR_F32 ? (sr ? &pack<float, true, u> : &pack<float, false, u>)
                            : (sr ? &pack<uint16_t, true, u> : &pack<uint16_t, false, u>);
  };
  auto* f = many == 1 ? pick(Const<1>{}) : pick(Const<kMany>{});
  return done(launch(f, dim3(grid_of(a.g)), 256, s, a), "pack_i8 launch");
}

int asr_unpack_i8(const int8_t* q, int64_t ldq, const float* scale, int64_t rows, int64_t cols, void* x,
                  int32_t dtype, int64_t ldx, void* stream) {
  if (int rc = check_size("unpack_i8", rows, cols, dtype)) return rc;
  if (rows == 0 || cols == 0) return ok();
  if (int rc = check_codes("unpack_i8", q, ldq, scale, cols)) return rc;
  if (int rc = check_matrix("unpack_i8", x, ldx, cols, dtype)) return rc;
  Pack a{};
  const int many = make_grid(a.g, rows, cols, kMany);
  if (!many) return fail(ASR_EINVAL, "unpack_i8: the matrix is too large for one call");
  a.x = x;
  a.ldx = ldx;
  a.c = Codes{const_cast<int8_t*>(q), const_cast<float*>(scale), ldq};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const auto pick = [&](auto u) { return dtype == ASR_F32 ? &unpack<float, u> : &unpack<uint16_t, u>; };
  auto* f = many == 1 ? pick(Const<1>{}) : pick(Const<kMany>{});
  return done(launch(f, dim3(grid_of(a.g)), 256, s, a), "unpack_i8 launch");
}

int asr_silu_mul_forward(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up, int32_t dtype,
                         int64_t rows, int64_t cols, void* y, int64_t ld_y, int8_t* q_gate, float* s_gate,
                         int8_t* q_up, float* s_up, int64_t ldq, void* stream) {
  if (int rc = check_size("silu_mul", rows, cols, dtype)) return rc;
  if (rows == 0 || cols == 0) return ok();
  if (int rc = check_matrix("silu_mul", gate, ld_gate, cols, dtype)) return rc;
  if (int rc = check_matrix("silu_mul", up, ld_up, cols, dtype)) return rc;
  if (int rc = check_matrix("silu_mul", y, ld_y, cols, dtype)) return rc;
  const bool save = q_gate || s_gate || q_up || s_up;
  if (save) {
    if (int rc = check_codes("silu_mul", q_gate, ldq, s_gate, cols)) return rc;
    if (int rc = check_codes("silu_mul", q_up, ldq, s_up, cols)) return rc;
  }
  Silu a{};
  const int many = make_grid(a.g, rows, cols, kMany);
  if (!many) return fail(ASR_EINVAL, "silu_mul: the matrix is too large for one call");
  a.gate = gate;
  a.up = up;
  a.y = y;
  a.ld_gate = ld_gate;
  a.ld_up = ld_up;
  a.ld_y = ld_y;
  a.cg = Codes{q_gate, s_gate, ldq};
  a.cu = Codes{q_up, s_up, ldq};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const auto pick = [&](auto u) {
    return dtype == ASR_F32 ? (save ? &silu_forward<float, true, u> : &silu_forward<float, false, u>)
                            : (save ? &silu_forward<uint16_t, true, u> : &silu_forward<uint16_t, false, u>);
  };
  auto* f = many == 1 ? pick(Const<1>{}) : pick(Const<kMany>{});
  return done(launch(f, dim3(grid_of(a.g)), 256, s, a), "silu_mul launch");
}

int asr_silu_mul_backward(const void* dy, int64_t ld_dy, const void* gate, int64_t ld_gate, const void* up,
                          int64_t ld_up, const int8_t* q_gate, const float* s_gate, const int8_t* q_up,
                          const float* s_up, int64_t ldq, int32_t dtype, int64_t rows, int64_t cols, void* dgate,
                          int64_t ld_dgate, void* dup, int64_t ld_dup, void* stream) {
  if (int rc = check_size("silu_mul", rows, cols, dtype)) return rc;
  if (rows == 0 || cols == 0) return ok();
  if (int rc = check_matrix("silu_mul", dy, ld_dy, cols, dtype)) return rc;
  if (int rc = check_matrix("silu_mul", dgate, ld_dgate, cols, dtype)) return rc;
  if (int rc = check_matrix("silu_mul", dup, ld_dup, cols, dtype)) return rc;
  const bool saved = q_gate || s_gate || q_up || s_up;
  if (saved) {
    if (gate || up) return fail(ASR_EINVAL, "silu_mul: gate and up, or their codes, not both");
    if (int rc = check_codes("silu_mul", q_gate, ldq, s_gate, cols)) return rc;
    if (int rc = check_codes("silu_mul", q_up, ldq, s_up, cols)) return rc;
  } else {
    if (int rc = check_matrix("silu_mul", gate, ld_gate, cols, dtype)) return rc;
    if (int rc = check_matrix("silu_mul", up, ld_up, cols, dtype)) return rc;
  }
  Silu a{};
  const int many = make_grid(a.g, rows, cols, kMany);
  if (!many) return fail(ASR_EINVAL, "silu_mul: the matrix is too large for one call");
  a.gate = gate;
  a.up = up;
  a.dy = dy;
  a.dgate = dgate;
  a.dup = dup;
  a.ld_gate = ld_gate;
  a.ld_up = ld_up;
  a.ld_dy = ld_dy;
  a.ld_dgate = ld_dgate;
  a.ld_dup = ld_dup;
  a.cg = Codes{const_cast<int8_t*>(q_gate), const_cast<float*>(s_gate), ldq};
  a.cu = Codes{const_cast<int8_t*>(q_up), const_cast<float*>(s_up), ldq};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const auto pick = [&](auto u) {
    return dtype == ASR_F32 ? (saved ? &silu_backward<float, true, u> : &silu_backward<float, false, u>)
                            : (saved ? &silu_backward<uint16_t, true, u> : &silu_backward<uint16_t, false, u>);
  };
  auto* f = many == 1 ? pick(Const<1>{}) : pick(Const<kMany>{});
  return done(launch(f, dim3(grid_of(a.g)), 256, s, a), "silu_mul launch");
}

int asr_layer_norm_forward(const void* x, int32_t dtype, int64_t ldx, int64_t rows, int64_t cols,
                           const void* weight, const void* bias, int32_t param_dtype, double eps, void* y,
                           float* stat, int8_t* q, int64_t ldq, float* scale, void* stream) {
  if (int rc = check_norm(rows, cols, dtype, param_dtype)) return rc;
  if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(ASR_EINVAL, "layer_norm: eps must be finite and >= 0");
  if (rows == 0 || cols == 0) return ok();
  if (int rc = check_matrix("layer_norm", x, ldx, cols, dtype)) return rc;
  if (int rc = check_matrix("layer_norm", y, cols, cols, dtype)) return rc;
  if (!aligned_to(weight, param_dtype == ASR_F32 ? 4 : 2) || !aligned_to(bias, param_dtype == ASR_F32 ? 4 : 2))
    return fail(ASR_EALIGN, "layer_norm: weight and bias aligned to their elements");
  if (!aligned_to(stat, 16)) return fail(ASR_EALIGN, "layer_norm: stat aligned to 16 bytes");
  if (q || scale)
    if (int rc = check_codes("layer_norm", q, ldq, scale, cols)) return rc;
  Norm a{};
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.y = y;
  a.stat = reinterpret_cast<RowStat*>(stat);
  a.c = Codes{q, scale, ldq};
  a.rows = rows;
  a.ldx = ldx;
  a.cols = static_cast<int32_t>(cols);
  a.blocks = static_cast<int32_t>(blocks_of(cols));
  a.eps = eps;
  a.inv_cols = 1.0 / static_cast<double>(cols);
  a.w_bf16 = param_dtype == ASR_BF16;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = dtype == ASR_F32 ? (q ? norm_forward<float, true>(a, s) : norm_forward<float, false>(a, s))
                                        : (q ? norm_forward<uint16_t, true>(a, s) : norm_forward<uint16_t, false>(a, s));
  return done(e, "layer_norm launch");
}

size_t asr_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || rows > kMaxBlocks || cols > kMaxNorm) return 0;
  return static_cast<size_t>(norm_parts(rows, cols) * 2 * cols * 4);
}

int asr_layer_norm_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ldx, const int8_t* q, int64_t ldq,
                            const float* scale, const float* stat, int32_t dtype, int64_t rows, int64_t cols,
                            const void* weight, int32_t param_dtype, void* dx, void* dweight, void* dbias,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_norm(rows, cols, dtype, param_dtype)) return rc;
  if (cols == 0 || (!dx && !dweight && !dbias)) return ok();
  const uintptr_t wide = param_dtype == ASR_F32 ? 4 : 2;
  if (!aligned_to(weight, wide) || !aligned_to(dweight, wide) || !aligned_to(dbias, wide))
    return fail(ASR_EALIGN, "layer_norm: weight, dweight and dbias aligned to their elements");
  hipStream_t s = static_cast<hipStream_t>(stream);
  Norm a{};
  a.cols = static_cast<int32_t>(cols);
  a.dw = dweight;
  a.db = dbias;
  a.w_bf16 = param_dtype == ASR_BF16;
  if (rows == 0) {  // empty sums
    if (!dweight && !dbias) return ok();
    return done(launch(&norm_params, dim3(static_cast<uint32_t>((cols + 63) / 64), 2), 1024, s, a, 0), "layer_norm launch");
  }
  if (int rc = check_matrix("layer_norm", dy, ld_dy, cols, dtype)) return rc;
  if (dx)
    if (int rc = check_matrix("layer_norm", dx, cols, cols, dtype)) return rc;
  if (q || scale) {
    if (x) return fail(ASR_EINVAL, "layer_norm: x or its codes, not both");
    if (int rc = check_codes("layer_norm", q, ldq, scale, cols)) return rc;
  } else if (int rc = check_matrix("layer_norm", x, ldx, cols, dtype)) {
    return rc;
  }
  if (!stat) return fail(ASR_EINVAL, "layer_norm: null pointer");
  if (!aligned_to(stat, 16)) return fail(ASR_EALIGN, "layer_norm: stat aligned to 16 bytes");
  if ((dweight || dbias) && (!workspace || !aligned_to(workspace, 16) ||
                             workspace_bytes < asr_layer_norm_backward_workspace_bytes(rows, cols)))
    return fail(ASR_EWORKSPACE, "layer_norm: workspace NULL, too small or not 16-byte aligned");
  a.x = x;
  a.w = weight;
  a.dy = dy;
  a.dx = dx;
  a.stat = reinterpret_cast<RowStat*>(const_cast<float*>(stat));
  a.part = static_cast<float*>(workspace);
  a.c = Codes{const_cast<int8_t*>(q), const_cast<float*>(scale), ldq};
  a.rows = rows;
  a.ldx = ldx;
  a.ld_dy = ld_dy;
  a.blocks = static_cast<int32_t>(blocks_of(cols));
  a.inv_cols = 1.0 / static_cast<double>(cols);
  a.inv_cols32 = static_cast<float>(a.inv_cols);
  const hipError_t e = dtype == ASR_F32 ? (q ? norm_back<float, true>(a, s) : norm_back<float, false>(a, s))
                                        : (q ? norm_back<uint16_t, true>(a, s) : norm_back<uint16_t, false>(a, s));
  return done(e, "layer_norm launch");
}

}  // extern "C"
