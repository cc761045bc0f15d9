// The K loop of the 8-bit and 16-bit matrix products of int8.hip and
// muon.hip: acc += A * B^T for one workgroup tile, A and B row-major with K
// contiguous, on gfx950's 32x32 matrix instructions.
//
// Both element types move the same bytes: a fragment is 16 bytes a lane (8
// f16 or 16 int8 values of one row), an instruction takes 32 bytes of K from
// 32 rows of each operand, and a K tile is 128 bytes (one cache line) a row.
// The operands are swapped (B rows feed the instruction's row side), so lane
// l holds, for row l % 32 of A, runs of 4 consecutive columns: register r is
// column 8 * (r / 4) + 4 * (l / 32) + r % 4.
//
// K tiles go through a ring of STAGES LDS buffers, filled by 16-byte buffer
// loads to LDS; the 16-byte chunks of a row are XOR-swizzled, which makes the
// fragment reads free of bank conflicts. One wave a SIMD copies. The copies
// of K tile kt + STAGES go into tile kt's buffer right after the barrier
// inside tile kt's last step (every fragment of tile kt is then in
// registers), and half of that step's matrix instructions follow the barrier
// to cover the first fragment reads of tile kt + 1. Each step's order is
// fenced with sched_barrier: one fragment read for the next step after each
// matrix instruction. This is the schedule of gemm_sr.hip's kernel, where it
// was measured variant by variant.
#pragma once

#include "device.hpp"

#include <type_traits>

#pragma clang fp contract(off)

namespace asr_mfma {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_void_ptr;

struct ElemF16 {
  using frag = f16x8;
  using acc = f32x16;
  static __device__ __forceinline__ acc mfma(frag b, frag a, acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(b, a, c, 0, 0, 0);
  }
};

struct ElemI8 {
  using frag = i32x4;
  using acc = i32x16;
  static __device__ __forceinline__ acc mfma(frag b, frag a, acc c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, c, 0, 0, 0);
  }
};

constexpr int kXcds = 8;
constexpr int kRowBytes = 128;  // bytes of K a row of one K tile holds
constexpr int kCopyBytes = 1024;  // one wave-wide copy: 8 rows

// A copy's resource starts at the tile's first row and K tile; lane offsets
// at or past kOutOfRange read zeros. Valid offsets are below 255 leading
// dimensions (< 2**23 bytes each), so below 2**31.
constexpr uint32_t kOutOfRange = 0x80000000u;
constexpr int64_t kMaxLdBytes = int64_t{1} << 23;

template <int BM_, int BN_, int WM_, int WN_, int STAGES_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
  static constexpr int kWavesN = BN / WN;
  static constexpr int kWaves = (BM / WM) * kWavesN;
  static constexpr int kThreads = kWaves * 64;
  // Waves a SIMD that the LDS leaves room for (two, or one for a 4-wave
  // workgroup that has a compute unit to itself).
  static constexpr int kMinWaves =
      kWaves <= 4 && STAGES_ * (BM_ + BN_) * kRowBytes > 80 * 1024 ? 1 : 2;
  static constexpr int kFragM = WM / 32, kFragN = WN / 32;
  static constexpr int kSlabs = (BM + BN) / 8;                // wave-wide copies a K tile
  static constexpr int kCopyWaves = kWaves > 4 ? 4 : kWaves;  // one a SIMD
  static constexpr int kSlabsPerWave = kSlabs / kCopyWaves;
  static constexpr int kSlabsA = BM / 8 / kCopyWaves;         // the first of them lie in A
  static constexpr int kStageBytes = (BM + BN) * kRowBytes;
  static constexpr int kLoopLds = STAGES * kStageBytes;
  static_assert(BM % WM == 0 && BN % WN == 0 && WM % 32 == 0 && WN % 32 == 0, "tile shape");
  static_assert(kSlabs % kCopyWaves == 0 && (BM / 8) % kCopyWaves == 0, "copies split evenly");
  static_assert(STAGES >= 2 && kLoopLds <= 160 * 1024, "LDS budget");
  static_assert((STAGES - 1) * kSlabsPerWave < 64, "vmcnt range");

  // Position of 16-byte chunk c in row r: a fragment read takes one chunk
  // index from 16 consecutive rows at a time, and rows pair up in a 256-byte
  // bank period, so (r >> 1) & 7 gives the 8 pairs 8 distinct places.
  static __device__ __forceinline__ uint32_t chunk_pos(uint32_t r, uint32_t c) {
    return c ^ ((r >> 1) & 7u);
  }
  static __device__ __forceinline__ uint32_t chunk_offset(uint32_t r, uint32_t c) {
    return r * kRowBytes + (chunk_pos(r, c) << 4);
  }
};

template <int N, typename F, int I = 0>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, F, I + 1>(static_cast<F&&>(f));
  }
}

// s_waitcnt vmcnt(N) alone.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Workgroup barrier that completes this wave's LDS accesses but leaves its
// copies to LDS in flight (the loop waits for those with wait_vmcnt).
__device__ __forceinline__ void barrier_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// One output tile's operands: `a` and `b` point at the tile's first rows;
// last_a and last_b are the tile-relative indexes of the operands' last rows
// (rows past them are clamped: they only feed outputs that are not stored).
// kbytes: bytes of K, a multiple of 16; ktiles: K tiles to walk, at least those
// that hold them (what lies past K counts as zeros, unread); ld_a, ld_b in
// bytes, below 2**23.
struct Operands {
  const char* a;
  const char* b;
  uint32_t ld_a, ld_b;
  int32_t last_a, last_b;
  int32_t kbytes, ktiles;
};

__host__ __device__ constexpr int32_t ktiles_of(int32_t kbytes) { return (kbytes + kRowBytes - 1) / kRowBytes; }

// acc[i][j] += the wave's 32 x 32 blocks of A * B^T over all of K. smem: T's
// kLoopLds bytes. Every wave of the workgroup calls it; a workgroup of several
// times T's waves walks as many K ranges at once, each in an LDS part of its own,
// with one ktiles for all of them (the barriers are the workgroup's). On return no copy is
// in flight, but other waves may still read the LDS: a barrier has to come
// before it is written.
template <typename T, typename E>
__device__ __forceinline__ void mfma_loop(const Operands& op, unsigned char* smem,
                                          typename E::acc (&acc)[T::kFragM][T::kFragN]) {
  using Frag = typename E::frag;
  constexpr int BM = T::BM, STAGES = T::STAGES;
  constexpr int kSteps = kRowBytes / 32;
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % T::kWaves;
  const bool copier = T::kCopyWaves == T::kWaves || wave < static_cast<uint32_t>(T::kCopyWaves);
  const uint32_t wm = wave / T::kWavesN, wn = wave % T::kWavesN;
  const uint32_t frag_row = lane & 31u, frag_half = lane >> 5;
  const int ktiles = op.ktiles;
  const int kfull = op.kbytes / kRowBytes;
  if (ktiles == 0) return;

  // Slab j of this wave is rows (wave + j * kCopyWaves) * 8 .. + 7 of the
  // stage (A's rows, then B's); the lane copies the chunk at position
  // lane % 8 of row lane / 8.
  uint32_t voff[T::kSlabsPerWave];
#pragma unroll
  for (int j = 0; j < T::kSlabsPerWave; ++j) {
    const int32_t row = static_cast<int32_t>((wave + j * T::kCopyWaves) * 8 + lane / 8);
    const uint32_t c = T::chunk_pos(row, lane % 8);  // the XOR is its own inverse
    if (j < T::kSlabsA)
      voff[j] = static_cast<uint32_t>(min(row, op.last_a)) * op.ld_a + c * 16;
    else
      voff[j] = static_cast<uint32_t>(min(row - BM, op.last_b)) * op.ld_b + c * 16;
  }
  auto copy_at = [&](int stage, int j, int kt, uint32_t off) {
    const char* base = (j < T::kSlabsA ? op.a : op.b) + static_cast<int64_t>(kt) * kRowBytes;
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(base), static_cast<short>(0), static_cast<int32_t>(kOutOfRange),
        0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc,
        (lds_void_ptr)(smem + stage * T::kStageBytes + (wave + j * T::kCopyWaves) * kCopyBytes),
        16, off, 0, 0, 0);
  };
  auto copy = [&](int stage, int j, int kt) { copy_at(stage, j, kt, voff[j]); };
  // K tiles that K does not fill: chunks past K read zeros
  auto copy_tail = [&](int stage, int j, int kt) {
    const uint32_t row = (wave + j * T::kCopyWaves) * 8 + lane / 8;
    const int k = kt * kRowBytes + static_cast<int>(T::chunk_pos(row, lane % 8)) * 16;
    copy_at(stage, j, kt, k < op.kbytes ? voff[j] : kOutOfRange);
  };

  Frag fa[2][T::kFragM], fb[2][T::kFragN];
  auto read_frag = [&](const unsigned char* sa, int kk, int buf, auto rc) {
    constexpr int r = decltype(rc)::value;
    const uint32_t c = 2 * kk + frag_half;
    if constexpr (r < T::kFragM)
      fa[buf][r] = *reinterpret_cast<const Frag*>(
          sa + T::chunk_offset(wm * T::WM + r * 32 + frag_row, c));
    else
      fb[buf][r - T::kFragM] = *reinterpret_cast<const Frag*>(
          sa + BM * kRowBytes +
          T::chunk_offset(wn * T::WN + (r - T::kFragM) * 32 + frag_row, c));
  };
  constexpr int kReads = T::kFragM + T::kFragN;

#pragma unroll
  for (int s = 0; s < STAGES; ++s) {
    if (!copier) {
    } else if (s < kfull) {
#pragma unroll
      for (int j = 0; j < T::kSlabsPerWave; ++j) copy(s, j, s);
    } else if (s < ktiles) {
#pragma unroll
      for (int j = 0; j < T::kSlabsPerWave; ++j) copy_tail(s, j, s);
    }
  }
  // K tile 0 has landed once at most STAGES - 1 tiles of copies are out
  if (STAGES <= ktiles) wait_vmcnt<(STAGES - 1) * T::kSlabsPerWave>();
  else wait_vmcnt<0>();
  barrier_lds();
  static_for<kReads>([&](auto rc) { read_frag(smem, 0, 0, rc); });

  int cur = 0;  // LDS buffer of tile kt
  // LOAD: the copies this body issues, of tile kt + STAGES: 0 none, 1 a whole
  // tile, 2 one that K does not fill.
  auto tile_body = [&](int kt, auto load_c) {
    constexpr int LOAD = decltype(load_c)::value;
    const unsigned char* sa = smem + cur * T::kStageBytes;
    const unsigned char* na = smem + (cur + 1 == STAGES ? 0 : cur + 1) * T::kStageBytes;
    static_for<kSteps>([&](auto kkc) {
      constexpr int kk = decltype(kkc)::value;
      constexpr bool kLast = kk + 1 == kSteps;
      constexpr int kNow = kLast ? 0 : kReads;
      constexpr int kRows = kLast ? T::kFragM / 2 : T::kFragM;
      constexpr int kMf = kRows * T::kFragN;
      auto mfma = [&](auto gc) {
        constexpr int i = decltype(gc)::value / T::kFragN, j = decltype(gc)::value % T::kFragN;
        acc[i][j] = E::mfma(fb[kk & 1][j], fa[kk & 1][i], acc[i][j]);
      };
      static_for<kMf>([&](auto gc) {
        constexpr int g = decltype(gc)::value;
        mfma(gc);
        if constexpr (g < kNow) read_frag(sa, kk + 1, (kk + 1) & 1, gc);
        __builtin_amdgcn_sched_barrier(0);
      });
      static_for<(kNow > kMf ? kNow - kMf : 0)>([&](auto rc) {
        read_frag(sa, kk + 1, (kk + 1) & 1,
                  std::integral_constant<int, kMf + decltype(rc)::value>{});
      });
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (kLast) {
        if (kt + 1 < ktiles) {
          if (kt + STAGES - 1 < ktiles) wait_vmcnt<(STAGES - 2) * T::kSlabsPerWave>();
          else wait_vmcnt<0>();
          barrier_lds();  // tile kt + 1 is visible; every wave has read tile kt
        }
        __builtin_amdgcn_sched_barrier(0);
        // the rest of the step; after the last tile the reads take stale LDS
        // inside the ring, and their values are not used
        constexpr int kRest = (T::kFragM - kRows) * T::kFragN;
        constexpr int kCopies = LOAD != 0 ? T::kSlabsPerWave : 0;
        constexpr int kPer = (kCopies + kRest - 1) / kRest;
        static_for<kRest>([&](auto gc) {
          constexpr int g = decltype(gc)::value;
          if constexpr (g < kReads) read_frag(na, 0, 0, gc);
          mfma(std::integral_constant<int, kMf + g>{});
          static_for<kPer>([&](auto dc) {
            constexpr int j = g * kPer + decltype(dc)::value;
            if constexpr (j < kCopies) {
              if (copier) {
                if constexpr (LOAD == 2) copy_tail(cur, j, kt + STAGES);
                else copy(cur, j, kt + STAGES);
              }
            }
          });
          __builtin_amdgcn_sched_barrier(0);
        });
        static_for<(kReads > kRest ? kReads - kRest : 0)>([&](auto rc) {
          read_frag(na, 0, 0, std::integral_constant<int, kRest + decltype(rc)::value>{});
        });
        __builtin_amdgcn_sched_barrier(0);
      }
    });
    cur = cur + 1 == STAGES ? 0 : cur + 1;
  };
  int kt = 0;
  for (; kt + STAGES < kfull; ++kt) tile_body(kt, std::integral_constant<int, 1>{});
  for (; kt + STAGES < ktiles; ++kt) tile_body(kt, std::integral_constant<int, 2>{});
  for (; kt < ktiles; ++kt) tile_body(kt, std::integral_constant<int, 0>{});
}

// The wave's 32 rows i * 32 .. + 31 of its accumulators, turned through a slice
// of LDS of its own into runs of 8 columns whose lanes cover whole rows: a
// store of 16 bytes a lane then writes whole 128-byte lines (64 f16 columns),
// where the accumulators' own order touches 32 lines with 32 bytes each, four
// times the address cycles. (The 256 x 256 product that updates X spent
// 16 us a tile on them, of 73.) Lanes l and l ^ 1 hold neighbouring rows of
// the same columns.
template <typename T>
struct Rows {
  static constexpr int kGroups = T::WN / 8;             // runs of 8 a row
  static constexpr int kPasses = 32 * kGroups / 64;     // runs a lane gets
  static constexpr int kLd = T::WN + 4;                 // words: no bank conflicts either way
  static constexpr int kSliceBytes = 32 * kLd * 4;
  static constexpr int kBytes = T::kWaves * kSliceBytes;
  static_assert(32 * kGroups % 64 == 0, "whole passes");

  // Row in the block and first column in the wave's tile of this lane's run.
  static __device__ __forceinline__ void place(int pass, uint32_t lane, uint32_t& row, uint32_t& col) {
    const uint32_t pair = (static_cast<uint32_t>(pass) * 64 + lane) >> 1;
    row = pair / kGroups * 2 + (lane & 1u);
    col = pair % kGroups * 8;
  }
  template <typename Acc>
  static __device__ __forceinline__ void put(uint32_t* slice, const Acc (&acc)[T::kFragN], uint32_t lane) {
    uint32_t* to = slice + (lane & 31u) * kLd + 4 * (lane >> 5);
    static_for<T::kFragN>([&](auto jc) {
      static_for<4>([&](auto qc) {
        constexpr int j = decltype(jc)::value, q = decltype(qc)::value;
        // (each element as a value first: a bit cast of an element of the
        // reference took element 0 of the vector)
        const auto v0 = acc[j][4 * q], v1 = acc[j][4 * q + 1], v2 = acc[j][4 * q + 2], v3 = acc[j][4 * q + 3];
        *reinterpret_cast<asr::u32x4*>(to + j * 32 + 8 * q) =
            asr::u32x4{__builtin_bit_cast(uint32_t, v0), __builtin_bit_cast(uint32_t, v1),
                       __builtin_bit_cast(uint32_t, v2), __builtin_bit_cast(uint32_t, v3)};
      });
    });
  }
  // (a wave's LDS accesses complete in order: no wait between put and get)
  static __device__ __forceinline__ void get(const uint32_t* slice, uint32_t row, uint32_t col, uint32_t (&v)[8]) {
    const asr::u32x4 a = *reinterpret_cast<const asr::u32x4*>(slice + row * kLd + col);
    const asr::u32x4 b = *reinterpret_cast<const asr::u32x4*>(slice + row * kLd + col + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  }
};

// Index of workgroup b in an order that gives each XCD (b % 8) a contiguous
// range of `total`.
__device__ __forceinline__ uint32_t xcd_order(uint32_t b, uint32_t total) {
  const uint32_t q = total / kXcds, r = total % kXcds, x = b % kXcds;
  return x * q + min(x, r) + b / kXcds;
}

// Tile t of tiles_m x tiles_n, taken in groups of 4 tile rows.
__device__ __forceinline__ void grouped_tile(uint32_t t, uint32_t tiles_m, uint32_t tiles_n,
                                             uint32_t& tm, uint32_t& tn) {
  constexpr uint32_t kGroup = 4;
  const uint32_t group = kGroup * tiles_n;
  const uint32_t first = (t / group) * kGroup;
  const uint32_t rows = min(tiles_m - first, kGroup);
  tm = first + (t % group) % rows;
  tn = (t % group) / rows;
}

// 16 random bits for stream positions p .. p + V - 1 (V = 4 or 8); aligned: p %
// 4 == 0. A run off a group of four takes one call more, and its words move
// down by 0 to 3 places, one bit of that number at a time. (As masks that the
// compiler cannot look through: of selects it made a branch for each number,
// calls included, and the lanes of a wave have all four: 333 x 1009 x 1111 took
// 14.7 us instead of 8.8.)
template <int V>
__device__ __forceinline__ void random_run(uint64_t p, bool aligned, uint32_t seed, uint32_t step,
                                           uint32_t (&r16)[V]) {
  static_assert(V % 4 == 0, "whole groups");
  if (aligned) {
    asr::stream_bits<0, V>(p, seed, step, r16);
    return;
  }
  constexpr int kCalls = V / 4 + 1;
  uint32_t w[4 * kCalls];
#pragma unroll
  for (int c = 0; c < kCalls; ++c) {
    const asr::Words4 f = asr::stream_call(((p >> 2) + c) & asr::kCounterMask, seed, step);
#pragma unroll
    for (int q = 0; q < 4; ++q) w[4 * c + q] = f.w[q];
  }
  uint32_t one = 0u - (static_cast<uint32_t>(p) & 1u), two = 0u - ((static_cast<uint32_t>(p) >> 1) & 1u);
  asm("" : "+v"(one), "+v"(two));
#pragma unroll
  for (int i = 0; i < V + 2; ++i) w[i] = (w[i + 1] & one) | (w[i] & ~one);
#pragma unroll
  for (int i = 0; i < V; ++i) r16[i] = ((w[i + 2] & two) | (w[i] & ~two)) & 0xFFFFu;
}

}  // namespace asr_mfma
