// Embedding: y[t] = scale * w[ids[t]], and the table's gradient
//   dw[v] = scale * (sum of dy[t] over the tokens t with ids[t] = v),
// a row of no token 0. Sums in f32, one rounding at the end: of a run of tokens in their
// order, of a long one as partial sums of consecutive shares, joined in theirs. The order
// of the additions is fixed by ids alone, so equal calls give equal bits.
//
// The gradient's steps. (1) Tokens are sorted by id, stable: 8 bits (or fewer) of the
// id a pass. Ids outside the table and the padding id get the key `vocab` and end up
// last. (2) Sorted rows are summed, `chunk` positions by one row of lanes; a run of one
// id inside a chunk is finished there, one that crosses a chunk's border leaves
// an f32 partial sum. (3) These are joined in order. The zeros of rows without a
// token, most of a large table, are written beside (1), over the whole table, where
// one workgroup's LDS holds the sort (up to 8192 tokens); else beside (2), where flags
// tell which rows these are.
#include "rows.hpp"
#include "status.hpp"

#include <adamw_sr.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#pragma clang fp contract(off)

namespace asr_embed {

using namespace asr_rows;

constexpr int kTile = 8192;     // tokens a workgroup sorts
constexpr int kBins = 256;
constexpr uint32_t kPast = 0xFFFFFFFFu;   // key of places past the last token

struct Ids {
  const void* ids;
  uint32_t wide;    // 64-bit ids
  int64_t n, vocab, padding;   // padding: the id without a gradient, or -1
};

__device__ __forceinline__ int64_t id_at(const Ids& a, int64_t i) {
  return a.wide ? static_cast<const int64_t*>(a.ids)[i] : static_cast<int64_t>(static_cast<const int32_t*>(a.ids)[i]);
}

__device__ __forceinline__ uint32_t key_at(const Ids& a, int64_t i) {
  const int64_t id = id_at(a, i);
  return static_cast<uint32_t>(id >= 0 && id < a.vocab && id != a.padding ? id : a.vocab);
}

// ------------------------------------------------------------- forward
struct Lookup {
  Ids ids;
  const void* table;
  void* y;
  int64_t ld, dim;
  float scale;
  int32_t log_lanes;    // lanes a row: 8 columns each
  uint32_t strips, items;
};

// Rows of up to 8 << log_lanes columns side by side, U rows of a lane loaded
// together; an id outside the table gives NaN. Bound by memory: 8192 rows of 4096
// bf16, 134 MB, in 21 us, 6.3 TB/s (by one row a lane as well); f32, 268 MB, in 53 us, by
// one row 55; 16 rows 3 us, the latency of an id's load and its row's.
template <typename S, int U>
__global__ __launch_bounds__(256) void lookup(Lookup a) {
  for (uint32_t item = blockIdx.x; item < a.items; item += gridDim.x) {
    const uint32_t up = item / a.strips, strip = item - up * a.strips;
    const int64_t t0 = (static_cast<int64_t>(up) * U << (8 - a.log_lanes)) + (threadIdx.x >> a.log_lanes);
    const int64_t col = ((static_cast<int64_t>(strip) << a.log_lanes) + (threadIdx.x & ((1u << a.log_lanes) - 1))) * 8;
    int64_t id[U];
    Run<S> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + (u << (8 - a.log_lanes));
      id[u] = t < a.ids.n ? id_at(a.ids, t) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool there = id[u] >= 0 && id[u] < a.ids.vocab;
      r[u].load(static_cast<const S*>(a.table) + (there ? id[u] : 0) * a.ld + col, there ? a.dim - col : 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + (u << (8 - a.log_lanes));
      const bool there = id[u] >= 0 && id[u] < a.ids.vocab;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = there ? r[u].get(e) * a.scale : __builtin_nanf("");
      store8(static_cast<S*>(a.y) + t * a.dim + col, t < a.ids.n ? a.dim - col : 0, x);
    }
  }
}

// ---------------------------------------------------------------- sort
struct Sort {
  Ids ids;
  const uint32_t* keys_in;   // NULL: the first pass, from the ids
  const uint32_t* toks_in;
  uint32_t* keys;
  uint32_t* toks;
  uint32_t* hist;            // [digit][tile], of several tiles
  uint32_t* flags;           // one bit an id: whether it has a token
  uint32_t tiles, shift, bits, passes;
};

// Zeros for the rows without a token (flags: a bit an id that has one; NULL: for all
// rows). A workgroup's lanes store 8 columns each and end: workgroups in the order of
// memory with one store a lane (bf16) reach 7.2 TB/s on a table of 1 GB, with 2 or 4 stores
// 6.4 and 5.8, as loops over the table 4.0 to 6.2; the wait for a flag costs a sixth.
struct Fill {
  void* dw;
  const uint32_t* flags;
  int64_t vocab, dim;
  int32_t log_lanes;         // lanes a row
  uint32_t strips;           // of a row
};

template <typename S, int THREADS>
__device__ __forceinline__ void fill_rows(const Fill& a, uint32_t block) {
  const uint32_t up = block / a.strips, strip = block - up * a.strips;
  const int64_t v = static_cast<int64_t>(up) * (THREADS >> a.log_lanes) + (threadIdx.x >> a.log_lanes);
  const int32_t lanes = 1 << a.log_lanes, lane = threadIdx.x & (lanes - 1);
  if (v >= a.vocab || (a.flags && ((a.flags[v / 32] >> (v % 32)) & 1u))) return;
  S* row = static_cast<S*>(a.dw) + v * a.dim;
  const int64_t first = (static_cast<int64_t>(strip) << a.log_lanes) * 8;
  if constexpr (std::is_same_v<S, float>) {
    // 16 bytes of a lane next to its neighbour's, so that a store covers whole lines (32
    // bytes a lane in two stores: 128256 x 4096 beside the sort 965 us, so 440)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t col = first + (k * lanes + lane) * 4;
      if (col + 4 <= a.dim) {
        store_stream(reinterpret_cast<f32x4_any*>(row + col), asr::f32x4{0.0f, 0.0f, 0.0f, 0.0f});
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (col + e < a.dim) row[col + e] = 0.0f;
      }
    }
  } else {
    const float zero[8] = {};
    const int64_t col = first + lane * 8;
    store8(row + col, a.dim - col, zero);
  }
}

// The place of each of a tile's keys when the tile is ordered by one digit, stable.
// A thread of W waves holds the keys at wave * 64 R + r * 64 + lane; counts[digit][wave]. A
// round of 64 keys finds the lanes of its own digit by ballots, the first of
// them adds their number to the wave's count. Ends with counts holding the
// place of each digit's first key of each wave.
template <int W, int R>
__device__ __forceinline__ void tile_places(const uint32_t (&key)[R], uint32_t shift, uint32_t bits, uint32_t* counts,
                                            uint32_t* totals, uint32_t (&place)[R]) {
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, mask = (1u << bits) - 1u;
#pragma unroll
  for (int i = 0; i < 4; ++i) counts[i * 64 * W + threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t digit = (key[r] >> shift) & mask;
    uint64_t peers = ~uint64_t{0};
    for (uint32_t b = 0; b < bits; ++b) {
      const bool one = (digit >> b) & 1u;
      const uint64_t with = __builtin_amdgcn_ballot_w64(one);
      peers &= one ? with : ~with;
    }
    const uint32_t first = static_cast<uint32_t>(__builtin_ctzll(peers));
    uint32_t before = 0;
    if (lane == first) before = atomicAdd(&counts[digit * W + wave], static_cast<uint32_t>(__builtin_popcountll(peers)));
    before = static_cast<uint32_t>(__shfl(static_cast<int>(before), static_cast<int>(first)));
    place[r] = before + static_cast<uint32_t>(__builtin_popcountll(peers & ((uint64_t{1} << lane) - 1)));
  }
  __syncthreads();
  // exclusive sums over counts, 4 a thread
  uint32_t c[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = sum;
    sum += counts[threadIdx.x * 4 + i];
  }
  uint32_t upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t below = static_cast<uint32_t>(__shfl_up(static_cast<int>(upto), d));
    if (lane >= static_cast<uint32_t>(d)) upto += below;
  }
  if (lane == 63) totals[wave] = upto;
  __syncthreads();
  uint32_t base = upto - sum;
#pragma unroll
  for (int i = 0; i < W - 1; ++i) base += static_cast<uint32_t>(i) < wave ? totals[i] : 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) counts[threadIdx.x * 4 + i] = base + c[i];
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) place[r] += counts[((key[r] >> shift) & mask) * W + wave];
}

// Up to 64 W R tokens, all passes, by the first workgroup. The others meanwhile write
// the table's zeros, 1 GB in 152 us by workgroups of 4 waves, 160 of 8, 172 of 16:
// the sort has as few as its registers allow (32 keys a lane would be 233).
template <typename S, int W, int R>
__global__ __launch_bounds__(64 * W) void sort_and_fill(Sort a, Fill fill) {
  __shared__ uint32_t counts[kBins * W], totals[W], keys[R * 64 * W];
  __shared__ uint16_t toks[R * 64 * W];
  if (blockIdx.x > 0) {
    fill_rows<S, 64 * W>(fill, blockIdx.x - 1);
    return;
  }
  const uint32_t at = (threadIdx.x >> 6) * (64 * R) + (threadIdx.x & 63u);
  uint32_t key[R], tok[R], place[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    tok[r] = at + r * 64;
    key[r] = tok[r] < a.ids.n ? key_at(a.ids, tok[r]) : kPast;
  }
  for (uint32_t pass = 0; pass < a.passes; ++pass) {
    tile_places<W, R>(key, pass * a.bits, a.bits, counts, totals, place);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      keys[place[r]] = key[r];
      toks[place[r]] = static_cast<uint16_t>(tok[r]);
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      key[r] = keys[at + r * 64];
      tok[r] = toks[at + r * 64];
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t i = at + r * 64;
    if (i < a.ids.n) {
      a.keys[i] = key[r];
      a.toks[i] = tok[r];
    }
  }
}

// More tokens: tiles of 8192, a pass at a time. The digits of each tile are counted,
__device__ __forceinline__ uint32_t sort_key(const Sort& a, int64_t i) {
  return i >= a.ids.n ? kPast : a.keys_in ? a.keys_in[i] : key_at(a.ids, i);
}

__global__ __launch_bounds__(1024) void count_digits(Sort a) {
  __shared__ uint32_t counts[kBins];
  const int64_t start = static_cast<int64_t>(blockIdx.x) * kTile;
  const uint32_t mask = (1u << a.bits) - 1u;
  if (threadIdx.x < kBins) counts[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int64_t i = start + r * 1024 + threadIdx.x;
    if (i < a.ids.n) {
      const uint32_t key = sort_key(a, i);
      atomicAdd(&counts[(key >> a.shift) & mask], 1u);
      if (!a.keys_in && key < a.ids.vocab) atomicOr(&a.flags[key / 32], 1u << (key % 32));
    }
  }
  __syncthreads();
  if (threadIdx.x < kBins) a.hist[static_cast<int64_t>(threadIdx.x) * a.tiles + blockIdx.x] = counts[threadIdx.x];
}

// the counts of all digits and tiles become places (one workgroup),
__global__ __launch_bounds__(1024) void scan_counts(uint32_t* hist, int64_t count) {
  __shared__ uint32_t totals[16];
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  uint32_t carry = 0;
  for (int64_t start = 0; start < count; start += 4096) {
    uint32_t c[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t k = start + threadIdx.x * 4 + i;
      c[i] = sum;
      sum += k < count ? hist[k] : 0u;
    }
    uint32_t upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t below = static_cast<uint32_t>(__shfl_up(static_cast<int>(upto), d));
      if (lane >= static_cast<uint32_t>(d)) upto += below;
    }
    if (lane == 63) totals[wave] = upto;
    __syncthreads();
    uint32_t base = carry + upto - sum;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      base += static_cast<uint32_t>(i) < wave ? totals[i] : 0u;
      carry += totals[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t k = start + threadIdx.x * 4 + i;
      if (k < count) hist[k] = base + c[i];
    }
    __syncthreads();  // (totals are read)
  }
}

// and each tile's keys go there.
__global__ __launch_bounds__(1024) void scatter_digits(Sort a) {
  __shared__ uint32_t counts[kBins * 16], totals[16];
  const int64_t start = static_cast<int64_t>(blockIdx.x) * kTile;
  const uint32_t at = (threadIdx.x >> 6) * 512 + (threadIdx.x & 63u), mask = (1u << a.bits) - 1u;
  uint32_t key[8], place[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) key[r] = sort_key(a, start + at + r * 64);
  tile_places<16, 8>(key, a.shift, a.bits, counts, totals, place);
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int64_t i = start + at + r * 64;
    if (i < a.ids.n) {
      const uint32_t digit = (key[r] >> a.shift) & mask;
      const uint32_t to = a.hist[static_cast<int64_t>(digit) * a.tiles + blockIdx.x] + place[r] - counts[digit * 16];
      a.keys[to] = key[r];
      a.toks[to] = a.toks_in ? a.toks_in[i] : static_cast<uint32_t>(i);
    }
  }
}

__global__ __launch_bounds__(256) void clear_flags(uint32_t* flags, int64_t words) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < words; i += static_cast<int64_t>(gridDim.x) * 256)
    flags[i] = 0;
}

// ---------------------------------------------------------------- sums
struct Sums {
  const uint32_t* keys;
  const uint32_t* toks;
  const void* dy;
  void* dw;
  float* part;               // [chunk][head, tail][dim]: runs that cross a border
  int64_t n, vocab, dim, ld;
  float scale;
  int32_t chunk;             // sorted positions a chunk, a multiple of 16
  int32_t chunks, log_lanes;
  int32_t fold;              // positions of a first sum
  uint32_t strips, sum_blocks;
  Fill fill;
};

// A workgroup's chunks side by side, each by a row of 16 or more lanes: 16 positions'
// keys and tokens go to LDS (one wait for all), then their rows, 8 at once, which each
// lane puts into its own part of LDS: the loop over the runs then has one copy of its
// code for all of them (unrolled over rows in registers it was 22 KB, and fetching it
// was most of a small call's time). 8192 tokens of 4096 bf16, 134 MB: 21 us, 6.4 TB/s.
// FOLDS: chunks of more than `fold` positions, whose runs are summed in two levels (8 more
// registers and their additions, a few per cent of a call of few thousand tokens).
template <typename S, bool FOLDS>
__global__ __launch_bounds__(256) void sum_and_fill(Sums a) {
  constexpr int kBatch = 16, kAhead = 8, kSide = 16;
  __shared__ Run<S> rows[kAhead * 256];
  __shared__ uint32_t keys[kSide * kBatch], toks[kSide * kBatch];
  if (blockIdx.x >= a.sum_blocks) {
    fill_rows<S, 256>(a.fill, blockIdx.x - a.sum_blocks);
    return;
  }
  const int lanes = 1 << a.log_lanes, side = 256 >> a.log_lanes;
  const uint32_t up = blockIdx.x / a.strips, strip = blockIdx.x - up * a.strips;
  const int mine = threadIdx.x >> a.log_lanes;
  const int64_t c0 = static_cast<int64_t>(up) * side, c = c0 + mine;
  const int64_t col = (static_cast<int64_t>(strip) * lanes + (threadIdx.x & (lanes - 1))) * 8, count = a.dim - col;
  const int64_t i0 = c * a.chunk, i1 = min(a.n, i0 + a.chunk);
  const bool there = c < a.chunks && count > 0;
  const S* dy = static_cast<const S*>(a.dy) + col;
  const uint32_t vocab = static_cast<uint32_t>(a.vocab);
  const uint32_t before = there && i0 > 0 ? a.keys[i0 - 1] : kPast, after = there && i1 < a.n ? a.keys[i1] : kPast;
  uint32_t run = kPast;      // of acc; no key of the table before the first
  bool head = false;
  float acc[8] = {};
  [[maybe_unused]] float all[8] = {};   // of the run's positions before the last fold
  [[maybe_unused]] int32_t held = 0;
  for (int32_t start = 0; start < a.chunk; start += kBatch) {
    if constexpr (FOLDS) {
      if (held == a.fold) {
        held = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          all[e] += acc[e];
          acc[e] = 0.0f;
        }
      }
      held += kBatch;
    }
    if (start > 0) __syncthreads();   // (the last batch is read)
    if (static_cast<int>(threadIdx.x) < side * kBatch) {
      const int64_t i = (c0 + threadIdx.x / kBatch) * a.chunk + start + threadIdx.x % kBatch;
      const bool in = i < a.n && c0 + threadIdx.x / kBatch < a.chunks;
      keys[threadIdx.x] = in ? a.keys[i] : kPast;
      toks[threadIdx.x] = in ? a.toks[i] : 0;
    }
    __syncthreads();
    if (!there) continue;
    const bool last = start + kBatch >= a.chunk;
    for (int half = 0; half < kBatch; half += kAhead) {
      Run<S> row[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int at = mine * kBatch + half + k;
        row[k].load(dy + static_cast<int64_t>(toks[at]) * a.ld, keys[at] < vocab ? count : 0);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) rows[k * 256 + threadIdx.x] = row[k];
      // one turn more after the last position, for the last run
      const int turns = last && half + kAhead == kBatch ? kAhead + 1 : kAhead;
      // (keys and rows are read from LDS a turn ahead)
      uint32_t key_next = keys[mine * kBatch + half];
      Run<S> row_next = rows[threadIdx.x];
#pragma unroll 1
      for (int k = 0; k < turns; ++k) {
        const uint32_t key = k < kAhead ? key_next : kPast;
        const Run<S> r = row_next;
        if (k + 1 < kAhead) {
          key_next = keys[mine * kBatch + half + k + 1];
          row_next = rows[(k + 1) * 256 + threadIdx.x];
        }
        if (key != run) {
          if (run < vocab) {
            const bool tail = k == kAhead ? after == run : false;
            if constexpr (FOLDS) {
#pragma unroll
              for (int e = 0; e < 8; ++e) acc[e] += all[e];
            }
            if (head || tail) {
              store8(a.part + (c * 2 + (head ? 0 : 1)) * a.dim + col, count, acc);
            } else {
              float x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = acc[e] * a.scale;
              store8(static_cast<S*>(a.dw) + static_cast<int64_t>(run) * a.dim + col, count, x);
            }
          }
          run = key;
          head = start + half + k == 0 && run == before;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
          if constexpr (FOLDS) {
#pragma unroll
            for (int e = 0; e < 8; ++e) all[e] = 0.0f;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += r.get(e);   // (what the turn after the last one adds, no one stores)
      }
    }
  }
}

// The runs that cross chunks: the chunk where one begins adds its tail and the
// heads of the chunks after it, in 4 shares side by side joined in their order.
// 256 columns a workgroup, 4 a lane. Bound by the latency of its few dependent loads
// and by its 8192 workgroups, most of which have nothing to join: 13 us at 8192
// tokens of 4096. (Two or four borders a workgroup, their keys loaded at once: 14 and 16.)
template <typename S>
__global__ __launch_bounds__(256) void join_runs(Sums a) {
  __shared__ asr::f32x4 lds[256];
  const int64_t c = blockIdx.x, i0 = c * a.chunk, i1 = i0 + a.chunk;
  if (i1 >= a.n) return;
  const uint32_t run = a.keys[i1], last = a.keys[i1 - 1], before = i0 > 0 ? a.keys[i0 - 1] : kPast;
  if (run >= a.vocab || last != run || before == run) return;   // none crosses, or it began before
  // the run starts the chunks up to hi (of 1024 at most, looked at 256 at once)
  int64_t hi = c + 1;
  for (int64_t from = hi; from == hi && from < a.chunks; from += 256) {
    const int64_t k = from + threadIdx.x;
    hi += __syncthreads_count(k < a.chunks && a.keys[k * a.chunk] == run);
  }
  const int64_t heads = hi - (c + 1), share = threadIdx.x / 64, each = (heads + 3) / 4;
  const int64_t from = c + 1 + share * each, to = min(hi, from + each);
  const int64_t col = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x % 64 * 4;
  const int left = static_cast<int>(max(int64_t{0}, min(int64_t{4}, a.dim - col)));
  asr::f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](int64_t slot) {
    const float* p = a.part + slot * a.dim + col;
    if (left == 4) {
      t += *reinterpret_cast<const f32x4_any*>(p);
    } else if (left > 0) {
#pragma unroll
      for (int e = 0; e < 3; ++e) t[e] += p[min(e, left - 1)];   // (what is past the end no one stores)
    }
  };
  if (share == 0) add(c * 2 + 1);
#pragma unroll 8
  for (int64_t k = from; k < to; ++k) add(k * 2);
  lds[threadIdx.x] = t;
  __syncthreads();
  if (share > 0) return;
  S* out = static_cast<S*>(a.dw) + static_cast<int64_t>(run) * a.dim + col;
#pragma unroll
  for (int k = 1; k < 4; ++k) t += lds[k * 64 + threadIdx.x];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (e < left) {
      if constexpr (std::is_same_v<S, float>) out[e] = t[e] * a.scale;
      else out[e] = static_cast<uint16_t>(bf16_pair(t[e] * a.scale, 0.0f));
    }
  }
}

// Few tokens and a small table in one launch: workgroup g of G takes the ids g, g + G,
// ... (up to 255: frequent ids are neighbours in many vocabularies), sorts the tokens by
// them (one digit, the others the last one), and sums and writes its rows: a row
// of lanes each where an id has up to 16 tokens, all of them together (consecutive
// shares, joined in their order) where it has more. Without the launches, partial sums
// and workspace of the above.
struct Direct {
  Ids ids;
  const void* dy;
  void* dw;
  int64_t dim, ld;
  float scale;
  int32_t log_lanes;         // lanes a row
  uint32_t strips, groups;   // of a row; G
};

template <typename S>
__global__ __launch_bounds__(1024) void sum_direct(Direct a) {
  constexpr uint32_t kAhead = 8, kLong = 16;
  __shared__ uint32_t counts[kBins * 16], totals[16];
  __shared__ uint16_t toks[1024];
  __shared__ asr::f32x4 joint[2][1024];
  __shared__ uint32_t longs[1024 / kLong], long_count;
  const uint32_t up = blockIdx.x / a.strips, strip = blockIdx.x - up * a.strips;
  const uint32_t vocab = static_cast<uint32_t>(a.ids.vocab), here = (vocab - up + a.groups - 1) / a.groups;
  const uint32_t id = threadIdx.x < a.ids.n ? key_at(a.ids, threadIdx.x) : vocab;
  const uint32_t turn = id / a.groups;
  uint32_t key[1] = {id < vocab && id - turn * a.groups == up ? turn : 255u}, place[1];
  if (threadIdx.x == 0) long_count = 0;
  tile_places<16, 1>(key, 0, 8, counts, totals, place);
  toks[place[0]] = static_cast<uint16_t>(threadIdx.x);
  if (threadIdx.x < here && counts[(threadIdx.x + 1) * 16] - counts[threadIdx.x * 16] > kLong)
    longs[atomicAdd(&long_count, 1u)] = threadIdx.x;   // (in any order: each is summed by itself)
  __syncthreads();
  const uint32_t lanes = 1u << a.log_lanes, groups = 1024u >> a.log_lanes, group = threadIdx.x >> a.log_lanes;
  const int64_t col = ((static_cast<int64_t>(strip) << a.log_lanes) + (threadIdx.x & (lanes - 1))) * 8;
  const int64_t count = a.dim - col;
  const S* dy = static_cast<const S*>(a.dy) + col;
  auto sum = [&](uint32_t from, uint32_t to, float (&acc)[8]) {
    for (uint32_t i = from; i < to; i += kAhead) {
      Run<S> row[kAhead];
#pragma unroll
      for (uint32_t k = 0; k < kAhead; ++k)
        row[k].load(dy + static_cast<int64_t>(toks[min(i + k, to - 1)]) * a.ld, i + k < to ? count : 0);
#pragma unroll
      for (uint32_t k = 0; k < kAhead; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += row[k].get(e);
    }
  };
  auto finish = [&](uint32_t v, float (&acc)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= a.scale;
    store8(static_cast<S*>(a.dw) + static_cast<int64_t>(up + v * a.groups) * a.dim + col, count, acc);
  };
  for (uint32_t v = group; v < here; v += groups) {
    const uint32_t from = counts[v * 16], to = counts[(v + 1) * 16];
    if (to - from > kLong) continue;
    float acc[8] = {};
    sum(from, to, acc);
    finish(v, acc);
  }
  for (uint32_t k = 0; k < long_count; ++k) {
    const uint32_t v = longs[k], from = counts[v * 16], to = counts[(v + 1) * 16];
    const uint32_t share = (to - from + groups - 1) / groups, mine = min(to, from + group * share);
    float acc[8] = {};
    sum(mine, min(to, mine + share), acc);
    joint[0][threadIdx.x] = asr::f32x4{acc[0], acc[1], acc[2], acc[3]};
    joint[1][threadIdx.x] = asr::f32x4{acc[4], acc[5], acc[6], acc[7]};
    __syncthreads();
    if (group == 0) {
      for (uint32_t g = 1; g < groups; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += joint[e / 4][(g << a.log_lanes) + threadIdx.x][e % 4];
      finish(v, acc);
    }
    __syncthreads();
  }
}

}  // namespace asr_embed

// =========================================================== host side
namespace {

using asr_host::fail;
using asr_host::hip_fail;
using asr_host::ok;
using namespace asr_embed;

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxDim = int64_t{1} << 31;
constexpr int64_t kMaxCols = int64_t{1} << 24;
constexpr int64_t kMaxBlocks = 0xFFFFFF;          // of 256 threads in a launch of fewer than 2**32
constexpr int64_t kMaxChunks = 1024;              // of sorted tokens: what the join of one id walks
constexpr int64_t kCus = 256;                     // compute units of an MI355X

template <typename... A>
hipError_t launch(void (*f)(A...), dim3 grid, int threads, hipStream_t s, std::common_type_t<A>... args) {
  void* argv[] = {&args...};
  return hipLaunchKernel(reinterpret_cast<const void*>(f), grid, dim3(threads), argv, 0, s);
}

// log2 of the lanes of a row: 8 columns each, at most a workgroup
int32_t lanes_of(int64_t dim, int32_t least = 0) {
  int32_t l = least;
  while (l < 8 && (int64_t{8} << l) < dim) ++l;
  return l;
}

struct Cut {
  int32_t chunk, chunks;
  int64_t tiles;
  explicit Cut(int64_t n) {
    // 16 positions a chunk at least: fewer leave more partial sums than rows are saved
    int64_t c = 16;
    while ((n + c - 1) / c > kMaxChunks) c *= 2;
    chunk = static_cast<int32_t>(c);
    chunks = static_cast<int32_t>((n + c - 1) / c);
    tiles = (n + kTile - 1) / kTile;
  }
};

// The buffers of the gradient in its workspace, each on a 256-byte boundary.
struct Buffers {
  char* base;
  int64_t at = 0;
  uint32_t *keys[2], *toks[2], *hist;
  uint32_t* flags;
  float* part;
  template <typename P>
  P* take(int64_t count) {
    P* p = reinterpret_cast<P*>(base + at);
    at += (count * static_cast<int64_t>(sizeof(P)) + 255) / 256 * 256;
    return p;
  }
  Buffers(void* ws, int64_t n, int64_t vocab, int64_t dim) : base(static_cast<char*>(ws)) {
    const Cut cut(n);
    const bool several = cut.tiles > 1;
    keys[0] = take<uint32_t>(n);
    toks[0] = take<uint32_t>(n);
    keys[1] = take<uint32_t>(several ? n : 0);
    toks[1] = take<uint32_t>(several ? n : 0);
    hist = take<uint32_t>(several ? kBins * cut.tiles : 0);
    flags = take<uint32_t>(several ? (vocab + 31) / 32 : 0);
    part = take<float>(static_cast<int64_t>(cut.chunks) * 2 * dim);
  }
};

// Few tokens (one a thread) and a small table: one launch. (us, that and the launches above,
// bf16: 16 tokens, 100 x 64: 5.0 and 11; 777, 1009 x 333: 6.7 and 22; 1024 of one id, 1009
// x 512: 15.7 and 21; 1024, 16000 x 1024: 13.6 and 17.7; 256, 100000 x 64: 11 and 17.
// Beyond, the order of the table's zeros counts more.)
bool direct(int64_t n, int64_t vocab, int64_t dim) {
  return n > 0 && n <= 1024 && vocab <= int64_t{1} << 17 && vocab * dim <= int64_t{1} << 24;
}

int check_table(int64_t n, int64_t vocab, int64_t dim, int32_t dtype) {
  if (n < 0 || n >= kMaxDim || vocab < 0 || vocab >= kMaxDim)
    return fail(ASR_EINVAL, "embedding: tokens and vocabulary must be in [0, 2**31)");
  if (dim < 0 || dim > kMaxCols) return fail(ASR_EINVAL, "embedding: dim must be in [0, 2**24]");
  if (dtype != ASR_F32 && dtype != ASR_BF16) return fail(ASR_EDTYPE, "embedding: unknown dtype");
  return ASR_OK;
}

Sort sort_args(const Ids& ids, const Buffers& b) {
  Sort a{};
  a.ids = ids;
  uint32_t bits = 1;
  while ((ids.vocab >> bits) != 0) ++bits;   // of the key `vocab`, the largest
  a.passes = (bits + 7) / 8;
  a.bits = (bits + a.passes - 1) / a.passes;
  a.keys = b.keys[0];
  a.toks = b.toks[0];
  a.flags = b.flags;
  return a;
}

// Workgroups that write a table's rows of no token
int64_t fill_blocks(const Fill& f, int threads) {
  const int64_t side = threads >> f.log_lanes;
  return (f.vocab + side - 1) / side * f.strips;
}

template <typename S>
hipError_t sort_one_tile(const Sort& a, const Fill& fill, hipStream_t s) {
  const auto one = [&](auto* f, int threads) {
    return launch(f, dim3(static_cast<uint32_t>(1 + fill_blocks(fill, threads))), threads, s, a, fill);
  };
  if (a.ids.n <= 1024) return one(&sort_and_fill<S, 4, 4>, 256);
  if (a.ids.n <= 2048) return one(&sort_and_fill<S, 4, 8>, 256);
  if (a.ids.n <= 4096) return one(&sort_and_fill<S, 4, 16>, 256);
  return one(&sort_and_fill<S, 8, 16>, 512);
}

// Several tiles: a ends with the sorted keys and tokens.
hipError_t sort_tiles(Sort& a, const Buffers& b, const Cut& cut, hipStream_t s) {
  a.hist = b.hist;
  a.tiles = static_cast<uint32_t>(cut.tiles);
  const int64_t words = (a.ids.vocab + 31) / 32;
  hipError_t e = launch(&clear_flags, dim3(static_cast<uint32_t>(std::min<int64_t>((words + 255) / 256, 1024))), 256, s,
                        b.flags, words);
  for (uint32_t pass = 0; pass < a.passes && e == hipSuccess; ++pass) {
    a.shift = pass * a.bits;
    a.keys = b.keys[pass % 2];
    a.toks = b.toks[pass % 2];
    e = launch(&count_digits, dim3(a.tiles), 1024, s, a);
    if (e == hipSuccess) e = launch(&scan_counts, dim3(1), 1024, s, b.hist, static_cast<int64_t>(kBins) * cut.tiles);
    if (e == hipSuccess) e = launch(&scatter_digits, dim3(a.tiles), 1024, s, a);
    a.keys_in = a.keys;
    a.toks_in = a.toks;
  }
  return e;
}

}  // namespace

extern "C" {

int asr_embedding_forward(const void* ids, int32_t ids_64, int64_t n, const void* table, int32_t dtype, int64_t ld,
                          int64_t vocab, int64_t dim, double scale, void* y, void* stream) {
  if (int rc = check_table(n, vocab, dim, dtype)) return rc;
  if (!std::isfinite(static_cast<float>(scale))) return fail(ASR_EINVAL, "embedding: scale must be finite in binary32");
  if (n == 0 || dim == 0) return ok();
  if (!ids || !y || (vocab > 0 && !table)) return fail(ASR_EINVAL, "embedding: null pointer");
  if (ld < dim) return fail(ASR_EINVAL, "embedding: a row stride is below the row's length");
  const uintptr_t size = dtype == ASR_F32 ? 4 : 2;
  if (!aligned_to(ids, ids_64 ? 8 : 4) || !aligned_to(table, size) || !aligned_to(y, size))
    return fail(ASR_EALIGN, "embedding: a pointer is not aligned to its elements");
  Lookup a{};
  a.ids = Ids{ids, ids_64 ? 1u : 0u, n, vocab, -1};
  a.table = table;
  a.y = y;
  a.ld = ld;
  a.dim = dim;
  a.scale = static_cast<float>(scale);
  a.log_lanes = lanes_of(dim);
  a.strips = static_cast<uint32_t>((dim + (int64_t{8} << a.log_lanes) - 1) / (int64_t{8} << a.log_lanes));
  // 4 rows of a lane, as long as that leaves enough workgroups for the chip (4 of them a
  // compute unit; 512 to 2048 rows of 4096 take 3.5 to 5.1 us either way)
  const int64_t rows = 256 >> a.log_lanes;
  const bool many = (n + 4 * rows - 1) / (4 * rows) * a.strips >= 4 * kCus;
  const int64_t up = (n + (many ? 4 : 1) * rows - 1) / ((many ? 4 : 1) * rows);
  if (up * a.strips >= kMaxDim) return fail(ASR_EINVAL, "embedding: too much for one call");
  a.items = static_cast<uint32_t>(up * a.strips);
  const uint32_t grid = std::min(a.items, 1u << 22);
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto* f = dtype == ASR_F32 ? (many ? &lookup<float, 4> : &lookup<float, 1>)
                             : (many ? &lookup<uint16_t, 4> : &lookup<uint16_t, 1>);
  const hipError_t e = launch(f, dim3(grid), 256, s, a);
  return e == hipSuccess ? ok() : hip_fail(e, "embedding launch");
}

size_t asr_embedding_backward_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
  if (n <= 0 || n >= kMaxDim || vocab <= 0 || vocab >= kMaxDim || dim <= 0 || dim > kMaxCols) return 0;
  return direct(n, vocab, dim) ? 0 : static_cast<size_t>(Buffers(nullptr, n, vocab, dim).at);
}

int asr_embedding_backward(const void* ids, int32_t ids_64, int64_t n, const void* dy, int64_t ld_dy, int32_t dtype,
                           int64_t vocab, int64_t dim, double scale, int64_t padding_idx, void* dtable,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_table(n, vocab, dim, dtype)) return rc;
  if (!std::isfinite(static_cast<float>(scale))) return fail(ASR_EINVAL, "embedding: scale must be finite in binary32");
  if (padding_idx < -1 || padding_idx >= std::max<int64_t>(vocab, 1))
    return fail(ASR_EINVAL, "embedding: padding_idx must be an id of the table, or -1");
  if (vocab == 0 || dim == 0) return ok();
  const int64_t size = dtype == ASR_F32 ? 4 : 2;
  Sums a{};
  a.log_lanes = lanes_of(dim, 4);
  a.strips = static_cast<uint32_t>((dim + (int64_t{8} << a.log_lanes) - 1) / (int64_t{8} << a.log_lanes));
  const int64_t side = 256 >> a.log_lanes;
  a.fill = Fill{dtable, nullptr, vocab, dim, a.log_lanes, a.strips};
  const int64_t filling = fill_blocks(a.fill, 256), summing = n > 0 ? (Cut(n).chunks + side - 1) / side * a.strips : 0;
  const int64_t strips4 = (dim + 255) / 256;   // of 256 columns: the join's
  if (filling + summing > kMaxBlocks || (n > 0 && Cut(n).chunks * strips4 > kMaxBlocks))
    return fail(ASR_EINVAL, "embedding: the table is too large for one call");
  if (!dtable || (n > 0 && (!ids || !dy))) return fail(ASR_EINVAL, "embedding: null pointer");
  if (n > 0 && ld_dy < dim) return fail(ASR_EINVAL, "embedding: a row stride is below the row's length");
  if (!aligned_to(ids, ids_64 ? 8 : 4) || !aligned_to(dy, size) || !aligned_to(dtable, size))
    return fail(ASR_EALIGN, "embedding: a pointer is not aligned to its elements");
  const bool small = direct(n, vocab, dim);
  if (n > 0 && !small && (!workspace || !aligned_to(workspace, 256) ||
                workspace_bytes < asr_embedding_backward_workspace_bytes(n, vocab, dim)))
    return fail(ASR_EWORKSPACE, "embedding: workspace NULL, too small or not 256-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (small) {
    Direct d{Ids{ids, ids_64 ? 1u : 0u, n, vocab, padding_idx}, dy, dtable, dim, ld_dy, static_cast<float>(scale),
             a.log_lanes, a.strips, 1};
    // about 512 workgroups, as long as every row of lanes has an id and none more than 255
    const int64_t rows = 1024 >> a.log_lanes;
    d.groups = static_cast<uint32_t>(std::max(std::min<int64_t>((vocab + rows - 1) / rows, std::max<int64_t>(512 / a.strips, 1)),
                                              (vocab + 254) / 255));
    const dim3 grid(d.groups * a.strips);
    const hipError_t e = launch(dtype == ASR_F32 ? &sum_direct<float> : &sum_direct<uint16_t>, grid, 1024, s, d);
    return e == hipSuccess ? ok() : hip_fail(e, "embedding launch");
  }
  a.dy = dy;
  a.dw = dtable;
  a.n = n;
  a.vocab = vocab;
  a.dim = dim;
  a.ld = ld_dy;
  a.scale = static_cast<float>(scale);
  a.sum_blocks = static_cast<uint32_t>(summing);
  hipError_t e = hipSuccess;
  bool filled = false;
  if (n > 0) {
    const Buffers b(workspace, n, vocab, dim);
    const Cut cut(n);
    a.part = b.part;
    a.chunk = cut.chunk;
    a.chunks = cut.chunks;
    a.fold = fold_of(cut.chunk);
    Sort sort = sort_args(Ids{ids, ids_64 ? 1u : 0u, n, vocab, padding_idx}, b);
    if (cut.tiles > 1) {
      e = sort_tiles(sort, b, cut, s);
    } else {
      // Zeros over the whole table beside the sort, those of rows with tokens too (8192
      // tokens; beside it and after it by flags: 128256 x 4096 bf16 183 us and 216, f32 440
      // and 430, 8000 x 4096 bf16 58 and 61, 30000 x 1024 f32 50 and 64).
      e = dtype == ASR_F32 ? sort_one_tile<float>(sort, a.fill, s) : sort_one_tile<uint16_t>(sort, a.fill, s);
      filled = true;
    }
    a.fill.flags = b.flags;
    a.keys = sort.keys;
    a.toks = sort.toks;
  }
  if (e == hipSuccess) {
    const bool folds = a.chunk > a.fold;
    auto* f = dtype == ASR_F32 ? (folds ? &sum_and_fill<float, true> : &sum_and_fill<float, false>)
                               : (folds ? &sum_and_fill<uint16_t, true> : &sum_and_fill<uint16_t, false>);
    e = launch(f, dim3(static_cast<uint32_t>(summing + (filled ? 0 : filling))), 256, s, a);
  }
  if (e == hipSuccess && a.chunks > 1)
    e = launch(dtype == ASR_F32 ? &join_runs<float> : &join_runs<uint16_t>,
               dim3(static_cast<uint32_t>(a.chunks), static_cast<uint32_t>(strips4)), 256, s, a);
  return e == hipSuccess ? ok() : hip_fail(e, "embedding launch");
}

}  // extern "C"
