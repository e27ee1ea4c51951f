// Rows sorted by expert: the arguments of the grouped kernels and the search for the rows, expert and
// tile that a wave works on, shared by the products (grouped.hip) and the bias gradient
// (grouped_bias.hip).
#pragma once
#include "mns_internal.h"

namespace mns {
namespace {

struct GroupedArgs {
  const void* A; const void* B; const void* D; void* C;
  int64_t lda, ldb, ldc;        // row pitches, elements (ldc: of C and D)
  int64_t sB, sC;               // per-expert strides of W (NT, NN) and of C, D (TN)
  const int64_t* offsets;
  int total_rows;
  int groups;
  int N, K;                     // NT, NN: output columns and reduction; TN: output rows, columns
  int tiles_n;
  int most_tiles;               // NT, NN: of rows that belong to one expert each
  int fill_rest;                // NT, NN: rows of no expert are written as zeros
  float beta;                   // TN
  int split_cap;                // most parts of a tile of the last round (k_grouped_big)
  float* partial;               // their sums, 256 KB a part
};

__device__ __forceinline__ int clamp_row(int64_t v, int lo, int hi) {
  return v < lo ? lo : v > hi ? hi : (int)v;
}

// Rows [lo, hi) of expert e.
__device__ __forceinline__ void expert_rows(const GroupedArgs& p, int e, int& lo, int& hi) {
  lo = clamp_row(p.offsets[e], 0, p.total_rows);
  hi = clamp_row(p.offsets[e + 1], lo, p.total_rows);
}

// Behind the last element of a token matrix.
template <typename T>
__device__ __forceinline__ const T* rows_end(const T* p, const GroupedArgs& a, int64_t ld, int width) {
  return p + ((int64_t)(a.total_rows - 1) * ld + width);
}

// Where a block of a forward or input-gradient call works: an expert (-1: the rows of no expert,
// to be filled with zeros), its rows [lo, hi), and the block's place among the expert's tiles.
struct Place {
  int expert, lo, hi, inside;
};

// The list of tiles that walks the experts in order, each cut into row tiles of BM rows with
// tiles_n tiles per row tile (with `rest`, the rows before the first expert and behind the last
// one come first and last). Every wave reads 64 experts' bounds at a time, one per lane, and adds
// their tile counts by a shuffle scan, so it finds its place by itself, without a launch or a
// barrier; up to 64 entries stay in registers for the next lookups.
struct Walk {
  int lo, hi;            // this lane's expert
  int incl;              // tiles up to and with it, from the start of its 64
  int total;             // tiles of all experts
};

// (least: row tiles of an expert without rows, 0 or 1)
__device__ __forceinline__ void walk_batch(const GroupedArgs& p, int BM, int tiles_n, int rest,
                                           int g0, Walk& w, int least = 0) {
  const int lane = threadIdx.x & 63;
  const int g = g0 + lane, e = g - rest;
  w.lo = w.hi = 0;
  int floor = 0;
  if (g < p.groups + 2 * rest) {
    if (e < 0) {
      w.hi = clamp_row(p.offsets[0], 0, p.total_rows);
    } else if (e >= p.groups) {
      int first;
      expert_rows(p, p.groups - 1, first, w.lo);     // from the last expert's end
      w.hi = p.total_rows;
    } else {
      expert_rows(p, e, w.lo, w.hi);
      floor = least * tiles_n;
    }
  }
  // The host refuses calls of 2^31 tiles; only offsets that overlap can add up to more (walk_start
  // then cuts the list off, find_place checks what it finds).
  w.incl = (w.hi - w.lo + (BM - 1)) / BM * tiles_n;
  if (least && w.incl < floor) w.incl = floor;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(w.incl, o);
    if (lane >= o) w.incl += up;
  }
}

// The first batch, and the total over all of them: at most most_tiles, so that overlapping offsets
// (experts that each claim all rows) do not multiply the rounds of blocks that go from tile to tile.
__device__ __forceinline__ Walk walk_start(const GroupedArgs& p, int BM, int tiles_n, int rest,
                                           int least = 0) {
  Walk w;
  const int count = p.groups + 2 * rest;
  int64_t total = 0;
  for (int g0 = (count - 1) / 64 * 64; g0 >= 0; g0 -= 64) {
    walk_batch(p, BM, tiles_n, rest, g0, w, least);
    total += (unsigned)__builtin_amdgcn_readlane(w.incl, 63);
  }
  w.total = total < p.most_tiles ? (int)total : p.most_tiles;
  return w;
}

// The place of position `lin` (false past the last tile). Everything found is read from one lane
// into scalar registers: a buffer resource computed from vector registers would make each load a
// loop over its values.
__device__ __forceinline__ bool find_place(const GroupedArgs& p, int BM, int tiles_n, int rest,
                                           Walk w, int lin, Place& at, int least = 0) {
  if (lin >= w.total) return false;
  const int count = p.groups + 2 * rest;
  int g0 = 0;
  if (count > 64) {
    for (; g0 < count; g0 += 64) {
      walk_batch(p, BM, tiles_n, rest, g0, w, least);
      const int sum = __builtin_amdgcn_readlane(w.incl, 63);
      if (lin < sum) break;
      lin -= sum;
    }
  }
  const unsigned long long over = __ballot(w.incl > lin);
  const int src = over ? __ffsll(over) - 1 : 63;
  at.inside = lin - (src ? __builtin_amdgcn_readlane(w.incl, src - 1) : 0);
  at.lo = __builtin_amdgcn_readlane(w.lo, src);
  at.hi = __builtin_amdgcn_readlane(w.hi, src);
  const int ge = g0 + src - rest;
  at.expert = ge >= 0 && ge < p.groups ? ge : -1;
  int tiles = (at.hi - at.lo + (BM - 1)) / BM * tiles_n;
  if (least && at.expert >= 0 && tiles == 0) tiles = tiles_n;
  return at.inside >= 0 && at.inside < tiles;
}

}  // namespace
}  // namespace mns
