// The tile schedule of the MLP gradient's persistent GEMMs over ragged rows: a
// table of row tiles over (problem, row group) entries and the order a CTA
// pair runs them in. The forward's GEMM (gemm_sm100.cu) keeps its own, on
// whose source its committed traffic captures are keyed.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int BM = 128;  // rows of one CTA's tile
constexpr int BK = 64;   // 64 bf16 = 128 bytes = one swizzle atom row
constexpr int kMaxEntries = 2 * kMaxLayerExperts + 2;  // (problem, group) entries of a launch

struct Sched {
  int n_entries;
  int total_tiles;
  int prob_end[2];  // tiles of problem 0 are [0, prob_end[0]), problem 1 [prob_end[0], prob_end[1])
  int tile_start[kMaxEntries + 1];
  int prob[kMaxEntries];
  int group[kMaxEntries];
  int row0[kMaxEntries];
  int row_end[kMaxEntries];
};

// The tiles one CTA pair runs, in order. Every tile of a problem costs the
// same (its K blocks), so with two problems of different K a round-robin
// deal can leave some pairs a whole long tile behind the others, which
// matters when there are few tiles per pair. Instead the longer problem's
// tiles are dealt round-robin first, and then each tile of the shorter
// problem, in order, goes to the pair that becomes free first (list
// scheduling with known durations, equal free times to the lower id). After
// the long deal the pairs below r hold one long tile more than the rest, so
// pair c's m-th short slot starts at a known time and its rank in the
// merged (start time, pair id) order, which is the short tile it gets, has a
// closed form. Tiles close in the order still run at about the same time,
// as with round-robin. Equal K (or one problem) is round-robin over the
// whole table.
struct TileSeq {
  int c, P;
  int startA, nA, startB, nB;
  int a, b, r, plo;
  int j, m;

  __device__ void init(const Sched &s, int kb0, int kb1, int n_probs, int id, int n) {
    c = id; P = n; j = id; m = 0;
    const int n0 = s.prob_end[0], n1 = n_probs > 1 ? s.prob_end[1] - s.prob_end[0] : 0;
    if (n1 == 0 || n0 == 0 || kb0 == kb1) {
      startA = 0; nA = s.total_tiles; startB = 0; nB = 0; a = b = 1;
    } else if (kb0 > kb1) {
      startA = 0; nA = n0; a = kb0; startB = n0; nB = n1; b = kb1;
    } else {
      startA = n0; nA = n1; a = kb1; startB = 0; nB = n0; b = kb0;
    }
    r = nA % P;
    plo = P - r;
  }
  // Next tile of this pair, or -1.
  __device__ int next() {
    if (j < nA) { const int t = startA + j; j += P; return t; }
    if (nB == 0) return -1;
    int pos;
    if (c >= r) {  // free at m*b (relative to the lower load after the long deal)
      const int t = m * b;
      const int hi_before = t >= a ? (t - a) / b + 1 : 0;  // slots of the r loaded pairs at times <= t
      pos = m * plo + (c - r) + r * hi_before;
    } else {       // free at a + m*b
      const int t = a + m * b;
      const int lo_before = (t + b - 1) / b;               // slots of the others at times < t
      pos = m * r + c + plo * lo_before;
    }
    ++m;
    return pos < nB ? startB + pos : -1;
  }
};

__device__ __forceinline__ int find_entry(const Sched &s, int t) {
  int lo = 0, hi = s.n_entries - 1;
  while (lo < hi) {
    int mid = (lo + hi + 1) >> 1;
    if (s.tile_start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Adds the row groups of one problem to the table (one warp): tiles of `bm`
// rows by ntn column tiles, column tiles fastest. `run` and `ne` count the
// tiles and entries so far.
__device__ __forceinline__ void sched_add(Sched &s, int pi, const int32_t *offsets, int n_groups, int64_t rows,
                                          int bm, int ntn, int32_t *status, int &run, int &ne) {
  const int lane = threadIdx.x & 31;
  for (int g0 = 0; g0 < n_groups; g0 += 32) {
    const int g = g0 + lane;
    int lo = 0, hi = 0;
    if (g < n_groups) {
      lo = offsets ? offsets[g] : 0;
      hi = offsets ? offsets[g + 1] : (int)rows;
      check_group_rows(lo, hi, rows, status);
    }
    const int tiles = hi > lo ? ((hi - lo + bm - 1) / bm) * ntn : 0;
    const int inc = warp_inclusive_scan(tiles);
    if (g < n_groups) {
      const int e = ne + lane;
      s.tile_start[e] = run + inc - tiles;
      s.prob[e] = pi;
      s.group[e] = g;
      s.row0[e] = lo;
      s.row_end[e] = hi;
    }
    run += __shfl_sync(0xffffffffu, inc, 31);
    ne += min(32, n_groups - g0);
  }
  if (lane == 0) s.prob_end[pi] = run;
}
// Ends the table of n_probs problems (the same warp).
__device__ __forceinline__ void sched_close(Sched &s, int n_probs, int run, int ne) {
  if ((threadIdx.x & 31) == 0) {
    if (n_probs < 2) s.prob_end[1] = run;
    s.n_entries = ne;
    s.total_tiles = run;
    s.tile_start[ne] = run;
  }
}

}  // namespace moe
