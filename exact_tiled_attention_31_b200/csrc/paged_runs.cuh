// paged_runs.cuh - how the work of paged_kernel and prefix_kernel is cut: the
// runs of a call's tiles and the ranges of its shared rows.  Plain arithmetic,
// without anything of CUDA's, so that it also compiles for the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FA_RUNS_FN __host__ __device__ __forceinline__
#else
#define FA_RUNS_FN inline
#endif

namespace fa {

// What beginning and ending a unit costs, in tiles.  Runs are cut at equal
// cost, so that a CTA with many short sequences is not the last; the cost lies
// in front of the unit's first tile.
constexpr int kUnitCost = 2;
// Where every unit is at most this many tiles and there is a CTA for each, no
// unit is cut: a CTA takes eight tiles in less time than joining parts costs.
constexpr int kWholeTiles = 8;
// Below this cost a run is not worth a CTA and a part.
constexpr int kMinRun = 4;
// From this many tiles a CTA on runs are handed out.
constexpr long long kClaimTiles = 48;

// The cost Hkv * sum_b (tiles(b) + kUnitCost) of a call, cut into runs.  CTAs do
// not stream equally fast: on B200 whole groups of SMs get up to 8 % less than
// the mean, others 8 % more (32 x 8 caches of 8192 rows in equal runs: the
// first SM done after 135 us, the last after 160, 149 on average).  So where
// there is enough to do, each of S equal stretches of the list is one long run
// and some short ones, in order; CTA c begins with the long run of stretch c,
// and then whoever comes first takes the next of the short ones, all second
// ones of the stretches before the third ones.  Which CTA takes a run does not
// change the runs, so results do not depend on it.  (With the short runs at the
// end of the list its last units came in up to a hundred parts, and joining
// them cost more than the balance gained.)
struct PagedRuns {
  int total;               // below 2^31: what begin() forms in 32 bits
  int S, runs, waves;      // CTAs; runs in all; runs of a stretch (1: `runs` equal ones)
  uint32_t quot, rest;     // one run a stretch: total = quot * runs + rest
  uint64_t step;           // several: cost of a 256th of a stretch, in 65536ths
  static constexpr int kMaxWaves = 3;
  static FA_RUNS_FN long long least(long long a, long long b) { return a < b ? a : b; }
  // where in a stretch its runs begin, in 256ths: they are 208, 32 and 16 long
  static FA_RUNS_FN int share(int w) { return w == 0 ? 0 : w == 1 ? 208 : 240; }
  FA_RUNS_FN PagedRuns(int total, long long units, int grid, bool claim)
      : total(total), S(grid), runs((int)least(grid, units > total / kMinRun ? units : total / kMinRun)), waves(1),
        step(0) {
    // Below 48 tiles a CTA (the shortest run then three) what a run costs is
    // what the balance gains: 8 x 8 caches of 8192 rows, 28 tiles, took 50.1 us
    // with two runs a stretch and 49.8 with one; 64 ragged ones, 62 tiles, 162.8
    // us with these three and 173.2 with one.
    const uint32_t per = (uint32_t)total / (uint32_t)S;
    if (claim && per >= kClaimTiles) {
      waves = kMaxWaves;
      runs = waves * S;
      step = (uint64_t)per * 256 + ((uint32_t)total - per * S) * 256u / (uint32_t)S;
    }
    quot = (uint32_t)total / (uint32_t)runs;
    rest = (uint32_t)total - quot * runs;
  }
  // place in the list of the i-th run to be taken
  FA_RUNS_FN int place(int i) const { return waves == 1 ? i : (i % S) * waves + i / S; }
  // cost in front of run c (by place)
  FA_RUNS_FN int begin(int c) const {
    if (waves == 1) return c * quot + c * rest / (uint32_t)runs;
    const int g = c / kMaxWaves, w = c - g * kMaxWaves;
    return c >= runs ? total : (int)(((uint32_t)(g * 256 + share(w)) * step) >> 16);
  }
  // the run that cost x lies in: the largest c with begin(c) <= x
  FA_RUNS_FN int of(int x) const {
    const int n = waves == 1 ? runs : S;
    int g = (int)least(n - 1, (int)((float)x * ((float)n / (float)total)));  // near
    while (g > 0 && begin(g * waves) > x) --g;
    while (g + 1 < n && begin((g + 1) * waves) <= x) ++g;
    int w = waves - 1;
    while (w > 0 && begin(g * waves + w) > x) --w;
    return g * waves + w;
  }
};

// The first 128-row tile of range s of the n that `tiles` of them are cut into,
// and the range that tile t lies in (n <= kMaxRanges and rows <= 2^30: 32 bits do).
constexpr int kMaxRanges = 64;
FA_RUNS_FN constexpr int range_begin(uint32_t s, uint32_t tiles, uint32_t n) { return (int)(s * tiles / n); }
FA_RUNS_FN constexpr int range_of(uint32_t t, uint32_t tiles, uint32_t n) { return (int)(((t + 1) * n - 1) / tiles); }

}  // namespace fa
