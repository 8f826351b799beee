// The library's own arithmetic of how paged work is cut, for the host:
// compiled and loaded by tests/test_paged_runs.py.
#include "../../exact_tiled_attention_31_b200/csrc/paged_runs.cuh"

using fa::PagedRuns;

extern "C" {
// total, units, grid, claim -> runs, waves
void runs_of_call(int total, long long units, int grid, int claim, int* out) {
  const PagedRuns r(total, units, grid, claim != 0);
  out[0] = r.runs, out[1] = r.waves;
}
int runs_begin(int total, long long units, int grid, int claim, int c) {
  return PagedRuns(total, units, grid, claim != 0).begin(c);
}
int runs_at(int total, long long units, int grid, int claim, int x) {
  return PagedRuns(total, units, grid, claim != 0).of(x);
}
int runs_place(int total, long long units, int grid, int claim, int i) {
  return PagedRuns(total, units, grid, claim != 0).place(i);
}
int unit_cost() { return fa::kUnitCost; }
int max_ranges() { return fa::kMaxRanges; }
int begin_of_range(unsigned s, unsigned tiles, unsigned n) { return fa::range_begin(s, tiles, n); }
int range_of_tile(unsigned t, unsigned tiles, unsigned n) { return fa::range_of(t, tiles, n); }
}
