// fa_paged.cuh - one decode step of exact attention over a paged KV cache.
//
// As in fa_decode.cuh each sequence brings one query token per query head,
// query head h reads KV head h / G, and every row of the sequence is visible;
// but the rows of sequence b live in pages: row i is row i % page_size of
// page table[b][i / page_size] of a pool [n_pages, Hkv, page_size, D].
//
//   m = max_j s_j,  l = sum_j exp(s_j - m),  O = sum_j exp(s_j - m) v_j / l,
// over the rows j in [start, len_b), one 64-row tile at a time; parts of a
// sequence computed apart are joined by LSE = log sum exp(LSE_s),
// O = sum exp(LSE_s - LSE) O_s.
//
// Bound: HBM, 4 D bytes a row and KV head, read once.  So the work is dealt
// out by rows: the tiles of all (sequence, KV head) units, in order, are cut
// into contiguous runs (PagedRuns) from the lengths on the device: a ragged
// batch keeps every SM streaming to the end, whatever its lengths.  A unit that
// one run covers whole is finished there; the units cut by a boundary (at most
// one begins in a run) leave normalised fp32 parts that paged_merge_kernel
// joins.
//
// A CTA has one producer warp, which fills a ring of stages (a tile's K and V
// rows) by TMA, a box per page, and runs ahead of the consumers over unit
// boundaries; and four consumer warps, each with 16 rows of every tile.  Two CTAs
// share an SM: what a unit costs besides its rows (queries in, four warps' parts
// joined, a result out) is latency, and the other CTA's stream covers it.  One
// CTA of eight consumer warps with the same 192 KB in flight took 28 us instead
// of 23 for 64 sequences of up to 512 rows.  The products are formed transposed,
// S^T = K Q^T and O^T = V^T P^T, with the cache rows (then the head's columns)
// as the 16-row side of m16n8k16: a group of up to 8 query heads then pads to
// 8 instead of 16, and one ldmatrix feeds a whole operand.
#pragma once

#include "fa_decode.cuh"
#include "paged_runs.cuh"
#include "pdl.cuh"

namespace fa {

struct PagedMap {       // how rows of a sequence are found
  const int* table;     // [B, max_pages] by table_stride
  long long table_stride;
  int n_pages, page_shift, max_len;  // max_len: rows the table holds
  const int* shared;    // the pages of the first n_shared rows of every sequence; null: those of shared_row's row of the table
  int n_shared;
};

// A cut unit: its first and last run.
struct PagedCut {
  int b, kvh;         // the unit; b = -1: none
  int first, last;
};

// What the producer tells the consumers of a segment: the tiles that a run has
// of one unit.
struct PagedSeg {
  int n, key0, end, q_row;  // tiles (0: no more segments), first row, the sequence's length, first query row
  int begins, ends;         // whether they are the unit's first, last
  int run, pad;
};

struct PagedParams {
  const uint16_t* q;     // [B, Hq, D]
  const int* seq_lens;   // [B]
  PagedMap map;
  float* o_part;         // [2 * max_runs, G, D] normalised parts: 2c for the unit run c goes on with, 2c + 1 begins
  float* lse_part;       // [2 * max_runs, G] log2 of the sums
  // What is cut, by run (the unit that it began and did not finish) where
  // by_unit is 0, else by unit (the run that begins it): whichever are fewer
  // (behind shared rows always by unit, for paged_join_kernel).
  PagedCut* cuts;
  int by_unit;
  int* next_run;         // zeroed, counts the short runs taken; null: CTA c has run c alone
  void* o;               // [B, Hq, D]
  float* lse;            // [B, Hq]
  // With shared rows [0, start) in front (n_pre > 0) nothing is finished here:
  // paged_join_kernel joins the shared rows' parts with what this kernel leaves.
  // They are cut into n_pre ranges; of a sequence that ends inside one this
  // kernel takes the rows from the range's first on, and that range's part and
  // those behind it are of no rows: in the product the rows that it does not see
  // would have weight 0, and 0 times what they hold need not be 0.
  const float* pre_o;    // [n_pre, B * Hq, D]
  const float* pre_lse;  // [n_pre, B * Hq]
  float* own_o;          // [B * Hq, D] parts of units that are not cut
  float* own_lse;        // [B * Hq]
  int n_pre, start;
  int B, Hq, Hkv, G, grid, max_runs;
  float scale_log2;
};

template <int D, int NB>
struct PagedCfg {
  static constexpr int KT = 64;                        // rows per tile
  static constexpr int ROWS = 8 * NB;                  // query rows, padded
  static constexpr int GROUP = D * 16;                 // 8 rows: D / 64 swizzle atoms of 1 KB
  static constexpr int TILE = KT * D * 2;              // K or V
  static constexpr int STAGE = 2 * TILE;
  static constexpr int STAGES = (D == 128 ? 3 : 6) - (NB == 2);  // 64 to 96 KB in flight per CTA
  static constexpr int CTAS = 2;  // per SM
  static constexpr int WARPS = 4;
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int OSTR = D + 4;                   // fp32 row stride of the scratch: conflict-free
  static constexpr int SCRATCH = ROWS * (3 + OSTR);    // floats of one warp's part
  static constexpr int QTILE = ROWS * D * 2;           // queries of a segment
  static constexpr uint32_t SMEM = STAGES * (STAGE + QTILE) + 2 * SCRATCH * 4 + 1024;
  // with the static part, and 1 KB a CTA that the system takes
  static constexpr uint32_t STATIC = 1408;
  static_assert(CTAS * (SMEM + STATIC + 1024) <= 228 * 1024, "shared memory of an SM");
};

enum : uint32_t { PAGED_SITE_FULL = 0x410, PAGED_SITE_EMPTY = 0x411, PAGED_SITE_DRAIN = 0x412, PAGED_SITE_PAGE = 0x413 };

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
      : "memory");
}
// Rows of one page and KV head into shared memory.  The pool is viewed as
// (64 columns, 8 rows, D / 64 halves, 8-row groups of all heads, pages), so
// that one copy brings whole rows and leaves them as [group][half][8][128
// bytes]: 8-row groups D / 64 KB apart, whatever the page size, each half an
// atom of the 128-byte swizzle.  (Boxes of 64 columns x rows need two copies
// for D = 128; with 16-row pages the 2 KB copies bound
// decode at 4.1 to 4.6 TB/s: 64 ragged sequences 233 us instead of 179.)
__device__ __forceinline__ void load_rows(void* dst, const CUtensorMap* m, uint64_t* bar, int group, int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %2, %2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(group), "r"(page), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// a plain copy of `bytes` (a multiple of 16) into shared memory
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(p)));
}
// named barrier over `count` threads: whether `ok` holds in all of them
__device__ __forceinline__ bool named_and(uint32_t id, uint32_t count, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ uint32_t movm_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// The page that a table entry names, or n_pages (out of the pool: TMA fills
// zeros) with an argument error where it names none.
__device__ __forceinline__ int page_ok(const PagedMap& m, int id) {
  if (id >= 0 && id < m.n_pages) return id;
  record_error(DEV_ERR_ARG, PAGED_SITE_PAGE);
  return m.n_pages;
}

// Whose row of the table names the pages of the first n_shared rows: the first
// sequence that has them all (so a padding row, or a row left over from a
// sequence that has gone, is not asked), else the first of the longest, which
// has every shared row that any sequence sees.  By all lanes of a warp; the
// callers ask only where the first sequence falls short.
__device__ __forceinline__ int shared_row(const int* seq_lens, int B, int max_len, int n_shared) {
  const int lane = threadIdx.x & 31;
  int at = 0, best = -1;
  for (int b0 = 0; b0 < B && best < n_shared; b0 += 32) {
    const int b = b0 + lane, rows = b < B ? min(min(max(seq_lens[b], 0), max_len), n_shared) : -1;
    const int most = __reduce_max_sync(0xffffffffu, rows);
    if (most > best) best = most, at = b0 + __ffs(__ballot_sync(0xffffffffu, rows == most)) - 1;
  }
  return at;
}

// A row joined from parts: a lane holds VEC columns of it.
template <int VEC>
struct RowSum {
  float m = -INFINITY, w = 0.f, o[VEC];
  __device__ __forceinline__ RowSum() {
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = 0.f;
  }
};

template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, float (&x)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x, x[1] = v.y;
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&x)[VEC]) {
  if constexpr (VEC == 4)
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  else
    *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
}
// The n parts s of a row, l2(s) the log2 of each one's sum (-inf: of no rows)
// and o(s) its normalised columns: the lanes take the logarithms of 32 parts at
// once, then eight parts' columns are in flight at a time.
template <int VEC, typename L, typename O>
__device__ __forceinline__ void add_parts(RowSum<VEC>& sum, int n, int lane, L&& l2, O&& o) {
  constexpr int FLY = 8;
  for (int s0 = 0; s0 < n; s0 += 32) {
    const int k = min(32, n - s0);
    const float l = lane < k ? l2(s0 + lane) : -INFINITY;
    float x[FLY][VEC];
    auto fetch = [&](int j) {
#pragma unroll
      for (int f = 0; f < FLY; ++f) load_vec<VEC>(o(s0 + min(j + f, k - 1)) + VEC * lane, x[f]);
    };
    fetch(0);
    float mn = l;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
    mn = fmaxf(mn, sum.m);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float a = ex2(sum.m - base), w = ex2(l - base);
    float wt = w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) wt += __shfl_xor_sync(0xffffffffu, wt, d);
    sum.m = mn;
    sum.w = sum.w * a + wt;
#pragma unroll
    for (int i = 0; i < VEC; ++i) sum.o[i] *= a;
    for (int j = 0; j < k; j += FLY) {
      if (j > 0) fetch(j);
#pragma unroll
      for (int f = 0; f < FLY; ++f) {
        const float wf = j + f < k ? __shfl_sync(0xffffffffu, w, j + f) : 0.f;
        if (wf != 0.f) {  // a part of no rows holds no columns
#pragma unroll
          for (int i = 0; i < VEC; ++i) sum.o[i] += wf * x[f][i];
        }
      }
    }
  }
}
// the finished row: O in 16 bits, LSE of the sum w in natural units (a row of
// nothing: 0 and -inf; NaN scores give NaN)
template <int VEC, bool BF16>
__device__ __forceinline__ void store_row(const PagedParams& p, size_t row, int D, int lane, const RowSum<VEC>& r,
                                          float w) {
  const float inv = r.w == 0.f ? 0.f : 1.f / r.w;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + row * D + VEC * lane);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) dst[i] = pack2<BF16>(r.o[2 * i] * inv, r.o[2 * i + 1] * inv);
  if (lane == 0) p.lse[row] = w == 0.f ? -INFINITY : (r.m + __log2f(w)) * 0.69314718055994531f;
}
template <int VEC, bool BF16>
__device__ __forceinline__ void store_row(const PagedParams& p, size_t row, int D, int lane, const RowSum<VEC>& r) {
  store_row<VEC, BF16>(p, row, D, lane, r, r.w);
}

// The first row that paged_kernel takes of a sequence that ends inside the shared
// rows (that of the range it ends in), and shared_row, as calls: few sequences
// come here, and short runs are bound by what they fetch and do before their
// first load (64 sequences behind 8192 shared rows took 44.8 us instead of 44.0
// with both inline).
__device__ __noinline__ int range_start(int end, int rows, int n) {
  const int tiles = (rows + 127) / 128;
  return 128 * range_begin(range_of(end / 128, tiles, n), tiles, n);
}
__device__ __noinline__ int shared_row_call(const int* seq_lens, int B, int max_len, int n_shared) {
  return shared_row(seq_lens, B, max_len, n_shared);
}

// A place in the list of tiles: (sequence, KV head) units in order, each of
// its sequence's tiles.  A sequence without rows of its own still has one
// (empty) tile, so that its outputs are written.
struct PagedWalk {
  int b, kvh, tile, tiles, start, end;  // start, end: the rows of the sequence that are taken
};

// PRE: behind shared rows (an instance of its own, so that the short calls that
// have none are not held up by what it takes to find their place in them).
template <int D, bool BF16, int NB, bool PRE>
__global__ void __launch_bounds__(PagedCfg<D, NB>::THREADS, PagedCfg<D, NB>::CTAS)
    paged_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const PagedParams p) {
  using C = PagedCfg<D, NB>;
  constexpr int VEC = D / 32;
  extern __shared__ uint8_t dsm_raw[];
  __shared__ uint64_t full[C::STAGES], empty[C::STAGES], seg_full[C::STAGES];
  __shared__ __align__(16) PagedSeg segs[C::STAGES];
  constexpr int FIND = 32 * C::WARPS;  // threads that sum the lengths, a chunk of sequences each
  __shared__ int warp_max[C::WARPS];
  __shared__ long long warp_sum[C::WARPS];
  __shared__ uint32_t sums[FIND];  // cost of the sequences before a chunk
  __shared__ int ends[FIND];       // with a sequence to a chunk: its length
  static_assert(sizeof(full) + sizeof(empty) + sizeof(seg_full) + sizeof(segs) + sizeof(warp_max) + sizeof(warp_sum) +
                        sizeof(sums) + sizeof(ends) <= C::STATIC,
                "static shared memory");
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* queries = ring + C::STAGES * C::STAGE;
  float* scratch = reinterpret_cast<float*>(queries + C::STAGES * C::QTILE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  const int behind = PRE ? p.start : 0;  // shared rows

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::WARPS);
      mbar_init(&seg_full[s], 1);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // On their way into L2 while the kernel ahead ends: the lengths, queries and
  // first lines of the table (only cached here, read after the wait).
  {
    const long long i = (long long)c * C::THREADS + threadIdx.x;
    if (i * 64 < (long long)p.B * p.Hq * D) prefetch_l2(p.q + i * 64);
    if (i * 32 < p.B) prefetch_l2(p.seq_lens + i * 32);
    if (i < p.B && behind < p.map.max_len)
      prefetch_l2(p.map.table + i * p.map.table_stride + (behind >> p.map.page_shift));
  }
  // Behind prefix_kernel (which has itself waited for all before it) this kernel
  // runs ahead: it reads nothing of that one's, and only waits for its end.
  if (!PRE) pdl_wait();
  pdl_launch();

  // ---- the cost of the call
  const int chunk = (p.B + FIND - 1) / FIND;
  auto length_of = [&](int b) { return min(max(p.seq_lens[b], 0), p.map.max_len); };
  // tiles of a sequence that is taken from row `start` on, and that row
  auto tiles_from = [&](int start, int end) { return max(1, (end - start + C::KT - 1) / C::KT); };
  auto start_of = [&](int end) { return !PRE || end >= behind ? behind : range_start(end, behind, p.n_pre); };
  long long total = 0;
  int most = 0;  // the largest cost of a sequence
  if (p.B <= FIND) {
    // few sequences: the producer alone looks, four to a lane
    __syncthreads();
    if (warp == C::WARPS) {
      constexpr int EACH = FIND / 32;
      int n[EACH], end[EACH], mine = 0;
#pragma unroll
      for (int k = 0; k < EACH; ++k)  // all on their way before the first is used
        end[k] = EACH * lane + k < p.B ? length_of(EACH * lane + k) : 0;
#pragma unroll
      for (int k = 0; k < EACH; ++k) {
        const int b = EACH * lane + k;
        n[k] = b < p.B ? tiles_from(start_of(end[k]), end[k]) + kUnitCost : 0;
        ends[b] = end[k];
        mine += n[k];
        most = max(most, n[k]);
      }
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      total = __shfl_sync(0xffffffffu, incl, 31);
      most = __reduce_max_sync(0xffffffffu, most);
      int before = incl - mine;
#pragma unroll
      for (int k = 0; k < EACH; ++k) {
        sums[EACH * lane + k] = before;
        before += n[k];
      }
      __syncwarp();
    }
  } else {
    const int b_lo = (int)min((long long)threadIdx.x * chunk, (long long)p.B);
    const int b_hi = threadIdx.x < FIND ? min(b_lo + chunk, p.B) : b_lo;
    long long mine = 0;
    for (int b = b_lo; b < b_hi; b += 4) {
      int end[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) end[k] = length_of(min(b + k, b_hi - 1));
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (b + k < b_hi) {
          const int n = tiles_from(start_of(end[k]), end[k]) + kUnitCost;
          mine += n;
          most = max(most, n);
        }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (warp < C::WARPS && lane == 31) {
      warp_sum[warp] = incl;
      warp_max[warp] = most;
    }
    __syncthreads();
    long long before = incl - mine;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
      most = max(most, warp_max[w]);
    }
    if (threadIdx.x < FIND) sums[threadIdx.x] = (uint32_t)before;
    __syncthreads();
  }

  if (warp == C::WARPS) {
    // ---------------------------------------------------------------- producer
    total *= p.Hkv;  // below 2^31 with every length at its longest (paged_call)
    const long long units = (long long)p.B * p.Hkv;
    const PagedRuns runs((int)total, units, p.grid, p.next_run != nullptr);
    const bool whole = units <= p.grid && most <= kWholeTiles + kUnitCost;  // the same in every CTA: a unit each
    // sequence at.b's rows and tiles
    auto go_to = [&](PagedWalk& at) {
      at.end = chunk == 1 ? ends[at.b] : length_of(at.b);
      at.start = start_of(at.end);
      at.tiles = tiles_from(at.start, at.end);
    };
    const int* shared = p.map.shared;
    if (p.map.n_shared && !shared) {
      shared = p.map.table;
      if ((chunk == 1 ? ends[0] : length_of(0)) < p.map.n_shared)
        shared += shared_row_call(p.seq_lens, p.B, p.map.max_len, p.map.n_shared) * p.map.table_stride;
    }
    // The first tile of run c and the cost of what the run holds from it on.
    // Tile k of a unit sits kUnitCost + k behind the unit's start; there are at
    // most as many runs as there is cost, so no run inside a unit is without a
    // tile.
    auto enter = [&](int c, PagedWalk& at, int& t1) -> int {
      const int t0 = runs.begin(c);
      t1 = runs.begin(c + 1);
      // the last chunk that begins at or before t0 (those behind the last
      // sequence begin at the total)
      int lo = 0;
#pragma unroll
      for (int k = 0; k < FIND; k += 32) lo += __popc(__ballot_sync(0xffffffffu, (int)(sums[k + lane] * p.Hkv) <= t0));
      int first = (int)sums[lo - 1];
      at.b = min((lo - 1) * chunk, p.B - 1);
      go_to(at);
      while (t0 >= (first + at.tiles + kUnitCost) * p.Hkv && at.b < p.B - 1) {
        first += at.tiles + kUnitCost;
        ++at.b;
        go_to(at);
      }
      first *= p.Hkv;
      const int cost = at.tiles + kUnitCost;
      at.kvh = (t0 - first) / cost;
      const int off = t0 - first - at.kvh * cost;  // into the unit
      at.tile = max(0, off - kUnitCost);
      return t1 - t0 - max(0, kUnitCost - off);
    };
    PagedWalk at;
    int run = c;
    int left = 0, t1 = 0;  // cost of what is left of the run, from tile at.tile on; the run's end
    if (whole) {
      if (c < units) {
        at.b = c / p.Hkv;
        go_to(at);
        at.kvh = c % p.Hkv;
        at.tile = 0;
        left = at.tiles;
      }
    } else if (c < runs.runs) {
      run = runs.place(c);
      left = enter(run, at, t1);
    }
    const int box = min(C::KT, 1 << p.map.page_shift), boxes = C::KT / box;  // rows per box, boxes per tile
    const int batch = 32 / boxes;                                            // tiles whose pages one load finds
    const int my_box = lane >> 1, my_v = lane & 1;                           // the copy this lane issues: <= 8 of them
    uint32_t it = 0, seg = 0;  // tiles, segments so far
    bool ok = true;
    // runs that there are not hold no cut
    if (!p.by_unit)
      for (int r = c + p.grid * lane; r < p.max_runs; r += 32 * p.grid)
        if (whole || r >= runs.runs) p.cuts[r].b = -1;
    // the stage of the next tile, free.  The tiles of the last STAGES - 1
    // segments and this one are in the ring at most, so a slot for each stage
    // is enough for what is told of segments.
    auto take = [&]() {
      const uint32_t st = it % C::STAGES, round = it / C::STAGES;
      if (round > 0) ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], (round - 1) & 1, PAGED_SITE_EMPTY));
      return st;
    };
    for (;;) {
      PagedCut run_cut{-1, 0, 0, 0};
      while (left > 0 && ok) {
        const int n = min(at.tiles - at.tile, left);
        const bool begins = at.tile == 0, ends = at.tile + n == at.tiles;
        const int* row = p.map.table + at.b * p.map.table_stride;
        // table entry of this lane's (tile, box) of the batch from tile k on
        auto find = [&](int k) {
          const int i = k + lane / boxes;
          const int first = at.start + (at.tile + i) * C::KT + (lane % boxes) * box;
          return i < n && lane < batch * boxes && first < at.end
                     ? (first < p.map.n_shared ? shared : row)[first >> p.map.page_shift]
                     : -1;
        };
        int ids = find(0);
        for (int k = 0; k < n && ok; k += batch) {
          const int ids_next = find(k + batch);
          for (int i = k; i < min(k + batch, n); ++i, ++it) {
            const uint32_t st = take();
            if (!ok) break;
            const int key0 = at.start + (at.tile + i) * C::KT;
            if (i == 0 && lane == 0) {
              const uint32_t sl = seg % C::STAGES;
              const int q_row = at.b * p.Hq + at.kvh * p.G;
              segs[sl] = PagedSeg{n, key0, at.end, q_row, begins, ends, run, 0};
              mbar_expect_tx(&seg_full[sl], p.G * D * 2);
              bulk_load(queries + sl * C::QTILE, p.q + (size_t)q_row * D, p.G * D * 2, &seg_full[sl]);
            }
            // boxes that hold rows of the sequence; the rest of the stage is left as it is and masked
            const int live = at.end > key0 ? min(boxes, (at.end - key0 + box - 1) / box) : 0;
            if (lane == 0) {
              if (live) mbar_expect_tx(&full[st], live * box * D * 4);
              else mbar_arrive(&full[st]);
            }
            __syncwarp();
            const int id = __shfl_sync(0xffffffffu, ids, (i - k) * boxes + min(my_box, boxes - 1));
            if (my_box < live) {
              uint8_t* dst = ring + st * C::STAGE + my_v * C::TILE + my_box * box * D * 2;
              const int first = (key0 + my_box * box) & ((1 << p.map.page_shift) - 1);  // row in its page
              load_rows(dst, my_v ? &tm_v : &tm_k, &full[st], ((at.kvh << p.map.page_shift) + first) >> 3,
                        page_ok(p.map, id));
            }
          }
          ids = ids_next;
        }
        ++seg;
        if (begins) {
          PagedCut cut{-1, 0, 0, 0};
          if (!ends) cut = PagedCut{at.b, at.kvh, run, runs.of(t1 + (at.tiles - at.tile - n) - 1)};
          if (!p.by_unit) run_cut = cut;
          else if (lane == 0) p.cuts[(size_t)at.b * p.Hkv + at.kvh] = cut;
        }
        left -= n + kUnitCost;  // the next unit's own cost too
        if (left > 0) {
          at.tile = 0;
          if (++at.kvh == p.Hkv) {
            at.kvh = 0;
            ++at.b;
            go_to(at);
          }
        }
      }
      if (lane == 0 && !p.by_unit && !whole && c < runs.runs) p.cuts[run] = run_cut;
      if (!ok || whole || runs.waves == 1) break;
      int i = 0;
      if (lane == 0) i = p.grid + atomicAdd(p.next_run, 1);
      i = __shfl_sync(0xffffffffu, i, 0);
      if (i >= runs.runs) break;
      run = runs.place(i);
      left = enter(run, at, t1);
    }
    if (ok) {  // no more
      take();
      if (ok) {
        if (lane == 0) {
          segs[seg % C::STAGES].n = 0;
          mbar_arrive(&seg_full[seg % C::STAGES]);
        }
        ++seg;
      }
    }
    // no copy may still be on its way into shared memory when the CTA ends: the
    // newest phase of every barrier
    for (uint32_t f = it > C::STAGES ? it - C::STAGES : 0; f < it; ++f)
      mbar_wait(&full[f % C::STAGES], (f / C::STAGES) & 1, PAGED_SITE_DRAIN);
    for (uint32_t f = seg > C::STAGES ? seg - C::STAGES : 0; f < seg; ++f)
      mbar_wait(&seg_full[f % C::STAGES], (f / C::STAGES) & 1, PAGED_SITE_DRAIN);
    __syncwarp();
    if (PRE) pdl_wait();
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int r0 = 2 * (lane & 3);  // this lane's query rows 8 nb + r0, + 1; its cache rows lane / 4, + 8
  // one of two parts in the scratch: of warps w and w + 2
  float* ws = scratch + (warp & 1) * C::SCRATCH;
  uint32_t it = 0, seg = 0;
  bool ok = true;
  for (;; ++seg) {
    const uint32_t sl = seg % C::STAGES;
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&seg_full[sl], (seg / C::STAGES) & 1, PAGED_SITE_FULL));
    // all four warps go on, or none does (this also ends the reads of the
    // scratch by the segment before)
    if (!named_and(1, 32 * C::WARPS, ok)) break;
    const PagedSeg sg = segs[sl];
    const int n = sg.n;
    if (n == 0) break;
    const size_t q_row = sg.q_row;
    // Q^T as the B operand: column lane / 4 of each 8 is a query row
    uint32_t qb[NB][D / 16][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = 8 * nb + (lane >> 2);
      const uint32_t* q = reinterpret_cast<const uint32_t*>(queries + sl * C::QTILE + r * D * 2) + (lane & 3);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qb[nb][kk][0] = r < p.G ? q[8 * kk] : 0u;
        qb[nb][kk][1] = r < p.G ? q[8 * kk + 4] : 0u;
      }
    }
    float oacc[D / 16][NB][4];
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) oacc[mt][nb][0] = oacc[mt][nb][1] = oacc[mt][nb][2] = oacc[mt][nb][3] = 0.f;
    float m[NB][2], l[NB][2], lr[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) m[nb][e] = -INFINITY, l[nb][e] = lr[nb][e] = 0.f;

    for (int i = 0; i < n; ++i, ++it) {
      const uint32_t st = it % C::STAGES;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[st], (it / C::STAGES) & 1, PAGED_SITE_FULL));
      if (!ok) continue;  // error recorded: take no more tiles, but keep to the barriers below
      const int key0 = sg.key0 + i * C::KT + 16 * warp;  // this warp's 16 rows
      const int live = sg.end - key0;                              // how many of them are rows of the sequence
      if (live > 0) {
        const uint32_t ks = smem_addr(ring + st * C::STAGE), vs = ks + C::TILE;
        // S^T = K Q^T
        float s[NB][4];
        {
          float s2[NB][4];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nb][e] = s2[nb][e] = 0.f;
          const int row = 16 * warp + (lane & 15);
          const uint32_t base = ks + (row >> 3) * C::GROUP + (row & 7) * 128;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t a[4];
            const int c8 = 2 * kk + (lane >> 4);
            ldsm_x4(base + (kk >> 2) * 1024 + (((c8 & 7) ^ (row & 7)) << 4), a);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816<BF16>(kk & 1 ? s2[nb] : s[nb], a, qb[nb][kk][0], qb[nb][kk][1]);
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nb][e] += s2[nb][e];
        }
        const int ka = lane >> 2;  // this lane's rows of the 16: ka, ka + 8
        uint32_t pb[NB][2];
        float alpha[NB][2];
        bool grew = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float pv[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)  // rows past the end drop out whatever they hold
            pv[e] = ka + 8 * (e >> 1) < live ? s[nb][e] * p.scale_log2 : -INFINITY;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(pv[e], pv[e + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m[nb][e], mx);
            alpha[nb][e] = mn > m[nb][e] ? ex2(m[nb][e] - mn) : 1.f;
            grew |= mn > m[nb][e];
            m[nb][e] = mn;
            const float neg = mn == -INFINITY ? 0.f : mn;
            pv[e] = ex2(pv[e] - neg);
            pv[e + 2] = ex2(pv[e + 2] - neg);
            l[nb][e] = l[nb][e] * alpha[nb][e] + (pv[e] + pv[e + 2]);
          }
          const uint32_t p0 = pack2<BF16>(pv[0], pv[1]), p1 = pack2<BF16>(pv[2], pv[3]);
          const float2 w0 = unpack2<BF16>(p0), w1 = unpack2<BF16>(p1);
          lr[nb][0] = lr[nb][0] * alpha[nb][0] + (w0.x + w1.x);
          lr[nb][1] = lr[nb][1] * alpha[nb][1] + (w0.y + w1.y);
          pb[nb][0] = movm_trans(p0);  // P^T as the B operand: its 8 x 8 blocks, transposed
          pb[nb][1] = movm_trans(p1);
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int e = 0; e < 4; ++e) oacc[mt][nb][e] *= alpha[nb][e & 1];
        }
        // O^T += V^T P^T.  In a tile that runs past the end the rows behind it
        // may hold anything (0 * inf): they are cleared in the operand.
        uint32_t keep_lo = 0xffffffffu, keep_hi = 0xffffffffu;
        if (live < 16) {
          keep_lo = (r0 < live ? 0xffffu : 0u) | (r0 + 1 < live ? 0xffff0000u : 0u);
          keep_hi = (r0 + 8 < live ? 0xffffu : 0u) | (r0 + 9 < live ? 0xffff0000u : 0u);
        }
        const int row = 16 * warp + (lane & 7) + 8 * (lane >> 4);
        const uint32_t base = vs + (row >> 3) * C::GROUP + (row & 7) * 128;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          uint32_t a[4];
          const int c8 = 2 * mt + ((lane >> 3) & 1);
          ldsm_x4_trans(base + (mt >> 2) * 1024 + (((c8 & 7) ^ (row & 7)) << 4), a);
          a[0] &= keep_lo;
          a[1] &= keep_lo;
          a[2] &= keep_hi;
          a[3] &= keep_hi;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma16816<BF16>(oacc[mt][nb], a, pb[nb][0], pb[nb][1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---- the four warps' parts of the unit, through shared memory: warps 2 and
    // 3 hand theirs to warps 0 and 1 as they hold them, which lay the sums out
    // by rows for all four to finish
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], o);
          lr[nb][e] += __shfl_xor_sync(0xffffffffu, lr[nb][e], o);
        }
    if (warp >= 2) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
          reinterpret_cast<float4*>(ws)[(mt * NB + nb) * 32 + lane] =
              make_float4(oacc[mt][nb][0], oacc[mt][nb][1], oacc[mt][nb][2], oacc[mt][nb][3]);
        if (lane < 4) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* x = ws + C::ROWS * D + 3 * (8 * nb + r0 + e);
            x[0] = m[nb][e], x[1] = l[nb][e], x[2] = lr[nb][e];
          }
        }
      }
    }
    named_sync(1, 32 * C::WARPS);
    if (warp < 2) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float f[2], g[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float* x = ws + C::ROWS * D + 3 * (8 * nb + r0 + e);
          const float mo = x[0], mn = fmaxf(m[nb][e], mo), base = mn == -INFINITY ? 0.f : mn;
          f[e] = ex2(m[nb][e] - base);
          g[e] = ex2(mo - base);
          m[nb][e] = mn;
          l[nb][e] = f[e] * l[nb][e] + g[e] * x[1];
          lr[nb][e] = f[e] * lr[nb][e] + g[e] * x[2];
        }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          const float4 x = reinterpret_cast<const float4*>(ws)[(mt * NB + nb) * 32 + lane];
          oacc[mt][nb][0] = f[0] * oacc[mt][nb][0] + g[0] * x.x;
          oacc[mt][nb][1] = f[1] * oacc[mt][nb][1] + g[1] * x.y;
          oacc[mt][nb][2] = f[0] * oacc[mt][nb][2] + g[0] * x.z;
          oacc[mt][nb][3] = f[1] * oacc[mt][nb][3] + g[1] * x.w;
        }
      }
      __syncwarp();  // every lane has read the other warp's part
      // m[ROWS] l[ROWS] lr[ROWS] O[ROWS][OSTR]
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * nb + r0 + e;
          if (lane < 4) {
            ws[r] = m[nb][e];
            ws[C::ROWS + r] = l[nb][e];
            ws[2 * C::ROWS + r] = lr[nb][e];
          }
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            float* dst = ws + 3 * C::ROWS + r * C::OSTR + 16 * mt + (lane >> 2);
            dst[0] = oacc[mt][nb][e];
            dst[8] = oacc[mt][nb][e + 2];
          }
        }
    }
    named_sync(1, 32 * C::WARPS);
    const bool begins = sg.begins, ends = sg.ends;
    for (int r = warp; r < p.G; r += C::WARPS) {
      const float *x0 = scratch + r, *x1 = x0 + C::SCRATCH;
      const float mn = fmaxf(x0[0], x1[0]), base = mn == -INFINITY ? 0.f : mn;
      const float f = ex2(x0[0] - base), g = ex2(x1[0] - base);
      const float lt = f * x0[C::ROWS] + g * x1[C::ROWS], lrt = f * x0[2 * C::ROWS] + g * x1[2 * C::ROWS];
      // O is normalised by the sum of the weights as rounded for the product,
      // the logarithm is that of the fp32 sum
      const float inv = lrt == 0.f ? 0.f : 1.f / lrt;
      float u[VEC], v[VEC];
      load_vec<VEC>(scratch + 3 * C::ROWS + r * C::OSTR + VEC * lane, u);
      load_vec<VEC>(scratch + C::SCRATCH + 3 * C::ROWS + r * C::OSTR + VEC * lane, v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) u[i] = (f * u[i] + g * v[i]) * inv;
      if (begins && ends && !PRE) {
        RowSum<VEC> sum;
        sum.m = mn;
        sum.w = 1.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum.o[i] = u[i];
        store_row<VEC, BF16>(p, q_row + r, D, lane, sum, lt);
      } else {
        const size_t slot = (size_t)(2 * sg.run + (begins ? 1 : 0)) * p.G + r;
        const bool whole = begins && ends;
        store_vec<VEC>((whole ? p.own_o + (q_row + r) * D : p.o_part + slot * D) + VEC * lane, u);
        if (lane == 0) (whole ? p.own_lse[q_row + r] : p.lse_part[slot]) = lt == 0.f ? -INFINITY : mn + __log2f(lt);
      }
    }
  }
  if (PRE) pdl_wait();
}

// Before a call that hands out runs: the count of them.
__global__ void __launch_bounds__(32) paged_zero_kernel(int* next_run) {
  pdl_launch();  // what follows waits for this kernel, and so for all before it
  pdl_wait();
  if (threadIdx.x == 0) *next_run = 0;
}

// Whether a cut is one (an erring paged_kernel may have left anything).
__device__ __forceinline__ bool cut_ok(const PagedParams& p, const PagedCut& cut) {
  return cut.b >= 0 && cut.b < p.B && cut.kvh >= 0 && cut.kvh < p.Hkv && cut.first >= 0 && cut.last > cut.first &&
         cut.last < p.max_runs;
}

// The units that a boundary between runs cut: a block joins the parts of the
// query rows of one of p.cuts, if it is a cut, grid.y blocks those of a unit;
// with few rows to a block several warps share a row's parts.  Bound: the latency of three dependent reads.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) paged_merge_kernel(const PagedParams p) {
  constexpr int VEC = D / 32, WARPS = 8;
  __shared__ __align__(16) float s_o[WARPS][D];
  __shared__ float s_l[WARPS];
  pdl_wait();
  pdl_launch();
  const PagedCut cut = p.cuts[blockIdx.x];
  if (!cut_ok(p, cut)) return;
  const int c0 = cut.first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int each = (p.G + gridDim.y - 1) / gridDim.y, r_lo = blockIdx.y * each;
  const int rows = min(each, p.G - r_lo);  // this block's rows
  if (rows <= 0) return;
  const int split = max(1, WARPS / rows);  // warps of a row
  const int sub = warp % split, own = cut.last - c0 + 1, per = (own + split - 1) / split, s0 = min(sub * per, own);
  const size_t row0 = (size_t)cut.b * p.Hq + cut.kvh * p.G;
  for (int r = r_lo + warp / split; r < r_lo + rows; r += WARPS / split) {
    auto slot = [&](int s) { return (size_t)(s == 0 ? 2 * c0 + 1 : 2 * (c0 + s)) * p.G + r; };
    RowSum<VEC> sum;
    add_parts<VEC>(
        sum, min(per, own - s0), lane, [&](int s) { return p.lse_part[slot(s0 + s)]; },
        [&](int s) { return p.o_part + slot(s0 + s) * D; });
    if (split == 1) {
      store_row<VEC, BF16>(p, row0 + r, D, lane, sum);
      continue;
    }
    const float inv = sum.w == 0.f ? 0.f : 1.f / sum.w;
#pragma unroll
    for (int i = 0; i < VEC; ++i) sum.o[i] *= inv;
    store_vec<VEC>(&s_o[warp][VEC * lane], sum.o);
    if (lane == 0) s_l[warp] = sum.w == 0.f ? -INFINITY : sum.m + __log2f(sum.w);
  }
  if (split == 1) return;
  __syncthreads();
  if (sub || warp / split >= rows) return;
  RowSum<VEC> all;
  add_parts<VEC>(all, split, lane, [&](int s) { return s_l[warp + s]; }, [&](int s) { return s_o[warp + s]; });
  store_row<VEC, BF16>(p, row0 + r_lo + warp / split, D, lane, all);
}

// Every row's shared rows' parts and its own, whole or cut: SPLIT warps per row,
// each a share of the parts.  Bound: the n_pre + 1 fp32 parts of every row read
// once, from L2 mostly; with few rows their latency, hence the split (2048 rows
// of 17 parts took 8 us with a warp each, 14 warps to an SM).  (Joining inside
// paged_kernel put this latency into every unit's chain.)
template <int D, bool BF16, int SPLIT>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedParams p) {
  constexpr int VEC = D / 32, ROWS = 8 / SPLIT;
  __shared__ __align__(16) float s_o[8][D];
  __shared__ float s_l[8];
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % SPLIT;
  const size_t rows = (size_t)p.B * p.Hq, row = (size_t)blockIdx.x * ROWS + warp / SPLIT;
  const bool in = row < rows;
  RowSum<VEC> sum;
  if (in) {
    const int b = (int)(row / p.Hq), h = (int)(row % p.Hq), kvh = h / p.G, r = h - kvh * p.G;
    const PagedCut cut = p.cuts[(size_t)b * p.Hkv + kvh];
    const bool is_cut = cut_ok(p, cut);
    const int c0 = cut.first, n = p.n_pre + (is_cut ? cut.last - c0 + 1 : 1);
    const int per = (n + SPLIT - 1) / SPLIT, s0 = min(sub * per, n);
    auto slot = [&](int s) { return (size_t)(s == 0 ? 2 * c0 + 1 : 2 * (c0 + s)) * p.G + r; };
    add_parts<VEC>(
        sum, min(per, n - s0), lane,
        [&](int i) {
          const int s = s0 + i;
          return s < p.n_pre ? p.pre_lse[s * rows + row] : is_cut ? p.lse_part[slot(s - p.n_pre)] : p.own_lse[row];
        },
        [&](int i) {
          const int s = s0 + i;
          return s < p.n_pre ? p.pre_o + (s * rows + row) * D
                 : is_cut    ? p.o_part + slot(s - p.n_pre) * D
                             : p.own_o + row * D;
        });
    if constexpr (SPLIT == 1) {
      store_row<VEC, BF16>(p, row, D, lane, sum);
    } else {
      const float inv = sum.w == 0.f ? 0.f : 1.f / sum.w;
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum.o[i] *= inv;
      store_vec<VEC>(&s_o[warp][VEC * lane], sum.o);
      if (lane == 0) s_l[warp] = sum.w == 0.f ? -INFINITY : sum.m + __log2f(sum.w);
    }
  }
  if constexpr (SPLIT > 1) {
    __syncthreads();
    if (sub || !in) return;
    RowSum<VEC> all;
    add_parts<VEC>(all, SPLIT, lane, [&](int s) { return s_l[warp + s]; }, [&](int s) { return s_o[warp + s]; });
    store_row<VEC, BF16>(p, row, D, lane, all);
  }
}

}  // namespace fa
