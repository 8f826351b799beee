// fa_paged.cu - host side of the rotary-position, paged-cache and
// shared-prefix entry points of include/fa.h: argument checks, tensor maps,
// launch configuration.  The kernels are in fa_rope.cuh, fa_paged.cuh and
// fa_prefix.cuh.
#include <algorithm>
#include <utility>

#include "fa_host.cuh"
#include "fa_prefix.cuh"
#include "fa_rope.cuh"

namespace {

// ---------------------------------------------------------------- shared checks
bool rows_ok(const fa_rows* r) {
  return r && r->data && aligned16(r->data) && r->batch_stride >= 0 && r->head_stride >= 0 && r->row_stride >= 0 &&
         !(r->batch_stride & 7) && !(r->head_stride & 7) && !(r->row_stride & 7) && r->heads > 0;
}
bool ints_ok(const int* p) { return !(reinterpret_cast<uintptr_t>(p) & 3u); }

fa::RowsIn rows_in(const fa_rows& r) {
  return {static_cast<const uint16_t*>(r.data), r.batch_stride, r.head_stride, r.row_stride};
}
fa::RowsOut rows_out(const fa_rows& r) {
  return {static_cast<uint16_t*>(r.data), r.batch_stride, r.head_stride, r.row_stride};
}

// ---------------------------------------------------------------- overlaps
// What a call reads or writes of a strided stack: `run` contiguous 16-bit
// values at `at` plus every sum of index * stride, strides falling.
struct Stack {
  uintptr_t at;
  long long run;
  int dims;
  bool repeats;  // an index that moves nothing (a broadcast)
  struct {
    long long n, stride, inner;  // inner: from the first to behind the last value of one index
  } dim[3];
  long long extent() const { return dims ? dim[0].inner + (dim[0].n - 1) * dim[0].stride : run; }
};

Stack stack_of(const void* data, long long run, std::initializer_list<std::pair<long long, long long>> dims) {
  Stack s = {reinterpret_cast<uintptr_t>(data), run, 0, false, {}};
  for (const auto& [n, stride] : dims) {
    if (n > 1 && stride == 0) s.repeats = true;
    if (n <= 1 || stride == 0) continue;
    int i = s.dims++;
    for (; i > 0 && s.dim[i - 1].stride < stride; --i) s.dim[i] = s.dim[i - 1];
    s.dim[i] = {n, stride, 0};
  }
  long long inner = run;
  for (int i = s.dims - 1; i >= 0; --i) {
    s.dim[i].inner = inner;
    inner += (s.dim[i].n - 1) * s.dim[i].stride;
  }
  return s;
}

// Whether index * stride stays within 2^46 values, 2^47 bytes: no device's
// addresses go further, and sums of it do not overflow.
bool within(long long n, long long stride) { return n <= 1 || stride <= (1LL << 46) / (n - 1); }
bool within(const fa_rows& r, int B, int S) {
  return within(B, r.batch_stride) && within(r.heads, r.head_stride) && within(S, r.row_stride);
}

long long floor_div(long long a, long long b) { return a / b - (a % b != 0 && a < 0); }

// Whether some run of a (from dimension i on, delta values behind b's start)
// meets one of b (from dimension j on); of one stack with itself (self) only
// where the indices differ.  Where the outer strides are equal only the
// difference of the two indices counts, and of nested strides (views of one
// buffer) only a few can bring the inner parts together; else the indices of
// one of them are tried.  `tries` bounds that: what has used it up counts as
// overlapping.
bool meet(const Stack& a, int i, const Stack& b, int j, long long delta, bool self, int& tries) {
  const long long ea = i < a.dims ? a.dim[i].inner + (a.dim[i].n - 1) * a.dim[i].stride : a.run;
  const long long eb = j < b.dims ? b.dim[j].inner + (b.dim[j].n - 1) * b.dim[j].stride : b.run;
  if (delta >= eb || -delta >= ea) return false;
  if (--tries < 0) return true;
  if (i == a.dims && j == b.dims) return !self;
  if (i < a.dims && j < b.dims && a.dim[i].stride == b.dim[j].stride) {
    const auto &da = a.dim[i], &db = b.dim[j];
    // -inner of a < delta + d * stride < inner of b
    const long long lo = std::max(-(db.n - 1), floor_div(-da.inner - delta, da.stride) + 1);
    const long long hi = std::min(da.n - 1, floor_div(db.inner - delta - 1, da.stride));
    for (long long d = lo; d <= hi; ++d)
      if (meet(a, i + 1, b, j + 1, delta + d * da.stride, self && d == 0, tries)) return true;
    return false;
  }
  if (j == b.dims || (i < a.dims && a.dim[i].stride > b.dim[j].stride)) {
    const auto& da = a.dim[i];
    const long long lo = std::max(0LL, floor_div(-da.inner - delta, da.stride) + 1);
    const long long hi = std::min(da.n - 1, floor_div(eb - delta - 1, da.stride));
    for (long long d = lo; d <= hi; ++d)
      if (meet(a, i + 1, b, j, delta + d * da.stride, self, tries)) return true;
    return false;
  }
  const auto& db = b.dim[j];
  const long long lo = std::max(0LL, floor_div(delta - db.inner, db.stride) + 1);
  const long long hi = std::min(db.n - 1, floor_div(delta + ea - 1, db.stride));
  for (long long d = lo; d <= hi; ++d)
    if (meet(a, i, b, j + 1, delta - d * db.stride, self, tries)) return true;
  return false;
}

bool overlap(const Stack& a, const Stack& b) {
  const long long ea = a.extent(), eb = b.extent();
  if (a.at >= b.at + 2 * (unsigned long long)eb || b.at >= a.at + 2 * (unsigned long long)ea) return false;
  int tries = 1 << 16;
  return meet(a, 0, b, 0, ((long long)a.at - (long long)b.at) / 2, false, tries);
}
// whether two indices of an output lead to one place
bool overlaps_itself(const Stack& a) {
  if (a.repeats) return true;
  bool nested = true;
  for (int i = 0; i < a.dims; ++i) nested &= a.dim[i].stride >= a.dim[i].inner;
  if (nested) return false;
  int tries = 1 << 16;
  return meet(a, 0, a, 0, 0, true, tries);
}
// the same rows, index by index: an output that is its input, in place
bool in_place(const fa_rows& y, const fa_rows& x, int B, int S) {
  return y.data == x.data && (B == 1 || y.batch_stride == x.batch_stride) &&
         (y.heads == 1 || y.head_stride == x.head_stride) && (S == 1 || y.row_stride == x.row_stride);
}
// [batch, heads, rows] of D values
Stack stack_of(const fa_rows& r, int B, int S, int D) {
  return stack_of(r.data, D, {{B, r.batch_stride}, {r.heads, r.head_stride}, {S, r.row_stride}});
}

// Pages: a pool of n_pages x heads x page_size x D, 16-byte aligned; a table.
fa_status pages_check(const fa_pages* pg, int D) {
  if (!pg || pg->n_pages < 0 || pg->max_pages < 0 || pg->heads <= 0 || pg->page_size <= 0) return FA_ERR_INVALID_ARG;
  if (pg->page_size < 16 || pg->page_size > 4096 || (pg->page_size & (pg->page_size - 1))) return FA_ERR_UNSUPPORTED;
  if (!ptrs_ok({pg->k, pg->v}) || !pg->block_table || !ints_ok(pg->block_table)) return FA_ERR_INVALID_ARG;
  if (pg->n_pages == 0 || pg->max_pages == 0) return FA_ERR_INVALID_ARG;
  if ((pg->page_stride & 7) || pg->page_stride < (long long)pg->heads * pg->page_size * D) return FA_ERR_INVALID_ARG;
  if (pg->table_stride < 0) return FA_ERR_INVALID_ARG;
  if ((long long)pg->max_pages * pg->page_size > (1LL << 30)) return FA_ERR_UNSUPPORTED;
  // tensor-map limits: strides below 2^40 bytes, coordinates below 2^31
  if (pg->page_stride >= (1LL << 39) || (long long)pg->heads * pg->page_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// A launch that may begin before the kernel ahead of it on the stream ends;
// every kernel here waits (pdl_wait) before it touches memory.
template <typename... A>
fa_status launch_after(void (*kern)(A...), dim3 grid, int block, uint32_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e == cudaSuccess) g_launches.fetch_add(1);
  return from_cuda(e);
}

// ---------------------------------------------------------------- rotary positions
// Blocks of `rows` tokens and `groups` groups of heads, the group's index first
// where the heads of a token are nearer than its neighbours (and the tokens'
// fits second).
template <int D>
dim3 rope_grid(long long rows, int groups, long long head_stride, long long row_stride, bool& heads_near) {
  constexpr int TOKENS = fa::kRopeThreads / (D / 16);
  const unsigned tiles = (unsigned)((rows + TOKENS - 1) / TOKENS);
  heads_near = head_stride < row_stride && tiles <= 65535;
  return heads_near ? dim3(groups, tiles) : dim3(tiles, groups);
}

template <int D, bool BF16>
fa_status launch_rope(fa::RopeParams& p, bool inter, bool fill, cudaStream_t st) {
  const dim3 grid = rope_grid<D>((long long)p.B * p.S, fa::rope_groups(p.heads[0]) + fa::rope_groups(p.heads[1]), p.x[0].head, p.x[0].row, p.heads_near);
  const auto kern = fill ? (inter ? fa::rope_kernel<D, BF16, true, true> : fa::rope_kernel<D, BF16, false, true>)
                         : (inter ? fa::rope_kernel<D, BF16, true, false> : fa::rope_kernel<D, BF16, false, false>);
  return launch_after(kern, grid, fa::kRopeThreads, 0, st, p);
}

template <int D, bool BF16>
fa_status launch_append(fa::AppendParams& p, bool inter, bool fill, cudaStream_t st) {
  const dim3 grid = rope_grid<D>(p.T, fa::rope_groups(p.Hq) + 2 * fa::rope_groups(p.Hkv), p.k.head, p.k.row, p.heads_near);
  const auto kern = fill ? (inter ? fa::append_kernel<D, BF16, true, true> : fa::append_kernel<D, BF16, false, true>)
                         : (inter ? fa::append_kernel<D, BF16, true, false> : fa::append_kernel<D, BF16, false, false>);
  return launch_after(kern, grid, fa::kRopeThreads, 0, st, p);
}

bool rot_ok(int rot_dim, int D) { return rot_dim >= 16 && rot_dim <= D && rot_dim % 16 == 0; }

// fill: rows of no sequence become zero
fa_status rope_call(const fa_rows* x, const fa_rows* y, int n, const double* freqs, int rot_dim, int interleaved,
                    float amp, int backward, const int* positions, long long positions_stride, const int* cu_seqlens,
                    int nseq, int B, int S, int D, fa_dtype dt, void* stream, bool fill) {
  if (B < 0 || S < 0 || nseq < 0 || positions_stride < 0 || n < 1 || n > 2 || !x || !y) return FA_ERR_INVALID_ARG;
  if (dt != FA_BF16 && dt != FA_FP16) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(amp)) return FA_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || !rot_ok(rot_dim, D)) return FA_ERR_UNSUPPORTED;
  if (cu_seqlens && B > 1) return FA_ERR_INVALID_ARG;
  if (B == 0 || S == 0 || (cu_seqlens && nseq == 0 && !fill)) return FA_OK;
  if (!freqs || (reinterpret_cast<uintptr_t>(freqs) & 7u) || !ints_ok(positions) || !ints_ok(cu_seqlens))
    return FA_ERR_INVALID_ARG;
  fa::RopeParams p = {};
  for (int i = 0; i < n; ++i) {
    if (!rows_ok(&x[i]) || !rows_ok(&y[i]) || x[i].heads != y[i].heads || !within(x[i], B, S) || !within(y[i], B, S))
      return FA_ERR_INVALID_ARG;
    p.x[i] = rows_in(x[i]);
    p.y[i] = rows_out(y[i]);
    p.heads[i] = x[i].heads;
  }
  if ((long long)p.heads[0] + p.heads[1] > 65535 || (long long)B * S > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  // an output is its own input, in place, or apart from everything else
  Stack in[2], out[2];
  for (int i = 0; i < n; ++i) in[i] = stack_of(x[i], B, S, D), out[i] = stack_of(y[i], B, S, D);
  for (int i = 0; i < n; ++i) {
    if (overlaps_itself(out[i])) return FA_ERR_INVALID_ARG;
    for (int j = 0; j < n; ++j)
      if (!(i == j && in_place(y[i], x[i], B, S)) && overlap(out[i], in[j])) return FA_ERR_INVALID_ARG;
  }
  if (n == 2 && overlap(out[0], out[1])) return FA_ERR_INVALID_ARG;
  p.freqs = freqs, p.positions = positions, p.pos_batch = positions_stride;
  p.cu = cu_seqlens, p.nseq = nseq, p.B = B, p.S = S, p.R = rot_dim;
  p.amp = amp, p.sign = backward ? -1.f : 1.f;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool il = interleaved != 0, zero = fill && cu_seqlens;
  if (D == 128) return dt == FA_BF16 ? launch_rope<128, true>(p, il, zero, st) : launch_rope<128, false>(p, il, zero, st);
  return dt == FA_BF16 ? launch_rope<64, true>(p, il, zero, st) : launch_rope<64, false>(p, il, zero, st);
}

fa_status append_call(const fa_rows* k, const fa_rows* v, const fa_rows* q, const fa_rows* q_out, const fa_pages* pages,
                      const int* seq_lens, const int* cu_seqlens, int nseq, int total, const double* freqs, int rot_dim,
                      int interleaved, float amp, const int* positions, int D, fa_dtype dt, void* stream, bool fill) {
  if (nseq < 0 || total < 0) return FA_ERR_INVALID_ARG;
  if (dt != FA_BF16 && dt != FA_FP16) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(amp)) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (freqs && !rot_ok(rot_dim, D)) return FA_ERR_UNSUPPORTED;
  if (!cu_seqlens && nseq != total) return FA_ERR_INVALID_ARG;
  if (fill && q && nseq == 0)  // every row is one of no sequence
    return rope_call(q, q_out, 1, freqs, rot_dim, interleaved, amp, 0, nullptr, 0, cu_seqlens, 0, 1, total, D, dt, stream,
                     true);
  if (nseq == 0 || total == 0) return FA_OK;
  const fa_status s = pages_check(pages, D);
  if (s != FA_OK) return s;
  if (!rows_ok(k) || !rows_ok(v) || k->heads != pages->heads || v->heads != pages->heads) return FA_ERR_INVALID_ARG;
  if (q && (!rows_ok(q) || !rows_ok(q_out) || q->heads != q_out->heads || !freqs)) return FA_ERR_INVALID_ARG;
  if (!seq_lens || !ints_ok(seq_lens) || !ints_ok(cu_seqlens) || !ints_ok(positions) ||
      (reinterpret_cast<uintptr_t>(freqs) & 7u))
    return FA_ERR_INVALID_ARG;
  fa::AppendParams p = {};
  p.k = rows_in(*k), p.v = rows_in(*v);
  if (q) p.q = rows_in(*q), p.q_out = rows_out(*q_out), p.Hq = q->heads;
  if ((long long)p.Hq + 2LL * pages->heads > 65535) return FA_ERR_UNSUPPORTED;
  // the pools apart from each other (one pool for both only where it takes the
  // same rows unrotated); q_out is q, in place, or apart from everything else
  if (!within(pages->n_pages, pages->page_stride) || !within(*k, 1, total) || !within(*v, 1, total) ||
      (q && (!within(*q, 1, total) || !within(*q_out, 1, total))))
    return FA_ERR_INVALID_ARG;
  const long long page = (long long)pages->heads * pages->page_size * D;
  const Stack pool_k = stack_of(pages->k, page, {{pages->n_pages, pages->page_stride}});
  const Stack pool_v = stack_of(pages->v, page, {{pages->n_pages, pages->page_stride}});
  const Stack ks = stack_of(*k, 1, total, D), vs = stack_of(*v, 1, total, D);
  if (overlap(pool_k, pool_v) && (freqs || pages->k != pages->v || !in_place(*k, *v, 1, total))) return FA_ERR_INVALID_ARG;
  if (q) {
    const Stack qs = stack_of(*q, 1, total, D), to = stack_of(*q_out, 1, total, D);
    if (overlaps_itself(to) || (!in_place(*q_out, *q, 1, total) && overlap(to, qs)) || overlap(to, ks) || overlap(to, vs) ||
        overlap(to, pool_k) || overlap(to, pool_v))
      return FA_ERR_INVALID_ARG;
  }
  p.k_pages = static_cast<uint16_t*>(pages->k);
  p.v_pages = static_cast<uint16_t*>(pages->v);
  p.page_stride = pages->page_stride, p.table = pages->block_table, p.table_stride = pages->table_stride;
  p.n_pages = pages->n_pages, p.page_shift = log2_of(pages->page_size), p.max_pages = pages->max_pages;
  p.seq_lens = seq_lens, p.cu = cu_seqlens, p.freqs = freqs, p.positions = positions;
  p.nseq = nseq, p.T = total, p.Hkv = pages->heads, p.R = freqs ? rot_dim : 0, p.amp = amp;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool in = interleaved != 0, zero = fill && q;
  if (D == 128) return dt == FA_BF16 ? launch_append<128, true>(p, in, zero, st) : launch_append<128, false>(p, in, zero, st);
  return dt == FA_BF16 ? launch_append<64, true>(p, in, zero, st) : launch_append<64, false>(p, in, zero, st);
}

// ---------------------------------------------------------------- paged decode
constexpr int kPagedCtas = 2;  // of paged_kernel on an SM
// Runs that a call can have: several waves of them (PagedRuns).
int paged_max_runs() { return kPagedCtas * sm_count() * fa::PagedRuns::kMaxWaves; }

// Ranges the shared rows are cut into: units = KV heads x query pairs CTAs run
// one range each.  The cost of n ranges is waves x (tiles of the longest range
// + the start and end of a CTA, about four tiles' worth); the fewest ranges of
// the least cost are taken.
int prefix_splits(long long units, int P) {
  const long long tiles = ((long long)P + 127) / 128, sms = sm_count();
  if (tiles <= 0) return 0;
  long long best = 1, cost = -1;
  for (long long n = 1; n <= std::min((long long)fa::kMaxRanges, tiles); ++n) {
    const long long c = ((units * n + sms - 1) / sms) * ((tiles + n - 1) / n + 4);
    if (cost < 0 || c < cost) best = n, cost = c;
  }
  return (int)best;
}

// Whether shared rows are worth a pass of their own.  Below 24 MB read once more
// than needed (from L2 mostly), or with up to three sequences, paged_kernel
// alone, reading them for each sequence, is done before prefix_kernel and the
// join are: 4 sequences x 1024 rows x 8 heads of 128, 13 MB more: 11.5 against
// 11.1 us on the GPU, but two launches instead of three (11.5 against 13.9 us
// for the call); 32 x 1024, 130 MB: 20.5 against 16.0; 4 x 16384: 27.8 against
// 27.6.  Two sequences, 8 heads of 128, read for each against a pass of their
// own: 16384 rows 22.0 against 27.6 us, 32768 33.9 against 44.7, 131072 106
// against 133; three: 4096 13.2 against 13.9, 16384 28.7 against 28.1.  Three
// behind longer rows, which the second and third reading no longer find in L2,
// are the rule's weak side: 32768 65.5 against 44.9 us, 131072 231 against 133.
bool shared_pass(int B, int Hkv, int P, int D) {
  return P > 0 && B > 3 && (double)(B - 1) * P * Hkv * D * 4 > 24e6;
}

struct PagedWs {
  size_t next_run, cuts, lse_part, o_part, pre_lse, pre_o, own_lse, own_o, total;
  int n_pre, n_pairs, per_tile;
};

PagedWs paged_layout(int B, int Hq, int Hkv, int P, int D) {
  const int G = Hq / Hkv;
  const int runs = paged_max_runs();
  const size_t parts = (size_t)2 * runs * G;
  PagedWs w;
  w.per_tile = 128 / G;
  w.n_pairs = (int)(((long long)B + 2 * w.per_tile - 1) / (2 * w.per_tile));
  w.n_pre = shared_pass(B, Hkv, P, D) ? prefix_splits((long long)Hkv * w.n_pairs, P) : 0;
  const size_t pre = (size_t)w.n_pre * B * Hq, own = w.n_pre ? (size_t)B * Hq : 0;
  w.next_run = 0;
  w.cuts = 256;
  // cuts of all units behind shared rows, else of the runs or units, whichever are fewer
  w.lse_part = w.cuts + up256((w.n_pre ? std::max((size_t)B * Hkv, (size_t)runs) : (size_t)runs) * sizeof(fa::PagedCut));
  w.o_part = w.lse_part + up256(parts * 4);
  w.pre_lse = w.o_part + up256(parts * D * 4);
  w.pre_o = w.pre_lse + up256(pre * 4);
  w.own_lse = w.pre_o + up256(pre * D * 4);
  w.own_o = w.own_lse + up256(own * 4);
  w.total = w.own_o + up256(own * D * 4);
  return w;
}

// One K or V pool as (64 columns, 8 rows, D / 64 halves, 8-row groups of all
// heads, pages), boxes of box whole rows (load_rows).
bool map_pages(CUtensorMap* m, const void* base, const fa_pages& pg, int D, bool bf16, int box) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint32_t halves = D / 64;
  const cuuint64_t dims[5] = {64, 8, halves, (cuuint64_t)pg.heads * pg.page_size / 8, (cuuint64_t)pg.n_pages};
  const cuuint64_t strides[4] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 16, (cuuint64_t)pg.page_stride * 2};
  const cuuint32_t boxes[5] = {64, 8, halves, (cuuint32_t)box / 8, 1}, estr[5] = {1, 1, 1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<void*>(base),
             dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q [B, Hkv, G, D] as (D, G, Hkv, B), boxes of 64 columns x G heads x per_tile sequences.
bool map_queries(CUtensorMap* m, const void* q, int B, int Hkv, int G, int D, bool bf16, int per_tile) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)G, (cuuint64_t)Hkv, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)G * D * 2, (cuuint64_t)Hkv * G * D * 2};
  const cuuint32_t boxes[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)per_tile}, estr[4] = {1, 1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(q), dims,
             strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tiles behind the shared rows of the longest sequence that the table can hold
// (one that ends inside them has at most a range of them to read, which is no
// reason for more CTAs), and whether a call may hand out runs (which takes one
// more small launch, about 1 us).
long long paged_tiles(const fa::PagedParams& p) { return std::max(1, (p.map.max_len - p.start + 63) / 64); }
bool hands_out(const fa::PagedParams& p, long long tiles) {
  return (long long)p.B * p.Hkv * tiles >= fa::kClaimTiles * kPagedCtas * sm_count();
}

template <int D, bool BF16, int NB, bool PRE>
fa_status launch_paged(const fa::PagedParams& p, const fa_pages& pg, cudaStream_t st) {
  using C = fa::PagedCfg<D, NB>;
  CUtensorMap mk, mv;
  const int box = std::min(C::KT, pg.page_size);
  if (!map_pages(&mk, pg.k, pg, D, BF16, box) || !map_pages(&mv, pg.v, pg, D, BF16, box)) return FA_ERR_CUDA;
  if (set_smem<fa::paged_kernel<D, BF16, NB, PRE>>(C::SMEM) != cudaSuccess) return FA_ERR_CUDA;
  fa::PagedParams a = p;
  const long long tiles = paged_tiles(p);
  static_assert(C::CTAS == kPagedCtas && C::KT == 64, "workspace for every run");
  const long long units = (long long)p.B * p.Hkv, ctas = (long long)C::CTAS * sm_count();
  a.grid = (int)std::min(ctas, units * tiles);
  const bool claim = hands_out(p, tiles);
  a.max_runs = claim ? a.grid * fa::PagedRuns::kMaxWaves : a.grid;
  a.by_unit = PRE || units <= a.max_runs;
  if (!claim) a.next_run = nullptr;
  // (behind shared rows the count was zeroed before them)
  if (claim && !PRE) {
    const fa_status s = launch_after(fa::paged_zero_kernel, dim3(1), 32, 0, st, a.next_run);
    if (s != FA_OK) return s;
  }
  const fa_status s = launch_after(fa::paged_kernel<D, BF16, NB, PRE>, dim3(a.grid), C::THREADS, C::SMEM, st, mk, mv, a);
  if (s != FA_OK) return s;
  if constexpr (PRE) {
    // four warps a row while all of them run at once (eight blocks to an SM)
    const long long rows = (long long)p.B * p.Hq;
    if (rows <= 16LL * sm_count() && p.n_pre >= 4)
      return launch_after(fa::paged_join_kernel<D, BF16, 4>, dim3((unsigned)((rows + 1) / 2)), 256, 0, st, a);
    return launch_after(fa::paged_join_kernel<D, BF16, 1>, dim3((unsigned)((rows + 7) / 8)), 256, 0, st, a);
  }
  // units that are never cut: of one tile, or all of them short and on an SM of their own
  if (tiles == 1 || (tiles <= fa::kWholeTiles && units <= a.grid)) return FA_OK;
  // few rows to a block (and so many warps to a row) as long as the blocks, three
  // to an SM, run at once
  const long long cuts = a.by_unit ? units : a.max_runs;
  const dim3 grid((unsigned)cuts, (unsigned)std::max(1LL, std::min<long long>(p.G, 3LL * sm_count() / cuts)));
  return launch_after(fa::paged_merge_kernel<D, BF16>, grid, 256, 0, st, a);
}

template <int D, bool BF16>
fa_status launch_prefix(const fa::PrefixParams& p, const void* q, const fa_pages& pg, cudaStream_t st) {
  using C = fa::FwdCfg<D>;
  CUtensorMap mq, mk, mv;
  const int box = std::min(128, pg.page_size);
  if (!map_queries(&mq, q, p.B, p.Hkv, p.G, D, BF16, p.per_tile) || !map_pages(&mk, pg.k, pg, D, BF16, box) ||
      !map_pages(&mv, pg.v, pg, D, BF16, box))
    return FA_ERR_CUDA;
  if (set_smem<fa::prefix_kernel<D, BF16>>(C::SMEM) != cudaSuccess) return FA_ERR_CUDA;
  const long long grid = (long long)p.n_pre * p.n_pairs * p.Hkv;
  if (grid > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  return launch_after(fa::prefix_kernel<D, BF16>, dim3((unsigned)grid), C::THREADS, C::SMEM, st, mq, mk, mv, p);
}

template <int D, bool BF16>
fa_status run_paged(const fa::PagedParams& p, const fa::PrefixParams& pre, const void* q, const fa_pages& pg,
                    cudaStream_t st) {
  if (p.n_pre) {
    if (hands_out(p, paged_tiles(p))) {
      const fa_status s = launch_after(fa::paged_zero_kernel, dim3(1), 32, 0, st, p.next_run);
      if (s != FA_OK) return s;
    }
    const fa_status s = launch_prefix<D, BF16>(pre, q, pg, st);
    if (s != FA_OK) return s;
    return p.G <= 8 ? launch_paged<D, BF16, 1, true>(p, pg, st) : launch_paged<D, BF16, 2, true>(p, pg, st);
  }
  return p.G <= 8 ? launch_paged<D, BF16, 1, false>(p, pg, st) : launch_paged<D, BF16, 2, false>(p, pg, st);
}

fa_status paged_call(const void* q, const fa_pages* pages, const int* seq_lens, int prefix_len, const int* prefix_table,
                     void* o, float* lse, int B, int Hq, int D, float scale, fa_dtype dt, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (B < 0 || Hq < 0 || prefix_len < 0) return FA_ERR_INVALID_ARG;
  if (dt != FA_BF16 && dt != FA_FP16) return FA_ERR_INVALID_ARG;
  if (!scale_ok(scale)) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (B == 0 || Hq == 0) return FA_OK;
  const fa_status s = pages_check(pages, D);
  if (s != FA_OK) return s;
  const int Hkv = pages->heads, max_len = pages->max_pages * pages->page_size;
  if (Hq % Hkv) return FA_ERR_INVALID_ARG;
  if (Hq / Hkv > 16) return FA_ERR_UNSUPPORTED;
  if (prefix_len % pages->page_size || prefix_len > max_len) return FA_ERR_INVALID_ARG;
  if ((long long)B * Hq > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  // paged_kernel counts what it has to do in 31 bits, whatever the lengths are
  if ((long long)B * Hkv > 0x7fffffffLL / ((max_len + 63LL) / 64 + fa::kUnitCost)) return FA_ERR_UNSUPPORTED;
  if (!ptrs_ok({q, o, lse}) || !seq_lens || !ints_ok(seq_lens) || !ints_ok(prefix_table)) return FA_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return FA_ERR_INVALID_ARG;
  const PagedWs w = paged_layout(B, Hq, Hkv, prefix_len, D);
  if (workspace_bytes < w.total) return FA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  fa::PagedParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.seq_lens = seq_lens;
  p.map = {pages->block_table, pages->table_stride, pages->n_pages, log2_of(pages->page_size), max_len, prefix_table,
           prefix_len};
  p.o_part = reinterpret_cast<float*>(ws + w.o_part);
  p.lse_part = reinterpret_cast<float*>(ws + w.lse_part);
  p.cuts = reinterpret_cast<fa::PagedCut*>(ws + w.cuts);
  p.next_run = reinterpret_cast<int*>(ws + w.next_run);
  p.o = o;
  p.lse = lse;
  p.pre_o = reinterpret_cast<float*>(ws + w.pre_o);
  p.pre_lse = reinterpret_cast<float*>(ws + w.pre_lse);
  p.own_o = reinterpret_cast<float*>(ws + w.own_o);
  p.own_lse = reinterpret_cast<float*>(ws + w.own_lse);
  p.n_pre = w.n_pre, p.start = w.n_pre ? prefix_len : 0;
  p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv;
  p.scale_log2 = scale * 1.4426950408889634f;
  fa::PrefixParams pre = {};
  pre.seq_lens = seq_lens;
  pre.map = p.map;
  pre.pre_o = reinterpret_cast<float*>(ws + w.pre_o);
  pre.pre_lse = reinterpret_cast<float*>(ws + w.pre_lse);
  pre.P = prefix_len, pre.n_pre = w.n_pre, pre.n_pairs = w.n_pairs, pre.per_tile = w.per_tile;
  pre.B = B, pre.Hq = Hq, pre.Hkv = Hkv, pre.G = p.G;
  pre.scale_log2 = p.scale_log2;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (D == 128)
    return dt == FA_BF16 ? run_paged<128, true>(p, pre, q, *pages, st) : run_paged<128, false>(p, pre, q, *pages, st);
  return dt == FA_BF16 ? run_paged<64, true>(p, pre, q, *pages, st) : run_paged<64, false>(p, pre, q, *pages, st);
}

}  // namespace

cudaError_t fa_host::take_paged_error(uint32_t* code) {
  cudaError_t e = cudaMemcpyFromSymbol(code, fa::g_dev_error, sizeof(*code));
  if (e != cudaSuccess || *code == 0) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(fa::g_dev_error, &zero, sizeof(zero));
}

extern "C" {

fa_status fa_rope_freqs(int rot_dim, double base, fa_rope_scaling scaling, double factor, int original_len,
                        double beta_fast, double beta_slow, double* freqs, float* amp) {
  constexpr double kTau = 6.283185307179586476925;
  if (rot_dim <= 0 || rot_dim % 2 || !freqs || !amp) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(base) || base <= 1.0) return FA_ERR_INVALID_ARG;
  if (scaling != FA_ROPE_PLAIN && scaling != FA_ROPE_LINEAR && scaling != FA_ROPE_NTK && scaling != FA_ROPE_YARN)
    return FA_ERR_INVALID_ARG;
  if (scaling != FA_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0)) return FA_ERR_INVALID_ARG;
  if (scaling == FA_ROPE_NTK) {
    if (rot_dim == 2) return FA_ERR_INVALID_ARG;
    base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  }
  double lo = 0, hi = 0;
  if (scaling == FA_ROPE_YARN) {
    if (original_len <= 0 || !std::isfinite(beta_fast) || !std::isfinite(beta_slow) || beta_slow <= 0 ||
        beta_fast < beta_slow)
      return FA_ERR_INVALID_ARG;
    // the pair that turns `beta` times over the trained length
    auto pair_of = [&](double beta) { return rot_dim * std::log(original_len / (beta * kTau)) / (2 * std::log(base)); };
    lo = std::max(std::floor(pair_of(beta_fast)), 0.0);
    hi = std::min(std::ceil(pair_of(beta_slow)), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == FA_ROPE_LINEAR) f /= factor;
    if (scaling == FA_ROPE_YARN) {
      const double keep = 1.0 - std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 1e-3)));
      f = f / factor * (1.0 - keep) + f * keep;
    }
    freqs[i] = f;
  }
  *amp = scaling == FA_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return FA_OK;
}

fa_status fa_rope(const fa_rows* x, const fa_rows* y, int n, const double* freqs, int rot_dim, int interleaved,
                  float amp, int backward, const int* positions, long long positions_stride,
                  const int* cu_seqlens, int nseq, int B, int S, int D, fa_dtype dt, void* stream) {
  return rope_call(x, y, n, freqs, rot_dim, interleaved, amp, backward, positions, positions_stride, cu_seqlens, nseq, B,
                   S, D, dt, stream, false);
}

fa_status fa_rope_fill(const fa_rows* x, const fa_rows* y, int n, const double* freqs, int rot_dim, int interleaved,
                       float amp, int backward, const int* positions, long long positions_stride,
                       const int* cu_seqlens, int nseq, int B, int S, int D, fa_dtype dt, void* stream) {
  return rope_call(x, y, n, freqs, rot_dim, interleaved, amp, backward, positions, positions_stride, cu_seqlens, nseq, B,
                   S, D, dt, stream, true);
}

fa_status fa_append_paged(const fa_rows* k, const fa_rows* v, const fa_rows* q, const fa_rows* q_out,
                          const fa_pages* pages, const int* seq_lens, const int* cu_seqlens, int nseq,
                          int total, const double* freqs, int rot_dim, int interleaved, float amp,
                          const int* positions, int D, fa_dtype dt, void* stream) {
  return append_call(k, v, q, q_out, pages, seq_lens, cu_seqlens, nseq, total, freqs, rot_dim, interleaved, amp,
                     positions, D, dt, stream, false);
}

fa_status fa_append_paged_fill(const fa_rows* k, const fa_rows* v, const fa_rows* q, const fa_rows* q_out,
                               const fa_pages* pages, const int* seq_lens, const int* cu_seqlens, int nseq,
                               int total, const double* freqs, int rot_dim, int interleaved, float amp,
                               const int* positions, int D, fa_dtype dt, void* stream) {
  return append_call(k, v, q, q_out, pages, seq_lens, cu_seqlens, nseq, total, freqs, rot_dim, interleaved, amp,
                     positions, D, dt, stream, true);
}

size_t fa_decode_paged_workspace_size(int B, int Hq, int Hkv, int D) {
  return fa_decode_prefix_workspace_size(B, Hq, Hkv, 0, D);
}

size_t fa_decode_prefix_workspace_size(int B, int Hq, int Hkv, int prefix_len, int D) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hq / Hkv > 16 || prefix_len < 0 || (D != 64 && D != 128)) return 0;
  if ((long long)B * Hq > 0x7fffffffLL) return 0;
  return paged_layout(B, Hq, Hkv, prefix_len, D).total;
}

fa_status fa_decode_paged(const void* q, const fa_pages* pages, const int* seq_lens, void* o, float* lse, int B, int Hq,
                          int D, float scale, fa_dtype dt, void* workspace, size_t workspace_bytes, void* stream) {
  return paged_call(q, pages, seq_lens, 0, nullptr, o, lse, B, Hq, D, scale, dt, workspace, workspace_bytes, stream);
}

fa_status fa_decode_prefix(const void* q, const fa_pages* pages, const int* seq_lens, int prefix_len,
                           const int* prefix_table, void* o, float* lse, int B, int Hq, int D, float scale, fa_dtype dt,
                           void* workspace, size_t workspace_bytes, void* stream) {
  return paged_call(q, pages, seq_lens, prefix_len, prefix_table, o, lse, B, Hq, D, scale, dt, workspace,
                    workspace_bytes, stream);
}

}  // extern "C"
