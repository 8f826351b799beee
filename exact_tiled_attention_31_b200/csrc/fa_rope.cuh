// fa_rope.cuh - rotary positions, on tensors and on the way into a paged cache.
//
// Pair i (i < R / 2) of the first R of a row's D columns is a point of the
// plane, turned by the angle pos * f_i and scaled by amp:
//     (a, b) -> amp * (a cos - b sin, b cos + a sin),
// and the columns from R on are copied.  The pairs are columns (i, i + R/2)
// ("half") or (2i, 2i + 1) ("interleaved").  The map is linear, so the
// gradient takes the transposed matrix: the same with the angle negated.
//
// Angles.  pos * f_i reaches 10^6 radians and more, where fp32 has lost the
// phase.  The turns pos * f_i / 2 pi are formed in fp64 and reduced to
// [-1/2, 1/2] there (error below 2^-34 turns up to position 2^20, 2^-23 at
// 2^31).  The reduced angle goes to fp32 and to the special-function unit's
// sine and cosine, whose error on [-pi, pi] is below 2^-21 (with the angle's
// own rounding the pair is off by at most 2^-20 of its length, 2^-9 of the
// half step of fp16; sincospif, 40 instructions instead of 3, was no closer
// after the rounding to 16 bits).
//
// Bound: HBM.  Every row is read once and written once, 2 x 2 D bytes, with
// three multiply-adds a pair.  A thread owns two 8-column chunks of one
// token that hold whole pairs (columns c and c + R/2 of the rotated part;
// likewise of the copied part) for four heads, all of whose loads are in
// flight before it forms the eight sines and cosines.  Four heads to a block,
// and 128 threads, not more: the angles are cheap, and many short blocks leave
// a short tail (q and k of 32 heads x 4096 rows, now 22.1 us; when tried:
// 24.0 with 256 threads and eight heads, 23.7 with four, 22.8 with 128 threads).  Where the heads of a
// token lie next to each other, neighbouring blocks take the heads of the same
// tokens instead of the next tokens (22.4 us; with rows of a head next to each
// other that costs 1 %: 81.0 against 80.2 us for 64 heads x 8192 twice).
#pragma once

#include "pdl.cuh"
#include "sm100.cuh"

namespace fa {

constexpr int kRopeThreads = 128;
constexpr int kRopeHeads = 4;  // heads of a block, all in flight

// A strided stack of rows of D contiguous 16-bit values (strides in elements).
struct RowsIn {
  const uint16_t* p;
  long long batch, head, row;
};
struct RowsOut {
  uint16_t* p;
  long long batch, head, row;
};

// The place of token t of a packed batch: its sequence s in [0, nseq) by the
// offsets cu[0 .. nseq], or -1 behind the last sequence (or before the first).
__device__ __forceinline__ int seq_of(const int* cu, int nseq, int t) {
  if (t < cu[0] || t >= cu[nseq]) return -1;
  int lo = 0, hi = nseq;  // the number of offsets cu[1 ..] that are <= t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid + 1] <= t) lo = mid + 1; else hi = mid;
  }
  return lo < nseq ? lo : -1;
}

// cosine and sine of pair `freq` at a position of `cycles` = position / 2 pi
__device__ __forceinline__ void rope_angle(double freq, double cycles, float amp, float& c, float& s) {
  double turns = cycles * freq;
  turns -= rint(turns);
  const float x = (float)turns * 6.2831853071795865f;
  c = __cosf(x) * amp;
  s = __sinf(x) * amp;
}

// The two 8-column chunks of item `it` (of D / 16 items), whether they are
// rotated, and for pair j of the thread's eight its frequency index.
template <int D, bool INTER>
struct RopeItem {
  int lo, hi;   // first columns of the two chunks
  bool turn;
  int f_lo, f_hi;
  __device__ __forceinline__ RopeItem(int it, int R) {
    turn = it < R / 16;
    const int base = turn ? 0 : R, width = turn ? R : D - R, i = turn ? it : it - R / 16;
    lo = base + 8 * i;
    hi = lo + width / 2;
    // half: pair j is (lo + j, hi + j), frequency lo + j; interleaved: each
    // chunk holds four pairs, frequencies from half its first column on
    f_lo = INTER ? lo / 2 : lo;
    f_hi = INTER ? hi / 2 : lo + 4;
  }
};

template <bool BF16, bool INTER>
__device__ __forceinline__ void rope_turn(uint4& a, uint4& b, const float (&c)[8], const float (&s)[8]) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&a);
  uint32_t* y = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (INTER) {
      const float2 u = unpack2<BF16>(x[j]), v = unpack2<BF16>(y[j]);
      x[j] = pack2<BF16>(u.x * c[j] - u.y * s[j], u.y * c[j] + u.x * s[j]);
      y[j] = pack2<BF16>(v.x * c[4 + j] - v.y * s[4 + j], v.y * c[4 + j] + v.x * s[4 + j]);
    } else {
      const float2 u = unpack2<BF16>(x[j]), v = unpack2<BF16>(y[j]);
      x[j] = pack2<BF16>(u.x * c[2 * j] - v.x * s[2 * j], u.y * c[2 * j + 1] - v.y * s[2 * j + 1]);
      y[j] = pack2<BF16>(v.x * c[2 * j] + u.x * s[2 * j], v.y * c[2 * j + 1] + u.y * s[2 * j + 1]);
    }
  }
}

// n <= kRopeHeads rows of one token, xs and ys elements apart: turned by `pos`
// (with sign -1 back) if `turn`, else copied; zeros in their place if FILL and
// `skip`.
template <int D, bool BF16, bool INTER, bool FILL>
__device__ __forceinline__ void rope_heads(const RopeItem<D, INTER>& item, const uint16_t* x, long long xs, uint16_t* y,
                                           long long ys, int n, bool turn, bool skip, const double* freqs, int pos,
                                           float amp, float sign) {
  uint4 lo[kRopeHeads], hi[kRopeHeads];
#pragma unroll
  for (int k = 0; k < kRopeHeads; ++k)
    if (k < n) {
      lo[k] = *reinterpret_cast<const uint4*>(x + item.lo);
      hi[k] = *reinterpret_cast<const uint4*>(x + item.hi);
      x += xs;
    }
  turn = turn && item.turn;
  float c[8], s[8];
  if (turn) {
    const double cycles = (double)pos * 0.15915494309189533577;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      rope_angle(freqs[(j < 4 ? item.f_lo : item.f_hi) + (j & 3)], cycles, amp, c[j], s[j]);
      s[j] *= sign;
    }
  }
#pragma unroll
  for (int k = 0; k < kRopeHeads; ++k)
    if (k < n) {
      if (turn) rope_turn<BF16, INTER>(lo[k], hi[k], c, s);
      if (FILL && skip) lo[k] = hi[k] = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(y + item.lo) = lo[k];
      *reinterpret_cast<uint4*>(y + item.hi) = hi[k];
      y += ys;
    }
}
// groups of kRopeHeads heads, none of them over two tensors
__host__ __device__ constexpr int rope_groups(int heads) { return (heads + kRopeHeads - 1) / kRopeHeads; }

struct RopeParams {
  RowsIn x[2];
  RowsOut y[2];
  int heads[2];
  const double* freqs;     // [R / 2] radians per position
  const int* positions;    // [B, S] by pos_batch, or null: the index in the sequence
  long long pos_batch;
  const int* cu;           // packed batch (B = 1, S rows): [nseq + 1] offsets, or null
  int nseq, B, S, R;
  bool heads_near;         // grid: (head groups, token tiles) instead of (token tiles, head groups)
  float amp;
  float sign;              // -1 turns back
};

// block: tokens x D / 16 items.  FILL: rows of no sequence become zero, by the
// same path as the others, in an instance of its own (q and k of 32 heads x 4096
// packed rows 20.4 us either way; 23.0 with a branch that stores zeros).
template <int D, bool BF16, bool INTER, bool FILL>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  pdl_wait();
  pdl_launch();
  constexpr int ITEMS = D / 16, TOKENS = kRopeThreads / ITEMS;
  const int it = threadIdx.x % ITEMS;
  const uint32_t tile = p.heads_near ? blockIdx.y : blockIdx.x, group = p.heads_near ? blockIdx.x : blockIdx.y;
  const uint32_t n = tile * TOKENS + threadIdx.x / ITEMS;
  if (n >= (uint32_t)p.B * (uint32_t)p.S) return;
  const int b = n / (uint32_t)p.S, t = n - b * (uint32_t)p.S;
  int pos = t;
  bool skip = false;
  if (p.cu) {
    const int s = seq_of(p.cu, p.nseq, t);
    skip = s < 0;
    if (!FILL && skip) return;  // rows of no sequence stay as they were
    pos = t - p.cu[FILL ? max(s, 0) : s];
  }
  if (p.positions) pos = p.positions[b * p.pos_batch + t];
  const int first = rope_groups(p.heads[0]);
  const bool w = group >= first;  // which tensor
  const int h = (group - (w ? first : 0)) * kRopeHeads;
  const RowsIn x = w ? p.x[1] : p.x[0];
  const RowsOut y = w ? p.y[1] : p.y[0];
  rope_heads<D, BF16, INTER, FILL>(RopeItem<D, INTER>(it, p.R), x.p + b * x.batch + h * x.head + t * x.row, x.head,
                                   y.p + b * y.batch + h * y.head + t * y.row, y.head,
                                   (w ? p.heads[1] : p.heads[0]) - h, !skip, skip, p.freqs, pos, p.amp, p.sign);
}

// ---------------------------------------------------------------------------
// New keys and values into the pages of their sequences.
//
// Token t is the j-th of the n new tokens of its sequence b; it becomes row
// i = seq_lens[b] - n + j of the sequence, which lives in row i % page_size
// of page table[b][i / page_size].  Its key is rotated by i (or positions[t])
// on the way, its value copied, and the query of the same token, if given,
// rotated into q_out by the same launch.  Tokens with i < 0 (a padded batch
// gives its padding rows length 0) and tokens of no sequence write nothing, or
// with FILL zeros to their queries' rows of q_out.
// A row past the table or a page outside the pool writes nothing and records
// an argument error.
// ---------------------------------------------------------------------------
enum : uint32_t { APPEND_SITE_PAGE = 0x400 };

struct AppendParams {
  RowsIn q, k, v;  // batch unused
  RowsOut q_out;
  uint16_t* k_pages;
  uint16_t* v_pages;
  long long page_stride;   // elements from one page to the next
  const int* table;        // [nseq, max_pages] by table_stride
  long long table_stride;
  const int* seq_lens;     // [nseq], the new tokens included
  const int* cu;           // [nseq + 1], or null: token t is the new one of sequence t
  const double* freqs;     // null (R = 0): no rotation
  const int* positions;    // [T], or null
  int n_pages, page_shift, max_pages;
  int nseq, T, Hq, Hkv, R;
  bool heads_near;         // as in RopeParams
  float amp;
};

template <int D, bool BF16, bool INTER, bool FILL>
__global__ void __launch_bounds__(kRopeThreads) append_kernel(const AppendParams p) {
  pdl_wait();
  pdl_launch();
  constexpr int ITEMS = D / 16, TOKENS = kRopeThreads / ITEMS;
  const int it = threadIdx.x % ITEMS;
  const uint32_t tile = p.heads_near ? blockIdx.y : blockIdx.x, group = p.heads_near ? blockIdx.x : blockIdx.y;
  const uint32_t n = tile * TOKENS + threadIdx.x / ITEMS;
  if (n >= (uint32_t)p.T) return;
  const int t = n;
  int b = t, i;
  if (p.cu) {
    b = seq_of(p.cu, p.nseq, t);
    if (!FILL && b < 0) return;
    i = FILL && b < 0 ? -1 : p.seq_lens[b] - (p.cu[b + 1] - t);
  } else {
    i = p.seq_lens[b] - 1;
  }
  const bool skip = i < 0;
  if (skip && (!FILL || group >= rope_groups(p.Hq))) return;
  const int pos = p.positions ? p.positions[t] : i;
  const int slot = i >> p.page_shift, row = i & ((1 << p.page_shift) - 1);
  const int page = !(FILL && skip) && slot < p.max_pages ? p.table[b * p.table_stride + slot] : -1;
  const bool placed = page >= 0 && page < p.n_pages;
  if (!placed && !(FILL && skip) && it == 0 && group == 0) record_error(DEV_ERR_ARG, APPEND_SITE_PAGE);
  // q's groups of heads, then k's, then v's
  const RopeItem<D, INTER> item(it, p.R);
  const int gq = rope_groups(p.Hq), gk = gq + rope_groups(p.Hkv);
  if (group < gq) {
    const int h = group * kRopeHeads;
    rope_heads<D, BF16, INTER, FILL>(item, p.q.p + h * p.q.head + t * p.q.row, p.q.head,
                                     p.q_out.p + h * p.q_out.head + t * p.q_out.row, p.q_out.head, p.Hq - h, !skip, skip,
                                     p.freqs, pos, p.amp, 1.f);
  } else if (placed) {
    const bool val = group >= gk;
    const int h = (group - (val ? gk : gq)) * kRopeHeads;
    const RowsIn x = val ? p.v : p.k;
    uint16_t* y = (val ? p.v_pages : p.k_pages) + page * p.page_stride + ((((long long)h << p.page_shift) + row) * D);
    rope_heads<D, BF16, INTER, false>(item, x.p + h * x.head + t * x.row, x.head, y, (long long)D << p.page_shift,
                                      p.Hkv - h, !val, false, p.freqs, pos, p.amp, 1.f);
  }
}

}  // namespace fa
