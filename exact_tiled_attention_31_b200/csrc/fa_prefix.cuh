// fa_prefix.cuh - attention of many single-token queries over shared rows.
//
// The first P rows of every sequence are the same pages.  For one KV head the
// B sequences' G query heads each are then B * G query rows against one and
// the same K and V: a matrix product, as in the forward, instead of B passes
// over the cache.  Row (b, g) takes the ranges that lie whole in [0, len_b);
// paged_kernel reads the rows of the one that the sequence ends in.  Each
// CTA runs two tiles of up to 128 query rows over a contiguous range of
// 128-row K/V tiles and writes normalised fp32 parts with the log2 of their
// sums; paged_kernel takes the rows that each sequence has of its own, and
// paged_join_kernel joins both.
//
// Bound: with R = B * G rows a KV head, 4 R D flop against 4 D bytes a shared
// row: HBM up to about 256 rows (the two tiles' products and exponentials of a
// K/V tile then take as long as its 64 KB at an SM's share of the bandwidth),
// the tensor cores and the exponentials above.  So K/V are split over enough
// CTAs to fill the SMs, and a CTA takes 256 query rows, not 128, to halve what
// it draws from L2 once there are that many.
//
// Roles, pipeline and arithmetic are those of fwd_kernel (fa_fwd.cuh): a TMA
// warp, a tcgen05 issuer, sixteen softmax warps, four correction warps; S, P
// and O in TMEM.  What differs is where tiles come from (a box per page, all
// lanes of the TMA warp issuing), the per-row limits, and the fp32 parts.  The
// maximum is exact, as there: the largest weight of a row is then 1 without
// rounding, and two keys that share the weight mix within half a step.  (One
// that moves only for a score above it by 2^8 saves 2.6 of 172 us for 250
// queries, 32 heads, against 32768 shared rows; both weights then round.)
#pragma once

#include "fa_fwd.cuh"
#include "fa_paged.cuh"

namespace fa {

struct PrefixParams {
  const int* seq_lens;  // [B]
  PagedMap map;         // n_shared: P; max_len clamps seq_lens
  float* pre_o;         // [n_pre, B * Hq, D]
  float* pre_lse;       // [n_pre, B * Hq]
  int P, n_pre, n_pairs;
  int B, Hq, Hkv, G;
  int per_tile;         // sequences per query tile: 128 / G
  float scale_log2;
};

// `bytes` (a multiple of 16) of shared memory that this thread wrote (and
// fenced) to global memory, and the wait for all of this thread's copies.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)),
               "r"(smem_addr(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_store_wait() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
}

template <int D, bool BF16>
__global__ void __launch_bounds__(768, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const PrefixParams p) {
  using C = FwdCfg<D>;

  // ---- work unit: (split, KV head, query pair); the pairs of one split and
  // head side by side, so that they share its K/V tiles in L2
  const int pair = blockIdx.x % p.n_pairs;
  const int rest = blockIdx.x / p.n_pairs;
  const int kvh = rest % p.Hkv, split = rest / p.Hkv;
  const int all_tiles = (p.P + 127) / 128;
  const int j0 = range_begin(split, all_tiles, p.n_pre);
  const int n_kv = range_begin(split + 1, all_tiles, p.n_pre) - j0;  // >= 1: n_pre <= all_tiles
  const int range_end = min(p.P, 128 * (j0 + n_kv));
  const int b0 = 2 * pair * p.per_tile;  // first sequence of query tile 0; tile 1 follows
  const bool has_t1 = b0 + p.per_tile < p.B;
  const int n0 = n_kv, n1 = has_t1 ? n_kv : 0;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* q_full = bars;
  uint64_t* kv_full = bars + 2;
  uint64_t* kv_empty = kv_full + C::NSLOT;
  uint64_t* s_full = kv_empty + C::NSLOT;
  uint64_t* p_full = s_full + 2;
  uint64_t* mx_full = p_full + 4;
  uint64_t* o_ready = mx_full + 8;
  uint64_t* pv_done = o_ready + 2;
  uint64_t* stats_ready = pv_done + 2;
  uint64_t* o_full = stats_ready + 2;
  uint64_t* drain = o_full + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  float* pmax_buf = reinterpret_cast<float*>(smem + C::XCH_OFF);  // [tile][half][128]
  float* sum_buf = pmax_buf + 2 * 2 * 128;                        // [tile][half][l, lr][128]

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&o_ready[i], 128);
      for (int q = 0; q < 4; ++q) mbar_init(&mx_full[4 * i + q], 64);
      mbar_init(&pv_done[i], 1);
      mbar_init(&stats_ready[i], 256);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&p_full[i], 256);  // both halves of a tile
    for (int i = 0; i < C::NSLOT; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t sq = smem_addr(smem + C::Q_OFF);
  const uint32_t skv = smem_addr(smem + C::KV_OFF);

  // row r of query tile t: its sequence (or -1) and query head
  auto seq_of_row = [&](int t, int r) {
    const int k = r / p.G, b = b0 + t * p.per_tile + k;
    return k < p.per_tile && b < p.B ? b : -1;
  };

  // register split over 768 threads launched with 80 each (61440)
  static_assert(128 * 48 + 512 * 96 + 128 * 48 == 768 * 80, "register split");
  if (warp < 4) {
    regs_dec<48>();
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      const int box = min(128, 1 << p.map.page_shift), boxes = 128 / box;  // rows per box, boxes per tile: <= 8
      const int my_box = (int)lane;
      const bool active = my_box < boxes;
      // table entry of this lane's box of tile j; past the shared rows zeros are filled
      const int* shared = p.map.shared ? p.map.shared : p.map.table;
      auto find = [&](int j) {
        const int first = (j0 + j) * 128 + my_box * box;
        return active && j < n_kv && first < p.P ? shared[first >> p.map.page_shift] : p.map.n_pages;
      };
      auto length_of = [&](int b) { return min(p.seq_lens[b], p.map.max_len); };
      // The first sequence's entries are on their way while its length shows
      // whether they are the ones.
      int id0 = find(0), id1 = find(1);
      if (!p.map.shared && length_of(0) < p.P) {
        shared += shared_row(p.seq_lens, p.B, p.map.max_len, p.P) * p.map.table_stride;
        id0 = find(0);
        id1 = find(1);
      }
      // The page of an entry, or zeros where it names none: an error where a
      // sequence of this CTA takes the range (entries that none has may be anything).
      auto page_of = [&](int j, int id) {
        const bool none = (id < 0 || id >= p.map.n_pages) && active && (j0 + j) * 128 + my_box * box < p.P;
        if (__any_sync(0xffffffffu, none)) {
          bool taken = false;
          for (int b = b0 + (int)lane; b < min(b0 + 2 * p.per_tile, p.B); b += 32) taken |= length_of(b) >= range_end;
          if (__any_sync(0xffffffffu, taken) && none) record_error(DEV_ERR_ARG, PAGED_SITE_PAGE);
        }
        return id >= 0 && id < p.map.n_pages ? id : p.map.n_pages;
      };
      if (lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        for (int t = 0; t < (has_t1 ? 2 : 1); ++t) {
          mbar_expect_tx(&q_full[t], p.per_tile * p.G * 128 * C::CH);
          for (int c = 0; c < C::CH; ++c)
            tma_load_4d(smem + C::Q_OFF + t * C::TILE + c * C::CHUNK, &tm_q, &q_full[t], c * 64, 0, kvh,
                        b0 + t * p.per_tile);
        }
      }
      __syncwarp();
      int fill = 0;
      bool ok = true;
      auto load = [&](bool is_v, int jj, int id) {
        const uint32_t slot = fill % C::NSLOT, round = fill / C::NSLOT;
        if (round > 0 &&
            !(ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[slot], (round - 1) & 1, FWD_SITE_PROD))))
          return;
        if (lane == 0) mbar_expect_tx(&kv_full[slot], C::TILE);
        __syncwarp();
        if (active) {
          const int first = ((j0 + jj) * 128 + my_box * box) & ((1 << p.map.page_shift) - 1);  // row in its page
          load_rows(smem + C::KV_OFF + slot * C::TILE + my_box * box * D * 2, is_v ? &tm_v : &tm_k, &kv_full[slot],
                    ((kvh << p.map.page_shift) + first) >> 3, id);
        }
        ++fill;
      };
      load(false, 0, page_of(0, id0));
      for (int jj = 0; jj < n_kv && ok; ++jj) {
        const int id2 = find(jj + 2);
        load(true, jj, page_of(jj, id0));
        if (ok && jj + 1 < n_kv) load(false, jj + 1, page_of(jj + 1, id1));
        id0 = id1;
        id1 = id2;
      }
      // never leave a copy in flight into shared memory about to be given back
      for (int f = (fill > C::NSLOT ? fill - C::NSLOT : 0); f < fill; ++f)
        mbar_wait(&kv_full[f % C::NSLOT], (f / C::NSLOT) & 1, FWD_SITE_PROD);
      for (int t = 0; t < (has_t1 ? 2 : 1); ++t) mbar_wait(&q_full[t], 0, FWD_SITE_PROD);
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      const uint32_t e = elect_one();
      constexpr uint32_t IDESC_QK = make_idesc(128, 128, BF16, false, false);
      constexpr uint32_t IDESC_PV = make_idesc(128, D, BF16, false, true);
      const uint64_t dq_base = make_sdesc(sq, 16, 1024);
      // K and V tiles are [8-row group][half][8][128 bytes] (load_rows): 8-row
      // groups GROUP apart, the second 64 columns 1 KB behind the first
      constexpr uint32_t GROUP = D * 16;
      const uint64_t dk_base = make_sdesc(skv, 16, GROUP);      // K-major
      const uint64_t dv_base = make_sdesc(skv, 1024, GROUP);    // MN-major
      bool ok = true;
      int fill = 0;
      auto take = [&](uint32_t& slot) {
        slot = fill % C::NSLOT;
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&kv_full[slot], (fill / C::NSLOT) & 1, FWD_SITE_KV));
        ++fill;
      };
      auto qk = [&](int t, uint32_t kslot) {
        const uint64_t a = desc_add(dq_base, t * C::TILE), bb = desc_add(dk_base, kslot * C::TILE);
        const uint32_t d = tmem + C::TM_S + 128 * t;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss_e(d, desc_add(a, (kk >> 2) * C::CHUNK + (kk & 3) * 32),
                   desc_add(bb, (kk >> 2) * 1024 + (kk & 3) * 32), IDESC_QK, kk > 0 ? 1u : 0u, e);
      };
      auto pv = [&](int t, int h, uint32_t vslot, uint32_t acc) {
        const uint64_t bb = desc_add(dv_base, vslot * C::TILE + h * 8 * GROUP);
        const uint32_t d = tmem + C::TM_O + D * t, pa = tmem + C::TM_S + 128 * t + 32 * h;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts_e(d, pa + kk * 8, desc_add(bb, kk * 2 * GROUP), IDESC_PV, kk > 0 ? 1u : acc, e);
      };
      uint32_t ks;
      take(ks);
      for (int t = 0; t < (has_t1 ? 2 : 1) && ok; ++t) {
        ok = __all_sync(0xffffffffu, mbar_wait(&q_full[t], 0, FWD_SITE_Q));
        if (!ok) break;
        tc_fence_after();
        qk(t, ks);
        mma_commit_e(&s_full[t], e);
      }
      if (ok) mma_commit_e(&kv_empty[ks], e);
      // Everything that is ready early is waited for before P, so that P V and
      // the next Q K^T of a tile go out back to back: every wait here is ahead of
      // the tile's next scores (each takes 150 to 200 cycles even when it has
      // nothing to wait for: four of them behind P were 1700 of a step's 3950).
      for (int j = 0; j < n_kv && ok; ++j) {
        uint32_t vs;
        take(vs);
        if (j + 1 < n_kv) take(ks);
        if (!ok) break;
        for (int t = 0; t < 2; ++t) {
          if (j >= (t ? n1 : n0)) continue;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&o_ready[t], j & 1, FWD_SITE_OR)))) break;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&p_full[t], j & 1, FWD_SITE_P)))) break;
          tc_fence_after();
          pv(t, 0, vs, j > 0 ? 1u : 0u);
          pv(t, 1, vs, 1u);
          mma_commit_e(&pv_done[t], e);
          if (j == n_kv - 1) {
            mma_commit_e(&o_full[t], e);
          } else {
            qk(t, ks);
            mma_commit_e(&s_full[t], e);
          }
        }
        if (!ok) break;
        mma_commit_e(&kv_empty[vs], e);
        if (j + 1 < n_kv) mma_commit_e(&kv_empty[ks], e);
      }
      mma_commit_e(drain, e);
      mbar_wait(drain, 0, FWD_SITE_DRAIN);
      __syncwarp();
    }
  } else if (warp < 20) {
    regs_inc<96>();
    // ------------------------------------------------------------ softmax
    const int t = (warp - 4) >> 3;
    const int h = ((warp - 4) >> 2) & 1;
    const int n_t = t == 0 ? n0 : n1;
    const int r = 32 * (warp & 3) + (int)lane;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + lane_off + C::TM_S + 128 * t;
    const float sl2 = p.scale_log2;
    float* my_max = pmax_buf + (2 * t + h) * 128 + r;
    const float* other_max = pmax_buf + (2 * t + (h ^ 1)) * 128 + r;
    // the range's end, if this query row takes it
    const int b = seq_of_row(t, r);
    const int sees = b >= 0 && min(p.seq_lens[b], p.map.max_len) >= range_end ? range_end : 0;
    float m = -INFINITY, l = 0.f, lr = 0.f;
    bool ok = true;
    for (int j = 0; j < n_t; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(&s_full[t], j & 1, FWD_SITE_S));
      if (!ok) break;
      tc_fence_after();
      uint32_t sv[2][32];
      tmem_ld32(tS + 64 * h, sv[0]);
      tmem_ld32(tS + 64 * h + 32, sv[1]);
      tmem_ld_wait(sv[0]);
      tmem_ld_wait(sv[1]);
      const int limit = sees - (128 * (j0 + j) + 64 * h);  // rows of this half tile: [0, limit)
      if (limit < 64) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i >= limit) sv[c][i] = __float_as_uint(-INFINITY);
      }
      float mx2[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float a = fmax3(__uint_as_float(sv[c][0]), __uint_as_float(sv[c][1]), __uint_as_float(sv[c][2]));
        float bb = fmax3(__uint_as_float(sv[c][3]), __uint_as_float(sv[c][4]), __uint_as_float(sv[c][5]));
#pragma unroll
        for (int i = 6; i < 30; i += 4) {
          a = fmax3(a, __uint_as_float(sv[c][i]), __uint_as_float(sv[c][i + 1]));
          bb = fmax3(bb, __uint_as_float(sv[c][i + 2]), __uint_as_float(sv[c][i + 3]));
        }
        mx2[c] = fmax3(a, bb, fmaxf(__uint_as_float(sv[c][30]), __uint_as_float(sv[c][31])));
      }
      const float pm = fmaxf(mx2[0], mx2[1]);
      *my_max = pm;
      mbar_arrive(&mx_full[4 * t + (warp & 3)]);
      ok = __all_sync(0xffffffffu, mbar_wait(&mx_full[4 * t + (warp & 3)], j & 1, FWD_SITE_MX));
      if (!ok) break;
      const float mx = fmaxf(pm, *other_max);
      const float m_new = fmaxf(m, mx * sl2);
      const float alpha = m_new > m ? ex2(m - m_new) : 1.f;
      const float neg = (m_new == -INFINITY) ? 0.f : -m_new;
      const uint64_t scale2 = f2(sl2, sl2), neg2 = f2(neg, neg);
      uint64_t fsum0 = f2(0.f, 0.f), fsum1 = f2(0.f, 0.f), rsum0 = f2(0.f, 0.f), rsum1 = f2(0.f, 0.f);
      auto exp_pair = [&](uint32_t x, uint32_t y, uint64_t& fs, uint64_t& rs) -> uint32_t {
        const uint64_t arg = ffma2(f2(__uint_as_float(x), __uint_as_float(y)), scale2, neg2);
        float a, bb;
        f2split(arg, a, bb);
        a = ex2(a);
        bb = ex2(bb);
        fs = fadd2(fs, f2(a, bb));
        const uint32_t pk = pack2<BF16>(a, bb);
        rs = fadd2(rs, widen2<BF16>(pk));
        return pk;
      };
      uint32_t pk[32];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        pk[i] = exp_pair(sv[0][2 * i], sv[0][2 * i + 1], fsum0, rsum0);
        pk[16 + i] = exp_pair(sv[1][2 * i], sv[1][2 * i + 1], fsum1, rsum1);
      }
      tmem_st32(tS + 32 * h, pk);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[t]);
      float f0, f1, f2_, f3, r0, r1, r2, r3;
      f2split(fsum0, f0, f1);
      f2split(fsum1, f2_, f3);
      f2split(rsum0, r0, r1);
      f2split(rsum1, r2, r3);
      l = l * alpha + ((f0 + f1) + (f2_ + f3));
      lr = lr * alpha + ((r0 + r1) + (r2 + r3));
      m = m_new;
    }
    // ---- normalised fp32 parts and the log2 of the fp32 sums: each warp its 32
    // rows and half of the columns, through the tile buffers (free once every
    // product of both tiles is done) in rows 16 bytes apart from a bank
    // conflict, and out as one bulk copy per row half.  (Four warps storing
    // from registers, a row a lane, took 6.5 us.)
    if (ok && n_t > 0) {
      sum_buf[((2 * t + h) * 2 + 0) * 128 + r] = l;
      sum_buf[((2 * t + h) * 2 + 1) * 128 + r] = lr;
      mbar_arrive(&stats_ready[t]);
      ok = __all_sync(0xffffffffu, mbar_wait(&stats_ready[t], 0, FWD_SITE_ST) && mbar_wait(&o_full[0], 0, FWD_SITE_O) &&
                                       (!has_t1 || mbar_wait(&o_full[1], 0, FWD_SITE_O)));
      if (ok) {
        tc_fence_after();
        const float lt = l + sum_buf[((2 * t + (h ^ 1)) * 2 + 0) * 128 + r];
        const float lrt = lr + sum_buf[((2 * t + (h ^ 1)) * 2 + 1) * 128 + r];
        const float inv = lrt == 0.f ? 0.f : 1.f / lrt;
        constexpr int HALF = D / 2, STRIDE = D * 4 + 16;
        static_assert(256 * STRIDE <= C::BAR_OFF, "parts fit the tile buffers");
        uint8_t* out = smem + (128 * t + r) * STRIDE + h * HALF * 4;
        const uint32_t tO = tmem + lane_off + C::TM_O + D * t + HALF * h;
#pragma unroll
        for (int c = 0; c < HALF / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(tO + 32 * c, ov);
          tmem_ld_wait(ov);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            reinterpret_cast<float4*>(out)[8 * c + i] =
                make_float4(__uint_as_float(ov[4 * i]) * inv, __uint_as_float(ov[4 * i + 1]) * inv,
                            __uint_as_float(ov[4 * i + 2]) * inv, __uint_as_float(ov[4 * i + 3]) * inv);
        }
        fence_proxy_async_smem();
        if (b >= 0) {
          const size_t row = (size_t)split * p.B * p.Hq + (size_t)b * p.Hq + kvh * p.G + r % p.G;
          bulk_store(p.pre_o + row * D + h * HALF, out, HALF * 4);
          if (h == 0) p.pre_lse[row] = lt == 0.f ? -INFINITY : m + __log2f(lt);
        }
        bulk_store_wait();
      }
    }
  } else {
    regs_dec<48>();
    // ------------------------------------------------------------ correction
    const int r = 32 * (warp & 3) + (int)lane;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const float sl2 = p.scale_log2;
    float m_row0 = -INFINITY, m_row1 = -INFINITY;
    bool ok = true;
    for (int j = 0; j < n_kv && ok; ++j) {
      for (int t = 0; t < 2; ++t) {
        if (j >= (t ? n1 : n0)) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(&mx_full[4 * t + (warp & 3)], j & 1, FWD_SITE_MX));
        if (!ok) break;
        const float mx = fmaxf(pmax_buf[(2 * t) * 128 + r], pmax_buf[(2 * t + 1) * 128 + r]);
        const float m = t ? m_row1 : m_row0;
        const float m_new = fmaxf(m, mx * sl2);
        const float alpha = m_new > m ? ex2(m - m_new) : 1.f;
        if (t) m_row1 = m_new; else m_row0 = m_new;
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[t], (j - 1) & 1, FWD_SITE_PV));
          if (!ok) break;
          tc_fence_after();
          const uint32_t tO = tmem + lane_off + C::TM_O + D * t;
          const uint64_t alpha2 = f2(alpha, alpha);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t ov[16];
            tmem_ld16(tO + 16 * c, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float x, y;
              f2split(fmul2(f2(__uint_as_float(ov[2 * i]), __uint_as_float(ov[2 * i + 1])), alpha2), x, y);
              ov[2 * i] = __float_as_uint(x);
              ov[2 * i + 1] = __float_as_uint(y);
            }
            tmem_st16(tO + 16 * c, ov);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(&o_ready[t]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa
