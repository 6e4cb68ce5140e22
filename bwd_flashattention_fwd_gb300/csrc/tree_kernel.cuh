// Attention of drafted tokens over a key/value cache and each other (tree
// attention), for sequences of unequal lengths.
//
//   s_tj = scale * q_t . k_j over the context (j < cache_len[b]) and the drafts
//   that t's mask row keeps; O_t = sum_j 2^(s'_tj - m) v_j / l, lse = m + log2 l,
//   with s' = s log2 e, m a running reference and l = sum_j 2^(s'_tj - m).
//
// Few query rows meet a long cache, so reading K and V once is the bound
// (4 D bytes per key and KV head).  Three choices follow from that.
//
// * Work is split over keys, evenly, whatever the lengths.  The G query heads
//   x T drafts of a KV head are consecutive rows of q and form one packed block
//   of R = G T rows.  A KV head's keys are a list of stages (64 keys, or 128), its drafts'
//   stages first; the lists of all KV heads form one list of N stages, which
//   the CTAs (one per SM) divide into equal ranges.  A range that holds a
//   whole KV head writes O and lse; a partial one writes (O / l, lse) in fp32
//   to the workspace, at most two per CTA, and attn_tree_combine_kernel merges
//   them.  Every CTA derives the same division from the lengths in device memory.
//
// * The tensor cores always compute 128 rows, so few rows leave lanes idle
//   unless they share the keys out: with R <= 32 the rows are loaded into all
//   four 32-lane quadrants (QS = 4) and each quadrant takes a quarter of a
//   stage's keys, with its own m, l and O; P is zero at the other quadrants'
//   keys, so O += P V keeps them apart.  R <= 64: two (QS = 2).  The quadrants
//   are merged when the range ends.  tree_plan has the rule and its figures.
//
// * More than 128 rows (NT = 2, D <= 128): a CTA takes 256 rows as two tiles
//   that share every stage, with a softmax warpgroup and an MMA warp each.
//   (With 128-key stages tensor memory holds one S buffer per tile, not two, and
//   products and softmax take turns: B16 T61 ragged 98.5 us, against 79.0 before the
//   mask and the combine kernel got faster.)
//   More than one block of rows: n_rb neighbouring CTAs walk the same keys
//   with different rows, so the keys come from memory once and then from L2.
//
// Warp roles: 4 NT softmax warps (thread = row of the tile = TMEM lane), one
// TMA producer, NT MMA issuers.  S has two buffers per tile, P is
// written over the S it came from, a row keeps its reference m until a stage
// raises its maximum by more than 8 (log2 units), so O is rescaled rarely;
// O / l and m + log2 l use the same reference.
//
// P is rounded to 16 bits because that is what the tensor cores multiply V by;
// l sums it unrounded.  The rounding is half a step of each p (2^-8 of it in
// bf16, 2^-11 in fp16): against 64 bits O is 1.1 to 1.4 times as far off as with
// P in 32 bits, whose only 16-bit rounding is O's own.  Two 16-bit parts of P
// would take it away for twice the products.  fp16 ends at 2^-25, where bf16
// goes on to 2^-133, and many light keys together weigh something: there P
// and l are kept times 2^7 (p <= 2^8 by the rule above, so 2^15 at most, in
// range), and a key counts in O down to 2^-32 of the row's reference.
//
// Rows of V behind the context's or the drafts' end share a stage with real
// ones and may hold anything: P is 0 there, but 0 * NaN is not, so the softmax
// warps clear them in shared memory before O += P V reads the stage.
//
// Measured (call and combine kernel, replayed): B4 32/8 heads T8 8192 keys
// D = 128 30.1 us for 134 MB (27 stages a CTA stream in 18.6 us, at the full copy
// rate; the rest is start, quadrant merge and combine); 131072 keys D = 256 85 us,
// 6.3 TB/s; B16 T61 ragged 70.2 us for 321 MB, which stream in 45 us, at the full rate too.
#pragma once

#include "cache.h"
#include "kernel_common.cuh"

namespace gbattn {

// What every block derives from the lengths.  The list that the CTAs divide
// counts units: a KV head's stages, and before them `extra` units for what a
// CTA spends on a head besides its stages (loading Q, merging and writing O):
// kTreeExtra, or a sixth of a CTA's range where that is less.
// pre[b]: units of one KV head of the sequences before b (pre[B] the total).
struct TreeTable {
  int extra;
  int pre[kTreeMaxB + 1];
  int len[kTreeMaxB];
  uint16_t tl[kTreeMaxB];
};
constexpr int kTreeStaticSmem = sizeof(TreeTable) + 4096;

template <int D, int QS, int NT>
struct TreeGeom {
  static constexpr int BK = tree_stage_keys(D, NT);  // keys per stage
  static constexpr int KPW = BK / QS;     // keys per softmax thread and stage,
  static constexpr int NV = KPW > 32 ? 32 : KPW;  // in NB blocks of NV
  static constexpr int NB = KPW / NV;
  static constexpr int ROWS = QS > 1 ? 128 / QS : 128 * NT;  // packed rows per CTA
  static constexpr int QROWS = 128 / QS;  // rows of a Q load
  static constexpr int NCH = n_chunks(D);
  static constexpr int Q_BYTES = NCH * 128 * 128;
  static constexpr int KV_BYTES = NCH * BK * 128;
  static constexpr int XCH_PITCH = 36;  // floats: 16-byte pieces of eight neighbouring rows fall into different banks
  static constexpr int XCH_BYTES = QS > 1 ? 128 * XCH_PITCH * 4 : 0;  // merging the quadrants' O
  static constexpr int AVAIL = kMaxDynSmem - kTreeStaticSmem - 1024 - NT * Q_BYTES - XCH_BYTES;
  static constexpr int SLOTS = AVAIL / KV_BYTES > 16 ? 16 : AVAIL / KV_BYTES;  // a K or a V tile each
  static constexpr int SMEM_BYTES = 1024 + NT * Q_BYTES + SLOTS * KV_BYTES + XCH_BYTES;
  static constexpr int O_W = D <= 128 ? 128 : 256;
  static constexpr int TMEM_COLS = NT * (O_W + 2 * BK) <= 256 ? 256 : 512;
  static constexpr int SOFTMAX_WARPS = 4 * NT;
  static constexpr int NUM_THREADS = 32 * (SOFTMAX_WARPS + 1 + NT);
  static constexpr float TAU = 8.0f;
  __host__ __device__ static constexpr int o_col(int t) { return t * O_W; }
  __host__ __device__ static constexpr int s_col(int t, int b) { return NT * O_W + (2 * t + b) * BK; }
  static_assert(NT * (O_W + 2 * BK) <= 512, "tensor memory budget");
  static_assert(SLOTS >= 4, "shared memory budget");  // K of two stages ahead of the oldest V
  static_assert(QS == 1 || NT == 1, "only a full tile comes in pairs");
};

// Lengths of sequence b, and the stages of one of its KV heads (the drafts' first, then the context's).
__device__ __forceinline__ void tree_lengths(const TreeParams& p, int b, int& len, int& tl) {
  len = min(max(p.cache_len[b], 0), p.Lk);
  tl = p.tree_len ? min(max(p.tree_len[b], 0), p.T) : p.T;
}
__device__ __forceinline__ int tree_stages(int len, int tl, int stage) {
  return tl == 0 ? 0 : (len + stage - 1) / stage + (tl + stage - 1) / stage;
}

// Fills the table: one warp for up to 32 sequences; for more, the whole block
// loads the lengths first (tree_lengths_of_all and a barrier).  Whatever
// follows needs a barrier, except in the calling warp.
__device__ __forceinline__ int tree_load(const TreeParams& p, TreeTable& tab, int b) {
  int len, tl;
  tree_lengths(p, b, len, tl);
  tab.len[b] = len;
  tab.tl[b] = static_cast<uint16_t>(tl);
  return tree_stages(len, tl, p.stage);
}
__device__ __forceinline__ void tree_lengths_of_all(const TreeParams& p, TreeTable& tab) {
  if (p.B <= 32) return;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) tab.pre[b + 1] = tree_load(p, tab, b);
  __syncthreads();
}
__device__ __forceinline__ void tree_table(const TreeParams& p, TreeTable& tab) {
  const int lane = threadIdx.x & 31;
  int mine = 0, all = 0;  // this lane's sequence (up to 32 of them); all stages of a KV head
  if (p.B > 32) {
    for (int b = lane; b < p.B; b += 32) all += tab.pre[b + 1];
  } else if (lane < p.B) {
    all = mine = tree_load(p, tab, lane);
  }
  all = __reduce_add_sync(0xffffffffu, all);
  const int extra = min(kTreeExtra, all * p.Hkv / (6 * p.n_groups));
  if (lane == 0) tab.extra = extra, tab.pre[0] = 0;
  int run = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    int x = b >= p.B ? 0 : p.B > 32 ? tab.pre[b + 1] : mine;
    if (x > 0) x += extra;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (b < p.B) tab.pre[b + 1] = run + x;
    run += __shfl_sync(0xffffffffu, x, 31);
  }
  __syncwarp();
}

// The sequence that unit x of the whole list belongs to: the largest b with pre[b] * Hkv <= x
// (pre[b] < pre[b + 1] there, as x is below the total).
__device__ __forceinline__ int tree_find(const int* pre, int B, int Hkv, int x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] * Hkv <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Units per CTA range.
__device__ __forceinline__ int tree_per(int total, int n_groups) { return (total + n_groups - 1) / n_groups; }

// Walks a CTA's range [lo, xe) of the list, one KV head at a time: the segment
// is stages j0 .. j1 - 1 of the n of head (b, hk).  A range that ends among a
// head's extra units leaves the head to the next one.
struct TreeWalk {
  const TreeTable& tab;
  int Hkv, lo, xe, s;
  int b, hk, n, j0, j1;
  bool more_;
  __device__ __forceinline__ TreeWalk(const TreeParams& p, const TreeTable& tab_, int group) : tab(tab_), Hkv(p.Hkv) {
    const int total = tab.pre[p.B] * p.Hkv, per = tree_per(total, p.n_groups);
    if (p.whole) {
      auto first = [&](int head) {
        const int i = head / Hkv;
        return i < p.B ? tab.pre[i] * Hkv + (head - i * Hkv) * (tab.pre[i + 1] - tab.pre[i]) : total;
      };
      lo = first(min(group * p.whole, p.B * Hkv));
      xe = first(min((group + 1) * p.whole, p.B * Hkv));
    } else {
      const long long from = static_cast<long long>(group) * per;
      lo = from < total ? static_cast<int>(from) : total;
      xe = from + per < total ? static_cast<int>(from + per) : total;
    }
    more_ = lo < xe;
    if (more_) {
      b = tree_find(tab.pre, p.B, p.Hkv, lo);
      hk = (lo - tab.pre[b] * Hkv) / (tab.pre[b + 1] - tab.pre[b]);
      set(lo);
    }
  }
  __device__ __forceinline__ bool more() const { return more_; }
  __device__ __forceinline__ void set(int x) {  // the segment that holds unit x
    const int units = tab.pre[b + 1] - tab.pre[b];
    s = tab.pre[b] * Hkv + hk * units;
    n = units - tab.extra;
    j0 = max(x - s - tab.extra, 0);
    j1 = min(xe - s, units) - tab.extra;
    more_ = j1 > j0;
  }
  __device__ __forceinline__ void next() {
    const int x = s + tab.extra + j1;
    more_ = x < xe;
    if (!more_) return;
    if (++hk == Hkv) {
      hk = 0;
      do ++b;
      while (tab.pre[b + 1] == tab.pre[b]);
    }
    set(x);
  }
  // the segment is the whole KV head
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == n; }
  // where a partial segment goes: 0 if it is the range's first, 1 behind another (cut off by the range's end)
  __device__ __forceinline__ int slot() const { return s > lo ? 1 : 0; }
};

// First partial row of (group, slot, row block): slot 0 holds the segment at
// the start of the group's range, slot 1 the one cut off by its end.  Its lse
// are consecutive; its O is kept for 32 rows at a time, as [D / 4][32 rows][4],
// so a warp whose lanes are rows stores and loads 512 consecutive bytes.
__device__ __forceinline__ size_t tree_slot_row(const TreeParams& p, int group, int slot, int rb, int rows) {
  return ((static_cast<size_t>(group) * 2 + slot) * p.n_rb + rb) * rows;
}

// see &= which of the N bytes mask[at], mask[at + 1], ... are not zero, 32 bits
// to a word; only the first `most` are needed, and the mask has n bytes.  The
// words that cover them are loaded together, each aligned (a mask row begins at
// any byte), so a stage waits for one latency.  (Rows read a byte per lane, 16
// at a time, and balloted took 18,000 clocks of a CTA's 100,000 at B16 T61.)
template <int N, int NB>
__device__ __forceinline__ void tree_mask_bits(const uint8_t* mask, size_t at, size_t n, int most, uint32_t (&see)[NB]) {
  constexpr int W = N / 4;
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(mask) + at) & 3u);
  uint32_t x[W + 1];
  if (at >= static_cast<size_t>(lead) && at - lead + 4 * (W + 1) <= n) {
    const uint32_t* word = reinterpret_cast<const uint32_t*>(mask + at - lead);
#pragma unroll
    for (int i = 0; i <= W; ++i) x[i] = 4 * i - lead < most ? word[i] : 0u;
#pragma unroll
    for (int i = 0; i < W; ++i) x[i] = __funnelshift_r(x[i], x[i + 1], 8 * lead);
  } else {  // at the mask's ends: byte by byte
#pragma unroll
    for (int i = 0; i < W; ++i) {
      x[i] = 0u;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (4 * i + c < most) x[i] |= static_cast<uint32_t>(mask[at + 4 * i + c]) << (8 * c);
    }
  }
#pragma unroll
  for (int h = 0; h < NB; ++h) {
    uint32_t bits = 0u;
#pragma unroll
    for (int i = 0; i < W / NB; ++i) {
      uint32_t y = x[h * (W / NB) + i];
      y |= y >> 4, y |= y >> 2, y |= y >> 1;            // bit 0 of a byte: any of its bits
      bits |= (((y & 0x01010101u) * 0x10204080u) >> 28) << (4 * i);  // the four of them side by side
    }
    see[h] &= bits;
  }
}

constexpr int kTreeReady = 3;  // named barrier (1 and 2: the tiles' softmax warps)

template <int D, bool BF16, int QS, int NT>
__global__ void __launch_bounds__(TreeGeom<D, QS, NT>::NUM_THREADS, 1)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKn,
                     const __grid_constant__ CUtensorMap tmVn, const TreeParams p) {
  using Gm = TreeGeom<D, QS, NT>;
  using E = Elem<BF16>;
  constexpr int BK = Gm::BK, NCH = Gm::NCH, SL = Gm::SLOTS, KPW = Gm::KPW, NV = Gm::NV, NB = Gm::NB;
  constexpr int PRODUCER = Gm::SOFTMAX_WARPS;
  // P and l are multiplied by 2^LIFT (see the head of this file)
  constexpr float LIFT = BF16 ? 0.f : 7.f, UNLIFT = BF16 ? 1.f : 1.f / 128;
  constexpr int kWait = wait_code<94>();  // every bounded wait of this kernel

  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_q, bar_qfree, bar_full[SL], bar_empty[SL], bar_sfull[NT][2], bar_pready[NT][2],
      bar_odone[NT][2], bar_mfin[NT];
  __shared__ TreeTable tab;
  __shared__ float2 ml[128 * NT];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = sbase;                  // tile t at sQ + t * Q_BYTES
  const uint32_t sKV = sQ + NT * Gm::Q_BYTES;  // slot s of the K / V ring at sKV + s * KV_BYTES
  const uint32_t sX = sKV + SL * Gm::KV_BYTES;
  const int group = blockIdx.x / p.n_rb, rb = blockIdx.x - group * p.n_rb;
  const WaitGuard g{&abort_flag, p.status, p.limit_ns};

  // The producer warp sets up the barriers and the division and goes on to its
  // loads at once; the others meet when that and tensor memory are ready.
  if (warp == PRODUCER) {
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmKn);
      tma_prefetch_desc(&tmVn);
      abort_flag = 0;
      mbar_init(smem_u32(&bar_q), 1);
      mbar_init(smem_u32(&bar_qfree), NT);
      for (int s = 0; s < SL; ++s) {
        mbar_init(smem_u32(&bar_full[s]), 1);
        mbar_init(smem_u32(&bar_empty[s]), NT);
      }
      for (int t = 0; t < NT; ++t) {
        for (int i = 0; i < 2; ++i) {
          mbar_init(smem_u32(&bar_sfull[t][i]), 1);
          mbar_init(smem_u32(&bar_pready[t][i]), 128);
          mbar_init(smem_u32(&bar_odone[t][i]), 1);
        }
        mbar_init(smem_u32(&bar_mfin[t]), 1);
      }
      fence_mbar_init();
    }
    __syncwarp();
  }
  grid_dependency_wait();  // the kernels before this one are complete
  // (Tensor memory is allocated behind that: a kernel before this one whose
  // CTA has not allocated its own yet cannot be left without.)
  if (warp == PRODUCER + 1) {
    tmem_alloc(smem_u32(&tmem_slot), Gm::TMEM_COLS);
    tmem_relinquish();
  }
  tree_lengths_of_all(p, tab);
  if (warp == PRODUCER) {
    tree_table(p, tab);
    named_bar_arrive(kTreeReady, Gm::NUM_THREADS);
  } else {
    tc_fence_before_sync();
    named_bar_sync(kTreeReady, Gm::NUM_THREADS);
    tc_fence_after_sync();
    // The combine kernel may start; it waits for this grid before it reads
    // partials.  (After tensor memory is allocated: a dependent that wants
    // some cannot get in front.)
    if (threadIdx.x == 0) grid_launch_dependents();
  }
  TreeWalk w(p, tab, group);

  if (warp == PRODUCER) {
    // ---------------- TMA producer (whole warp, one elected lane issues) ----------------
    // K and V tiles go into one ring in the order the MMA warps use them up:
    // K0, K1, V0, K2, V1, ..., K(n-1), V(n-2), V(n-1).
    RingPos<SL> st;
    int issued = 0, nq = 0;
    bool q_due = false;  // the segment's Q is still to be loaded (z, below)
    int z = 0;
    auto load_q = [&]() {
      mbar_arrive_expect_tx_w(smem_u32(&bar_q), NT * Gm::Q_BYTES);
      for (int t = 0; t < NT; ++t)
        for (int c = 0; c < NCH; ++c)
          for (int i = 0; i < QS; ++i)
            tma_load_3d_w(sQ + t * Gm::Q_BYTES + c * 128 * 128 + i * Gm::QROWS * 128, &tmQ, smem_u32(&bar_q), c * 64,
                          rb * Gm::ROWS + t * 128, z);
      ++nq;
      q_due = false;
    };
    // Q's buffer is free once the previous segment's S products, its only
    // readers, are complete.  The next segment's K and V do not wait for that:
    // while a slot is awaited, Q is loaded as soon as it can be.
    auto try_q = [&](bool block) {
      if (!q_due) return;
      if (nq > 0) {
        if (block) mbar_wait(smem_u32(&bar_qfree), (nq - 1) & 1, g, kWait);
        else if (!__all_sync(0xffffffffu, mbar_test(smem_u32(&bar_qfree), (nq - 1) & 1))) return;
      }
      if (!__any_sync(0xffffffffu, abort_flag)) load_q();
    };
    auto load_tile = [&](const CUtensorMap* map, int row) {
      const int s = st.slot;
      if (issued >= SL) {
        if (q_due) {  // whichever comes first; the limit is mbar_wait's, below
          const uint64_t t0 = global_timer_ns();
          while (q_due && !__any_sync(0xffffffffu, abort_flag || global_timer_ns() - t0 > p.limit_ns) &&
                 !__all_sync(0xffffffffu, mbar_test(smem_u32(&bar_empty[s]), st.phase ^ 1u)))
            try_q(false);
        }
        mbar_wait(smem_u32(&bar_empty[s]), st.phase ^ 1u, g, kWait);
      }
      if (__any_sync(0xffffffffu, abort_flag)) return;  // no further copy is issued
      const uint32_t bar = smem_u32(&bar_full[s]);
      mbar_arrive_expect_tx_w(bar, Gm::KV_BYTES);
      for (int c = 0; c < NCH; ++c) tma_load_3d_w(sKV + s * Gm::KV_BYTES + c * BK * 128, map, bar, c * 64, row, z);
      st.next();
      ++issued;
    };
    for (; w.more() && !abort_flag; w.next()) {
      z = w.b * p.Hkv + w.hk;
      q_due = true;
      try_q(false);
      const int nd = (tab.tl[w.b] + BK - 1) / BK;  // draft stages
      const int n = w.j1 - w.j0;
      auto row_of = [&](int j) { return j < nd ? j * BK : (j - nd) * BK; };
      load_tile(w.j0 < nd ? &tmKn : &tmK, row_of(w.j0));
      for (int i = 1; i <= n && !abort_flag; ++i) {
        const int jk = w.j0 + i, jv = jk - 1;
        if (i < n) load_tile(jk < nd ? &tmKn : &tmK, row_of(jk));
        load_tile(jv < nd ? &tmVn : &tmV, row_of(jv));
        try_q(false);
      }
      try_q(true);
    }
    // the last SL issued tiles (each slot holds at most one copy in flight) and the last Q
    for (int u = 0; u < SL && u < issued; ++u) {
      if (st.slot == 0) st.phase ^= 1u;
      st.slot = (st.slot == 0 ? SL : st.slot) - 1;
      mbar_wait_drain(smem_u32(&bar_full[st.slot]), st.phase);
    }
    if (nq > 0) mbar_wait_drain(smem_u32(&bar_q), (nq - 1) & 1);
    __syncwarp();
  } else if (warp > PRODUCER) {
    const uint32_t tmem = tmem_slot;
    // ---------------- MMA issuer of tile t ----------------
    const int t = warp - PRODUCER - 1;
    constexpr uint32_t IDESC_QK = make_idesc_f16(128, BK, BF16, false, false);
    constexpr uint32_t IDESC_PV = make_idesc_f16(128, D, BF16, false, true);
    const uint64_t dQd = make_sdesc_sw128(sQ + t * Gm::Q_BYTES, 16, 1024);      // this tile's Q, K-major
    const uint64_t dK = make_sdesc_sw128(sKV, 16, 1024);       // slot 0 as K, K-major
    const uint64_t dV = make_sdesc_sw128(sKV, BK * 128, 1024);  // slot 0 as V, MN-major
    RingPos<SL> st;
    int ts = 0, tp = 0;  // stages (all segments) of the next S and of the next P V
    auto issue_s = [&](bool last) {
      const int s = st.slot, bb = ts & 1;
      mbar_wait(smem_u32(&bar_full[s]), st.phase, g, kWait);
      st.next();
      ++ts;
      __syncwarp();
      tc_fence_after_sync();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t qo = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
        const uint32_t ko = s * Gm::KV_BYTES + (kk >> 2) * (BK * 128) + (kk & 3) * 32;
        mma_ss_w(tmem + Gm::s_col(t, bb), sdesc_add(dQd, qo), sdesc_add(dK, ko), IDESC_QK, kk > 0 ? 1u : 0u);
      }
      mma_commit_w(smem_u32(&bar_sfull[t][bb]));
      mma_commit_w(smem_u32(&bar_empty[s]));
      if (last) mma_commit_w(smem_u32(&bar_qfree));  // last read of this segment's Q
    };
    int r = 0;
    for (; w.more(); w.next(), ++r) {
      const int n = w.j1 - w.j0;
      mbar_wait(smem_u32(&bar_q), r & 1, g, kWait);
      __syncwarp();
      tc_fence_after_sync();
      issue_s(n == 1);
      if (n > 1) issue_s(n == 2);
      for (int j = 0; j < n; ++j) {
        const int s = st.slot, bb = tp & 1;
        mbar_wait(smem_u32(&bar_full[s]), st.phase, g, kWait);
        mbar_wait(smem_u32(&bar_pready[t][bb]), (tp >> 1) & 1, g, kWait);
        st.next();
        ++tp;
        __syncwarp();
        tc_fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          mma_ts_w(tmem + Gm::o_col(t), tmem + Gm::s_col(t, bb) + kk * 8,
                   sdesc_add(dV, s * Gm::KV_BYTES + kk * 2048), IDESC_PV, (j > 0 || kk > 0) ? 1u : 0u);
        mma_commit_w(smem_u32(&bar_empty[s]));
        mma_commit_w(smem_u32(&bar_odone[t][bb]));
        // S of stage j + 2 goes over P of stage j, which the products above read (issue order)
        if (j + 2 < n) issue_s(j + 3 == n);
      }
    }
    // every MMA this warp issued is complete before tensor memory is released
    mma_commit_w(smem_u32(&bar_mfin[t]));
    mbar_wait_drain(smem_u32(&bar_mfin[t]), 0);
    __syncwarp();
  } else {
    const uint32_t tmem = tmem_slot;
    // ---------------- softmax warps ----------------
    const int t = warp >> 2, quad = warp & 3;
    const int kq = QS == 4 ? quad : QS == 2 ? quad >> 1 : 0;  // which keys of a stage
    const int lrow = QS == 4 ? lane : QS == 2 ? (quad & 1) * 32 + lane : t * 128 + quad * 32 + lane;  // row of the CTA's block
    const int c0 = kq * KPW;
    const int R = p.G * p.T;
    const int row = rb * Gm::ROWS + lrow;  // packed row of the KV head
    const int trow = row % p.T;            // its draft
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t o_col = tmem + lanes + Gm::o_col(t);
    const float sl2 = p.scale_log2;
    const size_t n_mask = static_cast<size_t>(p.B) * p.T * p.T;
    // extents for the debug build's index checks: rows of o / lse, and of the partials
    [[maybe_unused]] const size_t n_rows = static_cast<size_t>(p.B) * p.Hkv * R;
    [[maybe_unused]] const size_t n_parts = static_cast<size_t>(p.n_groups) * 2 * p.n_rb * Gm::ROWS;
    // KV heads without a stage (no drafts): their rows see nothing
    for (int x = blockIdx.x; x < p.B * p.Hkv; x += gridDim.x) {
      if (tab.pre[x / p.Hkv + 1] != tab.pre[x / p.Hkv]) continue;
      if (!dbg_in_range(static_cast<size_t>(x) * R, R, n_rows, p.status, 62)) continue;
      uint4* o = reinterpret_cast<uint4*>(static_cast<typename E::T*>(p.o) + static_cast<size_t>(x) * R * D);
      for (long long i = threadIdx.x; i < static_cast<long long>(R) * (D / 8); i += 128 * NT) o[i] = make_uint4(0, 0, 0, 0);
      for (int i = threadIdx.x; i < R; i += 128 * NT) p.lse[static_cast<size_t>(x) * R + i] = INFINITY;
    }
    // O += P V of stage k is complete.  (One barrier for even and one for odd
    // stages: when stage k's P has just been handed over, the product of k - 1
    // may still run, and a single barrier's parity could not tell; k - 2 is
    // complete, S of stage k was issued behind it.)
    auto o_done = [&](int k) { mbar_wait(smem_u32(&bar_odone[t][k & 1]), (k >> 1) & 1, g, kWait); };
    int ts = 0;  // stages (all segments) so far
    for (; w.more(); w.next()) {
      const int len = tab.len[w.b], tl = tab.tl[w.b];
      const int ts0 = ts, n = w.j1 - w.j0;
      const int nd = (tl + BK - 1) / BK;
      float m = -INFINITY, l = 0.f;
      for (int j = w.j0; j < w.j1; ++j, ++ts) {
        const bool draft = j < nd;
        const int k0 = draft ? j * BK : (j - nd) * BK;
        const int valid = min((draft ? tl : len) - k0, BK);  // keys of the stage that exist
        // which of this thread's keys its row sees, NV bits at a time
        uint32_t see[NB];
        auto first_n = [&](int n) {  // the first n of them
#pragma unroll
          for (int h = 0; h < NB; ++h) {
            const int m = n - h * NV;
            see[h] = m <= 0 ? 0u : m >= 32 ? ~0u : (1u << m) - 1u;
          }
        };
        if (draft && p.mask) {
          // bytes of the lane's own mask row from this stage's keys on (only the first `most` of them count)
          const int most = min(valid - c0, KPW);
          const size_t at = (static_cast<size_t>(w.b) * p.T + trow) * p.T + k0 + c0;
          first_n(most);
          if (most > 0 && dbg_in_range(at, most, n_mask, p.status, 63)) tree_mask_bits<KPW, NB>(p.mask, at, n_mask, most, see);
        } else {
          first_n(draft ? min(valid - c0, trow - (k0 + c0) + 1) : valid - c0);
        }
        const int bb = ts & 1;
        const uint32_t s_col = tmem + lanes + Gm::s_col(t, bb);
        mbar_wait(smem_u32(&bar_sfull[t][bb]), (ts >> 1) & 1, g, kWait);
        if (valid < BK) {
          // V rows of no key: cleared, P = 0 does not hide a NaN there.  V of
          // the segment's stage i is tile 2 i + 2 of its ring order, the last one 2 n - 1.
          const int i = j - w.j0;
          const int tile = 2 * ts0 + (i == n - 1 ? 2 * n - 1 : 2 * i + 2);
          const int s = tile % SL;
          mbar_wait(smem_u32(&bar_full[s]), (tile / SL) & 1, g, kWait);
          const uint32_t sV = sKV + s * Gm::KV_BYTES;
          const int pieces = (BK - valid) * 8;
          for (int x = threadIdx.x & 127; x < NCH * pieces; x += 128) {
            const int c = x / pieces, y = x - c * pieces;
            st_shared_v4(sV + c * BK * 128 + valid * 128 + y * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        tc_fence_after_sync();
        uint32_t v[NB][NV];
#pragma unroll
        for (int h = 0; h < NB; ++h) {
          if constexpr (NV == 32) tmem_ld32(s_col + c0 + 32 * h, v[h]);
          else tmem_ld16(s_col + c0, v[h]);
        }
        tmem_ld_wait(v[0]);
#pragma unroll
        for (int h = 1; h < NB; ++h) reg_fence(v[h]);
        if (draft || valid < BK) {
#pragma unroll
          for (int h = 0; h < NB; ++h)
#pragma unroll
            for (int i = 0; i < NV; ++i)
              if (!((see[h] >> i) & 1u)) v[h][i] = __float_as_uint(-INFINITY);
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int h = 0; h < NB; ++h)
#pragma unroll
          for (int i = 0; i < NV; i += 2)
            mx[(i >> 1) & 3] = fmax3(mx[(i >> 1) & 3], __uint_as_float(v[h][i]), __uint_as_float(v[h][i + 1]));
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
        const float m_new = fmaxf(m, mt);
        if (__any_sync(0xffffffffu, m_new > m + Gm::TAU)) {
          // (a lane that has seen no key yet stays at -inf with l = 0 and O = 0)
          const float alpha = m_new == -INFINITY ? 1.f : ex2_approx(m - m_new);
          m = m_new;
          l *= alpha;
          if (j > w.j0) {
            o_done(ts - 1);  // O up to the stage before
            __syncwarp();
            tc_fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t rr[32];
              tmem_ld32(o_col + c * 32, rr);
              tmem_ld_wait(rr);
#pragma unroll
              for (int i = 0; i < 32; ++i) rr[i] = __float_as_uint(__uint_as_float(rr[i]) * alpha);
              tmem_st32(o_col + c * 32, rr);
            }
          }
        }
        const float mu = m == -INFINITY ? 0.f : m - LIFT;
        const uint64_t sl2x2 = f2_pack(sl2, sl2), nm2 = f2_pack(-mu, -mu);
        uint64_t sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
        uint32_t pk[NB][NV / 2];
#pragma unroll
        for (int h = 0; h < NB; ++h)
#pragma unroll
          for (int i = 0; i < NV / 2; ++i) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(v[h][2 * i]), __uint_as_float(v[h][2 * i + 1])), sl2x2, nm2), x0,
                      x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            sum[i & 1] = f2_add(sum[i & 1], f2_pack(p0, p1));
            pk[h][i] = E::pack(p0, p1);
          }
        {
          float s0, s1;
          f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
        }
        // P over the stage's S: pairs of keys, zeros at the other quadrants' keys
        uint32_t zero[NV / 2];
#pragma unroll
        for (int i = 0; i < NV / 2; ++i) zero[i] = 0u;
#pragma unroll
        for (int i = 0; i < QS; ++i)
#pragma unroll
          for (int h = 0; h < NB; ++h) {
            const uint32_t col = s_col + i * (KPW / 2) + h * 16;
            if constexpr (NV == 32) {
              if (i == kq) tmem_st16(col, pk[h]);
              else tmem_st16(col, zero);
            } else {
              if (i == kq) tmem_st8(col, pk[h]);
              else tmem_st8(col, zero);
            }
          }
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(smem_u32(&bar_pready[t][bb]));
      }
      // ---------------- end of the segment: merge the quadrants, write out ----------------
      const int me = threadIdx.x;  // 128 t + thread of the tile
      float f = 1.f;               // this lane's O counts f times
      if constexpr (QS > 1) {
        ml[me] = make_float2(m, l);
        named_bar_sync(1 + t, 128);
        float M = -INFINITY;
#pragma unroll
        for (int i = 0; i < QS; ++i) M = fmaxf(M, ml[i * Gm::QROWS + lrow].x);
        float L = 0.f;
#pragma unroll
        for (int i = 0; i < QS; ++i) {
          const float2 o = ml[i * Gm::QROWS + lrow];
          L += o.y == 0.f ? 0.f : o.y * ex2_approx(o.x - M);
        }
        f = l == 0.f ? 0.f : ex2_approx(m - M);
        m = M;
        l = L;
      }
      const bool live = row < R && trow < tl;
      const bool empty = !live || l == 0.f;  // (l NaN: the row's own scores are, and so is O)
      const float inv = empty ? 0.f : f / l;
      const bool whole = w.whole();
      const size_t grow = (static_cast<size_t>(w.b) * p.Hkv + w.hk) * R + row;  // row of o and lse
      const size_t prow = tree_slot_row(p, group, w.slot(), rb, Gm::ROWS) + lrow;  // row of the partials
      o_done(ts - 1);
      __syncwarp();
      tc_fence_after_sync();
      const bool mine = row < R && (whole ? dbg_in_range(grow, 1, n_rows, p.status, 64)
                                          : dbg_in_range(prow, 1, n_parts, p.status, 65));
      if (kq == 0 && mine) {
        const float lse = m + log2f(l * UNLIFT);
        if (whole) p.lse[grow] = empty ? INFINITY : lse;
        else p.part_lse[prow] = empty ? -INFINITY : lse;
      }
      typename E::T* orow = static_cast<typename E::T*>(p.o) + grow * D;
      float* prt = p.part + (prow - lrow % 32) * D + (lrow % 32) * 4;  // 4 columns every 128 floats
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t rr[32];
        tmem_ld32(o_col + c * 32, rr);
        tmem_ld_wait(rr);
        if constexpr (QS == 1) {
          if (empty) {
#pragma unroll
            for (int i = 0; i < 32; ++i) rr[i] = 0u;
          }
          if (mine) {
            const float mul = empty ? 1.f : inv;
            if (whole) store_row32<BF16>(orow + c * 32, rr, mul);
            else
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float4*>(prt + (c * 8 + i) * 128) =
                    make_float4(__uint_as_float(rr[4 * i]) * mul, __uint_as_float(rr[4 * i + 1]) * mul,
                                __uint_as_float(rr[4 * i + 2]) * mul, __uint_as_float(rr[4 * i + 3]) * mul);
          }
        } else {
          constexpr int W = 32 / QS;  // columns per thread once merged
          const bool drop = empty || f == 0.f;
          const uint32_t own = sX + (kq * Gm::QROWS + lrow) * (Gm::XCH_PITCH * 4);
#pragma unroll
          for (int i = 0; i < 32; ++i) rr[i] = drop ? 0u : __float_as_uint(__uint_as_float(rr[i]) * inv);
#pragma unroll
          for (int i = 0; i < 8; ++i) st_shared_v4(own + i * 16, rr[4 * i], rr[4 * i + 1], rr[4 * i + 2], rr[4 * i + 3]);
          named_bar_sync(1 + t, 128);
          float acc[W];
#pragma unroll
          for (int i = 0; i < W; ++i) acc[i] = 0.f;
#pragma unroll
          for (int k = 0; k < QS; ++k)
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
              const uint4 x = ld_shared_v4(sX + (k * Gm::QROWS + lrow) * (Gm::XCH_PITCH * 4) + kq * W * 4 + i * 16);
              acc[4 * i] += __uint_as_float(x.x);
              acc[4 * i + 1] += __uint_as_float(x.y);
              acc[4 * i + 2] += __uint_as_float(x.z);
              acc[4 * i + 3] += __uint_as_float(x.w);
            }
          if (mine) {
            if (whole) {
              uint4* d = reinterpret_cast<uint4*>(orow + c * 32 + kq * W);
#pragma unroll
              for (int i = 0; i < W / 8; ++i)
                d[i] = make_uint4(E::pack(acc[8 * i], acc[8 * i + 1]), E::pack(acc[8 * i + 2], acc[8 * i + 3]),
                                  E::pack(acc[8 * i + 4], acc[8 * i + 5]), E::pack(acc[8 * i + 6], acc[8 * i + 7]));
            } else {
#pragma unroll
              for (int i = 0; i < W / 4; ++i)
                *reinterpret_cast<float4*>(prt + (c * 8 + kq * (W / 4) + i) * 128) =
                    make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
            }
          }
          named_bar_sync(1 + t, 128);
        }
      }
      // the next segment's first P V overwrites O after this warp's next P arrival
      tc_fence_before_sync();
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == PRODUCER + 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_slot, Gm::TMEM_COLS);
  }
}

// Merges the partials of the KV heads that more than one CTA worked on.  With
// partial lse L_s and O_s: M = max L_s, w_s = 2^(L_s - M), O = sum w_s O_s /
// sum w_s, lse = M + log2 sum w_s.  Lane = row, QT times 4 columns per thread; NS warps
// share a head's partials out and are merged, in order, by the same rule.
// Launched as a programmatic dependent: the blocks derive the
// division while the attention kernel runs, then walk the (head, 32 rows,
// 32 QT / NS columns) tasks.
template <int D, bool BF16, int NS, int QT>
__global__ void __launch_bounds__(256) attn_tree_combine_kernel(const TreeParams p, int rows) {
  using E = Elem<BF16>;
  // QT column quads per thread, QPB quads at a time per block, QB blocks per row group
  constexpr int QPB = 8 / NS, QB = D / 4 / (QPB * QT), U = NS == 1 ? 3 : 4;
  static_assert(QB * QPB * QT * 4 == D, "whole blocks per row");
  __shared__ TreeTable tab;
  __shared__ float sM[8][32], sden[8][32];
  __shared__ float4 so[NS > 1 ? QT : 1][8][32];
  tree_lengths_of_all(p, tab);
  if (threadIdx.x < 32) tree_table(p, tab);
  __syncthreads();
  const int* pre = tab.pre;
  const int per = tree_per(pre[p.B] * p.Hkv, p.n_groups);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % NS;
  const int R = p.G * p.T, rgs = (R + 31) / 32;
  const long long tasks = static_cast<long long>(p.B) * p.Hkv * rgs * QB;
  grid_dependency_wait();  // the partials are written (and the whole call ends behind them)
  if (threadIdx.x == 0) grid_launch_dependents();
  for (long long task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int head = static_cast<int>(task / (rgs * QB)), rest = static_cast<int>(task % (rgs * QB));
    const int rg = rest / QB, q = (rest - rg * QB) * QPB * QT + warp / NS;  // and q + QPB, ...
    const int b = head / p.Hkv, hk = head - b * p.Hkv;
    const int n = pre[b + 1] - pre[b];
    const int s = pre[b] * p.Hkv + hk * n;  // the head's units; its stages begin at s + extra
    const int g0 = (s + tab.extra) / per, ng = n > 0 ? (s + n - 1) / per - g0 + 1 : 0;
    if (ng < 2) continue;  // written by its CTA (the same for the whole block)
    const int row = rg * 32 + lane, rb = rg * 32 / rows, r0 = rg * 32 - rb * rows;
    const int first = s > g0 * per ? 1 : 0;  // slot of the head's first partial
    auto part_row = [&](int i) { return tree_slot_row(p, g0 + i, i == 0 ? first : 0, rb, rows) + r0; };
    float M = -INFINITY, den = 0.f;
    float4 acc[QT];
#pragma unroll
    for (int c = 0; c < QT; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto scale = [](float4& y, float a) { y.x *= a, y.y *= a, y.z *= a, y.w *= a; };
    auto add = [](float4& y, float a, const float4& x) {
      y.x = fmaf(a, x.x, y.x), y.y = fmaf(a, x.y, y.y), y.z = fmaf(a, x.z, y.z), y.w = fmaf(a, x.w, y.w);
    };
    if (row < R) {
      // U partials at a time, all their loads in flight
      for (int i = sub; i < ng; i += U * NS) {
        float L[U];
        float4 x[U][QT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          L[u] = -INFINITY;
          if (i + u * NS < ng && dbg_in_range(part_row(i + u * NS), 32, static_cast<size_t>(p.n_groups) * 2 * p.n_rb * rows,
                                              p.status, 66)) {
            const size_t r = part_row(i + u * NS);
            L[u] = p.part_lse[r + lane];
#pragma unroll
            for (int c = 0; c < QT; ++c)
              x[u][c] = *reinterpret_cast<const float4*>(p.part + r * D + (q + c * QPB) * 128 + lane * 4);
          }
        }
        float Mn = M;
#pragma unroll
        for (int u = 0; u < U; ++u) Mn = fmaxf(Mn, L[u]);
        const float a = M == -INFINITY ? 0.f : exp2f(M - Mn);
        den *= a;
#pragma unroll
        for (int c = 0; c < QT; ++c) scale(acc[c], a);
        M = Mn;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (L[u] == -INFINITY) continue;
          const float wgt = exp2f(L[u] - M);
          den += wgt;
#pragma unroll
          for (int c = 0; c < QT; ++c) add(acc[c], wgt, x[u][c]);
        }
      }
    }
    if constexpr (NS > 1) {
      sM[warp][lane] = M, sden[warp][lane] = den;
#pragma unroll
      for (int c = 0; c < QT; ++c) so[c][warp][lane] = acc[c];
      __syncthreads();
      if (sub == 0) {
        for (int k = 1; k < NS; ++k) M = fmaxf(M, sM[warp + k][lane]);
        den = 0.f;
#pragma unroll
        for (int c = 0; c < QT; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < NS; ++k) {
          const float d = sden[warp + k][lane];
          const float wgt = d == 0.f ? 0.f : exp2f(sM[warp + k][lane] - M);
          den = fmaf(wgt, d, den);
#pragma unroll
          for (int c = 0; c < QT; ++c) add(acc[c], wgt, so[c][warp + k][lane]);
        }
      }
    }
    const size_t grow = static_cast<size_t>(head) * R + row;
    if (row < R && sub == 0 && dbg_in_range(grow, 1, static_cast<size_t>(p.B) * p.Hkv * R, p.status, 67)) {
      const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
      for (int c = 0; c < QT; ++c) {
        uint2 o;
        o.x = E::pack(acc[c].x * inv, acc[c].y * inv), o.y = E::pack(acc[c].z * inv, acc[c].w * inv);
        *reinterpret_cast<uint2*>(static_cast<typename E::T*>(p.o) + grow * D + (q + c * QPB) * 4) = o;
      }
      if (q == 0) p.lse[grow] = den == 0.f ? INFINITY : M + log2f(den);
    }
    if constexpr (NS > 1) __syncthreads();  // before the next task's values
  }
}

}  // namespace gbattn
