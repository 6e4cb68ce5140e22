// Accumulated attention weight of every cached key:
//   weight_out[j] = weight[j] + sum over the rows r that see j of 2^(s'_rj - lse_r),
//   s' = scale log2 e q_r . k_j.
//
// Keys are the rows of the products (S^T = K Q^T, thread = key = TMEM lane), so
// a key's sum stays in its thread, in a fixed order and without atomics.  A
// step's terms are summed apart from the running total, which keeps sums over
// tens of thousands of rows exact to a few ulp.
//
// Rows: the G query heads x Lq rows of a KV head, packed (consecutive in q and
// lse) where Lq is small or the limits are per row, else head by head.
// Each row has a limit (keys j < limit are seen) and -lse, in shared memory.
// A row of the padding (zero q, as loads past the end read zeros) has
// -lse = -inf and limit 0, but does not make a tile masked by itself; a row
// whose lse is +inf, or whose limit is 0, may hold anything and does.
//
// Two kernels share this:
// * few rows (G Lq <= 128): the rows stay in shared memory and K streams
//   through; bound by reading K once.
// * many rows: 256 keys stay in shared memory and 64-row tiles of Q stream
//   through; bound by the exponentials (one per pair; 16 a clock and SM).
#pragma once

#include "cache.h"
#include "kernel_common.cuh"

namespace gbattn {

// Where the keys of a row end, and -lse (see above).
__device__ __forceinline__ void key_weight_row(const KeyWeightParams& p, int b, int t, float lse, int& lim,
                                               float& nlse) {
  lim = p.limit ? min(max(p.limit[static_cast<size_t>(b) * p.Lq + t], 0), p.Lk) : p.causal ? t + p.Lk - p.Lq + 1 : p.Lk;
  nlse = -lse;
  if (lse == INFINITY) lim = 0;
}

// The sum over NC columns of this thread's key: S at TMEM columns col.., the
// rows' tables at nl / lim (shared memory, 16-byte aligned).
template <int NC, bool MASK>
__device__ __forceinline__ float key_weight_sum(uint32_t col, uint32_t nl, uint32_t lim, float sl2, int j) {
  const uint64_t sl2x2 = f2_pack(sl2, sl2);
  uint64_t acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
  constexpr int W = NC < 32 ? NC : 32;
#pragma unroll
  for (int c = 0; c < NC; c += W) {
    uint32_t v[W];
    if constexpr (W == 32) tmem_ld32(col + c, v);
    else tmem_ld16(col + c, v);
    tmem_ld_wait(v);
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 n = ld_shared_v4(nl + (c + i) * 4);
      float x0, x1, x2, x3;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sl2x2,
                       f2_pack(__uint_as_float(n.x), __uint_as_float(n.y))), x0, x1);
      f2_unpack(f2_fma(f2_pack(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), sl2x2,
                       f2_pack(__uint_as_float(n.z), __uint_as_float(n.w))), x2, x3);
      if constexpr (MASK) {
        const uint4 l = ld_shared_v4(lim + (c + i) * 4);
        if (j >= static_cast<int>(l.x)) x0 = -INFINITY;
        if (j >= static_cast<int>(l.y)) x1 = -INFINITY;
        if (j >= static_cast<int>(l.z)) x2 = -INFINITY;
        if (j >= static_cast<int>(l.w)) x3 = -INFINITY;
      }
      acc[0] = f2_add(acc[0], f2_pack(ex2_approx(x0), ex2_approx(x1)));
      acc[1] = f2_add(acc[1], f2_pack(ex2_approx(x2), ex2_approx(x3)));
    }
  }
  float a, b, c, d;
  f2_unpack(acc[0], a, b);
  f2_unpack(acc[1], c, d);
  return (a + b) + (c + d);
}

// Key tiles of BK keys that sequence b's rows reach (limit calls), as a prefix
// sum over the sequences: tab[b], tab[B] the total.  Whole block; the caller's
// next barrier publishes it.
template <int BK>
__device__ __forceinline__ void key_weight_table(const KeyWeightParams& p, int* tab) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  for (int b = warp; b < p.B; b += warps) {
    int most = 0;
    for (int t = lane; t < p.Lq; t += 32) most = max(most, p.limit[static_cast<size_t>(b) * p.Lq + t]);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) tab[b + 1] = (min(most, p.Lk) + BK - 1) / BK;
  }
  if (threadIdx.x == 0) tab[0] = 0;
  __syncthreads();
  if (warp == 0) {
    int run = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      int x = b0 + lane < p.B ? tab[b0 + lane + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      if (b0 + lane < p.B) tab[b0 + lane + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows: NQ >= G * Lq of them in one tile; CTAs share the 128-key tiles of
// all KV heads out in equal consecutive ranges.
// ---------------------------------------------------------------------------
template <int D, int NQ>
struct KeyWeightFewGeom {
  static constexpr int BK = 128;
  static constexpr int NCH = n_chunks(D);
  static constexpr int K_BYTES = NCH * BK * 128;
  static constexpr int Q_BYTES = NCH * NQ * 128;
  static constexpr int QBUF = Q_BYTES > 32768 ? 1 : 2;
  static constexpr int AVAIL = kMaxDynSmem - 8192 - 1024 - QBUF * Q_BYTES;
  static constexpr int SLOTS = AVAIL / K_BYTES > 8 ? 8 : AVAIL / K_BYTES;
  static constexpr int SMEM_BYTES = 1024 + QBUF * Q_BYTES + SLOTS * K_BYTES;
  static constexpr int NBUF = 4;  // S buffers
  static constexpr int TMEM_COLS = NBUF * NQ < 64 ? 64 : NBUF * NQ;
  static constexpr int PRODUCER = 8, MMA = 9, NUM_THREADS = 320;
  static_assert(SLOTS >= 2, "shared memory budget");
};

// Walks tiles [x, xe) of the list: the segment is tiles j0 .. j1 - 1 of KV head z = b * Hkv + hk.
struct KeyTileWalk {
  const int* tab;  // limit calls; else every sequence has `each` tiles
  int each, B, Hkv;
  long long x, xe;
  int b, hk, n, j0, j1;
  __device__ __forceinline__ long long pre(int i) const { return tab ? tab[i] : static_cast<long long>(i) * each; }
  __device__ __forceinline__ KeyTileWalk(const int* tab_, int each_, int B_, int Hkv_)
      : tab(tab_), each(each_), B(B_), Hkv(Hkv_) {
    const long long total = pre(B) * Hkv;
    const long long per = (total + gridDim.x - 1) / gridDim.x;
    x = min(static_cast<long long>(blockIdx.x) * per, total);
    xe = min(x + per, total);
    if (x >= xe) return;
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre(mid) * Hkv <= x) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    n = static_cast<int>(pre(b + 1) - pre(b));
    hk = static_cast<int>((x - pre(b) * Hkv) / n);
    set();
  }
  __device__ __forceinline__ bool more() const { return x < xe; }
  __device__ __forceinline__ void set() {
    const long long s = pre(b) * Hkv + static_cast<long long>(hk) * n;
    j0 = static_cast<int>(x - s);
    j1 = static_cast<int>(min(xe - s, static_cast<long long>(n)));
  }
  __device__ __forceinline__ void next() {
    x += j1 - j0;
    if (x >= xe) return;
    if (++hk == Hkv) {
      hk = 0;
      do {
        ++b;
        n = static_cast<int>(pre(b + 1) - pre(b));
      } while (n == 0);
    }
    set();
  }
};

template <int D, bool BF16, int NQ>
__global__ void __launch_bounds__(320, 1)
    attn_key_weight_few_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                               const KeyWeightParams p) {
  using Gm = KeyWeightFewGeom<D, NQ>;
  constexpr int BK = Gm::BK, NCH = Gm::NCH, SL = Gm::SLOTS, QB = Gm::QBUF, NB = Gm::NBUF;
  constexpr int kWait = wait_code<96>();  // every bounded wait of this kernel

  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_qfull[QB], bar_qempty[QB], bar_kfull[SL], bar_kempty[SL], bar_sfull[NB], bar_sempty[NB],
      bar_mfin;
  __shared__ __align__(16) float nlse[QB][NQ];
  __shared__ __align__(16) int lims[QB][NQ];
  __shared__ int lim_min[QB];  // the least limit of the rows
  __shared__ int tab[kTreeMaxB + 1];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = sbase, sK = sQ + QB * Gm::Q_BYTES;
  const WaitGuard g{&abort_flag, p.status, p.limit_ns};
  const int R = p.G * p.Lq;

  if (threadIdx.x == 32 * Gm::PRODUCER) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    abort_flag = 0;
    for (int i = 0; i < QB; ++i) {
      mbar_init(smem_u32(&bar_qfull[i]), 1 + 32);  // the copy, and the 32 lanes that fill the tables
      mbar_init(smem_u32(&bar_qempty[i]), 8);      // the epilogue warps (behind the products)
    }
    for (int i = 0; i < SL; ++i) {
      mbar_init(smem_u32(&bar_kfull[i]), 1);
      mbar_init(smem_u32(&bar_kempty[i]), 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(smem_u32(&bar_sfull[i]), 1);
      mbar_init(smem_u32(&bar_sempty[i]), 4);
    }
    mbar_init(smem_u32(&bar_mfin), 1);
    fence_mbar_init();
  }
  if (warp == Gm::MMA) {
    tmem_alloc(smem_u32(&tmem_slot), Gm::TMEM_COLS);
    tmem_relinquish();
  }
  if (p.limit) key_weight_table<BK>(p, tab);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  const int n_kt = (p.Lk + BK - 1) / BK;
  KeyTileWalk w(p.limit ? tab : nullptr, n_kt, p.B, p.Hkv);

  if (warp == Gm::PRODUCER) {
    // ---------------- TMA producer ----------------
    RingPos<SL> st;
    RingPos<QB> sq;
    int issued = 0, nq = 0;
    for (; w.more() && !abort_flag; w.next()) {
      const int z = w.b * p.Hkv + w.hk;
      const int qb = sq.slot;
      if (nq >= QB) mbar_wait(smem_u32(&bar_qempty[qb]), sq.phase ^ 1u, g, kWait);
      if (__any_sync(0xffffffffu, abort_flag)) break;
      mbar_arrive_expect_tx_w(smem_u32(&bar_qfull[qb]), Gm::Q_BYTES);
      for (int c = 0; c < NCH; ++c)
        tma_load_3d_w(sQ + qb * Gm::Q_BYTES + c * NQ * 128, &tmQ, smem_u32(&bar_qfull[qb]), c * 64, 0, z);
      sq.next();
      ++nq;
      auto tables = [&]() {
        int least = INT_MAX;
        for (int r = lane; r < NQ; r += 32) {
          int lim = 0;
          float nl = -INFINITY;
          if (r < R) {
            key_weight_row(p, w.b, r % p.Lq, p.lse[static_cast<size_t>(z) * R + r], lim, nl);
            least = min(least, lim);
          }
          nlse[qb][r] = nl;
          lims[qb][r] = lim;
        }
        least = __reduce_min_sync(0xffffffffu, least);
        if (lane == 0) lim_min[qb] = least;
        __syncwarp();
        mbar_arrive(smem_u32(&bar_qfull[qb]));
      };
      bool filled = false;
      for (int j = w.j0; j < w.j1; ++j, st.next(), ++issued) {
        const int s = st.slot;
        // the tables' loads wait behind the first keys' copies
        if (!filled && (issued >= SL || j == w.j0 + SL - 1)) tables(), filled = true;
        if (issued >= SL) mbar_wait(smem_u32(&bar_kempty[s]), st.phase ^ 1u, g, kWait);
        if (__any_sync(0xffffffffu, abort_flag)) break;
        const uint32_t bar = smem_u32(&bar_kfull[s]);
        mbar_arrive_expect_tx_w(bar, Gm::K_BYTES);
        for (int c = 0; c < NCH; ++c) tma_load_3d_w(sK + s * Gm::K_BYTES + c * BK * 128, &tmK, bar, c * 64, j * BK, z);
      }
      if (!filled) tables();
    }
    for (int u = 0; u < SL && u < issued; ++u) {
      if (st.slot == 0) st.phase ^= 1u;
      st.slot = (st.slot == 0 ? SL : st.slot) - 1;
      mbar_wait_drain(smem_u32(&bar_kfull[st.slot]), st.phase);
    }
    for (int u = 0; u < QB && u < nq; ++u) {
      if (sq.slot == 0) sq.phase ^= 1u;
      sq.slot = (sq.slot == 0 ? QB : sq.slot) - 1;
      mbar_wait_drain(smem_u32(&bar_qfull[sq.slot]), sq.phase);
    }
    __syncwarp();
  } else if (warp == Gm::MMA) {
    // ---------------- MMA issuer: S^T = K Q^T ----------------
    constexpr uint32_t IDESC = make_idesc_f16(128, NQ, BF16, false, false);
    const uint64_t dQ = make_sdesc_sw128(sQ, 16, 1024), dK = make_sdesc_sw128(sK, 16, 1024);
    RingPos<SL> st;
    RingPos<QB> sq;
    int i = 0;  // tiles so far
    for (; w.more(); w.next(), sq.next()) {
      mbar_wait(smem_u32(&bar_qfull[sq.slot]), sq.phase, g, kWait);
      for (int j = w.j0; j < w.j1; ++j, ++i, st.next()) {
        const int s = st.slot, bb = i % NB;
        if (i >= NB) mbar_wait(smem_u32(&bar_sempty[bb]), (i / NB - 1) & 1, g, kWait);
        mbar_wait(smem_u32(&bar_kfull[s]), st.phase, g, kWait);
        __syncwarp();
        tc_fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss_w(tmem + bb * NQ, sdesc_add(dK, s * Gm::K_BYTES + (kk >> 2) * (BK * 128) + (kk & 3) * 32),
                   sdesc_add(dQ, sq.slot * Gm::Q_BYTES + (kk >> 2) * (NQ * 128) + (kk & 3) * 32), IDESC, kk > 0 ? 1u : 0u);
        mma_commit_w(smem_u32(&bar_sfull[bb]));
        mma_commit_w(smem_u32(&bar_kempty[s]));
      }
    }
    mma_commit_w(smem_u32(&bar_mfin));
    mbar_wait_drain(smem_u32(&bar_mfin), 0);
    __syncwarp();
  } else {
    // ---------------- epilogue: warpgroup h takes every other tile, thread = key ----------------
    const int h = warp >> 2, quad = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    // keys that no row reaches keep their weight
    for (int z = blockIdx.x; z < p.B * p.Hkv; z += gridDim.x) {
      const int b = z / p.Hkv;
      const int from = p.limit ? (tab[b + 1] - tab[b]) * BK : p.Lk;
      for (int j = from + threadIdx.x; j < p.Lk; j += 256) {
        const size_t o = static_cast<size_t>(z) * p.Lk + j;
        p.weight_out[o] = p.weight ? p.weight[o] : 0.f;
      }
    }
    RingPos<QB> sq;
    int i = 0;
    for (; w.more(); w.next(), sq.next()) {
      const int qb = sq.slot;
      mbar_wait(smem_u32(&bar_qfull[qb]), sq.phase, g, kWait);
      const int least = lim_min[qb];
      const uint32_t nl = smem_u32(&nlse[qb][0]), lm = smem_u32(&lims[qb][0]);
      for (int j = w.j0; j < w.j1; ++j, ++i) {
        if ((i & 1) != h) continue;
        const int bb = i % NB;
        const int key = j * BK + quad * 32 + lane;
        const size_t o = (static_cast<size_t>(w.b) * p.Hkv + w.hk) * p.Lk + key;
        const float w0 = p.weight && key < p.Lk ? p.weight[o] : 0.f;
        mbar_wait(smem_u32(&bar_sfull[bb]), (i / NB) & 1, g, kWait);
        __syncwarp();
        tc_fence_after_sync();
        const uint32_t col = tmem + lanes + bb * NQ;
        const float sum = least < (j + 1) * BK ? key_weight_sum<NQ, true>(col, nl, lm, p.scale_log2, key)
                                               : key_weight_sum<NQ, false>(col, nl, lm, p.scale_log2, key);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_sempty[bb]));
        if (key < p.Lk) p.weight_out[o] = w0 + sum;
      }
      // every product with this Q that this warp waits for is complete; the
      // tables are read; (the other warpgroup's tiles are covered by its own arrival)
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_qempty[qb]));
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == Gm::MMA) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, Gm::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// Many rows.  Work: for every KV head and 256-key tile, the 64-row tiles of Q
// that reach it (steps).  CTAs share all steps out in equal consecutive ranges;
// a key tile that several CTAs work on leaves 256 floats per CTA in the
// workspace (at most two such sets each), which attn_key_weight_join_kernel adds up in order.
// ---------------------------------------------------------------------------
template <int D>
struct KeyWeightGeom {
  static constexpr int BK = 256, NQ = 64;
  static constexpr int NCH = n_chunks(D);
  static constexpr int K_BYTES = 2 * NCH * 128 * 128;  // two 128-key tiles
  static constexpr int Q_BYTES = NCH * NQ * 128;
  static constexpr int KBUF = K_BYTES > 65536 ? 1 : 2;
  static constexpr int AVAIL = kMaxDynSmem - 14336 - 1024 - KBUF * K_BYTES;
  static constexpr int SLOTS = AVAIL / Q_BYTES > 8 ? 8 : AVAIL / Q_BYTES;
  static constexpr int SMEM_BYTES = 1024 + KBUF * K_BYTES + SLOTS * Q_BYTES;
  static constexpr int NBUF = 4;   // S buffers per key tile
  static constexpr int TABS = 8;   // row tables in flight
  static constexpr int TMEM_COLS = 512;
  static constexpr int PRODUCER = 8, MMA = 9, ROWS = 10, NUM_THREADS = 352;
  static_assert(SLOTS >= 2, "shared memory budget");
};

// The steps of one KV head: key tile kt needs, in each of `heads` row lists
// (one per query head, or one packed list), row tiles q0(kt) .. tiles - 1.
struct KeyWeightSteps {
  int heads, tiles, shift;  // shift: causal, q0(kt) = max(0, 4 kt - shift); < 0: q0 = 0
  __device__ __forceinline__ int q0(int kt) const { return shift < 0 ? 0 : max(0, 4 * kt - shift); }
  __device__ __forceinline__ int steps(int kt) const { return heads * (tiles - q0(kt)); }
  // steps of the key tiles before kt
  __device__ __forceinline__ long long before(int kt) const {
    long long skipped = 0;
    if (shift >= 0) {
      const long long first = shift / 4 + 1;  // the first key tile with q0 > 0
      if (kt > first) skipped = 2 * (kt - first) * (kt - 1 + first) - static_cast<long long>(shift) * (kt - first);
    }
    return heads * (static_cast<long long>(kt) * tiles - skipped);
  }
};

__device__ __forceinline__ KeyWeightSteps key_weight_steps(const KeyWeightParams& p) {
  if (p.packed) return {1, (p.G * p.Lq + 63) / 64, -1};
  return {p.G, (p.Lq + 63) / 64, p.causal ? (p.Lk - p.Lq + 63) / 64 : -1};
}

// Walks steps [x, xe): the segment is steps s0 .. s1 - 1 of the n of key tile kt of KV head (b, hk).
struct KeyStepWalk {
  KeyWeightSteps st;
  const int* tab;  // limit calls: key tiles that the rows reach; else n_kt for every sequence
  int n_kt, B, Hkv;
  long long lo, x, xe;
  int b, hk, kt, n, s0, s1;
  __device__ __forceinline__ int tiles_of(int i) const { return tab ? tab[i + 1] - tab[i] : n_kt; }
  // first step of KV head (i, h)
  __device__ __forceinline__ long long start(int i, int h) const {
    if (tab) return (static_cast<long long>(tab[i]) * Hkv + static_cast<long long>(h) * tiles_of(i)) * st.heads * st.tiles;
    return (static_cast<long long>(i) * Hkv + h) * st.before(n_kt);
  }
  __device__ __forceinline__ long long total() const { return start(B - 1, Hkv - 1) + st.before(tiles_of(B - 1)); }
  __device__ __forceinline__ KeyStepWalk(const KeyWeightParams& p, const int* tab_)
      : st(key_weight_steps(p)), tab(tab_), n_kt((p.Lk + 255) / 256), B(p.B), Hkv(p.Hkv) {}
  __device__ __forceinline__ long long per(int groups) const { return (total() + groups - 1) / groups; }
  __device__ __forceinline__ void begin(int group, int groups) {
    const long long all = total(), each = per(groups);
    lo = x = min(group * each, all);
    xe = min(x + each, all);
    if (x >= xe) return;
    int a = 0, c = B - 1;
    while (a < c) {
      const int mid = (a + c + 1) >> 1;
      if (start(mid, 0) <= x) a = mid;
      else c = mid - 1;
    }
    b = a;
    hk = static_cast<int>((x - start(b, 0)) / st.before(tiles_of(b)));
    const long long in = x - start(b, hk);
    a = 0, c = tiles_of(b) - 1;
    while (a < c) {
      const int mid = (a + c + 1) >> 1;
      if (st.before(mid) <= in) a = mid;
      else c = mid - 1;
    }
    kt = a;
    set();
  }
  __device__ __forceinline__ bool more() const { return x < xe; }
  __device__ __forceinline__ void set() {
    const long long s = start(b, hk) + st.before(kt);
    n = st.steps(kt);
    s0 = static_cast<int>(x - s);
    s1 = static_cast<int>(min(xe - s, static_cast<long long>(n)));
  }
  __device__ __forceinline__ void next() {
    x += s1 - s0;
    if (x >= xe) return;
    if (++kt == tiles_of(b)) {
      kt = 0;
      if (++hk == Hkv) {
        hk = 0;
        do ++b;
        while (tiles_of(b) == 0);
      }
    }
    set();
  }
  __device__ __forceinline__ bool whole() const { return s0 == 0 && s1 == n; }
  __device__ __forceinline__ int slot() const { return x == lo ? 0 : 1; }
};

// Step s of key tile kt: row list g, row tile qt; and the next step.
struct KeyStepPos {
  int g, qt, q0;
  __device__ __forceinline__ KeyStepPos(const KeyWeightSteps& st, int kt, int s) : q0(st.q0(kt)) {
    const int each = st.tiles - q0;
    g = s / each;
    qt = q0 + s - g * each;
  }
  __device__ __forceinline__ void next(const KeyWeightSteps& st) {
    if (++qt == st.tiles) qt = q0, ++g;
  }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(352, 1)
    attn_key_weight_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const KeyWeightParams p) {
  using Gm = KeyWeightGeom<D>;
  constexpr int NCH = Gm::NCH, SL = Gm::SLOTS, KB = Gm::KBUF, NB = Gm::NBUF, NT = Gm::TABS, NQ = Gm::NQ;
  constexpr int kWait = wait_code<97>();  // every bounded wait of this kernel

  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_kfull[KB], bar_kempty[KB], bar_qfull[SL], bar_qempty[SL], bar_tfull[NT], bar_tempty[NT],
      bar_sfull[2][NB], bar_sempty[2][NB], bar_mfin;
  __shared__ __align__(16) float nlse[NT][NQ];
  __shared__ __align__(16) int lims[NT][NQ];
  __shared__ int lim_min[NT];
  __shared__ int tab[kTreeMaxB + 1];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  if (threadIdx.x == 0) grid_launch_dependents();  // the join kernel waits for this grid before it reads
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sK = sbase, sQ = sK + KB * Gm::K_BYTES;
  const WaitGuard g{&abort_flag, p.status, p.limit_ns};

  if (threadIdx.x == 32 * Gm::PRODUCER) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    abort_flag = 0;
    for (int i = 0; i < KB; ++i) {
      mbar_init(smem_u32(&bar_kfull[i]), 1);
      mbar_init(smem_u32(&bar_kempty[i]), 1);
    }
    for (int i = 0; i < SL; ++i) {
      mbar_init(smem_u32(&bar_qfull[i]), 1);
      mbar_init(smem_u32(&bar_qempty[i]), 1);
    }
    for (int i = 0; i < NT; ++i) {
      mbar_init(smem_u32(&bar_tfull[i]), 32);
      mbar_init(smem_u32(&bar_tempty[i]), 8);
    }
    for (int h = 0; h < 2; ++h)
      for (int i = 0; i < NB; ++i) {
        mbar_init(smem_u32(&bar_sfull[h][i]), 1);
        mbar_init(smem_u32(&bar_sempty[h][i]), 4);
      }
    mbar_init(smem_u32(&bar_mfin), 1);
    fence_mbar_init();
  }
  if (warp == Gm::MMA) {
    tmem_alloc(smem_u32(&tmem_slot), Gm::TMEM_COLS);
    tmem_relinquish();
  }
  if (p.limit) key_weight_table<256>(p, tab);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  KeyStepWalk w(p, p.limit ? tab : nullptr);
  w.begin(blockIdx.x, gridDim.x);

  if (warp == Gm::PRODUCER) {
    // ---------------- TMA producer: K of each segment, its Q tiles ----------------
    RingPos<SL> st;
    RingPos<KB> sk;
    int issued = 0, nk = 0;
    for (; w.more() && !abort_flag; w.next()) {
      const int z = w.b * p.Hkv + w.hk;
      if (nk >= KB) mbar_wait(smem_u32(&bar_kempty[sk.slot]), sk.phase ^ 1u, g, kWait);
      if (__any_sync(0xffffffffu, abort_flag)) break;
      mbar_arrive_expect_tx_w(smem_u32(&bar_kfull[sk.slot]), Gm::K_BYTES);
      for (int h = 0; h < 2; ++h)
        for (int c = 0; c < NCH; ++c)
          tma_load_3d_w(sK + sk.slot * Gm::K_BYTES + (h * NCH + c) * 128 * 128, &tmK, smem_u32(&bar_kfull[sk.slot]),
                        c * 64, w.kt * 256 + h * 128, z);
      sk.next();
      ++nk;
      KeyStepPos at(w.st, w.kt, w.s0);
      for (int s = w.s0; s < w.s1; ++s, at.next(w.st), st.next(), ++issued) {
        if (issued >= SL) mbar_wait(smem_u32(&bar_qempty[st.slot]), st.phase ^ 1u, g, kWait);
        if (__any_sync(0xffffffffu, abort_flag)) break;
        const uint32_t bar = smem_u32(&bar_qfull[st.slot]);
        mbar_arrive_expect_tx_w(bar, Gm::Q_BYTES);
        for (int c = 0; c < NCH; ++c)
          tma_load_3d_w(sQ + st.slot * Gm::Q_BYTES + c * NQ * 128, &tmQ, bar, c * 64, at.qt * NQ,
                        p.packed ? z : z * p.G + at.g);
      }
    }
    for (int u = 0; u < SL && u < issued; ++u) {
      if (st.slot == 0) st.phase ^= 1u;
      st.slot = (st.slot == 0 ? SL : st.slot) - 1;
      mbar_wait_drain(smem_u32(&bar_qfull[st.slot]), st.phase);
    }
    for (int u = 0; u < KB && u < nk; ++u) {
      if (sk.slot == 0) sk.phase ^= 1u;
      sk.slot = (sk.slot == 0 ? KB : sk.slot) - 1;
      mbar_wait_drain(smem_u32(&bar_kfull[sk.slot]), sk.phase);
    }
    __syncwarp();
  } else if (warp == Gm::ROWS) {
    // ---------------- row tables of each step, loaded a step ahead ----------------
    RingPos<NT> tb;
    int made = 0;
    const int rows = p.packed ? p.G * p.Lq : p.Lq;  // rows of a row list
    for (; w.more() && !abort_flag; w.next()) {
      const int z = w.b * p.Hkv + w.hk;
      KeyStepPos at(w.st, w.kt, w.s0);
      float nl[2];
      int lm[2];
      bool real[2];
      auto fetch = [&]() {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = at.qt * NQ + i * 32 + lane;
          nl[i] = -INFINITY;
          lm[i] = 0;
          real[i] = r < rows;
          if (real[i]) {
            const size_t row = (p.packed ? static_cast<size_t>(z) : static_cast<size_t>(z) * p.G + at.g) * rows + r;
            key_weight_row(p, w.b, p.packed ? r % p.Lq : r, p.lse[row], lm[i], nl[i]);
          }
        }
      };
      fetch();
      for (int s = w.s0; s < w.s1; ++s, tb.next(), ++made) {
        const float a0 = nl[0], a1 = nl[1];
        const int l0 = lm[0], l1 = lm[1];
        const int least = __reduce_min_sync(0xffffffffu, min(real[0] ? l0 : INT_MAX, real[1] ? l1 : INT_MAX));
        at.next(w.st);
        if (s + 1 < w.s1) fetch();
        if (made >= NT) mbar_wait(smem_u32(&bar_tempty[tb.slot]), tb.phase ^ 1u, g, kWait);
        nlse[tb.slot][lane] = a0;
        nlse[tb.slot][lane + 32] = a1;
        lims[tb.slot][lane] = l0;
        lims[tb.slot][lane + 32] = l1;
        if (lane == 0) lim_min[tb.slot] = least;
        mbar_arrive(smem_u32(&bar_tfull[tb.slot]));
      }
    }
  } else if (warp == Gm::MMA) {
    // ---------------- MMA issuer: S^T of both key tiles ----------------
    constexpr uint32_t IDESC = make_idesc_f16(128, NQ, BF16, false, false);
    const uint64_t dQ = make_sdesc_sw128(sQ, 16, 1024), dK = make_sdesc_sw128(sK, 16, 1024);
    RingPos<SL> st;
    RingPos<KB> sk;
    int i = 0;  // steps so far
    for (; w.more(); w.next()) {
      mbar_wait(smem_u32(&bar_kfull[sk.slot]), sk.phase, g, kWait);
      for (int s = w.s0; s < w.s1; ++s, ++i, st.next()) {
        const int bb = i % NB;
        mbar_wait(smem_u32(&bar_qfull[st.slot]), st.phase, g, kWait);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (i >= NB) mbar_wait(smem_u32(&bar_sempty[h][bb]), (i / NB - 1) & 1, g, kWait);
          __syncwarp();
          tc_fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss_w(tmem + (h * NB + bb) * NQ,
                     sdesc_add(dK, sk.slot * Gm::K_BYTES + (h * NCH + (kk >> 2)) * (128 * 128) + (kk & 3) * 32),
                     sdesc_add(dQ, st.slot * Gm::Q_BYTES + (kk >> 2) * (NQ * 128) + (kk & 3) * 32), IDESC,
                     kk > 0 ? 1u : 0u);
          mma_commit_w(smem_u32(&bar_sfull[h][bb]));
        }
        mma_commit_w(smem_u32(&bar_qempty[st.slot]));
      }
      mma_commit_w(smem_u32(&bar_kempty[sk.slot]));
      sk.next();
    }
    mma_commit_w(smem_u32(&bar_mfin));
    mbar_wait_drain(smem_u32(&bar_mfin), 0);
    __syncwarp();
  } else {
    // ---------------- epilogue: warpgroup h takes key tile h, thread = key ----------------
    const int h = warp >> 2, quad = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    RingPos<NT> tb;
    int i = 0;
    for (; w.more(); w.next()) {
      const int k0 = w.kt * 256 + h * 128;
      const int mine = h * 128 + quad * 32 + lane, key = w.kt * 256 + mine;
      float total = 0.f;
      for (int s = w.s0; s < w.s1; ++s, ++i, tb.next()) {
        const int bb = i % NB, ts = tb.slot;
        mbar_wait(smem_u32(&bar_tfull[ts]), tb.phase, g, kWait);
        mbar_wait(smem_u32(&bar_sfull[h][bb]), (i / NB) & 1, g, kWait);
        __syncwarp();
        tc_fence_after_sync();
        const uint32_t col = tmem + lanes + (h * NB + bb) * NQ;
        const uint32_t nl = smem_u32(&nlse[ts][0]), lm = smem_u32(&lims[ts][0]);
        total += lim_min[ts] < k0 + 128 ? key_weight_sum<NQ, true>(col, nl, lm, p.scale_log2, key)
                                        : key_weight_sum<NQ, false>(col, nl, lm, p.scale_log2, key);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bar_sempty[h][bb]));
          mbar_arrive(smem_u32(&bar_tempty[ts]));
        }
      }
      if (w.whole()) {
        if (key < p.Lk) {
          const size_t o = (static_cast<size_t>(w.b) * p.Hkv + w.hk) * p.Lk + key;
          p.weight_out[o] = (p.weight ? p.weight[o] : 0.f) + total;
        }
      } else {
        p.part[(static_cast<size_t>(blockIdx.x) * 2 + w.slot()) * 256 + mine] = total;
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == Gm::MMA) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, Gm::TMEM_COLS);
  }
}

// Adds up the partial sums of key tiles that several of the `groups` CTAs
// worked on, in order, and gives keys that no row reaches their weight.
static __global__ void __launch_bounds__(256) attn_key_weight_join_kernel(const KeyWeightParams p, int groups) {
  __shared__ int tab[kTreeMaxB + 1];
  if (p.limit) key_weight_table<256>(p, tab);
  __syncthreads();
  KeyStepWalk w(p, p.limit ? tab : nullptr);
  const long long per = w.per(groups), tiles = static_cast<long long>(p.B) * p.Hkv * w.n_kt;
  grid_dependency_wait();
  for (long long i = blockIdx.x; i < tiles; i += gridDim.x) {
    const int head = static_cast<int>(i / w.n_kt), kt = static_cast<int>(i - static_cast<long long>(head) * w.n_kt);
    const int b = head / p.Hkv, hk = head - b * p.Hkv;
    const int key = kt * 256 + threadIdx.x;
    const size_t o = static_cast<size_t>(head) * p.Lk + key;
    float sum = 0.f;
    if (kt < w.tiles_of(b)) {
      const long long s = w.start(b, hk) + w.st.before(kt);
      const long long g0 = s / per, g1 = (s + w.st.steps(kt) - 1) / per;
      if (g0 == g1) continue;  // written by its CTA
      for (long long g = g0; g <= g1; ++g)
        sum += p.part[(g * 2 + (g == g0 && s != g0 * per ? 1 : 0)) * 256 + threadIdx.x];
    }
    if (key < p.Lk) p.weight_out[o] = (p.weight ? p.weight[o] : 0.f) + sum;
  }
}

}  // namespace gbattn
