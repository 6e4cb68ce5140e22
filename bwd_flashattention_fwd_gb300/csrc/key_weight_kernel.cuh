// Accumulated attention weight of every cached key:
//   weight_out[j] = weight[j] + sum over the rows r that see j of 2^(s'_rj - lse_r),
//   s' = scale log2 e q_r . k_j.
//
// Keys are the rows of the products (S^T = K Q^T, thread = key = TMEM lane), so
// a key's sum stays in its thread, in a fixed order and without atomics.  A
// step's terms are summed, in four chains, apart from the running total: in a sum
// over R rows a term meets about ten roundings in its step and one per step after
// it, all in fp32, instead of R.  With the exponentials (2^-22 each, in hardware)
// the weights of an 8192-token prompt are off by 1.4e-7 of their size.
//
// Rows: the G query heads x Lq rows of a KV head, packed (consecutive in q and
// lse) where Lq is small or the limits are per row, else head by head.
// Each row has a limit (keys j < limit are seen) and -lse, in shared memory.
// A row of the padding (zero q, as loads past the end read zeros), a row whose
// lse is +inf and a row whose limit is 0 (both may hold anything) have limit 0,
// which makes their tile a masked one.  (In the kernel for few rows, padding alone does not.)
//
// Measured (replayed): a prompt of 8192 tokens, 32/8 heads, D = 128 225 us (1220
// TFLOP/s; 145 at the matrix rate); B4 T8 8192 keys 15.9 us for 67 MB, B8 T8
// 16384 keys D = 256 81 us (6.7 TB/s).
//
// Two kernels share this:
// * few rows (G Lq <= 128): the rows stay in shared memory and K streams
//   through; bound by reading K once.
// * many rows: 256 keys stay in tensor memory and tiles of 128 rows of Q (64
//   at D = 256) stream through.
#pragma once

#include "cache.h"
#include "kernel_common.cuh"

namespace gbattn {

// Row t's limit as given (limit calls).
__device__ __forceinline__ int key_weight_limit(const KeyWeightParams& p, int b, int t) {
  const size_t i = static_cast<size_t>(b) * p.Lq + t;
  return dbg_in_range(i, 1, static_cast<size_t>(p.B) * p.Lq, p.status, 70) ? p.limit[i] : 0;
}

// Where the keys of a row end, and -lse (see above).
__device__ __forceinline__ void key_weight_row(const KeyWeightParams& p, int b, int t, float lse, int& lim,
                                               float& nlse) {
  lim = p.limit ? min(max(key_weight_limit(p, b, t), 0), p.Lk) : p.causal ? t + p.Lk - p.Lq + 1 : p.Lk;
  nlse = -lse;
  if (lse == INFINITY) lim = 0;
}

// The sum of 2^(s' - lse) over W rows for this thread's key j: S in v, the
// rows' tables at nl / lim (shared memory, 16-byte aligned).
template <int W, bool MASK>
__device__ __forceinline__ float key_weight_terms(const uint32_t (&v)[W], uint32_t nl, uint32_t lim, float sl2, int j) {
  const uint64_t sl2x2 = f2_pack(sl2, sl2);
  uint64_t acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const uint4 n = ld_shared_v4(nl + i * 4);
    float x0, x1, x2, x3;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sl2x2,
                     f2_pack(__uint_as_float(n.x), __uint_as_float(n.y))), x0, x1);
    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), sl2x2,
                     f2_pack(__uint_as_float(n.z), __uint_as_float(n.w))), x2, x3);
    if constexpr (MASK) {
      const uint4 l = ld_shared_v4(lim + i * 4);
      if (j >= static_cast<int>(l.x)) x0 = -INFINITY;
      if (j >= static_cast<int>(l.y)) x1 = -INFINITY;
      if (j >= static_cast<int>(l.z)) x2 = -INFINITY;
      if (j >= static_cast<int>(l.w)) x3 = -INFINITY;
    }
    acc[0] = f2_add(acc[0], f2_pack(ex2_approx(x0), ex2_approx(x1)));
    acc[1] = f2_add(acc[1], f2_pack(ex2_approx(x2), ex2_approx(x3)));
  }
  float a, b, c, d;
  f2_unpack(acc[0], a, b);
  f2_unpack(acc[1], c, d);
  return (a + b) + (c + d);
}

// The sum over NC columns at TMEM column col.
template <int NC, bool MASK>
__device__ __forceinline__ float key_weight_sum(uint32_t col, uint32_t nl, uint32_t lim, float sl2, int j) {
  constexpr int W = NC < 32 ? NC : 32;
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < NC; c += W) {
    uint32_t v[W];
    if constexpr (W == 32) tmem_ld32(col + c, v);
    else tmem_ld16(col + c, v);
    tmem_ld_wait(v);
    sum += key_weight_terms<W, MASK>(v, nl + c * 4, lim + c * 4, sl2, j);
  }
  return sum;
}

// Key tiles of BK keys that sequence b's rows reach (limit calls), as a prefix
// sum over the sequences: tab[b], tab[B] the total.  Whole block; the caller's
// next barrier publishes it.
template <int BK>
__device__ __forceinline__ void key_weight_table(const KeyWeightParams& p, int* tab) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  for (int b = warp; b < p.B; b += warps) {
    int most = 0;
    for (int t = lane; t < p.Lq; t += 32) most = max(most, key_weight_limit(p, b, t));
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
  int x, xe;
  int b, hk, n, j0, j1;
  __device__ __forceinline__ int pre(int i) const { return tab ? tab[i] : i * each; }
  __device__ __forceinline__ KeyTileWalk(const int* tab_, int each_, int B_, int Hkv_)
      : tab(tab_), each(each_), B(B_), Hkv(Hkv_) {
    const int total = pre(B) * Hkv;  // below 2^31 - 2^10 tiles (the host's check)
    const int per = (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    x = static_cast<int>(min(static_cast<long long>(blockIdx.x) * per, static_cast<long long>(total)));
    xe = min(x + per, total);
    if (x >= xe) return;
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre(mid) * Hkv <= x) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    n = pre(b + 1) - pre(b);
    hk = (x - pre(b) * Hkv) / n;
    set();
  }
  __device__ __forceinline__ bool more() const { return x < xe; }
  __device__ __forceinline__ void set() {
    const int s = pre(b) * Hkv + hk * n;
    j0 = x - s;
    j1 = min(xe - s, n);
  }
  __device__ __forceinline__ void next() {
    x += j1 - j0;
    if (x >= xe) return;
    if (++hk == Hkv) {
      hk = 0;
      do {
        ++b;
        n = pre(b + 1) - pre(b);
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
  grid_dependency_wait();  // the kernels before this one are complete
  if (warp == Gm::MMA) {  // (behind that, so that those have had theirs)
    tmem_alloc(smem_u32(&tmem_slot), Gm::TMEM_COLS);
    tmem_relinquish();
  }
  if (p.limit) key_weight_table<BK>(p, tab);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (threadIdx.x == 0) grid_launch_dependents();  // after tensor memory is allocated
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
          if (r < R && dbg_in_range(static_cast<size_t>(z) * R + r, 1, static_cast<size_t>(p.B) * p.Hkv * R, p.status, 71)) {
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
    [[maybe_unused]] const size_t n_out = static_cast<size_t>(p.B) * p.Hkv * p.Lk;  // for the debug build's index checks
    // keys that no row reaches keep their weight
    for (int z = blockIdx.x; z < p.B * p.Hkv; z += gridDim.x) {
      const int b = z / p.Hkv;
      const int from = p.limit ? (tab[b + 1] - tab[b]) * BK : p.Lk;
      for (int j = from + threadIdx.x; j < p.Lk; j += 256) {
        const size_t o = static_cast<size_t>(z) * p.Lk + j;
        if (dbg_in_range(o, 1, n_out, p.status, 72)) p.weight_out[o] = p.weight ? p.weight[o] : 0.f;
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
        const bool mine = key < p.Lk && dbg_in_range(o, 1, n_out, p.status, 73);
        const float w0 = p.weight && mine ? p.weight[o] : 0.f;
        mbar_wait(smem_u32(&bar_sfull[bb]), (i / NB) & 1, g, kWait);
        __syncwarp();
        tc_fence_after_sync();
        const uint32_t col = tmem + lanes + bb * NQ;
        const float sum = least < (j + 1) * BK ? key_weight_sum<NQ, true>(col, nl, lm, p.scale_log2, key)
                                               : key_weight_sum<NQ, false>(col, nl, lm, p.scale_log2, key);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_sempty[bb]));
        if (mine) p.weight_out[o] = w0 + sum;
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
// Many rows.  Work: for every KV head and 256-key tile, the row tiles of Q
// that reach it (steps).  CTAs share all steps out in equal consecutive ranges;
// a key tile that several CTAs work on leaves 256 floats per CTA in the
// workspace (at most two such sets each), which attn_key_weight_join_kernel adds up in order.
// ---------------------------------------------------------------------------
template <int D>
struct KeyWeightGeom {
  static constexpr int BK = 256, NQ = key_weight_rows_per_step(D);
  static constexpr int NCH = n_chunks(D);
  static constexpr int K_BYTES = 2 * NCH * 128 * 128;  // two 128-key tiles
  static constexpr int Q_BYTES = NCH * NQ * 128;
  static constexpr int AVAIL = kMaxDynSmem - 14336 - 1024 - K_BYTES;
  static constexpr int SLOTS = AVAIL / Q_BYTES > 8 ? 8 : AVAIL / Q_BYTES;
  static constexpr int SMEM_BYTES = 1024 + K_BYTES + SLOTS * Q_BYTES;
  // Tensor memory: K of both key tiles (16-bit pairs) and a ring of S buffers
  // that the two key tiles take in turn; the epilogue empties one into
  // registers at once, so the products never wait.  (K in shared memory would
  // make the products read 8 KB of it per 64 clocks, all that it gives.)
  static constexpr int K_COLS = NCH * 32;
  static constexpr int S_COL = 2 * K_COLS;
  static constexpr int TMEM_COLS = 512;
  static constexpr int NBUF = (TMEM_COLS - S_COL) / NQ > 4 ? 4 : (TMEM_COLS - S_COL) / NQ;
  static constexpr int TABS = 512 / NQ;  // row tables in flight
  static constexpr int EPILOGUE = 4 * 2 * (NQ / 64);  // warps: half of the rows, key tile, lane quadrant
  static constexpr int PRODUCER = EPILOGUE, MMA = EPILOGUE + 1, ROWS = EPILOGUE + 2, NUM_THREADS = 32 * (EPILOGUE + 3);
  static_assert(NBUF >= 3 && S_COL + NBUF * NQ <= TMEM_COLS, "tensor memory budget");
  static_assert(SLOTS >= 2, "shared memory budget");
};

// The steps of one KV head: key tile kt needs, in each of `heads` row lists
// (one per query head, or one packed list), row tiles q0(kt) .. tiles - 1.
struct KeyWeightSteps {
  int heads, tiles;
  int per, shift;  // row tiles per key tile; causal: q0(kt) = max(0, per kt - shift), shift < 0: q0 = 0
  __device__ __forceinline__ int q0(int kt) const { return shift < 0 ? 0 : max(0, per * kt - shift); }
  __device__ __forceinline__ int steps(int kt) const { return heads * (tiles - q0(kt)); }
  // steps of the key tiles before kt
  // (32 bits: the host refuses calls of 2^31 steps or more)
  __device__ __forceinline__ int before(int kt) const {
    int skipped = 0;
    if (shift >= 0) {
      const int first = shift / per + 1;  // the first key tile with q0 > 0
      if (kt > first) skipped = (kt - first) * (per / 2 * (kt - 1 + first) - shift);
    }
    return heads * (kt * tiles - skipped);
  }
};

__device__ __forceinline__ KeyWeightSteps key_weight_steps(const KeyWeightParams& p) {
  const int nq = p.rows_per_step;
  if (p.packed) return {1, (p.G * p.Lq + nq - 1) / nq, 256 / nq, -1};
  return {p.G, (p.Lq + nq - 1) / nq, 256 / nq, p.causal ? (p.Lk - p.Lq + nq - 1) / nq : -1};
}

// A range [x, xe) of steps, and where it begins.
struct KeyStepStart {
  int x, xe, b, hk, kt;
};

// Walks the range: the segment is steps s0 .. s1 - 1 of the n of key tile kt of KV head (b, hk).
struct KeyStepWalk {
  KeyWeightSteps st;
  const int* tab;  // limit calls: key tiles that the rows reach; else n_kt for every sequence
  int n_kt, B, Hkv;
  int lo, x, xe;
  int b, hk, kt, n, s0, s1;
  __device__ __forceinline__ int tiles_of(int i) const { return tab ? tab[i + 1] - tab[i] : n_kt; }
  // first step of KV head (i, h)
  __device__ __forceinline__ int start(int i, int h) const {
    if (tab) return (tab[i] * Hkv + h * tiles_of(i)) * st.heads * st.tiles;
    return (i * Hkv + h) * st.before(n_kt);
  }
  __device__ __forceinline__ int total() const { return start(B - 1, Hkv - 1) + st.before(tiles_of(B - 1)); }
  __device__ __forceinline__ KeyStepWalk(const KeyWeightParams& p, const int* tab_)
      : st(key_weight_steps(p)), tab(tab_), n_kt((p.Lk + 255) / 256), B(p.B), Hkv(p.Hkv) {}
  __device__ __forceinline__ int per(int groups) const {
    const unsigned all = static_cast<unsigned>(total());
    return static_cast<int>((all + groups - 1) / groups);
  }
  // Where group's share begins (one thread; the searches take a microsecond).
  __device__ __forceinline__ KeyStepStart find(int group, int groups) const {
    const int all = total();
    const long long each = per(groups);
    KeyStepStart f;
    f.x = static_cast<int>(min(group * each, static_cast<long long>(all)));
    f.xe = static_cast<int>(min(f.x + each, static_cast<long long>(all)));
    f.b = f.hk = f.kt = 0;
    if (f.x >= f.xe) return f;
    int a = 0, c = B - 1;
    while (a < c) {
      const int mid = (a + c + 1) >> 1;
      if (start(mid, 0) <= f.x) a = mid;
      else c = mid - 1;
    }
    f.b = a;
    f.hk = (f.x - start(f.b, 0)) / st.before(tiles_of(f.b));
    const int in = f.x - start(f.b, f.hk);
    a = 0, c = tiles_of(f.b) - 1;
    while (a < c) {
      const int mid = (a + c + 1) >> 1;
      if (st.before(mid) <= in) a = mid;
      else c = mid - 1;
    }
    f.kt = a;
    return f;
  }
  __device__ __forceinline__ void begin(const KeyStepStart& f) {
    lo = x = f.x, xe = f.xe, b = f.b, hk = f.hk, kt = f.kt;
    if (x < xe) set();
  }
  __device__ __forceinline__ bool more() const { return x < xe; }
  __device__ __forceinline__ void set() {
    const int s = start(b, hk) + st.before(kt);
    n = st.steps(kt);
    s0 = x - s;
    s1 = min(xe - s, n);
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
    // a key tile's first step follows the last of the one before
    n = st.steps(kt);
    s0 = 0;
    s1 = min(xe - x, n);
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
__global__ void __launch_bounds__(KeyWeightGeom<D>::NUM_THREADS, 1)
    attn_key_weight_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const KeyWeightParams p) {
  using Gm = KeyWeightGeom<D>;
  constexpr int NCH = Gm::NCH, SL = Gm::SLOTS, NB = Gm::NBUF, NT = Gm::TABS, NQ = Gm::NQ;
  constexpr int kWait = wait_code<97>();  // every bounded wait of this kernel

  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_kfull, bar_kempty, bar_kready, bar_qfull[SL], bar_qempty[SL], bar_tfull[NT], bar_tempty[NT],
      bar_sfull[NB], bar_sempty[NB], bar_mfin;
  __shared__ __align__(16) float nlse[NT][NQ];
  __shared__ __align__(16) int lims[NT][NQ];
  __shared__ float upper[256];  // sums of the second half of the rows
  __shared__ int2 range[NT][NQ / 32];  // least and largest limit of each 32 rows
  __shared__ int tab[kTreeMaxB + 1];
  __shared__ KeyStepStart start;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sK = sbase, sQ = sK + Gm::K_BYTES;
  const WaitGuard g{&abort_flag, p.status, p.limit_ns};

  if (threadIdx.x == 32 * Gm::PRODUCER) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    abort_flag = 0;
    mbar_init(smem_u32(&bar_kfull), 1);
    mbar_init(smem_u32(&bar_kempty), Gm::EPILOGUE);
    mbar_init(smem_u32(&bar_kready), 32 * Gm::EPILOGUE);
    for (int i = 0; i < SL; ++i) {
      mbar_init(smem_u32(&bar_qfull[i]), 1);
      mbar_init(smem_u32(&bar_qempty[i]), 1);
    }
    for (int i = 0; i < NT; ++i) {
      mbar_init(smem_u32(&bar_tfull[i]), 32);
      mbar_init(smem_u32(&bar_tempty[i]), Gm::EPILOGUE);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(smem_u32(&bar_sfull[i]), 1);
      mbar_init(smem_u32(&bar_sempty[i]), Gm::EPILOGUE / 2);
    }
    mbar_init(smem_u32(&bar_mfin), 1);
    fence_mbar_init();
  }
  grid_dependency_wait();  // the kernels before this one are complete
  if (warp == Gm::MMA) {  // (behind that, so that those have had theirs)
    tmem_alloc(smem_u32(&tmem_slot), Gm::TMEM_COLS);
    tmem_relinquish();
  }
  if (p.limit) {
    key_weight_table<256>(p, tab);
    __syncthreads();
  }
  KeyStepWalk w(p, p.limit ? tab : nullptr);
  if (threadIdx.x == 32 * Gm::ROWS) start = w.find(blockIdx.x, gridDim.x);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  // the join kernel waits for this grid before it reads partials (after tensor memory is allocated)
  if (threadIdx.x == 0) grid_launch_dependents();
  const uint32_t tmem = tmem_slot;
  w.begin(start);

  if (warp == Gm::PRODUCER) {
    // ---------------- TMA producer: K of each segment, its Q tiles ----------------
    RingPos<SL> st;
    int issued = 0, nk = 0;
    for (; w.more() && !abort_flag; w.next()) {
      const int z = w.b * p.Hkv + w.hk;
      if (nk > 0) mbar_wait(smem_u32(&bar_kempty), (nk - 1) & 1, g, kWait);
      if (__any_sync(0xffffffffu, abort_flag)) break;
      mbar_arrive_expect_tx_w(smem_u32(&bar_kfull), Gm::K_BYTES);
      for (int h = 0; h < 2; ++h)
        for (int c = 0; c < NCH; ++c)
          tma_load_3d_w(sK + (h * NCH + c) * 128 * 128, &tmK, smem_u32(&bar_kfull), c * 64, w.kt * 256 + h * 128, z);
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
    if (nk > 0) mbar_wait_drain(smem_u32(&bar_kfull), (nk - 1) & 1);
    __syncwarp();
  } else if (warp == Gm::ROWS) {
    // ---------------- row tables of each step, loaded two to four steps ahead ----------------
    // (with each load used where it is made, the kernel ran at two loads' latency per step: 0.7 us)
    constexpr int AHEAD = 2, RPL = NQ / 32;  // rows per lane
    RingPos<NT> tb;
    int made = 0;
    const int rows = p.packed ? p.G * p.Lq : p.Lq;  // rows of a row list
    for (; w.more() && !abort_flag; w.next()) {
      const int z = w.b * p.Hkv + w.hk;
      KeyStepPos at(w.st, w.kt, w.s0);
      float raw[2][AHEAD][RPL];  // lse as loaded: used (and waited for) in publish only
      int lm[2][AHEAD][RPL];   // limits as loaded (limit calls), else the row's number; -1 past the end
      int fetched = w.s0;
      auto fetch = [&](float(&x)[AHEAD][RPL], int(&l)[AHEAD][RPL]) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
#pragma unroll
          for (int i = 0; i < RPL; ++i) {
            const int r = at.qt * NQ + i * 32 + lane, in = min(r, rows - 1);
            const int t = p.packed ? in % p.Lq : in;
            const size_t row = (p.packed ? static_cast<size_t>(z) : static_cast<size_t>(z) * p.G + at.g) * rows + in;
            const bool real = dbg_in_range(row, 1, static_cast<size_t>(p.B) * p.Hq * p.Lq, p.status, 74);
            x[u][i] = real ? p.lse[row] : INFINITY;
            l[u][i] = p.limit ? key_weight_limit(p, w.b, t) : t;
            if (r >= rows) l[u][i] = -1;
          }
          if (++fetched < w.s1) at.next(w.st);  // (the last step again, past the end)
        }
      };
      auto publish = [&](const float(&x)[AHEAD][RPL], const int(&l)[AHEAD][RPL], int s) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          if (s + u >= w.s1) break;
          if (made >= NT) mbar_wait(smem_u32(&bar_tempty[tb.slot]), tb.phase ^ 1u, g, kWait);
#pragma unroll
          for (int i = 0; i < RPL; ++i) {
            int lim = p.limit ? min(max(l[u][i], 0), p.Lk) : p.causal ? l[u][i] + p.Lk - p.Lq + 1 : p.Lk;
            if (l[u][i] < 0 || x[u][i] == INFINITY) lim = 0;
            nlse[tb.slot][i * 32 + lane] = -x[u][i];
            lims[tb.slot][i * 32 + lane] = lim;
            const int least = __reduce_min_sync(0xffffffffu, lim), most = __reduce_max_sync(0xffffffffu, lim);
            if (lane == 0) range[tb.slot][i] = make_int2(least, most);
          }
          mbar_arrive(smem_u32(&bar_tfull[tb.slot]));
          tb.next();
          ++made;
        }
      };
      fetch(raw[0], lm[0]);
      for (int s = w.s0; s < w.s1; s += 2 * AHEAD) {
        fetch(raw[1], lm[1]);
        publish(raw[0], lm[0], s);
        fetch(raw[0], lm[0]);
        publish(raw[1], lm[1], s + AHEAD);
      }
    }
  } else if (warp == Gm::MMA) {
    // ---------------- MMA issuer: S^T of both key tiles in turn ----------------
    constexpr uint32_t IDESC = make_idesc_f16(128, NQ, BF16, false, false);
    const uint64_t dQ = make_sdesc_sw128(sQ, 16, 1024);
    RingPos<SL> st;
    RingPos<NB> sb;
    int i = 0, r = 0;  // products and segments so far
    for (; w.more(); w.next(), ++r) {
      mbar_wait(smem_u32(&bar_kready), r & 1, g, kWait);  // K is in tensor memory
      for (int s = w.s0; s < w.s1; ++s, st.next()) {
        mbar_wait(smem_u32(&bar_qfull[st.slot]), st.phase, g, kWait);
#pragma unroll
        for (int h = 0; h < 2; ++h, ++i, sb.next()) {
          if (i >= NB) mbar_wait(smem_u32(&bar_sempty[sb.slot]), sb.phase ^ 1u, g, kWait);
          __syncwarp();
          tc_fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ts_w(tmem + Gm::S_COL + sb.slot * NQ, tmem + h * Gm::K_COLS + kk * 8,
                     sdesc_add(dQ, st.slot * Gm::Q_BYTES + (kk >> 2) * (NQ * 128) + (kk & 3) * 32), IDESC,
                     kk > 0 ? 1u : 0u);
          mma_commit_w(smem_u32(&bar_sfull[sb.slot]));
        }
        mma_commit_w(smem_u32(&bar_qempty[st.slot]));
      }
    }
    mma_commit_w(smem_u32(&bar_mfin));
    mbar_wait_drain(smem_u32(&bar_mfin), 0);
    __syncwarp();
  } else {
    // ---------------- epilogue: thread = key of key tile h, HQ of the step's rows ----------------
    // (four warps per scheduler hide one another's waits and loads: with two,
    // each holding 128 rows, an 8192-token prompt took 288 us; with six, three
    // groups of warps that take the products in turn, 216, but 1777 x 2111 at D =
    // 96 30.9 us against 28.5)
    constexpr int HALVES = NQ / 64, HQ = 64;
    const int h = (warp >> 2) & 1, half = warp >> 3, quad = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    RingPos<NT> tb;
    RingPos<NB> sb;  // this key tile's S: every other buffer of the ring
    if (h == 1) sb.next();
    int nk = 0;
    // K of the next segment from shared to tensor memory: this thread's key, 64
    // dims (128 bytes, swizzled) at a time.  Called when the last S of the segment
    // before is complete, so no product reads the old K any more.
    auto copy_k = [&]() {
      mbar_wait(smem_u32(&bar_kfull), nk & 1, g, kWait);
      const int r = quad * 32 + lane;
#pragma unroll 1
      for (int c = half; c < NCH; c += HALVES) {
        const uint32_t src = sK + (h * NCH + c) * 128 * 128 + r * 128;
        uint32_t x[32];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint4 y = ld_shared_v4(src + ((q ^ (r & 7)) << 4));
          x[4 * q] = y.x, x[4 * q + 1] = y.y, x[4 * q + 2] = y.z, x[4 * q + 3] = y.w;
        }
        tmem_st32(tmem + lanes + h * Gm::K_COLS + c * 32, x);
      }
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(smem_u32(&bar_kready));
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_kempty));
      ++nk;
    };
    if (w.more()) copy_k();
    for (; w.more(); w.next()) {
      const int w0 = w.kt * 256 + h * 128 + quad * 32;  // the warp's first key
      const int mine = h * 128 + quad * 32 + lane, key = w.kt * 256 + mine;
      float total = 0.f;
      for (int s = w.s0; s < w.s1; ++s, tb.next(), sb.next(), sb.next()) {
        // every wait comes before S is loaded: a wait's slow path is a call,
        // and S live across it would go through local memory
        const int ts = tb.slot;
        mbar_wait(smem_u32(&bar_tfull[ts]), tb.phase, g, kWait);
        mbar_wait(smem_u32(&bar_sfull[sb.slot]), sb.phase, g, kWait);
        __syncwarp();
        tc_fence_after_sync();
        if (s + 1 == w.s1 && w.x + (w.s1 - w.s0) < w.xe) copy_k();
        const uint32_t s_col = tmem + lanes + Gm::S_COL + sb.slot * NQ + half * HQ;
        const uint32_t nl = smem_u32(&nlse[ts][half * HQ]), lm = smem_u32(&lims[ts][half * HQ]);
        float sum = 0.f;
        // 32 columns at a time: all 64 at once 29.8 us at 1777 x 2111 D = 96, this
        // 28.5 (8192 tokens: 223 and 225)
#pragma unroll
        for (int c = 0; c < HQ / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(s_col + 32 * c, v);
          const int2 lr = range[ts][2 * half + c];
          tmem_ld_wait(v);
          if (c == HQ / 32 - 1) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar_sempty[sb.slot]));
          }
          if (lr.x >= w0 + 32) {  // these 32 rows see all of the warp's 32 keys
            sum += key_weight_terms<32, false>(v, nl + 128 * c, lm + 128 * c, p.scale_log2, key);
          } else if (lr.y > w0) {
            sum += key_weight_terms<32, true>(v, nl + 128 * c, lm + 128 * c, p.scale_log2, key);
          }
        }
        total += sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_tempty[ts]));
      }
      if constexpr (HALVES > 1) {  // the two halves of the rows, in order
        if (half == 1) upper[mine] = total;
        named_bar_sync(1 + h, 256);
        if (half == 0) total += upper[mine];
        named_bar_sync(1 + h, 256);
        if (half == 1) continue;
      }
      if (w.whole()) {
        const size_t o = (static_cast<size_t>(w.b) * p.Hkv + w.hk) * p.Lk + key;
        if (key < p.Lk && dbg_in_range(o, 1, static_cast<size_t>(p.B) * p.Hkv * p.Lk, p.status, 75)) {
          p.weight_out[o] = (p.weight ? p.weight[o] : 0.f) + total;
        }
      } else if (dbg_in_range((static_cast<size_t>(blockIdx.x) * 2 + w.slot()) * 256 + mine, 1,
                              static_cast<size_t>(kTreeMaxCtas) * 512, p.status, 76)) {
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
  const int per = w.per(groups);
  const long long tiles = static_cast<long long>(p.B) * p.Hkv * w.n_kt;
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  for (long long i = blockIdx.x; i < tiles; i += gridDim.x) {
    const int head = static_cast<int>(i / w.n_kt), kt = static_cast<int>(i - static_cast<long long>(head) * w.n_kt);
    const int b = head / p.Hkv, hk = head - b * p.Hkv;
    const int key = kt * 256 + threadIdx.x;
    const size_t o = static_cast<size_t>(head) * p.Lk + key;
    float sum = 0.f;
    if (kt < w.tiles_of(b)) {
      const int s = w.start(b, hk) + w.st.before(kt);
      const int g0 = s / per, g1 = (s + w.st.steps(kt) - 1) / per;
      if (g0 == g1) continue;  // written by its CTA
#pragma unroll 4
      for (int g = g0; g <= g1; ++g) {
        const size_t at = (g * 2 + (g == g0 && s != g0 * per ? 1 : 0)) * 256 + threadIdx.x;
        if (dbg_in_range(at, 1, static_cast<size_t>(kTreeMaxCtas) * 512, p.status, 77)) sum += p.part[at];
      }
    }
    if (key < p.Lk && dbg_in_range(o, 1, static_cast<size_t>(p.B) * p.Hkv * p.Lk, p.status, 78))
      p.weight_out[o] = (p.weight ? p.weight[o] : 0.f) + sum;
  }
}

}  // namespace gbattn
