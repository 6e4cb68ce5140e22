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
//   of R = G T rows.  A KV head's keys are a list of 64-key stages, its drafts'
//   stages first; the lists of all KV heads form one list of N stages, which
//   the CTAs (one per SM) divide into equal ranges.  A range that holds a
//   whole KV head writes O and lse; a partial one writes (O / l, lse) in fp32
//   to the workspace, at most two per CTA, and attn_tree_combine_kernel merges
//   them.  Every CTA derives the same division from the lengths in device memory.
//
// * The tensor cores always compute 128 rows, so few rows leave lanes idle
//   unless they share the keys out: with R <= 32 the rows are loaded into all
//   four 32-lane quadrants (QS = 4) and quadrant w takes keys 16w .. 16w + 15 of
//   each stage, with its own m, l and O; P is zero at the other quadrants'
//   keys, so O += P V keeps them apart.  R <= 64: two (QS = 2).  The quadrants
//   are merged when the range ends.  Per stage a softmax thread then handles
//   64 / QS keys, and the exponentials stay far below the time of the loads.
//
// * More than 128 rows (NT = 2, D <= 128): a CTA takes 256 rows as two tiles
//   that share every stage, with a softmax warpgroup and an MMA warp each.
//   More than one block of rows: n_rb neighbouring CTAs walk the same keys
//   with different rows, so the keys come from memory once and then from L2.
//
// Warp roles: 4 NT softmax warps (thread = row of the tile = TMEM lane), one
// TMA producer, NT MMA issuers.  S has two 64-column buffers per tile, P is
// written over the S it came from, a row keeps its reference m until a stage
// raises its maximum by more than 8 (log2 units), so O is rescaled rarely;
// O / l and m + log2 l use the same reference.
//
// Rows of V behind the context's or the drafts' end share a stage with real
// ones and may hold anything: P is 0 there, but 0 * NaN is not, so the softmax
// warps clear them in shared memory before O += P V reads the stage.
#pragma once

#include "cache.h"
#include "kernel_common.cuh"

namespace gbattn {

template <int D, int QS, int NT>
struct TreeGeom {
  static constexpr int BK = kTreeStage;   // keys per stage
  static constexpr int KPW = BK / QS;     // keys per softmax thread and stage
  static constexpr int ROWS = QS > 1 ? 128 / QS : 128 * NT;  // packed rows per CTA
  static constexpr int QROWS = 128 / QS;  // rows of a Q load
  static constexpr int NCH = n_chunks(D);
  static constexpr int Q_BYTES = NCH * 128 * 128;
  static constexpr int KV_BYTES = NCH * BK * 128;
  static constexpr int XCH_BYTES = QS > 1 ? 128 * 33 * 4 : 0;  // merging the quadrants' O
  static constexpr int AVAIL = kMaxDynSmem - 12288 - 1024 - NT * Q_BYTES - XCH_BYTES;
  static constexpr int STAGES = AVAIL / (2 * KV_BYTES) > 8 ? 8 : AVAIL / (2 * KV_BYTES);  // K and V each
  static constexpr int SMEM_BYTES = 1024 + NT * Q_BYTES + STAGES * 2 * KV_BYTES + XCH_BYTES;
  static constexpr int O_W = D <= 128 ? 128 : 256;
  static constexpr int TMEM_COLS = NT * (O_W + 2 * BK) <= 256 ? 256 : 512;
  static constexpr int SOFTMAX_WARPS = 4 * NT;
  static constexpr int NUM_THREADS = 32 * (SOFTMAX_WARPS + 1 + NT);
  static constexpr float TAU = 8.0f;
  __host__ __device__ static constexpr int o_col(int t) { return t * O_W; }
  __host__ __device__ static constexpr int s_col(int t, int b) { return NT * O_W + (2 * t + b) * BK; }
  static_assert(NT * (O_W + 2 * BK) <= 512, "tensor memory budget");
  static_assert(STAGES >= 2, "shared memory budget");
  static_assert(QS == 1 || NT == 1, "only a full tile comes in pairs");
};

// Stages of sequence b (its drafts' first, then its context's).
__device__ __forceinline__ void tree_lengths(const TreeParams& p, int b, int& len, int& tl) {
  len = min(max(p.cache_len[b], 0), p.Lk);
  tl = p.tree_len ? min(max(p.tree_len[b], 0), p.T) : p.T;
}
__device__ __forceinline__ int tree_stages(int len, int tl) {
  return tl == 0 ? 0 : (len + kTreeStage - 1) / kTreeStage + (tl + kTreeStage - 1) / kTreeStage;
}

// pre[b] = stages of one KV head of the sequences before b, pre[B] the total
// (whole block; ends with a barrier).
__device__ __forceinline__ void tree_prefix(const TreeParams& p, int* pre) {
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    int len, tl;
    tree_lengths(p, b, len, tl);
    pre[b + 1] = tree_stages(len, tl);
  }
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    int run = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      int x = b < p.B ? pre[b + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (static_cast<int>(threadIdx.x) >= d) x += y;
      }
      if (b < p.B) pre[b + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
}

// The sequence that stage x of the whole list belongs to: the largest b with pre[b] * Hkv <= x
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

// Stages per CTA range.
__device__ __forceinline__ int tree_per(int total, int n_groups) {
  const int per = (total + n_groups - 1) / n_groups;
  return per > kTreeMinStages ? per : kTreeMinStages;
}

// Walks a CTA's range [x, xe) of the stage list, one KV head at a time: the
// segment is stages j0 .. j1 - 1 of the n stages of head (b, hk).
struct TreeWalk {
  const int* pre;
  int Hkv, lo, x, xe;
  int b, hk, n, j0, j1;
  __device__ __forceinline__ TreeWalk(const TreeParams& p, const int* pre_, int group)
      : pre(pre_), Hkv(p.Hkv) {
    const int total = pre[p.B] * p.Hkv, per = tree_per(total, p.n_groups);
    const long long from = static_cast<long long>(group) * per;
    x = lo = from < total ? static_cast<int>(from) : total;
    xe = from + per < total ? static_cast<int>(from + per) : total;
    if (x < xe) {
      b = tree_find(pre, p.B, Hkv, x);
      n = pre[b + 1] - pre[b];
      hk = (x - pre[b] * Hkv) / n;
      set();
    }
  }
  __device__ __forceinline__ bool more() const { return x < xe; }
  __device__ __forceinline__ void set() {
    const int s = pre[b] * Hkv + hk * n;
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
        n = pre[b + 1] - pre[b];
      } while (n == 0);
    }
    set();
  }
  // the segment is the whole KV head
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == n; }
  // where a partial segment goes: 0 at the start of the range, 1 behind it (cut off by its end)
  __device__ __forceinline__ int slot() const { return x == lo ? 0 : 1; }
};

// First fp32 partial row of (group, slot, row block): slot 0 holds the segment
// at the start of the group's range, slot 1 the one cut off by its end.
__device__ __forceinline__ size_t tree_slot_row(const TreeParams& p, int group, int slot, int rb, int rows) {
  return ((static_cast<size_t>(group) * 2 + slot) * p.n_rb + rb) * rows;
}

template <int D, bool BF16, int QS, int NT>
__global__ void __launch_bounds__(TreeGeom<D, QS, NT>::NUM_THREADS, 1)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKn,
                     const __grid_constant__ CUtensorMap tmVn, const TreeParams p) {
  using Gm = TreeGeom<D, QS, NT>;
  using E = Elem<BF16>;
  constexpr int BK = Gm::BK, NCH = Gm::NCH, ST = Gm::STAGES, KPW = Gm::KPW;
  constexpr int PRODUCER = Gm::SOFTMAX_WARPS;
  constexpr int kWait = wait_code<94>();  // every bounded wait of this kernel

  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_q, bar_qfree, bar_kvfull[ST], bar_kvempty[ST], bar_sfull[NT][2], bar_pready[NT][2],
      bar_odone[NT][2], bar_mfin[NT];
  __shared__ int pre[kTreeMaxB + 1];
  __shared__ float2 ml[128 * NT];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  // the combine kernel may start; it waits for this grid before it reads
  if (threadIdx.x == 0) grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = sbase;                  // tile t at sQ + t * Q_BYTES
  const uint32_t sK0 = sQ + NT * Gm::Q_BYTES;  // stage s: K at sK0 + 2 s KV_BYTES, V right after
  float* xch = reinterpret_cast<float*>(smem_raw + (sK0 + ST * 2 * Gm::KV_BYTES - smem_u32(smem_raw)));
  const int group = blockIdx.x / p.n_rb, rb = blockIdx.x - group * p.n_rb;
  const WaitGuard g{&abort_flag, p.status, p.limit_ns};

  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(smem_u32(&bar_q), 1);
    mbar_init(smem_u32(&bar_qfree), NT);
    for (int s = 0; s < ST; ++s) {
      mbar_init(smem_u32(&bar_kvfull[s]), 1);
      mbar_init(smem_u32(&bar_kvempty[s]), NT);
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
  if (warp == PRODUCER + 1) {
    tmem_alloc(smem_u32(&tmem_slot), Gm::TMEM_COLS);
    tmem_relinquish();
  }
  tree_prefix(p, pre);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  TreeWalk w(p, pre, group);

  if (warp == PRODUCER) {
    // ---------------- TMA producer (whole warp, one elected lane issues) ----------------
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmKn);
      tma_prefetch_desc(&tmVn);
    }
    __syncwarp();
    RingPos<ST> st;
    int issued = 0, nq = 0;
    for (; w.more() && !abort_flag; w.next()) {
      const int z = w.b * p.Hkv + w.hk;
      int len, tl;
      tree_lengths(p, w.b, len, tl);
      const int nd = (tl + BK - 1) / BK;  // draft stages
      // the previous segment's S products, the only readers of Q, are complete
      if (nq > 0) mbar_wait(smem_u32(&bar_qfree), (nq - 1) & 1, g, kWait);
      __syncwarp();
      if (abort_flag) break;
      ++nq;
      mbar_arrive_expect_tx_w(smem_u32(&bar_q), NT * Gm::Q_BYTES);
      for (int t = 0; t < NT; ++t)
        for (int c = 0; c < NCH; ++c)
          for (int i = 0; i < QS; ++i)
            tma_load_3d_w(sQ + t * Gm::Q_BYTES + c * 128 * 128 + i * Gm::QROWS * 128, &tmQ, smem_u32(&bar_q), c * 64,
                          rb * Gm::ROWS + t * 128, z);
      for (int j = w.j0; j < w.j1; ++j, st.next(), ++issued) {
        const int s = st.slot;
        if (issued >= ST) mbar_wait(smem_u32(&bar_kvempty[s]), st.phase ^ 1u, g, kWait);
        __syncwarp();
        if (abort_flag) break;
        const uint32_t bar = smem_u32(&bar_kvfull[s]);
        const uint32_t dK = sK0 + 2 * s * Gm::KV_BYTES;
        mbar_arrive_expect_tx_w(bar, 2 * Gm::KV_BYTES);
        const bool draft = j < nd;
        const int row = draft ? j * BK : (j - nd) * BK;
        for (int c = 0; c < NCH; ++c) {
          tma_load_3d_w(dK + c * BK * 128, draft ? &tmKn : &tmK, bar, c * 64, row, z);
          tma_load_3d_w(dK + Gm::KV_BYTES + c * BK * 128, draft ? &tmVn : &tmV, bar, c * 64, row, z);
        }
      }
    }
    // the last ST issued stages (each slot holds at most one copy in flight) and the last Q
    for (int u = 0; u < ST && u < issued; ++u) {
      if (st.slot == 0) st.phase ^= 1u;
      st.slot = (st.slot == 0 ? ST : st.slot) - 1;
      mbar_wait_drain(smem_u32(&bar_kvfull[st.slot]), st.phase);
    }
    if (nq > 0) mbar_wait_drain(smem_u32(&bar_q), (nq - 1) & 1);
    __syncwarp();
  } else if (warp > PRODUCER) {
    // ---------------- MMA issuer of tile t ----------------
    const int t = warp - PRODUCER - 1;
    constexpr uint32_t IDESC_QK = make_idesc_f16(128, BK, BF16, false, false);
    constexpr uint32_t IDESC_PV = make_idesc_f16(128, D, BF16, false, true);
    const uint64_t dQd = make_sdesc_sw128(sQ + t * Gm::Q_BYTES, 16, 1024);      // this tile's Q, K-major
    const uint64_t dKk = make_sdesc_sw128(sK0, 16, 1024);                       // K stage 0, K-major
    const uint64_t dVm = make_sdesc_sw128(sK0 + Gm::KV_BYTES, BK * 128, 1024);  // V stage 0, MN-major
    RingPos<ST> st_s, st_pv;
    int ts = 0, tp = 0;  // stages (all segments) of the next S and of the next P V
    auto issue_s = [&]() {
      const int s = st_s.slot, bb = ts & 1;
      mbar_wait(smem_u32(&bar_kvfull[s]), st_s.phase, g, kWait);
      st_s.next();
      ++ts;
      __syncwarp();
      tc_fence_after_sync();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t qo = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
        const uint32_t ko = 2 * s * Gm::KV_BYTES + (kk >> 2) * (BK * 128) + (kk & 3) * 32;
        mma_ss_w(tmem + Gm::s_col(t, bb), sdesc_add(dQd, qo), sdesc_add(dKk, ko), IDESC_QK, kk > 0 ? 1u : 0u);
      }
      mma_commit_w(smem_u32(&bar_sfull[t][bb]));
    };
    int r = 0;
    for (; w.more(); w.next(), ++r) {
      const int n = w.j1 - w.j0;
      mbar_wait(smem_u32(&bar_q), r & 1, g, kWait);
      __syncwarp();
      tc_fence_after_sync();
      for (int j = 0; j < 2 && j < n; ++j) {
        issue_s();
        if (j == n - 1) mma_commit_w(smem_u32(&bar_qfree));  // last read of this segment's Q
      }
      for (int j = 0; j < n; ++j) {
        const int s = st_pv.slot, bb = tp & 1;
        mbar_wait(smem_u32(&bar_pready[t][bb]), (tp >> 1) & 1, g, kWait);
        st_pv.next();
        ++tp;
        __syncwarp();
        tc_fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          mma_ts_w(tmem + Gm::o_col(t), tmem + Gm::s_col(t, bb) + kk * 8,
                   sdesc_add(dVm, 2 * s * Gm::KV_BYTES + kk * 2048), IDESC_PV, (j > 0 || kk > 0) ? 1u : 0u);
        mma_commit_w(smem_u32(&bar_kvempty[s]));  // S and P V of this stage were its last reads
        mma_commit_w(smem_u32(&bar_odone[t][bb]));
        // S of stage j + 2 goes over P of stage j, which the products above read (issue order)
        if (j + 2 < n) {
          issue_s();
          if (j + 2 == n - 1) mma_commit_w(smem_u32(&bar_qfree));
        }
      }
    }
    // every MMA this warp issued is complete before tensor memory is released
    mma_commit_w(smem_u32(&bar_mfin[t]));
    mbar_wait_drain(smem_u32(&bar_mfin[t]), 0);
    __syncwarp();
  } else {
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
    // KV heads without a stage (no drafts): their rows see nothing
    for (int x = blockIdx.x; x < p.B * p.Hkv; x += gridDim.x) {
      if (pre[x / p.Hkv + 1] != pre[x / p.Hkv]) continue;
      uint4* o = reinterpret_cast<uint4*>(static_cast<typename E::T*>(p.o) + static_cast<size_t>(x) * R * D);
      for (long long i = threadIdx.x; i < static_cast<long long>(R) * (D / 8); i += 128 * NT) o[i] = make_uint4(0, 0, 0, 0);
      for (int i = threadIdx.x; i < R; i += 128 * NT) p.lse[static_cast<size_t>(x) * R + i] = INFINITY;
    }
    // O += P V of stage k is complete.  (One barrier for even and one for odd
    // stages: when stage k's P has just been handed over, the product of k - 1
    // may still run, and a single barrier's parity could not tell; k - 2 is
    // complete, S of stage k was issued behind it.)
    auto o_done = [&](int k) { mbar_wait(smem_u32(&bar_odone[t][k & 1]), (k >> 1) & 1, g, kWait); };
    RingPos<ST> st;
    int ts = 0;  // stages (all segments) so far
    for (; w.more(); w.next()) {
      int len, tl;
      tree_lengths(p, w.b, len, tl);
      const int nd = (tl + BK - 1) / BK;
      float m = -INFINITY, l = 0.f;
      for (int j = w.j0; j < w.j1; ++j, ++ts, st.next()) {
        const bool draft = j < nd;
        const int k0 = draft ? j * BK : (j - nd) * BK;
        const int valid = min((draft ? tl : len) - k0, BK);  // keys of the stage that exist
        // which of this thread's keys its row sees
        uint64_t see = ~0ull;
        if (draft) {
          see = 0ull;
          if (row < R) {
            const uint8_t* mrow = p.mask ? p.mask + (static_cast<size_t>(w.b) * p.T + trow) * p.T + k0 + c0 : nullptr;
#pragma unroll 8
            for (int i = 0; i < KPW; ++i) {
              if (c0 + i < valid && (mrow ? mrow[i] != 0 : k0 + c0 + i <= trow)) see |= 1ull << i;
            }
          }
        } else if (valid < BK) {
          const int mine = valid - c0;
          see = mine <= 0 ? 0ull : mine >= 64 ? ~0ull : (1ull << mine) - 1ull;
        }
        const int bb = ts & 1;
        const uint32_t s_col = tmem + lanes + Gm::s_col(t, bb);
        mbar_wait(smem_u32(&bar_sfull[t][bb]), (ts >> 1) & 1, g, kWait);
        if (valid < BK) {
          // V rows of no key: cleared, P = 0 does not hide a NaN there
          mbar_wait(smem_u32(&bar_kvfull[st.slot]), st.phase, g, kWait);
          const uint32_t sV = sK0 + 2 * st.slot * Gm::KV_BYTES + Gm::KV_BYTES;
          const int pieces = (BK - valid) * 8;
          for (int x = threadIdx.x & 127; x < NCH * pieces; x += 128) {
            const int c = x / pieces, y = x - c * pieces;
            st_shared_v4(sV + c * BK * 128 + valid * 128 + y * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        tc_fence_after_sync();
        constexpr int NV = KPW > 32 ? 32 : KPW;  // values per register block
        constexpr int NB = KPW / NV;
        uint32_t v[NB][NV];
#pragma unroll
        for (int h = 0; h < NB; ++h) {
          if constexpr (NV == 32) tmem_ld32(s_col + c0 + 32 * h, v[h]);
          else tmem_ld16(s_col + c0, v[h]);
        }
        tmem_ld_wait(v[0]);
        if constexpr (NB == 2) reg_fence(v[1]);
        if (draft || valid < BK) {
#pragma unroll
          for (int h = 0; h < NB; ++h)
#pragma unroll
            for (int i = 0; i < NV; ++i)
              if (!((see >> (h * NV + i)) & 1ull)) v[h][i] = __float_as_uint(-INFINITY);
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
        const float mu = m == -INFINITY ? 0.f : m;
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
        // P over the stage's S: pairs of keys in 32 columns, zeros at the other quadrants' keys
        if constexpr (QS == 1) {
          tmem_st16(s_col, pk[0]);
          tmem_st16(s_col + 16, pk[1]);
        } else {
          uint32_t zero[NV / 2];
#pragma unroll
          for (int i = 0; i < NV / 2; ++i) zero[i] = 0u;
#pragma unroll
          for (int i = 0; i < QS; ++i) {
            if constexpr (QS == 4) {
              if (i == kq) tmem_st8(s_col + i * 8, pk[0]);
              else tmem_st8(s_col + i * 8, zero);
            } else {
              if (i == kq) tmem_st16(s_col + i * 16, pk[0]);
              else tmem_st16(s_col + i * 16, zero);
            }
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
      if (kq == 0 && row < R) {
        const float lse = m + log2f(l);
        if (whole) p.lse[grow] = empty ? INFINITY : lse;
        else p.part_lse[prow] = empty ? -INFINITY : lse;
      }
      typename E::T* orow = static_cast<typename E::T*>(p.o) + grow * D;
      float* partrow = p.part + prow * D;
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
          if (row < R) {
            if (whole) store_row32<BF16>(orow + c * 32, rr, empty ? 1.f : inv);
            else store_row32_f32(partrow + c * 32, rr, empty ? 1.f : inv);
          }
        } else {
          constexpr int W = 32 / QS;  // columns per thread once merged
          const int slotrow = kq * Gm::QROWS + lrow;
          const bool drop = empty || f == 0.f;
#pragma unroll
          for (int i = 0; i < 32; ++i) xch[slotrow * 33 + i] = drop ? 0.f : __uint_as_float(rr[i]) * inv;
          named_bar_sync(1 + t, 128);
          float acc[W];
#pragma unroll
          for (int i = 0; i < W; ++i) {
            acc[i] = 0.f;
#pragma unroll
            for (int k = 0; k < QS; ++k) acc[i] += xch[(k * Gm::QROWS + lrow) * 33 + kq * W + i];
          }
          if (row < R) {
            if (whole) {
              uint4* d = reinterpret_cast<uint4*>(orow + c * 32 + kq * W);
#pragma unroll
              for (int i = 0; i < W / 8; ++i)
                d[i] = make_uint4(E::pack(acc[8 * i], acc[8 * i + 1]), E::pack(acc[8 * i + 2], acc[8 * i + 3]),
                                  E::pack(acc[8 * i + 4], acc[8 * i + 5]), E::pack(acc[8 * i + 6], acc[8 * i + 7]));
            } else {
              float4* d = reinterpret_cast<float4*>(partrow + c * 32 + kq * W);
#pragma unroll
              for (int i = 0; i < W / 4; ++i) d[i] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
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
    tmem_dealloc(tmem, Gm::TMEM_COLS);
  }
}

// Merges the partials of the KV heads that more than one CTA worked on.  A
// head is cut at the range boundaries inside it; block (x, y) takes the head
// whose first cut is the start of group x + 1, rows 8 / WPR * y and on, WPR
// warps per row.  With partial lse L_s and O_s: M = max L_s, w_s = 2^(L_s - M),
// O = sum w_s O_s / sum w_s, lse = M + log2 sum w_s, partials in order.
template <int D, bool BF16, int WPR>
__global__ void __launch_bounds__(256) attn_tree_combine_kernel(const TreeParams p, int rows) {
  using E = Elem<BF16>;
  constexpr int PER = D / 32;
  __shared__ int pre[kTreeMaxB + 1];
  __shared__ float sden[8], so[8][D];
  tree_prefix(p, pre);
  const int total = pre[p.B] * p.Hkv, per = tree_per(total, p.n_groups);
  const long long cut = (static_cast<long long>(blockIdx.x) + 1) * per;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % WPR;
  const int row = static_cast<int>(blockIdx.y) * (8 / WPR) + warp / WPR;
  bool mine = cut < total && row < p.G * p.T;
  int s = 0, e = 0, b = 0, hk = 0;
  if (cut < total) {
    b = tree_find(pre, p.B, p.Hkv, static_cast<int>(cut));
    const int n = pre[b + 1] - pre[b];
    hk = (static_cast<int>(cut) - pre[b] * p.Hkv) / n;
    s = pre[b] * p.Hkv + hk * n;
    e = s + n;
    // cut lies inside the head and is the first cut that does
    mine = mine && s < cut && cut - per <= s;
  }
  grid_dependency_wait();  // the partials are written (and the whole call ends behind them)
  float den = 0.f, M = -INFINITY, acc[PER];
#pragma unroll
  for (int c = 0; c < PER; ++c) acc[c] = 0.f;
  const int g0 = s / per, ng = mine ? (e - 1) / per - g0 + 1 : 0;
  const int rb = row / rows, lrow = row - rb * rows;
  auto part_row = [&](int i) {
    // the head's first partial is its group's second one, unless the head starts the group's range
    return tree_slot_row(p, g0 + i, i == 0 && s != g0 * per ? 1 : 0, rb, rows) + lrow;
  };
  for (int i = lane; i < ng; i += 32) M = fmaxf(M, p.part_lse[part_row(i)]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
#pragma unroll 4
  for (int i = sub; i < ng; i += WPR) {
    const size_t r = part_row(i);
    const float L = p.part_lse[r];
    const float wgt = L == -INFINITY ? 0.f : exp2f(L - M);
    den += wgt;
#pragma unroll
    for (int c = 0; c < PER; ++c) acc[c] = fmaf(wgt, p.part[r * D + lane + 32 * c], acc[c]);
  }
  if constexpr (WPR > 1) {
    if (lane == 0) sden[warp] = den;
#pragma unroll
    for (int c = 0; c < PER; ++c) so[warp][lane + 32 * c] = acc[c];
    __syncthreads();
    if (sub != 0) return;
    for (int k = 1; k < WPR; ++k) {
      den += sden[warp + k];
#pragma unroll
      for (int c = 0; c < PER; ++c) acc[c] += so[warp + k][lane + 32 * c];
    }
  }
  if (!mine) return;
  const size_t grow = (static_cast<size_t>(b) * p.Hkv + hk) * (p.G * p.T) + row;
  const bool empty = den == 0.f;
  typename E::T* o = static_cast<typename E::T*>(p.o) + grow * D;
#pragma unroll
  for (int c = 0; c < PER; ++c) o[lane + 32 * c] = E::from_float(empty ? 0.f : acc[c] / den);
  if (lane == 0) p.lse[grow] = empty ? INFINITY : M + log2f(den);
}

}  // namespace gbattn
