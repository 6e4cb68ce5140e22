// The two cache calls that move rows: appending accepted drafts and evicting
// the lightest keys.  Both are bound by memory traffic and latency: a prompt of
// 2 x 2048 tokens, 8 heads, D = 128 is appended in 7.1 us (33.6 MB, 4.7 TB/s,
// launch included), 8 drafts in 2.7.
#pragma once

#include "cache.h"
#include "kernel_common.cuh"

namespace gbattn {

__device__ __forceinline__ int clamp_len(int n, int most) { return n < 0 ? 0 : n > most ? most : n; }

// Elements of a cache buffer (16-byte pieces), for the debug build's checks.
__device__ __forceinline__ size_t cache_extent(int heads, int64_t pitch, int Lk, int row16) {
  return (static_cast<size_t>(heads - 1) * pitch + Lk) * row16;
}

constexpr int kAppendThreads = 256;

// Accepted drafts into the cache: the blocks (x, b * Hkv + h) of a KV head
// stride over the 16-byte pieces of the path's rows, one per thread; block
// (0, b * Hkv) writes the sequence's lengths and key limits.
__global__ void __launch_bounds__(kAppendThreads) attn_cache_append_kernel(const AppendParams p) {
  __shared__ int cut, lims[kTreeMaxT];  // (a path has at most kTreeMaxT entries)
  grid_dependency_wait();  // the kernels before this one are complete
  if (threadIdx.x == 0) grid_launch_dependents();
  const int bh = blockIdx.y, b = bh / p.Hkv;
  const int len = clamp_len(p.cache_len[b], p.Lk);
  int n = clamp_len(p.accept_len ? p.accept_len[b] : p.T, p.T);
  n = min(n, p.Lk - len);
  const int32_t* path = p.path ? p.path + static_cast<size_t>(b) * p.T : nullptr;
  if (path) {  // the path ends at its first entry that is no draft
    if (!dbg_in_range(static_cast<size_t>(b) * p.T, n, static_cast<size_t>(p.B) * p.T, p.status, 69)) n = 0;
    if (threadIdx.x == 0) cut = n;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kAppendThreads)
      if (path[i] < 0 || path[i] >= p.T) atomicMin(&cut, i);
    __syncthreads();
    n = cut;
  }
  const int seen = p.seen ? p.seen[b] : 0;
  const size_t src0 = static_cast<size_t>(bh) * p.T * p.row16;
  const size_t dst0 = (static_cast<size_t>(bh) * p.kv_pitch + len) * p.row16;
  [[maybe_unused]] const size_t n_src = static_cast<size_t>(p.B) * p.Hkv * p.T * p.row16;
  [[maybe_unused]] const size_t n_dst = cache_extent(p.B * p.Hkv, p.kv_pitch, p.Lk, p.row16);
  const uint4* ks = static_cast<const uint4*>(p.k_new) + src0;
  const uint4* vs = static_cast<const uint4*>(p.v_new) + src0;
  uint4* kd = static_cast<uint4*>(p.k) + dst0;
  uint4* vd = static_cast<uint4*>(p.v) + dst0;
  const long long total = static_cast<long long>(n) * p.row16;
  for (long long x = static_cast<long long>(blockIdx.x) * kAppendThreads + threadIdx.x; x < total;
       x += static_cast<long long>(gridDim.x) * kAppendThreads) {
    const int i = static_cast<int>(x / p.row16), c = static_cast<int>(x - static_cast<long long>(i) * p.row16);
    const size_t s = static_cast<size_t>(path ? path[i] : i) * p.row16 + c;
    if (dbg_in_range(src0 + s, 1, n_src, p.status, 60) && dbg_in_range(dst0 + x, 1, n_dst, p.status, 61)) {
      const uint4 a = ks[s], v = vs[s];
      kd[x] = a;
      vd[x] = v;
    }
  }
  if (p.pos) {
    const size_t at = static_cast<size_t>(bh) * p.Lk + len;
    for (int i = blockIdx.x * kAppendThreads + threadIdx.x; i < n; i += gridDim.x * kAppendThreads)
      if (dbg_in_range(at + i, 1, static_cast<size_t>(p.B) * p.Hkv * p.Lk, p.status, 68)) p.pos[at + i] = seen + i;
  }
  if (blockIdx.x == 0 && bh == b * p.Hkv) {
    if (threadIdx.x == 0) {
      p.cache_len_out[b] = len + n;
      if (p.seen_out) p.seen_out[b] = seen + n;
    }
    if (p.limit && dbg_in_range(static_cast<size_t>(b) * p.T, p.T, static_cast<size_t>(p.B) * p.T, p.status, 79)) {
      int32_t* limit = p.limit + static_cast<size_t>(b) * p.T;
      if (path) {
        // the last of equal entries: the largest limit, whatever the order of the maxima
        for (int t = threadIdx.x; t < p.T; t += kAppendThreads) lims[t] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kAppendThreads) atomicMax(&lims[path[i]], len + i + 1);
        __syncthreads();
        for (int t = threadIdx.x; t < p.T; t += kAppendThreads) limit[t] = lims[t];
      } else {
        for (int t = threadIdx.x; t < p.T; t += kAppendThreads) limit[t] = t < n ? len + t + 1 : 0;
      }
    }
  }
}

constexpr int kEvictThreads = 1024;  // one CTA per copy of the search
constexpr int kEvictClusterThreads = 512;
constexpr int kEvictKeys = 40960;  // keys that a CTA of a cluster keeps in shared memory

// Order of the slots as an unsigned key, larger = kept first: recent slots
// above all, then by weight (the usual monotone map of IEEE bits; -0 equals
// +0, NaN is below everything).
__device__ __forceinline__ uint32_t evict_key(float w, int pos, long long recent_from) {
  if (pos >= recent_from) return 0xffffffffu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One warp's 32 bins (-1: none) into a histogram.  Equal keys (fresh weights
// are all zero, recent slots share one key) would hit one counter 32 times: counted at once.
__device__ __forceinline__ void evict_count(int* hist, int bin) {
  if (__all_sync(0xffffffffu, bin == __shfl_sync(0xffffffffu, bin, 0))) {
    if (bin >= 0 && (threadIdx.x & 31) == 0) atomicAdd(&hist[bin], 32);
  } else if (bin >= 0) {
    atomicAdd(&hist[bin], 1);
  }
}

// Which slots a search keeps: those with key > threshold, and the first `need`
// of the `equal` ones in slot order (ties: not all of them).
struct EvictKept {
  uint32_t threshold;
  int need;
  bool ties;
  // The kept slots among the warp's 32 (bit per lane); in: the lane has a slot;
  // eq: equal slots before these, counted on (ties only).
  __device__ __forceinline__ uint32_t bits(bool in, uint32_t key, int& eq) const {
    if (!ties) return __ballot_sync(0xffffffffu, in && key >= threshold);
    const uint32_t e = __ballot_sync(0xffffffffu, in && key == threshold);
    const int before = eq + __popc(e & ((1u << (threadIdx.x & 31)) - 1u));
    eq += __popc(e);
    return __ballot_sync(0xffffffffu, in && (key > threshold || (key == threshold && before < need)));
  }
};

// Lanes of the strip of slots i .. i + 31 that lie below `keep`.
__device__ __forceinline__ uint32_t evict_below(int i, int keep) {
  return i + 32 <= keep ? ~0u : i >= keep ? 0u : (1u << (keep - i)) - 1u;
}

// Debug build: slot i of the weights and positions, piece i of a cache buffer.
__device__ __forceinline__ bool evict_slot_ok(const EvictParams& p, size_t i, int site) {
  return dbg_in_range(i, 1, static_cast<size_t>(p.B) * p.Hkv * p.Lk, p.status, site);
}

// The lists' entries of one strip of slots i .. i + 31 (k: kept, m: below
// `keep`, in: existing), with `below` / `above` kept slots before it on either
// side of `keep`; only pairs m0 .. m1 - 1 are listed.  The freed slot j is
// number j - kept(j), the moving one number kept(j) - kept(keep).
template <class Index>
__device__ __forceinline__ void evict_list(int i, uint32_t k, uint32_t m, int below, int above, int m0, int m1,
                                           Index* freed, Index* moving) {
  uint32_t h = ~k & m, v = k & ~m;
  int number = i - below;  // of the first freed slot
  if (number < m1 && number + __popc(h) > m0)
    for (; h; h &= h - 1, ++number)
      if (number >= m0 && number < m1) freed[number - m0] = static_cast<Index>(i + __ffs(static_cast<int>(h)) - 1);
  if (above < m1 && above + __popc(v) > m0)
    for (; v; v &= v - 1, ++above)
      if (above >= m0 && above < m1) moving[above - m0] = static_cast<Index>(i + __ffs(static_cast<int>(v)) - 1);
}

// Kept slots below `keep` keep their values: slots j0 + at, + by, ... below
// j1; bits: their kept strips from slot j0 on.
__device__ __forceinline__ void evict_stay(const EvictParams& p, int bh, const uint32_t* bits, int j0, int j1, int at,
                                           int by) {
  const size_t row = static_cast<size_t>(bh) * p.Lk;
  const int end = min(j1, p.keep);
  for (int j = j0 + at; j < end; j += 4 * by) {
    float w[4];
    int pos[4];
    bool on[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int x = j + u * by;
      on[u] = x < end && ((bits[(x - j0) >> 5] >> ((x - j0) & 31)) & 1u) && evict_slot_ok(p, row + x, 80);
      if (on[u]) w[u] = p.weight[row + x], pos[u] = p.pos[row + x];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (on[u]) p.weight_out[row + j + u * by] = w[u], p.pos_out[row + j + u * by] = pos[u];
  }
}

// The rows of the pairs (moving[i], freed[i]), i < n: threads `all` of `step`, in 16-byte pieces.
template <class Index>
__device__ __forceinline__ void evict_move(const EvictParams& p, int bh, const Index* moving, const Index* freed, int n,
                                           int all, int step) {
  uint4* k = static_cast<uint4*>(p.k) + static_cast<size_t>(bh) * p.kv_pitch * p.row16;
  uint4* v = static_cast<uint4*>(p.v) + static_cast<size_t>(bh) * p.kv_pitch * p.row16;
  const int pieces = n * p.row16;  // at most 2^19 x 32
  [[maybe_unused]] const size_t head = static_cast<size_t>(bh) * p.kv_pitch * p.row16;
  [[maybe_unused]] const size_t n_pieces = cache_extent(p.B * p.Hkv, p.kv_pitch, p.Lk, p.row16);
  constexpr int U = 4;
  for (int x0 = all; x0 < pieces; x0 += U * step) {
    uint4 a[U], e[U];
    size_t to[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = x0 + u * step;
      on[u] = x < pieces;
      if (on[u]) {
        const int i = x / p.row16, c = x - i * p.row16;
        const size_t from = static_cast<size_t>(moving[i]) * p.row16 + c;
        to[u] = static_cast<size_t>(freed[i]) * p.row16 + c;
        on[u] = dbg_in_range(head + from, 1, n_pieces, p.status, 81) && dbg_in_range(head + to[u], 1, n_pieces, p.status, 82);
        if (on[u]) a[u] = k[from], e[u] = v[from];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (on[u]) k[to[u]] = a[u], v[to[u]] = e[u];
  }
}

// Their weights and positions.
template <class Index>
__device__ __forceinline__ void evict_move_values(const EvictParams& p, int bh, const Index* moving, const Index* freed,
                                                  int n, int all, int step) {
  const size_t row = static_cast<size_t>(bh) * p.Lk;
  for (int i = all; i < n; i += step) {
    const int to = freed[i], from = moving[i];
    if (!evict_slot_ok(p, row + to, 83) || !evict_slot_ok(p, row + from, 84)) continue;
    p.weight_out[row + to] = p.weight[row + from];
    p.pos_out[row + to] = p.pos[row + from];
  }
}

// Slots from the new length on: weight 0, position -1.
__device__ __forceinline__ void evict_clear(const EvictParams& p, int bh, int from, int all, int step) {
  const size_t row = static_cast<size_t>(bh) * p.Lk;
  for (int j = from + all; j < p.Lk; j += step) {
    if (!evict_slot_ok(p, row + j, 85)) continue;
    p.weight_out[row + j] = 0.f;
    p.pos_out[row + j] = -1;
  }
}

// A KV head with at most `keep` tokens: nothing goes.
__device__ __forceinline__ void evict_nothing(const EvictParams& p, int bh, int len, int all, int step) {
  const size_t row = static_cast<size_t>(bh) * p.Lk;
  for (int j = all; j < len; j += step) {
    if (!evict_slot_ok(p, row + j, 86)) continue;
    p.weight_out[row + j] = p.weight[row + j];
    p.pos_out[row + j] = p.pos[row + j];
  }
  evict_clear(p, bh, len, all, step);
}

// Keys of the warp's slots w0 .. w1 - 1 into `keys` (from slot j0 on; null:
// not kept) and their first digit into the counters; U strips' loads at a time.
template <int U>
__device__ __forceinline__ void evict_load(const EvictParams& p, int bh, int w0, int w1, int j0, uint32_t* keys,
                                           long long recent_from, int* hist, int digit_shift) {
  const int lane = threadIdx.x & 31;
  const float* w = p.weight + static_cast<size_t>(bh) * p.Lk;
  const int32_t* pos = p.pos + static_cast<size_t>(bh) * p.Lk;
  for (int i = w0 + lane; i - lane < w1; i += 32 * U) {
    float x[U];
    int y[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + 32 * u < w1 && evict_slot_ok(p, static_cast<size_t>(bh) * p.Lk + i + 32 * u, 87))
        x[u] = w[i + 32 * u], y[u] = pos[i + 32 * u];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = i + 32 * u < w1;
      const uint32_t key = in ? evict_key(x[u], y[u], recent_from) : 0u;
      if (in && keys) keys[i + 32 * u - j0] = key;
      evict_count(hist, in ? static_cast<int>(key >> digit_shift) : -1);
    }
  }
}

// Shared memory of the kernel below: keys, and its share of the two lists (16 bits per slot).
__host__ __device__ inline int evict_share(int Lk, int copies) { return (Lk / 2 + copies - 1) / copies; }
__host__ __device__ inline size_t evict_smem(int Lk, int copies) {
  return static_cast<size_t>(Lk) * 4 + static_cast<size_t>(evict_share(Lk, copies)) * 4 + 16;
}

// Eviction with rows of up to kEvictRowKeys slots.
//   1. The keep-th largest key, by a radix search with digits of 11, 11 and 10
//      bits over histograms in shared memory (four, by lane, for the first
//      digit: the weights' exponents meet in few bins).
//   2. Kept tokens before each slot, in slot order (ballots within a warp's
//      consecutive slots, prefix sums over the warps): the freed slot j below
//      `keep` is number j - kept(j), the kept slot j above is number kept(j) -
//      kept(keep).  Of equal keys the lower slots are kept.
//   3. The i-th freed slot takes the i-th kept row from above.  Sources and
//      targets are disjoint, so the rows move in place and in any order.
// A single CTA's load/store unit would bound step 3, and a barrier between
// CTAs costs more than the search; so `copies` CTAs per KV head all do steps 1
// and 2 (every one holds all keys, 4 bytes a slot) and share step 3 out, which
// needs nothing from each other.
__global__ void __launch_bounds__(kEvictThreads, 1) attn_cache_evict_kernel(const EvictParams p, int copies) {
  constexpr int BINS = 2048, NH = 4;
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) int hist[NH][BINS];
  static_assert(__alignof__(hist) >= alignof(int2), "hist is read and cleared in pairs");
  __shared__ uint32_t bits[kEvictRowKeys / 32];  // kept slots
  __shared__ int warp_sum[32];
  __shared__ int2 warp_pair[32];
  __shared__ int s_digit, s_need, s_equal;
  grid_dependency_wait();  // the kernels before this one are complete
  if (threadIdx.x == 0) grid_launch_dependents();
  const int bh = blockIdx.x / copies, rank = blockIdx.x - bh * copies, b = bh / p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = clamp_len(p.cache_len[b], p.Lk);
  const int keep = p.keep;
  const int all = rank * kEvictThreads + tid, step = copies * kEvictThreads;  // this thread among the head's
  if (all == 0 && bh == b * p.Hkv) p.cache_len_out[b] = min(len, keep);
  if (len <= keep) {
    evict_nothing(p, bh, len, all, step);
    return;
  }
  const long long recent_from = static_cast<long long>(p.seen[b]) - p.recent;
  // every warp owns consecutive slots, a multiple of 32 of them
  const int per_warp = ((len + 31) / 32 + 31) & ~31;
  const int w0 = min(warp * per_warp, len), w1 = min(w0 + per_warp, len);
  for (int i = tid; i < NH * BINS; i += kEvictThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  evict_load<5>(p, bh, w0, w1, 0, keys, recent_from, hist[lane & (NH - 1)], 21);
  __syncthreads();
  uint32_t prefix = 0;
  int need = keep;  // how many of the slots that match the digits so far are kept
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
    // two bins per thread, from the top: thread 0 has the last two
    const int bin0 = BINS - 2 - 2 * tid;
    int lo = 0, hi = 0;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      int2* at = reinterpret_cast<int2*>(&hist[h][bin0]);
      lo += at->x, hi += at->y;
      *at = make_int2(0, 0);
    }
    const int mine = lo + hi;
    int incl = mine;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, k);
      if (lane >= k) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0) + incl - mine;
    if (before < need && need <= before + mine) {  // one thread
      const bool upper = need - before <= hi;
      s_digit = bin0 + upper;
      s_need = need - before - (upper ? 0 : hi);
      s_equal = upper ? hi : lo;
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    need = s_need;
    // every slot that matches so far is kept: the lower digits do not matter
    // (the usual end, as two digits leave one slot: 0.9 us less than all three)
    if (d == 2 || need == s_equal) break;
    // the next digit of the slots that match so far (few)
    const uint32_t above = ~0u << shift;
    const int next = d == 0 ? 10 : 0;
    const uint32_t mask = d == 0 ? 2047u : 1023u;
    for (int i0 = w0; i0 < w1; i0 += 128) {
      uint32_t key[4];  // four strips' loads before the first count
#pragma unroll
      for (int u = 0; u < 4; ++u) key[u] = i0 + 32 * u + lane < w1 ? keys[i0 + 32 * u + lane] : ~prefix;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool on = (key[u] & above) == prefix;
        if (__any_sync(0xffffffffu, on)) evict_count(hist[0], on ? static_cast<int>((key[u] >> next) & mask) : -1);
      }
    }
    __syncthreads();
  }
  const EvictKept kept{prefix, need, need < s_equal};
  int eq = 0;
  if (kept.ties) {  // equal slots before this warp's
    int n_eq = 0;
#pragma unroll 4
    for (int i = w0; i < w1; i += 32)
      n_eq += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && keys[i + lane] == prefix));
    if (lane == 0) warp_sum[warp] = n_eq;
    __syncthreads();
    eq = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0);
  }
#pragma unroll 4
  for (int i = w0; i < w1; i += 32) {
    const uint32_t k = kept.bits(i + lane < w1, i + lane < w1 ? keys[i + lane] : 0u, eq);
    if (lane == 0) bits[i >> 5] = k;
  }
  __syncthreads();
  // a strip of 32 slots per thread: kept slots before it, below `keep` and from there on
  const bool on = tid * 32 < len;
  const uint32_t k = on ? bits[tid] : 0u, m = on ? evict_below(tid * 32, keep) : 0u;
  int below = __popc(k & m), above = __popc(k & ~m);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, below, d), y = __shfl_up_sync(0xffffffffu, above, d);
    if (lane >= d) below += x, above += y;
  }
  if (lane == 31) warp_pair[warp] = make_int2(below, above);
  below -= __popc(k & m), above -= __popc(k & ~m);
  __syncthreads();
  const int2 of = warp_pair[lane];
  const int n = keep - __reduce_add_sync(0xffffffffu, of.x);  // freed slots, and as many moving ones
  below += __reduce_add_sync(0xffffffffu, lane < warp ? of.x : 0);
  above += __reduce_add_sync(0xffffffffu, lane < warp ? of.y : 0);
  // this CTA's pairs m0 .. m1 - 1, listed in shared memory
  const int share = evict_share(p.Lk, copies), each = (n + copies - 1) / copies;
  const int m0 = min(rank * each, n), m1 = min(m0 + each, n);
  uint16_t* freed = reinterpret_cast<uint16_t*>(keys + p.Lk);
  uint16_t* moving = freed + share;
  if (on && dbg_in_range(0, m1 - m0, share, p.status, 88)) evict_list(tid * 32, k, m, below, above, m0, m1, freed, moving);
  __syncthreads();
  // rows and values side by side: one's latency does not wait for the other's
  constexpr int ROW_THREADS = kEvictThreads * 3 / 4, VALUE_THREADS = kEvictThreads - ROW_THREADS;
  if (tid < ROW_THREADS) {
    evict_move(p, bh, moving, freed, m1 - m0, tid, ROW_THREADS);
  } else {
    const int t = tid - ROW_THREADS;
    evict_stay(p, bh, bits, 0, len, rank * VALUE_THREADS + t, copies * VALUE_THREADS);
    evict_move_values(p, bh, moving, freed, m1 - m0, t, VALUE_THREADS);
    evict_clear(p, bh, keep, rank * VALUE_THREADS + t, copies * VALUE_THREADS);
  }
}

// Value of another CTA's shared memory (cluster address).
__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// The same for longer rows, one cluster of 8 CTAs per KV head (8 heads of
// 32768 slots: 20 us; 5 more with the moves in this kernel); each CTA owns
// a consecutive part of the slots and keeps their keys in shared memory
// (CACHED; parts that do not fit are read again in each pass).  Four digits of
// 8 bits: what a digit costs is reading every CTA's histogram through
// distributed shared memory (2048 bins: 2.3 us a digit, 256: 0.6) and a cluster
// barrier.  Each digit has a histogram of its own, so none is cleared while
// others read it.  Prefix sums run over warps and CTAs; the lists are in the workspace.
template <bool CACHED>
__global__ void __launch_bounds__(kEvictClusterThreads) attn_cache_evict_cluster_kernel(const EvictParams p) {
  constexpr int NC = kEvictCluster;
  constexpr int NW = kEvictClusterThreads / 32, BINS = 256;
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) int hist[4][BINS];
  __shared__ int first[4][BINS];  // the first digit's, by lane: the weights' exponents meet in few bins
  __shared__ uint32_t bits[kEvictMaxLk / 8 / 32];  // kept slots
  __shared__ int warp_sum[NW];
  __shared__ int2 warp_pair[NW];
  __shared__ __align__(16) int4 quad_sum[NC][BINS / 4];
  __shared__ int s_digit, s_need, s_equal;
  __shared__ int s_counts[2];
  if (threadIdx.x == 0) grid_launch_dependents();  // the move kernel waits for this grid
  const int rank = static_cast<int>(cluster_ctarank());
  const int bh = blockIdx.x / NC, b = bh / p.Hkv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = clamp_len(p.cache_len[b], p.Lk);
  const int keep = p.keep;
  const int all = rank * kEvictClusterThreads + tid, step = NC * kEvictClusterThreads;  // this thread among the cluster's
  if (all == 0 && bh == b * p.Hkv) p.cache_len_out[b] = min(len, keep);
  if (len <= keep) {  // the same for the whole cluster
    if (all == 0) p.counts[bh] = 0;
    evict_nothing(p, bh, len, all, step);
    return;
  }
  const long long recent_from = static_cast<long long>(p.seen[b]) - p.recent;
  const size_t row = static_cast<size_t>(bh) * p.Lk;
  const float* w = p.weight + row;
  const int32_t* pos = p.pos + row;
  // this CTA's slots [j0, j1); every warp owns a consecutive multiple of 32 of them
  const int per_warp = ((len + NC * NW - 1) / (NC * NW) + 31) & ~31;
  const int j0 = min(rank * NW * per_warp, len), j1 = min(j0 + NW * per_warp, len);
  const int w0 = min(j0 + warp * per_warp, j1), w1 = min(w0 + per_warp, j1);
  auto key_at = [&](int j) {
    if constexpr (CACHED) return keys[j - j0];
    else return evict_slot_ok(p, row + j, 89) ? evict_key(w[j], pos[j], recent_from) : 0u;
  };
  for (int i = tid; i < 4 * BINS; i += kEvictClusterThreads) (&hist[0][0])[i] = (&first[0][0])[i] = 0;
  __syncthreads();
  evict_load<8>(p, bh, w0, w1, j0, CACHED ? keys : nullptr, recent_from, first[lane & 3], 24);
  __syncthreads();
  if (tid < BINS) hist[0][tid] = first[0][tid] + first[1][tid] + first[2][tid] + first[3][tid];
  uint32_t prefix = 0;
  int need = keep;
#pragma unroll 1
  for (int d = 0; d < 4; ++d) {
    const int shift = 24 - 8 * d;
    cluster_sync_all();
    // every CTA's histogram, four bins a thread; then the sums, one warp, eight bins a lane from the top
    for (int x = tid; x < NC * (BINS / 4); x += kEvictClusterThreads) {
      const int r = x / (BINS / 4), q = x % (BINS / 4);
      quad_sum[r][q] = ld_cluster_v4(cluster_map(smem_u32(&hist[d][4 * q]), r));
    }
    __syncthreads();
    if (warp == 0) {
      int c[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int4 t = make_int4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < NC; ++r) {
          const int4 x = quad_sum[r][BINS / 4 - 1 - 2 * lane - h];
          t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
        }
        c[4 * h] = t.w, c[4 * h + 1] = t.z, c[4 * h + 2] = t.y, c[4 * h + 3] = t.x;  // from the top
      }
      int mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += c[i];
      int incl = mine;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, k);
        if (lane >= k) incl += y;
      }
      int left = need - (incl - mine);
      if (left > 0 && left <= mine) {  // one lane
        int i = 0;
        bool found = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (!found) {
            i = k;
            if (left <= c[k]) found = true, s_equal = c[k];
            else left -= c[k];
          }
        }
        s_digit = BINS - 1 - 8 * lane - i;
        s_need = left;
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    need = s_need;
    if (d == 3 || need == s_equal) break;  // (as above; the same in every CTA)
    const uint32_t above = ~0u << shift;
    for (int i0 = w0; i0 < w1; i0 += 128) {
      uint32_t key[4];  // four strips' loads before the first count
#pragma unroll
      for (int u = 0; u < 4; ++u) key[u] = i0 + 32 * u + lane < w1 ? key_at(i0 + 32 * u + lane) : ~prefix;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool on = (key[u] & above) == prefix;
        if (__any_sync(0xffffffffu, on))
          evict_count(hist[d + 1], on ? static_cast<int>((key[u] >> (shift - 8)) & 255u) : -1);
      }
    }
  }
  const EvictKept kept{prefix, need, need < s_equal};
  int eq = 0;
  if (kept.ties) {  // equal slots before this warp's
    const int bin = static_cast<int>(prefix & 255u);
    int of[NC];
#pragma unroll
    for (int r = 0; r < NC; ++r) of[r] = ld_cluster(cluster_map(smem_u32(&hist[3][bin]), r));
#pragma unroll
    for (int r = 0; r < NC; ++r) eq += r < rank ? of[r] : 0;
    int n_eq = 0;
#pragma unroll 4
    for (int i = w0; i < w1; i += 32)
      n_eq += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && key_at(i + lane) == prefix));
    if (lane == 0) warp_sum[warp] = n_eq;
    __syncthreads();
    for (int k = 0; k < warp; ++k) eq += warp_sum[k];
  }
  int below = 0, above = 0;  // kept slots of the warp, on either side of `keep`
#pragma unroll 4
  for (int i = w0; i < w1; i += 32) {
    const uint32_t k = kept.bits(i + lane < w1, i + lane < w1 ? key_at(i + lane) : 0u, eq);
    const uint32_t m = evict_below(i, keep);
    if (lane == 0) bits[(i - j0) >> 5] = k;
    below += __popc(k & m), above += __popc(k & ~m);
  }
  if (lane == 0) warp_pair[warp] = make_int2(below, above);
  __syncthreads();
  const int2 of = lane < NW ? warp_pair[lane] : make_int2(0, 0);
  if (warp == 0) {
    const int x = __reduce_add_sync(0xffffffffu, of.x), y = __reduce_add_sync(0xffffffffu, of.y);
    if (lane == 0) s_counts[0] = x, s_counts[1] = y;
  }
  below = __reduce_add_sync(0xffffffffu, lane < warp ? of.x : 0);
  above = __reduce_add_sync(0xffffffffu, lane < warp ? of.y : 0);
  cluster_sync_all();
  int n = keep;  // freed slots, and as many moving ones
  {
    int bl[NC], ab[NC];
#pragma unroll
    for (int r = 0; r < NC; ++r) {
      const uint32_t at = cluster_map(smem_u32(&s_counts[0]), r);
      bl[r] = ld_cluster(at), ab[r] = ld_cluster(at + 4);
    }
#pragma unroll
    for (int r = 0; r < NC; ++r) {
      n -= bl[r];
      if (r < rank) below += bl[r], above += ab[r];
    }
  }
  const int cap = p.Lk / 2;  // min(keep, len - keep) slots at most
  int32_t* freed = p.lists + static_cast<size_t>(bh) * 2 * cap;
  int32_t* moving = freed + cap;
  auto list_ok = [&](int i) { return dbg_in_range(i, 1, cap, p.status, 90); };  // entry i of either
  // a strip of 32 slots per lane; then the warp writes the strips one by one, so
  // that a list's entries are stored side by side (a lane for each strip took
  // 134 us at 2 x 8 heads 200000 -> 20000, where one CTA has all the freed slots, this 123)
  for (int i0 = w0; i0 < w1; i0 += 1024) {
    const int i = i0 + 32 * lane;
    const uint32_t k = i < w1 ? bits[(i - j0) >> 5] : 0u, m = i < w1 ? evict_below(i, keep) : 0u;
    int b0 = __popc(k & m), a0 = __popc(k & ~m);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, b0, d), y = __shfl_up_sync(0xffffffffu, a0, d);
      if (lane >= d) b0 += x, a0 += y;
    }
    const int fb = i - (below + b0 - __popc(k & m)), mb = above + a0 - __popc(k & ~m);  // numbers of the strip's first ones
    for (uint32_t todo = __ballot_sync(0xffffffffu, i < w1 && ((~k & m) | (k & ~m)) != 0u); todo; todo &= todo - 1) {
      const int t = __ffs(static_cast<int>(todo)) - 1;
      const uint32_t kt = __shfl_sync(0xffffffffu, k, t), mt = __shfl_sync(0xffffffffu, m, t);
      const int f0 = __shfl_sync(0xffffffffu, fb, t), m0 = __shfl_sync(0xffffffffu, mb, t);
      const uint32_t h = ~kt & mt, v = kt & ~mt, below_me = (1u << lane) - 1u;
      const int fi = f0 + __popc(h & below_me), mi = m0 + __popc(v & below_me);
      if (((h >> lane) & 1u) && fi < n && list_ok(fi)) freed[fi] = i0 + 32 * t + lane;
      if (((v >> lane) & 1u) && mi < n && list_ok(mi)) moving[mi] = i0 + 32 * t + lane;
    }
    below += __shfl_sync(0xffffffffu, b0, 31), above += __shfl_sync(0xffffffffu, a0, 31);
  }
  if (all == 0) p.counts[bh] = n;
  evict_stay(p, bh, bits, j0, j1, tid, kEvictClusterThreads);
  evict_clear(p, bh, keep, all, step);
  cluster_sync_all();  // no CTA's shared memory is read any more
}

// The moves that the cluster kernel listed, over the whole GPU: block (x, bh).
__global__ void __launch_bounds__(256) attn_cache_move_kernel(const EvictParams p) {
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int bh = blockIdx.y, cap = p.Lk / 2;
  const int32_t* freed = p.lists + static_cast<size_t>(bh) * 2 * cap;
  const int all = static_cast<int>(blockIdx.x * 256 + threadIdx.x), step = static_cast<int>(gridDim.x * 256);
  const int n = p.counts[bh];
  if (!dbg_in_range(0, n, cap, p.status, 91)) return;
  evict_move(p, bh, freed + cap, freed, n, all, step);
  evict_move_values(p, bh, freed + cap, freed, n, all, step);
}

}  // namespace gbattn
