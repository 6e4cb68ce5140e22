// The two cache calls that move rows: appending accepted drafts and evicting
// the lightest keys.  Both are bound by memory traffic and latency.
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

// Accepted drafts into the cache: block (x, b * Hkv + h) copies rows x,
// x + gridDim.x, ... of the path, 16 bytes per thread; block (0, b * Hkv)
// writes the sequence's lengths and key limits.
__global__ void __launch_bounds__(kAppendThreads) attn_cache_append_kernel(const AppendParams p) {
  __shared__ int cut;
  const int bh = blockIdx.y, b = bh / p.Hkv;
  const int len = clamp_len(p.cache_len[b], p.Lk);
  int n = clamp_len(p.accept_len ? p.accept_len[b] : p.T, p.T);
  n = min(n, p.Lk - len);
  const int32_t* path = p.path ? p.path + static_cast<size_t>(b) * p.T : nullptr;
  if (path) {  // the path ends at its first entry that is no draft
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
    int32_t* pos = p.pos + static_cast<size_t>(bh) * p.Lk + len;
    for (int i = blockIdx.x * kAppendThreads + threadIdx.x; i < n; i += gridDim.x * kAppendThreads) pos[i] = seen + i;
  }
  if (blockIdx.x == 0 && bh == b * p.Hkv) {
    if (threadIdx.x == 0) {
      p.cache_len_out[b] = len + n;
      if (p.seen_out) p.seen_out[b] = seen + n;
    }
    if (p.limit) {
      int32_t* limit = p.limit + static_cast<size_t>(b) * p.T;
      for (int t = threadIdx.x; t < p.T; t += kAppendThreads) {
        int lim = 0;
        if (!path) {
          lim = t < n ? len + t + 1 : 0;
        } else {
          for (int i = 0; i < n; ++i)
            if (path[i] == t) lim = len + i + 1;
        }
        limit[t] = lim;
      }
    }
  }
}

constexpr int kEvictThreads = 1024;     // one CTA per copy of the search
constexpr int kEvictClusterThreads = 512;
constexpr int kEvictBins = 1 << 11;  // digits of the radix search: 11, 11 and 10 bits
constexpr int kEvictKeys = 40960;    // keys that a CTA of a cluster keeps in shared memory

// Order of the slots as an unsigned key, larger = kept first: recent slots
// above all, then by weight (the usual monotone map of IEEE bits; -0 equals
// +0, NaN is below everything).
__device__ __forceinline__ uint32_t evict_key(float w, int pos, long long recent_from) {
  if (pos >= recent_from) return 0xffffffffu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Digit d (0, 1, 2) of the radix search: its shift, its mask, and the bits of the digits before it.
struct EvictDigit {
  int shift;
  uint32_t mask, above;
};
__device__ __forceinline__ EvictDigit evict_digit(int d) {
  return d == 0 ? EvictDigit{21, 2047u, 0u} : d == 1 ? EvictDigit{10, 2047u, ~0u << 21} : EvictDigit{0, 1023u, ~0u << 10};
}

// One warp's 32 keys into a histogram.  Equal keys (fresh weights are all
// zero, recent slots share one key) would hit one counter 32 times: counted at once.
__device__ __forceinline__ void evict_count(int* hist, bool on, uint32_t key, const EvictDigit& dg) {
  const int bin = on ? static_cast<int>((key >> dg.shift) & dg.mask) : -1;
  if (__all_sync(0xffffffffu, bin == __shfl_sync(0xffffffffu, bin, 0))) {
    if (on && (threadIdx.x & 31) == 0) atomicAdd(&hist[bin], 32);
  } else if (on) {
    atomicAdd(&hist[bin], 1);
  }
}

// The rows of the pairs (moving[i], freed[i]), i < n, and their weights and
// positions: threads `all` of `step`, in 16-byte pieces.
template <class Index>
__device__ __forceinline__ void evict_move(const EvictParams& p, int bh, const Index* moving, const Index* freed, int n,
                                           int all, int step) {
  const size_t row = static_cast<size_t>(bh) * p.Lk;
  for (int i = all; i < n; i += step) {
    const int to = freed[i], from = moving[i];
    p.weight_out[row + to] = p.weight[row + from];
    p.pos_out[row + to] = p.pos[row + from];
  }
  uint4* k = static_cast<uint4*>(p.k) + static_cast<size_t>(bh) * p.kv_pitch * p.row16;
  uint4* v = static_cast<uint4*>(p.v) + static_cast<size_t>(bh) * p.kv_pitch * p.row16;
  const int pieces = n * p.row16;  // at most 2^19 x 32
  constexpr int U = 4;
  for (int x0 = all; x0 < pieces; x0 += U * step) {
    uint4 a[U], e[U];
    size_t to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = x0 + u * step;
      if (x < pieces) {
        const int i = x / p.row16, c = x - i * p.row16;
        const size_t from = static_cast<size_t>(moving[i]) * p.row16 + c;
        to[u] = static_cast<size_t>(freed[i]) * p.row16 + c;
        a[u] = k[from];
        e[u] = v[from];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (x0 + u * step < pieces) k[to[u]] = a[u], v[to[u]] = e[u];
  }
}

// Slots from the new length on: weight 0, position -1.
__device__ __forceinline__ void evict_clear(const EvictParams& p, int bh, int from, int all, int step) {
  const size_t row = static_cast<size_t>(bh) * p.Lk;
  for (int j = from + all; j < p.Lk; j += step) {
    p.weight_out[row + j] = 0.f;
    p.pos_out[row + j] = -1;
  }
}

// Shared memory of the kernel below: keys, and its share of the two lists (16 bits per slot).
__host__ __device__ inline int evict_share(int Lk, int copies) { return (Lk / 2 + copies - 1) / copies; }
__host__ __device__ inline size_t evict_smem(int Lk, int copies) {
  return static_cast<size_t>(Lk) * 4 + static_cast<size_t>(evict_share(Lk, copies)) * 4 + 16;
}

// Eviction with rows of up to kEvictRowKeys slots.
//   1. The keep-th largest key, by a radix search with digits of 11, 11 and 10
//      bits over histograms in shared memory.
//   2. Ranks in slot order (ballots within a warp's consecutive slots, prefix
//      sums over the warps) give every freed slot below `keep` and every kept
//      one above it its place in two lists; of equal keys the lower slots are kept.
//   3. The i-th freed slot takes the i-th kept row from above.  Sources and
//      targets are disjoint, so the rows move in place and in any order.
// A single CTA's load/store unit would bound step 3, and a barrier between
// CTAs costs more than the search; so `copies` CTAs per KV head all do steps 1
// and 2 (every one holds all keys, 4 bytes a slot) and share step 3 out, which
// needs nothing from each other.
__global__ void __launch_bounds__(kEvictThreads, 1) attn_cache_evict_kernel(const EvictParams p, int copies) {
  extern __shared__ uint32_t keys[];
  __shared__ int hist[2][kEvictBins];  // counters for even and odd lanes
  __shared__ int warp_sum[32];
  __shared__ int2 warp_pair[32];
  __shared__ int s_digit, s_need;
  const int bh = blockIdx.x / copies, rank = blockIdx.x - bh * copies, b = bh / p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = clamp_len(p.cache_len[b], p.Lk);
  const int keep = p.keep, new_len = min(len, keep);
  const long long recent_from = static_cast<long long>(p.seen[b]) - p.recent;
  const size_t row = static_cast<size_t>(bh) * p.Lk;
  const float* w = p.weight + row;
  const int32_t* pos = p.pos + row;
  float* wo = p.weight_out + row;
  int32_t* po = p.pos_out + row;
  const int all = rank * kEvictThreads + tid, step = copies * kEvictThreads;  // this thread among the head's
  if (all == 0 && bh == b * p.Hkv) p.cache_len_out[b] = new_len;
  if (len <= keep) {
    for (int j = all; j < len; j += step) {
      wo[j] = w[j];
      po[j] = pos[j];
    }
    evict_clear(p, bh, new_len, all, step);
    return;
  }
  // every warp owns consecutive slots, a multiple of 32 of them
  const int per_warp = ((len + 31) / 32 + 31) & ~31;
  const int w0 = min(warp * per_warp, len), w1 = min(w0 + per_warp, len);
  for (int i = tid; i < 2 * kEvictBins; i += kEvictThreads) (&hist[0][0])[i] = 0;
#pragma unroll 8
  for (int j = w0 + lane; j < w1; j += 32) keys[j] = evict_key(w[j], pos[j], recent_from);
  __syncthreads();
  uint32_t prefix = 0;
  int need = keep;  // how many of the slots that match the digits so far are kept
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    const EvictDigit dg = evict_digit(d);
    for (int i = w0; i < w1; i += 32) {
      const uint32_t key = i + lane < w1 ? keys[i + lane] : 0u;
      evict_count(hist[lane & 1], i + lane < w1 && (key & dg.above) == prefix, key, dg);
    }
    __syncthreads();
    // two bins per thread, from the top: thread 0 has the last two
    const int bin0 = kEvictBins - 2 - 2 * tid;
    const int lo = hist[0][bin0] + hist[1][bin0], hi = hist[0][bin0 + 1] + hist[1][bin0 + 1], mine = lo + hi;
    hist[0][bin0] = hist[1][bin0] = hist[0][bin0 + 1] = hist[1][bin0 + 1] = 0;
    int incl = mine;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, k);
      if (lane >= k) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = lane < warp ? warp_sum[lane] : 0;
    before = __reduce_add_sync(0xffffffffu, before) + incl - mine;  // keys in higher bins than this thread's
    if (before < need && need <= before + mine) {  // one thread
      const bool upper = need - before <= hi;
      s_digit = bin0 + upper;
      s_need = need - before - (upper ? 0 : hi);
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << dg.shift;
    need = s_need;
  }
  // ranks
  const uint32_t lower = (1u << lane) - 1u;
  int n_eq = 0;
  for (int i = w0; i < w1; i += 32) n_eq += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && keys[i + lane] == prefix));
  if (lane == 0) warp_sum[warp] = n_eq;
  __syncthreads();
  const int eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0);
  // the slots of one strip of 32: which are kept
  auto kept_of = [&](int i, int& eq) {
    const uint32_t key = i + lane < w1 ? keys[i + lane] : 0u;
    const uint32_t eqs = __ballot_sync(0xffffffffu, i + lane < w1 && key == prefix);
    const bool k = i + lane < w1 && (key > prefix || (key == prefix && eq + __popc(eqs & lower) < need));
    eq += __popc(eqs);
    return k;
  };
  int holes = 0, movers = 0;
  {
    int eq = eq_before;
    for (int i = w0; i < w1; i += 32) {
      const bool k = kept_of(i, eq);
      holes += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && !k && i + lane < keep));
      movers += __popc(__ballot_sync(0xffffffffu, k && i + lane >= keep));
    }
  }
  if (lane == 0) warp_pair[warp] = make_int2(holes, movers);
  __syncthreads();
  const int2 of = warp_pair[lane];
  const int n = __reduce_add_sync(0xffffffffu, of.x);  // freed slots, and as many moving ones
  holes = __reduce_add_sync(0xffffffffu, lane < warp ? of.x : 0);
  movers = __reduce_add_sync(0xffffffffu, lane < warp ? of.y : 0);
  // this CTA's pairs m0 .. m1 - 1, listed in shared memory
  const int share = evict_share(p.Lk, copies), mine_n = (n + copies - 1) / copies;
  const int m0 = min(rank * mine_n, n), m1 = min(m0 + mine_n, n);
  uint16_t* freed = reinterpret_cast<uint16_t*>(keys + p.Lk);
  uint16_t* moving = freed + share;
  {
    int eq = eq_before;
    for (int i = w0; i < w1; i += 32) {
      const int j = i + lane;
      const bool k = kept_of(i, eq);
      const bool hole = j < w1 && !k && j < keep, mover = k && j >= keep;
      const uint32_t hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, mover);
      const int hi = holes + __popc(hb & lower), mi = movers + __popc(mb & lower);
      if (hole && hi >= m0 && hi < m1) freed[hi - m0] = static_cast<uint16_t>(j);
      if (mover && mi >= m0 && mi < m1) moving[mi - m0] = static_cast<uint16_t>(j);
      if (k && j < keep && (i >> 5) % copies == rank) {  // strips are shared out, too
        wo[j] = w[j];
        po[j] = pos[j];
      }
      holes += __popc(hb), movers += __popc(mb);
    }
  }
  __syncthreads();
  evict_move(p, bh, moving, freed, m1 - m0, tid, kEvictThreads);
  evict_clear(p, bh, new_len, all, step);
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
// The same for longer rows, one cluster of CTAs per KV head; each CTA owns a
// consecutive part of the slots and keeps their keys in shared memory (CACHED;
// parts that do not fit are read again in each pass).  Every CTA adds the
// histograms up through distributed shared memory, one cluster barrier per
// digit (a histogram per digit, so none is cleared while others read it);
// prefix sums run over warps and CTAs, and the lists are in the workspace.
template <bool CACHED>
__global__ void __launch_bounds__(kEvictClusterThreads) attn_cache_evict_cluster_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) int hist[3][kEvictBins];
  __shared__ int warp_sum[16];
  __shared__ int2 warp_pair[16];
  __shared__ int s_digit, s_need;
  __shared__ int s_counts[2];
  constexpr int NW = kEvictClusterThreads / 32;
  constexpr int nc = kEvictCluster;  // constant, so that a thread's remote loads are all in flight at once
  const int rank = static_cast<int>(cluster_ctarank());
  const int bh = blockIdx.x / nc, b = bh / p.Hkv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = clamp_len(p.cache_len[b], p.Lk);
  const int keep = p.keep, new_len = min(len, keep);
  const long long recent_from = static_cast<long long>(p.seen[b]) - p.recent;
  const size_t row = static_cast<size_t>(bh) * p.Lk;
  const float* w = p.weight + row;
  const int32_t* pos = p.pos + row;
  float* wo = p.weight_out + row;
  int32_t* po = p.pos_out + row;
  const int all = rank * kEvictClusterThreads + tid, step = nc * kEvictClusterThreads;  // this thread among the cluster's
  if (all == 0 && bh == b * p.Hkv) p.cache_len_out[b] = new_len;
  if (len <= keep) {  // the same for the whole cluster
    for (int j = all; j < len; j += step) {
      wo[j] = w[j];
      po[j] = pos[j];
    }
    evict_clear(p, bh, new_len, all, step);
    return;
  }
  // this CTA's slots [j0, j1); every warp owns a consecutive multiple of 32 of them
  const int per_warp = ((len + nc * NW - 1) / (nc * NW) + 31) & ~31;
  const int j0 = min(rank * NW * per_warp, len), j1 = min(j0 + NW * per_warp, len);
  const int w0 = min(j0 + warp * per_warp, j1), w1 = min(w0 + per_warp, j1);
  auto key_at = [&](int j) { return CACHED ? keys[j - j0] : evict_key(w[j], pos[j], recent_from); };
  for (int i = tid; i < 3 * kEvictBins; i += kEvictClusterThreads) (&hist[0][0])[i] = 0;
  if constexpr (CACHED) {
#pragma unroll 4
    for (int j = w0 + lane; j < w1; j += 32) keys[j - j0] = evict_key(w[j], pos[j], recent_from);
  }
  __syncthreads();
  uint32_t prefix = 0;
  int need = keep;
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    const EvictDigit dg = evict_digit(d);
    for (int i = w0; i < w1; i += 32) {
      const uint32_t key = i + lane < w1 ? key_at(i + lane) : 0u;
      evict_count(hist[d], i + lane < w1 && (key & dg.above) == prefix, key, dg);
    }
    cluster_sync_all();
    // the cluster's counts of this thread's four bins, from the top: thread 0 has the last four
    const int bin0 = kEvictBins - 4 - 4 * tid;
    int4 part[nc], c = make_int4(0, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < nc; ++r) part[r] = ld_cluster_v4(cluster_map(smem_u32(&hist[d][bin0]), r));
#pragma unroll
    for (int r = 0; r < nc; ++r) c.x += part[r].x, c.y += part[r].y, c.z += part[r].z, c.w += part[r].w;
    const int mine = c.x + c.y + c.z + c.w;
    int incl = mine;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, k);
      if (lane >= k) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - mine;  // keys in higher bins than this thread's
#pragma unroll
    for (int k = 0; k < NW; ++k)
      if (k < warp) before += warp_sum[k];
    if (before < need && need <= before + mine) {  // one thread
      int left = need - before, bin = bin0 + 3;
      if (left > c.w) {
        left -= c.w, --bin;
        if (left > c.z) {
          left -= c.z, --bin;
          if (left > c.y) left -= c.y, --bin;
        }
      }
      s_digit = bin;
      s_need = left;
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << dg.shift;
    need = s_need;
  }
  // ranks.  Equal keys before this warp's slots:
  const int eq_bin = static_cast<int>(prefix & 1023u);
  int eq_before = 0, eq_of[nc];
#pragma unroll
  for (int r = 0; r < nc; ++r) eq_of[r] = ld_cluster(cluster_map(smem_u32(&hist[2][eq_bin]), r));
#pragma unroll
  for (int r = 0; r < nc; ++r) eq_before += r < rank ? eq_of[r] : 0;
  int n_eq = 0;
  for (int i = w0; i < w1; i += 32)
    n_eq += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && key_at(i + lane) == prefix));
  if (lane == 0) warp_sum[warp] = n_eq;
  __syncthreads();
  for (int k = 0; k < warp; ++k) eq_before += warp_sum[k];
  const uint32_t lower = (1u << lane) - 1u;
  // the slots of one strip of 32: which are kept
  auto kept_of = [&](int i, int& eq) {
    const uint32_t key = i + lane < w1 ? key_at(i + lane) : 0u;
    const uint32_t eqs = __ballot_sync(0xffffffffu, i + lane < w1 && key == prefix);
    const bool k = i + lane < w1 && (key > prefix || (key == prefix && eq + __popc(eqs & lower) < need));
    eq += __popc(eqs);
    return k;
  };
  int holes = 0, movers = 0;
  {
    int eq = eq_before;
    for (int i = w0; i < w1; i += 32) {
      const bool k = kept_of(i, eq);
      holes += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && !k && i + lane < keep));
      movers += __popc(__ballot_sync(0xffffffffu, k && i + lane >= keep));
    }
  }
  if (lane == 0) warp_pair[warp] = make_int2(holes, movers);
  __syncthreads();
  int hole0 = 0, mover0 = 0;
  for (int k = 0; k < NW; ++k) {
    if (k == warp) holes = hole0, movers = mover0;
    hole0 += warp_pair[k].x, mover0 += warp_pair[k].y;
  }
  if (tid == 0) s_counts[0] = hole0, s_counts[1] = mover0;
  cluster_sync_all();
  int n = 0, h_of[nc], m_of[nc];
#pragma unroll
  for (int r = 0; r < nc; ++r) {
    const uint32_t at = cluster_map(smem_u32(&s_counts[0]), r);
    h_of[r] = ld_cluster(at), m_of[r] = ld_cluster(at + 4);
  }
#pragma unroll
  for (int r = 0; r < nc; ++r) {
    if (r < rank) holes += h_of[r], movers += m_of[r];
    n += h_of[r];
  }
  const int cap = p.Lk / 2;  // min(keep, len - keep) slots at most
  int32_t* freed = p.lists + static_cast<size_t>(bh) * 2 * cap;
  int32_t* moving = freed + cap;
  {
    int eq = eq_before;
    for (int i = w0; i < w1; i += 32) {
      const int j = i + lane;
      const bool k = kept_of(i, eq);
      const uint32_t hb = __ballot_sync(0xffffffffu, j < w1 && !k && j < keep);
      const uint32_t mb = __ballot_sync(0xffffffffu, k && j >= keep);
      if (j < w1 && !k && j < keep) freed[holes + __popc(hb & lower)] = j;
      if (k && j >= keep) moving[movers + __popc(mb & lower)] = j;
      if (k && j < keep) {
        wo[j] = w[j];
        po[j] = pos[j];
      }
      holes += __popc(hb), movers += __popc(mb);
    }
  }
  cluster_sync_all();  // the lists are written (and no CTA's shared memory is read any more)
  evict_move(p, bh, moving, freed, n, all, step);
  evict_clear(p, bh, new_len, all, step);
}

}  // namespace gbattn
