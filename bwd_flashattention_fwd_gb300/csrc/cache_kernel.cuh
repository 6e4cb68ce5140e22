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

constexpr int kEvictThreads = 1024;

// Order of the slots as an unsigned key, larger = kept first: recent slots
// above all, then by weight (the usual monotone map of IEEE bits; -0 equals
// +0, NaN is below everything).
__device__ __forceinline__ uint32_t evict_key(float w, int pos, long long recent_from) {
  if (pos >= recent_from) return 0xffffffffu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the block of three counts at once; totals in tot.
__device__ __forceinline__ int3 block_scan3(int3 x, int3* warp_sums, int3& tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int3 s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, s.x, d), b = __shfl_up_sync(0xffffffffu, s.y, d),
              c = __shfl_up_sync(0xffffffffu, s.z, d);
    if (lane >= d) s.x += a, s.y += b, s.z += c;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int3 w = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, w.x, d), b = __shfl_up_sync(0xffffffffu, w.y, d),
                c = __shfl_up_sync(0xffffffffu, w.z, d);
      if (lane >= d) w.x += a, w.y += b, w.z += c;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  int3 base = make_int3(0, 0, 0);
  if (warp > 0) base = warp_sums[warp - 1];
  tot = warp_sums[31];
  __syncthreads();
  return make_int3(base.x + s.x - x.x, base.y + s.y - x.y, base.z + s.z - x.z);
}

// One block per KV head: the keep-th largest key by a radix search (8 bits a
// pass), then one pass in slot order that lists freed slots and moving tokens
// (ranks by prefix sums, so ties go to the lower slot), then the moves.
__global__ void __launch_bounds__(kEvictThreads) attn_cache_evict_kernel(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int3 warp_sums[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int bh = blockIdx.x, b = bh / p.Hkv, tid = threadIdx.x;
  const int len = clamp_len(p.cache_len[b], p.Lk);
  const int keep = p.keep;
  const long long recent_from = static_cast<long long>(p.seen[b]) - p.recent;
  const size_t row = static_cast<size_t>(bh) * p.Lk;
  const float* w = p.weight + row;
  const int32_t* pos = p.pos + row;
  float* wo = p.weight_out + row;
  int32_t* po = p.pos_out + row;
  const int new_len = min(len, keep);
  if (tid == 0 && bh == b * p.Hkv) p.cache_len_out[b] = new_len;
  for (int j = new_len + tid; j < p.Lk; j += kEvictThreads) {
    wo[j] = 0.f;
    po[j] = -1;
  }
  if (len <= keep) {
    for (int j = tid; j < len; j += kEvictThreads) {
      wo[j] = w[j];
      po[j] = pos[j];
    }
    return;
  }
  // the keep-th largest key; `need` of the slots that equal it are kept
  uint32_t prefix = 0;
  int need = keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kEvictThreads) hist[i] = 0;
    __syncthreads();
    for (int j = tid; j < len; j += kEvictThreads) {
      const uint32_t key = evict_key(w[j], pos[j], recent_from);
      if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int d = 255, left = need;
      while (d > 0 && hist[d] < left) left -= hist[d--];
      s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  const int cap = p.Lk / 2;
  int32_t* freed = p.lists + static_cast<size_t>(bh) * 2 * cap;
  int32_t* moving = freed + cap;
  int eq_base = 0, free_base = 0, move_base = 0;
  for (int j0 = 0; j0 < len; j0 += kEvictThreads) {
    const int j = j0 + tid;
    const bool in = j < len;
    const uint32_t key = in ? evict_key(w[j], pos[j], recent_from) : 0u;
    const bool eq = in && key == prefix;
    int3 tot;
    const int3 r = block_scan3(make_int3(eq, 0, 0), warp_sums, tot);
    const bool kept = in && (key > prefix || (eq && eq_base + r.x < need));
    eq_base += tot.x;
    const bool hole = in && !kept && j < keep, mover = kept && j >= keep;
    const int3 r2 = block_scan3(make_int3(hole, mover, 0), warp_sums, tot);
    if (hole) freed[free_base + r2.x] = j;
    if (mover) moving[move_base + r2.y] = j;
    if (kept && j < keep) {
      wo[j] = w[j];
      po[j] = pos[j];
    }
    free_base += tot.x;
    move_base += tot.y;
  }
  __syncthreads();
  const int n = min(free_base, move_base);  // equal: as many kept slots above as freed ones below
  uint4* k = static_cast<uint4*>(p.k) + static_cast<size_t>(bh) * p.kv_pitch * p.row16;
  uint4* v = static_cast<uint4*>(p.v) + static_cast<size_t>(bh) * p.kv_pitch * p.row16;
  for (int i = tid; i < n; i += kEvictThreads) {
    wo[freed[i]] = w[moving[i]];
    po[freed[i]] = pos[moving[i]];
  }
  for (long long x = tid; x < static_cast<long long>(n) * p.row16; x += kEvictThreads) {
    const int i = static_cast<int>(x / p.row16), c = static_cast<int>(x - static_cast<long long>(i) * p.row16);
    const size_t s = static_cast<size_t>(moving[i]) * p.row16 + c, d = static_cast<size_t>(freed[i]) * p.row16 + c;
    const uint4 a = k[s], e = v[s];
    k[d] = a;
    v[d] = e;
  }
}

}  // namespace gbattn
