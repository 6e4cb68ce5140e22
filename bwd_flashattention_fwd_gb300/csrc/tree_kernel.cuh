// Attention of drafted tokens over a cache and each other: one block per
// output row, one warp per key in turn, with an online softmax per warp that
// the block merges at the end.
#pragma once

#include "cache.h"
#include "kernel_common.cuh"

namespace gbattn {

constexpr int kTreeThreads = 256;

template <int D, bool BF16>
__global__ void __launch_bounds__(kTreeThreads) attn_tree_kernel(const TreeParams p) {
  using E = Elem<BF16>;
  constexpr int PER = D / 32;
  __shared__ float sm[8], sl[8], so[8][D];
  const int t = blockIdx.x % p.T;
  const int bhq = blockIdx.x / p.T;
  const int b = bhq / p.Hq, hk = (bhq % p.Hq) / p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = min(max(p.cache_len[b], 0), p.Lk);
  const int tl = p.tree_len ? min(max(p.tree_len[b], 0), p.T) : p.T;
  typename E::T* o = static_cast<typename E::T*>(p.o) + static_cast<size_t>(blockIdx.x) * D;
  const typename E::T* q = static_cast<const typename E::T*>(p.q) + static_cast<size_t>(blockIdx.x) * D;
  float qr[PER], acc[PER];
  for (int c = 0; c < PER; ++c) qr[c] = static_cast<float>(q[lane + 32 * c]) * p.scale_log2, acc[c] = 0.f;
  float m = -INFINITY, l = 0.f;
  if (t < tl) {
    const size_t head = static_cast<size_t>(b) * p.Hkv + hk;
    for (int j = warp; j < len + tl; j += 8) {
      const int u = j - len;
      if (u >= 0) {
        const bool see = p.mask ? p.mask[(static_cast<size_t>(b) * p.T + t) * p.T + u] != 0 : u <= t;
        if (!see) continue;
      }
      const size_t off = (u < 0 ? head * p.kv_pitch + j : head * p.T + u) * D;
      const typename E::T* k = static_cast<const typename E::T*>(u < 0 ? p.k : p.k_new) + off;
      const typename E::T* v = static_cast<const typename E::T*>(u < 0 ? p.v : p.v_new) + off;
      float s = 0.f;
      for (int c = 0; c < PER; ++c) s = fmaf(qr[c], static_cast<float>(k[lane + 32 * c]), s);
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      const float mn = fmaxf(m, s), a = exp2f(m - mn), e = exp2f(s - mn);
      l = l * a + e;
      m = mn;
      for (int c = 0; c < PER; ++c) acc[c] = acc[c] * a + e * static_cast<float>(v[lane + 32 * c]);
    }
  }
  for (int c = 0; c < PER; ++c) so[warp][lane + 32 * c] = acc[c];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  __syncthreads();
  if (warp != 0) return;
  float M = -INFINITY, L = 0.f;
  for (int i = 0; i < 8; ++i) M = fmaxf(M, sm[i]);
  const bool empty = M == -INFINITY;
  for (int c = 0; c < PER; ++c) acc[c] = 0.f;
  if (!empty)
    for (int i = 0; i < 8; ++i) {
      const float a = exp2f(sm[i] - M);
      L += sl[i] * a;
      for (int c = 0; c < PER; ++c) acc[c] += so[i][lane + 32 * c] * a;
    }
  for (int c = 0; c < PER; ++c) o[lane + 32 * c] = E::from_float(empty ? 0.f : acc[c] / L);
  if (lane == 0) p.lse[blockIdx.x] = empty ? INFINITY : M + log2f(L);
}

}  // namespace gbattn
