// Accumulated attention weight per key: thread = key, query rows in order.
#pragma once

#include "cache.h"
#include "kernel_common.cuh"

namespace gbattn {

constexpr int kKeyWeightKeys = 64;

template <int D, bool BF16>
__global__ void __launch_bounds__(kKeyWeightKeys) attn_key_weight_kernel(const KeyWeightParams p) {
  using E = Elem<BF16>;
  __shared__ float qs[D];
  extern __shared__ float ks[];  // [D][64]
  const int bhk = blockIdx.y, b = bhk / p.Hkv;
  const int j = blockIdx.x * kKeyWeightKeys + threadIdx.x;
  const size_t krow = static_cast<size_t>(bhk) * p.kv_pitch + j;
  if (j < p.Lk)
    for (int d = 0; d < D; ++d) ks[d * kKeyWeightKeys + threadIdx.x] = static_cast<float>(static_cast<const typename E::T*>(p.k)[krow * D + d]);
  float sum = 0.f;
  const int rows = p.G * p.Lq;
  for (int r = 0; r < rows; ++r) {
    const size_t qrow = static_cast<size_t>(bhk) * rows + r;
    const int i = r % p.Lq;
    const int lim = p.limit ? min(max(p.limit[static_cast<size_t>(b) * p.Lq + i], 0), p.Lk)
                            : p.causal ? i + (p.Lk - p.Lq) + 1 : p.Lk;
    if (lim <= blockIdx.x * kKeyWeightKeys) continue;
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kKeyWeightKeys) qs[d] = static_cast<float>(static_cast<const typename E::T*>(p.q)[qrow * D + d]);
    __syncthreads();
    if (j < lim) {
      float s = 0.f;
      for (int d = 0; d < D; ++d) s = fmaf(qs[d], ks[d * kKeyWeightKeys + threadIdx.x], s);
      sum += exp2f(s * p.scale_log2 - p.lse[qrow]);
    }
  }
  if (j < p.Lk) {
    const size_t o = static_cast<size_t>(bhk) * p.Lk + j;
    p.weight_out[o] = (p.weight ? p.weight[o] : 0.f) + sum;
  }
}

}  // namespace gbattn
