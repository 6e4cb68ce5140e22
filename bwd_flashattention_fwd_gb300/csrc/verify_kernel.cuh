// Verification of a chain of drafted tokens against the target's
// probabilities, from given uniform numbers (rejection sampling).
//
//   draft i is accepted while u_i q_i(x_i) < p_i(x_i), all before it accepted;
//   n accepted; the next token is drawn from the residual max(p_n - q_n, 0) of
//   the first rejected draft, or from p_n if none was rejected: the least x with
//   sum_{y <= x} w(y) > r sum w.
//
// Bound by reading one row of p and one of q per sequence (2 x 608 KB at 151936
// tokens), and for few sequences by latency: a cluster of CTAs shares a row,
// their sums meet in distributed shared memory.
//
// The token is a comparison of sums of up to 10^5 terms with a threshold
// between them, so the sums are exact: probabilities are taken as multiples of
// 2^-60 in 64-bit integers, whose sum depends on no order.  (32-bit floating
// sums choose another token in a few draws out of a hundred; 64-bit floating
// additions would take 25 us at 64 sequences on this GPU.)
#pragma once

#include "kernel_common.cuh"
#include "step.h"

namespace gbattn {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyCluster = 8;

// floor(x 2^60) of a probability; what is negative or NaN counts as 0, what is above 1 as 1.
__device__ __forceinline__ uint64_t prob_fixed(float x) {
  if (!(x > 0.f)) return 0;
  x = fminf(x, 1.f);
  const uint32_t bits = __float_as_uint(x);
  const int s = static_cast<int>(bits >> 23) - 90;
  const uint32_t m = (bits & 0x7fffffu) | 0x800000u;
  return s >= 0 ? static_cast<uint64_t>(m) << s : static_cast<uint64_t>(m >> min(-s, 31));
}

// The weight of a token: its probability, less the draft's where one was rejected (lost: the point where a
// deterministic draft's whole probability lies, or -1).
__device__ __forceinline__ uint64_t residual(float p, float q, bool lost) {
  const uint64_t a = prob_fixed(p), b = prob_fixed(q);
  return lost || a <= b ? 0 : a - b;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// A cluster per sequence; warp w of CTA c holds a contiguous part of the vocabulary.  VEC: rows start on 16 bytes.
template <bool VEC>
__global__ void __launch_bounds__(kVerifyThreads) attn_draft_verify_kernel(const VerifyParams p) {
  constexpr int WARPS = kVerifyThreads / 32, W = VEC ? 4 : 1;
  __shared__ int cut;
  __shared__ uint64_t part[2][WARPS];  // sums of this CTA's warps (second row: of p alone, where the residual is empty)
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int b = blockIdx.x / kVerifyCluster, c = blockIdx.x % kVerifyCluster;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int most = p.draft_len ? clamp_len(p.draft_len[b], p.T) : p.T;
  if (threadIdx.x == 0) cut = most;
  __syncthreads();
  for (int i = threadIdx.x; i < most; i += kVerifyThreads) {
    const int x = p.tokens[static_cast<size_t>(b) * p.T + i];
    bool good = x >= 0 && x < p.V;
    if (good) {
      const float t = p.target[(static_cast<size_t>(b) * (p.T + 1) + i) * p.V + x];
      const float q = p.draft ? p.draft[(static_cast<size_t>(b) * p.T + i) * p.V + x] : 1.f;
      // exact: 48 bits of product
      good = static_cast<double>(p.u[static_cast<size_t>(b) * p.T + i]) * static_cast<double>(q) < static_cast<double>(t);
    }
    if (!good) atomicMin(&cut, i);
  }
  __syncthreads();
  const int n = cut;
  const bool rejected = n < most;
  const float* prow = p.target + (static_cast<size_t>(b) * (p.T + 1) + n) * p.V;
  const float* qrow = rejected && p.draft ? p.draft + (static_cast<size_t>(b) * p.T + n) * p.V : nullptr;
  const int point = rejected && !p.draft ? p.tokens[static_cast<size_t>(b) * p.T + n] : -1;
  // parts: multiples of 32 W tokens
  const int per = ((p.V + kVerifyCluster * WARPS - 1) / (kVerifyCluster * WARPS) + 32 * W - 1) / (32 * W) * (32 * W);
  const long long lo = static_cast<long long>(c * WARPS + warp) * per;
  const int from = static_cast<int>(lo < p.V ? lo : p.V), to = static_cast<int>(lo + per < p.V ? lo + per : p.V);

  auto load = [&](int x, float (&a)[W], float (&q)[W]) {  // tokens x .. x + W - 1 of this lane (zeros past the part)
#pragma unroll
    for (int k = 0; k < W; ++k) a[k] = q[k] = 0.f;
    if (x >= to) return;
    if constexpr (VEC) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(prow + x));
      a[0] = v.x, a[1] = v.y, a[2] = v.z, a[3] = v.w;
      if (qrow) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(qrow + x));
        q[0] = w.x, q[1] = w.y, q[2] = w.z, q[3] = w.w;
      }
    } else {
      a[0] = __ldg(prow + x);
      if (qrow) q[0] = __ldg(qrow + x);
    }
  };

  uint64_t sum = 0;
#pragma unroll 4
  for (int x = from + lane * W; x < to; x += 32 * W) {
    float a[W], q[W];
    load(x, a, q);
#pragma unroll
    for (int k = 0; k < W; ++k) sum += residual(a[k], q[k], x + k == point);
  }
  sum = warp_sum(sum);
  if (lane == 0) part[0][warp] = sum;
  cluster_sync_all();
  const uint32_t at = smem_u32(&part[0][0]);
  // every warp: all parts' sums (128 of them, four a lane), their total and what lies before its own
  auto totals = [&](int which, uint64_t& total, uint64_t& before) {
    total = before = 0;
#pragma unroll
    for (int i = 0; i < kVerifyCluster * WARPS / 32; ++i) {
      const int w = i * 32 + lane;
      const uint64_t v = ld_cluster_u64(cluster_map(at + (which * WARPS + w % WARPS) * 8, w / WARPS));
      total += v;
      if (w < c * WARPS + warp) before += v;
    }
    total = warp_sum(total), before = warp_sum(before);
  };
  uint64_t total, before;
  totals(0, total, before);
  bool whole = false;
  if (total == 0 && rejected) {  // nothing is left (the same for the whole cluster): p itself
    whole = true;
    sum = 0;
    for (int x = from + lane * W; x < to; x += 32 * W) {
      float a[W], q[W];
      load(x, a, q);
#pragma unroll
      for (int k = 0; k < W; ++k) sum += prob_fixed(a[k]);
    }
    sum = warp_sum(sum);
    if (lane == 0) part[1][warp] = sum;
    cluster_sync_all();
    totals(1, total, before);
  }
  // r as a multiple of 2^-64 (a float below 1 has 24 bits, so this is exact from 2^-40 up)
  const float r = p.r[b];
  uint64_t rf = 0;
  if (r >= 1.f) {
    rf = ~0ull;
  } else if (r > 0.f) {
    const uint32_t bits = __float_as_uint(r);
    const int s = static_cast<int>(bits >> 23) - 86;
    const uint32_t m = (bits & 0x7fffffu) | 0x800000u;
    rf = s >= 0 ? static_cast<uint64_t>(m) << s : static_cast<uint64_t>(m >> min(-s, 31));
  }
  const uint64_t limit = __umul64hi(rf, total);  // floor(r total): a sum of integers is above r total where it is above this
  if (threadIdx.x == 0 && c == 0) {
    p.accept_len[b] = n;
    if (total == 0) p.token[b] = -1;
  }
  if (before <= limit && limit < before + sum) {  // this warp's part holds the token
    uint64_t run = before;
    for (int x0 = from; x0 < to; x0 += 32 * W) {
      const int x = x0 + lane * W;
      float a[W], q[W];
      load(x, a, q);
      uint64_t v[W], mine = 0;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        v[k] = x + k < to ? (whole ? prob_fixed(a[k]) : residual(a[k], q[k], x + k == point)) : 0;
        mine += v[k];
      }
      uint64_t upto = mine;  // inclusive sums over the lanes
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, upto, m);
        if (lane >= m) upto += o;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, run + upto > limit);
      if (hit) {
        if (lane == __ffs(static_cast<int>(hit)) - 1) {
          uint64_t s = run + upto - mine;
          int k = 0;
#pragma unroll
          for (int i = 0; i < W - 1; ++i) {
            s += v[i];
            if (s <= limit && k == i) k = i + 1;
          }
          p.token[b] = x + k;
        }
        break;
      }
      run += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  cluster_sync_all();  // no CTA leaves while others read its sums
}

}  // namespace gbattn
