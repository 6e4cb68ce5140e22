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
// 2^-45 in integers, whose sum depends on no order.  (32-bit floating sums
// choose another token in a few draws out of a hundred; 64-bit floating
// additions would take 25 us at 64 sequences on this GPU.)
#pragma once

#include "kernel_common.cuh"
#include "step.h"

namespace gbattn {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyCluster = 8;

// A probability as hi 2^-22 + lo 2^-45, both read off the bits of a float that a
// constant pushes into a known binade (so the constants' bits belong to hi and
// lo: differences of two are free of them); the nearest multiple of 2^-45, so a larger
// probability never becomes the smaller one.
struct Fixed {
  int hi, lo;
};
__device__ __forceinline__ Fixed prob_fixed(float x) {  // (0 <= x <= 1)
  const float a = __fadd_rn(x, 3.f), rest = __fsub_rn(x, __fsub_rn(a, 3.f));
  return {__float_as_int(a), __float_as_int(__fmaf_rn(rest, 4194304.f, 1.5f))};
}

// A sum of a few weights max(p - q, 0), in multiples of 2^-45 (32 bits hold 256 terms).
struct FixedSum {
  int hi = 0, lo = 0;
  __device__ __forceinline__ void add(float p, float q) {
    p = __saturatef(p), q = __saturatef(q);  // what is negative or NaN counts as 0, what is above 1 as 1, in the comparison as well
    const Fixed a = prob_fixed(p), b = prob_fixed(q);
    if (p > q) hi += a.hi - b.hi, lo += a.lo - b.lo;
  }
  __device__ __forceinline__ uint64_t value() const {
    return static_cast<uint64_t>(static_cast<long long>(hi) * (1 << 23) + lo);
  }
};

// Sums of weights.  Past 2^19 tokens entries of 1 could add up to 2^64 and more (probabilities come nowhere near): there
// (LONG) sums stop at 2^64 - 1, which is the same in any order, so that a token is still found where
// they first pass r times that.  (At 64 x 151936 tokens 19.0 us with such sums, 18.3 without.)
constexpr int kVerifyLong = 1 << 19;
template <bool LONG>
__device__ __forceinline__ uint64_t plus(uint64_t a, uint64_t b) {
  const uint64_t s = a + b;
  return LONG && s < a ? ~0ull : s;
}
template <bool LONG>
__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int m = 16; m; m >>= 1) x = plus<LONG>(x, __shfl_xor_sync(0xffffffffu, x, m));
  return x;
}

__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// A cluster per sequence; warp w of CTA c holds a contiguous part of the vocabulary.  VEC: rows start on 16 bytes.
template <bool VEC, bool LONG>
__global__ void __launch_bounds__(kVerifyThreads, 4) attn_draft_verify_kernel(const VerifyParams p) {
  constexpr int WARPS = kVerifyThreads / 32, W = VEC ? 4 : 1, STEP = 32 * W;
  __shared__ int cut;
  __shared__ uint64_t part[2][WARPS];  // sums of this CTA's warps (second row: of p alone, where the residual is empty)
  __shared__ uint64_t piece[WARPS];
  __shared__ int chosen;  // the warp whose part holds the token, or -1
  __shared__ uint64_t chosen_before;
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int b = blockIdx.x / kVerifyCluster, c = blockIdx.x % kVerifyCluster;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int most = p.draft_len ? clamp_len(p.draft_len[b], p.T) : p.T;
  const float r = p.r[b];
  if (threadIdx.x == 0) cut = p.T, chosen = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < p.T; i += kVerifyThreads) {  // (all of them: nothing waits for draft_len)
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
  const int n = min(cut, most);
  const bool rejected = n < most;
  const float* prow = p.target + (static_cast<size_t>(b) * (p.T + 1) + n) * p.V;
  const float* qrow = rejected && p.draft ? p.draft + (static_cast<size_t>(b) * p.T + n) * p.V : nullptr;
  const int point = rejected && !p.draft ? p.tokens[static_cast<size_t>(b) * p.T + n] : -1;
  // parts: multiples of 32 W tokens
  const int per = ((p.V + kVerifyCluster * WARPS - 1) / (kVerifyCluster * WARPS) + STEP - 1) / STEP * STEP;
  auto bound = [&](int w) {  // where warp w's part begins (of all warps of the cluster)
    const long long at = static_cast<long long>(w) * per;
    return static_cast<int>(at < p.V ? at : p.V);
  };

  auto load = [&](int x, bool with_q, float (&a)[W], float (&q)[W]) {  // tokens x .. x + W - 1
#pragma unroll
    for (int k = 0; k < W; ++k) q[k] = 0.f;
    if constexpr (kDebugChecks) {
#pragma unroll
      for (int k = 0; k < W; ++k) a[k] = 0.f;
      const size_t row = static_cast<size_t>(b) * p.T + n;
      if (!dbg_in_range((row + b) * p.V + x, W, static_cast<size_t>(p.B) * (p.T + 1) * p.V, p.status, 130)) return;
      if (with_q && !dbg_in_range(row * p.V + x, W, static_cast<size_t>(p.B) * p.T * p.V, p.status, 131)) return;
    }
    if constexpr (VEC) {
      const float4 v = *reinterpret_cast<const float4*>(prow + x);
      a[0] = v.x, a[1] = v.y, a[2] = v.z, a[3] = v.w;
      if (with_q) {
        const float4 w = *reinterpret_cast<const float4*>(qrow + x);
        q[0] = w.x, q[1] = w.y, q[2] = w.z, q[3] = w.w;
      }
    } else {
      a[0] = prow[x];
      if (with_q) q[0] = qrow[x];
    }
  };
  auto sum_of = [&](int from, int to, bool with_q, int without) {  // this lane's share of a part
    uint64_t sum = 0;
    constexpr int N = VEC ? 4 : 8;  // steps whose loads are in flight together
    for (int x0 = from; x0 < to; x0 += N * STEP) {
      const int x = x0 + lane * W;
      float a[N][W], q[N][W];
      if (x0 + N * STEP <= to) {
#pragma unroll
        for (int i = 0; i < N; ++i) load(x + i * STEP, with_q, a[i], q[i]);
      } else {  // the last ones: together too
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
          for (int k = 0; k < W; ++k) a[i][k] = q[i][k] = 0.f;
          if (x + i * STEP < to) load(x + i * STEP, with_q, a[i], q[i]);
        }
      }
      FixedSum s;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < W; ++k) s.add(a[i][k], q[i][k]);
      sum = plus<LONG>(sum, s.value());
    }
    if (without >= from && without < to && (without - from) / W % 32 == lane) {  // a deterministic draft's token has no weight
      FixedSum s;
      s.add(prow[without], 0.f);
      sum -= s.value();
    }
    return sum;
  };

  const int mine = c * WARPS + warp;
  bool with_q = qrow != nullptr;
  int without = point;
  uint64_t sum, total, before;  // of this warp's part, of all, of what lies before the part
  auto add_up = [&](int which) {
    sum = warp_sum<LONG>(sum_of(bound(mine), bound(mine + 1), with_q, without));
    if (lane == 0) part[which][warp] = sum;
    cluster_sync_all();
    total = before = 0;
#pragma unroll
    for (int i = 0; i < kVerifyCluster * WARPS / 32; ++i) {  // all warps' sums, a few a lane
      const int w = i * 32 + lane;
      const uint64_t v = ld_cluster_u64(cluster_map(smem_u32(&part[which][w % WARPS]), w / WARPS));
      total = plus<LONG>(total, v);
      if (w < mine) before = plus<LONG>(before, v);
    }
    total = warp_sum<LONG>(total), before = warp_sum<LONG>(before);
  };
  add_up(0);
  if (total == 0 && rejected) {  // nothing is left (the same for the whole cluster): p itself
    with_q = false, without = -1;
    add_up(1);
  }
  cluster_arrive_all();  // (this CTA has read the others' sums)
  // r as a multiple of 2^-64 (a float below 1 has 24 bits, so this is exact from 2^-40 up)
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
  if (lane == 0 && before <= limit && limit < plus<LONG>(before, sum)) chosen = warp, chosen_before = before;
  __syncthreads();
  if (chosen >= 0) {  // this CTA holds the token: its warps look at that part's steps, WARPS at a time
    const int from = bound(c * WARPS + chosen), to = bound(c * WARPS + chosen + 1);
    uint64_t run = chosen_before;
    for (int x0 = from; x0 < to; x0 += WARPS * STEP) {
      const int x = x0 + warp * STEP + lane * W;
      float a[W], q[W];
#pragma unroll
      for (int k = 0; k < W; ++k) a[k] = q[k] = 0.f;
      if (x < to) load(x, with_q, a, q);
      uint64_t v[W], own = 0;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        FixedSum s;
        s.add(a[k], q[k]);
        v[k] = x + k == without ? 0 : s.value();
        own += v[k];
      }
      uint64_t upto = own;  // inclusive sums over the lanes
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, upto, m);
        if (lane >= m) upto += o;
      }
      if (lane == 31) piece[warp] = upto;
      __syncthreads();
      uint64_t ahead = 0, all = 0;  // sums of the warps before this one, and of all
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const uint64_t y = piece[w];
        if (w < warp) ahead += y;
        all += y;
      }
      const uint64_t s0 = plus<LONG>(run, ahead + (upto - own));
      if (s0 <= limit && limit < plus<LONG>(s0, own)) {  // this lane's tokens
        uint64_t s = s0;
        int k = 0;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
          s = plus<LONG>(s, v[i]);
          if (s <= limit && k == i) k = i + 1;
        }
        p.token[b] = x + k;
      }
      run = plus<LONG>(run, all);
      __syncthreads();
      if (run > limit) break;
    }
  }
  cluster_wait_all();  // no CTA leaves while others read its sums
}

}  // namespace gbattn
