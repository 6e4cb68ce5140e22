// RMS norm of every head's query or key row and its rotation by the token's
// position, in one pass, and the gradient of both.
//
//   n = x * r * w,  r = 1 / sqrt(mean x^2 + eps)            (w null: n = x)
//   a pair (n_a, n_b) turns by  t = pos[axis] * freq:       y = (n_a c - n_b s, n_b c + n_a s)
// and backward, with g = dy turned by -t:
//   dw = sum over rows of g x r,   dx = r (g w - x r^2 mean(g w x))   (w null: dx = g)
//
// Bound by memory traffic: 40 heads x 8192 tokens, D = 128 are 168 MB forward
// and 252 MB backward.  A row belongs to D / 16 lanes, each with two 16-byte
// pieces that hold both members of its eight pairs, so the rotation needs no
// exchange and the norm's sums take log2(D / 16) shuffles.  A lane keeps its
// token's eight sines and cosines in registers over all heads it works on.
//
// Angles.  pos * freq of a far position loses its fraction in 32 bits (2^20
// radians leave 4 bits behind the point), so freq is taken once per CTA as a
// 64-bit fraction of a turn, F = freq / 2 pi mod 1, and pos * F mod 1 is an
// integer product that wraps: exact to pos * 2^-63 turns.
#pragma once

#include "row_lanes.cuh"
#include "step.h"

namespace gbattn {

// freq / (2 pi) mod 1 in units of 2^-64 turns (two's complement for a negative freq).
__device__ __forceinline__ uint64_t turn_fraction(float freq) {
  constexpr uint64_t kInvTwoPi = 0x28be60db9391054aull;  // 2^64 / (2 pi)
  const uint32_t bits = __float_as_uint(freq), e = (bits >> 23) & 255u;
  const uint32_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  const uint64_t lo = kInvTwoPi * m, hi = __umul64hi(kInvTwoPi, m);
  const int s = 150 - static_cast<int>(e ? e : 1u);  // freq = m 2^-s
  uint64_t f;
  if (s >= 128)
    f = 0;
  else if (s >= 64)
    f = hi >> (s - 64);
  else if (s > 0)
    f = (hi << (64 - s)) | (lo >> s);
  else
    f = s > -64 ? lo << -s : 0;
  return bits >> 31 ? 0 - f : f;
}

// cos and sin of pos * F turns (the upper 32 bits of the product are the angle: 2^-32 of a turn).
__device__ __forceinline__ void turn(int pos, uint64_t F, float& c, float& s) {
  const uint32_t fl = static_cast<uint32_t>(F), fh = static_cast<uint32_t>(F >> 32), p = static_cast<uint32_t>(pos);
  uint32_t t = p * fh + __umulhi(p, fl);
  if (pos < 0) t -= fl;
  sincospif(static_cast<float>(static_cast<int32_t>(t)) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
}

// Turn the eight pairs of a lane's two pieces f[0..7], f[8..15] by (c, sgn * s).
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate16(float (&f)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int a = INTERLEAVED ? 2 * i : i, b = INTERLEAVED ? 2 * i + 1 : 8 + i;
    const float x = f[a], y = f[b];
    f[a] = x * c[i] - y * s[i];
    f[b] = y * c[i] + x * s[i];
  }
}

// Units of work: a token and ROWS * per heads of q, then those of k.  `per` is
// the heads a lane goes through with one set of sines.
template <int D, bool BF16, bool INTERLEAVED, bool BWD>
__global__ void __launch_bounds__(kRopeThreads, BWD ? 2 : 3) rope_kernel(const RopeParams p, int per) {
  using Gm = RowLanes<D>;
  __shared__ uint64_t frac[D / 2];
  __shared__ float dw_sum[BWD ? kRopeThreads / 32 : 1][BWD ? D : 1];
  grid_dependency_wait();  // the kernels before this one are complete
  if (threadIdx.x == 0) grid_launch_dependents();
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < D / 2; i += kRopeThreads) frac[i] = i < half ? turn_fraction(p.freq[i]) : 0;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = lane % Gm::GROUP, row = lane / Gm::GROUP;
  const bool on = j < Gm::LANES;
  // The lane's pieces (8 elements each).  Halves: both members of the pairs 8 j ..
  // 8 j + 7, and what is not turned in equal shares; interleaved: any two.
  const int turned = p.rot / 16;
  int c0, c1;
  if (INTERLEAVED || j >= turned) {
    const int k = INTERLEAVED ? j : j - turned, base = INTERLEAVED ? 0 : 2 * turned;
    c0 = base + k;
    c1 = c0 + (INTERLEAVED ? D / 16 : D / 16 - turned);
  } else {
    c0 = j;
    c1 = j + turned;
  }
  const long long tokens = static_cast<long long>(p.B) * p.L;
  const long long n_warps = static_cast<long long>(gridDim.x) * (kRopeThreads / 32);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int H = p.x[which].H, step = Gm::ROWS * per, blocks = (H + step - 1) / step;
    const bool norm = p.w[which] != nullptr;
    uint4 wp[2] = {};
    if (norm && on) {
      const uint4* w = static_cast<const uint4*>(p.w[which]);
      wp[0] = __ldg(w + c0), wp[1] = __ldg(w + c1);
    }
    float dw[BWD ? 16 : 1];
#pragma unroll
    for (float& x : dw) x = 0.f;
#pragma unroll 1
    for (long long unit = static_cast<long long>(blockIdx.x) * (kRopeThreads / 32) + warp; unit < tokens * blocks;
         unit += n_warps) {
      const long long token = unit / blocks;
      const int hb = static_cast<int>(unit - token * blocks);
      const int b = static_cast<int>(token / p.L), l = static_cast<int>(token - static_cast<long long>(b) * p.L);
      const int h0 = hb * step + row;
      const uint16_t* xrow = static_cast<const uint16_t*>(p.x[which].at) + b * p.x[which].sb + l * p.x[which].sl;
      const size_t y0 = (static_cast<size_t>(b) * H * p.L + l) * D;
      [[maybe_unused]] const size_t n_x = (p.B - 1) * p.x[which].sb + (H - 1) * p.x[which].sh + (p.L - 1) * p.x[which].sl + D;
      [[maybe_unused]] const size_t n_y = static_cast<size_t>(p.B) * H * p.L * D;
      float c[8], s[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int pair = INTERLEAVED ? (i < 4 ? 4 * c0 + i : 4 * c1 + i - 4) : 8 * j + i;
        c[i] = 1.f, s[i] = 0.f;
        if (on && pair < half) {
          int a = p.axis ? p.axis[pair] : 0;
          a = a < p.axes ? a : p.axes - 1;
          turn(__ldg(p.pos + a * tokens + token), frac[pair], c[i], s[i]);
          if (BWD) s[i] = -s[i];
        }
      }
#pragma unroll 2
      for (int i = 0; i < per; ++i) {
        const int h = h0 + i * Gm::ROWS;
        const bool live = on && h < H;
        const size_t xo = xrow - static_cast<const uint16_t*>(p.x[which].at) + h * p.x[which].sh;
        const size_t yo = y0 + static_cast<size_t>(h) * p.L * D;
        uint4 xp[2] = {}, gp[2] = {};
        if (live && (!BWD || norm) && dbg_in_range(xo, D, n_x, p.status, 100)) {
          const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x[which].at) + xo);
          xp[0] = x[c0], xp[1] = x[c1];
        }
        if (BWD && live && dbg_in_range(yo, D, n_y, p.status, 101)) {
          const uint4* g = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.y[which]) + yo);
          gp[0] = g[c0], gp[1] = g[c1];
        }
        float f[16];
        if constexpr (!BWD) {
          unpack8<BF16>(xp[0], f), unpack8<BF16>(xp[1], f + 8);
          if (norm) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) ss = fmaf(f[e], f[e], ss);
            const float r = rsqrtf(group_sum<Gm::GROUP>(ss) * (1.f / D) + p.eps);
            float w[16];
            unpack8<BF16>(wp[0], w), unpack8<BF16>(wp[1], w + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] *= r * w[e];
          }
          rotate16<INTERLEAVED>(f, c, s);
          if (live && dbg_in_range(yo, D, n_y, p.status, 102)) {
            uint4* y = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y[which]) + yo);
            y[c0] = pack8<BF16>(f), y[c1] = pack8<BF16>(f + 8);
          }
        } else {
          unpack8<BF16>(gp[0], f), unpack8<BF16>(gp[1], f + 8);
          rotate16<INTERLEAVED>(f, c, s);
          if (norm) {
            float x[16], w[16], ss = 0.f, gx = 0.f;
            unpack8<BF16>(xp[0], x), unpack8<BF16>(xp[1], x + 8);
            unpack8<BF16>(wp[0], w), unpack8<BF16>(wp[1], w + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss), gx = fmaf(f[e] * w[e], x[e], gx);
            const float r = rsqrtf(group_sum<Gm::GROUP>(ss) * (1.f / D) + p.eps);
            const float m = group_sum<Gm::GROUP>(gx) * (1.f / D) * r * r;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              dw[e] = fmaf(f[e] * r, x[e], dw[e]);
              f[e] = r * (f[e] * w[e] - x[e] * m);
            }
          }
          const size_t dxo = b * p.dx[which].sb + l * p.dx[which].sl + h * p.dx[which].sh;
          if (live && dbg_in_range(dxo, D, (p.B - 1) * p.dx[which].sb + (H - 1) * p.dx[which].sh +
                                               (p.L - 1) * p.dx[which].sl + D, p.status, 103)) {
            uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dx[which].at) + dxo);
            d[c0] = pack8<BF16>(f), d[c1] = pack8<BF16>(f + 8);
          }
        }
      }
    }
    if constexpr (BWD) {
      if (!norm) continue;
      // rows of the warp, then its CTA's warps, in a fixed order
#pragma unroll
      for (int e = 0; e < 16; ++e)
#pragma unroll
        for (int m = Gm::GROUP; m < 32; m <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], m);
      __syncthreads();
      if (row == 0 && on) {
#pragma unroll
        for (int e = 0; e < 16; ++e) dw_sum[warp][(e < 8 ? c0 : c1) * 8 + (e & 7)] = dw[e];
      }
      __syncthreads();
      for (int d = threadIdx.x; d < D; d += kRopeThreads) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kRopeThreads / 32; ++w) x += dw_sum[w][d];
        p.part[(static_cast<size_t>(blockIdx.x) * 2 + which) * D + d] = x;
      }
    }
  }
}

// dw = the CTAs' partial sums, in a fixed order: a block per 32 columns, a warp per eighth of the CTAs.
__global__ void __launch_bounds__(256) rope_dw_kernel(const RopeParams p, int n) {
  __shared__ float sum[8][32];
  grid_dependency_wait();
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
  const int which = col / p.D, d = col - which * p.D;
  float x = 0.f;
#pragma unroll 8
  for (int i = warp; i < n; i += 8) x += p.part[(static_cast<size_t>(i) * 2 + which) * p.D + d];
  sum[warp][threadIdx.x & 31] = x;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < 8; ++w) x += sum[w][threadIdx.x & 31];
    p.dw[which][d] = x;
  }
}

}  // namespace gbattn
