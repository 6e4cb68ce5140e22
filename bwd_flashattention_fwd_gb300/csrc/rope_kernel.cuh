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
// exchange and the norm's sums take log2(D / 16) shuffles.
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

// A CTA takes an equal share of the tokens (and, where there are fewer tokens
// than CTAs, of the heads) in chunks of up to kRopeChunk: the chunk's sines and
// cosines go to shared memory once, then its rows (head by head, the chunk's
// tokens of each) go round the CTA's groups of lanes, each row loaded while the
// one before it is worked on.
constexpr int kRopeChunk = 8;

template <int D, bool BF16, bool INTERLEAVED, bool BWD>
__global__ void __launch_bounds__(kRopeThreads, BWD ? kRopeBwdPerSm : kRopeFwdPerSm) rope_kernel(const RopeParams p, int parts) {
  using Gm = RowLanes<D>;
  constexpr int GROUPS = kRopeThreads / Gm::GROUP, WARPS = kRopeThreads / 32;
  __shared__ uint64_t frac[D / 2];
  __shared__ __align__(16) float cs[kRopeChunk][2][D / 2];  // cosines, sines
  __shared__ float dw_sum[BWD ? WARPS : 1][BWD ? D : 1];
  grid_dependency_wait();  // the kernels before this one are complete
  if (threadIdx.x == 0) grid_launch_dependents();
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < D / 2; i += kRopeThreads) frac[i] = i < half ? turn_fraction(p.freq[i]) : 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = lane % Gm::GROUP, group = threadIdx.x / Gm::GROUP;
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
  // the first of its pairs in each half of the eight; pairs that are not turned have cosine 1, sine 0
  const int pair0 = INTERLEAVED ? 4 * c0 : 8 * j, pair1 = INTERLEAVED ? 4 * c1 : 8 * j + 4;
  const bool turns0 = on && pair0 < half, turns1 = on && pair1 < half;
  const bool norm = p.w[0] != nullptr;
  const long long tokens = static_cast<long long>(p.B) * p.L;
  const int part = blockIdx.x % parts;
  const long long block = blockIdx.x / parts, blocks = gridDim.x / parts;
  const long long t_first = tokens * block / blocks, t_end = tokens * (block + 1) / blocks;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const RowsView xv = p.x[which], dv = p.dx[which];
    uint16_t* const y = static_cast<uint16_t*>(p.y[which]);
    const int H = xv.H, h_lo = H * part / parts, h_hi = H * (part + 1) / parts;
    uint4 wp[2] = {};
    if (norm && on) {
      const uint4* w = static_cast<const uint4*>(p.w[which]);
      wp[0] = __ldg(w + c0), wp[1] = __ldg(w + c1);
    }
    float dw[BWD ? 16 : 1];
#pragma unroll
    for (float& x : dw) x = 0.f;
#pragma unroll 1
    for (long long t0 = t_first; t0 < t_end; t0 += kRopeChunk) {
      // the chunk: n tokens, rows in slots of 2^shift per head
      const int n = static_cast<int>(t_end - t0 < kRopeChunk ? t_end - t0 : kRopeChunk);
      const int shift = n > 4 ? 3 : n > 2 ? 2 : n > 1 ? 1 : 0;
      const int t = group & ((1 << shift) - 1), stride = GROUPS >> shift;  // a group's rows are all of one token
      const long long token = t0 + t;
      const int b = static_cast<int>(token / p.L), l = static_cast<int>(token - static_cast<long long>(b) * p.L);
      const int h0 = h_lo + (group >> shift);  // the group's first head
      const int rows = t < n && on && h0 < h_hi ? (h_hi - h0 + stride - 1) / stride : 0;  // of this lane
      const int rounds = (h_hi - h_lo + stride - 1) / stride;  // of the CTA: the shuffles take whole warps
      const uint16_t* xr = static_cast<const uint16_t*>(xv.at) + b * xv.sb + l * xv.sl + h0 * xv.sh;
      uint16_t* yr = y + ((static_cast<size_t>(b) * H + h0) * p.L + l) * D;
      uint16_t* dr = BWD ? static_cast<uint16_t*>(dv.at) + b * dv.sb + l * dv.sl + h0 * dv.sh : nullptr;
      const int64_t step_x = stride * xv.sh, step_y = static_cast<int64_t>(stride) * p.L * D, step_d = stride * dv.sh;
      auto inside = [&](const uint16_t* at, const RowsView& v, int site) {
        return dbg_in_range(at - static_cast<const uint16_t*>(v.at), D, (p.B - 1) * v.sb + (v.H - 1) * v.sh + (p.L - 1) * v.sl + D, p.status, site);
      };
      auto inside_y = [&](const uint16_t* at, int site) {
        return dbg_in_range(at - y, D, static_cast<size_t>(p.B) * H * p.L * D, p.status, site);
      };
      uint4 xn[2] = {}, gn[2] = {};
      auto load = [&](int i) {  // row i, at xr (and yr)
        if (i >= rows) return;
        if ((!BWD || norm) && inside(xr, xv, 100)) {
          const uint4* v = reinterpret_cast<const uint4*>(xr);
          xn[0] = v[c0], xn[1] = v[c1];
        }
        if (BWD && inside_y(yr, 101)) {
          const uint4* v = reinterpret_cast<const uint4*>(yr);
          gn[0] = v[c0], gn[1] = v[c1];
        }
      };
      load(0);
      __syncthreads();  // frac; the chunk before is done with cs
      for (int i = threadIdx.x; i < n * half; i += kRopeThreads) {
        const int ti = i / half, pair = i - ti * half;
        int a = p.axis ? __ldg(p.axis + pair) : 0;
        a = a < p.axes ? a : p.axes - 1;
        float c, s;
        turn(__ldg(p.pos + a * tokens + t0 + ti), frac[pair], c, s);
        cs[ti][0][pair] = c, cs[ti][1][pair] = BWD ? -s : s;
      }
      __syncthreads();
#pragma unroll 1
      for (int i = 0; i < rounds; ++i) {
        const bool live = i < rows;
        uint4 xp[2] = {xn[0], xn[1]}, gp[2] = {gn[0], gn[1]};
        xr += step_x;
        uint16_t* const yi = yr;
        yr += step_y;
        load(i + 1);
        float c[8], s[8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float4 cv = make_float4(1.f, 1.f, 1.f, 1.f), sv = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k ? turns1 : turns0) {
            cv = *reinterpret_cast<const float4*>(&cs[t][0][k ? pair1 : pair0]);
            sv = *reinterpret_cast<const float4*>(&cs[t][1][k ? pair1 : pair0]);
          }
          c[4 * k] = cv.x, c[4 * k + 1] = cv.y, c[4 * k + 2] = cv.z, c[4 * k + 3] = cv.w;
          s[4 * k] = sv.x, s[4 * k + 1] = sv.y, s[4 * k + 2] = sv.z, s[4 * k + 3] = sv.w;
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
          if (live && inside_y(yi, 102)) {
            uint4* v = reinterpret_cast<uint4*>(yi);
            v[c0] = pack8<BF16>(f), v[c1] = pack8<BF16>(f + 8);
          }
        } else {
          unpack8<BF16>(gp[0], f), unpack8<BF16>(gp[1], f + 8);
          rotate16<INTERLEAVED>(f, c, s);
          if (norm) {
            float x[16], ss = 0.f, gx = 0.f;
            unpack8<BF16>(xp[0], x), unpack8<BF16>(xp[1], x + 8);
            float w[16];
            unpack8<BF16>(wp[0], w), unpack8<BF16>(wp[1], w + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss), gx = fmaf(f[e] * w[e], x[e], gx);
            const float r = rsqrtf(group_sum<Gm::GROUP>(ss) * (1.f / D) + p.eps);
            const float m = group_sum<Gm::GROUP>(gx) * (1.f / D) * r * r;
            if (live) {  // (what an idle lane's registers hold adds nothing)
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                dw[e] = fmaf(f[e] * r, x[e], dw[e]);
                f[e] = r * (f[e] * w[e] - x[e] * m);
              }
            }
          }
          if (live && inside(dr, dv, 103)) {
            uint4* v = reinterpret_cast<uint4*>(dr);
            v[c0] = pack8<BF16>(f), v[c1] = pack8<BF16>(f + 8);
          }
          dr += step_d;
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
      if (lane < Gm::GROUP && on) {
#pragma unroll
        for (int e = 0; e < 16; ++e) dw_sum[warp][(e < 8 ? c0 : c1) * 8 + (e & 7)] = dw[e];
      }
      __syncthreads();
      for (int d = threadIdx.x; d < D; d += kRopeThreads) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) x += dw_sum[w][d];
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
