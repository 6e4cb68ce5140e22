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
// radians leave 4 bits behind the point), so freq is taken once per thread as a
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

// A lane's sixteen values as eight pairs of neighbours (two lanes of a 64-bit
// register, which one instruction multiplies or adds).
template <bool BF16>
__device__ __forceinline__ void unpack16(const uint4 (&u)[2], uint64_t (&f)[8]) {
  const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = Elem<BF16>::unpack(w[i]);
    f[i] = f2_pack(v.x, v.y);
  }
}

template <bool BF16>
__device__ __forceinline__ void store16(uint16_t* row, int c0, int c1, const uint64_t (&f)[8]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    f2_unpack(f[i], a, b);
    w[i] = Elem<BF16>::pack(a, b);
  }
  uint4* v = reinterpret_cast<uint4*>(row);
  v[c0] = make_uint4(w[0], w[1], w[2], w[3]);
  v[c1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Turn the eight pairs of a lane's two pieces.  Halves: neighbours f[i] turn with
// f[i + 4], c[i] and s[i] (i < 4) hold two pairs' cosines and sines.
// Interleaved: f[i] is one pair, c[i] = (cos, cos), s[i] = (-sin, sin) (i < 8).
// turn0, turn1: whether the first and the second piece hold pairs (halves: both or neither); what
// is not turned is left alone (turned by nothing, an infinite one would reach its neighbours).
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate16(uint64_t (&f)[8], const uint64_t (&c)[INTERLEAVED ? 8 : 4], const uint64_t (&s)[INTERLEAVED ? 8 : 4],
                                         bool turn0, bool turn1) {
  if constexpr (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!(i < 4 ? turn0 : turn1)) continue;
      float a, b;
      f2_unpack(f[i], a, b);
      f[i] = f2_fma(f[i], c[i], f2_mul(f2_pack(b, a), s[i]));
    }
  } else if (turn0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t a = f[i], b = f[i + 4];
      f[i] = f2_sub(f2_mul(a, c[i]), f2_mul(b, s[i]));
      f[i + 4] = f2_fma(b, c[i], f2_mul(a, s[i]));
    }
  }
}

__device__ __forceinline__ float f2_total(const uint64_t (&f)[2]) {
  float a, b;
  f2_unpack(f2_add(f[0], f[1]), a, b);
  return a + b;
}

// A CTA takes an equal share of the tokens (and, where there are fewer tokens
// than CTAs, of the heads), up to TOKENS of them at a time: their sines and
// cosines and the addresses of their rows go to shared memory, then their rows
// (head by head, every token of each) go round the CTA's groups of lanes.  A
// lane copies its pieces of the rows to come into a ring of its own (cp.async),
// DEPTH rows ahead: that many bytes in flight are more than the registers
// would hold (video prompt: 42 us with one row ahead in registers).
template <int D, bool BWD>
struct RopeGeom {
  static constexpr int GROUPS = kRopeThreads / RowLanes<D>::GROUP;
  static constexpr int PER_SM = BWD ? kRopeBwdPerSm : kRopeFwdPerSm;
  static constexpr int TOKENS = 4096 / D;                       // 16 KB of sines and cosines
  static constexpr int DEPTH = BWD ? 3 : 4;  // (gradient, 8192 tokens: 46.4 us, with 4 47.7, with 5 48.4; video prompt 30.9, with 3 31.1, with 6 31.1)
  static constexpr int PIECES = BWD ? 4 : 2;                    // 16-byte pieces of a row: x (and dy)
  static constexpr int RING = DEPTH * PIECES * kRopeThreads * 16;
  static constexpr int CS = TOKENS * D * 4;                     // [TOKENS][2][D / 2] floats
  static constexpr int ROWS_AT = TOKENS * 6 * 8;                // addresses in x, y and dx, of q and k
  static constexpr int SUMS = BWD ? 2 * kRopeThreads / 32 * D * 4 : 0;
  static constexpr int SMEM = RING + CS + ROWS_AT + SUMS;
};

template <int D, bool BF16, bool INTERLEAVED, bool BWD>
__global__ void __launch_bounds__(kRopeThreads, RopeGeom<D, BWD>::PER_SM) rope_kernel(const RopeParams p, int parts, int per, int more, int inv_half) {
  using Gm = RopeGeom<D, BWD>;
  using Ln = RowLanes<D>;
  constexpr int WARPS = kRopeThreads / 32, DEPTH = Gm::DEPTH;
  extern __shared__ __align__(128) uint8_t smem[];
  float* const cs = reinterpret_cast<float*>(smem + Gm::RING);                                  // [TOKENS][2][D / 2]
  uint64_t* const rows_at = reinterpret_cast<uint64_t*>(smem + Gm::RING + Gm::CS);              // [2][3][TOKENS]
  float* const dw_sum = reinterpret_cast<float*>(smem + Gm::RING + Gm::CS + Gm::ROWS_AT);       // [2][WARPS][D]
  grid_dependency_wait();  // the kernels before this one are complete
  if (threadIdx.x == 0) grid_launch_dependents();
  const int half = p.rot / 2;
  // This thread's part of the sines: one pair, of every `abreast`-th token.  What
  // they need is on its way long before they are worked out.
  // (Divisions cost a decode step as much as its loads: what the host can divide it passes, or passes as a factor of 2^-16.)
  const int abreast = kRopeThreads * inv_half >> 16, my_t = static_cast<int>(threadIdx.x) * inv_half >> 16, pair = threadIdx.x - my_t * half;
  float my_freq = 0.f;
  const int32_t* my_pos = p.pos;
  if (my_t < abreast) {
    my_freq = p.freq[pair];
    int a = p.axis ? p.axis[pair] : 0;
    a = a < p.axes ? a : p.axes - 1;
    my_pos += static_cast<long long>(a) * p.B * p.L;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = lane % Ln::GROUP, group = threadIdx.x / Ln::GROUP;
  const bool on = j < Ln::LANES;
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
  const bool turn0 = INTERLEAVED ? c0 < 2 * turned : j < turned, turn1 = INTERLEAVED ? c1 < 2 * turned : turn0;
  // Where the cosines (and, D / 2 floats on, sines) of its pairs lie in a token's part of cs, in fours: neighbouring
  // lanes' fours side by side.  (What lies there for elements that are not turned is not used.)
  const int four0 = 4 * (INTERLEAVED ? c0 : j), four1 = 4 * (INTERLEAVED ? c1 : D / 16 + j);
  auto place = [](int pair) { return INTERLEAVED ? pair : ((pair >> 2 & 1) * (D / 16) + (pair >> 3)) * 4 + (pair & 3); };
  const bool norm = p.w[0] != nullptr;
  const uint32_t ring = smem_u32(smem) + threadIdx.x * 16;  // piece k of slot s: + (s * PIECES + k) * kRopeThreads * 16
  const int tokens = p.B * p.L;  // (at most 2^30)
  // blocks of `per` tokens, the first `more` of them one more
  const int part = blockIdx.y, block = blockIdx.x;
  const int t_first = block * per + min(block, more), t_end = t_first + per + (block < more ? 1 : 0);
  const int q_lo = p.x[0].H * part / parts, q_n = p.x[0].H * (part + 1) / parts - q_lo;  // heads of q and of k
  const int k_lo = p.x[1].H * part / parts, k_n = p.x[1].H * (part + 1) / parts - k_lo;
  // bytes between heads
  const uint32_t x_head[2] = {static_cast<uint32_t>(p.x[0].sh * 2), static_cast<uint32_t>(p.x[1].sh * 2)};
  const uint32_t d_head[2] = {static_cast<uint32_t>(p.dx[0].sh * 2), static_cast<uint32_t>(p.dx[1].sh * 2)}, y_head = static_cast<uint32_t>(p.L) * (D * 2);
  const int chunks = max(1, (t_end - t_first + Gm::TOKENS - 1) / Gm::TOKENS), each = (t_end - t_first + chunks - 1) / chunks;  // (equal ones)
#pragma unroll 1
  for (int t0 = t_first; t0 < t_end; t0 += each) {
    const int n = min(t_end - t0, each);
    if (t0 != t_first) __syncthreads();  // the tokens before are done with
    constexpr int POS = (Gm::TOKENS + kRopeThreads / (D / 2) - 1) / (kRopeThreads / (D / 2));  // tokens of a thread, at most
    int pos[POS];
#pragma unroll
    for (int i = 0; i < POS; ++i) {
      const int t = my_t + i * abreast;
      const bool in = my_t < abreast && t < n &&
                      dbg_in_range(my_pos + t0 + t - p.pos, 1, static_cast<size_t>(p.axes) * tokens, p.status, 104);
      pos[i] = in ? my_pos[t0 + t] : 0;
    }
    if (threadIdx.x < n) {
      const int token = t0 + threadIdx.x, b = token / p.L, l = token - b * p.L;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        uint64_t* const at = rows_at + which * 3 * Gm::TOKENS + threadIdx.x;
        const int lo = which ? k_lo : q_lo;
        const RowsView &xv = p.x[which], &dv = p.dx[which];
        at[0] = reinterpret_cast<uint64_t>(static_cast<uint16_t*>(xv.at) + (b * xv.sb + l * xv.sl + lo * xv.sh));
        at[Gm::TOKENS] = reinterpret_cast<uint64_t>(static_cast<uint16_t*>(p.y[which]) + ((static_cast<long long>(b) * xv.H + lo) * p.L + l) * D);
        if (BWD) at[2 * Gm::TOKENS] = reinterpret_cast<uint64_t>(static_cast<uint16_t*>(dv.at) + (b * dv.sb + l * dv.sl + lo * dv.sh));
      }
    }
    __syncthreads();
    // Rows head by head, a round of GROUPS of them at a time (whole rounds of q, then of k): this group's row of round
    // r of q is row r * GROUPS + group of q_n * n.  (The shuffles take whole warps.)
    const int q_rounds = (q_n * n + Gm::GROUPS - 1) / Gm::GROUPS, k_rounds = (k_n * n + Gm::GROUPS - 1) / Gm::GROUPS;
    const int inv_n = 65536 / n + 1;  // (exact for what is below 65536 / n)
    const int step_h = Gm::GROUPS * inv_n >> 16, step_t = Gm::GROUPS - step_h * n;
    const int first_h = group * inv_n >> 16, first_t = group - first_h * n;
    auto inside = [&](uint64_t at, const RowsView& v, int site) {
      return dbg_in_range((at - reinterpret_cast<uint64_t>(v.at)) / 2, D, (p.B - 1) * v.sb + (v.H - 1) * v.sh + (p.L - 1) * v.sl + D, p.status, site);
    };
    auto inside_y = [&](uint64_t at, int which, int site) {
      return dbg_in_range((at - reinterpret_cast<uint64_t>(p.y[which])) / 2, D, static_cast<size_t>(p.B) * p.x[which].H * p.L * D, p.status, site);
    };
    int ahead = 0, ahead_h = first_h, ahead_t = first_t;  // the round that is fetched next, and its row
    auto fetch = [&]() {
      const bool is_k = ahead >= q_rounds;
      if (on && ahead < q_rounds + k_rounds && ahead_h < (is_k ? k_n : q_n)) {
        const uint32_t slot = ring + (ahead % DEPTH) * (Gm::PIECES * kRopeThreads * 16);
        const int which = is_k ? 1 : 0;
        const uint64_t* const at = rows_at + which * 3 * Gm::TOKENS + ahead_t;
        const uint64_t xo = at[0] + static_cast<uint64_t>(static_cast<uint32_t>(ahead_h)) * (is_k ? x_head[1] : x_head[0]);
        if ((!BWD || norm) && inside(xo, p.x[which], 100)) {
          const uint4* v = reinterpret_cast<const uint4*>(xo);
          cp_async16(slot, v + c0, true), cp_async16(slot + kRopeThreads * 16, v + c1, true);
        }
        if constexpr (BWD) {
          const uint64_t yo = at[Gm::TOKENS] + static_cast<uint64_t>(static_cast<uint32_t>(ahead_h)) * y_head;
          if (inside_y(yo, which, 101)) {
            const uint4* v = reinterpret_cast<const uint4*>(yo);
            cp_async16(slot + 2 * kRopeThreads * 16, v + c0, true), cp_async16(slot + 3 * kRopeThreads * 16, v + c1, true);
          }
        }
      }
      cp_async_commit();
      ++ahead, ahead_h += step_h, ahead_t += step_t;
      if (ahead_t >= n) ahead_t -= n, ++ahead_h;
      if (ahead == q_rounds) ahead_h = first_h, ahead_t = first_t;
    };
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) fetch();
    {  // (while the first rows are on their way)
      const uint64_t my_frac = turn_fraction(my_freq);
      const int at = place(pair);
#pragma unroll
      for (int i = 0; i < POS; ++i) {
        const int t = my_t + i * abreast;
        if (my_t < abreast && t < n) {
          float c, s;
          turn(pos[i], my_frac, c, s);
          cs[t * D + at] = c, cs[t * D + D / 2 + at] = BWD ? -s : s;
        }
      }
    }
    __syncthreads();
    int round = 0;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const int rounds = which ? k_rounds : q_rounds, h_n = which ? k_n : q_n;
      const uint64_t* const at = rows_at + which * 3 * Gm::TOKENS;
      uint64_t w[8], dw[BWD ? 8 : 1];
      {
        uint4 wp[2] = {};
        if (norm && on) {
          const uint4* v = static_cast<const uint4*>(p.w[which]);
          wp[0] = v[c0], wp[1] = v[c1];
        }
        unpack16<BF16>(wp, w);
      }
#pragma unroll
      for (uint64_t& x : dw) x = 0;
      int h = first_h, t = first_t;
#pragma unroll 1
      for (int i = 0; i < rounds; ++i, ++round) {
        const bool live = on && h < h_n;
        fetch();
        cp_async_wait<DEPTH - 1>();
        const uint32_t slot = ring + (round % DEPTH) * (Gm::PIECES * kRopeThreads * 16);
        // this token's cosines and sines, as rotate16 takes them
        constexpr int NC = INTERLEAVED ? 8 : 4;
        uint64_t c[NC], s[NC];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 cv = *reinterpret_cast<const float4*>(cs + t * D + (k ? four1 : four0));
          const float4 sv = *reinterpret_cast<const float4*>(cs + t * D + D / 2 + (k ? four1 : four0));
          if constexpr (INTERLEAVED) {
            c[4 * k] = f2_pack(cv.x, cv.x), c[4 * k + 1] = f2_pack(cv.y, cv.y), c[4 * k + 2] = f2_pack(cv.z, cv.z), c[4 * k + 3] = f2_pack(cv.w, cv.w);
            s[4 * k] = f2_pack(-sv.x, sv.x), s[4 * k + 1] = f2_pack(-sv.y, sv.y), s[4 * k + 2] = f2_pack(-sv.z, sv.z), s[4 * k + 3] = f2_pack(-sv.w, sv.w);
          } else {
            c[2 * k] = f2_pack(cv.x, cv.y), c[2 * k + 1] = f2_pack(cv.z, cv.w);
            s[2 * k] = f2_pack(sv.x, sv.y), s[2 * k + 1] = f2_pack(sv.z, sv.w);
          }
        }
        uint64_t f[8];
        if constexpr (!BWD) {
          const uint4 xp[2] = {ld_shared_v4(slot), ld_shared_v4(slot + kRopeThreads * 16)};
          unpack16<BF16>(xp, f);
          if (norm) {
            uint64_t ss[2] = {f2_mul(f[0], f[0]), f2_mul(f[1], f[1])};
#pragma unroll
            for (int e = 2; e < 8; ++e) ss[e & 1] = f2_fma(f[e], f[e], ss[e & 1]);
            const float r = rsqrtf(group_sum<Ln::GROUP>(on ? f2_total(ss) : 0.f) * (1.f / D) + p.eps);
            const uint64_t rr = f2_pack(r, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f2_mul(f2_mul(f[e], rr), w[e]);
          }
          rotate16<INTERLEAVED>(f, c, s, turn0, turn1);
          if (live) {
            const uint64_t yo = at[Gm::TOKENS + t] + static_cast<uint64_t>(static_cast<uint32_t>(h)) * y_head;
            if (inside_y(yo, which, 102)) store16<BF16>(reinterpret_cast<uint16_t*>(yo), c0, c1, f);
          }
        } else {
          const uint4 gp[2] = {ld_shared_v4(slot + 2 * kRopeThreads * 16), ld_shared_v4(slot + 3 * kRopeThreads * 16)};
          unpack16<BF16>(gp, f);
          rotate16<INTERLEAVED>(f, c, s, turn0, turn1);
          if (norm) {
            const uint4 xp[2] = {ld_shared_v4(slot), ld_shared_v4(slot + kRopeThreads * 16)};
            uint64_t x[8], ss[2] = {0, 0}, gx[2] = {0, 0};
            unpack16<BF16>(xp, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              ss[e & 1] = f2_fma(x[e], x[e], ss[e & 1]);
              gx[e & 1] = f2_fma(f2_mul(f[e], w[e]), x[e], gx[e & 1]);
            }
            const float r = rsqrtf(group_sum<Ln::GROUP>(on ? f2_total(ss) : 0.f) * (1.f / D) + p.eps);
            const float m = -group_sum<Ln::GROUP>(on ? f2_total(gx) : 0.f) * (1.f / D) * r * r;
            const uint64_t rr = f2_pack(r, r), mm = f2_pack(m, m);
            if (live) {  // (what an idle lane's ring holds adds nothing)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                dw[e] = f2_fma(f2_mul(f[e], rr), x[e], dw[e]);
                f[e] = f2_mul(rr, f2_fma(x[e], mm, f2_mul(f[e], w[e])));
              }
            }
          }
          if (live) {
            const uint64_t dxo = at[2 * Gm::TOKENS + t] + static_cast<uint64_t>(static_cast<uint32_t>(h)) * (which ? d_head[1] : d_head[0]);
            if (inside(dxo, p.dx[which], 103)) store16<BF16>(reinterpret_cast<uint16_t*>(dxo), c0, c1, f);
          }
        }
        h += step_h, t += step_t;
        if (t >= n) t -= n, ++h;
      }
      if constexpr (BWD) {
        if (!norm) continue;
        // the warp's rows, added to those of the tokens before, in a fixed order
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int m = Ln::GROUP; m < 32; m <<= 1) dw[e] = f2_add(dw[e], __shfl_xor_sync(0xffffffffu, dw[e], m));
        if (lane < Ln::GROUP && on) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint64_t* sum = reinterpret_cast<uint64_t*>(dw_sum + (which * WARPS + warp) * D + (e < 4 ? c0 : c1) * 8) + (e & 3);
            *sum = t0 == t_first ? dw[e] : f2_add(*sum, dw[e]);
          }
        }
      }
    }
    cp_async_wait<0>();
  }
  if constexpr (BWD) {
    if (!norm) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kRopeThreads) {  // the CTA's warps
      const int which = i / D, d = i - which * D;
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) x += dw_sum[(which * WARPS + k) * D + d];
      p.part[(static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * D + i] = x;
    }
  }
}

// dw = the CTAs' partial sums, in a fixed order: a block per 8 columns, 128 threads for each.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const RopeParams p, int n) {
  __shared__ float sum[128][9];
  grid_dependency_wait();
  const int c = threadIdx.x & 7, row = threadIdx.x >> 3, col = blockIdx.x * 8 + c;
  float x = 0.f;
#pragma unroll 4
  for (int i = row; i < n; i += 128) x += p.part[static_cast<size_t>(i) * 2 * p.D + col];
  sum[row][c] = x;
  __syncthreads();
  if (threadIdx.x < 256) {  // a warp per column
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    float y = (sum[lane][w] + sum[lane + 32][w]) + (sum[lane + 64][w] + sum[lane + 96][w]);
#pragma unroll
    for (int m = 16; m; m >>= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
    const int at = blockIdx.x * 8 + w, which = at / p.D;
    if (lane == 0) p.dw[which][at - which * p.D] = y;
  }
}

}  // namespace gbattn
