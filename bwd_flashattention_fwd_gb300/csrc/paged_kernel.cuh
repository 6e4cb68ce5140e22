// The paged cache: new rows into the pages (in 16 bits or quantised to e4m3)
// and pages back into contiguous rows.  Both are bound by memory traffic and,
// for a decode step, by latency.
//
// Quantised rows.  A row of D values (one token, one KV head, K or V) has one
// exponent e, the least with max |x| <= 448 * 2^e, and codes c = e4m3(x 2^-e),
// so x 2^-e is exact and each value is rounded once.  A power of two costs
// nothing against max / 448 as the scale, since the codes are floating-point
// (their relative error is the same wherever the row's largest value falls
// between 224 and 448), and makes reading back exact.
#pragma once

#include <cuda_fp8.h>

#include "row_lanes.cuh"
#include "step.h"

namespace gbattn {

// Row number (of D values) of token `at` of sequence b and head h in the pool, or -1 where its page is none.
__device__ __forceinline__ long long paged_row(const PagedCache& c, int b, int h, int at, [[maybe_unused]] int B, [[maybe_unused]] int* status) {
  if (!dbg_in_range(static_cast<size_t>(b) * c.per_seq + (at >> c.shift), 1, static_cast<size_t>(B) * c.per_seq, status, 113)) return -1;
  const int page = c.table[static_cast<size_t>(b) * c.per_seq + (at >> c.shift)];
  if (page < 0 || page >= c.n_pages) return -1;
  return ((static_cast<long long>(page) * c.Hkv + h) << c.shift) + (at & ((1 << c.shift) - 1));
}

// Exponent of a row whose largest finite magnitude is m.
__device__ __forceinline__ int row_exponent(float m) {
  // 448 = 1.75 * 2^8; m = f * 2^x with 1 <= f < 2
  const uint32_t bits = __float_as_uint(m);
  const int x = static_cast<int>(bits >> 23) - 127;
  const int e = x - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return bits < 0x00800000u ? kExpMin : min(max(e, kExpMin), kExpMax);  // (below 2^-126: far under the least exponent)
}

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// Two values as e4m3 codes, round to nearest even; CHECK: what is not finite becomes NaN.
template <bool CHECK>
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  uint32_t r = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  if constexpr (CHECK) {
    if (!(fabsf(a) < INFINITY)) r |= 0x007fu;
    if (!(fabsf(b) < INFINITY)) r |= 0x7f00u;
  }
  return r;
}

// Sixteen values times `by` as codes.
template <bool BF16, bool CHECK>
__device__ __forceinline__ uint4 e4m3_16(const uint4 (&x)[2], float by) {
  float f[16];
  uint32_t w[4];
  unpack8<BF16>(x[0], f), unpack8<BF16>(x[1], f + 8);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = e4m3_pair<CHECK>(f[4 * i] * by, f[4 * i + 1] * by) | e4m3_pair<CHECK>(f[4 * i + 2] * by, f[4 * i + 3] * by) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float2 e4m3_unpack(uint32_t pair) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(pair), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

constexpr int kPagedThreads = 256;

// A lane's 16 values of a row, 32 bytes: in one access where the arrays start on 32 bytes (WIDE), else in two.  (Two
// leave half a sector each: quantised prefixes read back in 27.9 us by halves, 22.3 by wholes.)
template <bool WIDE>
__device__ __forceinline__ void load32(const void* p, uint4 (&x)[2]) {
  if constexpr (WIDE) {
    ld_global_v8(p, x[0], x[1]);
  } else {
    x[0] = static_cast<const uint4*>(p)[0], x[1] = static_cast<const uint4*>(p)[1];
  }
}
template <bool WIDE>
__device__ __forceinline__ void store32(void* p, const uint4& a, const uint4& b) {
  if constexpr (WIDE) {
    st_global_v8(p, a, b);
  } else {
    static_cast<uint4*>(p)[0] = a, static_cast<uint4*>(p)[1] = b;
  }
}

// A token's row of K and its row of V belong to D / 16 lanes, 16 consecutive
// values each; both are loaded before the page is looked up.
template <int D, bool BF16, bool Q8, bool WIDE>
__global__ void __launch_bounds__(kPagedThreads) attn_paged_write_kernel(const PagedWriteParams p) {
  using Gm = RowLanes<D>;
  grid_dependency_wait();  // the kernels before this one are complete
  if (threadIdx.x == 0) grid_launch_dependents();
  const int lane = threadIdx.x & 31, j = lane % Gm::GROUP;
  const uint32_t rows = static_cast<uint32_t>(p.B) * p.c.Hkv * p.T;  // below 2^31
  const int room = p.c.per_seq << p.c.shift;
  [[maybe_unused]] const long long n_rows = (static_cast<long long>(p.c.n_pages) * p.c.Hkv) << p.c.shift;
  const uint32_t step = gridDim.x * (kPagedThreads / Gm::GROUP);
  // whole warps go round together: the shuffles below take every lane
  for (uint32_t base = (blockIdx.x * kPagedThreads + (threadIdx.x & ~31u)) / Gm::GROUP; base < rows; base += step) {
    const uint32_t r = base + lane / Gm::GROUP;  // (b, h, t)
    const bool in = r < rows;
    uint4 x[2][2] = {};
    if (in && j < Gm::LANES) {
      load32<WIDE>(static_cast<const uint4*>(p.k_new) + static_cast<size_t>(r) * (D / 8) + 2 * j, x[0]);
      load32<WIDE>(static_cast<const uint4*>(p.v_new) + static_cast<size_t>(r) * (D / 8) + 2 * j, x[1]);
    }
    long long dst = -1;
    if (in) {
      const uint32_t bh = p.T == 1 ? r : r / p.T;
      const int t = r - bh * p.T, b = bh / p.c.Hkv, h = bh - b * p.c.Hkv;
      const int len = clamp_len(p.cache_len[b], room);
      const int n = min(p.new_len ? clamp_len(p.new_len[b], p.T) : p.T, room - len);
      if (t < n) dst = paged_row(p.c, b, h, len + t, p.B, p.status);
      if (t == 0 && h == 0 && j == 0) p.cache_len_out[b] = len + n;
    }
    const bool live = dst >= 0 && j < Gm::LANES && dbg_in_range(dst, 1, n_rows, p.status, 110);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      if constexpr (!Q8) {
        if (live) store32<WIDE>(static_cast<uint4*>(v ? p.c.v : p.c.k) + dst * (D / 8) + 2 * j, x[v][0], x[v][1]);
      } else {
        // the row's largest magnitude, from the 16-bit patterns (which order as the values do)
        const uint32_t u[8] = {x[v][0].x, x[v][0].y, x[v][0].z, x[v][0].w, x[v][1].x, x[v][1].y, x[v][1].z, x[v][1].w};
        constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, u[i] & 0x7fff7fffu);
        m = max(m & 0xffffu, m >> 16);
#pragma unroll
        for (int k = Gm::GROUP / 2; k; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
        const bool fine = m < kInf;
        if (__any_sync(0xffffffffu, !fine)) {  // the largest finite one, for rows with others
          uint32_t f = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t y = u[i] >> (16 * k) & 0x7fffu;
              if (y < kInf) f = max(f, y);
            }
#pragma unroll
          for (int k = Gm::GROUP / 2; k; k >>= 1) f = max(f, __shfl_xor_sync(0xffffffffu, f, k));
          m = f;
        }
        const int e = row_exponent(Elem<BF16>::unpack(m).x);
        const uint4 w = fine ? e4m3_16<BF16, false>(x[v], exp2_int(-e)) : e4m3_16<BF16, true>(x[v], exp2_int(-e));
        if (live) {
          (static_cast<uint4*>(v ? p.c.v : p.c.k) + dst * (D / 16))[j] = w;
          if (j == 0) (v ? p.c.v_exp : p.c.k_exp)[dst] = static_cast<int8_t>(e);
        }
      }
    }
  }
}

// The codes' values in 16 bits; EDGE: one that rounds past the type's largest value becomes that.
template <bool BF16, bool EDGE>
__device__ __forceinline__ uint32_t dequant_pair(uint32_t pair, float by) {
  float2 v = e4m3_unpack(pair);
  v.x *= by, v.y *= by;
  if constexpr (EDGE) {
    constexpr float most = BF16 ? 3.3895313892515355e38f : 65504.f;
    if (fabsf(v.x) > most) v.x = copysignf(most, v.x);
    if (fabsf(v.y) > most) v.y = copysignf(most, v.y);
  }
  return Elem<BF16>::pack(v.x, v.y);
}

template <bool BF16, bool EDGE, bool WIDE>
__device__ __forceinline__ void dequant16(const uint4& w, float by, uint4* d) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    o[2 * k] = dequant_pair<BF16, EDGE>(u[k] & 0xffffu, by);
    o[2 * k + 1] = dequant_pair<BF16, EDGE>(u[k] >> 16, by);
  }
  store32<WIDE>(d, make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]));
}

// A block: read_rows tokens of one sequence and head.  A thread holds the same
// 16 values of several tokens' K and V, whose pages it looks up first, so that
// all its loads are in flight together.
constexpr int kReadTokens = 2;  // of a thread
constexpr int read_rows(int D) { return kReadTokens * (kPagedThreads / (D / 16)); }

template <int D, bool BF16, bool Q8, bool WIDE>
__global__ void __launch_bounds__(kPagedThreads) attn_paged_read_kernel(const PagedReadParams p) {
  constexpr int LANES = D / 16, GROUPS = kPagedThreads / LANES, N = kReadTokens, ROWS = N * GROUPS;
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int b = blockIdx.y / p.c.Hkv, h = blockIdx.y - b * p.c.Hkv;
  const int most = min(p.Lk, p.c.per_seq << p.c.shift), n = clamp_len(p.cache_len[b], most);
  [[maybe_unused]] const long long n_rows = (static_cast<long long>(p.c.n_pages) * p.c.Hkv) << p.c.shift;
  [[maybe_unused]] const size_t n_out = static_cast<size_t>(p.B * p.c.Hkv - 1) * p.pitch + p.Lk;
  const int group = threadIdx.x / LANES, c = threadIdx.x - group * LANES;
  const size_t out0 = static_cast<size_t>(blockIdx.y) * p.pitch;
  for (long long j0 = static_cast<long long>(blockIdx.x) * ROWS; j0 < most; j0 += static_cast<long long>(gridDim.x) * ROWS) {
    if (j0 != static_cast<long long>(blockIdx.x) * ROWS && j0 >= n) break;
    long long from[N];
    int row[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = i * GROUPS + group;
      row[i] = static_cast<int>(j0) + x;
      from[i] = group < GROUPS && row[i] < most ? paged_row(p.c, b, h, row[i], p.B, p.status) : -1;  // (not waiting for n)
      if (row[i] >= n) from[i] = -1;
      if (from[i] >= 0 && !(dbg_in_range(from[i], 1, n_rows, p.status, 111) && dbg_in_range(out0 + row[i], 1, n_out, p.status, 112))) from[i] = -1;
    }
    if constexpr (Q8) {
      uint4 w[2][N];
      int e[2][N];
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (from[i] >= 0) {
          w[0][i] = (static_cast<const uint4*>(p.c.k) + from[i] * LANES)[c], e[0][i] = p.c.k_exp[from[i]];
          w[1][i] = (static_cast<const uint4*>(p.c.v) + from[i] * LANES)[c], e[1][i] = p.c.v_exp[from[i]];
        }
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          if (from[i] < 0) continue;
          uint4* d = static_cast<uint4*>(v ? p.v : p.k) + (out0 + row[i]) * (D / 8) + 2 * c;
          // 448 * 2^e is within the type up to these
          if (e[v][i] <= (BF16 ? 118 : 7))
            dequant16<BF16, false, WIDE>(w[v][i], exp2_int(e[v][i]), d);
          else
            dequant16<BF16, true, WIDE>(w[v][i], exp2_int(e[v][i]), d);
        }
    } else {
      uint4 w[2][N][2];
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (from[i] >= 0) {
          load32<WIDE>(static_cast<const uint4*>(p.c.k) + from[i] * (D / 8) + 2 * c, w[0][i]);
          load32<WIDE>(static_cast<const uint4*>(p.c.v) + from[i] * (D / 8) + 2 * c, w[1][i]);
        }
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          if (from[i] < 0) continue;
          store32<WIDE>(static_cast<uint4*>(v ? p.v : p.k) + (out0 + row[i]) * (D / 8) + 2 * c, w[v][i][0], w[v][i][1]);
        }
    }
  }
}

}  // namespace gbattn
