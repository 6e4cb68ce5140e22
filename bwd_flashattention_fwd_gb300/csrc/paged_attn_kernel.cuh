// Attention of a sequence's newest tokens (one, or a few in a chain) over its
// paged cache, the keys shared out over the whole GPU.
//
// Row r = g T + t of KV head h (packed: G query heads x T tokens) sees the keys
// j < n - T + 1 + t of the n in the cache:
//   s_j = scale log2e q_r . k_j,   O_r = sum_j 2^(s_j - m) v_j / l,
//   l = sum_j 2^(s_j - m),   lse_r = m + log2 l,
// with running m and l per warp, joined over the warps of a CTA and then over
// the CTAs that share a KV head.
//
// Bound by HBM: every key and value is read once, 4 G T products an element.
// A KV head has few rows, so the products are taken transposed, S^T = K Q^T and
// O^T = V^T P^T, with the keys (or the columns of V) on the 16 rows of a
// warp-level matrix instruction and the rows on its 8 columns: eight rows fill
// it.  (tcgen05's smallest tile has 64 rows of which 4 to 8 would be used, and
// it takes no 8-bit operand beside a 16-bit one, so quantised tiles would have
// to go through shared memory twice more.)  Its C fragment holds keys down a
// column of lanes and its B fragment along a row: movmatrix turns one into the
// other without shared memory.
//
// Every warp works on tiles of its own (16 or 32 keys) out of a ring of its
// own that cp.async fills, so the loop has no CTA barrier; row pitches are an odd
// number of 16-byte pieces, so ldmatrix meets no bank twice.  Pages only change
// the address of a row: a lane looks a key's page up one tile ahead.
//
// Quantised pages: codes are widened to fp16 in registers (exact; one
// conversion instruction for two).  ldmatrix moves pairs of bytes, which makes
// a lane's four codes neighbours along D: Q's fragments take the same order of
// D, and V's come out as two rows of V^T after one byte permutation.  A
// key's 2^e multiplies its score; a value's goes into the exponent, p'_j =
// 2^(s_j + e_j - m') with m' the running maximum of s_j + e_j, so p' <= 1 whatever
// the exponents, and l sums p'_j 2^-e_j in 32 bits: O = sum p' c / l.  Rows of Q
// are scaled by a power of two to use fp16's range.
//
// fp16 P: times 2^15, so that what counts as nothing is 2^-40 of the row's
// largest (2^-25 otherwise, and 10^5 such keys add up).
#pragma once

#include "paged_kernel.cuh"

namespace gbattn {

template <int D, bool Q8>
struct PagedGeom {
  static constexpr int NW = 4;                             // warps of a CTA
  static constexpr int THREADS = NW * 32;
  static constexpr int ROWB = D * (Q8 ? 1 : 2);            // bytes of a row
  static constexpr int CH = ROWB / 16;                     // its 16-byte pieces
  static constexpr int PITCH = (CH | 1) * 16;              // and its pitch in shared memory
  static constexpr int KT = ROWB <= 128 ? 32 : 16;         // keys of a warp's tile
  static constexpr int ST = 3;                             // tiles in flight
  static constexpr int KS = NW * KT;                       // keys of a CTA's step
  static constexpr int EXP = Q8 ? 2 * KT : 0;              // exponents of K, then of V
  static constexpr int TILE = 2 * KT * PITCH + (EXP + 15) / 16 * 16;
  static constexpr int RING = NW * ST * TILE;
  static constexpr int join_pitch = D + 4;  // floats of a row where the warps meet
  __host__ __device__ static constexpr int smem(int rows) {  // (and the B + 1 starts behind)
    const int join = NW * rows * join_pitch * 4;
    return (RING > join ? RING : join) + (D / 16) * (rows / 8) * 256;
  }
};

// The division of the work: the heads (b, h, row block) one after the other,
// each with its steps of keys and kPagedExtra more for what a head costs by
// itself; CTA c of n takes [total c / n, total (c + 1) / n), n = min(n_groups,
// total), so that every CTA of a head's range has some of it.
constexpr int kPagedExtra = 2;

struct PagedHead {
  int b, h, rb;
  int start;        // first unit
  int steps;        // of keys
};

// Prefix sums of the sequences' units (fewer than 2^31 in all: the host sees to
// it) into starts[0..B] (shared memory); every thread calls it.
__device__ __forceinline__ void paged_starts(const PagedAttnParams& p, int ks, int* starts) {
  __shared__ int warp_total[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  const int room = p.c.per_seq << p.c.shift;
  const int heads = p.c.Hkv * p.n_rb;
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int x = b < p.B ? ((clamp_len(p.cache_len[b], room) + ks - 1) / ks + kPagedExtra) * heads : 0;
    const int own = x;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, x, m);
      if (lane >= m) x += o;
    }
    if (lane == 31) warp_total[warp] = x;
    __syncthreads();
    int before = base;
    for (int w = 0; w < warp; ++w) before += warp_total[w];
    if (b < p.B) starts[b] = before + x - own;
    for (int w = 0; w < n_warps; ++w) base += warp_total[w];
    __syncthreads();
  }
  if (threadIdx.x == 0) starts[p.B] = base;
  __syncthreads();
}

// The head that unit u belongs to.
__device__ __forceinline__ PagedHead paged_head(const PagedAttnParams& p, const int* starts, int u) {
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (starts[mid] <= u) lo = mid; else hi = mid - 1;
  }
  const int heads = p.c.Hkv * p.n_rb;
  const int per = (starts[lo + 1] - starts[lo]) / heads, i = (u - starts[lo]) / per;
  return {lo, i / p.n_rb, i % p.n_rb, starts[lo] + i * per, per - kPagedExtra};
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t mat_trans(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// c += A (16 x 16) B (16 x 8), fp32 sums
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The e4m3 codes of a register, low and high pair, as fp16 pairs.
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}

// Row r's 16 values of Q that a lane's B fragment of k-step kk needs, as (b0, b1), in the operands' type.
template <int D, bool BF16, bool Q8>
__device__ __forceinline__ uint2 q_fragment(const uint16_t* qrow, int kk, int t, float by) {
  if constexpr (!Q8) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(qrow) + kk * 8;
    return make_uint2(w[t], w[t + 4]);
  } else {  // four neighbours along D, as ldmatrix hands out codes
    const uint2 w = *reinterpret_cast<const uint2*>(qrow + kk * 16 + 4 * t);
    const float2 a = Elem<BF16>::unpack(w.x), b = Elem<BF16>::unpack(w.y);
    return make_uint2(Elem<false>::pack(a.x * by, a.y * by), Elem<false>::pack(b.x * by, b.y * by));
  }
}

template <int D, bool BF16, bool Q8, int NT>
__global__ void __launch_bounds__(PagedGeom<D, Q8>::THREADS, D == 256 && !Q8 ? 1 : 2)
    attn_paged_kernel(const PagedAttnParams p) {
  using Gm = PagedGeom<D, Q8>;
  constexpr int NW = Gm::NW, KT = Gm::KT, ST = Gm::ST, MB = KT / 16, ROWS = 8 * NT, KK = D / 16;
  constexpr bool MMA_BF16 = BF16 && !Q8;          // type of the products' operands
  constexpr float kPShift = MMA_BF16 ? 0.f : 15.f;  // P is kept times 2^kPShift
  constexpr bool Q_REGS = KK * NT * 2 <= 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float q_exp[ROWS];       // log2 of what row r of Q was multiplied by
  __shared__ uint32_t key_mask[NW][ST];
  __shared__ float ml[NW][ROWS][2];
  uint2* qf = reinterpret_cast<uint2*>(smem + (Gm::smem(ROWS) - KK * NT * 256));
  int* starts = reinterpret_cast<int*>(smem + Gm::smem(ROWS));  // [B + 1]
  float* join = reinterpret_cast<float*>(smem);
  grid_dependency_wait();  // the kernels before this one are complete
  if (threadIdx.x == 0) grid_launch_dependents();
  paged_starts(p, Gm::KS, starts);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * ST * Gm::TILE;
  const int room = p.c.per_seq << p.c.shift;
  const long long n_rows = (static_cast<long long>(p.c.n_pages) * p.c.Hkv) << p.c.shift;
  const long long total = starts[p.B], groups = total < p.n_groups ? total : p.n_groups;
  if (blockIdx.x >= groups) return;
  int u = static_cast<int>(total * blockIdx.x / groups);
  const int u_end = static_cast<int>(total * (blockIdx.x + 1) / groups);
  while (u < u_end) {
    const PagedHead hd = paged_head(p, starts, u);
    const int s0 = u - hd.start, left = hd.start + hd.steps + kPagedExtra - u;
    const int s1 = min(hd.steps, s0 + min(left, u_end - u));
    u += left;  // the next head, if any
    if (s0 >= s1 && !(hd.steps == 0 && s0 == 0)) continue;  // only the head's extra units
    const int n = clamp_len(p.cache_len[hd.b], room);
    const int row0 = hd.rb * ROWS;  // first packed row
    __syncthreads();                // the join buffer of the head before is read

    // ---- the warp's ring of tiles ----
    int page = -1;  // of this lane's key in the tile that is issued next
    auto look_up = [&](int s) {
      const int key = (s * NW + warp) * KT + (lane & (KT - 1));
      page = s < s1 && key < n ? __ldg(p.c.table + static_cast<size_t>(hd.b) * p.c.per_seq + (key >> p.c.shift)) : -1;
      if (page >= p.c.n_pages) page = -1;
    };
    auto issue = [&](int s) {
      if (s < s1) {
        const int slot = (s - s0) % ST, key0 = (s * NW + warp) * KT;
        const uint32_t dst = ring + slot * Gm::TILE;
        const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) key_mask[warp][slot] = there;
#pragma unroll
        for (int i = 0; i < (KT * Gm::CH + 31) / 32; ++i) {
          const int x = i * 32 + lane, row = x / Gm::CH, c = x - row * Gm::CH;
          const int pg = __shfl_sync(0xffffffffu, page, row & (KT - 1));
          const int key = key0 + row;
          const long long r = ((static_cast<long long>(pg) * p.c.Hkv + hd.h) << p.c.shift) + (key & ((1 << p.c.shift) - 1));
          const bool in = pg >= 0 && dbg_in_range(r, 1, n_rows, p.status, 120);
          const size_t off = in ? static_cast<size_t>(r) * Gm::ROWB + c * 16 : 0;
          if (KT * Gm::CH % 32 == 0 || x < KT * Gm::CH) {
            cp_async16(dst + row * Gm::PITCH + c * 16, static_cast<const uint8_t*>(p.c.k) + off, in);
            cp_async16(dst + (KT + row) * Gm::PITCH + c * 16, static_cast<const uint8_t*>(p.c.v) + off, in);
          }
        }
        if constexpr (Q8) {  // four exponents at a time (a page has at least 8 rows)
          const int i = lane & (KT / 4 - 1), key = key0 + 4 * i;
          const int pg = __shfl_sync(0xffffffffu, page, 4 * i);
          const long long r = ((static_cast<long long>(pg) * p.c.Hkv + hd.h) << p.c.shift) + (key & ((1 << p.c.shift) - 1));
          const bool in = pg >= 0 && dbg_in_range(r, 4, n_rows, p.status, 121);
          const bool is_v = lane >= KT / 4;
          if (lane < KT / 2)
            cp_async4(dst + 2 * KT * Gm::PITCH + (is_v ? KT : 0) + 4 * i, (is_v ? p.c.v_exp : p.c.k_exp) + (in ? r : 0), in);
        }
        look_up(s + 1);
      }
      cp_async_commit();
    };
    look_up(s0);
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) issue(s0 + i);

    // ---- Q as B fragments, the same for every warp ----
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + (static_cast<size_t>(hd.b) * p.c.Hkv + hd.h) * p.R * D;
    if constexpr (Q8) {
      for (int r = warp; r < ROWS; r += NW) {
        float m = 0.f;
        if (row0 + r < p.R)
          for (int d = lane; d < D / 2; d += 32) {
            const float2 v = Elem<BF16>::unpack(reinterpret_cast<const uint32_t*>(q + static_cast<size_t>(row0 + r) * D)[d]);
            m = fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
#pragma unroll
        for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        // to a largest value in 2^14 .. 2^15 (a row of zeros or with an infinity as it is)
        const int e = m > 0.f && m < INFINITY ? min(max(141 - static_cast<int>(__float_as_uint(m) >> 23), -110), 110) : 0;
        if (lane == 0) q_exp[r] = static_cast<float>(e);
      }
      __syncthreads();
    }
    for (int x = threadIdx.x; x < KK * NT * 32; x += Gm::THREADS) {
      const int kk = x / (NT * 32), r = (x / 32 % NT) * 8 + (x % 32) / 4;
      uint2 w = make_uint2(0u, 0u);
      if (row0 + r < p.R)
        w = q_fragment<D, BF16, Q8>(q + static_cast<size_t>(row0 + r) * D, kk, x & 3, Q8 ? exp2_int(static_cast<int>(q_exp[r])) : 1.f);
      qf[x] = w;
    }
    __syncthreads();
    uint2 qr[Q_REGS ? KK * NT : 1];
    if constexpr (Q_REGS) {
#pragma unroll
      for (int i = 0; i < KK * NT; ++i) qr[i] = qf[i * 32 + lane];
    }
    float mul[NT][2];  // of the scores of rows 2 t4, 2 t4 + 1
    int lim[NT][2];    // and how many keys they see
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = i * 8 + 2 * t4 + k;
        mul[i][k] = p.scale_log2 * (Q8 ? exp2_int(-static_cast<int>(q_exp[r])) : 1.f);
        lim[i][k] = n - p.T + 1 + (row0 + r) % p.T;
      }

    // ---- the keys ----
    float acc[KK][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      m[i][0] = m[i][1] = -INFINITY, l[i][0] = l[i][1] = 0.f;
#pragma unroll
      for (int d = 0; d < KK; ++d) acc[d][i][0] = acc[d][i][1] = acc[d][i][2] = acc[d][i][3] = 0.f;
    }
    for (int s = s0; s < s1; ++s) {
      cp_async_wait<ST - 2>();
      __syncwarp();
      issue(s + ST - 1);
      const int slot = (s - s0) % ST, key0 = (s * NW + warp) * KT;
      const uint32_t tile = ring + slot * Gm::TILE;
      const uint32_t there = key_mask[warp][slot];
      if (there == 0) continue;  // past the end, or all holes
      // S^T = K Q^T
      float sc[MB][NT][4];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
        for (int i = 0; i < NT; ++i) sc[mb][i][0] = sc[mb][i][1] = sc[mb][i][2] = sc[mb][i][3] = 0.f;
        const uint32_t at = tile + (mb * 16 + (lane & 15)) * Gm::PITCH + (lane >> 4) * 16;
        if constexpr (!Q8) {
#pragma unroll
          for (int kk = 0; kk < KK; ++kk) {
            uint32_t a[4];
            ldsm4(a, at + kk * 32);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              const uint2 b = Q_REGS ? qr[kk * NT + i] : qf[(kk * NT + i) * 32 + lane];
              mma16816<MMA_BF16>(sc[mb][i], a, b.x, b.y);
            }
          }
        } else {
#pragma unroll
          for (int k2 = 0; k2 < KK / 2; ++k2) {
            uint32_t w[4];  // keys 0-7 and 8-15 of 16 codes, then of the next 16
            ldsm4(w, at + k2 * 32);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t a[4];
              widen(w[2 * half], a[0], a[2]);
              widen(w[2 * half + 1], a[1], a[3]);
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                const int kk = 2 * k2 + half;
                const uint2 b = Q_REGS ? qr[kk * NT + i] : qf[(kk * NT + i) * 32 + lane];
                mma16816<MMA_BF16>(sc[mb][i], a, b.x, b.y);
              }
            }
          }
        }
      }
      // scores, masked, and their running maxima
      float ev[MB][2];  // exponents of this lane's keys' values
      const bool edge = there != 0xffffffffu || key0 + KT > n - p.T + 1;
      float top[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i) top[i][0] = m[i][0], top[i][1] = m[i][1];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // key mb * 16 + g + 8 k
          const int at = mb * 16 + g + 8 * k;
          float fk = 1.f;
          ev[mb][k] = 0.f;
          if constexpr (Q8) {
            const int8_t* ex = reinterpret_cast<const int8_t*>(smem) + (tile - smem_u32(smem)) + 2 * KT * Gm::PITCH;
            fk = exp2_int(ex[at]);
            ev[mb][k] = static_cast<float>(ex[KT + at]);
          }
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = sc[mb][i][2 * k + e] * mul[i][e];
              if constexpr (Q8) x = fmaf(x, fk, ev[mb][k]);
              if (edge && (!(there >> at & 1u) || key0 + at >= lim[i][e])) x = -INFINITY;
              sc[mb][i][2 * k + e] = x;
              top[i][e] = fmaxf(top[i][e], x);
            }
        }
      bool same = true;
      float fix[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) top[i][e] = fmaxf(top[i][e], __shfl_xor_sync(0xffffffffu, top[i][e], x));
          const float ref = top[i][e] == -INFINITY ? 0.f : top[i][e];
          fix[i][e] = ex2_approx(m[i][e] - ref);
          same = same && top[i][e] == m[i][e];
          m[i][e] = top[i][e];
          top[i][e] = ref - kPShift;
        }
      if (!__all_sync(0xffffffffu, same)) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          l[i][0] *= fix[i][0], l[i][1] *= fix[i][1];
#pragma unroll
          for (int d = 0; d < KK; ++d) {
            acc[d][i][0] *= fix[i][0], acc[d][i][1] *= fix[i][1];
            acc[d][i][2] *= fix[i][0], acc[d][i][3] *= fix[i][1];
          }
        }
      }
      // P^T, and O^T += V^T P^T
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        uint32_t b[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float p0 = ex2_approx(sc[mb][i][2 * k] - top[i][0]), p1 = ex2_approx(sc[mb][i][2 * k + 1] - top[i][1]);
            const float w = Q8 ? exp2_int(-static_cast<int>(ev[mb][k])) : 1.f;
            l[i][0] = fmaf(p0, w, l[i][0]), l[i][1] = fmaf(p1, w, l[i][1]);
            b[i][k] = mat_trans(Elem<MMA_BF16>::pack(p0, p1));
          }
        const uint32_t vt = tile + (KT + mb * 16) * Gm::PITCH;
        if constexpr (!Q8) {
          const uint32_t at = vt + ((lane >> 4) * 8 + (lane & 7)) * Gm::PITCH + (lane >> 3 & 1) * 16;
#pragma unroll
          for (int d = 0; d < KK; ++d) {
            uint32_t a[4];
            ldsm4_t(a, at + d * 32);
#pragma unroll
            for (int i = 0; i < NT; ++i) mma16816<MMA_BF16>(acc[d][i], a, b[i][0], b[i][1]);
          }
        } else {
          const uint32_t at = vt + (lane & 15) * Gm::PITCH + (lane >> 4) * 16;
#pragma unroll
          for (int d2 = 0; d2 < KK / 2; ++d2) {
            uint32_t w[4];
            ldsm4_t(w, at + d2 * 32);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t a[4];  // rows 2 g and 2 g + 1 of these 16 columns of V
              widen(__byte_perm(w[2 * half], 0, 0x3120), a[0], a[1]);
              widen(__byte_perm(w[2 * half + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
              for (int i = 0; i < NT; ++i) mma16816<MMA_BF16>(acc[2 * d2 + half][i], a, b[i][0], b[i][1]);
            }
          }
        }
      }
    }
    cp_async_wait<0>();
    __syncthreads();  // every warp is done with its ring: the warps' results go there

    // ---- the warps' results ----
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], x);
        const int r = i * 8 + 2 * t4 + e;
        if (g == 0) ml[warp][r][0] = m[i][e], ml[warp][r][1] = l[i][e];
        float* dst = join + (warp * ROWS + r) * Gm::join_pitch;
#pragma unroll
        for (int d = 0; d < KK; ++d) {
          if constexpr (Q8) {
            *reinterpret_cast<float2*>(dst + d * 16 + 2 * g) = make_float2(acc[d][i][e], acc[d][i][2 + e]);
          } else {
            dst[d * 16 + g] = acc[d][i][e];
            dst[d * 16 + 8 + g] = acc[d][i][2 + e];
          }
        }
      }
    __syncthreads();
    const bool whole = s0 == 0 && s1 == hd.steps;
    const int slot = s0 == 0 ? 1 : 0;
    const size_t out0 = (static_cast<size_t>(hd.b) * p.c.Hkv + hd.h) * p.R + row0;
    for (int x = threadIdx.x; x < ROWS * (D / 4); x += Gm::THREADS) {
      const int r = x / (D / 4), c = x - r * (D / 4);
      if (row0 + r >= p.R) continue;
      float mx = ml[0][r][0];
#pragma unroll
      for (int w = 1; w < NW; ++w) mx = fmaxf(mx, ml[w][r][0]);
      const float ref = mx == -INFINITY ? 0.f : mx;
      float lsum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = ex2_approx(ml[w][r][0] - ref);
        const float4 a = *reinterpret_cast<const float4*>(join + (w * ROWS + r) * Gm::join_pitch + 4 * c);
        lsum = fmaf(ml[w][r][1], f, lsum);
        o.x = fmaf(a.x, f, o.x), o.y = fmaf(a.y, f, o.y), o.z = fmaf(a.z, f, o.z), o.w = fmaf(a.w, f, o.w);
      }
      if (whole) {
        const float by = mx == -INFINITY ? 0.f : 1.f / lsum;
        const size_t at = out0 + r;
        if (!dbg_in_range(at, 1, static_cast<size_t>(p.B) * p.Hq * p.T, p.status, 122)) continue;
        reinterpret_cast<uint2*>(p.o)[at * (D / 4) + c] =
            make_uint2(Elem<BF16>::pack(o.x * by, o.y * by), Elem<BF16>::pack(o.z * by, o.w * by));
        if (c == 0) p.lse[at] = mx == -INFINITY ? INFINITY : mx - kPShift + log2f(lsum);
      } else {
        const size_t at = (static_cast<size_t>(blockIdx.x) * 2 + slot) * ROWS + r;
        if (!dbg_in_range(at, 1, static_cast<size_t>(p.n_groups) * 2 * ROWS, p.status, 123)) continue;
        reinterpret_cast<float4*>(p.part)[at * (D / 4) + c] = o;
        if (c == 0) reinterpret_cast<float2*>(p.part_ml)[at] = make_float2(mx, lsum);
      }
    }
  }
}

// Joins the partial results of a head that several CTAs worked on: a block per
// packed row, 32 lanes' worth of column quads times slices of the CTAs.
constexpr int kPagedJoinThreads = 256;

template <int D, bool BF16, bool Q8, int NT>
__global__ void __launch_bounds__(kPagedJoinThreads) attn_paged_join_kernel(const PagedAttnParams p) {
  using Gm = PagedGeom<D, Q8>;
  constexpr int ROWS = 8 * NT, QUADS = D / 4, SLICES = kPagedJoinThreads / QUADS;
  constexpr float kPShift = BF16 && !Q8 ? 0.f : 15.f;
  __shared__ int starts[kPagedMaxB + 1];
  __shared__ float weight[kPagedMaxCtas];
  __shared__ float4 sum[SLICES][QUADS];
  __shared__ float red[2][kPagedJoinThreads / 32];
  paged_starts(p, Gm::KS, starts);  // (lengths: nothing that the kernel before writes)
  grid_dependency_wait();
  const long long total = starts[p.B], groups = total < p.n_groups ? total : p.n_groups;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long tasks = static_cast<long long>(p.B) * p.c.Hkv * p.R;
  for (long long task = blockIdx.x; task < tasks; task += gridDim.x) {
    const long long bh = task / p.R;
    const int pr = static_cast<int>(task - bh * p.R), rb = pr / ROWS, r = pr - rb * ROWS;
    const int b = static_cast<int>(bh / p.c.Hkv), h = static_cast<int>(bh - static_cast<long long>(b) * p.c.Hkv);
    const int per = (starts[b + 1] - starts[b]) / (p.c.Hkv * p.n_rb);
    const long long s = starts[b] + (h * p.n_rb + rb) * per;
    const int steps = per - kPagedExtra;
    if (steps == 0) continue;
    const int c0 = static_cast<int>(((s + 1) * groups - 1) / total);
    const int c1 = static_cast<int>(((s + steps) * groups - 1) / total);
    if (c0 == c1) continue;  // one CTA had it all
    const int n = c1 - c0 + 1;
    // weights of the partial results
    auto at = [&](int i) { return (static_cast<size_t>(c0 + i) * 2 + (i == 0 ? 1 : 0)) * ROWS + r; };
    float mx = -INFINITY;
    for (int i = threadIdx.x; i < n; i += kPagedJoinThreads) mx = fmaxf(mx, reinterpret_cast<const float2*>(p.part_ml)[at(i)].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    if (lane == 0) red[0][warp] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPagedJoinThreads / 32; ++w) mx = fmaxf(mx, red[0][w]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    float l = 0.f;
    for (int i = threadIdx.x; i < n; i += kPagedJoinThreads) {
      const float2 v = reinterpret_cast<const float2*>(p.part_ml)[at(i)];
      const float f = ex2_approx(v.x - ref);
      weight[i] = f;
      l = fmaf(v.y, f, l);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    if (lane == 0) red[1][warp] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kPagedJoinThreads / 32; ++w) l += red[1][w];
    const int q = threadIdx.x % QUADS, slice = threadIdx.x / QUADS;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (slice < SLICES) {
#pragma unroll 4
      for (int i = slice; i < n; i += SLICES) {
        const float4 a = reinterpret_cast<const float4*>(p.part)[at(i) * QUADS + q];
        const float f = weight[i];
        o.x = fmaf(a.x, f, o.x), o.y = fmaf(a.y, f, o.y), o.z = fmaf(a.z, f, o.z), o.w = fmaf(a.w, f, o.w);
      }
      sum[slice][q] = o;
    }
    __syncthreads();
    if (slice == 0) {
#pragma unroll
      for (int i = 1; i < SLICES; ++i) {
        const float4 a = sum[i][q];
        o.x += a.x, o.y += a.y, o.z += a.z, o.w += a.w;
      }
      const float by = mx == -INFINITY ? 0.f : 1.f / l;
      if (dbg_in_range(task, 1, static_cast<size_t>(tasks), p.status, 124)) {
        reinterpret_cast<uint2*>(p.o)[static_cast<size_t>(task) * QUADS + q] =
            make_uint2(Elem<BF16>::pack(o.x * by, o.y * by), Elem<BF16>::pack(o.z * by, o.w * by));
        if (q == 0) p.lse[task] = mx == -INFINITY ? INFINITY : mx - kPShift + log2f(l);
      }
    }
    __syncthreads();  // the shared arrays are used again
  }
}

}  // namespace gbattn
