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
// Bound by HBM: every key and value is read once for each block of rows (32 at
// most, 16 at D = 256), 4 G T products an element.  (The blocks of a head follow one another in the order of
// the work: with two of them at D = 256 the second finds the keys in L2, 134.3 MB read for 134.2 of
// keys; with four of 32 rows at D = 128, 4 x 8192 keys, memory gives them 2.9 times.)
// A KV head has few rows, so the products are taken transposed, S^T = K Q^T and
// O^T = V^T P^T, with the keys (or the columns of V) on the 16 rows of a
// warp-level matrix instruction and the rows on its 8 columns: eight rows fill
// it.  (tcgen05 would take 64 or 128 keys on its rows the same way, widened codes by way of tensor
// memory.  With 8 rows that has little to win, the tensor pipe being 8 to 16% busy; for
// more rows over quantised pages it was not tried.)  Its C fragment holds keys down a
// column of lanes and its B fragment along a row: movmatrix turns one into the
// other without shared memory.
//
// Every warp works on tiles of its own (16 keys) out of a ring of its
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
// the exponents, and l sums the weights 2^(s_j - m') in 32 bits: O = sum p' c / l.
// The largest weight of l is between 2^-120 and 2^64 (e is -64 .. 120), and l is kept
// times 2^kPLift, so that a weight counts down to 2^-37 of it.  (p' comes from the weight and not
// the other way round, which would be one instruction less for two: p' of a row of zeros, e = -64, beside
// one of 2^100 is nothing where its weight is not.  32 rows over 4 sequences of 32768 quantised
// keys 85.6 us, 83.8 so; D = 64 59.0 and 56.4; 4 x 8192 keys, 4 rows 16.6 and 16.4.)  Rows of Q
// are scaled by a power of two to use fp16's range.
//
// fp16 P: times 2^15, so that what counts as nothing is 2^-40 of the row's
// largest (2^-25 otherwise, and 10^5 such keys add up; beside exponents above 117 2^-37).
//
// Past a few rows, or with codes to widen, the instructions of a tile bound it (46
// to 62% of the issue slots): scores and sums in packed pairs, masks only in tiles that need
// one, the rows' references moved only by scores well above them, offsets of copies in the
// instructions: 32 rows over 4 sequences of 65536 quantised keys 150 us (166 without), D = 64 102 (120).
#pragma once

#include <cfloat>
#include <utility>

#include "paged_kernel.cuh"

namespace gbattn {

// Warps: as many as hide the latency of a tile's chain (look-up, copy, products,
// exponentials), which registers limit: 8 rows over quantised pages take 128
// registers, 16 warps on an SM (8192 keys, 4 sequences: 16.4 us; 8 warps of 32-key tiles 3.5 more).
template <int D, bool Q8, int NT>
struct PagedGeom {
  static constexpr int NW = D == 256 && !Q8 ? 2 : Q8 && D * NT <= 128 ? 8 : 4;  // warps of a CTA
  static constexpr int PER_SM = Q8 && NT == 2 && NW == 4 && D <= 128 ? 3 : 2;              // CTAs on an SM, as far as registers allow
  static constexpr int THREADS = NW * 32;
  static constexpr int ROWS = 8 * NT;
  static constexpr int ROWB = D * (Q8 ? 1 : 2);            // bytes of a row
  static constexpr int CH = ROWB / 16;                     // its 16-byte pieces
  static constexpr int PITCH = (CH | 1) * 16;              // and its pitch in shared memory
  static constexpr int KT = 16;                            // keys of a warp's tile
  static constexpr int ST = 3;                             // tiles in flight
  static constexpr int KS = NW * KT;                       // keys of a CTA's step
  static constexpr int EXP = Q8 ? 2 * KT : 0;              // exponents of K, then of V
  static constexpr int TILE = 2 * KT * PITCH + EXP;        // K, V, exponents
  static constexpr int RING = NW * ST * TILE;
  static constexpr int JOIN_PITCH = D + 4;                 // floats of a row where the warps meet
  static constexpr int JOIN = NW * ROWS * JOIN_PITCH * 4;
  static constexpr int Q_AT = RING > JOIN ? RING : JOIN;   // Q's rows, then fragments
  static constexpr int SMEM = Q_AT + ROWS * D * 2;         // (and the B + 1 starts and B lengths behind)
};

// The division of the work: the heads (b, h, row block) one after the other,
// each with its steps of keys and kPagedExtra more for what a head costs by
// itself, cut into equal pieces, one for each CTA that runs at once.  (The SMs
// do not get equal shares of the memory's bandwidth: equal pieces of 131072 keys
// end between 61 and 89 us, by the number of SMs in their part of the chip.  Smaller
// pieces behind large ones, 80, 8, 7 and 5% of a CTA's share, ended at 96: a
// CTA's start costs more than they even out.)
constexpr int kPagedExtra = 2;

struct PagedPieces {
  int n, each, more;  // pieces; units of each, and how many (the first ones) have one more
  __device__ __forceinline__ PagedPieces(int total, int ctas) : n(total < ctas ? total : ctas), each(total / n), more(total - each * n) {}
  __device__ __forceinline__ int first(int c) const { return c * each + min(c, more); }  // unit of piece c
  __device__ __forceinline__ int of(int u) const {  // the piece that unit u belongs to
    const int longer = more * (each + 1);
    return u < longer ? u / (each + 1) : more + (u - longer) / each;
  }
};

struct PagedHead {
  int b, h, rb;
  int start;        // first unit
  int steps;        // of keys
};

// Prefix sums of the sequences' units (fewer than 2^31 in all: the host sees to
// it) into starts[0..B], and their lengths into lens (shared memory; may be null); every thread calls it.
__device__ __forceinline__ void paged_starts(const PagedAttnParams& p, int ks, int* starts, int* lens) {
  __shared__ int warp_total[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  const int room = p.c.per_seq << p.c.shift;
  const int heads = p.c.Hkv * p.n_rb;
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    const int len = b < p.B ? clamp_len(p.cache_len[b], room) : 0;
    if (lens && b < p.B) lens[b] = len;
    int x = b < p.B ? ((len + ks - 1) / ks + kPagedExtra) * heads : 0;
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

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
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

// 16 bytes each from src, src + SRC, ..., whose offsets go into the instructions.
template <int DST, int SRC>
__device__ __forceinline__ void cp_async16_at(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(DST), "n"(SRC) : "memory");
}
template <int DST, int SRC, int... I>
__device__ __forceinline__ void cp_async16_rows(uint32_t dst, const void* src, std::integer_sequence<int, I...>) {
  (..., cp_async16_at<I * DST, I * SRC>(dst, src));
}

constexpr int kPLift = 16;  // l is at most 2^(64 + 16 + kPLift) times the number of keys, 2^30

// What results of reference `from` are multiplied by beside ones of reference `to`, d = from - to: O by o, l by l0 and then by l1.
// Over quantised pages l 2^d may be of ordinary size where 2^d is below what 32 bits hold: by halves.
template <bool Q8>
struct PagedRescale {
  float o, l0, l1;
  __device__ __forceinline__ explicit PagedRescale(float d) {
    if constexpr (Q8) {
      l0 = l1 = ex2_approx(0.5f * d);
      o = l0 * l1;
    } else {
      l0 = 1.f, o = l1 = ex2_approx(d);
    }
  }
};

// What the warps of a CTA share besides the ring.
template <int NW, int ST, int ROWS>
struct PagedShared {
  float q_exp[ROWS];  // log2 of what row r of Q was multiplied by
  uint32_t key_mask[NW][ST];
  float ml[NW][ROWS][2];
};

// Steps s0 .. s1 - 1 of a head's keys, n in all, for one block of its rows: leaves the warps' results in
// smem (rows of JOIN_PITCH floats) and sh.ml.
template <int D, bool BF16, bool Q8, int NT>
__device__ __forceinline__ void paged_part(const PagedAttnParams& p, const PagedHead& hd, int s0, int s1, int n, uint8_t* smem,
                                           PagedShared<PagedGeom<D, Q8, NT>::NW, PagedGeom<D, Q8, NT>::ST, 8 * NT>& sh) {
  using Gm = PagedGeom<D, Q8, NT>;
  constexpr int NW = Gm::NW, KT = Gm::KT, ST = Gm::ST, MB = KT / 16, ROWS = 8 * NT, KK = D / 16;
  constexpr bool MMA_BF16 = BF16 && !Q8;          // type of the products' operands
  constexpr float kPShift = MMA_BF16 ? 0.f : 15.f;  // P is kept times 2^kPShift,
  constexpr float kPMost = kPShift + 0.9f;          // and no larger than 2^kPMost (fp16 ends at 2^16)
  constexpr bool Q_REGS = KK * NT * 2 <= 32;
  auto& q_exp = sh.q_exp;
  auto& key_mask = sh.key_mask;
  auto& ml = sh.ml;
  uint16_t* const q_rows = reinterpret_cast<uint16_t*>(smem + Gm::Q_AT);  // [ROWS][D], then
  uint2* const qf = reinterpret_cast<uint2*>(q_rows);                         // as fragments
  float* join = reinterpret_cast<float*>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * ST * Gm::TILE;
  [[maybe_unused]] const long long n_rows = (static_cast<long long>(p.c.n_pages) * p.c.Hkv) << p.c.shift;
  const int row0 = hd.rb * ROWS;  // first packed row

  // ---- Q, ahead of everything ----
  const uint8_t* q = static_cast<const uint8_t*>(p.q) + ((static_cast<size_t>(hd.b) * p.c.Hkv + hd.h) * p.R + row0) * (D * 2);
  for (int x = threadIdx.x; x < ROWS * (D / 8); x += Gm::THREADS) {
    const bool in = row0 + x / (D / 8) < p.R &&
                    dbg_in_range(static_cast<size_t>(q - static_cast<const uint8_t*>(p.q)) + x * 16, 16, static_cast<size_t>(p.B) * p.Hq * p.T * D * 2, p.status, 126);
    cp_async16(smem_u32(q_rows) + x * 16, in ? q + static_cast<size_t>(x) * 16 : static_cast<const uint8_t*>(p.q), in);
  }
  cp_async_commit();

  // ---- the warp's ring of tiles ----
  auto look_up = [&](int s) {  // page of this lane's key in the tile of step s
    const int key = (s * NW + warp) * KT + (lane & (KT - 1));
    if (s >= s1 || key >= n) return -1;
    if (!dbg_in_range(static_cast<size_t>(hd.b) * p.c.per_seq + (key >> p.c.shift), 1, static_cast<size_t>(p.B) * p.c.per_seq, p.status, 125)) return -1;
    const int pg = p.c.table[static_cast<size_t>(hd.b) * p.c.per_seq + (key >> p.c.shift)];
    return pg < p.c.n_pages ? pg : -1;
  };
  int page[ST];  // of the tiles that are issued next: the first ones' are looked up together, then one at a time
#pragma unroll
  for (int i = 0; i < ST; ++i) page[i] = look_up(s0 + i);
  // Where the tile's rows lie in the pool, by eights (a page has at least eight), and which of them are there.
  long long src[KT / 8];
  uint32_t there_next = 0;
  auto copy_rows = [&](uint32_t dst, const void* pool) {
    const uint8_t* base = static_cast<const uint8_t*>(pool);
    if constexpr (32 % Gm::CH == 0) {
      constexpr int RPI = 32 / Gm::CH;  // rows per instruction: whole ones, all in one eight
      const int row = lane / Gm::CH, c = lane % Gm::CH;
#pragma unroll
      for (int e = 0; e < KT / 8; ++e) {
        const uint32_t to = dst + (e * 8 + row) * Gm::PITCH + c * 16;
        const uint8_t* from = base + src[e] * Gm::ROWB + (row * Gm::ROWB + c * 16);
        if (there_next == 0xffffffffu) {
          cp_async16_rows<RPI * Gm::PITCH, RPI * Gm::ROWB>(to, from, std::make_integer_sequence<int, 8 / RPI>());
        } else {
#pragma unroll
          for (int j = 0; j < 8; j += RPI) cp_async16(to + j * Gm::PITCH, from + j * Gm::ROWB, there_next >> (e * 8 + j + row) & 1u);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < KT * Gm::CH / 32; ++i) {
        const int x = i * 32 + lane, row = x / Gm::CH, c = x - row * Gm::CH;
        long long at = src[0];
#pragma unroll
        for (int e = 1; e < KT / 8; ++e) at = row / 8 == e ? src[e] : at;
        cp_async16(dst + row * Gm::PITCH + c * 16, base + (at + (row & 7)) * Gm::ROWB + c * 16, there_next >> row & 1u);
      }
    }
  };
  auto issue_k = [&](int s, int slot, int pages) {
    if (s < s1) {
      const int key0 = (s * NW + warp) * KT;
      there_next = __ballot_sync(0xffffffffu, pages >= 0);
#pragma unroll
      for (int e = 0; e < KT / 8; ++e) {
        const int pg = __shfl_sync(0xffffffffu, pages, 8 * e);
        const long long r = ((static_cast<long long>(pg) * p.c.Hkv + hd.h) << p.c.shift) + ((key0 + 8 * e) & ((1 << p.c.shift) - 1));
        src[e] = r;
        if (pg < 0 || !dbg_in_range(r, 8, n_rows, p.status, 120)) {  // (a hole, or past the end)
          src[e] = 0;
          there_next &= ~(0xffu << (8 * e));
        }
      }
      if (lane == 0) key_mask[warp][slot] = there_next;
      const uint32_t dst = ring + slot * Gm::TILE;
      copy_rows(dst, p.c.k);
      if constexpr (Q8) {  // four exponents at a time
        const int i = lane & (KT / 4 - 1);
        const bool is_v = lane >= KT / 4;
        long long at = src[0];
#pragma unroll
        for (int e = 1; e < KT / 8; ++e) at = i / 2 == e ? src[e] : at;
        if (lane < KT / 2)
          cp_async4(dst + 2 * KT * Gm::PITCH + (is_v ? KT : 0) + 4 * i, (is_v ? p.c.v_exp : p.c.k_exp) + at + 4 * (i & 1),
                    there_next >> (4 * i) & 1u);
      }
    }
    cp_async_commit();
  };
  auto issue_v = [&](int s, int slot) {  // (behind issue_k of the same tile)
    if (s < s1) copy_rows(ring + slot * Gm::TILE + KT * Gm::PITCH, p.c.v);
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < ST; ++i) {
    issue_k(s0 + i, i, page[i]);
    issue_v(s0 + i, i);
  }
  int next_page = look_up(s0 + ST);

  // ---- Q as B fragments, the same for every warp ----
  cp_async_wait<2 * ST>();
  __syncthreads();
  if constexpr (Q8) {
    for (int r = warp; r < ROWS; r += NW) {
      float m = 0.f;
      for (int d = lane; d < D / 2; d += 32) {
        const float2 v = Elem<BF16>::unpack(reinterpret_cast<const uint32_t*>(q_rows + r * D)[d]);
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
  constexpr int FRAGMENTS = (KK * NT * 32 + Gm::THREADS - 1) / Gm::THREADS;  // of a thread
  {
    uint2 w[FRAGMENTS];
#pragma unroll
    for (int i = 0; i < FRAGMENTS; ++i) {
      const int x = i * Gm::THREADS + threadIdx.x, kk = x / (NT * 32), r = (x / 32 % NT) * 8 + (x % 32) / 4;
      if (x < KK * NT * 32) w[i] = q_fragment<D, BF16, Q8>(q_rows + r * D, kk, x & 3, Q8 ? exp2_int(static_cast<int>(q_exp[r])) : 1.f);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < FRAGMENTS; ++i)
      if (i * Gm::THREADS + threadIdx.x < KK * NT * 32) qf[i * Gm::THREADS + threadIdx.x] = w[i];
  }
  __syncthreads();
  uint2 qr[Q_REGS ? KK * NT : 1];
  if constexpr (Q_REGS) {
#pragma unroll
    for (int i = 0; i < KK * NT; ++i) qr[i] = qf[i * 32 + lane];
  }
  uint64_t mul[NT];  // of the scores of rows 2 t4, 2 t4 + 1
  int lim[NT][2];    // and how many keys they see
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int r = i * 8 + 2 * t4;
    mul[i] = Q8 ? f2_pack(p.scale_log2 * exp2_int(-static_cast<int>(q_exp[r])), p.scale_log2 * exp2_int(-static_cast<int>(q_exp[r + 1])))
                : f2_pack(p.scale_log2, p.scale_log2);
    lim[i][0] = n - p.T + 1 + (row0 + r) % p.T, lim[i][1] = n - p.T + 1 + (row0 + r + 1) % p.T;
  }

  // ---- the keys ----
  // (m: a row's reference, 2^kPShift below a score that was its largest; see below)
  float acc[KK][NT][4];
  uint64_t m[NT], l[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    m[i] = f2_pack(-FLT_MAX, -FLT_MAX), l[i] = 0;
#pragma unroll
    for (int d = 0; d < KK; ++d) acc[d][i][0] = acc[d][i][1] = acc[d][i][2] = acc[d][i][3] = 0.f;
  }
  for (int s = s0, slot = 0; s < s1; ++s, slot = slot + 1 == ST ? 0 : slot + 1) {
    cp_async_wait<2 * ST - 1>();  // K of this tile
    __syncwarp();
    const int key0 = (s * NW + warp) * KT;
    const uint32_t tile = ring + slot * Gm::TILE;
    const uint32_t there = key_mask[warp][slot];
    if (there == 0) {  // past the end, or all holes
      __syncwarp();
      issue_k(s + ST, slot, next_page);
      next_page = look_up(s + ST + 1);
      cp_async_wait<2 * ST - 1>();
      issue_v(s + ST, slot);
      continue;
    }
    // S^T = K Q^T
    // (two chains of products where the registers allow it: each waits for the one before)
    constexpr int CHAINS = MB * NT == 1 ? 2 : 1;
    float sc2[CHAINS][MB][NT][4];
    float(&sc)[MB][NT][4] = sc2[0];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < CHAINS; ++x) sc2[x][mb][i][0] = sc2[x][mb][i][1] = sc2[x][mb][i][2] = sc2[x][mb][i][3] = 0.f;
      const uint32_t at = tile + (mb * 16 + (lane & 15)) * Gm::PITCH + (lane >> 4) * 16;
      if constexpr (!Q8) {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          uint32_t a[4];
          ldsm4(a, at + kk * 32);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const uint2 b = Q_REGS ? qr[kk * NT + i] : qf[(kk * NT + i) * 32 + lane];
            mma16816<MMA_BF16>(sc2[kk % CHAINS][mb][i], a, b.x, b.y);
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
              mma16816<MMA_BF16>(sc2[kk % CHAINS][mb][i], a, b.x, b.y);
            }
          }
        }
      }
      if constexpr (CHAINS == 2) {
#pragma unroll
        for (int x = 0; x < 4; ++x) sc[0][0][x] += sc2[1][0][0][x];
      }
    }
    // scores, masked
    int ev[MB][2];  // exponents of this lane's keys' values
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // key mb * 16 + g + 8 k
        uint64_t fk = 0, fe = 0;
        if constexpr (Q8) {
          const int8_t* ex = reinterpret_cast<const int8_t*>(smem) + (tile - smem_u32(smem)) + 2 * KT * Gm::PITCH + mb * 16 + g + 8 * k;
          ev[mb][k] = ex[KT];
          const float f = exp2_int(ex[0]), e = static_cast<float>(ev[mb][k]);
          fk = f2_pack(f, f), fe = f2_pack(e, e);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          uint64_t x = f2_mul(f2_pack(sc[mb][i][2 * k], sc[mb][i][2 * k + 1]), mul[i]);
          if constexpr (Q8) x = f2_fma(x, fk, fe);
          f2_unpack(x, sc[mb][i][2 * k], sc[mb][i][2 * k + 1]);
        }
      }
    if (there != 0xffffffffu || key0 + KT > n - p.T + 1) {
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int at = mb * 16 + g + 8 * k;
          const bool in = there >> at & 1u;
          if (!in) ev[mb][k] = 0;  // (such a row may hold any exponent: 2^128 times its weight 0 would not be 0)
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!in || key0 + at >= lim[i][e]) sc[mb][i][2 * k + e] = -INFINITY;
        }
    }
    // The rows' references.  A score may be 0.9 above the one that set its row's before it moves, which
    // saves the lanes' common maximum and the sums' rescaling in nearly every tile.
    bool up = false;
    float top[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      top[i][0] = sc[0][i][0], top[i][1] = sc[0][i][1];
#pragma unroll
      for (int x = 2; x < 4 * MB; ++x) top[i][x & 1] = fmaxf(top[i][x & 1], sc[x / 4][i][x & 3]);
      float d0, d1;  // (the difference that P is the power of, not a rounded bound on the score: P may not pass 2^kPMost)
      f2_unpack(f2_sub(f2_pack(top[i][0], top[i][1]), m[i]), d0, d1);
      up = up || d0 > kPMost || d1 > kPMost;
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float old[2], fix[2], l0[2], l1[2];
        f2_unpack(m[i], old[0], old[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) top[i][e] = fmaxf(top[i][e], __shfl_xor_sync(0xffffffffu, top[i][e], x));
          // (no row's result depends on another's scores; upwards, so that large scores too give at most 2^kPShift)
          top[i][e] = top[i][e] - old[e] > kPMost ? __fadd_ru(top[i][e], -kPShift) : old[e];
          const PagedRescale<Q8> by(old[e] - top[i][e]);
          fix[e] = by.o, l0[e] = by.l0, l1[e] = by.l1;
        }
        m[i] = f2_pack(top[i][0], top[i][1]);
        if constexpr (Q8) l[i] = f2_mul(l[i], f2_pack(l0[0], l0[1]));
        l[i] = f2_mul(l[i], f2_pack(l1[0], l1[1]));
#pragma unroll
        for (int d = 0; d < KK; ++d) {
          acc[d][i][0] *= fix[0], acc[d][i][1] *= fix[1];
          acc[d][i][2] *= fix[0], acc[d][i][3] *= fix[1];
        }
      }
    }
    __syncwarp();  // every lane has read K and the exponents
    issue_k(s + ST, slot, next_page);
    next_page = look_up(s + ST + 1);
    cp_async_wait<2 * ST - 1>();  // V of this tile
    __syncwarp();
    // P^T, and O^T += V^T P^T
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      uint32_t b[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint64_t x = f2_sub(f2_pack(sc[mb][i][2 * k], sc[mb][i][2 * k + 1]), m[i]);
          if constexpr (Q8) {
            const float e = static_cast<float>(ev[mb][k] - kPLift);
            x = f2_sub(x, f2_pack(e, e));
          }
          float p0, p1;
          f2_unpack(x, p0, p1);
          p0 = ex2_approx(p0), p1 = ex2_approx(p1);
          l[i] = f2_add(l[i], f2_pack(p0, p1));
          if constexpr (Q8) {
            const float e = exp2_int(ev[mb][k] - kPLift);
            f2_unpack(f2_mul(f2_pack(p0, p1), f2_pack(e, e)), p0, p1);
          }
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
    __syncwarp();  // every lane has read V
    issue_v(s + ST, slot);
  }
  cp_async_wait<0>();
  __syncthreads();  // every warp is done with its ring: the warps' results go there

  // ---- the warps' results ----
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    float mi[2], li[2];
    f2_unpack(m[i], mi[0], mi[1]);
    f2_unpack(l[i], li[0], li[1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) li[e] += __shfl_xor_sync(0xffffffffu, li[e], x);
      const int r = i * 8 + 2 * t4 + e;
      if (g == 0) ml[warp][r][0] = mi[e], ml[warp][r][1] = li[e];
      float* dst = join + (warp * ROWS + r) * Gm::JOIN_PITCH;
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
  }
  __syncthreads();
}

// Row r, column quad c of a CTA's warps' results joined: O (unnormalised) and its maximum and sum.
template <int D, bool Q8, int NT, class Shared>
__device__ __forceinline__ float4 paged_join_warps(const float* join, const Shared& sh, int r, int c, float& mx, float& lsum) {
  using Gm = PagedGeom<D, Q8, NT>;
  mx = sh.ml[0][r][0];
#pragma unroll
  for (int w = 1; w < Gm::NW; ++w) mx = fmaxf(mx, sh.ml[w][r][0]);
  lsum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < Gm::NW; ++w) {
    const PagedRescale<Q8> f(sh.ml[w][r][0] - mx);
    const float4 a = *reinterpret_cast<const float4*>(join + (w * Gm::ROWS + r) * Gm::JOIN_PITCH + 4 * c);
    lsum = fmaf(sh.ml[w][r][1] * f.l0, f.l1, lsum);
    o.x = fmaf(a.x, f.o, o.x), o.y = fmaf(a.y, f.o, o.y), o.z = fmaf(a.z, f.o, o.z), o.w = fmaf(a.w, f.o, o.w);
  }
  return o;
}

// A finished row's column quad (and, with the first, its lse): mx and lsum its reference and sum (0: it saw no key).
template <int D, bool BF16, bool Q8>
__device__ __forceinline__ void paged_store(const PagedAttnParams& p, size_t row, int c, const float4& o, float mx, float lsum) {
  if constexpr (Q8) lsum *= exp2_int(-kPLift);
  const float by = lsum == 0.f ? 0.f : 1.f / lsum;
  if (!dbg_in_range(row, 1, static_cast<size_t>(p.B) * p.Hq * p.T, p.status, 122)) return;
  reinterpret_cast<uint2*>(p.o)[row * (D / 4) + c] = make_uint2(Elem<BF16>::pack(o.x * by, o.y * by), Elem<BF16>::pack(o.z * by, o.w * by));
  if (c == 0) p.lse[row] = lsum == 0.f ? INFINITY : mx + log2f(lsum);
}

// A piece of the work per CTA; heads that several pieces share leave partial results.
template <int D, bool BF16, bool Q8, int NT>
__global__ void __launch_bounds__(PagedGeom<D, Q8, NT>::THREADS, PagedGeom<D, Q8, NT>::PER_SM) attn_paged_kernel(const PagedAttnParams p) {
  using Gm = PagedGeom<D, Q8, NT>;
  constexpr int ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ PagedShared<Gm::NW, Gm::ST, ROWS> sh;
  const float* join = reinterpret_cast<const float*>(smem);
  int* starts = reinterpret_cast<int*>(smem + Gm::SMEM);  // [B + 1], then lengths [B]
  grid_dependency_wait();  // the kernels before this one are complete
  if (threadIdx.x == 0) grid_launch_dependents();
  paged_starts(p, Gm::KS, starts, starts + p.B + 1);
  const PagedPieces pieces(starts[p.B], p.n_groups);
  if (blockIdx.x >= pieces.n) return;
  int u = pieces.first(blockIdx.x);
  const int u_end = pieces.first(blockIdx.x + 1);
  while (u < u_end) {
    const PagedHead hd = paged_head(p, starts, u);
    const int s0 = u - hd.start, left = hd.start + hd.steps + kPagedExtra - u;
    const int s1 = min(hd.steps, s0 + min(left, u_end - u));
    u += left;  // the next head, if any
    if (s0 >= s1 && !(hd.steps == 0 && s0 == 0)) continue;  // only the head's extra units
    __syncthreads();  // the results of the head before are read
    paged_part<D, BF16, Q8, NT>(p, hd, s0, s1, starts[p.B + 1 + hd.b], smem, sh);
    const bool whole = s0 == 0 && s1 == hd.steps;
    const size_t part0 = (static_cast<size_t>(blockIdx.x) * 2 + (s0 == 0 ? 1 : 0)) * ROWS;
    const size_t out0 = (static_cast<size_t>(hd.b) * p.c.Hkv + hd.h) * p.R + hd.rb * ROWS;
    for (int x = threadIdx.x; x < ROWS * (D / 4); x += Gm::THREADS) {
      const int r = x / (D / 4), c = x - r * (D / 4);
      if (hd.rb * ROWS + r >= p.R) continue;
      float mx, lsum;
      const float4 o = paged_join_warps<D, Q8, NT>(join, sh, r, c, mx, lsum);
      if (whole) {
        paged_store<D, BF16, Q8>(p, out0 + r, c, o, mx, lsum);
      } else if (dbg_in_range(part0 + r, 1, static_cast<size_t>(p.n_groups) * 2 * ROWS, p.status, 123)) {
        reinterpret_cast<float4*>(p.part)[(part0 + r) * (D / 4) + c] = o;
        if (c == 0) reinterpret_cast<float2*>(p.part_ml)[part0 + r] = make_float2(mx, lsum);
      }
    }
  }
}

// Short caches: a cluster of `size` CTAs per head shares its steps out and joins their results through distributed
// shared memory, in one launch.
template <int D, bool BF16, bool Q8, int NT>
__global__ void __launch_bounds__(PagedGeom<D, Q8, NT>::THREADS, PagedGeom<D, Q8, NT>::PER_SM) attn_paged_cluster_kernel(const PagedAttnParams p, int size) {
  using Gm = PagedGeom<D, Q8, NT>;
  constexpr int ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ PagedShared<Gm::NW, Gm::ST, ROWS> sh;
  __shared__ float2 stat[ROWS];  // the CTA's maxima and sums
  float* join = reinterpret_cast<float*>(smem);
  grid_dependency_wait();  // the kernels before this one are complete
  if (threadIdx.x == 0) grid_launch_dependents();
  const int rank = blockIdx.x % size, i = blockIdx.x / size;
  PagedHead hd;
  hd.rb = i % p.n_rb, hd.h = i / p.n_rb % p.c.Hkv, hd.b = i / (p.n_rb * p.c.Hkv), hd.start = 0;
  const int n = clamp_len(p.cache_len[hd.b], p.c.per_seq << p.c.shift);
  hd.steps = (n + Gm::KS - 1) / Gm::KS;
  paged_part<D, BF16, Q8, NT>(p, hd, hd.steps * rank / size, hd.steps * (rank + 1) / size, n, smem, sh);
  const size_t out0 = (static_cast<size_t>(hd.b) * p.c.Hkv + hd.h) * p.R + hd.rb * ROWS;
  const int rows = min(ROWS, p.R - hd.rb * ROWS);
  for (int x = threadIdx.x; x < rows * (D / 4); x += Gm::THREADS) {
    const int r = x / (D / 4), c = x - r * (D / 4);
    float mx, lsum;
    const float4 o = paged_join_warps<D, Q8, NT>(join, sh, r, c, mx, lsum);
    if (size == 1) {
      paged_store<D, BF16, Q8>(p, out0 + r, c, o, mx, lsum);
    } else {  // over the first warp's, which no other thread reads here
      *reinterpret_cast<float4*>(join + r * Gm::JOIN_PITCH + 4 * c) = o;
      if (c == 0) stat[r] = make_float2(mx, lsum);
    }
  }
  if (size == 1) return;
  cluster_sync_all();
  const uint32_t join_at = smem_u32(join), stat_at = smem_u32(stat);
  for (int x = rank * Gm::THREADS + threadIdx.x; x < rows * (D / 4); x += size * Gm::THREADS) {
    const int r = x / (D / 4), c = x - r * (D / 4);
    float mx = -INFINITY, lsum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float2 ml[kPagedCluster];
#pragma unroll
    for (int k = 0; k < kPagedCluster; ++k) {
      ml[k] = k < size ? ld_cluster_f2(cluster_map(stat_at + r * 8, k)) : make_float2(-INFINITY, 0.f);
      mx = fmaxf(mx, ml[k].x);
    }
#pragma unroll
    for (int k = 0; k < kPagedCluster; ++k) {
      if (k >= size) continue;
      const PagedRescale<Q8> f(ml[k].x - mx);
      const float4 a = ld_cluster_f4(cluster_map(join_at + (r * Gm::JOIN_PITCH + 4 * c) * 4, k));
      lsum = fmaf(ml[k].y * f.l0, f.l1, lsum);
      o.x = fmaf(a.x, f.o, o.x), o.y = fmaf(a.y, f.o, o.y), o.z = fmaf(a.z, f.o, o.z), o.w = fmaf(a.w, f.o, o.w);
    }
    paged_store<D, BF16, Q8>(p, out0 + r, c, o, mx, lsum);
  }
  cluster_sync_all();  // no CTA leaves while others read its results
}

// Joins the partial results of the heads that several CTAs worked on: WARPS
// warps of a block share out a packed row's partial results (1: a warp per row).
constexpr int kPagedJoinThreads = 256;

template <int D, bool BF16, bool Q8, int NT, int WARPS>
__global__ void __launch_bounds__(kPagedJoinThreads) attn_paged_join_kernel(const PagedAttnParams p) {
  using Gm = PagedGeom<D, Q8, NT>;
  constexpr int ROWS = 8 * NT, QUADS = D / 4, Q = (QUADS + 31) / 32;  // column quads, and a lane's
  __shared__ int starts[kPagedMaxB + 1];
  __shared__ float4 sum[WARPS > 1 ? WARPS : 1][QUADS];
  __shared__ float2 stat[WARPS];
  // (lengths: nothing that the kernel before writes; it has waited for what did.  So the first row's part of the plan is
  // worked out before the wait.)
  paged_starts(p, Gm::KS, starts, nullptr);
  bool waited = false;
  const PagedPieces pieces(starts[p.B], p.n_groups);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // (a lane past the columns loads the last again: no branch around the loads)
  const float4* part = reinterpret_cast<const float4*>(p.part) + min(lane, QUADS - 1);
  const long long tasks = static_cast<long long>(p.B) * p.c.Hkv * p.R;
  constexpr int PER = kPagedJoinThreads / 32 / WARPS;  // rows of a block
  for (long long task = static_cast<long long>(blockIdx.x) * PER + (WARPS > 1 ? 0 : warp); task < tasks;
       task += static_cast<long long>(gridDim.x) * PER) {
    const long long bh = task / p.R;
    const int pr = static_cast<int>(task - bh * p.R), rb = pr / ROWS, r = pr - rb * ROWS;
    const int b = static_cast<int>(bh / p.c.Hkv), h = static_cast<int>(bh - static_cast<long long>(b) * p.c.Hkv);
    const int per = (starts[b + 1] - starts[b]) / (p.c.Hkv * p.n_rb);
    const int s = starts[b] + (h * p.n_rb + rb) * per;
    const int steps = per - kPagedExtra;
    if (steps == 0) continue;
    const int c0 = pieces.of(s), c1 = pieces.of(s + steps - 1);
    if (c0 == c1) continue;  // one CTA had it all
    if (!waited) grid_dependency_wait();
    waited = true;
    const int n = c1 - c0 + 1, first = WARPS > 1 ? n * warp / WARPS : 0, last = WARPS > 1 ? n * (warp + 1) / WARPS : n;
    auto at = [&](int i) { return ((c0 + i) * 2 + (i == 0 ? 1 : 0)) * ROWS + r; };
    // this warp's partial results: running maximum and sums, 32 of them at a time
    float mx = -INFINITY, l = 0.f;
    float4 o[Q];
#pragma unroll
    for (int x = 0; x < Q; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = first; i0 < last; i0 += 32) {
      const int k = min(32, last - i0);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < k) ml = reinterpret_cast<const float2*>(p.part_ml)[at(i0 + lane)];
      // The first rows are on their way while the weights are worked out, the others loaded so many at a time, all before the
      // first is used (one head of 24137 quantised keys, 12 rows: 11.7 us; 21.6 where the sums and loads took turns).
      constexpr int AHEAD = 6, AT_ONCE = WARPS > 1 ? 13 : 8;
      float4 early[AHEAD][Q];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
#pragma unroll
        for (int x = 0; x < Q; ++x)
          if (i < k) early[i][x] = part[at(i0 + i) * QUADS + x * 32];
      float top = ml.x;
#pragma unroll
      for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      top = fmaxf(top, mx);
      const PagedRescale<Q8> part_by(ml.x - top), by(mx - top);
      const float w = part_by.o, fix = by.o;
      float add = ml.y * part_by.l0 * part_by.l1;
#pragma unroll
      for (int x = 16; x; x >>= 1) add += __shfl_xor_sync(0xffffffffu, add, x);
      l = fmaf(l * by.l0, by.l1, add);
      mx = top;
#pragma unroll
      for (int x = 0; x < Q; ++x) o[x].x *= fix, o[x].y *= fix, o[x].z *= fix, o[x].w *= fix;
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const float f = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
        for (int x = 0; x < Q; ++x) {
          if (i >= k) continue;
          const float4 a = early[i][x];
          o[x].x = fmaf(a.x, f, o[x].x), o[x].y = fmaf(a.y, f, o[x].y), o[x].z = fmaf(a.z, f, o[x].z), o[x].w = fmaf(a.w, f, o[x].w);
        }
      }
      for (int j = AHEAD; j < k; j += AT_ONCE) {
        float4 more[AT_ONCE][Q];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
          for (int x = 0; x < Q; ++x) more[i][x] = part[at(i0 + min(j + i, k - 1)) * QUADS + x * 32];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
          const float f = __shfl_sync(0xffffffffu, w, (j + i) & 31);
#pragma unroll
          for (int x = 0; x < Q; ++x) {
            if (j + i >= k) continue;
            const float4 a = more[i][x];
            o[x].x = fmaf(a.x, f, o[x].x), o[x].y = fmaf(a.y, f, o[x].y), o[x].z = fmaf(a.z, f, o[x].z), o[x].w = fmaf(a.w, f, o[x].w);
          }
        }
      }
    }
    if constexpr (WARPS > 1) {
      __syncthreads();  // (the row before is read)
      if (lane == 0) stat[warp] = make_float2(mx, l);
#pragma unroll
      for (int x = 0; x < Q; ++x)
        if (QUADS % 32 == 0 || x * 32 + lane < QUADS) sum[warp][x * 32 + lane] = o[x];
      __syncthreads();
      if (warp != 0) continue;
      float top = mx;
#pragma unroll
      for (int w = 1; w < WARPS; ++w) top = fmaxf(top, stat[w].x);
      l = 0.f;
#pragma unroll
      for (int x = 0; x < Q; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const PagedRescale<Q8> by(stat[w].x - top);
        const float f = by.o;
        l = fmaf(stat[w].y * by.l0, by.l1, l);
#pragma unroll
        for (int x = 0; x < Q; ++x) {
          if (QUADS % 32 != 0 && x * 32 + lane >= QUADS) continue;
          const float4 a = sum[w][x * 32 + lane];
          o[x].x = fmaf(a.x, f, o[x].x), o[x].y = fmaf(a.y, f, o[x].y), o[x].z = fmaf(a.z, f, o[x].z), o[x].w = fmaf(a.w, f, o[x].w);
        }
      }
      mx = top;
    }
    if constexpr (Q8) l *= exp2_int(-kPLift);
    const float by = l == 0.f ? 0.f : 1.f / l;
    if (dbg_in_range(task, 1, static_cast<size_t>(tasks), p.status, 124)) {
#pragma unroll
      for (int x = 0; x < Q; ++x)
        if (QUADS % 32 == 0 || x * 32 + lane < QUADS)
          reinterpret_cast<uint2*>(p.o)[static_cast<size_t>(task) * QUADS + x * 32 + lane] =
              make_uint2(Elem<BF16>::pack(o[x].x * by, o[x].y * by), Elem<BF16>::pack(o[x].z * by, o[x].w * by));
      if (lane == 0) p.lse[task] = l == 0.f ? INFINITY : mx + log2f(l);
    }
  }
  // (a grid that ended before the one ahead of it would let the next one in early)
  if (!waited) grid_dependency_wait();
}

}  // namespace gbattn
