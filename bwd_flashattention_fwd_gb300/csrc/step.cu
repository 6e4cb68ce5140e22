// C ABI of the calls around attention in a model step (declared in
// include/gbattn.h): norm and rotation of queries and keys, the paged cache,
// verification of drafts.  Validation is on the host and touches no device
// memory; lengths, pages and tokens that live on the device are brought into
// range by the kernels.
#include "step.h"

#include "abi.h"
#include "paged_kernel.cuh"
#include "rope_kernel.cuh"
#include "verify_kernel.cuh"

namespace gbattn {
namespace {

// Rows [B, H, L, D] at strides: none negative, each a multiple of 8 elements
// (16 bytes); a size of 1 has no stride.
attn_status_t check_strides(const int64_t* st, int B, int H, int L) {
  const int size[3] = {B, H, L};
  for (int i = 0; i < 3; ++i) {
    if (size[i] == 1) continue;
    if (st[i] < 0 || st[i] % 8 != 0) return ATTN_ERR_INVALID_ARG;
    // (bytes between heads are counted in 32 bits)
    if (st[i] > (int64_t{1} << 40) || (i == 1 && st[i] > 0x7fffffffLL)) return ATTN_ERR_UNSUPPORTED;
  }
  return ATTN_OK;
}

// Whether no two rows of [B, H, L, D] at these strides share an element: each
// stride reaches past all that the smaller ones span.
bool disjoint_rows(int B, int H, int L, int D, const int64_t* st) {
  const int size[3] = {B, H, L};
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[order[j]] < st[order[i]]) { const int t = order[i]; order[i] = order[j], order[j] = t; }
  int64_t span = D;
  for (const int i : order) {
    if (size[i] == 1) continue;
    if (st[i] < span) return false;
    span += (size[i] - 1) * st[i];
  }
  return true;
}

Span rows_span(const void* at, int B, int H, int L, int D, const int64_t* st) {
  return {at, 2 * ((B - 1) * st[0] + (H - 1) * st[1] + (L - 1) * st[2] + D)};
}

// Whether off + sum n_i s_i, lo_i <= n_i <= hi_i, comes within D of 0 for the dimensions order[i] on, the widest stride
// first.  What the narrower ones span is at most a stride, so each n_i is one of the two that bring the sum across 0.
bool rows_meet(int64_t off, const int64_t (&s)[3], const int (&lo)[3], const int (&hi)[3], const int (&order)[3], int i, int D) {
  if (i == 3) return off > -D && off < D;
  const int k = order[i];
  if (lo[k] == 0 && hi[k] == 0) return rows_meet(off, s, lo, hi, order, i + 1, D);
  const int64_t n = off <= 0 ? -off / s[k] : -((off + s[k] - 1) / s[k]);  // floor(-off / s)
  for (int64_t x = n; x <= n + 1; ++x)
    if (x >= lo[k] && x <= hi[k] && rows_meet(off + x * s[k], s, lo, hi, order, i + 1, D)) return true;
  return false;
}

// Whether two sets of rows (each with no element twice) have an element in common, exact for views of one packed array:
// strides alike wherever a size has them, starts a whole number of rows apart.  Others are taken to, where what they span overlaps.
bool rows_overlap(const void* a, int Ha, const int64_t* sa, const void* b, int Hb, const int64_t* sb, int B, int L, int D) {
  if (!overlap(rows_span(a, B, Ha, L, D, sa), rows_span(b, B, Hb, L, D, sb))) return false;
  if ((B > 1 && sa[0] != sb[0]) || (Ha > 1 && Hb > 1 && sa[1] != sb[1]) || (L > 1 && sa[2] != sb[2])) return true;
  const int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  if (off % (2 * D) != 0) return true;
  const int64_t s[3] = {sa[0], Ha > 1 ? sa[1] : sb[1], sa[2]};
  const int lo[3] = {1 - B, 1 - Ha, 1 - L}, hi[3] = {B - 1, Hb - 1, L - 1};
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (s[order[j]] > s[order[i]]) { const int t = order[i]; order[i] = order[j], order[j] = t; }
  return rows_meet(off / 2, s, lo, hi, order, 0, D);
}

void dense(int64_t* st, int H, int L, int D) {
  st[0] = static_cast<int64_t>(H) * L * D, st[1] = static_cast<int64_t>(L) * D, st[2] = D;
}

attn_status_t check_rope(const void* q, const void* k, const void* qw, const void* kw, const int32_t* pos,
                         const float* freq, const void* y0, const void* y1, const int64_t* qs, const int64_t* ks, int B,
                         int Hq, int Hkv, int L, int D, int rot, int axes, float eps, int interleaved,
                         attn_dtype_t dtype) {
  if (!q || !k || !pos || !freq || !y0 || !y1 || !qs || !ks || !qw != !kw) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(qw) || !aligned16(kw) || !aligned16(y0) || !aligned16(y1) ||
      !aligned4(pos) || !aligned4(freq))
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || L < 1 || rot < 2 || rot > D || axes < 1) return ATTN_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps) || (interleaved != 0 && interleaved != 1)) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_DTYPE_FP16 && dtype != ATTN_DTYPE_BF16) return ATTN_ERR_INVALID_ARG;
  if (!supported_d(D) || rot % 16 != 0 || axes > kRopeMaxAxes) return ATTN_ERR_UNSUPPORTED;
  // units of work and rows are counted in 32 bits beside a token's number
  if (static_cast<long long>(B) * L > (1 << 30) || Hq > 65535 || Hkv > 65535 || static_cast<long long>(L) * D > 0x7fffffffLL)
    return ATTN_ERR_UNSUPPORTED;
  const attn_status_t a = check_strides(qs, B, Hq, L), b = check_strides(ks, B, Hkv, L);
  return a != ATTN_OK ? a : b;
}

template <int D, bool BF16, bool INTERLEAVED, bool BWD>
int rope_impl(const RopeParams& p, int num_sms, cudaStream_t stream) {
  using Gm = RopeGeom<D, BWD>;
  const int sms = num_sms < kTreeMaxCtas ? num_sms : kTreeMaxCtas;
  const long long tokens = static_cast<long long>(p.B) * p.L;
  long long most = static_cast<long long>(Gm::PER_SM) * sms;
  // Three CTAs after one another where each has work enough: SMs that get less of the memory's bandwidth take fewer
  // (32768 tokens 110.0 us, one each 121.6; 16384 56.2 and 57.5; 12000 46.1 and 45.4; the gradient, 32768 tokens: 167.6
  // and 166.6).
  if (!BWD && tokens >= 32 * most) most *= 3;
  // few tokens: their heads are shared out too, one round of the CTA's groups at least
  const int blocks = static_cast<int>(tokens < most ? tokens : most), heads = (p.x[0].H + Gm::GROUPS - 1) / Gm::GROUPS;
  const int parts = most / blocks < heads ? static_cast<int>(most / blocks) : heads, grid = blocks * parts;
  const int per = static_cast<int>(tokens / blocks), more = static_cast<int>(tokens % blocks), half = p.rot / 2;
  const auto kern = rope_kernel<D, BF16, INTERLEAVED, BWD>;
  static std::atomic<uint64_t> done{0};
  if (!set_smem_limit(kern, Gm::SMEM, done)) return kLaunchCudaError;
  const int r = launch_dependent(kern, dim3(blocks, parts), kRopeThreads, Gm::SMEM, stream, p, parts, per, more, (65536 + half - 1) / half);
  if (r != kLaunchOk || !BWD || !p.w[0]) return r;
  return launch_dependent(rope_dw_kernel, dim3(2 * D / 8), 1024, 0, stream, p, grid);
}

template <int D, bool BF16>
int rope_dispatch(const RopeParams& p, bool interleaved, bool bwd, int num_sms, cudaStream_t stream) {
  if (bwd) return interleaved ? rope_impl<D, BF16, true, true>(p, num_sms, stream) : rope_impl<D, BF16, false, true>(p, num_sms, stream);
  return interleaved ? rope_impl<D, BF16, true, false>(p, num_sms, stream) : rope_impl<D, BF16, false, false>(p, num_sms, stream);
}

template <bool BF16>
int rope_by_d(const RopeParams& p, bool interleaved, bool bwd, int num_sms, cudaStream_t stream) {
  switch (p.D) {
    case 64: return rope_dispatch<64, BF16>(p, interleaved, bwd, num_sms, stream);
    case 96: return rope_dispatch<96, BF16>(p, interleaved, bwd, num_sms, stream);
    case 128: return rope_dispatch<128, BF16>(p, interleaved, bwd, num_sms, stream);
    default: return rope_dispatch<256, BF16>(p, interleaved, bwd, num_sms, stream);
  }
}

// Whether a paged cache of these (positive) sizes is served.
bool paged_sizes(int B, int Hkv, int page_size, int per_seq) {
  // a page's rows are found by shifts, and hold a multiple of four exponents
  if (page_size < 8 || page_size > 4096 || (page_size & (page_size - 1)) != 0) return false;
  return static_cast<long long>(per_seq) * page_size <= kPagedMaxTokens && B <= kPagedMaxB && static_cast<long long>(B) * Hkv <= 65535;
}

// Sizes, types and alignment of a paged cache.
attn_status_t check_paged(const void* k, const void* v, const int8_t* ke, const int8_t* ve, const int32_t* table, int B,
                          int Hkv, int n_pages, int page_size, int per_seq, int D, attn_dtype_t dtype) {
  if (!k || !v || !table || !ke != !ve) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned4(ke) || !aligned4(ve) || !aligned4(table)) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hkv < 1 || n_pages < 1 || page_size < 1 || per_seq < 1) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_DTYPE_FP16 && dtype != ATTN_DTYPE_BF16) return ATTN_ERR_INVALID_ARG;
  if (!supported_d(D)) return ATTN_ERR_UNSUPPORTED;
  return paged_sizes(B, Hkv, page_size, per_seq) ? ATTN_OK : ATTN_ERR_UNSUPPORTED;
}

PagedCache paged_cache(const void* k, const void* v, const int8_t* ke, const int8_t* ve, const int32_t* table, int Hkv,
                       int n_pages, int page_size, int per_seq, int D) {
  int shift = 0;
  while ((1 << shift) < page_size) ++shift;
  return {const_cast<void*>(k), const_cast<void*>(v), const_cast<int8_t*>(ke), const_cast<int8_t*>(ve), table, n_pages, shift, per_seq, Hkv, D};
}

long long pool_rows(int Hkv, int n_pages, int page_size) { return static_cast<long long>(n_pages) * Hkv * page_size; }

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

template <int D, bool BF16, bool WIDE>
int write_impl(const PagedWriteParams& p, int num_sms, cudaStream_t stream) {
  constexpr int per_cta = kPagedThreads / RowLanes<D>::GROUP;
  const long long ctas = (static_cast<long long>(p.B) * p.c.Hkv * p.T + per_cta - 1) / per_cta, most = 8LL * num_sms;
  const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most));
  return p.c.k_exp ? launch_dependent(attn_paged_write_kernel<D, BF16, true, WIDE>, grid, kPagedThreads, 0, stream, p)
                   : launch_dependent(attn_paged_write_kernel<D, BF16, false, WIDE>, grid, kPagedThreads, 0, stream, p);
}

template <int D, bool BF16, bool WIDE>
int read_impl(const PagedReadParams& p, int num_sms, cudaStream_t stream) {
  const int room = p.c.per_seq << p.c.shift, heads = p.B * p.c.Hkv;
  const long long blocks = (static_cast<long long>(p.Lk < room ? p.Lk : room) + read_rows(D) - 1) / read_rows(D);
  const long long most = 64LL * num_sms / heads + 1;  // (blocks past a sequence's end leave at once)
  const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most), heads);
  return p.c.k_exp ? launch_dependent(attn_paged_read_kernel<D, BF16, true, WIDE>, grid, kPagedThreads, 0, stream, p)
                   : launch_dependent(attn_paged_read_kernel<D, BF16, false, WIDE>, grid, kPagedThreads, 0, stream, p);
}

template <template <int, bool> class F, typename P>
int by_type(const P& p, int D, bool bf16, int num_sms, cudaStream_t stream) {
  switch (D) {
    case 64: return bf16 ? F<64, true>::run(p, num_sms, stream) : F<64, false>::run(p, num_sms, stream);
    case 96: return bf16 ? F<96, true>::run(p, num_sms, stream) : F<96, false>::run(p, num_sms, stream);
    case 128: return bf16 ? F<128, true>::run(p, num_sms, stream) : F<128, false>::run(p, num_sms, stream);
    default: return bf16 ? F<256, true>::run(p, num_sms, stream) : F<256, false>::run(p, num_sms, stream);
  }
}
template <int D, bool BF16>
struct Write {
  static int run(const PagedWriteParams& p, int n, cudaStream_t s) {
    const bool wide = aligned32(p.k_new) && aligned32(p.v_new) && (p.c.k_exp || (aligned32(p.c.k) && aligned32(p.c.v)));
    return wide ? write_impl<D, BF16, true>(p, n, s) : write_impl<D, BF16, false>(p, n, s);
  }
};
template <int D, bool BF16>
struct Read {
  static int run(const PagedReadParams& p, int n, cudaStream_t s) {
    const bool wide = aligned32(p.k) && aligned32(p.v) && (p.c.k_exp || (aligned32(p.c.k) && aligned32(p.c.v)));
    return wide ? read_impl<D, BF16, true>(p, n, s) : read_impl<D, BF16, false>(p, n, s);
  }
};

attn_status_t check_paged_attn(int B, int Hq, int Hkv, int T, int page_size, int per_seq, int D) {
  if (B < 1 || Hq < 1 || Hkv < 1 || T < 1 || page_size < 1 || per_seq < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (!supported_d(D) || !paged_sizes(B, Hkv, page_size, per_seq)) return ATTN_ERR_UNSUPPORTED;
  const long long rows = static_cast<long long>(Hq / Hkv) * T, room = static_cast<long long>(per_seq) * page_size;
  if (rows > kPagedMaxRows) return ATTN_ERR_UNSUPPORTED;
  // the units of work of the whole call are ints (steps of 32 keys at least)
  const long long blocks = (rows + paged_rows(static_cast<int>(rows), D) - 1) / paged_rows(static_cast<int>(rows), D);
  if ((room / 32 + 4) * B * Hkv * blocks > 0x7fff0000LL) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" attn_status_t attn_qk_norm_rope(const void* q, const void* k, const void* q_weight, const void* k_weight,
                                           const int32_t* pos, const float* freq, const uint8_t* axis, void* q_out,
                                           void* k_out, const int64_t* q_strides, const int64_t* k_strides, int B,
                                           int Hq, int Hkv, int L, int D, int rot, int axes, float eps,
                                           int interleaved, attn_dtype_t dtype, cudaStream_t stream) {
  const attn_status_t s = check_rope(q, k, q_weight, k_weight, pos, freq, q_out, k_out, q_strides, k_strides, B, Hq,
                                     Hkv, L, D, rot, axes, eps, interleaved, dtype);
  if (s != ATTN_OK) return s;
  int64_t qd[3], kd[3];
  dense(qd, Hq, L, D), dense(kd, Hkv, L, D);
  const Span qo = rows_span(q_out, B, Hq, L, D, qd), ko = rows_span(k_out, B, Hkv, L, D, kd);
  const Span qi = rows_span(q, B, Hq, L, D, q_strides), ki = rows_span(k, B, Hkv, L, D, k_strides);
  const long long tokens = static_cast<long long>(B) * L;
  const Span spans[] = {qo, ko, {q_weight, 2 * D}, {k_weight, 2 * D}, {pos, 4 * tokens * axes}, {freq, 2 * rot}, {axis, rot / 2}};
  if (outputs_overlap(spans, 2) || overlap(qo, ki) || overlap(ko, qi)) return ATTN_ERR_INVALID_ARG;
  // in place a row's lanes read all of it before they write it; any other shared storage would be read after
  auto in_place = [&](const void* out, const void* in, int H, const int64_t* st, const int64_t* d) {
    return out == in && (B == 1 || st[0] == d[0]) && (H == 1 || st[1] == d[1]) && (L == 1 || st[2] == d[2]);
  };
  if (overlap(qo, qi) && !in_place(q_out, q, Hq, q_strides, qd)) return ATTN_ERR_INVALID_ARG;
  if (overlap(ko, ki) && !in_place(k_out, k, Hkv, k_strides, kd)) return ATTN_ERR_INVALID_ARG;
  int dev, num_sms, *status;
  EncodeTiledFn enc;
  const attn_status_t ds = call_state(stream, &dev, &enc, &status, &num_sms);
  if (ds != ATTN_OK) return ds;
  RopeParams p{};
  p.x[0] = {const_cast<void*>(q), q_strides[0], q_strides[1], q_strides[2], Hq};
  p.x[1] = {const_cast<void*>(k), k_strides[0], k_strides[1], k_strides[2], Hkv};
  p.y[0] = q_out, p.y[1] = k_out, p.w[0] = q_weight, p.w[1] = k_weight;
  p.pos = pos, p.freq = freq, p.axis = axis;
  p.B = B, p.L = L, p.D = D, p.rot = rot, p.axes = axes, p.eps = eps, p.status = status;
  return finish(dtype == ATTN_DTYPE_BF16 ? rope_by_d<true>(p, interleaved, false, num_sms, stream)
                                         : rope_by_d<false>(p, interleaved, false, num_sms, stream));
}

extern "C" size_t attn_qk_norm_rope_workspace_bytes(int D) {
  return supported_d(D) ? static_cast<size_t>(kRopeBwdPerSm) * kTreeMaxCtas * 2 * D * sizeof(float) : 0;
}

extern "C" attn_status_t attn_qk_norm_rope_bwd(const void* q, const void* k, const void* q_weight,
                                               const void* k_weight, const int32_t* pos, const float* freq,
                                               const uint8_t* axis, const void* dq_out, const void* dk_out, void* dq,
                                               void* dk, float* dq_weight, float* dk_weight, void* workspace,
                                               size_t workspace_bytes, const int64_t* q_strides,
                                               const int64_t* k_strides, const int64_t* dq_strides,
                                               const int64_t* dk_strides, int B, int Hq, int Hkv, int L, int D,
                                               int rot, int axes, float eps, int interleaved, attn_dtype_t dtype,
                                               cudaStream_t stream) {
  if (!dq || !dk || !dq_strides || !dk_strides || !workspace || !aligned16(dq) || !aligned16(dk) || !aligned16(workspace))
    return ATTN_ERR_INVALID_ARG;
  if (!dq_weight != !q_weight || !dk_weight != !k_weight || !aligned4(dq_weight) || !aligned4(dk_weight)) return ATTN_ERR_INVALID_ARG;
  attn_status_t s = check_rope(q, k, q_weight, k_weight, pos, freq, dq_out, dk_out, q_strides, k_strides, B, Hq, Hkv, L,
                               D, rot, axes, eps, interleaved, dtype);
  if (s != ATTN_OK) return s;
  s = check_strides(dq_strides, B, Hq, L);
  if (s == ATTN_OK) s = check_strides(dk_strides, B, Hkv, L);
  if (s != ATTN_OK) return s;
  if (workspace_bytes < attn_qk_norm_rope_workspace_bytes(D)) return ATTN_ERR_INVALID_ARG;
  if (!disjoint_rows(B, Hq, L, D, dq_strides) || !disjoint_rows(B, Hkv, L, D, dk_strides)) return ATTN_ERR_INVALID_ARG;
  if (rows_overlap(dq, Hq, dq_strides, dk, Hkv, dk_strides, B, L, D)) return ATTN_ERR_INVALID_ARG;
  int64_t qd[3], kd[3];
  dense(qd, Hq, L, D), dense(kd, Hkv, L, D);
  const long long tokens = static_cast<long long>(B) * L;
  const Span ins[] = {rows_span(q, B, Hq, L, D, q_strides), rows_span(k, B, Hkv, L, D, k_strides), rows_span(dq_out, B, Hq, L, D, qd),
                      rows_span(dk_out, B, Hkv, L, D, kd), {q_weight, 2 * D}, {k_weight, 2 * D}, {pos, 4 * tokens * axes}, {freq, 2 * rot},
                      {axis, rot / 2}};
  const Span gq = rows_span(dq, B, Hq, L, D, dq_strides), gk = rows_span(dk, B, Hkv, L, D, dk_strides);
  const Span wq = {dq_weight, 4 * D}, wk = {dk_weight, 4 * D}, ws = {workspace, static_cast<long long>(workspace_bytes)};
  for (const Span& in : ins)
    for (const Span& out : {gq, gk, wq, wk})
      if (overlap(in, out)) return ATTN_ERR_INVALID_ARG;
  if (overlap(wq, wk) || overlap(wq, gq) || overlap(wq, gk) || overlap(wk, gq) || overlap(wk, gk)) return ATTN_ERR_INVALID_ARG;
  for (const Span& x : {gq, gk, wq, wk})
    if (overlap(x, ws)) return ATTN_ERR_INVALID_ARG;
  int dev, num_sms, *status;
  EncodeTiledFn enc;
  const attn_status_t ds = call_state(stream, &dev, &enc, &status, &num_sms);
  if (ds != ATTN_OK) return ds;
  RopeParams p{};
  p.x[0] = {const_cast<void*>(q), q_strides[0], q_strides[1], q_strides[2], Hq};
  p.x[1] = {const_cast<void*>(k), k_strides[0], k_strides[1], k_strides[2], Hkv};
  p.dx[0] = {dq, dq_strides[0], dq_strides[1], dq_strides[2], Hq};
  p.dx[1] = {dk, dk_strides[0], dk_strides[1], dk_strides[2], Hkv};
  p.y[0] = const_cast<void*>(dq_out), p.y[1] = const_cast<void*>(dk_out), p.w[0] = q_weight, p.w[1] = k_weight;
  p.dw[0] = dq_weight, p.dw[1] = dk_weight, p.part = static_cast<float*>(workspace);
  p.pos = pos, p.freq = freq, p.axis = axis;
  p.B = B, p.L = L, p.D = D, p.rot = rot, p.axes = axes, p.eps = eps, p.status = status;
  return finish(dtype == ATTN_DTYPE_BF16 ? rope_by_d<true>(p, interleaved, true, num_sms, stream)
                                         : rope_by_d<false>(p, interleaved, true, num_sms, stream));
}

extern "C" attn_status_t attn_paged_write(const void* k_new, const void* v_new, void* k_pages, void* v_pages,
                                          int8_t* k_exp, int8_t* v_exp, const int32_t* table, const int32_t* cache_len,
                                          const int32_t* new_len, int32_t* cache_len_out, int B, int Hkv, int T,
                                          int n_pages, int page_size, int per_seq, int D, attn_dtype_t dtype,
                                          cudaStream_t stream) {
  if (!k_new || !v_new || !cache_len || !cache_len_out || T < 1) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned4(cache_len) || !aligned4(new_len) || !aligned4(cache_len_out))
    return ATTN_ERR_INVALID_ARG;
  const attn_status_t s = check_paged(k_pages, v_pages, k_exp, v_exp, table, B, Hkv, n_pages, page_size, per_seq, D, dtype);
  if (s != ATTN_OK) return s;
  // rows are counted in 32 bits (a row has 128 bytes at least)
  if (T > kPagedMaxTokens || static_cast<long long>(B) * Hkv * T > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  const long long pool = pool_rows(Hkv, n_pages, page_size), ints = 4LL * B, fresh = 2LL * B * Hkv * T * D;
  const long long bytes = pool * D * (k_exp ? 1 : 2);
  const Span spans[] = {{cache_len_out, ints}, {k_pages, bytes}, {v_pages, bytes}, {k_exp, pool}, {v_exp, pool}, {k_new, fresh},
                        {v_new, fresh}, {table, ints * per_seq}, {cache_len, ints}, {new_len, ints}};
  if (outputs_overlap(spans, 5)) return ATTN_ERR_INVALID_ARG;
  int dev, num_sms, *status;
  EncodeTiledFn enc;
  const attn_status_t ds = call_state(stream, &dev, &enc, &status, &num_sms);
  if (ds != ATTN_OK) return ds;
  const PagedWriteParams p{paged_cache(k_pages, v_pages, k_exp, v_exp, table, Hkv, n_pages, page_size, per_seq, D),
                           k_new, v_new, cache_len, new_len, cache_len_out, B, T, status};
  return finish(by_type<Write>(p, D, dtype == ATTN_DTYPE_BF16, num_sms, stream));
}

extern "C" attn_status_t attn_paged_read(const void* k_pages, const void* v_pages, const int8_t* k_exp,
                                         const int8_t* v_exp, const int32_t* table, const int32_t* cache_len, void* k,
                                         void* v, int64_t kv_pitch, int B, int Hkv, int Lk, int n_pages, int page_size,
                                         int per_seq, int D, attn_dtype_t dtype, cudaStream_t stream) {
  if (!cache_len || !k || !v || !aligned4(cache_len) || !aligned16(k) || !aligned16(v)) return ATTN_ERR_INVALID_ARG;
  if (Lk < 1 || kv_pitch < 0 || (kv_pitch != 0 && kv_pitch < Lk)) return ATTN_ERR_INVALID_ARG;
  const attn_status_t s = check_paged(k_pages, v_pages, k_exp, v_exp, table, B, Hkv, n_pages, page_size, per_seq, D, dtype);
  if (s != ATTN_OK) return s;
  if (Lk > kCacheMaxLk || kv_pitch > (int64_t{1} << 40) / (2 * D)) return ATTN_ERR_UNSUPPORTED;
  const int64_t pitch = kv_pitch ? kv_pitch : Lk;
  const long long pool = pool_rows(Hkv, n_pages, page_size), ints = 4LL * B, out = 2LL * D * ((static_cast<long long>(B) * Hkv - 1) * pitch + Lk);
  const long long bytes = pool * D * (k_exp ? 1 : 2);
  const Span spans[] = {{k, out}, {v, out}, {k_pages, bytes}, {v_pages, bytes}, {k_exp, pool}, {v_exp, pool},
                        {table, ints * per_seq}, {cache_len, ints}};
  if (outputs_overlap(spans, 2)) return ATTN_ERR_INVALID_ARG;
  int dev, num_sms, *status;
  EncodeTiledFn enc;
  const attn_status_t ds = call_state(stream, &dev, &enc, &status, &num_sms);
  if (ds != ATTN_OK) return ds;
  const PagedReadParams p{paged_cache(k_pages, v_pages, k_exp, v_exp, table, Hkv, n_pages, page_size, per_seq, D), cache_len,
                          k, v, pitch, B, Lk, status};
  return finish(by_type<Read>(p, D, dtype == ATTN_DTYPE_BF16, num_sms, stream));
}

extern "C" size_t attn_paged_workspace_bytes(int B, int Hq, int Hkv, int T, int page_size, int per_seq, int D) {
  if (check_paged_attn(B, Hq, Hkv, T, page_size, per_seq, D) != ATTN_OK) return 0;
  return static_cast<size_t>(kPagedMaxCtas) * 2 * paged_rows(Hq / Hkv * T, D) * (D + 2) * sizeof(float);
}

extern "C" attn_status_t attn_fwd_paged(const void* q, const void* k_pages, const void* v_pages, const int8_t* k_exp,
                                        const int8_t* v_exp, const int32_t* table, const int32_t* cache_len, void* o,
                                        float* lse, void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv,
                                        int T, int n_pages, int page_size, int per_seq, int D, float scale,
                                        attn_dtype_t dtype, cudaStream_t stream) {
  if (!q || !cache_len || !o || !lse || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned4(cache_len) || !aligned16(o) || !aligned16(lse) || !aligned16(workspace)) return ATTN_ERR_INVALID_ARG;
  attn_status_t s = check_scale(scale);
  if (s != ATTN_OK) return s;
  s = check_paged_attn(B, Hq, Hkv, T, page_size, per_seq, D);
  if (s == ATTN_ERR_INVALID_ARG) return s;
  const attn_status_t c = check_paged(k_pages, v_pages, k_exp, v_exp, table, B, Hkv, n_pages, page_size, per_seq, D, dtype);
  if (c != ATTN_OK) return c;
  if (s != ATTN_OK) return s;
  if (workspace_bytes < attn_paged_workspace_bytes(B, Hq, Hkv, T, page_size, per_seq, D)) return ATTN_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(B) * Hq * T, pool = pool_rows(Hkv, n_pages, page_size), ints = 4LL * B;
  const long long bytes = pool * D * (k_exp ? 1 : 2);
  const Span spans[] = {{o, rows * D * 2}, {lse, rows * 4}, {workspace, static_cast<long long>(workspace_bytes)}, {q, rows * D * 2},
                        {k_pages, bytes}, {v_pages, bytes}, {k_exp, pool}, {v_exp, pool}, {table, ints * per_seq}, {cache_len, ints}};
  if (outputs_overlap(spans, 3)) return ATTN_ERR_INVALID_ARG;
  int dev, num_sms, *status;
  EncodeTiledFn enc;
  const attn_status_t ds = call_state(stream, &dev, &enc, &status, &num_sms);
  if (ds != ATTN_OK) return ds;
  PagedAttnParams p{};
  p.c = paged_cache(k_pages, v_pages, k_exp, v_exp, table, Hkv, n_pages, page_size, per_seq, D);
  p.q = q, p.cache_len = cache_len, p.o = o, p.lse = lse, p.part = static_cast<float*>(workspace);
  p.B = B, p.Hq = Hq, p.G = Hq / Hkv, p.T = T, p.R = p.G * T;
  p.scale_log2 = scale_log2_of(scale), p.status = status;
  const bool bf16 = dtype == ATTN_DTYPE_BF16;
  switch (D) {
    case 64: return finish(launch_paged_d64(p, bf16, num_sms, stream));
    case 96: return finish(launch_paged_d96(p, bf16, num_sms, stream));
    case 128: return finish(launch_paged_d128(p, bf16, num_sms, stream));
    default: return finish(launch_paged_d256(p, bf16, num_sms, stream));
  }
}

extern "C" attn_status_t attn_draft_verify(const float* target, const float* draft, const int32_t* tokens,
                                           const float* u, const float* r, const int32_t* draft_len,
                                           int32_t* accept_len, int32_t* token, int B, int T, int V,
                                           cudaStream_t stream) {
  if (!target || !tokens || !u || !r || !accept_len || !token) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(target) || !aligned16(draft) || !aligned4(tokens) || !aligned4(u) || !aligned4(r) || !aligned4(draft_len) ||
      !aligned4(accept_len) || !aligned4(token))
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || V < 1) return ATTN_ERR_INVALID_ARG;
  if (T > kTreeMaxT || B > 65535 || V > (1 << 30)) return ATTN_ERR_UNSUPPORTED;
  const long long ints = 4LL * B, rows = ints * V;
  const Span spans[] = {{accept_len, ints}, {token, ints}, {target, rows * (T + 1)}, {draft, rows * T}, {tokens, ints * T},
                        {u, ints * T}, {r, ints}, {draft_len, ints}};
  if (outputs_overlap(spans, 2)) return ATTN_ERR_INVALID_ARG;
  int dev, num_sms, *status;
  EncodeTiledFn enc;
  const attn_status_t ds = call_state(stream, &dev, &enc, &status, &num_sms);
  if (ds != ATTN_OK) return ds;
  const VerifyParams p{target, draft, tokens, u, r, draft_len, accept_len, token, B, T, V, status};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B) * kVerifyCluster);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kVerifyCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const auto kern = V < kVerifyLong ? (V % 4 == 0 ? attn_draft_verify_kernel<true, false> : attn_draft_verify_kernel<false, false>)
                                    : (V % 4 == 0 ? attn_draft_verify_kernel<true, true> : attn_draft_verify_kernel<false, true>);
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
