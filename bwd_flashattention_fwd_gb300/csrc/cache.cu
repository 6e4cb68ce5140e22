// C ABI of the cache calls (declared in include/gbattn.h): tree attention
// over a cache, appending, accumulated key weights, eviction.  Validation is
// on the host and touches no device memory; lengths, limits and indices that
// live on the device are brought into range by the kernels.
#include "../../include/gbattn.h"
#include "abi.h"
#include "cache.h"
#include "cache_kernel.cuh"

namespace gbattn {
namespace {

// Sizes and type of a cache [B, Hkv, Lk (kv_pitch), D].
attn_status_t check_cache(int B, int Hkv, int Lk, int D, int64_t kv_pitch, attn_dtype_t dtype) {
  if (B < 1 || Hkv < 1 || Lk < 1) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_DTYPE_FP16 && dtype != ATTN_DTYPE_BF16) return ATTN_ERR_INVALID_ARG;
  if (kv_pitch < 0 || (kv_pitch != 0 && kv_pitch < Lk)) return ATTN_ERR_INVALID_ARG;
  if (!supported_d(D)) return ATTN_ERR_UNSUPPORTED;
  // the TMA stride limit between heads (2^40 bytes), head counts that a grid takes
  if (kv_pitch > (int64_t{1} << 40) / (2 * D)) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Hkv > 65535) return ATTN_ERR_UNSUPPORTED;
  if (Lk > kCacheMaxLk) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

attn_status_t check_tree(int B, int Hq, int Hkv, int T, int Lk, int D) {
  if (Hq < 1 || T < 1) return ATTN_ERR_INVALID_ARG;
  const attn_status_t s = check_cache(B, Hkv, Lk, D, 0, ATTN_DTYPE_BF16);
  if (s == ATTN_ERR_INVALID_ARG) return s;
  if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (s != ATTN_OK) return s;
  if (T > kTreeMaxT || B > kTreeMaxB) return ATTN_ERR_UNSUPPORTED;
  // stages of the whole call, and the combine kernel's rows per KV head, are ints that a grid takes
  const long long stages = (Lk + 63) / 64 + (T + 63) / 64 + kTreeExtra;
  if (stages * B * Hkv > 0x7fff0000LL) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(Hq / Hkv) * T > 65535) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

attn_status_t check_key_weight(int B, int Hq, int Hkv, int Lq, int Lk, int D) {
  if (Hq < 1 || Lq < 1) return ATTN_ERR_INVALID_ARG;
  const attn_status_t s = check_cache(B, Hkv, Lk, D, 0, ATTN_DTYPE_BF16);
  if (s == ATTN_ERR_INVALID_ARG) return s;
  if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (s != ATTN_OK) return s;
  const long long rows = static_cast<long long>(Hq / Hkv) * Lq;
  if (rows > (1 << 30)) return ATTN_ERR_UNSUPPORTED;
  // the kernels count key tiles of 128, or steps of 256 keys x 64 rows (at
  // most G partly filled row tiles more), in 32 bits
  const long long heads = static_cast<long long>(B) * Hkv, row_tiles = rows / 64 + Hq / Hkv + 1;
  if (heads * ((Lk + 127) / 128) > 0x7fff0000LL) return ATTN_ERR_UNSUPPORTED;
  if (rows > kKeyWeightFewRows && heads * ((Lk + 255) / 256) > 0x7fff0000LL / row_tiles) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" size_t attn_tree_workspace_bytes(int B, int Hq, int Hkv, int T, int Lk, int D) {
  if (check_tree(B, Hq, Hkv, T, Lk, D) != ATTN_OK) return 0;
  const TreePlan t = tree_plan(static_cast<long long>(Hq / Hkv) * T, D, kTreeMaxCtas);
  return static_cast<size_t>(t.n_groups) * 2 * t.n_rb * t.rows * (D + 1) * sizeof(float);
}

extern "C" attn_status_t attn_fwd_tree(const void* q, const void* k, const void* v, const void* k_new,
                                       const void* v_new, const uint8_t* tree_mask, const int32_t* cache_len,
                                       const int32_t* tree_len, void* o, float* lse, void* workspace,
                                       size_t workspace_bytes, int64_t kv_pitch, int B, int Hq, int Hkv, int T,
                                       int Lk, int D, float scale, attn_dtype_t dtype, cudaStream_t stream) {
  if (!q || !k || !v || !k_new || !v_new || !cache_len || !o || !lse || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(o) ||
      !aligned16(lse) || !aligned16(workspace) || !aligned4(cache_len) || !aligned4(tree_len))
    return ATTN_ERR_INVALID_ARG;
  if (o == q) return ATTN_ERR_INVALID_ARG;
  attn_status_t s = check_scale(scale);
  if (s != ATTN_OK) return s;
  s = check_tree(B, Hq, Hkv, T, Lk, D);
  if (s == ATTN_ERR_INVALID_ARG) return s;
  const attn_status_t c = check_cache(B, Hkv, Lk, D, kv_pitch, dtype);
  if (c != ATTN_OK) return c;
  if (s != ATTN_OK) return s;
  if (workspace_bytes < attn_tree_workspace_bytes(B, Hq, Hkv, T, Lk, D)) return ATTN_ERR_INVALID_ARG;
  // several CTAs read a row of q, of the drafts, of the mask
  const long long rows = static_cast<long long>(B) * Hq * T, drafts = static_cast<long long>(B) * Hkv * T, ints = 4LL * B;
  const Span spans[] = {{o, rows * D * 2}, {lse, rows * 4}, {q, rows * D * 2}, {k_new, drafts * D * 2},
                        {v_new, drafts * D * 2}, {tree_mask, static_cast<long long>(B) * T * T}, {cache_len, ints},
                        {tree_len, ints}};
  if (outputs_overlap(spans, 2)) return ATTN_ERR_INVALID_ARG;
  int dev, num_sms, *status;
  EncodeTiledFn enc;
  const attn_status_t ds = call_state(stream, &dev, &enc, &status, &num_sms);
  if (ds != ATTN_OK) return ds;
  TreeParams p{};
  p.q = q, p.k = k, p.v = v, p.k_new = k_new, p.v_new = v_new;
  p.mask = tree_mask, p.cache_len = cache_len, p.tree_len = tree_len;
  p.o = o, p.lse = lse, p.part = static_cast<float*>(workspace);
  p.kv_pitch = kv_pitch ? kv_pitch : Lk;
  p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv, p.T = T, p.Lk = Lk;
  p.scale_log2 = scale_log2_of(scale), p.status = status, p.limit_ns = shared_wait_limit_ns();
  const bool bf16 = dtype == ATTN_DTYPE_BF16;
  switch (D) {
    case 64: return finish(launch_tree_d64(p, bf16, num_sms, enc, stream));
    case 96: return finish(launch_tree_d96(p, bf16, num_sms, enc, stream));
    case 128: return finish(launch_tree_d128(p, bf16, num_sms, enc, stream));
    default: return finish(launch_tree_d256(p, bf16, num_sms, enc, stream));
  }
}

extern "C" size_t attn_key_weight_workspace_bytes(int B, int Hq, int Hkv, int Lq, int Lk, int D) {
  if (check_key_weight(B, Hq, Hkv, Lq, Lk, D) != ATTN_OK) return 0;
  // two sets of partial sums per CTA where the rows do not fit shared memory together
  if (static_cast<long long>(Hq / Hkv) * Lq <= kKeyWeightFewRows) return 16;
  return static_cast<size_t>(kTreeMaxCtas) * 2 * 256 * sizeof(float);
}

extern "C" attn_status_t attn_key_weight(const void* q, const void* k, const float* lse, const int32_t* limit,
                                         const float* weight, float* weight_out, void* workspace,
                                         size_t workspace_bytes, int64_t kv_pitch, int B, int Hq, int Hkv, int Lq,
                                         int Lk, int D, float scale, int causal, attn_dtype_t dtype,
                                         cudaStream_t stream) {
  if (!q || !k || !lse || !weight_out || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(lse) || !aligned16(weight) || !aligned16(weight_out) ||
      !aligned16(workspace) || !aligned4(limit))
    return ATTN_ERR_INVALID_ARG;
  attn_status_t s = check_scale(scale);
  if (s != ATTN_OK) return s;
  s = check_key_weight(B, Hq, Hkv, Lq, Lk, D);
  if (s == ATTN_ERR_INVALID_ARG) return s;
  const attn_status_t c = check_cache(B, Hkv, Lk, D, kv_pitch, dtype);
  if (c == ATTN_ERR_INVALID_ARG) return c;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (causal && (limit || Lq > Lk)) return ATTN_ERR_INVALID_ARG;
  if (c != ATTN_OK) return c;
  if (s != ATTN_OK) return s;
  // every CTA reads all B x Lq limits before it starts (how far each sequence's
  // rows reach decides the division), and holds B sums
  if (limit && (Lq > kTreeMaxT || B > kTreeMaxB)) return ATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < attn_key_weight_workspace_bytes(B, Hq, Hkv, Lq, Lk, D)) return ATTN_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(B) * Hq * Lq, slots = 4LL * B * Hkv * Lk;
  const Span out = {weight_out, slots}, spans[] = {out, {q, rows * D * 2}, {lse, rows * 4}, {limit, 4LL * B * Lq}};
  if (outputs_overlap(spans, 1)) return ATTN_ERR_INVALID_ARG;
  // in place a thread reads an element before it writes it; a shifted array would be read after
  if (weight != weight_out && overlap(out, {weight, slots})) return ATTN_ERR_INVALID_ARG;
  int dev, num_sms, *status;
  EncodeTiledFn enc;
  const attn_status_t ds = call_state(stream, &dev, &enc, &status, &num_sms);
  if (ds != ATTN_OK) return ds;
  KeyWeightParams p{};
  p.q = q, p.k = k, p.lse = lse, p.limit = limit, p.weight = weight, p.weight_out = weight_out;
  p.part = static_cast<float*>(workspace);
  p.kv_pitch = kv_pitch ? kv_pitch : Lk;
  p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv, p.Lq = Lq, p.Lk = Lk, p.causal = causal;
  // a list per query head lets causal calls leave out the row tiles above the
  // diagonal; short or individually limited rows fill tiles better packed (B4
  // G4 Lq 48 over 8192 keys: 30.0 us packed, 51.5 as lists)
  p.packed = limit || Lq < 64;
  p.rows_per_step = key_weight_rows_per_step(D);
  p.scale_log2 = scale_log2_of(scale), p.status = status, p.limit_ns = shared_wait_limit_ns();
  const bool bf16 = dtype == ATTN_DTYPE_BF16;
  switch (D) {
    case 64: return finish(launch_key_weight_d64(p, bf16, num_sms, enc, stream));
    case 96: return finish(launch_key_weight_d96(p, bf16, num_sms, enc, stream));
    case 128: return finish(launch_key_weight_d128(p, bf16, num_sms, enc, stream));
    default: return finish(launch_key_weight_d256(p, bf16, num_sms, enc, stream));
  }
}

extern "C" attn_status_t attn_cache_append(const void* k_new, const void* v_new, const int32_t* path,
                                           const int32_t* accept_len, const int32_t* cache_len, const int32_t* seen,
                                           void* k, void* v, int32_t* pos, int32_t* cache_len_out, int32_t* seen_out,
                                           int32_t* limit, int64_t kv_pitch, int B, int Hkv, int T, int Lk, int D,
                                           attn_dtype_t dtype, cudaStream_t stream) {
  if (!k_new || !v_new || !cache_len || !k || !v || !cache_len_out) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k) || !aligned16(v) || !aligned4(path) ||
      !aligned4(accept_len) || !aligned4(cache_len) || !aligned4(seen) || !aligned4(pos) || !aligned4(cache_len_out) ||
      !aligned4(seen_out) || !aligned4(limit))
    return ATTN_ERR_INVALID_ARG;
  if ((pos || seen_out) && !seen) return ATTN_ERR_INVALID_ARG;
  if (cache_len_out == cache_len || (seen_out && seen_out == seen)) return ATTN_ERR_INVALID_ARG;
  if (T < 1) return ATTN_ERR_INVALID_ARG;
  const attn_status_t s = check_cache(B, Hkv, Lk, D, kv_pitch, dtype);
  if (s != ATTN_OK) return s;
  if (path && T > kTreeMaxT) return ATTN_ERR_UNSUPPORTED;
  const long long ints = 4LL * B;
  const Span spans[] = {{cache_len_out, ints}, {seen_out, ints}, {limit, ints * T}, {pos, ints * Hkv * Lk}, {cache_len, ints},
                        {seen, ints}, {accept_len, ints}, {path, ints * T}};
  if (outputs_overlap(spans, 4)) return ATTN_ERR_INVALID_ARG;
  int dev, num_sms, *status;
  EncodeTiledFn enc;
  const attn_status_t ds = call_state(stream, &dev, &enc, &status, &num_sms);
  if (ds != ATTN_OK) return ds;
  AppendParams p{k_new, v_new, path, accept_len, cache_len, seen, k, v, pos, cache_len_out, seen_out, limit,
                 kv_pitch ? kv_pitch : Lk, B, Hkv, T, Lk, D / 8, status};
  const long long pieces = (static_cast<long long>(T) * p.row16 + kAppendThreads - 1) / kAppendThreads;
  const int gx = static_cast<int>(pieces < 64 ? pieces : 64);
  return finish(launch_dependent(attn_cache_append_kernel, dim3(gx, B * Hkv), kAppendThreads, 0, stream, p));
}

extern "C" size_t attn_cache_evict_workspace_bytes(int B, int Hkv, int Lk) {
  if (B < 1 || Hkv < 1 || Lk < 1 || static_cast<long long>(B) * Hkv > 65535 || Lk > kEvictMaxLk) return 0;
  // per KV head: two lists of at most Lk / 2 slots and their length
  return round16(static_cast<size_t>(B) * Hkv * ((Lk / 2) * 2 + 1) * sizeof(int32_t));
}

extern "C" attn_status_t attn_cache_evict(void* k, void* v, const float* weight, const int32_t* pos,
                                          const int32_t* cache_len, const int32_t* seen, float* weight_out,
                                          int32_t* pos_out, int32_t* cache_len_out, void* workspace,
                                          size_t workspace_bytes, int64_t kv_pitch, int B, int Hkv, int Lk, int D,
                                          int keep, int recent, attn_dtype_t dtype, cudaStream_t stream) {
  if (!k || !v || !weight || !pos || !cache_len || !seen || !weight_out || !pos_out || !cache_len_out || !workspace)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(weight) || !aligned16(pos) || !aligned16(weight_out) ||
      !aligned16(pos_out) || !aligned16(workspace) || !aligned4(cache_len) || !aligned4(seen) ||
      !aligned4(cache_len_out))
    return ATTN_ERR_INVALID_ARG;
  if (weight_out == weight || pos_out == pos || cache_len_out == cache_len) return ATTN_ERR_INVALID_ARG;
  const attn_status_t s = check_cache(B, Hkv, Lk, D, kv_pitch, dtype);
  if (s == ATTN_ERR_INVALID_ARG) return s;
  if (keep < 1 || keep > Lk || recent < 0 || recent > keep) return ATTN_ERR_INVALID_ARG;
  if (s != ATTN_OK) return s;
  if (Lk > kEvictMaxLk) return ATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < attn_cache_evict_workspace_bytes(B, Hkv, Lk)) return ATTN_ERR_INVALID_ARG;
  // CTAs that share a KV head read the same weights, positions and lengths and have to choose the same slots
  const long long ints = 4LL * B, slots = ints * Hkv * Lk;
  const Span spans[] = {{weight_out, slots}, {pos_out, slots}, {cache_len_out, ints}, {weight, slots}, {pos, slots},
                        {cache_len, ints}, {seen, ints}};
  if (outputs_overlap(spans, 3)) return ATTN_ERR_INVALID_ARG;
  int dev, num_sms, *status;
  EncodeTiledFn enc;
  const attn_status_t ds = call_state(stream, &dev, &enc, &status, &num_sms);
  if (ds != ATTN_OK) return ds;
  EvictParams p{k, v, weight, pos, cache_len, seen, weight_out, pos_out, cache_len_out,
                static_cast<int32_t*>(workspace),
                static_cast<int32_t*>(workspace) + static_cast<size_t>(B) * Hkv * (Lk / 2) * 2,
                kv_pitch ? kv_pitch : Lk, B, Hkv, Lk, D / 8, keep, recent, status};
  const int heads = B * Hkv;
  if (Lk <= kEvictRowKeys) {
    // about one CTA per SM, so that the moves run at the memory's rate (4 x 8
    // heads 8448 -> 8192: 11.3 us, by clusters 15.6; 16384 -> 8192: 37.9 and 40.1,
    // -> 16128: 15.2 and 16.2; 2 heads 8448 -> 8192: 9.7 and 12.2, 16384 -> 8192:
    // 13.7 and 13.3, -> 16128: 12.0 and 12.5, so the number of heads is left out of
    // the rule; past 16384 one CTA's search takes too long: 8 heads of 32768 55 us,
    // by clusters 20)
    const int copies = heads < num_sms ? num_sms / heads : 1;
    static std::atomic<uint64_t> done{0};
    if (!set_smem_limit(attn_cache_evict_kernel, evict_smem(kEvictRowKeys, 1), done)) return ATTN_ERR_CUDA;
    return finish(launch_dependent(attn_cache_evict_kernel, dim3(heads * copies), kEvictThreads,
                                   evict_smem(Lk, copies), stream, p, copies));
  }
  // a CTA's part of the slots: every warp's share is a multiple of 32
  constexpr int nc = kEvictCluster, warps = kEvictClusterThreads / 32;
  const long long part = static_cast<long long>((((Lk + nc * warps - 1) / (nc * warps)) + 31) & ~31) * warps;
  const bool cached = part <= kEvictKeys;
  auto kern = cached ? attn_cache_evict_cluster_kernel<true> : attn_cache_evict_cluster_kernel<false>;
  const size_t smem = cached ? static_cast<size_t>(part) * 4 : 0;
  static std::atomic<uint64_t> done[2] = {};
  if (!set_smem_limit(kern, kEvictKeys * 4, done[cached])) return ATTN_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(heads) * nc);
  cfg.blockDim = dim3(kEvictClusterThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return ATTN_ERR_CUDA;
  const int blocks = 4 * num_sms / heads;
  return finish(launch_dependent(attn_cache_move_kernel, dim3(blocks > 1 ? blocks : 1, heads), 256, 0, stream, p));
}
