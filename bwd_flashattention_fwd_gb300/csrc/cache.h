// Host-side interface between the C ABI of the cache calls (cache.cu) and
// their kernels.
#pragma once

#include <atomic>

#include "launch.h"

namespace gbattn {

constexpr int kTreeMaxT = 1024;   // drafts per sequence (the mask is T x T bytes per sequence)
constexpr int kTreeMaxB = 1024;   // sequences (each CTA holds the lengths' prefix sums in shared memory)
// Keys per pipeline stage.  64 keys of K and V at D = 64 arrive in 0.37 us, less
// than a stage's chain of S, softmax and P V takes, so small heads take 128
// (16384 keys D = 64: B8 T8 50.7 us, with 64 keys 67.1; T30 58.9 and 72.4).
constexpr int tree_stage_keys(int D, int nt) { return D <= 96 && nt == 1 ? 128 : 64; }
// What a CTA spends on a KV head besides its stages, in stages (B16 T61 ragged
// 70.4 us, with 4 72.5, 10 70.7, 14 70.9).
constexpr int kTreeExtra = 7;
// Small caches: KV heads are not divided, which saves the partials and the
// second launch, where a CTA's stages are at most kTreeWholeMost and at most
// kTreeWholeMore above an even share.  B2 T47 200 keys D = 64 (5 stages) 10.1
// us, divided 12.7; B24 T4 400 keys D = 128 (2 heads of 8 stages) 18.3 and
// 19.4; B18 T8 1400 keys (24 stages) 22.5 and 27.9; B1 T8 400 keys (8 stages) 9.9
// and 9.1 on the device, but one launch for the host instead of two (10.9 us a
// call and 13.7).  Beyond the rule: B1 T8 700 keys (12 stages) 11.6, divided 9.5;
// B4 T1 1000 keys D = 256 20.0 and 10.8; the other way round B8 T8 1000 keys, 64
// heads of 17 stages on 152 CTAs: 15.4 and 18.4.
constexpr int kTreeWholeMost = 24, kTreeWholeMore = 8;
constexpr int kTreeMaxCtas = 152;  // one per SM of a GB300
constexpr int kCacheMaxLk = 1 << 30;  // rows of a KV head (row numbers are ints)
constexpr int kEvictMaxLk = 1 << 20;
constexpr int kEvictCluster = 8;      // CTAs per KV head beyond that
constexpr int kEvictRowKeys = 16384;  // slots up to which one CTA holds a KV head's keys in shared memory

struct TreeParams {
  const void *q, *k, *v, *k_new, *v_new;
  const uint8_t* mask;       // [B][T][T] or null (chain)
  const int32_t* cache_len;  // [B]
  const int32_t* tree_len;   // [B] or null
  void* o;
  float* lse;
  int64_t kv_pitch;
  int B, Hq, Hkv, G, T, Lk;
  float scale_log2;
  int* status;
  uint64_t limit_ns;
  // division of the work (tree_plan) and the partials of KV heads that several CTAs share
  int stage, n_rb, n_groups;
  int whole;        // > 0: KV heads per group, undivided; no partials, no combine
  float* part;      // [n_groups][2][n_rb][rows][D]
  float* part_lse;  // [n_groups][2][n_rb][rows]
};

// How the packed rows of a KV head (R = G * T) are laid out over CTAs: rows
// per CTA, row blocks, and groups of n_rb CTAs that share out the keys.
struct TreePlan {
  int qs, nt, rows, stage, n_rb, n_groups;
};

// R <= 32 / 64: the rows sit in four / two lane quadrants that share the keys
// out, where that pays: B8 T8 16384 keys D = 64, 32 rows, 50.7 us against 58.1
// with one full tile; B4 T8 8192 keys D = 128 29.9 and 30.1; 64 rows at D = 128
// 31.9 against 31.3, and D = 256 (8 rows, 131072 keys) 86.2 against 85.6, so
// those take the full tile.
// Above 128 rows: 256 rows per CTA where two accumulators fit tensor memory
// (D <= 128): B16 T61 ragged 70.3 us, with 128 rows per CTA 83.1.
inline TreePlan tree_plan(long long R, int D, int num_sms) {
  TreePlan t;
  t.qs = R <= 32 && D <= 128 ? 4 : R <= 64 && D <= 96 ? 2 : 1;
  t.nt = R > 128 && D <= 128 ? 2 : 1;
  t.stage = tree_stage_keys(D, t.nt);
  t.rows = t.qs > 1 ? 128 / t.qs : 128 * t.nt;
  t.n_rb = static_cast<int>((R + t.rows - 1) / t.rows);
  const int ctas = num_sms < kTreeMaxCtas ? num_sms : kTreeMaxCtas;
  t.n_groups = ctas / t.n_rb > 1 ? ctas / t.n_rb : 1;
  return t;
}

struct KeyWeightParams {
  const void *q, *k;
  const float* lse;
  const int32_t* limit;  // [B][Lq] or null
  const float* weight;   // or null
  float* weight_out;
  int64_t kv_pitch;
  int B, Hq, Hkv, G, Lq, Lk;
  int causal;
  float scale_log2;
  int* status;
  uint64_t limit_ns;
  int rows_per_step;  // many rows: Q rows per step
  int packed;   // many rows: the G x Lq rows of a KV head form one list (else a list per query head)
  float* part;  // many rows: [CTAs][2][256] partial sums
};

// Q rows per step of the kernel for many rows: what tensor memory holds beside K of 256 keys.
__host__ __device__ constexpr int key_weight_rows_per_step(int D) { return D <= 128 ? 128 : 64; }

// G * Lq rows up to which a KV head's rows stay in shared memory together.
constexpr int kKeyWeightFewRows = 128;

struct AppendParams {
  const void *k_new, *v_new;
  const int32_t *path, *accept_len, *cache_len, *seen;
  void *k, *v;
  int32_t *pos, *cache_len_out, *seen_out, *limit;
  int64_t kv_pitch;
  int B, Hkv, T, Lk, row16;  // row16: 16-byte pieces of a row
  int* status;
};

struct EvictParams {
  void *k, *v;
  const float* weight;
  const int32_t *pos, *cache_len, *seen;
  float* weight_out;
  int32_t *pos_out, *cache_len_out;
  int32_t* lists;   // [B * Hkv][2][Lk / 2]: freed slots, then the kept slots that move into them
  int32_t* counts;  // [B * Hkv]: how many
  int64_t kv_pitch;
  int B, Hkv, Lk, row16, keep, recent;
  int* status;
};

// Launchers of one head dimension (cache_inst.cu); LaunchResult codes.
#define GBATTN_DECLARE_CACHE_LAUNCHERS(DIM)                                                                   \
  int launch_tree_d##DIM(const TreeParams& p, bool bf16, int num_sms, EncodeTiledFn enc, cudaStream_t stream);      \
  int launch_key_weight_d##DIM(const KeyWeightParams& p, bool bf16, int num_sms, EncodeTiledFn enc, cudaStream_t stream);

GBATTN_DECLARE_CACHE_LAUNCHERS(64)
GBATTN_DECLARE_CACHE_LAUNCHERS(96)
GBATTN_DECLARE_CACHE_LAUNCHERS(128)
GBATTN_DECLARE_CACHE_LAUNCHERS(256)

#undef GBATTN_DECLARE_CACHE_LAUNCHERS

// A kernel's shared-memory limit, once per device: `done` is that kernel's own record.
template <typename Kern>
bool set_smem_limit(Kern kern, size_t smem, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return false;
  done.fetch_or(bit, std::memory_order_release);
  return true;
}

// Launch as a programmatic dependent of the kernel before it on the stream:
// its CTAs may start (and set up) while that kernel finishes.  A call's first
// kernel waits for it (griddepcontrol.wait) before it reads or writes global
// memory or allocates tensor memory, and lets its own dependents start behind
// that; a second kernel reads nothing but lengths before its wait.  So stream
// order holds for the caller.
template <typename... Params, typename... Args>
int launch_dependent(void (*kern)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return kLaunchCudaError;
  return cudaPeekAtLastError() == cudaSuccess ? kLaunchOk : kLaunchCudaError;
}

}  // namespace gbattn
