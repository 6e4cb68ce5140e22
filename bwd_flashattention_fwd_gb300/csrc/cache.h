// Host-side interface between the C ABI of the cache calls (cache.cu) and
// their kernels.
#pragma once

#include "launch.h"

namespace gbattn {

constexpr int kTreeMaxT = 1024;   // drafts per sequence (the mask is T x T bytes per sequence)
constexpr int kTreeMaxB = 1024;   // sequences (each CTA holds the lengths' prefix sums in shared memory)
constexpr int kEvictMaxLk = 1 << 20;

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
};

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
};

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
  int32_t* lists;  // [B * Hkv][2][Lk / 2]: freed slots, then the kept slots that move into them
  int64_t kv_pitch;
  int B, Hkv, Lk, row16, keep, recent;
  int* status;
};

}  // namespace gbattn
