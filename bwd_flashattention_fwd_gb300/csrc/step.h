// Host-side interface between the C ABI of the calls around attention in a
// model step (step.cu) and their kernels: norm and rotation of queries and
// keys, the paged cache, verification of drafts.
#pragma once

#include "cache.h"

namespace gbattn {

// A [B, H, L, D] tensor with D contiguous; strides in elements.
struct RowsView {
  void* at;
  int64_t sb, sh, sl;
  int H;
};

constexpr int kRopeThreads = 256;
constexpr int kRopeFwdPerSm = 3, kRopeBwdPerSm = 2;  // CTAs of rope_kernel on an SM
constexpr int kRopeMaxAxes = 8;

struct RopeParams {
  RowsView x[2];         // q and k as they come (dx of the backward pass goes to dx)
  RowsView dx[2];
  void* y[2];            // forward: rotated q and k; backward: their gradients (contiguous)
  const void* w[2];      // norm weights [D], both or neither
  float* dw[2];          // their gradients
  float* part;           // backward: [CTAs][2][D] partial sums of dw
  const int32_t* pos;    // [axes][B][L]
  const float* freq;     // [rot / 2]
  const uint8_t* axis;   // [rot / 2] or null
  int B, L, D, rot, axes;
  float eps;
  int* status;
};

constexpr int kPagedMaxB = 1024;        // sequences (each CTA holds the lengths' prefix sums in shared memory)
constexpr int kPagedMaxRows = 128;      // G * T
constexpr int kPagedMaxTokens = 1 << 30;  // a sequence's room (token numbers are ints)
constexpr int kPagedMaxCtas = 3 * kTreeMaxCtas;
constexpr int kPagedCluster = 8;  // CTAs that share a head of a short cache, at most
// A quantised row's exponent.  (The largest is what bf16's values need; below the least lie 2^-73 and less.)
constexpr int kExpMin = -64, kExpMax = 120;

// The cache: pages [n_pages][Hkv][2^shift][D], 16-bit or e4m3 with an exponent per row.
struct PagedCache {
  void *k, *v;
  int8_t *k_exp, *v_exp;       // [n_pages][Hkv][2^shift], or null (16-bit)
  const int32_t* table;        // [B][per_seq]
  int n_pages, shift, per_seq, Hkv, D;
};

struct PagedWriteParams {
  PagedCache c;
  const void *k_new, *v_new;  // [B][Hkv][T][D]
  const int32_t *cache_len, *new_len;
  int32_t* cache_len_out;
  int B, T;
  int* status;
};

struct PagedReadParams {
  PagedCache c;
  const int32_t* cache_len;
  void *k, *v;  // [B][Hkv][Lk (pitch)][D]
  int64_t pitch;
  int B, Lk;
  int* status;
};

struct PagedAttnParams {
  PagedCache c;
  const void* q;
  const int32_t* cache_len;
  void* o;
  float* lse;
  int B, Hq, G, T, R;  // R = G * T rows of a KV head
  int n_rb, n_groups;  // blocks of rows, CTAs that share the keys out
  float scale_log2;
  float* part;     // [n_groups][2][rows][D]
  float* part_ml;  // [n_groups][2][rows][2]
  int* status;
};

// Rows that a CTA of the paged attention works on: 8, 16 or 32 (D = 256: 16 at most; the accumulators are registers).
inline int paged_rows(int R, int D) { return R <= 8 ? 8 : R <= 16 || D == 256 ? 16 : 32; }

struct VerifyParams {
  const float *target, *draft;  // [B][T + 1][V], [B][T][V] or null
  const int32_t* tokens;        // [B][T]
  const float *u, *r;           // [B][T], [B]
  const int32_t* draft_len;     // [B] or null
  int32_t *accept_len, *token;
  int B, T, V;
  int* status;
};


#define GBATTN_DECLARE_PAGED_LAUNCHERS(DIM) \
  int launch_paged_d##DIM(const PagedAttnParams& p, bool bf16, int num_sms, cudaStream_t stream);

GBATTN_DECLARE_PAGED_LAUNCHERS(64)
GBATTN_DECLARE_PAGED_LAUNCHERS(96)
GBATTN_DECLARE_PAGED_LAUNCHERS(128)
GBATTN_DECLARE_PAGED_LAUNCHERS(256)

#undef GBATTN_DECLARE_PAGED_LAUNCHERS

}  // namespace gbattn
