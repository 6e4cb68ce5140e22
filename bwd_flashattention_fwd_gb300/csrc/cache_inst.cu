// Instantiations and launchers of the cache kernels for one head dimension
// (compiled once per supported D with -DGBATTN_HEAD_DIM=<D>, like inst.cu).
#include "cache.h"
#include "key_weight_kernel.cuh"
#include "tree_kernel.cuh"

#ifndef GBATTN_HEAD_DIM
#error "compile with -DGBATTN_HEAD_DIM=<64|96|128|256>"
#endif

#define GBATTN_CAT2(a, b) a##b
#define GBATTN_CAT(a, b) GBATTN_CAT2(a, b)

namespace gbattn {
namespace GBATTN_CAT(cache_d, GBATTN_HEAD_DIM) {

constexpr int kD = GBATTN_HEAD_DIM;

// Rank-3 view [heads, L, D] with `pitch` rows between heads; boxes of 64
// columns x box_rows rows with the 128-byte swizzle.  Rows past L and columns
// past D read as zeros.
bool make_map(EncodeTiledFn enc, bool bf16, CUtensorMap* m, const void* base, long long L, long long heads,
              int box_rows, long long pitch) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(L),
                              static_cast<cuuint64_t>(heads)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kD) * 2,
                                 static_cast<cuuint64_t>(kD) * 2 * static_cast<cuuint64_t>(pitch)};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_rows), 1u};
  const cuuint32_t elem_strides[3] = {1u, 1u, 1u};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF16, int QS, int NT>
int tree_impl(const TreeParams& p, EncodeTiledFn enc, cudaStream_t stream) {
  using Gm = TreeGeom<kD, QS, NT>;
  const long long R = static_cast<long long>(p.G) * p.T, heads = static_cast<long long>(p.B) * p.Hkv;
  CUtensorMap tq, tk, tv, tkn, tvn;
  if (!make_map(enc, BF16, &tq, p.q, R, heads, Gm::QROWS, R) ||
      !make_map(enc, BF16, &tk, p.k, p.Lk, heads, Gm::BK, p.kv_pitch) ||
      !make_map(enc, BF16, &tv, p.v, p.Lk, heads, Gm::BK, p.kv_pitch) ||
      !make_map(enc, BF16, &tkn, p.k_new, p.T, heads, Gm::BK, p.T) ||
      !make_map(enc, BF16, &tvn, p.v_new, p.T, heads, Gm::BK, p.T))
    return kLaunchBadMap;
  auto kern = attn_tree_kernel<kD, BF16, QS, NT>;
  static std::atomic<uint64_t> done{0};
  if (!set_smem_limit(kern, Gm::SMEM_BYTES, done)) return kLaunchCudaError;
  const int r = launch_dependent(kern, dim3(p.n_groups * p.n_rb), Gm::NUM_THREADS,
                                 Gm::SMEM_BYTES, stream, tq, tk, tv, tkn, tvn, p);
  if (r != kLaunchOk) return r;
  if (p.n_groups == 1 || p.whole) return kLaunchOk;  // no KV head is shared
  // Warps that share a head's partials out by how many it has on average (131072
  // keys D = 256, 38 partials: 84.6 us with 8, 92.4 with one; B1 T8 1000 keys, 17:
  // 9.8 and 16.0), and column quads per thread, which are the loads in flight
  // (B16 T61 ragged: 70.7 us with 2, 76.4 with one; B6 T26 ragged, 12 partials: 27.3
  // with 4, 31.6 with one; B2 T27 1219 keys D = 96: 11.6 and 14.0)
  const long long avg = p.n_groups / heads + 1;
  // blocks walk the tasks: those that few warps share in more blocks (B16 T61 with
  // 3 per SM 74.5 us), those with barriers in fewer (61 x 8 rows 60000 keys with 8 per SM 82.3, 80.8 with 3)
  auto combine = [&](auto kern_c, int cols_per_block, int blocks_per_sm) {
    const long long tasks = heads * ((R + 31) / 32) * (kD / cols_per_block);
    const long long most = static_cast<long long>(blocks_per_sm) * kTreeMaxCtas;
    return launch_dependent(kern_c, dim3(static_cast<unsigned>(tasks < most ? tasks : most)), 256, 0, stream, p,
                            static_cast<int>(Gm::ROWS));
  };
  constexpr int QT = kD == 96 ? 3 : 2;
  if (avg > 8) return combine(attn_tree_combine_kernel<kD, BF16, 8, 4>, 16, 3);
  if (avg > 3) return combine(attn_tree_combine_kernel<kD, BF16, 2, 2>, 32, 3);
  return combine(attn_tree_combine_kernel<kD, BF16, 1, QT>, 32 * QT, 8);
}

template <bool BF16>
int tree_dispatch(const TreeParams& p, const TreePlan& plan, EncodeTiledFn enc, cudaStream_t stream) {
  if constexpr (kD <= 96) {
    if (plan.qs == 2) return tree_impl<BF16, 2, 1>(p, enc, stream);
  }
  if constexpr (kD <= 128) {
    if (plan.qs == 4) return tree_impl<BF16, 4, 1>(p, enc, stream);
    if (plan.nt == 2) return tree_impl<BF16, 1, 2>(p, enc, stream);
  }
  return tree_impl<BF16, 1, 1>(p, enc, stream);
}

template <bool BF16, int NQ>
int key_weight_few(const KeyWeightParams& p, int num_sms, EncodeTiledFn enc, cudaStream_t stream) {
  using Gm = KeyWeightFewGeom<kD, NQ>;
  const long long R = static_cast<long long>(p.G) * p.Lq, heads = static_cast<long long>(p.B) * p.Hkv;
  CUtensorMap tq, tk;
  if (!make_map(enc, BF16, &tq, p.q, R, heads, NQ, R) || !make_map(enc, BF16, &tk, p.k, p.Lk, heads, Gm::BK, p.kv_pitch))
    return kLaunchBadMap;
  const long long tiles = heads * ((p.Lk + Gm::BK - 1) / Gm::BK);
  auto kern = attn_key_weight_few_kernel<kD, BF16, NQ>;
  static std::atomic<uint64_t> done{0};
  if (!set_smem_limit(kern, Gm::SMEM_BYTES, done)) return kLaunchCudaError;
  return launch_dependent(kern, dim3(static_cast<unsigned>(tiles < num_sms ? tiles : num_sms)), Gm::NUM_THREADS,
                          Gm::SMEM_BYTES, stream, tq, tk, p);
}

template <bool BF16>
int key_weight_many(const KeyWeightParams& p, int num_sms, EncodeTiledFn enc, cudaStream_t stream) {
  using Gm = KeyWeightGeom<kD>;
  const long long heads = static_cast<long long>(p.B) * p.Hkv;
  const long long rows = p.packed ? static_cast<long long>(p.G) * p.Lq : p.Lq;
  CUtensorMap tq, tk;
  if (!make_map(enc, BF16, &tq, p.q, rows, p.packed ? heads : heads * p.G, Gm::NQ, rows) ||
      !make_map(enc, BF16, &tk, p.k, p.Lk, heads, 128, p.kv_pitch))
    return kLaunchBadMap;
  const int groups = num_sms < kTreeMaxCtas ? num_sms : kTreeMaxCtas;
  auto kern = attn_key_weight_kernel<kD, BF16>;
  static std::atomic<uint64_t> done{0};
  if (!set_smem_limit(kern, Gm::SMEM_BYTES, done)) return kLaunchCudaError;
  const int r = launch_dependent(kern, dim3(groups), Gm::NUM_THREADS, Gm::SMEM_BYTES, stream, tq, tk, p);
  if (r != kLaunchOk) return r;
  const long long tiles = heads * ((p.Lk + Gm::BK - 1) / Gm::BK), most = 4LL * kTreeMaxCtas;
  return launch_dependent(attn_key_weight_join_kernel, dim3(static_cast<unsigned>(tiles < most ? tiles : most)), 256, 0,
                          stream, p, groups);
}

template <bool BF16>
int key_weight_dispatch(const KeyWeightParams& p, int num_sms, EncodeTiledFn enc, cudaStream_t stream) {
  const long long R = static_cast<long long>(p.G) * p.Lq;
  // the smallest tile that holds the rows: 32 rows over 4 x 8192 keys 15.9 us, in
  // a 128-row tile 16.9; 128 rows 19.7, by the kernel for many rows 31.7
  if (R <= 16) return key_weight_few<BF16, 16>(p, num_sms, enc, stream);
  if (R <= 32) return key_weight_few<BF16, 32>(p, num_sms, enc, stream);
  if (R <= 64) return key_weight_few<BF16, 64>(p, num_sms, enc, stream);
  if (R <= kKeyWeightFewRows) return key_weight_few<BF16, 128>(p, num_sms, enc, stream);
  return key_weight_many<BF16>(p, num_sms, enc, stream);
}

}  // namespace GBATTN_CAT(cache_d, GBATTN_HEAD_DIM)

using namespace GBATTN_CAT(cache_d, GBATTN_HEAD_DIM);

int GBATTN_CAT(launch_tree_d, GBATTN_HEAD_DIM)(const TreeParams& p0, bool bf16, int num_sms, EncodeTiledFn enc,
                                               cudaStream_t stream) {
  const TreePlan plan = tree_plan(static_cast<long long>(p0.G) * p0.T, kD, num_sms);
  TreeParams p = p0;
  p.stage = plan.stage, p.n_rb = plan.n_rb, p.n_groups = plan.n_groups;
  p.part_lse = p.part + static_cast<size_t>(plan.n_groups) * 2 * plan.n_rb * plan.rows * kD;
  const long long heads = static_cast<long long>(p.B) * p.Hkv, each = (heads + p.n_groups - 1) / p.n_groups;
  const long long stages = (p.Lk + p.stage - 1) / p.stage + (p.T + p.stage - 1) / p.stage;
  if (each * stages <= kTreeWholeMost && (each * p.n_groups - heads) * stages <= kTreeWholeMore * p.n_groups) {
    p.whole = static_cast<int>(each);
    p.n_groups = static_cast<int>((heads + each - 1) / each);
  }
  return bf16 ? tree_dispatch<true>(p, plan, enc, stream) : tree_dispatch<false>(p, plan, enc, stream);
}

int GBATTN_CAT(launch_key_weight_d, GBATTN_HEAD_DIM)(const KeyWeightParams& p, bool bf16, int num_sms,
                                                     EncodeTiledFn enc, cudaStream_t stream) {
  return bf16 ? key_weight_dispatch<true>(p, num_sms, enc, stream) : key_weight_dispatch<false>(p, num_sms, enc, stream);
}

}  // namespace gbattn
