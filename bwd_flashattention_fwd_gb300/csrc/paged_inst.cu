// Instantiations and launchers of the paged attention for one head dimension
// (compiled once per supported D with -DGBATTN_HEAD_DIM=<D>, like inst.cu).
#include "paged_attn_kernel.cuh"

#ifndef GBATTN_HEAD_DIM
#error "compile with -DGBATTN_HEAD_DIM=<64|96|128|256>"
#endif

#define GBATTN_CAT2(a, b) a##b
#define GBATTN_CAT(a, b) GBATTN_CAT2(a, b)

namespace gbattn {
namespace GBATTN_CAT(paged_d, GBATTN_HEAD_DIM) {

constexpr int kD = GBATTN_HEAD_DIM;

// A cluster of CTAs per head, in one launch, or equal pieces and a second one.
// A cluster saves the join, but its CTAs get what their head has.  A step alone
// takes kPagedAlone us; where clusters fill the GPU, their steps take what the
// memory gives (6.6 TB/s), with rooms half full on average half as long.  A
// cluster is taken where the longest possible sequence would so be late by
// kPagedLate us at most (32 heads of 8192 keys 25.9 us, by pieces 27.4, quantised 16.4 and 19.0; 1000 keys
// of one sequence 5.4 and 6.0, 4000 keys 8.7 and 8.3; D = 64, 128 heads of 250 to
// 2000 keys 13.3 and 13.1, of 125 to 1000 7.5 and 8.3; 1024 to 8192 keys quantised 28.2 and 22.6).
// The longest possible sequence is the table's room: 1000 keys in room for 32768 go by pieces, 5.9 us for 5.2.
// Past kPagedShort steps a single long sequence among short ones would be waited for too long.
constexpr int kPagedShort = 32;
constexpr float kPagedLate = 3.f;
template <bool Q8>
constexpr float kPagedAlone = Q8 ? 0.9f : 0.7f;

template <typename... Params, typename... Args>
int launch_cluster(void (*kern)(Params...), unsigned grid, int size, int threads, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? kLaunchOk : kLaunchCudaError;
}

template <bool BF16, bool Q8, int NT>
int impl(const PagedAttnParams& p0, int num_sms, cudaStream_t stream) {
  using Gm = PagedGeom<kD, Q8, NT>;
  PagedAttnParams p = p0;
  constexpr int rows = 8 * NT;
  p.n_rb = (p.R + rows - 1) / rows;
  const int smem = Gm::SMEM + (2 * p.B + 1) * 4;
  // CTAs per SM: shared memory (1 KB more each, 228 KB in all) and static arrays
  constexpr int fixed = 1024 + 256 + Gm::NW * (rows * 8 + Gm::ST * 4) + rows * 12;
  int per_sm = Gm::PER_SM;
  while (per_sm > 1 && per_sm * (smem + fixed) > 233472) --per_sm;
  p.n_groups = per_sm * (num_sms < kTreeMaxCtas ? num_sms : kTreeMaxCtas);
  const long long all = static_cast<long long>(p.B) * p.c.Hkv * p.n_rb, room = static_cast<long long>(p.c.per_seq) << p.c.shift;
  const long long steps = (room + Gm::KS - 1) / Gm::KS;
  int size = 1;
  while (size < kPagedCluster && 2 * size * all <= p.n_groups && size < steps) size *= 2;
  const long long per = (steps + size - 1) / size;
  const float half_full = static_cast<float>(size * all) * Gm::KS * Gm::ROWB / 6.6e6f;  // us of a step
  if (per <= kPagedShort && per * (kPagedAlone<Q8> - half_full) <= kPagedLate) {
    auto kern = attn_paged_cluster_kernel<kD, BF16, Q8, NT>;
    static std::atomic<uint64_t> done{0};
    if (!set_smem_limit(kern, Gm::SMEM, done)) return kLaunchCudaError;
    return launch_cluster(kern, static_cast<unsigned>(all) * size, size, Gm::THREADS, Gm::SMEM, stream, p, size);
  }
  p.part_ml = p.part + static_cast<size_t>(kPagedMaxCtas) * 2 * rows * kD;
  auto kern = attn_paged_kernel<kD, BF16, Q8, NT>;
  static std::atomic<uint64_t> done{0};
  if (!set_smem_limit(kern, Gm::SMEM + (2 * kPagedMaxB + 1) * 4, done)) return kLaunchCudaError;
  const int r = launch_dependent(kern, dim3(p.n_groups), Gm::THREADS, smem, stream, p);
  if (r != kLaunchOk || p.n_groups == 1) return r;
  // a block's warps share a row's partial results where there are many, and few rows: past two blocks on an SM a warp
  // per row is faster (7 x 8 heads of 8943 quantised keys, D = 96, 12 rows: 30.6 us, 35.4)
  const long long tasks = static_cast<long long>(p.B) * p.c.Hkv * p.R;
  auto join = [&](auto kern_j, int per) {
    const long long blocks = (tasks + per - 1) / per, most = 8LL * kTreeMaxCtas;
    return launch_dependent(kern_j, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), kPagedJoinThreads, 0, stream, p);
  };
  if (p.n_groups > (tasks <= 2LL * num_sms ? 8 : 32) * all) return join(attn_paged_join_kernel<kD, BF16, Q8, NT, 8>, 1);
  return join(attn_paged_join_kernel<kD, BF16, Q8, NT, 1>, kPagedJoinThreads / 32);
}

template <bool BF16, bool Q8>
int by_rows(const PagedAttnParams& p, int num_sms, cudaStream_t stream) {
  const int rows = paged_rows(p.R, kD);
  if (rows == 8) return impl<BF16, Q8, 1>(p, num_sms, stream);
  if constexpr (kD <= 128) {
    if (rows == 32) return impl<BF16, Q8, 4>(p, num_sms, stream);
  }
  return impl<BF16, Q8, 2>(p, num_sms, stream);
}

}  // namespace GBATTN_CAT(paged_d, GBATTN_HEAD_DIM)

using namespace GBATTN_CAT(paged_d, GBATTN_HEAD_DIM);

int GBATTN_CAT(launch_paged_d, GBATTN_HEAD_DIM)(const PagedAttnParams& p, bool bf16, int num_sms, cudaStream_t stream) {
  if (p.c.k_exp) return bf16 ? by_rows<true, true>(p, num_sms, stream) : by_rows<false, true>(p, num_sms, stream);
  return bf16 ? by_rows<true, false>(p, num_sms, stream) : by_rows<false, false>(p, num_sms, stream);
}

}  // namespace gbattn
