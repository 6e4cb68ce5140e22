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

template <bool BF16, bool Q8, int NT>
int impl(const PagedAttnParams& p0, int num_sms, cudaStream_t stream) {
  using Gm = PagedGeom<kD, Q8>;
  PagedAttnParams p = p0;
  constexpr int rows = 8 * NT;
  p.n_rb = (p.R + rows - 1) / rows;
  const int smem = Gm::smem(rows) + (p.B + 1) * 4;
  // two CTAs per SM where their shared memory (1 KB more each, 228 KB in all) and static arrays allow it
  constexpr int fixed = 1024 + 256 + Gm::NW * (rows * 8 + Gm::ST * 4) + rows * 4;
  const int per_sm = 2 * (smem + fixed) <= 233472 ? 2 : 1;
  p.n_groups = per_sm * (num_sms < kTreeMaxCtas ? num_sms : kTreeMaxCtas);
  p.part_ml = p.part + static_cast<size_t>(kPagedMaxCtas) * 2 * rows * kD;
  auto kern = attn_paged_kernel<kD, BF16, Q8, NT>;
  static std::atomic<uint64_t> done{0};
  if (!set_smem_limit(kern, Gm::smem(rows) + (kPagedMaxB + 1) * 4, done)) return kLaunchCudaError;
  const int r = launch_dependent(kern, dim3(p.n_groups), Gm::THREADS, smem, stream, p);
  if (r != kLaunchOk || p.n_groups == 1) return r;
  const long long tasks = static_cast<long long>(p.B) * p.c.Hkv * p.R, most = 8LL * kTreeMaxCtas;
  return launch_dependent(attn_paged_join_kernel<kD, BF16, Q8, NT>, dim3(static_cast<unsigned>(tasks < most ? tasks : most)),
                          kPagedJoinThreads, 0, stream, p);
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
