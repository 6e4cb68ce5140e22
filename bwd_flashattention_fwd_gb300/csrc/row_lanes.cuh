// Rows of D 16-bit values held by the lanes of a warp, 16 values each.
#pragma once

#include "kernel_common.cuh"

namespace gbattn {

template <int D>
struct RowLanes {
  static constexpr int LANES = D / 16;                            // lanes that hold a row
  static constexpr int GROUP = LANES <= 4 ? 4 : LANES <= 8 ? 8 : 16;  // lanes set aside for it (a power of two)
  static constexpr int ROWS = 32 / GROUP;                         // rows of a warp
};

template <int GROUP>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int m = GROUP / 2; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = Elem<BF16>::unpack(w[i]);
    f[2 * i] = v.x, f[2 * i + 1] = v.y;
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(Elem<BF16>::pack(f[0], f[1]), Elem<BF16>::pack(f[2], f[3]), Elem<BF16>::pack(f[4], f[5]),
                    Elem<BF16>::pack(f[6], f[7]));
}

}  // namespace gbattn
