// Host-side checks and device state that the C ABI units of the serving calls share.
#pragma once

#include <cmath>

#include "launch.h"

namespace gbattn {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline bool supported_d(int D) { return D == 64 || D == 96 || D == 128 || D == 256; }

inline size_t round16(size_t x) { return (x + 15) & ~static_cast<size_t>(15); }

inline attn_status_t check_scale(float scale) {
  return std::isfinite(scale) && scale > 0.f ? ATTN_OK : ATTN_ERR_INVALID_ARG;
}

inline float scale_log2_of(float scale) { return static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074); }

// An array of a call, for the checks that no output shares storage with an
// input (blocks read the one while others write the other) or another output.
struct Span {
  const void* at;
  long long bytes;
};

inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.at && b.at && (x < y ? y - x < static_cast<uintptr_t>(a.bytes) : x - y < static_cast<uintptr_t>(b.bytes));
}

// Whether one of the first n_out spans overlaps any other of the n.
template <int N>
bool outputs_overlap(const Span (&s)[N], int n_out) {
  for (int i = 0; i < n_out; ++i)
    for (int j = i + 1; j < N; ++j)
      if (overlap(s[i], s[j])) return true;
  return false;
}

// The device's state for a call on `stream`.  It is allocated by the first call
// on a device, which a stream capture does not allow and would not survive: such
// a first call is refused before it touches anything.
inline attn_status_t call_state(cudaStream_t stream, int* dev, EncodeTiledFn* enc, int** status, int* num_sms) {
  if (!shared_device_ready()) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess || cs != cudaStreamCaptureStatusNone) {
      cudaGetLastError();  // an implicit-capture error must not linger for later calls
      return ATTN_ERR_INVALID_ARG;
    }
  }
  return shared_device_state(dev, enc, status, num_sms);
}

inline attn_status_t finish(int r) {
  return r == kLaunchOk ? ATTN_OK : r == kLaunchBadMap ? ATTN_ERR_INVALID_ARG : ATTN_ERR_CUDA;
}

}  // namespace gbattn
