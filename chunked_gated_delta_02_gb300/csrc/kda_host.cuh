// Host-side helpers that the entry points of several source files share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

inline bool aligned(const void *ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

// NVTX range for the host-side enqueue of one stage (shows up around the launches in a trace).
struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

// Device address of the current device's sticky status word, or null (kda_api.cu).
int *device_status_address();

// SM count of the current device, or 0 if it cannot be read (kda_recur.cu).
int device_sm_count();

// Tensor map over a 16-bit token tensor, dims (D, H, T, B) with D contiguous and the strides of H, T
// and B in bytes, loaded in boxes of 64 columns x 1 head x `rows` tokens x 1 batch row into
// 128-byte-swizzled rows; positions past a dimension read as zeros (kda_api.cu).
bool encode_swizzled_token_map(CUtensorMap *m, const void *base, int D, int H, int T, int B,
                               const long long (&stride_bytes)[3], int rows);

}  // namespace kda
