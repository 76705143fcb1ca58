// Global gradient norm and clipping (bfly_clip.hip): the interface between
// the C-ABI layer and the kernels.
#pragma once

#include "bfly_internal.h"

namespace bfly {

// The tensors are cut into granules of kClipGranule elements (a tensor's last
// one may be shorter), numbered through all tensors; a slot is a run of
// consecutive granules, summed by one workgroup.
constexpr int kClipGranule = 4096;
constexpr int kClipSlots = 1024;

inline int64_t clip_granules(int64_t numel) { return (numel + kClipGranule - 1) / kClipGranule; }

// One tensor in the workspace's table.
struct ClipTensor {
  const void* in;
  void* out;
  int64_t numel;
  int32_t first;  // its first granule
  int32_t bf16;   // 1: bf16, 0: fp32
};

// Workspace: the slots' sums of squares, then the table.
constexpr size_t kClipTableOffset = kClipSlots * sizeof(double);
inline size_t clip_workspace_bytes(int32_t count) {
  return kClipTableOffset + (size_t)count * sizeof(ClipTensor);
}

struct ClipParams {
  int32_t count;                // tensors, none of them empty
  const void* const* in;        // host arrays
  void* const* out;
  const int64_t* numel;
  const int32_t* dtype;         // 1: bf16, 0: fp32
  float max_norm;
  float* norm;                  // device [2]: the norm, the factor
  void* workspace;
};
hipError_t launch_grad_clip(const ClipParams& p, hipStream_t s);

}  // namespace bfly
