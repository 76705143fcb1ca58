// Global gradient norm and clipping (bfly_clip.hip): the interface between
// the C-ABI layer and the kernels.
#pragma once

#include "bfly_internal.h"

namespace bfly {

// The tensors are cut into granules of kClipGranule elements, numbered through
// all tensors; a slot is a run of consecutive granules, summed by one
// workgroup.  A tensor's granules start at the 16-byte boundary at or below
// its first element, so that every whole vector in them is aligned.
constexpr int kClipGranule = 4096;
// Slots at most, of a call of up to kClipFewBytes bytes of gradients and of a
// larger one.  300 tensors, 27M bf16 elements (54 MB): 40.8 us with 2048, 44.7
// with 1024.  The larger calls' way (bfly_clip.hip) against the other: 52 MB
// 32.3 us and 31.5, 54 MB in 300 tensors 46 and 41, 67 MB 33.4 and 39.7, 108 MB
// 63.5 and 74.4, 154 MB 80 and 104.
constexpr int kClipSlots = 2048, kClipManySlots = 8192;
constexpr int64_t kClipFewBytes = 56 << 20;

// One tensor of the table.
struct ClipTensor {
  const char* in;  // that boundary
  char* out;       // the output's address of it
  int64_t end;     // elements from there to the tensor's end
  int32_t first;   // the tensor's first granule
  int32_t kind;    // 1: bf16, 0: fp32; + 2 * the elements before the tensor's first
};
// Tensors whose table goes into a launch's arguments; for more of them it is
// written to the workspace first, kClipSources to a launch.
constexpr int kClipBatch = 112, kClipSources = 160;

// Workspace: the slots' sums of squares, then the table.
constexpr size_t kClipTableOffset = kClipManySlots * sizeof(double);
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
