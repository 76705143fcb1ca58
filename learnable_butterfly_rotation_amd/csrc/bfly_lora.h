// Low-rank adapters beside a shared product (bfly_lora.hip): launch
// parameters shared by the C-ABI layer and the kernels.
#pragma once

#include "bfly_internal.h"

namespace bfly {

constexpr int kLoraMaxRank = 256;
constexpr int kLoraMaxAdapters = 1 << 22;

struct LoraParams {
  const uint16_t* x;      // bf16 [rows][k]
  const int32_t* ids;     // [rows]: the row's adapter; outside [0, n_adapters): none
  const uint16_t* a;      // bf16 [n_adapters][rank][k]
  const uint16_t* b;      // bf16 [n_adapters][n_out][rank]
  const float* scaling;   // [n_adapters]
  const void* base;       // [rows][n_out] of base_bf16 or fp32, or nullptr (zeros)
  void* y;                // [rows][n_out] of y_bf16 or fp32; may be base (same type)
  void* workspace;        // lora_workspace_bytes
  int64_t rows;
  int32_t n_out, k, n_adapters, rank;
  int32_t base_bf16, y_bf16;
};
// Workspace bytes of a call: a function of the sizes only, that never falls
// with any of them.
size_t lora_workspace_bytes(int64_t rows, int k, int rank);
hipError_t launch_lora(const LoraParams& p, hipStream_t s);

}  // namespace bfly
