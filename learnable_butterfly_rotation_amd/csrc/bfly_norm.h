// Root-mean-square norm of rows (bfly_norm.hip): launch parameters shared by
// the C-ABI layer and the kernels.
#pragma once

#include "bfly_internal.h"

namespace bfly {

constexpr int kNormMaxN = 16384;  // longest row: a row stays in the registers of one workgroup

struct NormParams {
  const void* x;         // [rows][n], bf16 (x_bf16) or fp32
  const void* residual;  // of x's type, or nullptr
  void* h;               // x + residual in x's type, or nullptr
  const void* weight;    // [n], bf16 (w_bf16) or fp32, or nullptr (ones)
  void* y;               // [rows][n], bf16 (y_bf16) or fp32, or nullptr
  uint8_t* codes;        // [rows][n], or nullptr
  uint16_t* scales;      // [rows][n / group]
  float* rstd;           // [rows], or nullptr
  int64_t rows;
  int32_t n, group;
  int32_t x_bf16, w_bf16, y_bf16;
  int32_t e4m3;          // 1: e4m3 codes, 0: int8
  float eps;
};
hipError_t launch_rmsnorm(const NormParams& p, hipStream_t s);

struct NormBwdParams {
  const void* h;         // [rows][n], bf16 (h_bf16) or fp32
  const void* weight;    // [n] or nullptr
  const float* rstd;     // [rows]
  const void* dy;        // [rows][n], bf16 (g_bf16) or fp32
  const void* dh;        // of dy's type, or nullptr
  void* dx;              // of dy's type
  float* dweight;        // [n], or nullptr
  float* partials;       // [rmsnorm_bwd_slots(rows, n)][n] when dweight is asked for
  int64_t rows;
  int32_t n;
  int32_t h_bf16, w_bf16, g_bf16;
};
// Row slots of the weight gradient: a function of (rows, n) only, so that the
// order of its sum never depends on the device.
int rmsnorm_bwd_slots(int64_t rows, int n);
hipError_t launch_rmsnorm_backward(NormBwdParams p, hipStream_t s);

}  // namespace bfly
