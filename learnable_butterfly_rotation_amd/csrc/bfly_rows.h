// Device helpers of the row kernels: loads and stores of eight elements of a
// bf16 or fp32 row, and sums and maxima over a wave.
#pragma once

#include "bfly_common.h"

namespace bfly {

// Where the eight elements (v, 0..7) of thread t of T lie in a row.
//   VEC     chunk v*T + t, eight consecutive elements: 16-byte accesses (rows
//           whose length is a multiple of 8, so that every row is aligned)
//   not VEC element (8v + e)*T + t: accesses of one element, consecutive over
//           the lanes (rows of any length)
// Reads past the row's end give zeros and writes there are dropped (the
// buffer's range check).  With T < 64 the buffer holds the 64 / T rows of a
// wave, `row` is the element its lane's row starts at and `n` the rows' length.
template <int T, bool VEC, bool BF>
struct RowIo {
  // eight elements as they lie in memory (BF: four words, else eight)
  struct Raw {
    uint32_t w[BF && VEC ? 4 : 8];
  };
  static __device__ __forceinline__ int index(int t, int v, int e) {
    return VEC ? (v * T + t) * 8 + e : (v * 8 + e) * T + t;
  }
  static constexpr uint32_t es = BF ? 2u : 4u;
  // byte offset of element (v, e), beyond every range where it is past the row
  static __device__ __forceinline__ uint32_t offset(int t, int v, int e, int row, int n) {
    const int i = index(t, v, e);
    if constexpr (T < 64) return i < n ? (uint32_t)(row + i) * es : kOutOfRange - 64u;
    return (uint32_t)i * es;
  }
  static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t r, int t, int v, int row,
                                             int n) {
    Raw q;
    if constexpr (VEC) {
      const uint32_t off = offset(t, v, 0, row, n);
      const uint4 a = buf_ld16(r, off);
      q.w[0] = a.x;
      q.w[1] = a.y;
      q.w[2] = a.z;
      q.w[3] = a.w;
      if constexpr (!BF) {
        const uint4 b = buf_ld16(r, off + 16u);
        q.w[4] = b.x;
        q.w[5] = b.y;
        q.w[6] = b.z;
        q.w[7] = b.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t off = offset(t, v, e, row, n);
        if constexpr (BF)
          q.w[e] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
        else
          q.w[e] = buf_ld4(r, off);
      }
    }
    return q;
  }
  static __device__ __forceinline__ void unpack(const Raw& q, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (!BF)
        f[e] = __uint_as_float(q.w[e]);
      else if constexpr (!VEC)
        f[e] = bf16_lo(q.w[e]);
      else
        f[e] = (e & 1) ? bf16_hi(q.w[e >> 1]) : bf16_lo(q.w[e >> 1]);
    }
  }
  // fp32 values rounded to the row's type (bf16: to nearest even)
  static __device__ __forceinline__ Raw pack(const float (&f)[8]) {
    Raw q;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (!BF)
        q.w[e] = __float_as_uint(f[e]);
      else if constexpr (!VEC)
        q.w[e] = pack_bf16(f[e], 0.f) & 0xFFFFu;
      else if (!(e & 1))
        q.w[e >> 1] = pack_bf16(f[e], f[e + 1]);
    }
    return q;
  }
  template <int POLICY = kCached>
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, int t, int v, int row,
                                               int n, const Raw& q) {
    if constexpr (VEC) {
      const uint32_t off = offset(t, v, 0, row, n);
      buf_st16<POLICY>(r, off, make_uint4(q.w[0], q.w[1], q.w[2], q.w[3]));
      if constexpr (!BF)
        buf_st16<POLICY>(r, off + 16u, make_uint4(q.w[4], q.w[5], q.w[6], q.w[7]));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t off = offset(t, v, e, row, n);
        if constexpr (BF)
          buf_st2<POLICY>(r, off, (uint16_t)q.w[e]);
        else
          buf_st4<POLICY>(r, off, q.w[e]);
      }
    }
  }
};

// Rows r .. r + count - 1 of n elements of es bytes; empty where there is no
// matrix.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_range(const void* base, int64_t r, int n,
                                                            int es, int count = 1) {
  return buffer_range32(static_cast<const char*>(base) + r * n * es,
                        base ? (uint32_t)count * (uint32_t)n * (uint32_t)es : 0u);
}

// The value of another lane of the same 16 (DPP): 0xB1 lane ^ 1, 0x4E lane ^ 2,
// 0x141 mirrored within 8, 0x140 mirrored within 16.  Applied in this order,
// a symmetric operation leaves its result over 2, 4, 8, 16 lanes in each of them.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
      0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF,
                                                            false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF,
                                                            0xF, false);
  return __builtin_bit_cast(double, (uint64_t)lo | (uint64_t)hi << 32);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)lo | (uint64_t)hi << 32);
}
// Sum over the wave's 64 lanes (or each 16 of them), in a fixed order, the
// same in every lane.
template <int LANES = 64, typename F>
__device__ __forceinline__ F wave_sum(F v) {
  static_assert(LANES == 16 || LANES == 64, "16 or 64 lanes");
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  if constexpr (LANES == 16) return v;
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
// Maximum over 1, 2, 4 .. 64 consecutive lanes (an aligned run of `lanes`).
__device__ __forceinline__ float run_max(float v, int lanes) {
  if (lanes > 1) v = fmaxf(v, dpp<0xB1>(v));
  if (lanes > 2) v = fmaxf(v, dpp<0x4E>(v));
  if (lanes > 4) v = fmaxf(v, dpp<0x141>(v));
  if (lanes > 8) v = fmaxf(v, dpp<0x140>(v));
  if (lanes > 16) v = fmaxf(v, __shfl_xor(v, 16));
  if (lanes > 32) v = fmaxf(v, __shfl_xor(v, 32));
  return v;
}

}  // namespace bfly
