// The 2-norm over many tensors, and all of them scaled to a largest norm:
//
//   norm = sqrt(sum over all elements of g^2),  c = norm > max_norm ? max_norm / norm : 1
//   out = g c
//
// Squares are summed in fp64 (an fp32 square overflows above 1.8e19 and loses
// everything below 1e-23, and a sum over 10^9 elements loses half its digits).
// Two passes over the data: the slots' sums, then the scaling, whose every
// workgroup first adds the (at most 1024) slot sums in a fixed order.
#include "bfly_clip.h"
#include "bfly_rows.h"

namespace bfly {
namespace {

constexpr int kThreads = 256;

// The table's entries of up to kBatch tensors, as kernel arguments.
constexpr int kBatch = 120;
struct Batch {
  ClipTensor t[kBatch];
};
__global__ void __launch_bounds__(128) table_kernel(Batch b, int count, ClipTensor* to) {
  const int i = threadIdx.x;
  if (i < count) to[i] = b.t[i];
}

// The tensor that holds granule g: the last one whose first granule is not
// beyond it.  All threads of the workgroup look, one of them finds it.
__device__ __forceinline__ int find_tensor(const ClipTensor* tab, int count, int g, int* found) {
  for (int i = threadIdx.x; i < count; i += kThreads)
    if (tab[i].first <= g && (i + 1 == count || tab[i + 1].first > g)) *found = i;
  __syncthreads();
  return *found;
}

// One granule's elements of thread t, four at a time: 16-byte loads of fp32
// or 8-byte loads of bf16 where the tensor is aligned to them, else single
// elements.  f(values, offset of the first, how many are valid).
template <typename F>
__device__ __forceinline__ void each_four(const ClipTensor& c, int64_t at, int len, F f) {
  const int t = threadIdx.x;
  if (c.bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(c.in) + at;
    const bool wide = ((uintptr_t)p & 7) == 0;
#pragma unroll
    for (int k = 0; k < kClipGranule / (4 * kThreads); ++k) {
      const int i = (k * kThreads + t) * 4, m = len - i < 4 ? len - i : 4;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (wide && m == 4) {
        const uint2 q = *reinterpret_cast<const uint2*>(p + i);
        v[0] = bf16_lo(q.x);
        v[1] = bf16_hi(q.x);
        v[2] = bf16_lo(q.y);
        v[3] = bf16_hi(q.y);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < m) v[e] = bf16_lo(p[i + e]);
      }
      f(v, i, m);
    }
  } else {
    const float* p = static_cast<const float*>(c.in) + at;
    const bool wide = ((uintptr_t)p & 15) == 0;
#pragma unroll
    for (int k = 0; k < kClipGranule / (4 * kThreads); ++k) {
      const int i = (k * kThreads + t) * 4, m = len - i < 4 ? len - i : 4;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (wide && m == 4) {
        const float4 q = *reinterpret_cast<const float4*>(p + i);
        v[0] = q.x;
        v[1] = q.y;
        v[2] = q.z;
        v[3] = q.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < m) v[e] = p[i + e];
      }
      f(v, i, m);
    }
  }
}

// Calls f(tensor, offset of the granule in it, its length) for a slot's granules.
template <typename F>
__device__ __forceinline__ void each_granule(const ClipTensor* tab, int count, int g0, int g1,
                                             int* found, F f) {
  if (g0 >= g1) return;
  int i = find_tensor(tab, count, g0, found);
  for (int g = g0; g < g1; ++g) {
    while (i + 1 < count && tab[i + 1].first <= g) ++i;
    const ClipTensor c = tab[i];
    const int64_t at = (int64_t)(g - c.first) * kClipGranule;
    const int64_t left = c.numel - at;
    f(c, at, (int)(left < kClipGranule ? left : kClipGranule));
  }
}

__device__ __forceinline__ double block_total(double v, double* buf) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  return (buf[0] + buf[1]) + (buf[2] + buf[3]);
}

__global__ void __launch_bounds__(kThreads) square_kernel(const ClipTensor* tab, int count,
                                                          int granules, int per_slot,
                                                          double* sums) {
  __shared__ int found;
  __shared__ double buf[kThreads / 64];
  const int g0 = blockIdx.x * per_slot;
  const int g1 = g0 + per_slot < granules ? g0 + per_slot : granules;
  double s = 0.0;
  each_granule(tab, count, g0, g1, &found, [&](const ClipTensor& c, int64_t at, int len) {
    each_four(c, at, len, [&](const float (&v)[4], int, int) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s = fma((double)v[e], (double)v[e], s);
    });
  });
  s = block_total(s, buf);
  if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) scale_kernel(const ClipTensor* tab, int count,
                                                         int granules, int per_slot, int slots,
                                                         const double* sums, float max_norm,
                                                         float* norm) {
  __shared__ int found;
  __shared__ double buf[kThreads / 64];
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < kClipSlots / kThreads; ++k) {
    const int i = k * kThreads + threadIdx.x;
    s += i < slots ? sums[i] : 0.0;
  }
  const double all = sqrt(block_total(s, buf));
  // a norm that is not finite scales nothing: it is reported, and the caller drops the step
  const float c = all > (double)max_norm && all < __builtin_inf() ? (float)(max_norm / all) : 1.f;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    norm[0] = (float)all;
    norm[1] = c;
  }
  const int g0 = blockIdx.x * per_slot;
  const int g1 = g0 + per_slot < granules ? g0 + per_slot : granules;
  each_granule(tab, count, g0, g1, &found, [&](const ClipTensor& t, int64_t at, int len) {
    if (c == 1.f && t.in == t.out) return;  // in place and not scaled: nothing to write
    each_four(t, at, len, [&](const float (&v)[4], int i, int m) {
      if (m <= 0) return;
      if (t.bf16) {
        uint16_t* o = static_cast<uint16_t*>(t.out) + at + i;
        const uint2 q = make_uint2(pack_bf16(v[0] * c, v[1] * c), pack_bf16(v[2] * c, v[3] * c));
        if (m == 4 && ((uintptr_t)o & 7) == 0) {
          *reinterpret_cast<uint2*>(o) = q;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < m) o[e] = (uint16_t)((e < 2 ? q.x : q.y) >> (16 * (e & 1)));
        }
      } else {
        float* o = static_cast<float*>(t.out) + at + i;
        if (m == 4 && ((uintptr_t)o & 15) == 0) {
          *reinterpret_cast<float4*>(o) = make_float4(v[0] * c, v[1] * c, v[2] * c, v[3] * c);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < m) o[e] = v[e] * c;
        }
      }
    });
  });
}

}  // namespace

hipError_t launch_grad_clip(const ClipParams& p, hipStream_t s) {
  double* sums = static_cast<double*>(p.workspace);
  ClipTensor* tab = reinterpret_cast<ClipTensor*>(static_cast<char*>(p.workspace) + kClipTableOffset);
  int64_t granules = 0;
  int count = 0;
  Batch b;
  int filled = 0;
  for (int i = 0; i <= p.count; ++i) {
    if (filled == kBatch || (i == p.count && filled > 0)) {
      hipLaunchKernelGGL(table_kernel, dim3(1), dim3(128), 0, s, b, filled, tab + count - filled);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      filled = 0;
    }
    if (i == p.count || p.numel[i] == 0) continue;
    ClipTensor& t = b.t[filled++];
    t.in = p.in[i];
    t.out = p.out[i];
    t.numel = p.numel[i];
    t.first = (int32_t)granules;
    t.bf16 = p.dtype[i];
    granules += clip_granules(p.numel[i]);
    ++count;
  }
  const int64_t per_slot = granules > kClipSlots ? (granules + kClipSlots - 1) / kClipSlots : 1;
  const int slots = (int)((granules + per_slot - 1) / per_slot);
  if (slots > 0) {
    hipLaunchKernelGGL(square_kernel, dim3(slots), dim3(kThreads), 0, s, tab, count, (int)granules,
                       (int)per_slot, sums);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(scale_kernel, dim3(slots > 0 ? slots : 1), dim3(kThreads), 0, s, tab, count,
                     (int)granules, (int)per_slot, slots, sums, p.max_norm, p.norm);
  return hipGetLastError();
}

}  // namespace bfly
