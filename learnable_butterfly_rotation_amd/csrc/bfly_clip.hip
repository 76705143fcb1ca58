// The 2-norm over many tensors, and all of them scaled to a largest norm:
//
//   norm = sqrt(sum over all elements of g^2),  c = norm > max_norm ? max_norm / norm : 1
//   out = g c
//
// Squares are summed in fp64 (an fp32 square overflows above 1.8e19 and loses
// everything below 1e-23, and a sum over 10^9 elements loses half its digits).
// Two passes over the data, both bound by memory: the slots' sums, then the
// scaling.  With few bytes its every workgroup first adds the (at most
// 2048) slot sums itself, in a fixed order; with many a launch between does.
#include "bfly_clip.h"
#include "bfly_rows.h"

namespace bfly {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // vectors of a thread in flight

// The table's entries of up to kClipBatch tensors, as kernel arguments.  Those
// of a call with no more tensors go to the first pass, which writes them down
// for the second (3.5 KiB of arguments less: 96 tensors take the host 8.1 us,
// 8.3 to 8.7 where both passes get them).
struct Batch {
  ClipTensor t[kClipBatch];
};
// More tensors than that: what the table is made from, in as few launches as
// 4 KiB of arguments allow (300 tensors of 54 MB: 38.7 us with 2 of them, 40.5 with the
// entries themselves and 3).
struct ClipSource {
  const char* in;
  char* out;
  uint64_t numel;  // the top bit: bf16
};
struct Sources {
  ClipSource t[kClipSources];
};

// A tensor's entry but for its first granule, and how many granules it has.
__host__ __device__ __forceinline__ int entry_of(const char* in, char* out, int64_t numel,
                                                 int bf16, ClipTensor& t) {
  const int es = bf16 ? 2 : 4, skip = (int)((uintptr_t)in & 15) / es;
  t.in = in - skip * es;
  t.out = out - skip * es;
  t.end = numel + skip;
  t.kind = bf16 + 2 * skip;
  return (int)((t.end + kClipGranule - 1) / kClipGranule);
}

// Entries of `count` tensors, the first of which starts at granule `first`.
__global__ void __launch_bounds__(kThreads) table_kernel(Sources b, int count, int first,
                                                         ClipTensor* to) {
  static_assert(kClipSources <= kThreads, "a thread to a tensor");
  __shared__ int sums[kThreads / 64];
  const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
  ClipTensor t;
  int mine = 0;
  if (i < count) {
    const ClipSource& s = b.t[i];
    mine = entry_of(s.in, s.out, (int64_t)(s.numel & ~(1ull << 63)), (int)(s.numel >> 63), t);
  }
  int upto = mine;  // and those before it in the wave
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  for (int w = 0; w < wave; ++w) first += sums[w];
  if (i < count) {
    t.first = first + upto - mine;
    to[i] = t;
  }
}

// The tensor that holds granule g: the last one whose first granule is not
// beyond it.  All threads of the workgroup look, one of them finds it.
__device__ __forceinline__ int find_tensor(const ClipTensor* tab, int count, int g, int* found) {
  for (int i = threadIdx.x; i < count; i += kThreads)
    if (tab[i].first <= g && (i + 1 == count || tab[i + 1].first > g)) *found = i;
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*found);
}

// A 16-byte vector of a tensor's elements, as fp32.
// NT: loads and whole stores marked as used once.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <bool BF, bool NT>
struct Vec {
  static constexpr int W = BF ? 8 : 4;
  float v[W];
  __device__ __forceinline__ void load(const char* p) {
    const u32x4* const from = reinterpret_cast<const u32x4*>(p);
    const u32x4 w = NT ? __builtin_nontemporal_load(from) : *from;
#pragma unroll
    for (int e = 0; e < W; ++e)
      v[e] = !BF ? __uint_as_float(w[e]) : (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
  }
  // elements [lo, hi) of the vector, the others 0
  __device__ __forceinline__ void load_some(const char* p, int lo, int hi) {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      v[e] = 0.f;
      if (e >= lo && e < hi)
        v[e] = BF ? bf16_lo(reinterpret_cast<const uint16_t*>(p)[e])
                  : reinterpret_cast<const float*>(p)[e];
    }
  }
  __device__ __forceinline__ void words(uint32_t (&w)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = BF ? pack_bf16(v[(2 * i) % W], v[(2 * i + 1) % W]) : __float_as_uint(v[i]);
  }
  __device__ __forceinline__ void store(char* p) const {
    uint32_t w[4];
    words(w);
    const u32x4 q = {w[0], w[1], w[2], w[3]};
    if (NT) __builtin_nontemporal_store(q, reinterpret_cast<u32x4*>(p));
    else *reinterpret_cast<u32x4*>(p) = q;
  }
  __device__ __forceinline__ void store_some(char* p, int lo, int hi) const {
    uint32_t w[4];
    words(w);
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (e >= lo && e < hi) {
        if constexpr (BF) reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        else reinterpret_cast<uint32_t*>(p)[e] = w[e];
      }
  }
};

// The elements [from, to) of a tensor, counted from its boundary, vector by
// vector over the workgroup: f(vector, offset of it, first and last + 1 of
// its elements that are the tensor's).  Where there are kAhead whole vectors,
// their loads are in flight together.
template <bool BF, bool NT, typename F>
__device__ __forceinline__ void each_vector(const char* in, int64_t from, int64_t to, F f) {
  using V = Vec<BF, NT>;
  constexpr int es = BF ? 2 : 4, W = V::W, step = kThreads * W;
  const int64_t first = from / W * W;  // of a vector; from is inside it
  int64_t at = first + threadIdx.x * W;
  V v[kAhead];
  if (from > first) {  // the tensor starts inside its first vector
    if (threadIdx.x == 0) {
      const int hi = to - at < W ? (int)(to - at) : W;
      v[0].load_some(in + at * es, (int)(from - first), hi);
      f(v[0], at, (int)(from - first), hi);
    }
    if (threadIdx.x == 0) at += step;
  }
  for (; at + (kAhead - 1) * step + W <= to; at += kAhead * step) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) v[k].load(in + (at + k * step) * es);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) f(v[k], at + k * step, 0, W);
  }
  for (; at < to; at += step) {
    if (at + W <= to) {
      v[0].load(in + at * es);
      f(v[0], at, 0, W);
    } else {
      v[0].load_some(in + at * es, 0, (int)(to - at));
      f(v[0], at, 0, (int)(to - at));
    }
  }
}

// Calls f(tensor, from, to) for a slot's granules, one range to a tensor.
template <typename F>
__device__ __forceinline__ void each_range(const ClipTensor* tab, int count, int g0, int g1,
                                           int* found, F f) {
  if (g0 >= g1) return;
  int i = find_tensor(tab, count, g0, found);
  for (int g = g0; g < g1; ++i) {
    const ClipTensor c = tab[i];
    const int next = i + 1 < count ? tab[i + 1].first : g1;
    const int stop = next < g1 ? next : g1;
    const int64_t skip = c.kind >> 1;
    const int64_t from = (int64_t)(g - c.first) * kClipGranule;
    const int64_t to = (int64_t)(stop - c.first) * kClipGranule;
    f(c, from > skip ? from : skip, to < c.end ? to : c.end);
    g = stop;
  }
}

__device__ __forceinline__ double block_total(double v, double* buf) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  return (buf[0] + buf[1]) + (buf[2] + buf[3]);
}

// How the granules are dealt out, and the table in memory.
struct Slots {
  ClipTensor* table;
  int count, granules, per_slot, slots;
};

__device__ __forceinline__ void square_slot(const ClipTensor* tab, const Slots& S, double* sums) {
  __shared__ int found;
  __shared__ double buf[kThreads / 64];
  const int g0 = blockIdx.x * S.per_slot;
  const int g1 = g0 + S.per_slot < S.granules ? g0 + S.per_slot : S.granules;
  double s = 0.0;
  each_range(tab, S.count, g0, g1, &found, [&](const ClipTensor& c, int64_t from, int64_t to) {
    const auto add = [&](const auto& v, int64_t, int, int) {
#pragma unroll
      for (float e : v.v) s = fma((double)e, (double)e, s);
    };
    if (c.kind & 1) each_vector<true, false>(c.in, from, to, add);
    else each_vector<false, false>(c.in, from, to, add);
  });
  s = block_total(s, buf);
  if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

// The norm and the factor from the sum of squares.  A norm that is not finite
// as it is reported, in fp32, scales nothing: the caller sees it and drops the
// step.
__device__ __forceinline__ float factor_of(double squares, float max_norm, float* norm) {
  const double all = sqrt(squares);
  const float reported = (float)all;
  const bool scale = all > (double)max_norm && reported < __builtin_inff();
  const float c = scale ? (float)(max_norm / all) : 1.f;
  if (norm) {
    norm[0] = reported;
    norm[1] = c;
  }
  return c;
}

template <bool NT>
__device__ __forceinline__ void scale_range(const ClipTensor& t, int64_t from, int64_t to,
                                            float c) {
  if (c == 1.f && t.in == t.out) return;  // in place and not scaled: nothing to write
  const bool wide = ((uintptr_t)t.out & 15) == 0;  // the output is aligned as the input is
  const auto put = [&](auto v, int64_t at, int lo, int hi) {
    constexpr int W = decltype(v)::W;
#pragma unroll
    for (float& e : v.v) e *= c;
    char* const o = t.out + at * (16 / W);
    if (wide && hi - lo == W) v.store(o);
    else v.store_some(o, lo, hi);
  };
  if (t.kind & 1) each_vector<true, NT>(t.in, from, to, put);
  else each_vector<false, NT>(t.in, from, to, put);
}

__device__ __forceinline__ void scale_slot(const ClipTensor* tab, const Slots& S,
                                           const double* sums, float max_norm, float* norm) {
  __shared__ int found;
  __shared__ double buf[kThreads / 64];
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < kClipSlots / kThreads; ++k) {
    const int i = k * kThreads + threadIdx.x;
    s += i < S.slots ? sums[i] : 0.0;
  }
  const float c = factor_of(block_total(s, buf), max_norm,
                            blockIdx.x == 0 && threadIdx.x == 0 ? norm : nullptr);
  const int g0 = blockIdx.x * S.per_slot;
  const int g1 = g0 + S.per_slot < S.granules ? g0 + S.per_slot : S.granules;
  each_range(tab, S.count, g0, g1, &found, [&](const ClipTensor& t, int64_t from, int64_t to) {
    scale_range<false>(t, from, to, c);
  });
}

// Many bytes: the norm by one workgroup, then a granule to a workgroup at
// a time, neighbours together, past the caches (721M fp32 elements: 1429 us
// as 1024 ranges through the caches).
__global__ void __launch_bounds__(kThreads) factor_kernel(Slots S, const double* sums,
                                                          float max_norm, float* norm) {
  __shared__ double buf[kThreads / 64];
  double s = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < S.slots; i += kThreads) s += sums[i];
  s = block_total(s, buf);
  if (threadIdx.x == 0) factor_of(s, max_norm, norm);
}
__device__ __forceinline__ void scale_granules(const ClipTensor* tab, const Slots& S,
                                               const float* norm) {
  __shared__ int found[2];
  const float c = norm[1];
  int turn = 0;
  for (int g = blockIdx.x; g < S.granules; g += gridDim.x, turn ^= 1)
    each_range(tab, S.count, g, g + 1, &found[turn],
               [&](const ClipTensor& t, int64_t from, int64_t to) {
                 scale_range<true>(t, from, to, c);
               });
}

__global__ void __launch_bounds__(kThreads) square_kernel(Slots S, double* sums) {
  square_slot(S.table, S, sums);
}
__global__ void __launch_bounds__(kThreads) square_few_kernel(Batch b, Slots S, double* sums) {
  if (blockIdx.x == 0 && threadIdx.x < S.count) S.table[threadIdx.x] = b.t[threadIdx.x];
  square_slot(b.t, S, sums);
}
__global__ void __launch_bounds__(kThreads) scale_kernel(Slots S, const double* sums,
                                                         float max_norm, float* norm) {
  scale_slot(S.table, S, sums, max_norm, norm);
}
__global__ void __launch_bounds__(kThreads) scale_many_kernel(Slots S, const float* norm) {
  scale_granules(S.table, S, norm);
}

}  // namespace

hipError_t launch_grad_clip(const ClipParams& p, hipStream_t s) {
  double* sums = static_cast<double*>(p.workspace);
  ClipTensor* tab = reinterpret_cast<ClipTensor*>(static_cast<char*>(p.workspace) + kClipTableOffset);
  int64_t granules = 0, bytes = 0;
  int count = 0;  // tensors that are not empty
  for (int i = 0; i < p.count; ++i) count += p.numel[i] > 0;
  const bool few = count <= kClipBatch;
  static_assert(kClipBatch <= kThreads, "a thread to a tensor");
  Batch b;  // entries past the last tensor's are not looked at, here and there
  Sources src;
  int held = 0, first = 0;  // in src; its first tensor's first granule
  for (int i = 0, at = 0; i < p.count; ++i) {
    if (p.numel[i] == 0) continue;
    const char* const in = static_cast<const char*>(p.in[i]);
    char* const out = static_cast<char*>(p.out[i]);
    const int bf16 = p.dtype[i] != 0;
    ClipTensor t;
    t.first = (int32_t)granules;
    granules += entry_of(in, out, p.numel[i], bf16, t);
    bytes += p.numel[i] * (bf16 ? 2 : 4);
    ++at;
    if (few) {
      b.t[at - 1] = t;
      continue;
    }
    src.t[held++] = {in, out, (uint64_t)p.numel[i] | (uint64_t)bf16 << 63};
    if (held == kClipSources || at == count) {
      hipLaunchKernelGGL(table_kernel, dim3(1), dim3(kThreads), 0, s, src, held, first,
                         tab + at - held);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      held = 0;
      first = (int)granules;
    }
  }
  Slots S;
  S.table = tab;
  S.count = count;
  S.granules = (int)granules;
  const bool many = bytes > kClipFewBytes;
  const int most = many ? kClipManySlots : kClipSlots;
  S.per_slot = (int)(granules > most ? (granules + most - 1) / most : 1);
  S.slots = (int)((granules + S.per_slot - 1) / S.per_slot);
  hipError_t e = hipSuccess;
  if (S.slots > 0) {
    if (few) hipLaunchKernelGGL(square_few_kernel, dim3(S.slots), dim3(kThreads), 0, s, b, S, sums);
    else hipLaunchKernelGGL(square_kernel, dim3(S.slots), dim3(kThreads), 0, s, S, sums);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (many) {
    hipLaunchKernelGGL(factor_kernel, dim3(1), dim3(kThreads), 0, s, S, sums, p.max_norm, p.norm);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const dim3 grid(S.granules < 65536 ? S.granules : 65536);
    hipLaunchKernelGGL(scale_many_kernel, grid, dim3(kThreads), 0, s, S, p.norm);
    return hipGetLastError();
  }
  const dim3 grid(S.slots > 0 ? S.slots : 1);
  hipLaunchKernelGGL(scale_kernel, grid, dim3(kThreads), 0, s, S, sums, p.max_norm, p.norm);
  return hipGetLastError();
}

}  // namespace bfly
