// Rows of keys and values into the pages of a cache, in few bits, and back.
//
//   scale = fp16(max |x| / top),  code_i = rnd(x_i / scale),  x_i ~ code_i scale
//
// top = 127 (int8), 448 (e4m3) or 7 (int4); bf16 rows are rounded and have no
// scale.  The quotients are rounded from their exact values: max |x| / top by
// a division, x / scale as codes of an IEEE quotient (quotient() below).  No
// double rounding is possible: a value of 24 bits over one of at most 11 lies
// further from a rounding border than half of the fp32 quotient's last bit.
#include "bfly_cache.h"
#include "bfly_rows.h"

#include <type_traits>

namespace bfly {
namespace {

constexpr float top_of(int format) {
  return format == kCacheInt8 ? 127.f : format == kCacheE4M3 ? 448.f : 7.f;
}

// Largest over the `lanes` (8, 16 or 32) of a row.
__device__ __forceinline__ uint32_t row_max(uint32_t v, int lanes) {
  const auto other = [](uint32_t x, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xF, 0xF, false);
  };
  v = max(v, other(v, std::integral_constant<int, 0xB1>{}));
  v = max(v, other(v, std::integral_constant<int, 0x4E>{}));
  v = max(v, other(v, std::integral_constant<int, 0x141>{}));
  if (lanes > 8) v = max(v, other(v, std::integral_constant<int, 0x140>{}));
  if (lanes > 16) v = max(v, (uint32_t)__shfl_xor((int)v, 16));
  return v;
}

// Eight elements of a row that its lane holds, as they lie in memory: 8 lane ...
// of bf16 rows; of fp32 rows 4 lane ... of each half, so that the wave's loads
// and stores cover whole lines.
template <int D, bool BF>
struct Eight {
  static constexpr int EACH = BF ? 8 : 4, STEP = BF ? 4 : D / 2;  // consecutive; from four to four
  uint32_t w[BF ? 4 : 8];
  __device__ __forceinline__ void load(const char* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    if constexpr (!BF) {
      const uint4 b = *reinterpret_cast<const uint4*>(p + 4 * STEP);
      w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
  }
  __device__ __forceinline__ float at(int e) const {
    if constexpr (BF) return (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
    return __uint_as_float(w[e]);
  }
};

// x / d correctly rounded; r the rounded reciprocal of d, which has at most 11
// bits, so one correction by the exact remainder is enough (Markstein).
__device__ __forceinline__ float quotient(float x, float d, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, d, x), r, q);
}

// A row's scale from the bits of its largest |x| (a NaN's are larger than an
// infinity's), its codes, and where they go.  A row with a NaN has scale NaN
// and codes 0: it reads back as NaN.  An infinity has code +-top and the
// largest scale.
template <int FMT, int D, bool BF>
__device__ __forceinline__ void put_row(const Eight<D, BF>& x, int lane, char* row,
                                        uint16_t* scale, bool there) {
  // where the second four's codes go
  char* const row4 = row + cache_bytes(FMT, Eight<D, BF>::STEP);
  if constexpr (FMT == kCacheBF16) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = BF ? x.w[i] : pack_bf16(x.at(2 * i), x.at(2 * i + 1));
    if (there) {
      *reinterpret_cast<uint2*>(row) = make_uint2(q[0], q[1]);
      *reinterpret_cast<uint2*>(row4) = make_uint2(q[2], q[3]);
    }
  } else {
    constexpr float top = top_of(FMT);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x.at(e)) & 0x7FFFFFFFu);
    m = row_max(m, D / 8);
    const bool nan = m > 0x7F800000u;
    const _Float16 s = (_Float16)fminf(__uint_as_float(m) / top, 65504.f);
    const float d = (float)s, r = d > 0.f && !nan ? 1.f / d : 0.f;
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = x.at(e);
      if (m >= 0x7F800000u) v = __builtin_amdgcn_fmed3f(v, -3.40282347e38f, 3.40282347e38f);
      q[e] = __builtin_amdgcn_fmed3f(quotient(v, d, r), -top, top);
    }
    const uint32_t any = r > 0.f ? ~0u : 0u;
    if constexpr (FMT == kCacheE4M3) {
      uint32_t w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
        w[i] = any & (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], lo, true);
      }
      if (there) {
        *reinterpret_cast<uint32_t*>(row) = w[0];
        *reinterpret_cast<uint32_t*>(row4) = w[1];
      }
    } else {
      // 1.5 * 2^23 + q is rounded to nearest even at the unit: its low bits are the code
      constexpr int bits = FMT == kCacheInt8 ? 8 : 4;
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e / 4] |= (__float_as_uint(q[e] + 12582912.f) & ((1u << bits) - 1u)) << (e % 4 * bits);
      if (there) {
        if constexpr (bits == 8) {
          *reinterpret_cast<uint32_t*>(row) = w[0] & any;
          *reinterpret_cast<uint32_t*>(row4) = w[1] & any;
        } else {
          *reinterpret_cast<uint16_t*>(row) = (uint16_t)(w[0] & any);
          *reinterpret_cast<uint16_t*>(row4) = (uint16_t)(w[1] & any);
        }
      }
    }
    if (there && lane == 0) *scale = nan ? (uint16_t)0x7E00 : __builtin_bit_cast(uint16_t, s);
  }
}

// Four consecutive codes of a row as numbers.
template <int FMT>
struct Four {
  uint32_t w[FMT == kCacheBF16 ? 2 : 1];
  __device__ __forceinline__ void load(const char* p) {
    if constexpr (FMT == kCacheBF16) {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      w[0] = a.x, w[1] = a.y;
    } else if constexpr (FMT == kCacheInt4) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  }
  __device__ __forceinline__ void numbers(float* f) const {
    if constexpr (FMT == kCacheE4M3) {
      const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[0], false);
      const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[0], true);
      f[0] = lo.x, f[1] = lo.y, f[2] = hi.x, f[3] = hi.y;
    } else
#pragma unroll
      for (int e = 0; e < 4; ++e)
        f[e] = FMT == kCacheBF16   ? ((e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]))
               : FMT == kCacheInt4 ? (float)((int32_t)(w[0] << (28 - 4 * e)) >> 28)
                                   : (float)((int32_t)(w[0] << (24 - 8 * e)) >> 24);
  }
};

// A workgroup: one head's keys and values of 2048 / D consecutive tokens, D / 8
// lanes to a row.  Consecutive tokens' rows mostly lie together in a page, so a
// wave writes (or reads) whole lines there, and 2 D bytes or more of each token
// on the other side.
template <int D, int FMT, bool BF, bool WRITE>
__global__ void __launch_bounds__(256) cache_kernel(CacheParams P) {
  constexpr int L = D / 8, TOK = 256 / L;
  const int lane = threadIdx.x % L;
  const int head = blockIdx.x % P.kv_heads;
  const int64_t token = (int64_t)(blockIdx.x / P.kv_heads) * TOK + threadIdx.x / L;
  if (token >= P.tokens) return;  // whole rows: no lane of a row that goes on is missing
  const int32_t slot = P.slots[token];
  const int32_t page = slot >> P.page_shift, place = slot & ((1 << P.page_shift) - 1);
  const bool there = slot >= 0 && page < P.pages;
  const int64_t at = (((int64_t)(there ? page : 0) * P.kv_heads + head) << P.page_shift) + place;
  constexpr int EACH = Eight<D, BF>::EACH, STEP = Eight<D, BF>::STEP;
  const int64_t code = at * cache_bytes(FMT, D) + cache_bytes(FMT, EACH) * lane;
  const int64_t col = ((int64_t)head * D + EACH * lane) * (BF ? 2 : 4);
  const int64_t xk = token * P.k_stride * (BF ? 2 : 4) + col;
  const int64_t xv = token * P.v_stride * (BF ? 2 : 4) + col;
  char* const kc = static_cast<char*>(P.k_cache) + code;
  char* const vc = static_cast<char*>(P.v_cache) + code;
  if constexpr (WRITE) {
    Eight<D, BF> k, v;
    k.load(static_cast<const char*>(P.k) + xk);
    v.load(static_cast<const char*>(P.v) + xv);
    put_row<FMT, D>(k, lane, kc, P.k_scales + at, there);
    put_row<FMT, D>(v, lane, vc, P.v_scales + at, there);
  } else {
    // The rows go past the caches (32768 tokens of 8 heads int4 to bf16 38.9 ->
    // 25.1 us), which wants whole lines from a store of the wave (4099 tokens of
    // 40 heads fp32, written and read: 67 us; 99 with eight consecutive elements
    // to a lane, 80 with those through the caches).
    const char* const from[2] = {kc, vc};
    char* const out[2] = {const_cast<char*>(static_cast<const char*>(P.k)) + xk,
                          const_cast<char*>(static_cast<const char*>(P.v)) + xv};
    Four<FMT> c[2][2] = {};
    float s[2] = {0.f, 0.f};
    if (there) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        c[i][0].load(from[i]);
        c[i][1].load(from[i] + cache_bytes(FMT, STEP));
      }
      s[0] = s[1] = 1.f;
      if constexpr (FMT != kCacheBF16) {
        s[0] = (float)__builtin_bit_cast(_Float16, P.k_scales[at]);
        s[1] = (float)__builtin_bit_cast(_Float16, P.v_scales[at]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float f[8];
      c[i][0].numbers(f);
      c[i][1].numbers(f + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= s[i];
      if constexpr (BF) {
        __builtin_nontemporal_store(u32x4_t{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                            pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])},
                                    reinterpret_cast<u32x4_t*>(out[i]));
      } else {
        typedef float f32x4_t __attribute__((ext_vector_type(4)));
        __builtin_nontemporal_store(f32x4_t{f[0], f[1], f[2], f[3]},
                                    reinterpret_cast<f32x4_t*>(out[i]));
        __builtin_nontemporal_store(f32x4_t{f[4], f[5], f[6], f[7]},
                                    reinterpret_cast<f32x4_t*>(out[i] + 4 * STEP));
      }
    }
  }
}

template <bool WRITE>
hipError_t launch(const CacheParams& p, hipStream_t s) {
  const int tok = 2048 / p.head_dim;
  const dim3 grid((unsigned)((p.tokens + tok - 1) / tok * p.kv_heads));
  const auto go = [&](auto d, auto f) {
    constexpr int D = decltype(d)::value, F = decltype(f)::value;
    if (p.x_bf16) cache_kernel<D, F, true, WRITE><<<grid, 256, 0, s>>>(p);
    else cache_kernel<D, F, false, WRITE><<<grid, 256, 0, s>>>(p);
  };
  const auto by_format = [&](auto d) {
    switch (p.format) {
      case kCacheBF16: return go(d, std::integral_constant<int, kCacheBF16>{});
      case kCacheInt8: return go(d, std::integral_constant<int, kCacheInt8>{});
      case kCacheE4M3: return go(d, std::integral_constant<int, kCacheE4M3>{});
      default: return go(d, std::integral_constant<int, kCacheInt4>{});
    }
  };
  switch (p.head_dim) {
    case 64: by_format(std::integral_constant<int, 64>{}); break;
    case 128: by_format(std::integral_constant<int, 128>{}); break;
    default: by_format(std::integral_constant<int, 256>{}); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_write(const CacheParams& p, hipStream_t s) { return launch<true>(p, s); }
hipError_t launch_cache_read(const CacheParams& p, hipStream_t s) { return launch<false>(p, s); }

}  // namespace bfly
