// Attention of one new token per sequence over a paged cache in few bits.
//
//   s_t = scale q . k_t,  m = max_t s_t,  y = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m)
//
// One pass over the cache with a running maximum: the codes go from memory to
// the matrix cores, and their scales are applied to the scores instead of the
// rows,
//   s_t = (q . code_t) ks_t,   y = sum_t (p_t vs_t) code_t / sum_t p_t,
// so that a row of d elements costs one product per query head and not d.
#include "bfly_cache.h"
#include "bfly_common.h"

#include <algorithm>
#include <type_traits>

namespace bfly {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4, kStep = 32;         // tokens of a wave's step: two tiles of 16
constexpr int kRound = kWaves * kStep;        // tokens of a workgroup's round
constexpr int kHeads = 16;                    // query heads a workgroup takes (matrix-core columns)
constexpr float kNone = -3.0e38f;             // below every score: nothing seen yet
constexpr float kLog2e = 1.44269504088896341f;

// Eight operand values of a matrix-core instruction's lane.
struct Operand {
  uint32_t w[4];
};
template <int FMT>
__device__ __forceinline__ f32x4 product(const Operand& a, const Operand& b, f32x4 c) {
  if constexpr (FMT == kCacheBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ f16x2 halves(uint32_t w) { return __builtin_bit_cast(f16x2, w); }
__device__ __forceinline__ uint32_t bits_of(f16x2 v) { return __builtin_bit_cast(uint32_t, v); }

// Nibbles 0 and 4 (or 1 and 5, `odd`) of a word of int4 codes with their signs
// flipped, c + 8, as fp16 pairs: with the bits of 1024 above them they read as
// 1024 + (c + 8), or 1024 + 16 (c + 8); one exact operation leaves c.
template <bool ODD>
__device__ __forceinline__ uint32_t nibbles(uint32_t w) {
  if constexpr (ODD) {
    const f16x2 v = halves((w & 0x00F000F0u) | 0x64006400u);
    const f16x2 k = {(_Float16)0.0625f, (_Float16)0.0625f}, z = {(_Float16)-72.f, (_Float16)-72.f};
    return bits_of(__builtin_elementwise_fma(v, k, z));
  } else {
    const f16x2 v = halves((w & 0x000F000Fu) | 0x64006400u);
    const f16x2 z = {(_Float16)-1032.f, (_Float16)-1032.f};
    return bits_of(v + z);
  }
}
// Bytes SEL of (hi, lo), c + 128 each, under the exponent of 1024 -> c.
__device__ __forceinline__ uint32_t byte_pair(uint32_t bytes, uint32_t sel) {
  const f16x2 v = halves(__builtin_amdgcn_perm(0x64646464u, bytes, sel));
  const f16x2 z = {(_Float16)-1152.f, (_Float16)-1152.f};
  return bits_of(v + z);
}
template <bool HIGH>
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t bytes) {
  return bits_of(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)bytes, 1.0f, HIGH));
}

// The order in which eight consecutive elements of a key enter the product.
template <int FMT>
__host__ __device__ constexpr int key_order(int j) {
  return FMT == kCacheInt4 ? (j & 1) * 4 + (j >> 1) : j;
}
// Words of eight codes.
template <int FMT>
constexpr int kWords8 = FMT == kCacheBF16 ? 4 : FMT == kCacheInt4 ? 1 : 2;

template <int FMT>
__device__ __forceinline__ Operand key_operand(const uint32_t* w) {
  if constexpr (FMT == kCacheBF16) {
    return Operand{{w[0], w[1], w[2], w[3]}};
  } else if constexpr (FMT == kCacheInt4) {
    const uint32_t a = w[0] ^ 0x88888888u, b = a >> 8;
    return Operand{{nibbles<false>(a), nibbles<true>(a), nibbles<false>(b), nibbles<true>(b)}};
  } else if constexpr (FMT == kCacheInt8) {
    const uint32_t a = w[0] ^ 0x80808080u, b = w[1] ^ 0x80808080u;
    return Operand{{byte_pair(a, 0x04010400u), byte_pair(a, 0x04030402u),
                    byte_pair(b, 0x04010400u), byte_pair(b, 0x04030402u)}};
  } else {
    return Operand{{e4m3_pair<false>(w[0]), e4m3_pair<true>(w[0]), e4m3_pair<false>(w[1]),
                    e4m3_pair<true>(w[1])}};
  }
}

// The values' operands: a lane holds E = D / 16 consecutive elements of eight
// tokens; operand i is element i of the eight.  w[t] are token t's words.
template <int FMT, int E, int W>
__device__ __forceinline__ void value_operands(const uint32_t (&w)[8][W], Operand (&out)[E]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t(&a)[W] = w[2 * p];
    const uint32_t(&b)[W] = w[2 * p + 1];
    if constexpr (FMT == kCacheInt4) {
      // 16-bit halves of both tokens side by side: four nibbles of each
#pragma unroll
      for (int h = 0; h < E / 4; ++h) {
        const uint32_t x = 0x88888888u ^ __builtin_amdgcn_perm(b[h / 2], a[h / 2],
                                                               h % 2 ? 0x07060302u : 0x05040100u);
        const uint32_t y = x >> 8;
        out[4 * h].w[p] = nibbles<false>(x);
        out[4 * h + 1].w[p] = nibbles<true>(x);
        out[4 * h + 2].w[p] = nibbles<false>(y);
        out[4 * h + 3].w[p] = nibbles<true>(y);
      }
    } else if constexpr (FMT == kCacheBF16) {
#pragma unroll
      for (int h = 0; h < E / 2; ++h) {
        out[2 * h].w[p] = __builtin_amdgcn_perm(b[h], a[h], 0x05040100u);
        out[2 * h + 1].w[p] = __builtin_amdgcn_perm(b[h], a[h], 0x07060302u);
      }
    } else {
      // bytes a0 b0 a1 b1 and a2 b2 a3 b3
#pragma unroll
      for (int h = 0; h < E / 4; ++h) {
        uint32_t x = __builtin_amdgcn_perm(b[h], a[h], 0x05010400u);
        uint32_t y = __builtin_amdgcn_perm(b[h], a[h], 0x07030602u);
        if constexpr (FMT == kCacheInt8) {
          x ^= 0x80808080u;
          y ^= 0x80808080u;
          out[4 * h].w[p] = byte_pair(x, 0x04010400u);
          out[4 * h + 1].w[p] = byte_pair(x, 0x04030402u);
          out[4 * h + 2].w[p] = byte_pair(y, 0x04010400u);
          out[4 * h + 3].w[p] = byte_pair(y, 0x04030402u);
        } else {
          out[4 * h].w[p] = e4m3_pair<false>(x);
          out[4 * h + 1].w[p] = e4m3_pair<true>(x);
          out[4 * h + 2].w[p] = e4m3_pair<false>(y);
          out[4 * h + 3].w[p] = e4m3_pair<true>(y);
        }
      }
    }
  }
}

// `bytes` (2 to 64) from memory into words; two bytes leave a word's upper half 0.
template <int BYTES>
__device__ __forceinline__ void fetch(const char* p, uint32_t* w) {
  if constexpr (BYTES == 2) {
    w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else if constexpr (BYTES == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (BYTES == 8) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    w[0] = a.x, w[1] = a.y;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 a = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
    }
  }
}

// The four groups of 16 lanes brought together: f of the lanes l, l ^ 16,
// l ^ 32, l ^ 48.
template <typename F>
__device__ __forceinline__ float across_groups(float v, F f) {
  v = f(v, __shfl_xor(v, 16));
  return f(v, __shfl_xor(v, 32));
}

// N fp16 (bf16 for a bf16 cache) parts of eight values that add up to them.
// fp16 parts: each the rounding of what the earlier ones leave.  bf16 parts
// are truncations from below, so that every part of a positive weight is
// positive and an infinity in a value meets no zero and no other sign.
template <int FMT, int N>
__device__ __forceinline__ void weight_parts(const float (&w)[8], Operand (&out)[N]) {
  if constexpr (FMT == kCacheBF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = w[2 * i], b = w[2 * i + 1];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        uint32_t ha, hb;
        if (n + 1 < N) {
          ha = __builtin_elementwise_sub_sat(__float_as_uint(a), 1u) & 0xFFFF0000u;
          hb = __builtin_elementwise_sub_sat(__float_as_uint(b), 1u) & 0xFFFF0000u;
          a -= __uint_as_float(ha);
          b -= __uint_as_float(hb);
          out[n].w[i] = (ha >> 16) | hb;
        } else {
          out[n].w[i] = pack_bf16(a, b);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f32x2_t v = {w[2 * i], w[2 * i + 1]};
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const f16x2 h = __builtin_convertvector(v, f16x2);
        out[n].w[i] = bits_of(h);
        v.x -= (float)h.x;
        v.y -= (float)h.y;
      }
    }
  }
}

// Parts of the queries and of the weights: with bf16 queries and results one
// fp16 part of each is exact (queries) or rounds a weight by 2^-12 (a quarter
// of what the result's own rounding does); a bf16 weight of one part would
// round by 2^-9, as much as the result itself, so it has two.  fp32 results
// take 22 (fp16) or 24 (bf16) bits of both.
template <int FMT, bool EXACT>
constexpr int kQueryParts = !EXACT ? 1 : FMT == kCacheBF16 ? 3 : 2;
template <int FMT, bool EXACT>
constexpr int kWeightParts = (FMT == kCacheBF16 ? 2 : 1) + (EXACT ? 1 : 0);

// Which tokens of row `row` a call looks at: [first, end), cut into chunks
// that start at a multiple of 32.
struct Reach {
  int first, end, base;
};
__device__ __forceinline__ Reach reach_of(const AttendParams& P, int64_t row) {
  Reach r;
  r.end = min(max(P.lens[row], 0), P.max_len);
  r.first = P.window > 0 ? max(0, r.end - P.window) : 0;
  r.base = r.first & ~(kStep - 1);
  return r;
}

// One head of the partial results of a call whose length is split: the
// running maximum, the sum of the weights and the unnormalised result.
template <int D>
struct Partial {
  float top, total, pad[2];
  float y[D];
};

// Four elements of a result, from the sums; a row that saw nothing gives 0.
__device__ __forceinline__ void put_result(const AttendParams& P, int64_t at, f32x4 o, float l) {
  const float by = 1.f / l;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = l == 0.f ? 0.f : o[e] * by;
  if (P.y_bf16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.y) + at) =
        make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
  else
    *reinterpret_cast<f32x4*>(static_cast<float*>(P.y) + at) = o;
}
__device__ __forceinline__ float log_sum(float top, float l) {
  return l == 0.f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(l)) / kLog2e;
}

template <int FMT, int D, bool EXACT>
__global__ void __launch_bounds__(256) attend_kernel(AttendParams P, int splits, int chunk,
                                                     int blocks) {
  constexpr int E = D / 16;                     // a lane's elements of a value
  constexpr int QN = kQueryParts<FMT, EXACT>, WN = kWeightParts<FMT, EXACT>;
  constexpr int KB = cache_bytes(FMT, D / 4);   // a lane's bytes of a key
  constexpr int VB = cache_bytes(FMT, E);       // and of a value
  constexpr int KW = KB / 4, VW = VB < 4 ? 1 : VB / 4;
  constexpr int ROW = cache_bytes(FMT, D);
  constexpr bool SCALED = FMT != kCacheBF16;
  __shared__ float factors[kWaves][3][kStep];   // of a step's tokens: ks, log2 vs, 1 / vs
  __shared__ float stats[kWaves][2][kHeads];
  constexpr int PARTS = D > 128 ? 2 : 1, DP = D / PARTS;   // of the waves' results, one at a time
  __shared__ float sums[kWaves][kHeads][DP + 4];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int col = lane & 15, group = lane >> 4;
  const int share = P.heads / P.kv_heads;
  int at = (int)blockIdx.x;
  const int split = at % splits;
  at /= splits;
  const int block = at % blocks;
  at /= blocks;
  const int kvh = at % P.kv_heads;
  const int64_t row = at / P.kv_heads;
  const int head0 = kvh * share + block * kHeads;            // the block's first query head
  const int heads = min(kHeads, share - block * kHeads);     // and how many it has
  const Reach R = reach_of(P, row);
  const int t0 = R.base + split * chunk, t1 = min(R.end, t0 + chunk);
  if (t0 >= t1 && splits > 1) return;           // nothing to add: the join does not look here

  // the queries: column `col` is head head0 + col, a lane holds its D / 4 elements
  Operand q[QN][D / 32];
  float qscale;
  {
    float f[D / 4];
    const bool mine = col < heads;
    const int64_t from = row * P.q_stride + (int64_t)(head0 + (mine ? col : 0)) * D + group * (D / 4);
    if (P.q_bf16) {
      uint32_t w[D / 8];
      fetch<D / 2>(static_cast<const char*>(P.q) + from * 2, w);
#pragma unroll
      for (int i = 0; i < D / 4; ++i) f[i] = (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    } else {
      uint32_t w[D / 4];
      fetch<D>(static_cast<const char*>(P.q) + from * 4, w);
#pragma unroll
      for (int i = 0; i < D / 4; ++i) f[i] = __uint_as_float(w[i]);
    }
    qscale = P.scale * kLog2e;
    float by = 1.f;
    if constexpr (SCALED) {
      // a power of two that brings the largest element to [2^14, 2^15): fp16
      // then holds every element down to 2^-29 of it with all its bits
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(f[i]));
      top = across_groups(top, [](float a, float b) { return fmaxf(a, b); });
      int e = top > 0.f ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
      e = min(max(e, -120), 120);
      by = top < __builtin_inff() ? ldexpf(1.f, e) : __builtin_nanf("");
      qscale = ldexpf(qscale, -e);
    }
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = mine ? f[8 * s + key_order<FMT>(j)] * by : 0.f;
#pragma unroll
      for (int n = 0; n < QN; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (SCALED) {
            const f32x2_t pair = {v[2 * i], v[2 * i + 1]};
            const f16x2 h = __builtin_convertvector(pair, f16x2);
            q[n][s].w[i] = bits_of(h);
            v[2 * i] -= (float)h.x;
            v[2 * i + 1] -= (float)h.y;
          } else {
            const uint32_t h = pack_bf16(v[2 * i], v[2 * i + 1]);
            q[n][s].w[i] = h;
            v[2 * i] -= bf16_lo(h);
            v[2 * i + 1] -= bf16_hi(h);
          }
        }
    }
  }

  const int shift = P.page_shift, in_page = (1 << shift) - 1;
  const int32_t* const table = P.tables + row * P.table_width;
  // page of the tile of 16 tokens at t, or -1: past the end, or none in the table
  const auto page_of = [&](int t) {
    if (t >= t1) return -1;
    const int id = __builtin_amdgcn_readfirstlane(table[t >> shift]);
    return (uint32_t)id < (uint32_t)P.pages ? id : -1;
  };
  const int64_t head_rows = (int64_t)1 << shift;
  // a page's first row of this head; page 0 stands in where there is none
  const auto row_of = [&](int page, int t) {
    return ((int64_t)max(page, 0) * P.kv_heads + kvh) * head_rows + (t & in_page);
  };
  const char* const kc = static_cast<const char*>(P.k_cache);
  const char* const vc = static_cast<const char*>(P.v_cache);

  uint32_t k[2][KW], v[8][VW];
  uint16_t raw_ks = 0, raw_vs = 0;   // lane t: token t of the step (the tile of a lane above 31 is not used)
  const int my_tile = (lane >> 4) & 1;
  const auto load_keys = [&](int t, const int (&page)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const char* const p = kc + row_of(page[j], t + 16 * j) * ROW;
      fetch<KB>(p + (uint32_t)(col * ROW + group * KB), k[j]);
    }
    if constexpr (SCALED) {
      const int64_t r0 = row_of(page[0], t), r1 = row_of(page[1], t + 16);
      const int64_t r = (my_tile ? r1 : r0) + col;
      raw_ks = P.k_scales[r];
      raw_vs = P.v_scales[r];
    }
  };
  const auto load_values = [&](int t, const int (&page)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const char* const p = vc + row_of(page[j], t + 16 * j) * ROW;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        fetch<VB>(p + (uint32_t)((4 * group + i) * ROW + col * VB), v[4 * j + i]);
    }
  };

  float m = kNone, total = 0.f;
  f32x4 acc[E];
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};

  int t = t0 + wave * kStep;
  int page[2], next[2];
  if (t < t1) {
    page[0] = page_of(t), page[1] = page_of(t + 16);
    load_keys(t, page);
    load_values(t, page);
  }
  for (; t < t1; t += kRound) {
    const int tn = t + kRound;
    if (tn < t1) next[0] = page_of(tn), next[1] = page_of(tn + 16);
    // a step that has tokens nobody may look at
    const bool edge = t < R.first || t + kStep > t1 || page[0] < 0 || page[1] < 0;

    f32x4 s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const Operand a = key_operand<FMT>(&k[j][c * kWords8<FMT>]);
#pragma unroll
        for (int n = 0; n < QN; ++n) s[j] = product<FMT>(a, q[n][c], s[j]);
      }
    }
    // a token of the step that may be looked at
    const auto seen = [&](int i) {
      const int at_t = t + i;
      return at_t >= R.first && at_t < t1 && (i < 16 ? page[0] : page[1]) >= 0;
    };
    float u[8], inv[8];
    if constexpr (SCALED) {
      if (lane < kStep) {
        const float ks = (float)__builtin_bit_cast(_Float16, raw_ks);
        // a value scale of 0 stands for a row of codes 0: any scale will do
        float vs = (float)__builtin_bit_cast(_Float16, raw_vs);
        vs = vs == 0.f ? 1.f : vs;
        factors[wave][0][lane] = ks;
        factors[wave][1][lane] = __builtin_amdgcn_logf(vs);
        factors[wave][2][lane] = __builtin_amdgcn_rcpf(vs);
      }
      wave_lds_sync();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const f32x4 ks = *reinterpret_cast<const f32x4*>(&factors[wave][0][16 * j + 4 * group]);
        const f32x4 lv = *reinterpret_cast<const f32x4*>(&factors[wave][1][16 * j + 4 * group]);
        const f32x4 iv = *reinterpret_cast<const f32x4*>(&factors[wave][2][16 * j + 4 * group]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[4 * j + i] = fmaf(s[j][i] * qscale, ks[i], lv[i]);
          inv[4 * j + i] = iv[i];
        }
      }
      wave_lds_sync();
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = s[i >> 2][i & 3] * qscale;
    }
    if (edge) {
      // what lies there may be anything: it enters nothing (integer codes are
      // finite, so that a weight of 0 is enough for them)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool ok = seen(16 * (i >> 2) + 4 * group + (i & 3));
        u[i] = ok ? u[i] : -__builtin_inff();
        if constexpr (SCALED) inv[i] = ok ? inv[i] : 0.f;
        if constexpr (FMT == kCacheBF16 || FMT == kCacheE4M3)
#pragma unroll
          for (int h = 0; h < VW; ++h) v[i][h] = ok ? v[i][h] : 0u;
      }
    }
    float top = fmaxf(fmaxf(fmaxf(u[0], u[1]), fmaxf(u[2], u[3])),
                      fmaxf(fmaxf(u[4], u[5]), fmaxf(u[6], u[7])));
    top = across_groups(top, [](float a, float b) { return fmaxf(a, b); });
    // weights are 2^(u - m) with m between 15 below the largest u and 8 below
    // it, so that it seldom moves and fp16 holds them down to 2^-22 of the
    // largest with all bits
    if (__any(top > m + 15.f)) {
      const float to = top > m + 15.f ? top - 8.f : m;
      const float fade = __builtin_amdgcn_exp2f(m - to);
      m = to;
      total *= fade;
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] *= fade;
    }
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = __builtin_amdgcn_exp2f(u[i] - m);
      total = SCALED ? fmaf(w[i], inv[i], total) : total + w[i];
    }
    if (tn < t1) load_keys(tn, next);

    Operand p[WN];
    weight_parts<FMT, WN>(w, p);
    Operand x[E];
    value_operands<FMT, E, VW>(v, x);
#pragma unroll
    for (int i = 0; i < E; ++i)
#pragma unroll
      for (int n = 0; n < WN; ++n) acc[i] = product<FMT>(x[i], p[n], acc[i]);
    if (tn < t1) load_values(tn, next);
    page[0] = next[0], page[1] = next[1];
  }

  // the waves' results joined
  total = across_groups(total, [](float a, float b) { return a + b; });
  if (group == 0) {
    stats[wave][0][col] = m;
    stats[wave][1][col] = total;
  }
  __syncthreads();
  float top = stats[0][0][col];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) top = fmaxf(top, stats[i][0][col]);
  const float fade = __builtin_amdgcn_exp2f(m - top);
  // operand i's row 4 group + r of the product is element (4 group + r) E + i
  constexpr int RP = 4 / PARTS;
#pragma unroll
  for (int part = 0; part < PARTS; ++part) {
    if (part > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < RP; ++r)
#pragma unroll
      for (int i = 0; i < E; ++i)
        sums[wave][col][(RP * group + r) * E + i] = acc[i][RP * part + r] * fade;
    __syncthreads();
    for (int i = threadIdx.x; i < heads * (DP / 4); i += 256) {
      const int h = i / (DP / 4), x = i % (DP / 4) * 4, r = x / E;
      const int d = (r / RP * 4 + RP * part + r % RP) * E + x % E;
      float all = stats[0][0][h], l = 0.f;
#pragma unroll
      for (int n = 1; n < kWaves; ++n) all = fmaxf(all, stats[n][0][h]);
      f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < kWaves; ++n) {
        l = fmaf(stats[n][1][h], __builtin_amdgcn_exp2f(stats[n][0][h] - all), l);
        o += *reinterpret_cast<const f32x4*>(&sums[n][h][x]);
      }
      const int64_t to = row * P.heads + head0 + h;
      if (splits > 1) {
        Partial<D>* const result = reinterpret_cast<Partial<D>*>(P.partials) + to * splits + split;
        *reinterpret_cast<f32x4*>(&result->y[d]) = o;
        if (d == 0) result->top = all, result->total = l;
      } else {
        put_result(P, to * D + d, o, l);
        if (P.lse && d == 0) P.lse[to] = log_sum(all, l);
      }
    }
  }
}

// The partial results of a row's head joined: a workgroup to each.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(AttendParams P, int splits, int chunk) {
  constexpr int L = D / 4, G = 256 / L;         // lanes to a partial result, results at a time
  __shared__ f32x4 sums[G][L];
  __shared__ float totals[G];
  const int64_t to = blockIdx.x;
  const Reach R = reach_of(P, to / P.heads);
  const int used = (R.end - R.base + chunk - 1) / chunk;
  const Partial<D>* const part = reinterpret_cast<const Partial<D>*>(P.partials) + to * splits;
  const int g = threadIdx.x / L, d = threadIdx.x % L * 4;
  float top = kNone;
  for (int i = 0; i < used; ++i) top = fmaxf(top, part[i].top);
  float l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  for (int i = g; i < used; i += G) {
    const float by = __builtin_amdgcn_exp2f(part[i].top - top);
    l = fmaf(part[i].total, by, l);
    o += *reinterpret_cast<const f32x4*>(&part[i].y[d]) * by;
  }
  sums[g][threadIdx.x % L] = o;
  if (threadIdx.x % L == 0) totals[g] = l;
  __syncthreads();
  if (g != 0) return;
#pragma unroll
  for (int i = 1; i < G; ++i) {
    o += sums[i][threadIdx.x % L];
    l += totals[i];
  }
  put_result(P, to * D + d, o, l);
  if (P.lse && threadIdx.x == 0) P.lse[to] = log_sum(top, l);
}

constexpr int kWorkgroups = 1024;    // that fill the card
constexpr int kLeast = 256;          // tokens that are worth a workgroup

int most_splits(int max_len) { return (max_len + kStep - 1 + kLeast - 1) / kLeast; }

}  // namespace

size_t attend_workspace_bytes(int64_t rows, int heads, int head_dim, int max_len) {
  const int64_t results = rows * heads, most = most_splits(max_len);
  if (most <= 1) return 0;
  // splits <= min(most, 1 + kWorkgroups / items), and 16 items cover 16 heads each
  const int64_t parts = std::min(results * most, results + (int64_t)kHeads * kWorkgroups);
  return (size_t)parts * (size_t)(head_dim + 4) * sizeof(float);
}

hipError_t launch_attend(const AttendParams& p, hipStream_t s) {
  const int share = p.heads / p.kv_heads, blocks = (share + kHeads - 1) / kHeads;
  const int64_t items = p.rows * p.kv_heads * blocks;
  const int reach = p.window > 0 ? std::min(p.max_len, p.window + kStep - 1) : p.max_len;
  const int64_t want = 1 + (kWorkgroups - 1) / items;   // rounded up
  int splits = (int)std::max<int64_t>(1, std::min<int64_t>((reach + kLeast - 1) / kLeast, want));
  const int chunk = std::max(kRound, ((reach + splits - 1) / splits + kRound - 1) / kRound * kRound);
  splits = std::max(1, (reach + chunk - 1) / chunk);
  const dim3 grid((unsigned)(items * splits));
  const auto go = [&](auto d, auto f) {
    constexpr int D = decltype(d)::value, F = decltype(f)::value;
    if (p.q_bf16 && p.y_bf16) attend_kernel<F, D, false><<<grid, 256, 0, s>>>(p, splits, chunk, blocks);
    else attend_kernel<F, D, true><<<grid, 256, 0, s>>>(p, splits, chunk, blocks);
  };
  const auto by_format = [&](auto d) {
    constexpr int D = decltype(d)::value;
    switch (p.format) {
      case kCacheBF16: go(d, std::integral_constant<int, kCacheBF16>{}); break;
      case kCacheInt8: go(d, std::integral_constant<int, kCacheInt8>{}); break;
      case kCacheE4M3: go(d, std::integral_constant<int, kCacheE4M3>{}); break;
      default: go(d, std::integral_constant<int, kCacheInt4>{}); break;
    }
    if (splits > 1) join_kernel<D><<<(unsigned)(p.rows * p.heads), 256, 0, s>>>(p, splits, chunk);
  };
  switch (p.head_dim) {
    case 64: by_format(std::integral_constant<int, 64>{}); break;
    case 128: by_format(std::integral_constant<int, 128>{}); break;
    default: by_format(std::integral_constant<int, 256>{}); break;
  }
  return hipGetLastError();
}

}  // namespace bfly
