// Attention of one new token per sequence over a paged cache in few bits.
//
//   s_t = scale q . k_t,  m = max_t s_t,  y = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m)
//
// One pass over the cache with a running maximum: the codes go from memory to
// the matrix cores, and their scales are applied to the scores instead of the
// rows,
//   s_t = (q . code_t) ks_t,   y = sum_t (p_t vs_t) code_t / sum_t p_t,
// so that a row of d elements costs one product per query head and not d.
#include "bfly_attend_cut.h"
#include "bfly_cache.h"
#include "bfly_rows.h"

#include <algorithm>
#include <type_traits>

namespace bfly {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = kAttendStep, kHeads = kAttendHeads;
constexpr float kNone = -3.0e38f;             // below every score: nothing seen yet
constexpr float kLog2e = 1.44269504088896341f;

// Eight operand values of a matrix-core instruction's lane.
struct __align__(16) Operand {
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

// Nibbles 0 and 4 (or 1 and 5, ODD) of a word of int4 codes as fp16 pairs.  The
// mask and the bits of 1024 with the sign's flip, in one operation, leave
// 1024 + (c + 8), or 1024 + 16 (c + 8); one exact operation more leaves c.  The
// second constant of the first has to be in a register (Magic).
struct Magic {
  uint32_t even = 0x64086408u, odd = 0x64806480u;
  __device__ __forceinline__ void keep() { asm("" : "+v"(even), "+v"(odd)); }
};
template <bool ODD>
__device__ __forceinline__ uint32_t nibbles(uint32_t w, const Magic& g) {
  if constexpr (ODD) {
    const f16x2 v = halves((w & 0x00F000F0u) ^ g.odd);
    const f16x2 k = {(_Float16)0.0625f, (_Float16)0.0625f}, z = {(_Float16)-72.f, (_Float16)-72.f};
    return bits_of(__builtin_elementwise_fma(v, k, z));
  } else {
    const f16x2 v = halves((w & 0x000F000Fu) ^ g.even);
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

// Which elements a lane holds.  Of a key its group of 16 lanes takes every
// fourth piece of up to 16 bytes, so that a load of the wave covers 64
// consecutive bytes of each of 16 tokens: kKeyRuns runs of eight elements to a
// piece.  Of a value it takes pieces of up to 16 bytes, the 16 lanes' side by
// side: kValueRun elements to a piece.
template <int FMT, int D>
constexpr int kKeyRuns = (cache_bytes(FMT, D / 4) < 16 ? cache_bytes(FMT, D / 4) : 16) /
                         cache_bytes(FMT, 8);
template <int FMT, int D>
constexpr int kValueRun = cache_bytes(FMT, D / 16) > 16 ? D / 32 : D / 16;

template <int FMT>
__device__ __forceinline__ Operand key_operand(const uint32_t* w, const Magic& g) {
  if constexpr (FMT == kCacheBF16) {
    return Operand{{w[0], w[1], w[2], w[3]}};
  } else if constexpr (FMT == kCacheInt4) {
    const uint32_t a = w[0], b = a >> 8;
    return Operand{{nibbles<false>(a, g), nibbles<true>(a, g), nibbles<false>(b, g),
                    nibbles<true>(b, g)}};
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
// tokens, w[t] token t's words, and operand i is element i of the eight.  Run
// `h` of operands: those of a word's half (int4) or word.
template <int FMT>
constexpr int kRun = FMT == kCacheBF16 ? 2 : 4;
template <int FMT, int W>
__device__ __forceinline__ void value_operands(const uint32_t (&w)[8][W], int h,
                                               Operand (&out)[kRun<FMT>], const Magic& g) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t(&a)[W] = w[2 * p];
    const uint32_t(&b)[W] = w[2 * p + 1];
    if constexpr (FMT == kCacheInt4) {
      // 16-bit halves of both tokens side by side: four nibbles of each
      const uint32_t x = __builtin_amdgcn_perm(b[h / 2], a[h / 2],
                                               h % 2 ? 0x07060302u : 0x05040100u);
      const uint32_t y = x >> 8;
      out[0].w[p] = nibbles<false>(x, g);
      out[1].w[p] = nibbles<true>(x, g);
      out[2].w[p] = nibbles<false>(y, g);
      out[3].w[p] = nibbles<true>(y, g);
    } else if constexpr (FMT == kCacheBF16) {
      out[0].w[p] = __builtin_amdgcn_perm(b[h], a[h], 0x05040100u);
      out[1].w[p] = __builtin_amdgcn_perm(b[h], a[h], 0x07060302u);
    } else {
      // bytes a0 b0 a1 b1 and a2 b2 a3 b3
      uint32_t x = __builtin_amdgcn_perm(b[h], a[h], 0x05010400u);
      uint32_t y = __builtin_amdgcn_perm(b[h], a[h], 0x07030602u);
      if constexpr (FMT == kCacheInt8) {
        x ^= 0x80808080u;
        y ^= 0x80808080u;
        out[0].w[p] = byte_pair(x, 0x04010400u);
        out[1].w[p] = byte_pair(x, 0x04030402u);
        out[2].w[p] = byte_pair(y, 0x04010400u);
        out[3].w[p] = byte_pair(y, 0x04030402u);
      } else {
        out[0].w[p] = e4m3_pair<false>(x);
        out[1].w[p] = e4m3_pair<true>(x);
        out[2].w[p] = e4m3_pair<false>(y);
        out[3].w[p] = e4m3_pair<true>(y);
      }
    }
  }
}

// BYTES from memory into words, 16 at a time STRIDE bytes apart; two bytes
// leave a word's upper half 0.  NT: memory that is read once.
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
template <bool NT, typename T>
__device__ __forceinline__ T fetched(const char* p) {
  if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
  else return *reinterpret_cast<const T*>(p);
}
template <int BYTES, int STRIDE = 16, bool NT = false>
__device__ __forceinline__ void fetch(const char* p, uint32_t* w) {
  if constexpr (BYTES == 2) {
    w[0] = fetched<NT, uint16_t>(p);
  } else if constexpr (BYTES == 4) {
    w[0] = fetched<NT, uint32_t>(p);
  } else if constexpr (BYTES == 8) {
    const u32x2_t a = fetched<NT, u32x2_t>(p);
    w[0] = a.x, w[1] = a.y;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const u32x4_t a = fetched<NT, u32x4_t>(p + i * STRIDE);
      w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
    }
  }
}

// The four groups of 16 lanes brought together: f of the lanes l, l ^ 16,
// l ^ 32, l ^ 48.  A swap of two copies leaves the even groups (the lower half)
// in one and the odd ones (the upper half) in the other.
template <typename F>
__device__ __forceinline__ float across_groups(float v, F f) {
  const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = f(__uint_as_float(x[0]), __uint_as_float(x[1]));
  const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(y[0]), __uint_as_float(y[1]));
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

// Parts of the queries and of the weights.  With bf16 queries and results one
// fp16 part of each is exact (queries) or off by 2^-11 (a weight, where the
// result's own rounding is 2^-8); a bf16 weight of one part would be off by
// 2^-8 as well, so it has two (2^-15).  fp32 queries or results: 2^-22 of a
// weight, 2^-22 (fp16) or 2^-24 (bf16) of a query.
template <int FMT, bool EXACT>
constexpr int kQueryParts = !EXACT ? 1 : FMT == kCacheBF16 ? 3 : 2;
template <int FMT, bool EXACT>
constexpr int kWeightParts = (FMT == kCacheBF16 ? 2 : 1) + (EXACT ? 1 : 0);

// Which tokens of row `row` a call looks at: [first, end), cut into chunks
// that start at a multiple of 32.
struct Reach {
  int first, end, base;
};
// Words that no one writes during the call, at a uniform index: a scalar load,
// which does not wait for the vector loads in flight.
__device__ __forceinline__ int uniform_word(const int32_t* p, int64_t i) {
  typedef const __attribute__((address_space(4))) int32_t* Constant;
  return ((Constant)(uintptr_t)p)[i];
}
__device__ __forceinline__ Reach reach_of(const AttendParams& P, int len) {
  Reach r;
  r.end = min(max(len, 0), P.max_len);
  r.first = P.window > 0 ? max(0, r.end - P.window) : 0;
  r.base = r.first & ~(kStep - 1);
  return r;
}

// Sum of v over the lanes up to this one.
__device__ __forceinline__ int lanes_before(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // the lane before in its 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // the last of the 16 before
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // lane 31 to the upper half
  return v;
}
// Chunk `at` of all rows' chunks, rows one after the other: its row and which
// of the row's it is; false past the last.
__device__ __forceinline__ bool find_chunk(const AttendParams& P, int chunk, int at, int& row,
                                           int& split) {
  const int lane = threadIdx.x & 63;
  for (int r0 = 0; r0 < (int)P.rows; r0 += 64) {
    int mine = 0;
    if (r0 + lane < (int)P.rows) {
      const Reach r = reach_of(P, P.lens[r0 + lane]);
      mine = (r.end - r.base + chunk - 1) / chunk;
    }
    const int upto = lanes_before(mine);
    const uint64_t past = __ballot(upto > at);
    if (past) {
      const int l = __builtin_ctzll(past);
      row = r0 + l;
      split = at - __builtin_amdgcn_readlane(upto - mine, l);
      return true;
    }
    at -= __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
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

// Whether a step's registers leave none for the queries, which then stay in LDS
// (24 rows of a window of 2047: 15.8 us in registers, 15.3).
template <int FMT, int D>
constexpr bool kQueriesInLds = FMT == kCacheBF16 && D == 256;

// A workgroup of W waves: one row, up to 16 query heads of a key-value head,
// one chunk of the length.  Its waves take steps of 32 tokens in turn.
template <int FMT, int D, bool EXACT, int W, bool NT>
__global__ void __launch_bounds__(64 * W, 2)
    attend_kernel(AttendParams P, int share, int blocks, int splits, int chunk, int packed) {
  constexpr int E = D / 16;                     // a lane's elements of a value
  constexpr int VR = kValueRun<FMT, D>;
  constexpr int QN = kQueryParts<FMT, EXACT>, WN = kWeightParts<FMT, EXACT>;
  constexpr int KB = cache_bytes(FMT, D / 4);   // a lane's bytes of a key
  constexpr int VB = cache_bytes(FMT, E);       // and of a value
  constexpr int KW = KB / 4, VW = VB < 4 ? 1 : VB / 4;
  constexpr int ROW = cache_bytes(FMT, D);
  constexpr bool SCALED = FMT != kCacheBF16;
  constexpr int ROUND = W * kStep;
  // heads whose results are joined at a time, as many as leave room for two
  // workgroups in a CU's 160 KiB (24 rows of a window of 2047, 16 heads of 256:
  // eight heads 15.7 us, sixteen 15.3); of eight waves less (the same: 321 tokens 6.05)
  constexpr int QUERIES = QN * (D / 32) * 64 * 16, EACH = W * (D + 4) * 4;
  constexpr int MOST = ((W > 4 ? 48 : 77) * 1024 - QUERIES) / EACH;
  constexpr int COLS = MOST >= kHeads ? kHeads : MOST >= kHeads / 2 ? kHeads / 2 : kHeads / 4;
  constexpr int SUMS = COLS * EACH;
  __shared__ float factors[W][3][kStep];        // of a step's tokens: ks, log2 vs, 1 / vs
  __shared__ float query_scales[kHeads];
  // a wave may join its results while another has yet to read the queries: they
  // share no memory (a barrier instead: 321 tokens 6.28 us for 6.10)
  constexpr bool IN_LDS = kQueriesInLds<FMT, D>;
  constexpr bool APART = W > 1 || IN_LDS;
  __shared__ __align__(16) char room[APART ? SUMS + QUERIES : SUMS > QUERIES ? SUMS : QUERIES];
  float(*const sums)[COLS][D + 4] = reinterpret_cast<float(*)[COLS][D + 4]>(room);
  Operand(*const queries)[D / 32][64] =
      reinterpret_cast<Operand(*)[D / 32][64]>(room + (APART ? SUMS : 0));

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int col = lane & 15, group = lane >> 4;
  // packed: the y axis counts the chunks that there are, else x goes over the
  // rows too and y over the chunks that there may be
  int x = blockIdx.x, row32 = 0, split = blockIdx.y;
  if (packed) {
    if (!find_chunk(P, chunk, blockIdx.y, row32, split)) return;
  } else if (P.rows > 1) {
    row32 = blockIdx.x / (uint32_t)(P.kv_heads * blocks);
    x -= row32 * (P.kv_heads * blocks);
  }
  const int64_t row = row32;
  const int kvh = blocks == 1 ? x : (uint32_t)x / (uint32_t)blocks, block = x - kvh * blocks;
  const int head0 = kvh * share + block * kHeads;            // the block's first query head
  const int heads = min(kHeads, share - block * kHeads);     // and how many it has
  const int shift = P.page_shift, in_page = (1 << shift) - 1;
  const int32_t* const table = P.tables + row * P.table_width;
  // without a window the first pages are known before the length is
  int early[2] = {0, 0};
  if (P.window == 0) {
    const int t = split * chunk + wave * kStep;
    early[0] = uniform_word(table, min(t >> shift, P.table_width - 1));
    early[1] = uniform_word(table, min((t + 16) >> shift, P.table_width - 1));
  }
  // the queries' elements, eight to a thread: D / 8 lanes to a head
  constexpr int QL = D / 8, QC = (kHeads * QL + 64 * W - 1) / (64 * W);
  uint32_t raw_q[QC][8];
#pragma unroll
  for (int n = 0; n < QC; ++n) {
    const int c = threadIdx.x + n * 64 * W, h = c / QL;
    const int64_t from = row * P.q_stride + (int64_t)(head0 + h) * D + c % QL * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) raw_q[n][i] = 0;
    if (h < heads) {
      if (!EXACT || P.q_bf16) fetch<16>(static_cast<const char*>(P.q) + from * 2, raw_q[n]);
      else fetch<32>(static_cast<const char*>(P.q) + from * 4, raw_q[n]);
    }
  }
  const Reach R = reach_of(P, uniform_word(P.lens, row));
  const int t0 = R.base + split * chunk, t1 = min(R.end, t0 + chunk);
  if (t0 >= t1 && splits > 1) return;           // nothing to add: the join does not look here

  // page of the tile of 16 tokens at t from its table entry, or -1: past the
  // end, or none in the cache
  const auto page_of = [&](int t, int id) {
    return t < t1 && (uint32_t)id < (uint32_t)P.pages ? id : -1;
  };
  const auto entry = [&](int t) { return t < t1 ? uniform_word(table, t >> shift) : -1; };
  // a page's first row of this head; page 0 stands in where there is none
  const auto row_of = [&](int page, int t) {
    return (((int64_t)max(page, 0) * P.kv_heads + kvh) << shift) + (t & in_page);
  };
  const char* const kc = static_cast<const char*>(P.k_cache);
  const char* const vc = static_cast<const char*>(P.v_cache);

  // what a step needs: the next step's keys go out as soon as this one's are
  // used, its values likewise
  uint32_t k[2][KW], v[8][VW];
  uint16_t raw_ks, raw_vs;    // lane t: token t's scales (lanes above 31 repeat them)
  int page[2];
  const bool upper = lane & 16;
  // Of a wave's first tiles the rows in front of what is in reach and behind it
  // are fetched as the first and the last of that: a short sequence touches no
  // row that has no part in it (113 rows of up to 6 tokens of 18 heads of 256
  // bf16 14.0 us without, 9.8).  A long one's last tiles
  // are not worth the registers.
  const auto inside = [&](auto first, int i, int t) {
    if constexpr (!decltype(first)::value) return i;
    return max(min(i, min(max(t1 - 1 - t, 0), 15)), min(max(R.first - t, 0), 15));
  };
  const auto load_keys = [&](auto first, int t) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const char* const p = kc + row_of(page[j], t + 16 * j) * ROW;
      fetch<KB, 64, NT>(p + (uint32_t)(inside(first, col, t + 16 * j) * ROW +
                                       group * (KB < 16 ? KB : 16)), k[j]);
    }
    if constexpr (SCALED) {
      const int64_t r0 = row_of(page[0], t), r1 = row_of(page[1], t + 16);
      const int64_t r = (upper ? r1 : r0) + col;
      raw_ks = P.k_scales[r];
      raw_vs = P.v_scales[r];
    }
  };
  const auto load_values = [&](auto first, int t) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const char* const p = vc + row_of(page[j], t + 16 * j) * ROW;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        fetch<VB, 256, NT>(p + (uint32_t)(inside(first, 4 * group + i, t + 16 * j) * ROW +
                                          col * (VB < 16 ? VB : 16)), v[4 * j + i]);
    }
  };
  int t = t0 + wave * kStep;
  if (t < t1) {
    page[0] = page_of(t, P.window == 0 ? early[0] : entry(t));
    page[1] = page_of(t + 16, P.window == 0 ? early[1] : entry(t + 16));
    load_keys(std::true_type{}, t);
    load_values(std::true_type{}, t);
  }

  // from each thread's eight elements to the operands of the waves
#pragma unroll
  for (int n = 0; n < QC; ++n) {
    const int c = threadIdx.x + n * 64 * W, h = c / QL, chunk8 = c % QL;
    if (n * 64 * W >= heads * QL) break;        // columns behind the heads hold anything
    if (64 * W > kHeads * QL && h >= kHeads) break;
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = EXACT && !P.q_bf16 ? __uint_as_float(raw_q[n][i])
             : (i & 1) ? bf16_hi(raw_q[n][i >> 1]) : bf16_lo(raw_q[n][i >> 1]);
    if constexpr (SCALED) {
      // a power of two that brings the largest element to [2^14, 2^15): fp16
      // then holds every element down to 2^-29 of it with all its bits
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
      top = run_max(top, QL);
      int e = top > 0.f ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
      e = min(max(e, -120), 120);
      const float by = top < __builtin_inff() ? ldexpf(1.f, e) : __builtin_nanf("");
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= by;
      if (chunk8 == 0) query_scales[h] = ldexpf(P.scale * kLog2e, -e);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = fmaf(f[i], 0.f, f[i]);  // an infinity counts as NaN here too
    }
    // the operand and the lane that these eight belong to
    constexpr int KR = kKeyRuns<FMT, D>;
    const int operand = chunk8 / (4 * KR) * KR + chunk8 % KR, to_group = chunk8 / KR % 4;
#pragma unroll
    for (int part = 0; part < QN; ++part) {
      Operand o;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float &x = f[key_order<FMT>(2 * i)], &y = f[key_order<FMT>(2 * i + 1)];
        if constexpr (SCALED) {
          const f32x2_t pair = {x, y};
          const f16x2 r = __builtin_convertvector(pair, f16x2);
          o.w[i] = bits_of(r);
          x -= (float)r.x;
          y -= (float)r.y;
        } else {
          o.w[i] = pack_bf16(x, y);
          x -= bf16_lo(o.w[i]);
          y -= bf16_hi(o.w[i]);
        }
      }
      queries[part][operand][to_group * 16 + h] = o;
    }
  }
  __syncthreads();
  Operand q[IN_LDS ? 1 : QN][IN_LDS ? 1 : D / 32];
  if constexpr (!IN_LDS)
#pragma unroll
    for (int part = 0; part < QN; ++part)
#pragma unroll
      for (int c = 0; c < D / 32; ++c) q[part][c] = queries[part][c][lane];
  const float qscale = SCALED ? query_scales[col] : P.scale * kLog2e;

  Magic magic;
  magic.keep();
  float m = kNone, total = 0.f;
  f32x4 acc[E];
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};

  // the table's entries of the step to load next
  int ids[2] = {entry(t + ROUND), entry(t + ROUND + 16)};
  for (; t < t1; t += ROUND) {
    const int tn = t + ROUND, id[2] = {ids[0], ids[1]};
    ids[0] = entry(tn + ROUND);
    ids[1] = entry(tn + ROUND + 16);
    // a step that has tokens nobody may look at
    const bool edge = t < R.first || t + kStep > t1 || page[0] < 0 || page[1] < 0;

    if constexpr (IN_LDS) wave_lds_sync();      // read again in every step, not kept
    f32x4 s[2] = {};
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      Operand a[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) a[j] = key_operand<FMT>(&k[j][c * kWords8<FMT>], magic);
#pragma unroll
      for (int n = 0; n < QN; ++n) {
        Operand with;
        if constexpr (IN_LDS) with = queries[n][c][lane];
        else with = q[n][c];
#pragma unroll
        for (int j = 0; j < 2; ++j) s[j] = product<FMT>(a[j], with, s[j]);
      }
      if constexpr (IN_LDS) __builtin_amdgcn_sched_barrier(0);  // nor all of them at once
    }
    if constexpr (SCALED) {
      if (lane < kStep) {
        const float ks = (float)__builtin_bit_cast(_Float16, raw_ks);
        // A value scale of 0 stands for a row of codes 0: any scale gives its part
        // of the sums, but a large one raises the maximum that the others' fp16
        // weights are held to.  With 2^-60 a weight has all of its bits while the
        // zero row's is at most 2^82 vs times it: 47 nats beside values of 0.01 in
        // int8 (22 with fp16's least scale, 2^-24, 6 with 1).  Its inverse, in
        // the total, is far from fp32's ends.
        float vs = (float)__builtin_bit_cast(_Float16, raw_vs);
        vs = vs == 0.f ? 0x1p-60f : vs;
        factors[wave][0][lane] = ks;
        factors[wave][1][lane] = __builtin_amdgcn_logf(vs);
        factors[wave][2][lane] = __builtin_amdgcn_rcpf(vs);
      }
    }
    const bool gone[2] = {page[0] < 0, page[1] < 0};
    if (tn < t1) {
      page[0] = page_of(tn, id[0]);
      page[1] = page_of(tn + 16, id[1]);
      load_keys(std::false_type{}, tn);
    }
    float u[8], inv[8];
    if constexpr (SCALED) {
      wave_lds_sync();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const f32x4 ks = *reinterpret_cast<const f32x4*>(&factors[wave][0][16 * j + 4 * group]);
        const f32x4 lv = *reinterpret_cast<const f32x4*>(&factors[wave][1][16 * j + 4 * group]);
        const f32x4 iv = *reinterpret_cast<const f32x4*>(&factors[wave][2][16 * j + 4 * group]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // (the factors first: with the sum first a score within fp32 could pass
          // through an infinity)
          u[4 * j + i] = fmaf(s[j][i], qscale * ks[i], lv[i]);
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
        const int at = t + 16 * (i >> 2) + 4 * group + (i & 3);
        const bool ok = at >= R.first && at < t1 && !gone[i >> 2];
        u[i] = ok ? u[i] : -__builtin_inff();
        if constexpr (SCALED) inv[i] = ok ? inv[i] : 0.f;
        if constexpr (FMT == kCacheBF16 || FMT == kCacheE4M3)
#pragma unroll
          for (int h = 0; h < VW; ++h) v[i][h] = ok ? v[i][h] : 0u;
      }
    }
    // weights are 2^(u - m) with m between 15 below the largest u and 8 below
    // it, so that it seldom moves and fp16 holds them down to 2^-22 of the
    // largest with all bits.  Both are differences from top, exact where they
    // matter: for scores from 2^24 on m + 15 may round to m + 16 and top - 8 to
    // top - 16, and fp16 does not hold 2^16.
    float top = fmaxf(fmaxf(fmaxf(u[0], u[1]), fmaxf(u[2], u[3])),
                      fmaxf(fmaxf(u[4], u[5]), fmaxf(u[6], u[7])));
    if (__any(top - m > 15.f)) {
      top = across_groups(top, [](float a, float b) { return fmaxf(a, b); });
      const float below = top - (top - 8.f) > 15.f ? top : top - 8.f;
      const float to = top - m > 15.f ? below : m;
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
    Operand p[WN];
    weight_parts<FMT, WN>(w, p);
    constexpr int RUN = kRun<FMT>;
#pragma unroll
    for (int h = 0; h < E / RUN; ++h) {
      Operand x[RUN];
      value_operands<FMT, VW>(v, h, x, magic);
#pragma unroll
      for (int i = 0; i < RUN; ++i)
#pragma unroll
        for (int n = 0; n < WN; ++n)
          acc[h * RUN + i] = product<FMT>(x[i], p[n], acc[h * RUN + i]);
    }
    if (tn < t1) load_values(std::false_type{}, tn);
  }

  // the waves' results joined, COLS heads at a time; behind a head's sums its
  // maximum and total
  total = across_groups(total, [](float a, float b) { return a + b; });
#pragma unroll 1
  for (int c0 = 0; c0 < heads; c0 += COLS) {
    if (c0 > 0) __syncthreads();
    // row 4 group + r of operand i's product is a value's element
    if ((uint32_t)(col - c0) < (uint32_t)COLS) {
      float* const to = sums[wave][col - c0];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < E; ++i)
          to[i / VR * 16 * VR + (4 * group + r) * VR + i % VR] = acc[i][r];
      if (group == 0) to[D] = m, to[D + 1] = total;
    }
    __syncthreads();
    const int here = min(COLS, heads - c0);
    for (int i = threadIdx.x; i < here * (D / 4); i += 64 * W) {
      const int x = i / (D / 4), d = i % (D / 4) * 4;
      float top = sums[0][x][D], l = 0.f;
#pragma unroll
      for (int n = 1; n < W; ++n) top = fmaxf(top, sums[n][x][D]);
      f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < W; ++n) {
        const float by = __builtin_amdgcn_exp2f(sums[n][x][D] - top);
        l = fmaf(sums[n][x][D + 1], by, l);
        o += *reinterpret_cast<const f32x4*>(&sums[n][x][d]) * by;
      }
      const int64_t to = row * P.heads + head0 + c0 + x;
      if (splits > 1) {
        Partial<D>* const result = reinterpret_cast<Partial<D>*>(P.partials) + to * splits + split;
        *reinterpret_cast<f32x4*>(&result->y[d]) = o;
        if (d == 0) result->top = top, result->total = l;
      } else {
        put_result(P, to * D + d, o, l);
        if (P.lse && d == 0) P.lse[to] = log_sum(top, l);
      }
    }
  }
}

// The partial results of a row's head joined: a workgroup of N threads to each,
// D / 4 of them to a partial result.  A thread brings what it reads together
// with a maximum of its own; all its loads go out before the length is known.
template <int D, int N>
__global__ void __launch_bounds__(N) join_kernel(AttendParams P, int splits, int chunk) {
  constexpr int L = D / 4, G = N / L, AHEAD = 4;
  __shared__ f32x4 sums[G][L];
  __shared__ float tops[G], totals[G];
  const int64_t to = blockIdx.x;
  const Partial<D>* const part = reinterpret_cast<const Partial<D>*>(P.partials) + to * splits;
  const int g = threadIdx.x / L, d = threadIdx.x % L * 4;
  int used = splits;
  float top = kNone, l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  for (int i0 = g; i0 < used; i0 += AHEAD * G) {
    float2 s[AHEAD];
    f32x4 y[AHEAD];
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      const int i = min(i0 + n * G, splits - 1);
      s[n] = *reinterpret_cast<const float2*>(&part[i].top);
      y[n] = *reinterpret_cast<const f32x4*>(&part[i].y[d]);
    }
    if (i0 == g) {
      const Reach R = reach_of(P, uniform_word(P.lens, blockIdx.x / (uint32_t)P.heads));
      used = (R.end - R.base + chunk - 1) / chunk;
    }
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      if (i0 + n * G >= used) break;
      const float all = fmaxf(top, s[n].x);
      const float was = __builtin_amdgcn_exp2f(top - all), is = __builtin_amdgcn_exp2f(s[n].x - all);
      l = fmaf(s[n].y, is, l * was);
      o = o * was + y[n] * is;
      top = all;
    }
  }
  sums[g][threadIdx.x % L] = o;
  if (threadIdx.x % L == 0) tops[g] = top, totals[g] = l;
  __syncthreads();
  if (g != 0) return;
  float all = tops[0];
#pragma unroll
  for (int i = 1; i < G; ++i) all = fmaxf(all, tops[i]);
  l = 0.f;
  o = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const float by = __builtin_amdgcn_exp2f(tops[i] - all);
    l = fmaf(totals[i], by, l);
    o += sums[i][threadIdx.x % L] * by;
  }
  put_result(P, to * D + d, o, l);
  if (P.lse && threadIdx.x == 0) P.lse[to] = log_sum(all, l);
}

}  // namespace

hipError_t launch_attend(const AttendParams& p, hipStream_t s) {
  const int share = p.heads / p.kv_heads, blocks = attend_blocks(share);
  const int64_t items = p.rows * p.kv_heads * blocks;
  const int reach = attend_reach(p.max_len, p.window);
  const Cut cut = cut_of(p.rows, items, share, p.head_dim, reach);
  const int chunk = cut.chunk, splits = cut.splits;
  // a chunk each of up to 256 rows is looked for among their lengths, so that no
  // workgroup is there for what a short row does not have (64 ragged rows of up
  // to 8192: 45.1 us, 52.8 without)
  const bool packed = splits > 1 && p.rows > 1 && p.rows <= 256 && p.rows * splits < 65536;
  const unsigned across = (unsigned)(p.kv_heads * blocks);
  const dim3 grid = packed ? dim3(across, (unsigned)(p.rows * splits))
                           : dim3((unsigned)items, (unsigned)splits);
  // What the last-level cache (256 MiB) cannot hold until the next call goes
  // past it: 272 MB of one sequence 48.5 us, 53.8 through the caches; 64 ragged
  // rows of up to 553 MB together, 178 as it was, 45.1 and 48.0.  Below, it costs
  // what the cache would have kept (80 MB of up to 272 MB 22.0 us for 19.5).
  // Lengths spread, so of several rows half of what there may be is counted; what
  // several workgroups read, for more than 16 query heads, stays.
  const double bytes = 2.0 * (double)p.rows * p.kv_heads * reach * cache_bytes(p.format, p.head_dim);
  const bool once = blocks == 1 && reach > 128 &&
                    (p.rows > 1 ? bytes / 2 : bytes) >= 256.0 * (1 << 20);
  // Waves of a workgroup that has a row's whole length.  One where there are more
  // rows and heads than the card has room for and their lengths are short: 904
  // items of 32 tokens int8 4.8 us, with four waves 6.9; from 256 tokens on it is
  // the same, 904 items 14.6 and 14.3, 4096 56.0 and 55.3.  Eight where each of up
  // to 256 has a CU to itself and more than one round of four: 256 items of 512
  // tokens 9.2, with four 10.0, of 256 tokens 7.0 and 7.1; but 800 items of 512
  // tokens int4 16.4 and 14.2.  (Pages of their own, three sets of them in turn.)
  const int waves = splits > 1 || once                             ? 4
                    : items > 8 * (int64_t)std::max(reach, kStep) ? 1
                    : reach > 256 && items <= 256                 ? 8
                                                                  : 4;
  const auto go = [&](auto d, auto f, auto exact) {
    constexpr int D = decltype(d)::value, F = decltype(f)::value;
    constexpr bool X = decltype(exact)::value;
    const auto run = [&](auto w, auto nt) {
      constexpr int W2 = decltype(w)::value;
      attend_kernel<F, D, X, W2, decltype(nt)::value>
          <<<grid, 64 * W2, 0, s>>>(p, share, blocks, splits, chunk, packed);
    };
    if (waves == 1) run(std::integral_constant<int, 1>{}, std::false_type{});
    else if (waves == 8) run(std::integral_constant<int, 8>{}, std::false_type{});
    else if (once) run(std::integral_constant<int, 4>{}, std::true_type{});
    else run(std::integral_constant<int, 4>{}, std::false_type{});
  };
  const auto by_type = [&](auto d, auto f) {
    if (p.q_bf16 && p.y_bf16) go(d, f, std::false_type{});
    else go(d, f, std::true_type{});
  };
  const auto by_format = [&](auto d) {
    constexpr int D = decltype(d)::value;
    switch (p.format) {
      case kCacheBF16: by_type(d, std::integral_constant<int, kCacheBF16>{}); break;
      case kCacheInt8: by_type(d, std::integral_constant<int, kCacheInt8>{}); break;
      case kCacheE4M3: by_type(d, std::integral_constant<int, kCacheE4M3>{}); break;
      default: by_type(d, std::integral_constant<int, kCacheInt4>{}); break;
    }
    if (splits > 1) {
      const unsigned results = (unsigned)(p.rows * p.heads);
      if (splits > 16) join_kernel<D, 1024><<<results, 1024, 0, s>>>(p, splits, chunk);
      else join_kernel<D, 256><<<results, 256, 0, s>>>(p, splits, chunk);
    }
  };
  switch (p.head_dim) {
    case 64: by_format(std::integral_constant<int, 64>{}); break;
    case 128: by_format(std::integral_constant<int, 128>{}); break;
    default: by_format(std::integral_constant<int, 256>{}); break;
  }
  return hipGetLastError();
}

}  // namespace bfly
