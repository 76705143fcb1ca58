// Low-rank adapters of many requests beside a shared product:
//
//   y[r] = base[r] + s_id * B_id (A_id x[r]),  id = ids[r]  (none: y[r] = base[r])
//
// Two launches.  shrink: t = A_id x in fp32, the k axis split over workgroups
// when there are few rows (their partial sums are added in a fixed order by
// the second launch).  expand: y = base + B_id (s_id t).  Both on the matrix
// cores; rows of one adapter share a tile, whatever their order in the batch.
//
// s_id t is fp32 and goes through the bf16 matrix cores as a sum of bf16
// terms, each the rounding of what the ones before left: two terms (2^-16 of t
// is lost at worst) where y is bf16, three (2^-24) where it is fp32.
#include "bfly_lora.h"
#include "bfly_rows.h"

#include <type_traits>

namespace bfly {
namespace {

typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kBlockRows = 256;  // rows whose order a workgroup works out
constexpr int kTileRows = 64;    // rows of one adapter in a tile at most
constexpr int kNoAdapter = kLoraMaxAdapters;

// The rows of a block in the order of their adapters, cut into tiles of at
// most kTileRows rows of one adapter; rows without one come last.
struct Tiles {
  uint32_t key[kBlockRows];    // by row, adapter * 256 + row; a missing row: the largest value
  uint32_t sorted[kBlockRows];  // the keys in their order
  uint64_t heads[kBlockRows / 64];  // places where a tile begins
  uint64_t runs[kBlockRows / 64];   // places where an adapter's rows begin
  uint16_t start[kBlockRows];  // by tile: its first place
  int count;
  __device__ int row(int place) const { return (int)(sorted[place] & 255u); }
  __device__ int id(int place) const { return (int)(sorted[place] >> 8); }
};

// Every thread ranks its own row against all the others (the keys are in LDS,
// read four at a time as broadcasts): no sort, no atomics, and any ids.
__device__ __forceinline__ void make_tiles(Tiles& s, const int32_t* ids, int nr, int n_adapters) {
  const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
  uint32_t key = ~0u;
  if (i < nr) {
    const int id = ids[i];
    key = (uint32_t)(id >= 0 && id < n_adapters ? id : kNoAdapter) << 8 | (uint32_t)i;
  }
  s.key[i] = key;
  __syncthreads();
  int place = 0;
#pragma unroll 4
  for (int j = 0; j < nr; j += 4) {  // past nr: the largest value, never below
    const uint4 o = *reinterpret_cast<const uint4*>(s.key + j);
    place += (o.x < key) + (o.y < key) + (o.z < key) + (o.w < key);
  }
  if (i < nr) s.sorted[place] = key;
  __syncthreads();
  const uint32_t mine = i < nr ? s.sorted[i] >> 8 : ~0u;
  const uint32_t left = i > 0 && i < nr ? s.sorted[i - 1] >> 8 : ~0u;
  const uint64_t runs = __ballot(i < nr && mine != left);
  if (lane == 0) s.runs[wave] = runs;
  __syncthreads();
  // the first place of this place's adapter: the last run mark not beyond it
  int first = 0;
  for (int w = 0; w <= wave; ++w) {
    const uint64_t m = w < wave ? s.runs[w] : runs & (~0ull >> (63 - lane));
    if (m) first = w * 64 + 63 - __clzll((long long)m);
  }
  const bool head = i < nr && ((i - first) & (kTileRows - 1)) == 0;
  const uint64_t heads = __ballot(head);
  if (lane == 0) s.heads[wave] = heads;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kBlockRows / 64; ++w) {
    const int c = __popcll(s.heads[w]);
    before += w < wave ? c : 0;
    all += c;
  }
  if (head) s.start[before + __popcll(heads & ((1ull << lane) - 1))] = (uint16_t)i;
  if (i == 0) s.count = all;
  __syncthreads();
}
// First place, number of rows and adapter of a tile, uniform over the wave.
struct Tile {
  int start, len, id;
};
__device__ __forceinline__ Tile tile_at(const Tiles& s, int tile, int nr) {
  Tile t;
  t.start = __builtin_amdgcn_readfirstlane((int)s.start[tile]);
  const int end = tile + 1 < s.count ? (int)s.start[tile + 1] : nr;
  t.len = __builtin_amdgcn_readfirstlane(end) - t.start;
  t.id = __builtin_amdgcn_readfirstlane(s.id(t.start));
  return t;
}

__device__ __forceinline__ f32x4 mfma(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// t[split][row][j] = sum over the split's k of A_id[j][k] x[row][k].
// Grid: (blocks of rows, tile lanes, splits * rank blocks).  RT tiles of 16
// ranks; the four waves take every fourth run of 128 k and add their sums
// through LDS.
template <int RT>
struct ShrinkArgs {
  __amdgpu_buffer_rsrc_t rx, ra;  // the block's rows of x, the adapter's rows of A
  const Tiles* tiles;
  float* t;      // the split's sums of the block's first row, at the rank block
  f32x4* part;   // LDS [2][RT * NT][64]
  int k, kbeg, kend, stride;
};

// NT * 16 rows of a tile (`len` of them, the others read as zeros).  The loop
// has no branch around its loads: all of a run's loads are in flight together.
template <int RT, int NT>
__device__ __forceinline__ void shrink_rows(const ShrinkArgs<RT>& P, int start, int len) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  uint32_t xo[NT], ao[RT];
  int row[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int at = q * 16 + n;
    row[q] = at < len ? P.tiles->row(start + at) : -1;
    xo[q] = row[q] >= 0 ? (uint32_t)row[q] * (uint32_t)P.k * 2u : kOutOfRange;
  }
#pragma unroll
  for (int j = 0; j < RT; ++j) ao[j] = (uint32_t)(j * 16 + n) * (uint32_t)P.k * 2u;
  f32x4 acc[RT][NT];
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int q = 0; q < NT; ++q) acc[j][q] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int kc = P.kbeg + wave * 128; kc < P.kend; kc += 512) {
    uint4 fa[4][RT], fx[4][NT];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int kk = kc + u * 32 + g * 8;
      const bool in = kk < P.kend;
#pragma unroll
      for (int q = 0; q < NT; ++q)
        fx[u][q] = buf_ld16(P.rx, in && row[q] >= 0 ? xo[q] + 2u * kk : kOutOfRange);
#pragma unroll
      for (int j = 0; j < RT; ++j) fa[u][j] = buf_ld16(P.ra, in ? ao[j] + 2u * kk : kOutOfRange);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[j][q] = mfma(fa[u][j], fx[u][q], acc[j][q]);
  }
  // waves 2 and 3 to 0 and 1, then 1 to 0
  constexpr int half = RT * NT * 64;
  __syncthreads();  // the turn before has read `part`
  if (wave >= 2) {
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int q = 0; q < NT; ++q) P.part[(wave - 2) * half + (j * NT + q) * 64 + lane] = acc[j][q];
  }
  __syncthreads();
  if (wave < 2) {
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int q = 0; q < NT; ++q) acc[j][q] += P.part[wave * half + (j * NT + q) * 64 + lane];
  }
  if (wave == 1) {
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int q = 0; q < NT; ++q) P.part[half + (j * NT + q) * 64 + lane] = acc[j][q];
  }
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      if (row[q] < 0) continue;
      float* const to = P.t + (int64_t)row[q] * P.stride + 4 * g;
#pragma unroll
      for (int j = 0; j < RT; ++j)
        *reinterpret_cast<f32x4*>(to + 16 * j) =
            acc[j][q] + P.part[half + (j * NT + q) * 64 + lane];
    }
  }
}

template <int RT>
__global__ void __launch_bounds__(kThreads) shrink_kernel(LoraParams P, int splits, int slice,
                                                          int stride) {
  constexpr int NT = RT == 8 ? 2 : 4;  // 16-row tiles at a time at most
  __shared__ Tiles tiles;
  __shared__ f32x4 part[2 * RT * NT * 64];
  const int64_t row0 = (int64_t)blockIdx.x * kBlockRows;
  const int nr = P.rows - row0 < kBlockRows ? (int)(P.rows - row0) : kBlockRows;
  const int split = blockIdx.z % splits, rank0 = blockIdx.z / splits * (RT * 16);
  make_tiles(tiles, P.ids + row0, nr, P.n_adapters);
  ShrinkArgs<RT> a;
  a.rx = buffer_range(P.x + row0 * P.k, (int64_t)nr * P.k * 2);
  a.tiles = &tiles;
  a.t = P.t + ((int64_t)split * P.rows + row0) * stride + rank0;
  a.part = part;
  a.k = P.k;
  a.kbeg = split * slice;
  a.kend = P.k - a.kbeg < slice ? P.k : a.kbeg + slice;
  a.stride = stride;
  const int count = tiles.count;
  for (int tile = blockIdx.y; tile < count; tile += gridDim.y) {
    const Tile t = tile_at(tiles, tile, nr);
    if (t.id == kNoAdapter) break;  // the rows without an adapter come last
    a.ra = buffer_range(P.a + ((int64_t)t.id * P.rank + rank0) * P.k,
                        (int64_t)(P.rank - rank0) * P.k * 2);
    for (int first = 0; first < t.len; first += NT * 16) {
      const int len = t.len - first;
      if (len <= 16) shrink_rows<RT, 1>(a, t.start + first, len);
      else if (len <= 32 || NT == 2) shrink_rows<RT, 2>(a, t.start + first, len);
      else shrink_rows<RT, NT>(a, t.start + first, len);
    }
  }
}

// y = base + B_id (s_id t).  Grid: (column tiles, blocks of rows, tile lanes).
// The matrix cores' rows are columns of y, in an order that leaves eight
// consecutive columns of one row of y to a lane: tile j of a pair takes column
// 8 (m / 4) + 4 j + m % 4 of a run of 32 as its row m.  DK: runs of 32 ranks.
// CG: runs of 32 columns to a wave, the next one's loads ahead of this one's
// products.
template <int TERMS, bool BB, bool YB, int DK, int CG>
struct Expand {
  static constexpr int QN = DK == 8 ? 2 : 4;  // 16-row tiles at a time
  static constexpr int kRows = QN * 16;
  static constexpr int kDepth = DK * 32;
  static constexpr int kPitch = kDepth + 8;
  static constexpr int kCols = 128 * CG;
  struct Frag {
    uint4 b[2][DK];
    uint4 base[QN][BB ? 1 : 2];
  };
  static __device__ __forceinline__ void load(const LoraParams& P, __amdgpu_buffer_rsrc_t rb,
                                              __amdgpu_buffer_rsrc_t rbase,
                                              const uint32_t (&ro)[QN], int c0, bool none, Frag& f) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    if (!none) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = c0 + 8 * (n >> 2) + 4 * j + (n & 3);
#pragma unroll
        for (int d = 0; d < DK; ++d) {
          const int r = d * 32 + 8 * g;
          f.b[j][d] = buf_ld16(rb, r < P.rank && c < P.n_out
                                       ? ((uint32_t)c * (uint32_t)P.rank + r) * 2u
                                       : kOutOfRange);
        }
      }
    }
    if (P.base) {
      const int c = c0 + 8 * g;
#pragma unroll
      for (int q = 0; q < QN; ++q) {
        const bool in = ro[q] != kOutOfRange && c < P.n_out;
        const uint32_t at = (ro[q] + (uint32_t)c) * (BB ? 2u : 4u);
        f.base[q][0] = buf_ld16(rbase, in ? at : kOutOfRange);
        if constexpr (!BB) f.base[q][1] = buf_ld16(rbase, in ? at + 16u : kOutOfRange);
      }
    }
  }
  static __device__ __forceinline__ void finish(const LoraParams& P, __amdgpu_buffer_rsrc_t ry,
                                                const uint16_t* terms, const uint32_t (&ro)[QN],
                                                int c0, int len, bool none, const Frag& f) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int c = c0 + 8 * g;
#pragma unroll
    for (int q = 0; q < QN; ++q) {
      if (q * 16 >= len) break;
      f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      if (!none) {
        const int at = q * 16 + n < len ? q * 16 + n : len - 1;
#pragma unroll
        for (int d = 0; d < DK; ++d)
#pragma unroll
          for (int k = 0; k < TERMS; ++k) {
            const uint4 ft =
                *reinterpret_cast<const uint4*>(terms + (k * kRows + at) * kPitch + d * 32 + 8 * g);
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[j] = mfma(f.b[j][d], ft, acc[j]);
          }
      }
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = acc[e >> 2][e & 3];
      if (P.base) {
        const uint4 w0 = f.base[q][0], w1 = f.base[q][BB ? 0 : 1];
        const uint32_t ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] += !BB ? __uint_as_float(ww[e]) : (e & 1) ? bf16_hi(ww[e >> 1]) : bf16_lo(ww[e >> 1]);
      }
      const bool in = ro[q] != kOutOfRange && c < P.n_out;
      const uint32_t to = (ro[q] + (uint32_t)c) * (YB ? 2u : 4u);
      if constexpr (YB) {
        buf_st16(ry, in ? to : kOutOfRange,
                 make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                            pack_bf16(v[6], v[7])));
      } else {
        buf_st16(ry, in ? to : kOutOfRange,
                 make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                            __float_as_uint(v[3])));
        buf_st16(ry, in ? to + 16u : kOutOfRange,
                 make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                            __float_as_uint(v[7])));
      }
    }
  }
};

template <int TERMS, bool BB, bool YB, int DK, int CG>
__global__ void __launch_bounds__(kThreads) expand_kernel(LoraParams P, int splits, int stride) {
  using E = Expand<TERMS, BB, YB, DK, CG>;
  __shared__ Tiles tiles;
  __shared__ __align__(16) uint16_t terms[TERMS * E::kRows * E::kPitch];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t row0 = (int64_t)blockIdx.y * kBlockRows;
  const int nr = P.rows - row0 < kBlockRows ? (int)(P.rows - row0) : kBlockRows;
  const int col0 = blockIdx.x * E::kCols + wave * 32 * CG;
  make_tiles(tiles, P.ids + row0, nr, P.n_adapters);
  constexpr int bs = BB ? 2 : 4, ys = YB ? 2 : 4;
  const __amdgpu_buffer_rsrc_t rbase =
      buffer_range(static_cast<const char*>(P.base) + row0 * P.n_out * bs,
                   P.base ? (int64_t)nr * P.n_out * bs : 0);
  const __amdgpu_buffer_rsrc_t ry =
      buffer_range(static_cast<char*>(P.y) + row0 * P.n_out * ys, (int64_t)nr * P.n_out * ys);
  const int count = tiles.count;
  for (int tile = blockIdx.z; tile < count; tile += gridDim.z) {
    const Tile t = tile_at(tiles, tile, nr);
    const bool none = t.id == kNoAdapter;
    if (none && P.base == P.y) break;  // in place: those rows stay as they are
    const __amdgpu_buffer_rsrc_t rb = none
        ? buffer_range32(nullptr, 0)
        : buffer_range(P.b + (int64_t)t.id * P.n_out * P.rank, (int64_t)P.n_out * P.rank * 2);
    for (int part = 0; part < t.len; part += E::kRows) {
      const int len = t.len - part < E::kRows ? t.len - part : E::kRows;
      uint32_t ro[E::QN];
#pragma unroll
      for (int q = 0; q < E::QN; ++q) {
        const int at = q * 16 + (lane & 15);
        ro[q] = at < len ? (uint32_t)tiles.row(t.start + part + at) * (uint32_t)P.n_out
                         : kOutOfRange;
      }
      typename E::Frag f[CG];
      E::load(P, rb, rbase, ro, col0, none, f[0]);
      if (!none) {
        // the terms of s t, four ranks to a thread at a time
        const float s = P.scaling[t.id];
        __syncthreads();  // the turn before has read them
        for (int i = threadIdx.x; i < len * (E::kDepth / 4); i += kThreads) {
          const int r = i / (E::kDepth / 4), c = i % (E::kDepth / 4) * 4;
          f32x4 v = {0.f, 0.f, 0.f, 0.f};
          if (c < stride) {
            const float* from = P.t + (row0 + tiles.row(t.start + part + r)) * stride + c;
#pragma unroll 4
            for (int k = 0; k < splits; ++k)
              v += *reinterpret_cast<const f32x4*>(from + k * P.rows * stride);
            v *= s;
          }
#pragma unroll
          for (int q = 0; q < TERMS; ++q) {
            const uint32_t lo = pack_bf16(v.x, v.y), hi = pack_bf16(v.z, v.w);
            *reinterpret_cast<uint2*>(terms + (q * E::kRows + r) * E::kPitch + c) =
                make_uint2(lo, hi);
            v -= f32x4{bf16_lo(lo), bf16_hi(lo), bf16_lo(hi), bf16_hi(hi)};
          }
        }
        __syncthreads();
      }
#pragma unroll
      for (int cg = 0; cg < CG; ++cg) {
        if (cg + 1 < CG) E::load(P, rb, rbase, ro, col0 + 32 * (cg + 1), none, f[cg + 1]);
        E::finish(P, ry, terms, ro, col0 + 32 * cg, len, none, f[cg]);
      }
    }
  }
}

// How a call is cut up: a function of the sizes only.
struct Cut {
  int rt;        // tiles of 16 ranks in a shrink workgroup
  int ranks;     // rank blocks of 16 rt
  int stride;    // floats of a row of t
  int64_t blocks;  // blocks of rows
  int splits, slice;  // of the k axis
};
// Workgroups that share a block's tiles: as many as it can have tiles, up to
// a number that leaves few of them idle when there are many blocks.
int tile_lanes(int64_t rows, int64_t blocks, int n_adapters) {
  const int64_t r = rows < kBlockRows ? rows : kBlockRows;
  const int64_t most = (r < n_adapters ? r : n_adapters) + r / kTileRows + 1;
  const int64_t cap = blocks <= 2 ? 32 : blocks <= 8 ? 16 : 4;
  return (int)(most < cap ? most : cap);
}
Cut cut(int64_t rows, int k, int rank) {
  Cut c;
  c.rt = rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8;
  c.ranks = (rank + 16 * c.rt - 1) / (16 * c.rt);
  c.stride = c.ranks * c.rt * 16;
  c.blocks = (rows + kBlockRows - 1) / kBlockRows;
  // tiles there are at least: one to 64 rows
  const int64_t groups = (rows + kTileRows - 1) / kTileRows * c.ranks;
  const int most = (k + 511) / 512;
  const int64_t want = (512 + groups - 1) / groups;
  c.splits = (int)(want < most ? want : most);
  c.slice = ((k + c.splits - 1) / c.splits + 127) / 128 * 128;
  c.splits = (k + c.slice - 1) / c.slice;
  return c;
}

template <int RT>
void shrink(const LoraParams& p, const Cut& c, hipStream_t s) {
  hipLaunchKernelGGL((shrink_kernel<RT>),
                     dim3((unsigned)c.blocks, tile_lanes(p.rows, c.blocks, p.n_adapters),
                          c.splits * c.ranks),
                     dim3(kThreads), 0, s, p, c.splits, c.slice, c.stride);
}

template <int TERMS, bool BB, bool YB, int DK, int CG>
void expand(const LoraParams& p, const Cut& c, hipStream_t s) {
  using E = Expand<TERMS, BB, YB, DK, CG>;
  // few rows: a workgroup to a tile; many: a workgroup to a block
  const int lanes = c.blocks <= 8 ? tile_lanes(p.rows, c.blocks, p.n_adapters) : 1;
  hipLaunchKernelGGL((expand_kernel<TERMS, BB, YB, DK, CG>),
                     dim3((p.n_out + E::kCols - 1) / E::kCols, (unsigned)c.blocks, lanes),
                     dim3(kThreads), 0, s, p, c.splits, c.stride);
}
template <int TERMS, bool BB, bool YB, int DK>
void expand_cg(const LoraParams& p, const Cut& c, hipStream_t s) {
  if (c.blocks <= 8) expand<TERMS, BB, YB, DK, 1>(p, c, s);
  else expand<TERMS, BB, YB, DK, 2>(p, c, s);
}
template <int TERMS, bool BB, bool YB>
void expand_dk(const LoraParams& p, const Cut& c, hipStream_t s) {
  if (c.stride <= 32) expand_cg<TERMS, BB, YB, 1>(p, c, s);
  else if (c.stride <= 64) expand_cg<TERMS, BB, YB, 2>(p, c, s);
  else if (c.stride <= 128) expand_cg<TERMS, BB, YB, 4>(p, c, s);
  else expand_cg<TERMS, BB, YB, 8>(p, c, s);
}

}  // namespace

size_t lora_workspace_bytes(int64_t rows, int k, int rank) {
  const Cut c = cut(rows, k, rank);
  return (size_t)c.splits * (size_t)rows * (size_t)c.stride * sizeof(float);
}

hipError_t launch_lora(const LoraParams& p, hipStream_t s) {
  const Cut c = cut(p.rows, p.k, p.rank);
  switch (c.rt) {
    case 1: shrink<1>(p, c, s); break;
    case 2: shrink<2>(p, c, s); break;
    case 4: shrink<4>(p, c, s); break;
    default: shrink<8>(p, c, s); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.y_bf16) {
    if (p.base_bf16) expand_dk<2, true, true>(p, c, s);
    else expand_dk<2, false, true>(p, c, s);
  } else {
    if (p.base_bf16) expand_dk<3, true, false>(p, c, s);
    else expand_dk<3, false, false>(p, c, s);
  }
  return hipGetLastError();
}

}  // namespace bfly
