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
constexpr int kNoAdapter = 0x7FFFFFFF;

// The rows of a block in the order of their adapters, cut into tiles of at
// most kTileRows rows of one adapter; rows without one come last.
struct Tiles {
  int key[kBlockRows];                 // by row; a missing row: kNoAdapter
  uint8_t order[kBlockRows];           // row at every place
  int id[kBlockRows];                  // by tile
  uint16_t start[kBlockRows], len[kBlockRows];
  int count;
};

// Every thread ranks its own row against all the others (the ids are in LDS,
// read as broadcasts): no sort, no atomics, any number of adapters.
__device__ __forceinline__ void make_tiles(Tiles& s, const int32_t* ids, int nr, int n_adapters) {
  __shared__ uint64_t starts[kBlockRows / 64];
  __shared__ uint8_t head[kBlockRows];
  const int i = threadIdx.x;
  int id = kNoAdapter;
  if (i < nr) {
    id = ids[i];
    if (id < 0 || id >= n_adapters) id = kNoAdapter;
  }
  s.key[i] = id;
  __syncthreads();
  int less = 0, before = 0, same = 0;
  for (int j = 0; j < nr; ++j) {
    const int o = s.key[j];
    less += o < id;
    same += o == id;
    before += o == id && j < i;
  }
  const int place = less + before;
  const bool first = i < nr && before % kTileRows == 0;
  if (i < nr) {
    s.order[place] = (uint8_t)i;
    head[place] = first;
  } else {
    head[i] = 0;
  }
  __syncthreads();
  const uint64_t m = __ballot(head[i] != 0);
  if ((i & 63) == 0) starts[i >> 6] = m;
  __syncthreads();
  if (first) {
    int tile = 0;
    for (int w = 0; w < kBlockRows / 64; ++w) {
      const uint64_t b = starts[w];
      if (w < place >> 6) tile += __popcll(b);
      else if (w == place >> 6) tile += __popcll(b & ((1ull << (place & 63)) - 1));
    }
    const int left = same - before;
    s.id[tile] = id;
    s.start[tile] = (uint16_t)place;
    s.len[tile] = (uint16_t)(left < kTileRows ? left : kTileRows);
  }
  if (i == 0) {
    int c = 0;
    for (int w = 0; w < kBlockRows / 64; ++w) c += __popcll(starts[w]);
    s.count = c;
  }
  __syncthreads();
}

__device__ __forceinline__ f32x4 mfma(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// t[split][row][j] = sum over the split's k of A_id[j][k] x[row][k].
// Grid: (blocks of rows, tile lanes, splits * rank blocks).  RT tiles of 16
// ranks, NT of 16 rows at a time; the four waves take every fourth run of 128 k and
// add their sums through LDS.
template <int RT, int NT>
__global__ void __launch_bounds__(kThreads) shrink_kernel(LoraParams P, int splits, int slice,
                                                          int stride) {
  __shared__ Tiles tiles;
  __shared__ f32x4 part[2][RT * NT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int64_t row0 = (int64_t)blockIdx.x * kBlockRows;
  const int nr = P.rows - row0 < kBlockRows ? (int)(P.rows - row0) : kBlockRows;
  const int split = blockIdx.z % splits, rank0 = blockIdx.z / splits * (RT * 16);
  const int kbeg = split * slice, kend = P.k - kbeg < slice ? P.k : kbeg + slice;
  make_tiles(tiles, P.ids + row0, nr, P.n_adapters);
  const __amdgpu_buffer_rsrc_t rx = buffer_range(P.x + row0 * P.k, (int64_t)nr * P.k * 2);
  const int count = tiles.count;
  for (int tile = blockIdx.y; tile < count; tile += gridDim.y) {
    const int id = __builtin_amdgcn_readfirstlane(tiles.id[tile]);
    if (id == kNoAdapter) break;  // the rows without an adapter come last
    const int start = __builtin_amdgcn_readfirstlane((int)tiles.start[tile]);
    const int all = __builtin_amdgcn_readfirstlane((int)tiles.len[tile]);
    const __amdgpu_buffer_rsrc_t ra =
        buffer_range(P.a + ((int64_t)id * P.rank + rank0) * P.k, (int64_t)(P.rank - rank0) * P.k * 2);
    uint32_t ao[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) ao[j] = (uint32_t)(j * 16 + n) * (uint32_t)P.k * 2u;
    for (int first = 0; first < all; first += NT * 16) {
      const int len = all - first;  // NT * 16 of them at most are taken here
      uint32_t xo[NT];
      int row[NT];
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        const int at = q * 16 + n;
        row[q] = at < len ? tiles.order[start + first + at] : -1;
        xo[q] = (uint32_t)row[q] * (uint32_t)P.k * 2u;
      }
      f32x4 acc[RT][NT];
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int q = 0; q < NT; ++q) acc[j][q] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int kc = kbeg + wave * 128; kc < kend; kc += 512) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int kk = kc + u * 32 + g * 8;
          const bool in = kk < kend;
          uint4 fa[RT];
#pragma unroll
          for (int j = 0; j < RT; ++j) fa[j] = buf_ld16(ra, in ? ao[j] + 2u * kk : kOutOfRange);
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            if (q * 16 < len) {
              const uint4 fx = buf_ld16(rx, in && row[q] >= 0 ? xo[q] + 2u * kk : kOutOfRange);
#pragma unroll
              for (int j = 0; j < RT; ++j) acc[j][q] = mfma(fa[j], fx, acc[j][q]);
            }
          }
        }
      }
      // waves 2 and 3 to 0 and 1, then 1 to 0
      __syncthreads();  // the turn before has read `part`
      if (wave >= 2) {
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int q = 0; q < NT; ++q) part[wave - 2][j * NT + q][lane] = acc[j][q];
      }
      __syncthreads();
      if (wave < 2) {
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int q = 0; q < NT; ++q) acc[j][q] += part[wave][j * NT + q][lane];
      }
      if (wave == 1) {
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int q = 0; q < NT; ++q) part[1][j * NT + q][lane] = acc[j][q];
      }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          if (row[q] < 0) continue;
          float* const to =
              P.t + ((int64_t)split * P.rows + row0 + row[q]) * stride + rank0 + 4 * g;
#pragma unroll
          for (int j = 0; j < RT; ++j)
            *reinterpret_cast<f32x4*>(to + 16 * j) = acc[j][q] + part[1][j * NT + q][lane];
        }
      }
    }
  }
}

// y = base + B_id (s_id t).  Grid: (column tiles, blocks of rows).  The
// matrix cores' rows are columns of y, in an order that leaves eight
// consecutive columns of one row of y to a lane: tile j of a pair takes column
// 8 (m / 4) + 4 j + m % 4 of a run of 32 as its row m.
constexpr int kCols = 256;  // columns of a workgroup, 64 to a wave
template <int TERMS, bool BB, bool YB>
__global__ void __launch_bounds__(kThreads) expand_kernel(LoraParams P, int splits, int stride,
                                                          int depth, int tile_rows) {
  __shared__ Tiles tiles;
  extern __shared__ __align__(16) uint16_t terms[];  // [TERMS][tile_rows][depth + 8]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int64_t row0 = (int64_t)blockIdx.y * kBlockRows;
  const int nr = P.rows - row0 < kBlockRows ? (int)(P.rows - row0) : kBlockRows;
  const int col0 = blockIdx.x * kCols + wave * 64;
  const int pitch = depth + 8;
  make_tiles(tiles, P.ids + row0, nr, P.n_adapters);
  constexpr int bs = BB ? 2 : 4, ys = YB ? 2 : 4;
  const __amdgpu_buffer_rsrc_t rbase =
      buffer_range(static_cast<const char*>(P.base) + row0 * P.n_out * bs,
                   P.base ? (int64_t)nr * P.n_out * bs : 0);
  const __amdgpu_buffer_rsrc_t ry =
      buffer_range(static_cast<char*>(P.y) + row0 * P.n_out * ys, (int64_t)nr * P.n_out * ys);
  const int count = tiles.count;
  for (int tile = 0; tile < count; ++tile) {
    const int id = __builtin_amdgcn_readfirstlane(tiles.id[tile]);
    const bool none = id == kNoAdapter;
    if (none && P.base == P.y) break;  // in place: those rows stay as they are
    const int start = __builtin_amdgcn_readfirstlane((int)tiles.start[tile]);
    const int all = __builtin_amdgcn_readfirstlane((int)tiles.len[tile]);
    const __amdgpu_buffer_rsrc_t rb = none
        ? buffer_range32(nullptr, 0)
        : buffer_range(P.b + (int64_t)id * P.n_out * P.rank, (int64_t)P.n_out * P.rank * 2);
    for (int part = 0; part < all; part += tile_rows) {
      const int len = all - part < tile_rows ? all - part : tile_rows;
      if (!none) {
        // the terms of s t, four ranks to a thread at a time
        const float s = P.scaling[id];
        __syncthreads();
        const int quads = depth / 4;
        for (int i = threadIdx.x; i < len * quads; i += kThreads) {
          const int r = i / quads, c = i % quads * 4;
          f32x4 v = {0.f, 0.f, 0.f, 0.f};
          if (c < stride) {
            const float* from = P.t + (row0 + tiles.order[start + part + r]) * stride + c;
            for (int k = 0; k < splits; ++k)
              v += *reinterpret_cast<const f32x4*>(from + k * P.rows * stride);
            v *= s;
          }
#pragma unroll
          for (int q = 0; q < TERMS; ++q) {
            const uint32_t lo = pack_bf16(v.x, v.y), hi = pack_bf16(v.z, v.w);
            *reinterpret_cast<uint2*>(terms + (q * tile_rows + r) * pitch + c) = make_uint2(lo, hi);
            v -= f32x4{bf16_lo(lo), bf16_hi(lo), bf16_lo(hi), bf16_hi(hi)};
          }
        }
        __syncthreads();
      }
      for (int c32 = 0; c32 < 64; c32 += 32) {
        const int c0 = col0 + c32;
        if (c0 >= P.n_out) break;
        for (int q = 0; q < len; q += 16) {
          f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
          if (!none) {
            for (int d = 0; d < depth; d += 32) {
              const int r = d + 8 * g;
              uint4 fb[2];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int c = c0 + 8 * (n >> 2) + 4 * j + (n & 3);
                fb[j] = buf_ld16(rb, r < P.rank && c < P.n_out
                                         ? ((uint32_t)c * (uint32_t)P.rank + r) * 2u
                                         : kOutOfRange);
              }
#pragma unroll
              for (int k = 0; k < TERMS; ++k) {
                const int at = q + n < len ? q + n : len - 1;
                const uint4 ft = *reinterpret_cast<const uint4*>(
                    terms + (k * tile_rows + at) * pitch + r);
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[j] = mfma(fb[j], ft, acc[j]);
              }
            }
          }
          // lane: row q + n, columns c0 + 8 g .. + 7
          const int c = c0 + 8 * g;
          const bool in = q + n < len && c < P.n_out;
          const uint32_t at = in ? (uint32_t)tiles.order[start + part + q + n] * (uint32_t)P.n_out +
                                       (uint32_t)c
                                 : 0u;
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = acc[e >> 2][e & 3];
          if (P.base) {
            if constexpr (BB) {
              const uint4 w = buf_ld16(rbase, in ? at * 2u : kOutOfRange);
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] += (e & 1) ? bf16_hi(ww[e >> 1]) : bf16_lo(ww[e >> 1]);
            } else {
              const uint4 w0 = buf_ld16(rbase, in ? at * 4u : kOutOfRange);
              const uint4 w1 = buf_ld16(rbase, in ? at * 4u + 16u : kOutOfRange);
              const uint32_t ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] += __uint_as_float(ww[e]);
            }
          }
          if constexpr (YB) {
            buf_st16(ry, in ? at * 2u : kOutOfRange,
                     make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])));
          } else {
            buf_st16(ry, in ? at * 4u : kOutOfRange,
                     make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                __float_as_uint(v[2]), __float_as_uint(v[3])));
            buf_st16(ry, in ? at * 4u + 16u : kOutOfRange,
                     make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]),
                                __float_as_uint(v[6]), __float_as_uint(v[7])));
          }
        }
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
  int lanes;     // shrink workgroups that share a block's tiles
  int splits, slice;  // of the k axis
};
Cut cut(int64_t rows, int k, int rank) {
  Cut c;
  c.rt = rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8;
  c.ranks = (rank + 16 * c.rt - 1) / (16 * c.rt);
  c.stride = c.ranks * c.rt * 16;
  c.blocks = (rows + kBlockRows - 1) / kBlockRows;
  c.lanes = c.blocks > 1 ? 4 : (int)(rows < 16 ? rows : 16);
  const int64_t groups = c.blocks * c.lanes * c.ranks;
  const int most = (k + 511) / 512;
  const int64_t want = (768 + groups - 1) / groups;
  c.splits = (int)(want < most ? want : most);
  c.slice = ((k + c.splits - 1) / c.splits + 127) / 128 * 128;
  c.splits = (k + c.slice - 1) / c.slice;
  return c;
}

template <int RT, int NT>
void shrink(const LoraParams& p, const Cut& c, hipStream_t s) {
  hipLaunchKernelGGL((shrink_kernel<RT, NT>),
                     dim3((unsigned)c.blocks, c.lanes, c.splits * c.ranks), dim3(kThreads), 0, s, p,
                     c.splits, c.slice, c.stride);
}

template <int TERMS, bool BB, bool YB>
void expand(const LoraParams& p, const Cut& c, hipStream_t s) {
  const int depth = (c.stride + 31) / 32 * 32;
  const int tile_rows = depth > 128 ? 32 : 64;
  hipLaunchKernelGGL((expand_kernel<TERMS, BB, YB>),
                     dim3((p.n_out + kCols - 1) / kCols, (unsigned)c.blocks), dim3(kThreads),
                     TERMS * tile_rows * (depth + 8) * sizeof(uint16_t), s, p, c.splits, c.stride,
                     depth, tile_rows);
}

}  // namespace

size_t lora_workspace_bytes(int64_t rows, int k, int rank) {
  const Cut c = cut(rows, k, rank);
  return (size_t)c.splits * (size_t)rows * (size_t)c.stride * sizeof(float);
}

hipError_t launch_lora(const LoraParams& p, hipStream_t s) {
  const Cut c = cut(p.rows, p.k, p.rank);
  switch (c.rt) {
    case 1: shrink<1, 4>(p, c, s); break;
    case 2: shrink<2, 4>(p, c, s); break;
    case 4: shrink<4, 4>(p, c, s); break;
    default: shrink<8, 2>(p, c, s); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.y_bf16) {
    if (p.base_bf16) expand<2, true, true>(p, c, s);
    else expand<2, false, true>(p, c, s);
  } else {
    if (p.base_bf16) expand<3, true, false>(p, c, s);
    else expand<3, false, false>(p, c, s);
  }
  return hipGetLastError();
}

}  // namespace bfly
