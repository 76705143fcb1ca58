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
// is lost at worst) where y is bf16, three (2^-24) where it is fp32.  An
// infinity of B times a term of zero or of the other sign would leave NaN where
// the formula has an infinity: infinities of B enter the products as +-2^-100
// and their own products with t are added to y afterwards.  (A NaN is right as
// it is.)
#include "bfly_lora.h"
#include "bfly_rows.h"

namespace bfly {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kBlockRows = 256;  // rows whose order a workgroup works out
constexpr int kTileRows = 64;    // rows of one adapter in a tile at most
constexpr int kNoAdapter = kLoraMaxAdapters;

// The rows of a block in the order of their adapters, cut into tiles of at
// most kTileRows rows of one adapter; rows without one come last.
struct Tiles {
  __align__(16) uint32_t key[kBlockRows];  // by row, adapter * 256 + row; missing: the largest
  uint32_t sorted[kBlockRows];             // the keys in their order
  uint64_t runs[kBlockRows / 64];          // places where an adapter's rows begin
  uint64_t ordered[kBlockRows / 64];       // rows whose key is not below the one before
  uint16_t start[kBlockRows];              // by tile: its first place
  int count;
  __device__ int row(int place) const { return (int)(sorted[place] & 255u); }
  __device__ int id(int place) const { return (int)(sorted[place] >> 8); }
};

__device__ __forceinline__ int adapter_of(int id, int n_adapters) {
  return id < 0 || id >= n_adapters ? kNoAdapter : id;
}

// A row's place by counting, for adapters below 256 (`none`: the number that
// stands for no adapter): its rank among its wave's rows of the same adapter
// from ballots over the number's bits, after the rows of the same adapter in
// earlier waves and those of smaller numbers.  Every workgroup of a block gets
// the same order, which atomics would not give.
__device__ __forceinline__ int count_place(uint16_t (&bins)[kBlockRows / 64][256],
                                           int (&totals)[kBlockRows / 64], int id, bool valid) {
  const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
#pragma unroll
  for (int w = 0; w < kBlockRows / 64; ++w) bins[w][i] = 0;
  uint64_t same = __ballot(valid);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const bool bit = (id >> b) & 1;
    const uint64_t m = __ballot(bit);
    same &= bit ? m : ~m;
  }
  const int before = __popcll(same & ((1ull << lane) - 1));
  __syncthreads();
  if (valid && before == 0) bins[wave][id] = (uint16_t)__popcll(same);
  __syncthreads();
  // thread i adds bin i of the waves up, then all bins below it
  int of[kBlockRows / 64], sum = 0;
#pragma unroll
  for (int w = 0; w < kBlockRows / 64; ++w) {
    of[w] = sum;
    sum += bins[w][i];
  }
  int upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int v = __shfl_up(upto, d);
    upto += lane >= d ? v : 0;
  }
  if (lane == 63) totals[wave] = upto;
  __syncthreads();
  int base = upto - sum;
  for (int w = 0; w < wave; ++w) base += totals[w];
#pragma unroll
  for (int w = 0; w < kBlockRows / 64; ++w) bins[w][i] = (uint16_t)(base + of[w]);
  __syncthreads();
  return valid ? bins[wave][id] + before : i;
}

// Up to 64 rows: every wave works the order out by itself and all write the
// same values down, without a barrier.  A row's place is the number of smaller
// keys, counted lane by lane.
__device__ __forceinline__ void make_few_tiles(Tiles& s, const int32_t* ids, int nr,
                                               int n_adapters, int tile_rows) {
  const int lane = threadIdx.x & 63;
  uint32_t key = ~0u;
  if (lane < nr) key = (uint32_t)adapter_of(ids[lane], n_adapters) << 8 | (uint32_t)lane;
  int place = lane;
  const uint32_t before = (uint32_t)__shfl_up((int)key, 1);
  if (__ballot(lane > 0 && before > key)) {  // packed prompts mostly come in order
    place = 0;
    for (int j = 0; j < nr; j += 8)
#pragma unroll
      for (int u = 0; u < 8; ++u)  // past nr: the largest value, never below
        place += (uint32_t)__builtin_amdgcn_readlane((int)key, j + u) < key ? 1 : 0;
  }
  if (lane < nr) s.sorted[place] = key;
  wave_lds_sync();
  const uint32_t mine = s.sorted[lane] >> 8, left = s.sorted[lane ? lane - 1 : 0] >> 8;
  const uint64_t runs = __ballot(lane == 0 || mine != left) & (~0ull >> (63 - lane));
  const int first = 63 - __clzll((long long)runs);  // of this place's adapter
  const bool head = lane < nr && ((lane - first) & (tile_rows - 1)) == 0;
  const uint64_t heads = __ballot(head);
  if (head) s.start[__popcll(heads & ((1ull << lane) - 1))] = (uint16_t)lane;
  if (lane == 0) s.count = __popcll(heads);
  wave_lds_sync();
}

// More rows.  Where they are not in order already, the places come from
// counting where the adapters are below 256, and every thread ranks its own row
// against all the others where they are not (the keys are in LDS, read four at
// a time as broadcasts): no sort, no atomics, and any ids.
// Counting and ranking, a whole call: 512 rows of 4 adapters, rank 16, 12.0 us
// and 13.8; 257 rows of 32, rank 64, 23.2 and 25.0.
__device__ __forceinline__ void make_tiles(Tiles& s, const int32_t* ids, int nr, int n_adapters,
                                           int tile_rows) {
  if (nr <= 64) return make_few_tiles(s, ids, nr, n_adapters, tile_rows);
  const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
  uint32_t key = ~0u;
  int id = kNoAdapter, before = -1;
  if (i < nr) {
    id = adapter_of(ids[i], n_adapters);
    if (i > 0) before = adapter_of(ids[i - 1], n_adapters);
    key = (uint32_t)id << 8 | (uint32_t)i;
  }
  s.key[i] = s.sorted[i] = key;
  const uint64_t runs = __ballot(i < nr && id != before);
  const uint64_t ordered = __ballot(before <= id);
  if (lane == 0) {
    s.runs[wave] = runs;
    s.ordered[wave] = ordered;
  }
  __syncthreads();
  uint64_t all = ~0ull;
#pragma unroll
  for (int w = 0; w < kBlockRows / 64; ++w) all &= s.ordered[w];
  if (all != ~0ull) {
    int place = 0;
    if (n_adapters < 256) {
      __shared__ uint16_t bins[kBlockRows / 64][256];
      __shared__ int totals[kBlockRows / 64];
      place = count_place(bins, totals, id == kNoAdapter ? n_adapters : id, i < nr);
    } else {
#pragma unroll 4
      for (int j = 0; j < nr; j += 4) {  // past nr: the largest value, never below
        const uint4 o = *reinterpret_cast<const uint4*>(s.key + j);
        place += (o.x < key) + (o.y < key) + (o.z < key) + (o.w < key);
      }
    }
    if (i < nr) s.sorted[place] = key;
    __syncthreads();
    const uint32_t mine = s.sorted[i] >> 8, left = s.sorted[i ? i - 1 : 0] >> 8;
    const uint64_t again = __ballot(i < nr && (i == 0 || mine != left));
    if (lane == 0) s.runs[wave] = again;
    __syncthreads();
  }
  // the tiles' first places: every wave goes through all places by itself and
  // they all write the same values down
  int count = 0;
#pragma unroll
  for (int w = 0; w < kBlockRows / 64; ++w) {
    const int at = w * 64 + lane;
    // the first place of this place's adapter: the last run mark not beyond it
    int first = 0;
#pragma unroll
    for (int v = 0; v <= w; ++v) {
      const uint64_t m = s.runs[v] & (v < w ? ~0ull : ~0ull >> (63 - lane));
      if (m) first = v * 64 + 63 - __clzll((long long)m);
    }
    const bool head = at < nr && ((at - first) & (tile_rows - 1)) == 0;
    const uint64_t heads = __ballot(head);
    if (head) s.start[count + __popcll(heads & ((1ull << lane) - 1))] = (uint16_t)at;
    count += __popcll(heads);
  }
  if (lane == 0) s.count = count;
  wave_lds_sync();
}

// The order that shrink works out, as it leaves it for expand in the workspace.
struct Order {
  uint32_t sorted[kBlockRows];
  uint16_t start[kBlockRows];
  int32_t count, pad[3];
};
__device__ __forceinline__ void put_order(Order* o, const Tiles& s) {
  const int i = threadIdx.x;
  o->sorted[i] = s.sorted[i];
  o->start[i] = s.start[i];
  if (i == 0) o->count = s.count;
}
__device__ __forceinline__ void get_order(Tiles& s, const Order* o) {
  const int i = threadIdx.x;
  s.sorted[i] = o->sorted[i];
  s.start[i] = o->start[i];
  if (i == 0) s.count = o->count;
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

// The workspace: the orders of the blocks, then t.
__device__ __forceinline__ Order* order_at(const LoraParams& P) {
  return static_cast<Order*>(P.workspace);
}
__device__ __forceinline__ float* t_at(const LoraParams& P) {
  return reinterpret_cast<float*>(order_at(P) + (P.rows + kBlockRows - 1) / kBlockRows);
}

__device__ __forceinline__ f32x4 mfma(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Two bf16: the larger exponent bits of each half so far.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 most_exponent(u16x2 m, uint32_t w) {
  return __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w & 0x7F807F80u));
}
// Whether the low half is an infinity (the high one: of the word shifted), and
// a word with small numbers of the same sign in the place of infinities (an
// infinite t stays what it is).
__device__ __forceinline__ bool infinite(uint32_t w) { return (w & 0x7FFFu) == 0x7F80u; }
__device__ __forceinline__ uint32_t tamed(uint32_t w) {
  if (infinite(w)) w = (w & 0xFFFF8000u) | 0x0D80u;
  if (infinite(w >> 16)) w = (w & 0x8000FFFFu) | 0x0D800000u;
  return w;
}

// A row of 64 k in LDS: 128 bytes and 16 of padding, so that eight lanes
// reading one 16-byte column of eight rows touch every bank once.
constexpr int kRun = 64;
constexpr int kRunPitch = 2 * kRun + 16;

// t[split][row][j] = sum over the split's k of A_id[j][k] x[row][k].
// Grid: (blocks' tile lanes, splits * rank blocks).  RT tiles of 16
// ranks; the four waves take every fourth run of 64 k, each by itself, and
// add their sums through LDS at the end.
//
// A matrix-core operand wants row l % 16 in lane l, so loading it straight
// from memory makes four neighbouring lanes touch four lines and a load of
// the wave take 64 cycles of the address unit instead of 16: for few rows
// that, not the memory, was the bound (2.2 us for 512 k of 64 ranks, 1.2 so).
// So eight neighbouring lanes load a row's 128 bytes and the operands are
// read back from LDS.
template <int RT>
struct ShrinkArgs {
  static constexpr int kMaxTiles = 4;                // 16-row tiles at a time at most
  static constexpr int kStaged = RT == 4 ? 2 : 4;    // of them in LDS at once
  static constexpr int kWaveBytes = (RT + kStaged) * 16 * kRunPitch;
  __amdgpu_buffer_rsrc_t rx, ra;  // the block's rows of x, the adapter's rows of A
  const Tiles* tiles;
  float* t;      // the split's sums of the block's first row, at the rank block
  uint8_t* lds;  // [4][kWaveBytes]; then the sums of two waves
  int k, kbeg, kend, stride;
  int ranks;  // of t from the rank block's first on
};

// NT * 16 rows of a tile (`len` of them, the others read as zeros).
template <int RT, int NT>
__device__ __forceinline__ void shrink_rows(const ShrinkArgs<RT>& P, int start, int len) {
  using S = ShrinkArgs<RT>;
  constexpr int XS = NT < S::kStaged ? NT : S::kStaged;
  static_assert(2 * RT * S::kMaxTiles * 64 * 16 <= 4 * S::kWaveBytes, "the sums fit");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  uint8_t* const mine = P.lds + wave * S::kWaveBytes;
  // loading: row 8 i + lane / 8, its 16-byte piece lane % 8
  const int piece = lane & 7;
  uint32_t xo[2 * NT];
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) {
    const int at = i * 8 + (lane >> 3);
    xo[i] = at < len ? (uint32_t)P.tiles->row(start + at) * (uint32_t)P.k * 2u : kOutOfRange;
  }
  const uint32_t ao = (uint32_t)(lane >> 3) * (uint32_t)P.k * 2u;
  uint4 qa[2 * RT], qx[2 * NT];
  const auto load_a = [&](int kc) {
    const int kk = kc + piece * 8;
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i)
      qa[i] = buf_ld16(P.ra, kk < P.kend ? ao + (uint32_t)(i * 8 * P.k + kk) * 2u : kOutOfRange);
  };
  const auto load_x = [&](int kc, int first) {
    const int kk = kc + piece * 8;
#pragma unroll
    for (int i = 0; i < 2 * XS; ++i)
      qx[2 * first + i] = buf_ld16(P.rx, kk < P.kend && xo[2 * first + i] != kOutOfRange
                                             ? xo[2 * first + i] + 2u * kk
                                             : kOutOfRange);
  };
  uint8_t* const put = mine + (lane >> 3) * kRunPitch + piece * 16;
  const uint8_t* const get = mine + n * kRunPitch + g * 16;
  f32x4 acc[RT][NT];
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int q = 0; q < NT; ++q) acc[j][q] = f32x4{0.f, 0.f, 0.f, 0.f};

  int kc = P.kbeg + wave * kRun;
  load_a(kc);
#pragma unroll
  for (int f = 0; f < NT; f += XS) load_x(kc, f);
  for (; kc < P.kend; kc += 4 * kRun) {
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i) *reinterpret_cast<uint4*>(put + i * 8 * kRunPitch) = qa[i];
    load_a(kc + 4 * kRun);
#pragma unroll
    for (int f = 0; f < NT; f += XS) {
      if (f > 0) wave_lds_sync();
#pragma unroll
      for (int i = 0; i < 2 * XS; ++i)
        *reinterpret_cast<uint4*>(put + (RT * 16 + i * 8) * kRunPitch) = qx[2 * f + i];
      load_x(kc + 4 * kRun, f);
      wave_lds_sync();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint4 fa[RT], fx[XS];
#pragma unroll
        for (int j = 0; j < RT; ++j)
          fa[j] = *reinterpret_cast<const uint4*>(get + j * 16 * kRunPitch + u * 64);
#pragma unroll
        for (int q = 0; q < XS; ++q)
          fx[q] = *reinterpret_cast<const uint4*>(get + (RT + q) * 16 * kRunPitch + u * 64);
#pragma unroll
        for (int q = 0; q < XS; ++q)
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[j][f + q] = mfma(fa[j], fx[q], acc[j][f + q]);
      }
    }
  }

  // waves 2 and 3 to 0 and 1, then 1 to 0
  f32x4* const part = reinterpret_cast<f32x4*>(P.lds);
  constexpr int half = RT * NT * 64;
  __syncthreads();
  if (wave >= 2) {
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int q = 0; q < NT; ++q) part[(wave - 2) * half + (j * NT + q) * 64 + lane] = acc[j][q];
  }
  __syncthreads();
  if (wave < 2) {
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int q = 0; q < NT; ++q) acc[j][q] += part[wave * half + (j * NT + q) * 64 + lane];
  }
  if (wave == 1) {
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int q = 0; q < NT; ++q) part[half + (j * NT + q) * 64 + lane] = acc[j][q];
  }
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      if (q * 16 + n < len) {
        float* const to =
            P.t + (int64_t)P.tiles->row(start + q * 16 + n) * P.stride + 4 * g;
#pragma unroll
        for (int j = 0; j < RT; ++j)
          if (16 * j < P.ranks)
            *reinterpret_cast<f32x4*>(to + 16 * j) =
                acc[j][q] + part[half + (j * NT + q) * 64 + lane];
      }
    }
  }
  __syncthreads();  // the next turn writes over the sums
}

// The tile lanes of the blocks of rows (workgroups that share a block's tiles),
// numbered block by block within a lane.  The last block, with fewer rows, has
// `last` of `lanes`: workgroups without a tile would take the places of others
// (257 rows of 32 adapters, k = 11008, rank 64: 27.7 us in all for 23.6).
struct TileLanes {
  int blocks, lanes, last;
  int tile_rows;  // of a tile at most: a power of two up to kTileRows
  __host__ __device__ int count() const { return (blocks - 1) * lanes + last; }
  __device__ __forceinline__ int of(int block) const { return block + 1 < blocks ? lanes : last; }
  __device__ __forceinline__ void place(int i, int& block, int& lane) const {
    block = 0, lane = i;
    if (blocks == 1) return;
    const bool all = i < blocks * last;  // lanes that every block has
    const int j = all ? i : i - blocks * last, n = all ? blocks : blocks - 1;
    block = j % n;
    lane = j / n + (all ? 0 : last);
  }
};

template <int RT>
__global__ void __launch_bounds__(kThreads) shrink_kernel(LoraParams P, TileLanes L, int splits,
                                                          int slice, int stride) {
  using S = ShrinkArgs<RT>;
  __shared__ Tiles tiles;
  __shared__ __align__(16) uint8_t lds[4 * S::kWaveBytes];
  int block, first;
  L.place(blockIdx.x, block, first);
  const int64_t row0 = (int64_t)block * kBlockRows;
  const int nr = P.rows - row0 < kBlockRows ? (int)(P.rows - row0) : kBlockRows;
  const int split = blockIdx.y % splits, rank0 = blockIdx.y / splits * (RT * 16);
  make_tiles(tiles, P.ids + row0, nr, P.n_adapters, L.tile_rows);
  if (first == 0 && blockIdx.y == 0) put_order(order_at(P) + block, tiles);
  S a;
  a.rx = buffer_range(P.x + row0 * P.k, (int64_t)nr * P.k * 2);
  a.tiles = &tiles;
  a.t = t_at(P) + ((int64_t)split * P.rows + row0) * stride + rank0;
  a.lds = lds;
  a.k = P.k;
  a.kbeg = split * slice;
  a.kend = P.k - a.kbeg < slice ? P.k : a.kbeg + slice;
  a.stride = stride;
  a.ranks = stride - rank0;
  const int count = tiles.count;
  const int lanes = L.of(block);
  for (int tile = first; tile < count; tile += lanes) {
    const Tile t = tile_at(tiles, tile, nr);
    if (t.id == kNoAdapter) break;  // the rows without an adapter come last
    a.ra = buffer_range(P.a + ((int64_t)t.id * P.rank + rank0) * P.k,
                        (int64_t)(P.rank - rank0) * P.k * 2);
    if (t.len <= 16) shrink_rows<RT, 1>(a, t.start, t.len);
    else if (t.len <= 32) shrink_rows<RT, 2>(a, t.start, t.len);
    else shrink_rows<RT, 4>(a, t.start, t.len);
  }
}

// y = base + B_id (s_id t).  Grid: (column tiles, blocks' tile lanes in two axes).
// The matrix cores' columns are columns of y: tile j of JT takes columns
// JT n + j as its columns n, so that a lane is left with JT consecutive
// columns of a row and 16 lanes with a run of 16 JT (memory in whole lines).
// DK: runs of 32 ranks at a time, H times after each other.  H is 2 above 128
// ranks, with the sums of a tile's rows waiting in registers: all of B's 256
// ranks at once leave one wave to a SIMD (8192 x 4096 to 4096: 157 us, 104 so).
// base and y go past the caches (nt): through them they drive out B and t,
// which every column tile and block of rows reads again (8192 rows, 4096 to
// 11008, rank 32: 458 MB fetched and 134.6 us, 399 MB and 120.4 so; either of
// the two alone 130 and 136 us).
template <int TERMS, bool BB, bool YB, int DK>
struct Expand {
  static constexpr int JT = 4;  // 8: 138 us for 135 of a prompt's call
  static constexpr int QN = 4;  // 16-row tiles at a time
  static constexpr int kRows = QN * 16;
  static constexpr int kDepth = DK * 32;
  static constexpr int kPitch = kDepth + 8;
  static constexpr int kCols = 64 * JT;  // columns of a workgroup
  static constexpr int kBaseWords = JT * (BB ? 2 : 4) / 4, kYWords = JT * (YB ? 2 : 4) / 4;
  struct Base {
    uint32_t w[4][kBaseWords];
  };
  static __device__ __forceinline__ void load_base(__amdgpu_buffer_rsrc_t r,
                                                   const uint32_t (&ro)[4], int c, int n_out,
                                                   Base& f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = ro[i] != kOutOfRange && c < n_out;
      const uint32_t at = in ? (ro[i] + (uint32_t)c) * (BB ? 2u : 4u) : kOutOfRange;
      if constexpr (kBaseWords == 2) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)at, 0, kNonTemporal);
        f.w[i][0] = v.x;
        f.w[i][1] = v.y;
      } else {
#pragma unroll
        for (int k = 0; k < kBaseWords; k += 4) {
          const uint4 v = buf_ld16<kNonTemporal>(r, in ? at + 4u * k : kOutOfRange);
          f.w[i][k] = v.x;
          f.w[i][k + 1] = v.y;
          f.w[i][k + 2] = v.z;
          f.w[i][k + 3] = v.w;
        }
      }
    }
  }
  static __device__ __forceinline__ float base_at(const Base& f, int i, int j) {
    if constexpr (!BB) return __uint_as_float(f.w[i][j]);
    else return (j & 1) ? bf16_hi(f.w[i][j >> 1]) : bf16_lo(f.w[i][j >> 1]);
  }
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t ro, int c,
                                               int n_out, const float (&v)[JT]) {
    const bool in = ro != kOutOfRange && c < n_out;
    const uint32_t at = in ? (ro + (uint32_t)c) * (YB ? 2u : 4u) : kOutOfRange;
    uint32_t w[kYWords];
#pragma unroll
    for (int k = 0; k < kYWords; ++k)
      w[k] = YB ? pack_bf16(v[(2 * k) % JT], v[(2 * k + 1) % JT]) : __float_as_uint(v[k % JT]);
    if constexpr (kYWords == 2) {
      const u32x2 q = {w[0], w[1]};
      __builtin_amdgcn_raw_buffer_store_b64(q, r, (int)at, 0, kNonTemporal);
    } else {
#pragma unroll
      for (int k = 0; k < kYWords; k += 4)
        buf_st16<kNonTemporal>(r, in ? at + 4u * k : kOutOfRange,
                 make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]));
    }
  }
};

// Waves to a SIMD asked for where the compiler would give one fewer: what the
// loads of one workgroup wait for, another's fill (a whole call, 8192 x 4096 to
// 4096: rank 64 58.0 us unasked, 57.0 with 4 waves; rank 128 91.2 and 81.4 with
// 3; rank 256 213 and 158 with 2; all of a tile's base loaded ahead instead, 2
// waves at rank 64: 10 us more).  Up to rank 32 a bf16 base leaves room for 4,
// which fp32 y misses by two registers unasked.
template <int TERMS, bool BB, bool YB, int DK, int H>
__global__ void __launch_bounds__(kThreads,
                                  H > 1 ? 2 : DK == 2 || (DK == 1 && BB) ? 4 : DK == 4 && TERMS == 2 ? 3 : 1)
    expand_kernel(LoraParams P, TileLanes L, int splits, int stride) {
  using E = Expand<TERMS, BB, YB, DK>;
  constexpr int JT = E::JT;
  __shared__ Tiles tiles;
  __shared__ __align__(16) uint16_t terms[TERMS * E::kRows * E::kPitch];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int at = blockIdx.y + blockIdx.z * gridDim.y;
  if (at >= L.count()) return;
  int block, first;
  L.place(at, block, first);
  const int64_t row0 = (int64_t)block * kBlockRows;
  const int nr = P.rows - row0 < kBlockRows ? (int)(P.rows - row0) : kBlockRows;
  const int col = blockIdx.x * E::kCols + wave * 16 * JT + JT * n;  // the lane's first column
  get_order(tiles, order_at(P) + block);
  constexpr int bs = BB ? 2 : 4, ys = YB ? 2 : 4;
  const __amdgpu_buffer_rsrc_t rbase =
      buffer_range(static_cast<const char*>(P.base) + row0 * P.n_out * bs,
                   P.base ? (int64_t)nr * P.n_out * bs : 0);
  const __amdgpu_buffer_rsrc_t ry =
      buffer_range(static_cast<char*>(P.y) + row0 * P.n_out * ys, (int64_t)nr * P.n_out * ys);
  const float* const t_all = t_at(P);
  const int count = tiles.count, lanes = L.of(block);
  for (int tile = first; tile < count; tile += lanes) {
    const Tile t = tile_at(tiles, tile, nr);
    const bool none = t.id == kNoAdapter;
    if (none && P.base == P.y) break;  // in place: those rows stay as they are
    // B's operands of depth run h
    uint4 fb[JT][DK];
    const auto load_b = [&](int h) {
      const __amdgpu_buffer_rsrc_t rb = buffer_range(
          P.b + (int64_t)t.id * P.n_out * P.rank, (int64_t)P.n_out * P.rank * 2);
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int d = 0; d < DK; ++d) {
          const int r = h * E::kDepth + d * 32 + 8 * g;
          fb[j][d] = buf_ld16(rb, r < P.rank && col + j < P.n_out
                                      ? ((uint32_t)(col + j) * (uint32_t)P.rank + r) * 2u
                                      : kOutOfRange);
        }
    };
    if (!none) load_b(0);
    const int len = t.len;  // kRows at most
    // offsets of the lane's rows 16 q + 4 g + i, and their base one tile ahead
    const auto rows_of = [&](int q, uint32_t (&ro)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = 16 * q + 4 * g + i;
        ro[i] = at < len ? (uint32_t)tiles.row(t.start + at) * (uint32_t)P.n_out : kOutOfRange;
      }
    };
    uint32_t ro[2][4];
    typename E::Base base[2];
    rows_of(0, ro[0]);
    if (P.base) E::load_base(rbase, ro[0], col, P.n_out, base[0]);
    // the terms of s t in depth run h, four ranks to a thread at a time
    const auto stage = [&](int h) {
      const float s = P.scaling[t.id];
      __syncthreads();  // the turn before has read them
      for (int i = threadIdx.x; i < len * (E::kDepth / 4); i += kThreads) {
        const int r = i / (E::kDepth / 4), c = i % (E::kDepth / 4) * 4;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (h * E::kDepth + c < P.rank) {  // t's other columns may be infinity times 0
          const float* from =
              t_all + (row0 + tiles.row(t.start + r)) * stride + h * E::kDepth + c;
          int k = 0;
          for (; k + 4 <= splits; k += 4) {
            f32x4 w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              w[u] = *reinterpret_cast<const f32x4*>(from + (k + u) * P.rows * stride);
            // all four on their way before the first is waited for: the
            // compiler, short of registers, would take them one by one (512
            // rows of 4 adapters, rank 64: 25.8 us for 20.0)
            asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]));
#pragma unroll
            for (int u = 0; u < 4; ++u) v += w[u];
          }
          for (; k < splits; ++k)
            v += *reinterpret_cast<const f32x4*>(from + k * P.rows * stride);
          v *= s;
        }
#pragma unroll
        for (int q = 0; q < TERMS; ++q) {
          const uint32_t lo = pack_bf16(v.x, v.y), hi = pack_bf16(v.z, v.w);
          *reinterpret_cast<uint2*>(terms + (q * E::kRows + r) * E::kPitch + c) =
              make_uint2(lo, hi);
          // what is left of v; nothing of an infinity, where it would be NaN
          const f32x4 term = {bf16_lo(lo), bf16_hi(lo), bf16_lo(hi), bf16_hi(hi)};
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = isinf(term[e]) ? 0.f : v[e] - term[e];
        }
      }
      __syncthreads();
    };
    const auto multiply = [&](int q, f32x4 (&acc)[JT]) {
      const int at = q * 16 + n < len ? q * 16 + n : len - 1;
#pragma unroll
      for (int d = 0; d < DK; ++d)
#pragma unroll
        for (int k = 0; k < TERMS; ++k) {
          const uint4 ft = *reinterpret_cast<const uint4*>(
              terms + (k * E::kRows + at) * E::kPitch + d * 32 + 8 * g);
#pragma unroll
          for (int j = 0; j < JT; ++j) acc[j] = mfma(ft, fb[j][d], acc[j]);
        }
    };
    // Tames B's operands at hand and says whether an element of them, in any lane
    // of the wave, is not finite.  Looking costs two operations for two elements (whole
    // calls, 8192 rows of 8 adapters, 4096 to 4096: rank 64 57.4 us without and
    // 58.2 with, 128 84.8 and 86.1, 256 158 and 160; looking for NaN in every
    // row's sums instead breaks up the loop: 8192 x 4096 to 11008, rank 32,
    // 119.1 without, 118.9 so, 122.9).
    const auto tame_b = [&]() __attribute__((always_inline)) {
      u16x2 m = {0, 0};
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int d = 0; d < DK; ++d) {
          const uint4 w = fb[j][d];
          m = most_exponent(most_exponent(most_exponent(most_exponent(m, w.x), w.y), w.z), w.w);
        }
      const bool any = __any(m.x == 0x7F80u || m.y == 0x7F80u) != 0;
      if (any) {
#pragma unroll
        for (int j = 0; j < JT; ++j)
#pragma unroll
          for (int d = 0; d < DK; ++d) {
            uint4& w = fb[j][d];
            w = make_uint4(tamed(w.x), tamed(w.y), tamed(w.z), tamed(w.w));
          }
      }
      return any;
    };
    // The products of B's infinities in the lane's columns, added to the rows of
    // y that the lane has stored: 64 ranks at a time, so that a column full of
    // them is read once, and no further than to a NaN (8192 rows, rank 256: 0.26
    // ms with one infinity in every adapter, 0.29 all NaN, 0.92 all infinities).
    const auto add_infinities = [&]() {
      __threadfence_block();
      const float s = P.scaling[t.id];
#pragma unroll 1
      for (int c = col; c < col + JT && c < P.n_out; ++c)
#pragma unroll 1
        for (int r0 = 0; r0 < P.rank; r0 += 64) {
          const uint16_t* const b = P.b + ((int64_t)t.id * P.n_out + c) * P.rank + r0;
          const int ranks = P.rank - r0 < 64 ? P.rank - r0 : 64;
          uint64_t where = 0;
#pragma unroll 1
          for (int u = 0; u < ranks; u += 8) {
            const uint4 w = *reinterpret_cast<const uint4*>(b + u);
            const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
              where |= (uint64_t)infinite(h[e >> 1] >> (16 * (e & 1))) << (u + e);
          }
          if (!where) continue;
#pragma unroll 1
          for (int i = 4 * g; i < len; i += (i & 3) == 3 ? 13 : 1) {  // 16 q + 4 g + 0..3
            const int64_t row = row0 + tiles.row(t.start + i), at = row * P.n_out + c;
            float v = YB ? bf16_lo(static_cast<const uint16_t*>(P.y)[at])
                         : static_cast<const float*>(P.y)[at];
#pragma unroll 1
            for (uint64_t left = where; left && v == v; left &= left - 1) {
              const int r = __builtin_ctzll(left);
              float of = 0.f;
#pragma unroll 1
              for (int k = 0; k < splits; ++k) of += t_all[(k * P.rows + row) * stride + r0 + r];
              v = fmaf(of * s, bf16_lo(b[r]), v);
            }
            if constexpr (YB) static_cast<uint16_t*>(P.y)[at] = (uint16_t)pack_bf16(v, 0.f);
            else static_cast<float*>(P.y)[at] = v;
          }
        }
    };
    f32x4 acc[H > 1 ? E::QN : 1][JT];
    if constexpr (H > 1) {
#pragma unroll
      for (int q = 0; q < E::QN; ++q)
#pragma unroll
        for (int j = 0; j < JT; ++j) acc[q][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    bool beyond = false;
    if (!none) {
      stage(0);
      beyond = tame_b();
      if constexpr (H > 1) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          if (h > 0) {
            load_b(h);
            stage(h);
            beyond |= tame_b();
          }
#pragma unroll
          for (int q = 0; q < E::QN; ++q)
            if (q * 16 < len) multiply(q, acc[q]);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < E::QN; ++q) {
      if (q * 16 >= len) break;
      if (q + 1 < E::QN) {
        rows_of(q + 1, ro[(q + 1) & 1]);
        if (P.base) E::load_base(rbase, ro[(q + 1) & 1], col, P.n_out, base[(q + 1) & 1]);
      }
      f32x4(&sum)[JT] = acc[H > 1 ? q : 0];
      if constexpr (H == 1) {
#pragma unroll
        for (int j = 0; j < JT; ++j) sum[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (!none) multiply(q, sum);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[JT];
#pragma unroll
        for (int j = 0; j < JT; ++j)
          v[j] = P.base ? sum[j][i] + E::base_at(base[q & 1], i, j) : sum[j][i];
        E::store(ry, ro[q & 1][i], col, P.n_out, v);
      }
    }
    if (beyond) add_infinities();
  }
}

// How a call is cut up: a function of the sizes only.
struct Cut {
  int rt;        // tiles of 16 ranks in a shrink workgroup
  int ranks;     // rank blocks of 16 rt
  int stride;    // floats of a row of t
  int64_t blocks;  // blocks of rows
  int splits, slice;  // of the k axis
  int tile_rows;      // 16, 32 or 64
};
// Workgroups that share a block's tiles: as many as it can have tiles, and
// where there are many blocks as many as packed prompts have (four, and one
// more for every change of adapter within 256 rows): the others would start
// only to find nothing (257 rows of 32 adapters: 29.8 us with 16, 23.4 with 33;
// 700 rows of 5 22.7 with 8, 19.3 with 10; 8192 rows of 6 118.9 with 8, 120.2
// with 11).
TileLanes tile_lanes(int64_t rows, int64_t blocks, int n_adapters, int tile_rows) {
  const int cap = blocks <= 2 ? 64 : blocks <= 8 ? 16 : 8;
  const auto lanes = [&](int r) {
    const int most = (r < n_adapters ? r : n_adapters) + r / tile_rows + 1;
    return most < r ? (most < cap ? most : cap) : (r < cap ? r : cap);
  };
  TileLanes t;
  t.blocks = (int)blocks;
  t.tile_rows = tile_rows;
  t.last = lanes((int)(rows - (blocks - 1) * kBlockRows));
  t.lanes = blocks > 1 ? lanes(kBlockRows) : t.last;
  return t;
}
Cut cut(int64_t rows, int n_out, int k, int n_adapters, int rank) {
  Cut c;
  c.stride = (rank + 15) / 16 * 16;
  c.blocks = (rows + kBlockRows - 1) / kBlockRows;
  // The k axis is split until there is a workgroup for every CU, counting the
  // tiles there can be: one to 64 rows, and one more for every adapter of a
  // block.  More of them cost more to start than they save (2048 rows of 4
  // adapters, k = 4096, rank 64: 30 us with 192 workgroups wanted, 26.1 with
  // 256, 29.1 with 384; 257 rows of 32, k = 11008: 23.8 with 256, 24.3 with 384).
  // A workgroup takes 512 k at least, which its waves wait for twice.
  const int64_t tail = rows - (c.blocks - 1) * kBlockRows;
  const int64_t changes =
      (c.blocks - 1) * (n_adapters < kBlockRows ? n_adapters : kBlockRows) +
      (n_adapters < tail ? n_adapters : tail);
  const auto tiles_of = [&](int tile_rows) { return (rows + tile_rows - 1) / tile_rows + changes; };
  const auto ranks_of = [&](int rt) { return (rank + 16 * rt - 1) / (16 * rt); };
  const int64_t tiles = tiles_of(kTileRows);
  const int most = (k + 511) / 512;
  c.rt = rank <= 16 ? 1 : rank <= 32 ? 2 : 4;
  const int64_t want = 256 / (tiles * ranks_of(c.rt));
  c.splits = (int)(want < 1 ? 1 : want < most ? want : most);
  c.slice = ((k + c.splits - 1) / c.splits + 127) / 128 * 128;
  c.splits = (k + c.slice - 1) / c.slice;
  // Where that leaves CUs idle, tiles of fewer rows, as far as the adapters have
  // rows for them on average (99 rows of 2, 1024 to 1024, rank 40: 14.2 us for
  // 10.2; 512 of 4, 4096 to 4096, rank 16: 14.0 for 12.0; up to 256 workgroups
  // instead of 512: 1000 of 6, 8192 to 4096, rank 32 19.8 for 17.6), with at most
  // 1024 workgroups of expand (132 of 3, 5120 to 11008, rank 64: 15.3 us, up to
  // 512 16.9); then workgroups of fewer ranks (64 of 1, 4096 to 4096, rank 64:
  // 13.0 us for 11.6; up to 512 workgroups instead of 256: 2048 of 4 26.4 for
  // 25.7, 64 of 8 14.4 for 14.9).
  c.tile_rows = kTileRows;
  const int64_t cols = (n_out + 255) / 256;
  const int64_t mean = (rows < kBlockRows ? rows : kBlockRows) / n_adapters;
  const auto work = [&](int tile_rows, int rt) {
    return tiles_of(tile_rows) * c.splits * ranks_of(rt);
  };
  while (c.tile_rows > 16 && mean > c.tile_rows / 2 && work(c.tile_rows / 2, c.rt) <= 512 &&
         tiles_of(c.tile_rows / 2) * cols <= 1024)
    c.tile_rows /= 2;
  while (c.rt > 1 && work(c.tile_rows, c.rt / 2) <= 256) c.rt /= 2;
  c.ranks = ranks_of(c.rt);
  return c;
}

template <int RT>
void shrink(const LoraParams& p, const Cut& c, hipStream_t s) {
  const TileLanes lanes = tile_lanes(p.rows, c.blocks, p.n_adapters, c.tile_rows);
  hipLaunchKernelGGL((shrink_kernel<RT>), dim3((unsigned)lanes.count(), c.splits * c.ranks),
                     dim3(kThreads), 0, s, p, lanes, c.splits, c.slice, c.stride);
}

constexpr int kMaxGridY = 32768;
template <int TERMS, bool BB, bool YB, int DK, int H>
void expand(const LoraParams& p, const Cut& c, hipStream_t s) {
  using E = Expand<TERMS, BB, YB, DK>;
  static_assert(E::kRows == kTileRows, "a tile's rows are taken at once");
  const TileLanes lanes = tile_lanes(p.rows, c.blocks, p.n_adapters, c.tile_rows);
  const int y = lanes.count() < kMaxGridY ? lanes.count() : kMaxGridY;
  hipLaunchKernelGGL((expand_kernel<TERMS, BB, YB, DK, H>),
                     dim3((p.n_out + E::kCols - 1) / E::kCols, y, (lanes.count() + y - 1) / y),
                     dim3(kThreads), 0, s, p, lanes, c.splits, c.stride);
}
template <int TERMS, bool BB, bool YB>
void expand_by_rank(const LoraParams& p, const Cut& c, hipStream_t s) {
  if (c.stride <= 32) expand<TERMS, BB, YB, 1, 1>(p, c, s);
  else if (c.stride <= 64) expand<TERMS, BB, YB, 2, 1>(p, c, s);
  else if (c.stride <= 128) expand<TERMS, BB, YB, 4, 1>(p, c, s);
  else expand<TERMS, BB, YB, 4, 2>(p, c, s);
}

}  // namespace

// The orders, and t for as many rows as calls of up to `rows` rows can want:
// more splits than one take 256 workgroups at most, with a tile to 64 rows and
// one more to 256, so splits * rows <= 256 * 256 / 5 rows of t for every 64
// ranks, and at most one split to 512 k.  An upper bound that never falls with
// rows, k or rank, where the splits themselves do (at k = 4096 and rank 64, 2048
// rows of one adapter take 6 of them and 8192 rows one).
size_t lora_workspace_bytes(int64_t rows, int k, int rank) {
  constexpr int64_t kSplitRows = 256 * 256 / 5 + 1;
  const int64_t stride = (rank + 15) / 16 * 16, most = (k + 511) / 512;
  const int64_t many = rows * most * stride, cap = kSplitRows * (stride < 64 ? stride : 64);
  const int64_t split = many < cap ? many : cap, whole = rows * stride;
  return (size_t)((rows + kBlockRows - 1) / kBlockRows) * sizeof(Order) +
         (size_t)(split > whole ? split : whole) * sizeof(float);
}

hipError_t launch_lora(const LoraParams& p, hipStream_t s) {
  const Cut c = cut(p.rows, p.n_out, p.k, p.n_adapters, p.rank);
  switch (c.rt) {
    case 1: shrink<1>(p, c, s); break;
    case 2: shrink<2>(p, c, s); break;
    default: shrink<4>(p, c, s); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.y_bf16) {
    if (p.base_bf16) expand_by_rank<2, true, true>(p, c, s);
    else expand_by_rank<2, false, true>(p, c, s);
  } else {
    if (p.base_bf16) expand_by_rank<3, true, false>(p, c, s);
    else expand_by_rank<3, false, false>(p, c, s);
  }
  return hipGetLastError();
}

}  // namespace bfly
