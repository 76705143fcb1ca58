// Root-mean-square norm of rows, with the residual's addition in front and
// the round-to-nearest group quantizer at 8 bits behind, and its gradient.
//
//   h = x + residual (rounded to x's type)
//   rstd = (mean_i h_i^2 + eps)^(-1/2),  y_i = (h_i rstd) w_i
//   scale = fp16(max |y| / top) over a group, code_i = rnd(y_i / scale)
//
// One pass: a row stays in the registers of the threads that own it (16 to
// 1024 of them, eight elements a chunk) from its load to its last store.
#include "bfly_norm.h"
#include "bfly_rows.h"

#include <type_traits>

namespace bfly {
namespace {

// rstd from the mean square, in fp64: the hardware's reciprocal square root
// and two Newton steps (each squares the relative error), so that the fp32
// value is the correctly rounded one but for ties and the codes next to a
// rounding border do not depend on the order of the sum.
__device__ __forceinline__ float inv_sqrt(double m) {
  double r = __builtin_amdgcn_rsq(m);
  r = r * fma(-0.5 * m * r, r, 1.5);
  r = r * fma(-0.5 * m * r, r, 1.5);
  return m == __builtin_inf() ? 0.f : (float)r;
}

// Sum (or maximum) over the T threads of a row from each wave's value.  One
// barrier: the caller alternates between two buffers, so that a wave still
// reading one is never overtaken by a wave that writes it again.
template <int T, typename F>
__device__ __forceinline__ F block_sum(F v, F* buf, int t) {
  if constexpr (T <= 64) return v;
  if ((t & 63) == 0) buf[t >> 6] = v;
  __syncthreads();
  F s = buf[0];
#pragma unroll
  for (int i = 1; i < T / 64; ++i) s += buf[i];
  return s;
}
template <int T>
__device__ __forceinline__ float block_max(float v, float* buf, int t) {
  if constexpr (T <= 64) return v;
  if ((t & 63) == 0) buf[t >> 6] = v;
  __syncthreads();
  float s = buf[0];
#pragma unroll
  for (int i = 1; i < T / 64; ++i) s = fmaxf(s, buf[i]);
  return s;
}

// fp16(amax / top), saturated at the largest fp16 value; the quotient as a
// product with top's fp32 reciprocal, as the forward's quantizer takes it (it
// can differ from the rounded quotient only next to an fp16 rounding midpoint).
__device__ __forceinline__ _Float16 group_scale(float amax, float inv_top) {
  return (_Float16)fminf(amax * inv_top, 65504.f);
}

// The codes of eight values, four to a word; d the group's scale, r = 1 / d
// (0 for a zero scale: codes 0).  y / d is the IEEE quotient, as a division
// gives it: r is the rounded reciprocal and d has 11 bits, so one correction
// of y r by its exact remainder rounds the quotient correctly (Markstein).  y
// is finite (finite_group).
template <bool E4M3>
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float d, float r) {
  constexpr float top = E4M3 ? 448.f : 127.f;
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float q0 = y[e] * r;
    q[e] = __builtin_amdgcn_fmed3f(fmaf(fmaf(-q0, d, y[e]), r, q0), -top, top);
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (E4M3) {
      int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
      w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], v, true);
    } else {
      // 1.5 * 2^23 + q is rounded to nearest even at the unit: its low byte is the code
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = __float_as_uint(q[4 * i + e] + 12582912.f);
      w[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(u[3], u[2], 0x0C0C0400u),
                                   __builtin_amdgcn_perm(u[1], u[0], 0x0C0C0400u), 0x05040100u);
    }
  }
  const uint32_t any = d > 0.f ? ~0u : 0u;  // a zero scale: no negative zero either
  return make_uint2(w[0] & any, w[1] & any);
}
// An infinite y, beyond fp32 by its weight, would have the remainder infinity
// minus infinity: where the group's maximum says that there is one, the largest
// number stands for it, whose code is +-top as well.  (4096 rows, one scale
// each, to e4m3: of 4096 columns 13.9 us without this, 14.2 so, 14.8 with y r
// held to 2 top in every element; of 11008 34.5, 34.7, 36.4.)
__device__ __forceinline__ void finite_group(float (&y)[8], float amax) {
  if (amax < __builtin_inff()) return;
  constexpr float most = 3.40282347e38f;
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = __builtin_amdgcn_fmed3f(y[e], -most, most);
}
__device__ __forceinline__ float reciprocal(float d) { return d > 0.f ? 1.f / d : 0.f; }

// T threads to a row, V chunks of eight elements to a thread; VEC: n is a
// multiple of 8 (RowIo).  Q: 0 no codes, 1 int8, 2 e4m3.
template <int T, int V, bool VEC, bool XB, int Q>
__global__ void __launch_bounds__(T < 256 ? 256 : T) norm_kernel(NormParams P) {
  constexpr int RPB = T < 256 ? 256 / T : 1;  // rows a workgroup works on at once
  __shared__ double sums[2][T / 64];
  __shared__ float tops[2][T / 64];
  using X = RowIo<T, VEC, XB>;
  constexpr int RPW = T < 64 ? 64 / T : 1;  // rows of a wave
  const int t = threadIdx.x & (T - 1);
  // the wave's first row in the workgroup, the lane's row in the wave
  const int sub = T < 256 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64) * RPW : 0;
  const int mine = T < 64 ? (int)(threadIdx.x & 63) / T : 0;
  const int n = P.n, off = mine * n;
  const double inv_n = 1.0 / n;
  constexpr int es = XB ? 2 : 4;

  float w[V][8];
  {
    const __amdgpu_buffer_rsrc_t rw = row_range(P.weight, 0, n, P.w_bf16 ? 2 : 4);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!P.weight) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[v][e] = 1.f;
      } else if (P.w_bf16) {
        RowIo<T, VEC, true>::unpack(RowIo<T, VEC, true>::load(rw, t, v, 0, n), w[v]);
      } else {
        RowIo<T, VEC, false>::unpack(RowIo<T, VEC, false>::load(rw, t, v, 0, n), w[v]);
      }
    }
  }

  typename X::Raw qx[V], qr[V];
  const auto load = [&](int64_t row) {  // past the last row: nothing is read
    const int64_t left = P.rows - row;
    const int count = left < 0 ? 0 : left < RPW ? (int)left : RPW;
    const int64_t at = count ? row : 0;
    const __amdgpu_buffer_rsrc_t rx = row_range(P.x, at, n, es, count);
#pragma unroll
    for (int v = 0; v < V; ++v) qx[v] = X::load(rx, t, v, off, n);
    if (P.residual) {
      const __amdgpu_buffer_rsrc_t rr = row_range(P.residual, at, n, es, count);
#pragma unroll
      for (int v = 0; v < V; ++v) qr[v] = X::load(rr, t, v, off, n);
    }
  };
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + sub;
  load(row);
  for (; row < P.rows; row += step, turn ^= 1) {  // uniform over a row's threads
    const int count = P.rows - row < RPW ? (int)(P.rows - row) : RPW;
    const bool first = t == 0 && mine < count;  // the lane that writes a row's statistics
    float h[V][8];
    if (P.residual) {
      const __amdgpu_buffer_rsrc_t rh = row_range(P.h, row, n, es, count);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float a[8], b[8];
        X::unpack(qx[v], a);
        X::unpack(qr[v], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] += b[e];
        const typename X::Raw q = X::pack(a);
        if (P.h) X::store(rh, t, v, off, n, q);
        X::unpack(q, h[v]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) X::unpack(qx[v], h[v]);
    }
    load(row + step);  // the next row's, in flight during this one's work
    double ss = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fma((double)h[v][e], (double)h[v][e], ss);
    ss = block_sum<T>(wave_sum<T < 64 ? T : 64>(ss), sums[turn], t);
    const float rstd = inv_sqrt(fma(ss, inv_n, (double)P.eps));
    if (P.rstd && first) P.rstd[row + mine] = rstd;
    float top = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] = (h[v][e] * rstd) * w[v][e];
    if (P.y) {
      if (P.y_bf16) {
        const __amdgpu_buffer_rsrc_t ry = row_range(P.y, row, n, 2, count);
#pragma unroll
        for (int v = 0; v < V; ++v)
          RowIo<T, VEC, true>::store(ry, t, v, off, n, RowIo<T, VEC, true>::pack(h[v]));
      } else {
        const __amdgpu_buffer_rsrc_t ry = row_range(P.y, row, n, 4, count);
#pragma unroll
        for (int v = 0; v < V; ++v)
          RowIo<T, VEC, false>::store(ry, t, v, off, n, RowIo<T, VEC, false>::pack(h[v]));
      }
    }
    if constexpr (Q != 0) {
      constexpr float inv_top = 1.f / (Q == 2 ? 448.f : 127.f);
      const __amdgpu_buffer_rsrc_t rc = row_range(P.codes, row, n, 1, count);
      const int per_row = n / P.group;
      uint16_t* const sc = P.scales + (row + mine) * per_row;
      const auto code_offset = [&](int v, int e) {
        const int i = X::index(t, v, e);
        return T < 64 && i >= n ? kOutOfRange - 64u : (uint32_t)(off + i);
      };
      float d = 0.f, r = 0.f;
      if (P.group == n) {  // one scale for the row
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(h[v][e]));
        top = block_max<T>(run_max(top, T < 64 ? T : 64), tops[turn], t);
        const _Float16 s = group_scale(top, inv_top);
        d = (float)s;
        r = reciprocal(d);
        if (first) sc[0] = __builtin_bit_cast(uint16_t, s);
#pragma unroll
        for (int v = 0; v < V; ++v) finite_group(h[v], top);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (VEC && P.group != n) {  // a run of group / 8 lanes shares a scale
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(h[v][e]));
          m = run_max(m, P.group >> 3);
          finite_group(h[v], m);
          const _Float16 s = group_scale(m, inv_top);
          d = (float)s;
          r = reciprocal(d);
          const int i = X::index(t, v, 0);
          if (i < n && mine < count && (i & (P.group - 1)) == 0)
            sc[i / P.group] = __builtin_bit_cast(uint16_t, s);
        }
        const uint2 c = codes8<Q == 2>(h[v], d, r);
        if constexpr (VEC) {
          typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
          const u32x2 cw = {c.x, c.y};
          __builtin_amdgcn_raw_buffer_store_b64(cw, rc, (int)code_offset(v, 0), 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            __builtin_amdgcn_raw_buffer_store_b8(
                (uint8_t)((e < 4 ? c.x : c.y) >> (8 * (e & 3))), rc, (int)code_offset(v, e), 0, 0);
        }
      }
    }
  }
}

// ---- gradient --------------------------------------------------------------
//
//   g = dy w,  dx = (g - xhat mean(g xhat)) rstd + dh,  xhat = h rstd
//   dw = sum over rows of dy xhat
// Workgroup b takes row groups b, b + slots, ...; each thread sums dw of its
// columns over them in fp32 and writes one row of `partials`, which
// norm_dw_kernel adds up in a fixed order.
template <int T, int V, bool VEC, bool HB, bool GB>
__global__ void __launch_bounds__(T < 256 ? 256 : T) norm_bwd_kernel(NormBwdParams P) {
  constexpr int RPB = T < 256 ? 256 / T : 1;
  // a second row's loads, where the registers of a thread hold them
  constexpr bool AHEAD = T < 1024;
  __shared__ float sums[2][T / 64];
  using H = RowIo<T, VEC, HB>;
  using G = RowIo<T, VEC, GB>;
  constexpr int RPW = T < 64 ? 64 / T : 1;  // rows of a wave
  const int t = threadIdx.x & (T - 1);
  // the wave's first row in the workgroup, the lane's row in the wave
  const int sub = T < 256 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64) * RPW : 0;
  const int mine = T < 64 ? (int)(threadIdx.x & 63) / T : 0;
  const int n = P.n, off = mine * n;
  const float inv_n = 1.f / (float)n;

  float w[V][8], dw[V][8];
  {
    const __amdgpu_buffer_rsrc_t rw = row_range(P.weight, 0, n, P.w_bf16 ? 2 : 4);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!P.weight) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[v][e] = 1.f;
      } else if (P.w_bf16) {
        RowIo<T, VEC, true>::unpack(RowIo<T, VEC, true>::load(rw, t, v, 0, n), w[v]);
      } else {
        RowIo<T, VEC, false>::unpack(RowIo<T, VEC, false>::load(rw, t, v, 0, n), w[v]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[v][e] = 0.f;
    }
  }

  typename H::Raw qh[V];
  typename G::Raw qg[V], qd[V];
  float rstd;
  const auto load = [&](int64_t row, typename H::Raw (&h)[V], typename G::Raw (&g)[V],
                        typename G::Raw (&d)[V], float& r) {
    const int64_t left = P.rows - row;  // past the last row: nothing is read
    const int count = left < 0 ? 0 : left < RPW ? (int)left : RPW;
    const int64_t at = count ? row : 0;
    const __amdgpu_buffer_rsrc_t rh = row_range(P.h, at, n, HB ? 2 : 4, count);
    const __amdgpu_buffer_rsrc_t rg = row_range(P.dy, at, n, GB ? 2 : 4, count);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = H::load(rh, t, v, off, n);
#pragma unroll
    for (int v = 0; v < V; ++v) g[v] = G::load(rg, t, v, off, n);
    if (P.dh) {
      const __amdgpu_buffer_rsrc_t rd = row_range(P.dh, at, n, GB ? 2 : 4, count);
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = G::load(rd, t, v, off, n);
    }
    r = mine < count ? P.rstd[at + mine] : 0.f;
  };
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + sub;
  load(row, qh, qg, qd, rstd);
  for (; row < P.rows; row += step, turn ^= 1) {  // uniform over a row's threads
    typename H::Raw nh[V];
    typename G::Raw ng[V], nd[V];
    float next;
    if constexpr (AHEAD) load(row + step, nh, ng, nd, next);  // in flight during this row's work
    float c = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float h[8], g[8];
      H::unpack(qh[v], h);
      G::unpack(qg[v], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = g[e] * (h[e] * rstd);
        dw[v][e] += a;
        c = fmaf(a, w[v][e], c);
      }
    }
    c = block_sum<T>(wave_sum<T < 64 ? T : 64>(c), sums[turn], t) * inv_n;
    const __amdgpu_buffer_rsrc_t ro = row_range(
        P.dx, row, n, GB ? 2 : 4, P.rows - row < RPW ? (int)(P.rows - row) : RPW);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float h[8], g[8], d[8];
      H::unpack(qh[v], h);
      G::unpack(qg[v], g);
      if (P.dh) {
        G::unpack(qd[v], d);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        d[e] = fmaf(fmaf(-c, h[e] * rstd, g[e] * w[v][e]), rstd, d[e]);
      G::store(ro, t, v, off, n, G::pack(d));
    }
    if constexpr (AHEAD) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        qh[v] = nh[v];
        qg[v] = ng[v];
        if (P.dh) qd[v] = nd[v];
      }
      rstd = next;
    } else {
      load(row + step, qh, qg, qd, rstd);
    }
  }

  if (!P.dweight) return;
  const __amdgpu_buffer_rsrc_t rp = row_range(P.partials, blockIdx.x, n, 4);
  if constexpr (RPB > 1) {  // the rows of a workgroup, added in order
    __shared__ float all[RPB][V * 8][T];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) all[sub + mine][v * 8 + e][t] = dw[v][e];
    __syncthreads();
    if (sub + mine != 0) return;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int s = 1; s < RPB; ++s) dw[v][e] += all[s][v * 8 + e][t];
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    RowIo<T, VEC, false>::store(rp, t, v, 0, n, RowIo<T, VEC, false>::pack(dw[v]));
}

// dweight[i] = sum over slots of partials[slot][i]: 64 columns to a workgroup,
// wave k of 16 adding slots k, k + 16, ..., then the 16 sums in order.
constexpr int kDwWays = 16;
__global__ void __launch_bounds__(64 * kDwWays) norm_dw_kernel(const float* partials,
                                                               float* dweight, int slots, int n) {
  __shared__ float part[kDwWays][64];
  const int c = threadIdx.x & 63, k = threadIdx.x >> 6;
  const int i = blockIdx.x * 64 + c;
  float s = 0.f;
  if (i < n) {
#pragma unroll 8
    for (int j = k; j < slots; j += kDwWays) s += partials[(int64_t)j * n + i];
  }
  part[k][c] = s;
  __syncthreads();
  if (k == 0 && i < n) {
#pragma unroll
    for (int j = 1; j < kDwWays; ++j) s += part[j][c];
    dweight[i] = s;
  }
}

// Threads and chunks to a row: the fewest threads that hold it (777 x 5120
// bf16 to e4m3: 17.6 us with 1024 threads and one chunk, of which 384 threads
// had nothing, 9.9 with 256 and three).  But where a row has a CU to itself,
// one chunk a thread: the chunks of a thread take their turns (1 x 4096 bf16 to
// int8 in a graph 3.7 us with 256 threads and 3.3 with 512, 256 x 4096 4.4 and
// 4.0, 16 x 8192 4.95 and 4.35 with 1024; 320 x 8192 7.6 and 8.1).
#define BFLY_WIDTH(T, V) \
  if (n <= T * V * 8) return f(std::integral_constant<int, T>{}, std::integral_constant<int, V>{})
template <typename F>
hipError_t by_width(int64_t rows, int n, F f) {
  BFLY_WIDTH(16, 1);
  BFLY_WIDTH(64, 1);
  BFLY_WIDTH(64, 2);
  BFLY_WIDTH(256, 1);
  if (rows <= 256) {
    BFLY_WIDTH(512, 1);
    BFLY_WIDTH(1024, 1);
  }
  BFLY_WIDTH(256, 2);
  BFLY_WIDTH(256, 3);
  BFLY_WIDTH(256, 4);
  BFLY_WIDTH(512, 3);
  BFLY_WIDTH(1024, 2);
  return hipErrorInvalidValue;
}
// dw and the next row's loads need registers too: one chunk a thread where two
// would do (16384 x 4096 bf16 104 us with 256 threads and two, 99 with 512; fp32
// 193 us either way).
template <typename F>
hipError_t by_width_bwd(int n, F f) {
  BFLY_WIDTH(16, 1);
  BFLY_WIDTH(64, 1);
  BFLY_WIDTH(64, 2);
  BFLY_WIDTH(256, 1);
  BFLY_WIDTH(512, 1);
  BFLY_WIDTH(512, 2);
  BFLY_WIDTH(512, 3);
  BFLY_WIDTH(1024, 2);
  return hipErrorInvalidValue;
}
#undef BFLY_WIDTH
int rows_per_block(int n) { return n <= 128 ? 16 : n <= 1024 ? 4 : 1; }

// Workgroups of a forward launch at most: enough to give each of 8192 rows its
// own (8192 x 4096: 44.0 us; 1024 workgroups that load their next row ahead
// 45.2, 512 of them 50.4).
constexpr int64_t kNormBlocks = 8192;

template <bool VEC, bool XB, int Q>
hipError_t norm_run(const NormParams& p, hipStream_t s) {
  return by_width(p.rows, p.n, [&](auto T, auto V) {
    const int64_t need = (p.rows + rows_per_block(p.n) - 1) / rows_per_block(p.n);
    const int grid = (int)(need < kNormBlocks ? need : kNormBlocks);
    hipLaunchKernelGGL((norm_kernel<T(), V(), VEC, XB, Q>), dim3(grid),
                       dim3(T() < 256 ? 256 : T()), 0, s, p);
    return hipGetLastError();
  });
}

template <bool VEC, bool HB, bool GB>
hipError_t norm_bwd_run(const NormBwdParams& p, hipStream_t s) {
  return by_width_bwd(p.n, [&](auto T, auto V) {
    hipLaunchKernelGGL((norm_bwd_kernel<T(), V(), VEC, HB, GB>),
                       dim3(rmsnorm_bwd_slots(p.rows, p.n)), dim3(T() < 256 ? 256 : T()), 0, s, p);
    return hipGetLastError();
  });
}

}  // namespace

// 256 to 1024 slots, 4 MiB of partial sums where that allows it: writing and
// adding them costs 16384 x 5120 fp32 6 us at 256 slots and 18 at 1024
// (182 and 194 us in all), while narrow rows need the workgroups to have
// enough loads in flight.  With many rows more of them, so that a thread's
// fp32 sum goes over about 128 rows, up to 2048 slots: beyond 262144 groups of
// rows it grows with them (540000 x 4096: 264 rows).  A single one for two or three groups of
// rows: it is the sum already, and a launch less (3 rows of 4096: 4.6 us in a
// graph for 5.3, but 4 rows 5.4; 2 rows of 11008 5.7 for 6.6, 3 rows 7.0).
int rmsnorm_bwd_slots(int64_t rows, int n) {
  const int64_t need = (rows + rows_per_block(n) - 1) / rows_per_block(n);
  if (need > 0 && need <= (n <= 8192 ? 3 : 2)) return 1;
  int64_t most = n <= 1024 ? 1024 : n >= 4096 ? 256 : (1 << 20) / n;
  const int64_t many = need / 128 < 2048 ? need / 128 : 2048;
  if (most < many) most = many;
  return (int)(need < most ? need : most);
}

hipError_t launch_rmsnorm(const NormParams& p, hipStream_t s) {
  const int q = !p.codes ? 0 : p.e4m3 ? 2 : 1;
  const bool vec = p.n % 8 == 0;
#define BFLY_NORM(VEC, XB)                                    \
  (q == 0   ? norm_run<VEC, XB, 0>(p, s)                      \
   : q == 1 ? norm_run<VEC, XB, 1>(p, s)                      \
            : norm_run<VEC, XB, 2>(p, s))
  return vec ? (p.x_bf16 ? BFLY_NORM(true, true) : BFLY_NORM(true, false))
             : (p.x_bf16 ? BFLY_NORM(false, true) : BFLY_NORM(false, false));
#undef BFLY_NORM
}

hipError_t launch_rmsnorm_backward(NormBwdParams p, hipStream_t s) {
  const bool vec = p.n % 8 == 0;
  // one partial sum: straight to its place, where 16-byte stores can go there
  const bool alone = p.rows > 0 && rmsnorm_bwd_slots(p.rows, p.n) == 1 &&
                     ((uintptr_t)p.dweight & 15) == 0;
  if (alone) p.partials = p.dweight;
  hipError_t e = hipSuccess;
#define BFLY_NORM_BWD(HB, GB) (vec ? norm_bwd_run<true, HB, GB>(p, s) : norm_bwd_run<false, HB, GB>(p, s))
  if (p.rows > 0)
    e = p.h_bf16 ? (p.g_bf16 ? BFLY_NORM_BWD(true, true) : BFLY_NORM_BWD(true, false))
                 : (p.g_bf16 ? BFLY_NORM_BWD(false, true) : BFLY_NORM_BWD(false, false));
#undef BFLY_NORM_BWD
  if (e != hipSuccess || !p.dweight || alone) return e;
  hipLaunchKernelGGL(norm_dw_kernel, dim3((p.n + 63) / 64), dim3(64 * kDwWays), 0, s,
                     p.partials, p.dweight, rmsnorm_bwd_slots(p.rows, p.n), p.n);
  return hipGetLastError();
}

}  // namespace bfly
