// tg_norm.cu — layer normalisation of fp16 rows, forward and backward (Ba, Kiros & Hinton, 2016).
//
//   forward:   mu = sum_j x_j / N,  rstd = 1 / sqrt(sum_j (x_j - mu)^2 / N + eps)
//              y_j = (x_j - mu) rstd gamma_j + beta_j
//   backward:  h_j = (x_j - mu) rstd,  g_j = dy_j gamma_j
//              dx_j = rstd (g_j - (1/N) sum_i g_i - h_j (1/N) sum_i g_i h_i)
//              dgamma_j = sum over rows of dy_j h_j,  dbeta_j = sum over rows of dy_j
//
// Every sum is kept in float32; fp16 appears only where x and dy are read and y and dx (and
// gradients of fp16 parameters) are written, one rounding each.
//
// Both directions are bound by HBM: forward reads x and writes y (4 bytes an element), backward
// reads x and dy and writes dx (6 bytes).  So a row is read once, as fp16, into registers, and
// everything else happens there; the variance is summed from the centred values, since the row is
// at hand.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "tg_gemm_relu.h"
#include "tg_internal.h"

namespace {

// Eight fp16 values of a row: elements [8c, 8c + 8), zeros from n on.  b: the bytes by which the
// row's start misses a 16-byte boundary (even).  With b == 0 a whole chunk is one 16-byte load.
// Otherwise it lies in two aligned blocks, which are loaded and shifted together where both lie
// inside the row; at the row's ends, element by element, so that nothing outside it is read.
// VEC: every row starts on such a boundary and n is a multiple of 8.
template <bool VEC>
__device__ __forceinline__ uint4 load_chunk(const uint16_t* row, int c, int n) {
  const int e0 = c << 3;
  if (e0 >= n) return make_uint4(0, 0, 0, 0);
  if constexpr (VEC) return __ldg(reinterpret_cast<const uint4*>(row + e0));
  const uint32_t b = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u);
  if (b == 0 && e0 + 8 <= n) return __ldg(reinterpret_cast<const uint4*>(row + e0));
  if (b != 0 && c > 0 && e0 + 16 - static_cast<int>(b >> 1) <= n) {
    const uint4* blk = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(row) - b) + c;
    const uint4 lo = __ldg(blk), hi = __ldg(blk + 1);
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const uint32_t q = b >> 2;
    uint32_t t[7], u[5], o[4];
#pragma unroll
    for (int i = 0; i < 7; ++i) t[i] = (q & 1u) ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) u[i] = (q & 2u) ? t[i + 2] : t[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (b & 2u) ? __funnelshift_r(u[i], u[i + 1], 16) : u[i];
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = e0 + 2 * i < n ? __ldg(row + e0 + 2 * i) : 0u;
    const uint32_t hi = e0 + 2 * i + 1 < n ? __ldg(row + e0 + 2 * i + 1) : 0u;
    o[i] = lo | (hi << 16);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Stores chunk c = [8c, 8c + 8) of a row (values from n on are dropped).  The lanes of a warp hold
// consecutive chunks, and all of them call this together.  With b == 0 a whole chunk is one
// 16-byte store.  Otherwise a lane stores the aligned block that starts b bytes before its chunk:
// the last b bytes of the previous lane's chunk and the first 16 - b of its own; what no block
// covers (a warp's first and last elements, a row's last) is stored element by element.
template <bool VEC>
__device__ __forceinline__ void store_chunk(uint16_t* row, int c, int n, uint4 v, int lane) {
  const int e0 = c << 3;
  if constexpr (VEC) {
    if (e0 < n) *reinterpret_cast<uint4*>(row + e0) = v;
    return;
  }
  const uint32_t b = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u);
  if (b == 0) {  // the same for every lane of the warp
    if (e0 + 8 <= n) {
      *reinterpret_cast<uint4*>(row + e0) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e0 + i < n) row[e0 + i] = static_cast<uint16_t>(w[i >> 1] >> ((i & 1) << 4));
    }
    return;
  }
  const int own = 8 - static_cast<int>(b >> 1);  // elements of this chunk in its aligned block
  uint32_t w[8];
  w[4] = v.x;
  w[5] = v.y;
  w[6] = v.z;
  w[7] = v.w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xffffffffu, w[4 + i], 1);
  const bool whole = lane > 0 && e0 + own <= n;
  const bool next_whole = lane < 31 && e0 + 8 + own <= n;
  if (whole) {  // 16 bytes of w, starting 16 - b bytes in
    const uint32_t s = 16u - b, q = s >> 2;
    uint32_t t[7], u[5], o[4];
#pragma unroll
    for (int i = 0; i < 7; ++i) t[i] = (q & 1u) ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) u[i] = (q & 2u) ? t[i + 2] : t[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (s & 2u) ? __funnelshift_r(u[i], u[i + 1], 16) : u[i];
    *reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(row + e0) - b) =
        make_uint4(o[0], o[1], o[2], o[3]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool covered = i < own ? whole : next_whole;
    if (!covered && e0 + i < n) row[e0 + i] = static_cast<uint16_t>(w[4 + (i >> 1)] >> ((i & 1) << 4));
  }
}

// Two float32 values in a 64-bit register pair, and the arithmetic on such pairs (one instruction
// for both, each rounded as usual): the kernels below spend most of their issue slots on it.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 halves(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(f32x2 v) {
  const float2 f = halves(v);
  return f.x + f.y;
}

// Eight fp16 values <-> four pairs.
__device__ __forceinline__ void unpack8(const uint4& v, f32x2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[i] = pair(p.x, p.y);
  }
}

__device__ __forceinline__ uint4 pack8(const f32x2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = halves(f[i]);
    const __half2 h = __floats2half2_rn(p.x, p.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float as_float(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float as_float(const float* p) { return *p; }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// Eight parameters from column 8c on (`none` where there are none: a null pointer or past n).
// VEC: the pointer is 16-byte aligned and n a multiple of 8.
template <bool VEC, typename P>
__device__ __forceinline__ void load_param(const P* p, int c, int n, float none, f32x2 (&f)[4]) {
  const int e0 = c << 3;
  if (VEC && p != nullptr && e0 < n) {
    if constexpr (sizeof(P) == 2) {
      unpack8(__ldg(reinterpret_cast<const uint4*>(p + e0)), f);
    } else {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p + e0));
      const float4 b = __ldg(reinterpret_cast<const float4*>(p + e0) + 1);
      f[0] = pair(a.x, a.y), f[1] = pair(a.z, a.w), f[2] = pair(b.x, b.y), f[3] = pair(b.z, b.w);
    }
    return;
  }
  float g[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    g[i] = (!VEC && p != nullptr && e0 + i < n) ? as_float(p + e0 + i) : none;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pair(g[2 * i], g[2 * i + 1]);
}

// Sum of v over a row's threads: a warp, or (BLOCK) the whole block, which then calls it together.
// slots: 32 floats, not in use by the call before (callers alternate).
template <bool BLOCK>
__device__ __forceinline__ float row_sum(float v, float* slots) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if constexpr (BLOCK) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < static_cast<int>(blockDim.x >> 5) ? slots[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  }
  return v;
}

// 1 for the columns 8c .. 8c + 7 that a row of n has, 0 for the others (VEC: all or none).
template <bool VEC>
__device__ __forceinline__ f32x2 there(int c, int n, int i) {
  const int e0 = c << 3;
  if constexpr (VEC) return e0 < n ? pair(1.0f, 1.0f) : pair(0.0f, 0.0f);
  return pair(e0 + 2 * i < n ? 1.0f : 0.0f, e0 + 2 * i + 1 < n ? 1.0f : 0.0f);
}

// Forward: a row a warp (BLOCK false) or a row a block, CH chunks of eight a thread, THREADS at
// most a block.  Warps or blocks walk the rows in steps of the grid, so with CH <= 2 gamma and
// beta stay in registers, and the next row is loaded before the current one is reduced: its
// latency passes under the current row's arithmetic and barriers.
template <int CH, bool BLOCK, bool VEC, int THREADS, typename P>
__global__ void __launch_bounds__(THREADS)
    tg_layernorm_kernel(const uint16_t* __restrict__ x, int64_t ldx, const P* __restrict__ gamma,
                        const P* __restrict__ beta, uint16_t* __restrict__ y, int64_t ldy,
                        float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int n,
                        float eps) {
  __shared__ float slots[2][32];
  constexpr bool kKeep = CH <= 2;
  const int tpr = BLOCK ? blockDim.x : 32;  // threads of a row
  const int lane = threadIdx.x & 31, t = BLOCK ? threadIdx.x : lane;
  const int64_t step = BLOCK ? gridDim.x : int64_t(gridDim.x) * (blockDim.x >> 5);
  int64_t r = BLOCK ? blockIdx.x : blockIdx.x * int64_t(blockDim.x >> 5) + (threadIdx.x >> 5);
  const float inv_n = 1.0f / static_cast<float>(n);
  uint4 next[CH];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < CH; ++i) next[i] = load_chunk<VEC>(x + row * ldx, i * tpr + t, n);
  };
  if (r < rows) load(r);
  f32x2 g[kKeep ? CH : 1][4], o[kKeep ? CH : 1][4];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      load_param<VEC>(gamma, i * tpr + t, n, 1.0f, g[i]);
      load_param<VEC>(beta, i * tpr + t, n, 0.0f, o[i]);
    }
  }
  for (; r < rows; r += step) {
    f32x2 v[CH][4];
#pragma unroll
    for (int i = 0; i < CH; ++i) unpack8(next[i], v[i]);
    if (kKeep && r + step < rows) load(r + step);
    f32x2 s = pair(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < CH; ++i)
      s = add2(s, add2(add2(v[i][0], v[i][1]), add2(v[i][2], v[i][3])));
    const float mu = row_sum<BLOCK>(sum2(s), slots[0]) * inv_n;
    const f32x2 less = pair(-mu, -mu);
    f32x2 q = pair(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[i][j] = mul2(add2(v[i][j], less), there<VEC>(i * tpr + t, n, j));
        q = fma2(v[i][j], v[i][j], q);
      }
    }
    const float rs = 1.0f / sqrtf(row_sum<BLOCK>(sum2(q), slots[1]) * inv_n + eps);
    if (t == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
    const f32x2 times = pair(rs, rs);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = i * tpr + t, k = kKeep ? i : 0;
      if constexpr (!kKeep) {
        load_param<VEC>(gamma, c, n, 1.0f, g[0]);
        load_param<VEC>(beta, c, n, 0.0f, o[0]);
      }
      f32x2 out[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) out[j] = fma2(mul2(v[i][j], times), g[k][j], o[k][j]);
      store_chunk<VEC>(y + r * ldy, c, n, pack8(out), lane);
    }
    if (!kKeep && r + step < rows) load(r + step);
  }
}

// Backward, a row a warp or a row a block as above.  A thread keeps the same columns for all of
// its rows, so its part of dgamma and dbeta stays in registers, and each block writes one partial
// row of both (of np floats): part[0][block], part[1][block].  With CH <= 2 the row (as h and g)
// and the next one stay in registers; a longer row is read a second time for dx, from L2.
template <int CH, bool BLOCK, bool VEC, int THREADS, typename P>
__global__ void __launch_bounds__(THREADS)
    tg_layernorm_backward_kernel(const uint16_t* __restrict__ dy, int64_t lddy,
                                 const uint16_t* __restrict__ x, int64_t ldx,
                                 const P* __restrict__ gamma, const float* __restrict__ mean,
                                 const float* __restrict__ rstd, uint16_t* __restrict__ dx,
                                 int64_t lddx, float* __restrict__ part, int64_t np, int64_t rows,
                                 int n) {
  extern __shared__ float groups[];  // a row a warp: [warps][2][np]
  __shared__ float slots[2][2][32];
  constexpr bool kKeep = CH <= 2;
  constexpr int kHold = kKeep ? CH : 1;
  const int tpr = BLOCK ? blockDim.x : 32;
  const int lane = threadIdx.x & 31, t = BLOCK ? threadIdx.x : lane;
  const int64_t step = BLOCK ? gridDim.x : int64_t(gridDim.x) * (blockDim.x >> 5);
  int64_t r = BLOCK ? blockIdx.x : blockIdx.x * int64_t(blockDim.x >> 5) + (threadIdx.x >> 5);
  const float inv_n = 1.0f / static_cast<float>(n);
  f32x2 dg[CH][4], db[CH][4];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dg[i][j] = db[i][j] = pair(0.0f, 0.0f);
  uint4 next_x[kHold], next_dy[kHold];
  float next_mu = 0.0f, next_rs = 0.0f;
  auto load = [&](int64_t row) {
    if constexpr (kKeep) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        next_x[i] = load_chunk<VEC>(x + row * ldx, i * tpr + t, n);
        next_dy[i] = load_chunk<VEC>(dy + row * lddy, i * tpr + t, n);
      }
    }
    next_mu = __ldg(mean + row);
    next_rs = __ldg(rstd + row);
  };
  if (r < rows) load(r);
  f32x2 gm[kHold][4];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < CH; ++i) load_param<VEC>(gamma, i * tpr + t, n, 1.0f, gm[i]);
  }
  // h and g of chunk i of a row; past the row's end dy, and with it g, is 0
  auto terms = [&](int64_t row, int i, f32x2 less, f32x2 times, f32x2(&h)[4], f32x2(&d)[4],
                   f32x2(&g)[4]) {
    const int c = i * tpr + t, k = kKeep ? i : 0;
    if constexpr (!kKeep) {
      next_x[0] = load_chunk<VEC>(x + row * ldx, c, n);
      next_dy[0] = load_chunk<VEC>(dy + row * lddy, c, n);
      load_param<VEC>(gamma, c, n, 1.0f, gm[0]);
    }
    unpack8(next_x[k], h);
    unpack8(next_dy[k], d);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = mul2(add2(h[j], less), times);
      g[j] = mul2(d[j], gm[k][j]);
    }
  };
  for (int turn = 0; r < rows; r += step, turn ^= 1) {
    const float rs = next_rs;
    const f32x2 less = pair(-next_mu, -next_mu), times = pair(rs, rs);
    f32x2 h[kHold][4], g[kHold][4], a2 = pair(0.0f, 0.0f), b2 = pair(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int k = kKeep ? i : 0;
      f32x2 d[4];
      terms(r, i, less, times, h[k], d, g[k]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a2 = add2(a2, g[k][j]);
        b2 = fma2(g[k][j], h[k][j], b2);
        dg[i][j] = fma2(d[j], h[k][j], dg[i][j]);
        db[i][j] = add2(db[i][j], d[j]);
      }
    }
    if (r + step < rows) load(r + step);
    if (dx != nullptr) {
      const float a = row_sum<BLOCK>(sum2(a2), slots[turn][0]) * inv_n;
      const float b = row_sum<BLOCK>(sum2(b2), slots[turn][1]) * inv_n;
      const f32x2 less_a = pair(-a, -a), less_b = pair(-b, -b);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int k = kKeep ? i : 0;
        if constexpr (!kKeep) {
          f32x2 d[4];
          terms(r, i, less, times, h[0], d, g[0]);
        }
        f32x2 out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          out[j] = mul2(times, fma2(h[k][j], less_b, add2(g[k][j], less_a)));
        store_chunk<VEC>(dx + r * lddx, i * tpr + t, n, pack8(out), lane);
      }
    }
  }
  if (part == nullptr) return;
  float* out_g = part + int64_t(blockIdx.x) * np;
  float* out_b = part + (int64_t(gridDim.x) + blockIdx.x) * np;
  float* to_g = BLOCK ? out_g : groups + int64_t(threadIdx.x >> 5) * 2 * np;
  float* to_b = BLOCK ? out_b : to_g + np;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int e0 = (i * tpr + t) << 3;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 fg = halves(dg[i][j]), fb = halves(db[i][j]);
      if (e0 + 2 * j < n) to_g[e0 + 2 * j] = fg.x, to_b[e0 + 2 * j] = fb.x;
      if (e0 + 2 * j + 1 < n) to_g[e0 + 2 * j + 1] = fg.y, to_b[e0 + 2 * j + 1] = fb.y;
    }
  }
  if constexpr (!BLOCK) {  // the block's warps are added in their order
    __syncthreads();
    for (int e = threadIdx.x; e < n; e += blockDim.x) {
      float sg = 0.0f, sb = 0.0f;
      for (int k = 0; k < static_cast<int>(blockDim.x >> 5); ++k) {
        sg += groups[int64_t(k) * 2 * np + e];
        sb += groups[(int64_t(k) * 2 + 1) * np + e];
      }
      out_g[e] = sg;
      out_b[e] = sb;
    }
  }
}

// dgamma and dbeta from the blocks' partial rows, in a fixed order: 32 columns a block, four a
// thread; each of the 32 thread rows adds every 32nd partial row, four loads in flight, then the
// thread rows are added in order.  Bound by the latency of its few loads: 304 partial rows of 8192
// columns (20 MB, in L2) took 9.5 us with one load in flight and 16 thread rows.
constexpr int kPartRows = 32;
template <typename P>
__global__ void __launch_bounds__(8 * kPartRows)
    tg_layernorm_params_kernel(const float* __restrict__ part, int parts, int64_t np, int n,
                               P* dgamma, P* dbeta) {
  __shared__ float4 sum[2][kPartRows][8];
  const int j = blockIdx.x * 32 + threadIdx.x * 4;  // np is a multiple of 4
  float4 acc[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    acc[w] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (j >= n) continue;
    const float* src = part + int64_t(w) * parts * np + j;
#pragma unroll 4
    for (int p = threadIdx.y; p < parts; p += kPartRows) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(src + p * np));
      acc[w].x += v.x;
      acc[w].y += v.y;
      acc[w].z += v.z;
      acc[w].w += v.w;
    }
  }
  sum[0][threadIdx.y][threadIdx.x] = acc[0];
  sum[1][threadIdx.y][threadIdx.x] = acc[1];
  __syncthreads();
  const int e = threadIdx.y * 8 + threadIdx.x;  // 32 columns of both
  if (e >= 64 || blockIdx.x * 32 + (e & 31) >= n) return;
  P* out = e < 32 ? dgamma : dbeta;
  if (out == nullptr) return;
  float s = 0.0f;
#pragma unroll
  for (int p = 0; p < kPartRows; ++p)
    s += reinterpret_cast<const float*>(&sum[e >> 5][p][0])[e & 31];
  put(out + blockIdx.x * 32 + (e & 31), s);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up4(int64_t n) { return (n + 3) & ~int64_t{3}; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kWarpThreads = 256;  // of a block whose warps have a row each

// Threads of a block that has a row of n columns, CH chunks of eight a thread.
int block_threads(int64_t n, int ch) {
  return static_cast<int>(cdiv(cdiv(n, 8 * ch), 32) * 32);
}

template <bool VEC, typename P>
cudaError_t forward(const void* x, const void* gamma, const void* beta, void* y, float* mean,
                    float* rstd, int64_t rows, int64_t n, int64_t ldx, int64_t ldy, float eps,
                    int sms, cudaStream_t st) {
  auto go = [&](auto kern, int threads, int64_t blocks) {
    kern<<<static_cast<unsigned>(blocks), threads, 0, st>>>(
        static_cast<const uint16_t*>(x), ldx, static_cast<const P*>(gamma),
        static_cast<const P*>(beta), static_cast<uint16_t*>(y), ldy, mean, rstd, rows,
        static_cast<int>(n), eps);
    return cudaGetLastError();
  };
  constexpr int kT = kWarpThreads;
  if (n <= 512) {
    const int64_t blocks = std::min<int64_t>(cdiv(rows, kT / 32), int64_t(sms) * 4);
    return n <= 256 ? go(tg_layernorm_kernel<1, false, VEC, kT, P>, kT, blocks)
                    : go(tg_layernorm_kernel<2, false, VEC, kT, P>, kT, blocks);
  }
  if (n <= 8192) {
    const int threads = block_threads(n, 2);
    return go(tg_layernorm_kernel<2, true, VEC, 512, P>, threads,
              std::min<int64_t>(rows, int64_t(sms) * std::min(16, 1024 / threads)));
  }
  const int threads = block_threads(n, n <= 16384 ? 4 : 8);
  return go(n <= 16384 ? tg_layernorm_kernel<4, true, VEC, 512, P>
                       : tg_layernorm_kernel<8, true, VEC, 512, P>,
            threads, std::min<int64_t>(rows, int64_t(sms) * 2));
}

// Threads of a block, and blocks, of the backward pass.
struct BackwardShape {
  int threads, blocks;
};
BackwardShape backward_shape(int64_t rows, int64_t n, int sms) {
  if (n <= 512)  // a row a warp
    return {kWarpThreads,
            static_cast<int>(std::min<int64_t>(cdiv(rows, kWarpThreads / 32), int64_t(sms) * 2))};
  const int threads = block_threads(n, n <= 8192 ? 2 : 4);
  const int per_sm = std::min(8, std::max(1, 512 / threads));
  return {threads, static_cast<int>(std::min<int64_t>(rows, int64_t(sms) * per_sm))};
}

template <bool VEC, typename P>
cudaError_t backward(const void* dy, const void* x, const void* gamma, const float* mean,
                     const float* rstd, void* dx, void* dgamma, void* dbeta, float* part,
                     int64_t rows, int64_t n, int64_t lddy, int64_t ldx, int64_t lddx,
                     const BackwardShape& s, cudaStream_t st) {
  auto go = [&](auto kern, size_t smem) {
    kern<<<s.blocks, s.threads, smem, st>>>(
        static_cast<const uint16_t*>(dy), lddy, static_cast<const uint16_t*>(x), ldx,
        static_cast<const P*>(gamma), mean, rstd, static_cast<uint16_t*>(dx), lddx, part,
        round_up4(n), rows, static_cast<int>(n));
    return cudaGetLastError();
  };
  const size_t groups = part ? size_t(kWarpThreads / 32) * 2 * round_up4(n) * 4 : 0;  // <= 32 KB
  cudaError_t e;
  if (n <= 256) e = go(tg_layernorm_backward_kernel<1, false, VEC, kWarpThreads, P>, groups);
  else if (n <= 512) e = go(tg_layernorm_backward_kernel<2, false, VEC, kWarpThreads, P>, groups);
  else if (n <= 8192) e = go(tg_layernorm_backward_kernel<2, true, VEC, 512, P>, 0);
  else if (n <= 16384) e = go(tg_layernorm_backward_kernel<4, true, VEC, 512, P>, 0);
  else e = go(tg_layernorm_backward_kernel<4, true, VEC, 1024, P>, 0);
  if (e != cudaSuccess || part == nullptr) return e;
  tg_layernorm_params_kernel<P><<<static_cast<unsigned>(cdiv(n, 32)), dim3(8, kPartRows), 0, st>>>(
      part, s.blocks, round_up4(n), static_cast<int>(n), static_cast<P*>(dgamma), static_cast<P*>(dbeta));
  return cudaGetLastError();
}

bool misaligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

constexpr int64_t kMaxLd = int64_t{1} << 36;

bool bad_ld(int64_t ld, int64_t n) { return ld < std::max<int64_t>(1, n) || ld > kMaxLd; }

}  // namespace

extern "C" {

tg_status tg_layernorm_f16(const void* X, const void* gamma, const void* beta, void* Y,
                           float* mean, float* rstd, int64_t M, int64_t N, int64_t ldx,
                           int64_t ldy, float eps, int param_type, tg_stream_t stream) {
  if (M < 0 || N < 1 || M > INT32_MAX || N > TG_NORM_MAX_WIDTH) return TG_ERR_INVALID_ARG;
  if (bad_ld(ldx, N) || bad_ld(ldy, N) || !(eps >= 0.0f)) return TG_ERR_INVALID_ARG;
  if (param_type != TG_TYPE_F16 && param_type != TG_TYPE_F32) return TG_ERR_INVALID_ARG;
  if (M == 0) return TG_OK;
  if (!X || !Y) return TG_ERR_INVALID_ARG;
  const unsigned pa = param_type == TG_TYPE_F16 ? 2 : 4;
  if (misaligned(X, 2) || misaligned(Y, 2) || misaligned(gamma, pa) || misaligned(beta, pa) ||
      misaligned(mean, 4) || misaligned(rstd, 4))
    return TG_ERR_MISALIGNED;
  int sms = 0;
  unsigned* err = nullptr;
  const tg_status st = tg::device_info(&sms, &err);
  if (st != TG_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool vec = aligned16(X) && aligned16(Y) && aligned16(gamma) && aligned16(beta) &&
                   ldx % 8 == 0 && ldy % 8 == 0 && N % 8 == 0;
  auto run = [&](auto f) { return f(X, gamma, beta, Y, mean, rstd, M, N, ldx, ldy, eps, sms, s); };
  const cudaError_t e = param_type == TG_TYPE_F16
                            ? (vec ? run(forward<true, __half>) : run(forward<false, __half>))
                            : (vec ? run(forward<true, float>) : run(forward<false, float>));
  return e == cudaSuccess ? TG_OK : tg::record_cuda_error(e);
}

tg_status tg_layernorm_backward_f16(const void* dY, const void* X, const void* gamma,
                                    const float* mean, const float* rstd, void* dX, void* dgamma,
                                    void* dbeta, int64_t M, int64_t N, int64_t lddy, int64_t ldx,
                                    int64_t lddx, int param_type, tg_stream_t stream) {
  if (M < 0 || N < 1 || M > INT32_MAX || N > TG_NORM_MAX_WIDTH) return TG_ERR_INVALID_ARG;
  if (bad_ld(lddy, N) || bad_ld(ldx, N) || (dX && bad_ld(lddx, N))) return TG_ERR_INVALID_ARG;
  if (param_type != TG_TYPE_F16 && param_type != TG_TYPE_F32) return TG_ERR_INVALID_ARG;
  const unsigned pa = param_type == TG_TYPE_F16 ? 2 : 4;
  if (misaligned(X, 2) || misaligned(dY, 2) || misaligned(dX, 2) || misaligned(gamma, pa) ||
      misaligned(dgamma, pa) || misaligned(dbeta, pa) || misaligned(mean, 4) ||
      misaligned(rstd, 4))
    return TG_ERR_MISALIGNED;
  if (!dX && !dgamma && !dbeta) return TG_OK;
  if (M > 0 && (!dY || !X || !mean || !rstd)) return TG_ERR_INVALID_ARG;
  int sms = 0;
  unsigned* err = nullptr;
  tg_status st = tg::device_info(&sms, &err);
  if (st != TG_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (M == 0) {  // sums over no rows
    for (void* p : {dgamma, dbeta})
      if (p && (e = cudaMemsetAsync(p, 0, size_t(N) * pa, s)) != cudaSuccess)
        return tg::record_cuda_error(e);
    return TG_OK;
  }
  const BackwardShape shape = backward_shape(M, N, sms);
  float* part = nullptr;
  if (dgamma || dbeta) {
    st = tg::scratch_alloc(size_t(2) * shape.blocks * round_up4(N) * 4, s, reinterpret_cast<void**>(&part));
    if (st != TG_OK) return st;
  }
  const bool vec = aligned16(dY) && aligned16(X) && aligned16(dX) && aligned16(gamma) &&
                   lddy % 8 == 0 && ldx % 8 == 0 && (!dX || lddx % 8 == 0) && N % 8 == 0;
  auto run = [&](auto f) {
    return f(dY, X, gamma, mean, rstd, dX, dgamma, dbeta, part, M, N, lddy, ldx, lddx, shape, s);
  };
  e = param_type == TG_TYPE_F16 ? (vec ? run(backward<true, __half>) : run(backward<false, __half>))
                                : (vec ? run(backward<true, float>) : run(backward<false, float>));
  if (part) {
    const cudaError_t fe = cudaFreeAsync(part, s);
    if (e == cudaSuccess) e = fe;
  }
  return e == cudaSuccess ? TG_OK : tg::record_cuda_error(e);
}

}  // extern "C"
