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

constexpr int kNormThreads = 256;  // threads of a block whose rows need at most that many

// Eight fp16 values of a row: elements [8c, 8c + 8), zeros from n on.  b: bytes by which the row's
// start misses a 16-byte boundary (even).  With b == 0 a whole chunk is one 16-byte load.
// Otherwise it lies in two aligned blocks, which are loaded and shifted together where both lie
// inside the row; at the row's ends, element by element, so that nothing outside it is read.
__device__ __forceinline__ uint4 load_chunk(const uint16_t* row, uint32_t b, int c, int n) {
  const int e0 = c << 3;
  if (e0 >= n) return make_uint4(0, 0, 0, 0);
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
__device__ __forceinline__ void store_chunk(uint16_t* row, uint32_t b, int c, int n, uint4 v,
                                            int lane) {
  const int e0 = c << 3;
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

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float as_float(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float as_float(const float* p) { return *p; }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// Eight parameters from column 8c on (`none` where there are none: a null pointer or past n).
// vec: the pointer is 16-byte aligned.
template <typename P>
__device__ __forceinline__ void load_param(const P* p, bool vec, int c, int n, float none,
                                           float (&f)[8]) {
  const int e0 = c << 3;
  if (p != nullptr && vec && e0 + 8 <= n) {
    if constexpr (sizeof(P) == 2) {
      unpack8(__ldg(reinterpret_cast<const uint4*>(p + e0)), f);
    } else {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p + e0));
      const float4 b = __ldg(reinterpret_cast<const float4*>(p + e0) + 1);
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
      f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = (p != nullptr && e0 + i < n) ? as_float(p + e0 + i) : none;
}

// Sum of v over the tpr threads of a row (a power of two >= 32, aligned in the block); every thread
// of the block calls it the same number of times.  slots: 32 floats, not in use by the call before
// (callers alternate between two).
__device__ __forceinline__ float row_sum(float v, int tpr, float* slots) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (tpr == 32) return v;
  const int warp = threadIdx.x >> 5, wpr = tpr >> 5;
  if ((threadIdx.x & 31) == 0) slots[warp] = v;
  __syncthreads();
  const int first = warp & ~(wpr - 1);
  float s = slots[first + (threadIdx.x & (wpr - 1))];
  for (int d = wpr >> 1; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}

// tpr threads a row, CH chunks of eight a thread, blockDim.x / tpr rows a block.
template <int CH, typename P>
__global__ void __launch_bounds__(1024)
    tg_layernorm_kernel(const uint16_t* __restrict__ x, int64_t ldx, const P* __restrict__ gamma,
                        const P* __restrict__ beta, uint16_t* __restrict__ y, int64_t ldy,
                        float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int n,
                        float eps, int tpr, bool vec) {
  __shared__ float slots[2][32];
  const int t = threadIdx.x & (tpr - 1), lane = threadIdx.x & 31;
  const int64_t r = blockIdx.x * int64_t(blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = r < rows;  // threads of a row that is not there run along with nothing
  const uint16_t* xr = x + (live ? r : 0) * ldx;
  const uint32_t bx = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(xr) & 15u);
  const int width = live ? n : 0;
  uint4 v[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) v[i] = load_chunk(xr, bx, i * tpr + t, width);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    float f[8];
    unpack8(v[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += f[j];
  }
  const float mu = row_sum(s, tpr, slots[0]) / static_cast<float>(n);
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    float f[8];
    unpack8(v[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = f[j] - mu;
      if (((i * tpr + t) << 3) + j < width) q = fmaf(d, d, q);
    }
  }
  const float rs = 1.0f / sqrtf(row_sum(q, tpr, slots[1]) / static_cast<float>(n) + eps);
  if (t == 0 && live) {
    if (mean) mean[r] = mu;
    if (rstd) rstd[r] = rs;
  }
  uint16_t* yr = y + (live ? r : 0) * ldy;
  const uint32_t by = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(yr) & 15u);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = i * tpr + t;
    float f[8], g[8], o[8];
    unpack8(v[i], f);
    load_param(gamma, vec, c, width, 1.0f, g);
    load_param(beta, vec, c, width, 0.0f, o);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = fmaf((f[j] - mu) * rs, g[j], o[j]);
    store_chunk(yr, by, c, width, pack8(o), lane);
  }
}

// Backward.  A block walks rows blockIdx.x * R + group, + gridDim.x * R, ...; a thread keeps the
// same columns for all of them, so its part of dgamma and dbeta stays in registers, and each block
// writes one partial row of both: part[0][block][n] and part[1][block][n].
template <int CH, typename P>
__global__ void __launch_bounds__(1024)
    tg_layernorm_backward_kernel(const uint16_t* __restrict__ dy, int64_t lddy,
                                 const uint16_t* __restrict__ x, int64_t ldx,
                                 const P* __restrict__ gamma, const float* __restrict__ mean,
                                 const float* __restrict__ rstd, uint16_t* __restrict__ dx,
                                 int64_t lddx, float* __restrict__ part, int64_t rows, int n,
                                 int tpr, bool vec) {
  extern __shared__ float groups[];  // [rows of a block][2][n], where a block has several
  __shared__ float slots[2][2][32];
  const int t = threadIdx.x & (tpr - 1), lane = threadIdx.x & 31;
  const int per_block = blockDim.x / tpr, group = threadIdx.x / tpr;
  const float inv_n = 1.0f / static_cast<float>(n);
  float dg[CH][8], db[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = db[i][j] = 0.0f;
  int turn = 0;
  for (int64_t r0 = blockIdx.x * int64_t(per_block); r0 < rows;
       r0 += int64_t(gridDim.x) * per_block, turn ^= 1) {
    const int64_t r = r0 + group;
    const bool live = r < rows;
    const int width = live ? n : 0;
    const uint16_t* xr = x + (live ? r : 0) * ldx;
    const uint16_t* dyr = dy + (live ? r : 0) * lddy;
    const uint32_t bx = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(xr) & 15u);
    const uint32_t bd = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dyr) & 15u);
    uint4 xv[CH], dv[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      xv[i] = load_chunk(xr, bx, i * tpr + t, width);
      dv[i] = load_chunk(dyr, bd, i * tpr + t, width);
    }
    const float mu = live ? mean[r] : 0.0f, rs = live ? rstd[r] : 0.0f;
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = i * tpr + t;
      float f[8], d[8], g[8];
      unpack8(xv[i], f);
      unpack8(dv[i], d);
      load_param(gamma, vec, c, width, 1.0f, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if ((c << 3) + j < width) {
          const float h = (f[j] - mu) * rs;
          const float gj = d[j] * g[j];
          a += gj;
          b = fmaf(gj, h, b);
          dg[i][j] = fmaf(d[j], h, dg[i][j]);
          db[i][j] += d[j];
        }
      }
    }
    if (dx != nullptr) {
      a = row_sum(a, tpr, slots[turn][0]) * inv_n;
      b = row_sum(b, tpr, slots[turn][1]) * inv_n;
      uint16_t* dxr = dx + (live ? r : 0) * lddx;
      const uint32_t bo = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dxr) & 15u);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = i * tpr + t;
        float f[8], d[8], g[8], o[8];
        unpack8(xv[i], f);
        unpack8(dv[i], d);
        load_param(gamma, vec, c, width, 1.0f, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float h = (f[j] - mu) * rs;
          o[j] = rs * (d[j] * g[j] - a - h * b);
        }
        store_chunk(dxr, bo, c, width, pack8(o), lane);
      }
    }
  }
  if (part == nullptr) return;
  // the block's row groups are added in their order
  float* mine = per_block > 1 ? groups + int64_t(group) * 2 * n : nullptr;
  float* out_g = part + int64_t(blockIdx.x) * n;
  float* out_b = part + (int64_t(gridDim.x) + blockIdx.x) * n;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int e0 = (i * tpr + t) << 3;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (e0 + j < n) {
        (mine ? mine : out_g)[e0 + j] = dg[i][j];
        (mine ? mine + n : out_b)[e0 + j] = db[i][j];
      }
    }
  }
  if (per_block > 1) {
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * n; e += blockDim.x) {
      float s = 0.0f;
      for (int k = 0; k < per_block; ++k) s += groups[int64_t(k) * 2 * n + e];
      (e < n ? out_g : out_b - n)[e] = s;
    }
  }
}

// dgamma and dbeta from the blocks' partial rows, in a fixed order: 32 columns a block, each
// thread row adds every kReduceRows-th partial row, then the thread rows are added in order.
constexpr int kReduceRows = 16;
template <typename P>
__global__ void __launch_bounds__(32 * kReduceRows)
    tg_layernorm_params_kernel(const float* __restrict__ part, int parts, int n, P* dgamma,
                               P* dbeta) {
  __shared__ float sum[2][kReduceRows][32];
  const int j = blockIdx.x * 32 + threadIdx.x;
  float g = 0.0f, b = 0.0f;
  if (j < n) {
    for (int p = threadIdx.y; p < parts; p += kReduceRows) {
      g += part[int64_t(p) * n + j];
      b += part[(int64_t(parts) + p) * n + j];
    }
  }
  sum[0][threadIdx.y][threadIdx.x] = g;
  sum[1][threadIdx.y][threadIdx.x] = b;
  __syncthreads();
  if (threadIdx.y < 2 && j < n) {
    float s = 0.0f;
    for (int p = 0; p < kReduceRows; ++p) s += sum[threadIdx.y][p][threadIdx.x];
    P* out = threadIdx.y == 0 ? dgamma : dbeta;
    if (out) put(out + j, s);
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads of a row and chunks of a thread for n columns.
struct RowShape {
  int tpr, ch;
};
RowShape row_shape(int64_t n, int max_tpr_two) {
  const int64_t chunks = cdiv(n, 8);
  int tpr = 32;
  while (tpr < 1024 && tpr * (tpr < max_tpr_two ? 1 : 2) < chunks) tpr <<= 1;
  int ch = 1;
  while (int64_t(tpr) * ch < chunks) ch <<= 1;
  return {tpr, ch};
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename P>
cudaError_t forward(const void* x, const void* gamma, const void* beta, void* y, float* mean,
                    float* rstd, int64_t rows, int64_t n, int64_t ldx, int64_t ldy, float eps,
                    cudaStream_t st) {
  const RowShape s = row_shape(n, kNormThreads);
  const int threads = std::max(s.tpr, kNormThreads);
  const unsigned grid = static_cast<unsigned>(cdiv(rows, threads / s.tpr));
  const bool vec = aligned16(gamma) && aligned16(beta);
  auto go = [&](auto kern) {
    kern<<<grid, threads, 0, st>>>(static_cast<const uint16_t*>(x), ldx,
                                   static_cast<const P*>(gamma), static_cast<const P*>(beta),
                                   static_cast<uint16_t*>(y), ldy, mean, rstd, rows,
                                   static_cast<int>(n), eps, s.tpr, vec);
    return cudaGetLastError();
  };
  switch (s.ch) {
    case 1: return go(tg_layernorm_kernel<1, P>);
    case 2: return go(tg_layernorm_kernel<2, P>);
    default: return go(tg_layernorm_kernel<4, P>);
  }
}

template <typename P>
cudaError_t backward(const void* dy, const void* x, const void* gamma, const float* mean,
                     const float* rstd, void* dx, void* dgamma, void* dbeta, float* part,
                     int64_t rows, int64_t n, int64_t lddy, int64_t ldx, int64_t lddx,
                     const RowShape& s, int threads, int grid, cudaStream_t st) {
  const int per_block = threads / s.tpr;
  const size_t smem = per_block > 1 && part ? size_t(per_block) * 2 * n * 4 : 0;
  const bool vec = aligned16(gamma);
  auto go = [&](auto kern) {
    if (smem > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(
          kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (e != cudaSuccess) return e;
    }
    kern<<<grid, threads, smem, st>>>(
        static_cast<const uint16_t*>(dy), lddy, static_cast<const uint16_t*>(x), ldx,
        static_cast<const P*>(gamma), mean, rstd, static_cast<uint16_t*>(dx), lddx, part, rows,
        static_cast<int>(n), s.tpr, vec);
    return cudaGetLastError();
  };
  cudaError_t e;
  switch (s.ch) {
    case 1: e = go(tg_layernorm_backward_kernel<1, P>); break;
    case 2: e = go(tg_layernorm_backward_kernel<2, P>); break;
    default: e = go(tg_layernorm_backward_kernel<4, P>); break;
  }
  if (e != cudaSuccess || part == nullptr) return e;
  tg_layernorm_params_kernel<P><<<static_cast<unsigned>(cdiv(n, 32)), dim3(32, kReduceRows), 0, st>>>(
      part, grid, static_cast<int>(n), static_cast<P*>(dgamma), static_cast<P*>(dbeta));
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
  const cudaError_t e =
      param_type == TG_TYPE_F16
          ? forward<__half>(X, gamma, beta, Y, mean, rstd, M, N, ldx, ldy, eps, s)
          : forward<float>(X, gamma, beta, Y, mean, rstd, M, N, ldx, ldy, eps, s);
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
  const RowShape shape = row_shape(N, kNormThreads);
  const int threads = std::max(shape.tpr, kNormThreads);
  const int grid = static_cast<int>(
      std::min<int64_t>(cdiv(M, threads / shape.tpr), int64_t(sms) * (threads > 512 ? 1 : 2)));
  float* part = nullptr;
  if (dgamma || dbeta) {
    st = tg::scratch_alloc(size_t(2) * grid * N * 4, s, reinterpret_cast<void**>(&part));
    if (st != TG_OK) return st;
  }
  e = param_type == TG_TYPE_F16
          ? backward<__half>(dY, X, gamma, mean, rstd, dX, dgamma, dbeta, part, M, N, lddy, ldx,
                             lddx, shape, threads, grid, s)
          : backward<float>(dY, X, gamma, mean, rstd, dX, dgamma, dbeta, part, M, N, lddy, ldx,
                            lddx, shape, threads, grid, s);
  if (part) {
    const cudaError_t fe = cudaFreeAsync(part, s);
    if (e == cudaSuccess) e = fe;
  }
  return e == cudaSuccess ? TG_OK : tg::record_cuda_error(e);
}

}  // extern "C"
