// tg_clip.cu — the global norm of many gradients, and the gradients unscaled and clipped by it.
//
//   norm = sqrt(sum over all tensors of g^2) / scale,   out = g * min(1, max_norm / norm) / scale
//
// Two passes: squares are summed by blocks over fixed chunks (so the result does not depend on
// timing), then every block adds the blocks' sums in the same order, and scales its chunks.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <utility>
#include <vector>

#include "tg_gemm_relu.h"
#include "tg_internal.h"

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;                                 // elements a thread takes at a time
constexpr int kChunk = kThreads * kVec * 4;             // elements of a chunk
constexpr int kTensors = 256;                           // tensors of a launch
constexpr int kBlocksPerSm = 8;

struct Tensor {
  const void* data;
  void* out;
  int64_t count;
  unsigned first;  // number of its first chunk in the launch
  int kind;        // bit 0: float32 input, bit 1: float32 output, bit 2: vectors of kVec
};
struct Table {
  Tensor t[kTensors];
  int n;
  unsigned chunks;
};

// The tensor that chunk c is of.
__device__ __forceinline__ int tensor_of(const Table& tb, unsigned c) {
  int lo = 0, hi = tb.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tb.t[mid].first <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <bool F32>
__device__ __forceinline__ void load_vec(const void* p, int64_t i, float (&v)[kVec]) {
  if constexpr (F32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const __half*>(p) + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
  }
}
__device__ __forceinline__ float load_one(const void* p, int64_t i, int kind) {
  return kind & 1 ? static_cast<const float*>(p)[i] : __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_one(void* p, int64_t i, int kind, float v) {
  if (kind & 2)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

template <bool F32>
__device__ __forceinline__ void squares(const void* p, int64_t i0, int64_t n, float (&s)[4]) {
#pragma unroll
  for (int k = 0; k < kChunk / (kThreads * kVec); ++k) {
    const int64_t i = i0 + (int64_t(k) * kThreads + threadIdx.x) * kVec;
    if (i + kVec <= n) {
      float v[kVec];
      load_vec<F32>(p, i, v);
#pragma unroll
      for (int j = 0; j < kVec; ++j) s[j & 3] = fmaf(v[j], v[j], s[j & 3]);
    } else {
      for (int64_t j = i; j < n; ++j) {
        const float v = load_one(p, j, F32 ? 1 : 0);
        s[0] = fmaf(v, v, s[0]);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    tg_grad_squares_kernel(const __grid_constant__ Table tb, float* part) {
  __shared__ float slots[kThreads / 32];
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (unsigned c = blockIdx.x; c < tb.chunks; c += gridDim.x) {
    const Tensor& t = tb.t[tensor_of(tb, c)];
    const int64_t i0 = int64_t(c - t.first) * kChunk, n = min(t.count, i0 + kChunk);
    if (!(t.kind & 4)) {
      for (int64_t i = i0 + threadIdx.x; i < n; i += kThreads) {
        const float v = load_one(t.data, i, t.kind);
        s[0] = fmaf(v, v, s[0]);
      }
    } else if (t.kind & 1) {
      squares<true>(t.data, i0, n, s);
    } else {
      squares<false>(t.data, i0, n, s);
    }
  }
  const float w = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = w;
  __syncthreads();
  if (threadIdx.x != 0) return;
  float sum = 0.0f;
  for (int i = 0; i < kThreads / 32; ++i) sum += slots[i];
  part[blockIdx.x] = sum;
}

// The norm from the blocks' sums, added in float64, and the gradients' factor: by every block alike.
// A norm that is not finite clips nothing.
__device__ __forceinline__ float factor_of(const float* part, int parts, float scale, float max_norm,
                                           float* norm) {
  __shared__ double slots[kThreads / 32];
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.0;
  for (int i = 0; i < kThreads / 32; ++i) s += slots[i];
  const double r = sqrt(s) / scale;
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(r);
  const double c = r > max_norm && r < INFINITY ? max_norm / r : 1.0;
  return static_cast<float>(c / scale);
}

__global__ void __launch_bounds__(kThreads)
    tg_grad_norm_kernel(const float* part, int parts, float scale, float* norm) {
  factor_of(part, parts, scale, INFINITY, norm);
}

template <bool F32, bool OUT32>
__device__ __forceinline__ void scaled(const Tensor& t, int64_t i0, int64_t n, float f) {
  float v[kChunk / (kThreads * kVec)][kVec];
#pragma unroll
  for (int k = 0; k < kChunk / (kThreads * kVec); ++k) {
    const int64_t i = i0 + (int64_t(k) * kThreads + threadIdx.x) * kVec;
    if (i + kVec <= n) load_vec<F32>(t.data, i, v[k]);
  }
#pragma unroll
  for (int k = 0; k < kChunk / (kThreads * kVec); ++k) {
    const int64_t i = i0 + (int64_t(k) * kThreads + threadIdx.x) * kVec;
    if (i + kVec <= n) {
      if constexpr (OUT32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(t.out) + i);
        d[0] = make_float4(v[k][0] * f, v[k][1] * f, v[k][2] * f, v[k][3] * f);
        d[1] = make_float4(v[k][4] * f, v[k][5] * f, v[k][6] * f, v[k][7] * f);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2 h = __floats2half2_rn(v[k][2 * j] * f, v[k][2 * j + 1] * f);
          w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(static_cast<__half*>(t.out) + i) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
      for (int64_t j = i; j < n; ++j)
        store_one(t.out, j, OUT32 ? 2 : 0, load_one(t.data, j, F32 ? 1 : 0) * f);
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    tg_grad_clip_kernel(const __grid_constant__ Table tb, const float* part, int parts, float scale,
                        float max_norm, float* norm) {
  const float f = factor_of(part, parts, scale, max_norm, norm);
  for (unsigned c = blockIdx.x; c < tb.chunks; c += gridDim.x) {
    const Tensor& t = tb.t[tensor_of(tb, c)];
    const int64_t i0 = int64_t(c - t.first) * kChunk, n = min(t.count, i0 + kChunk);
    switch (t.kind) {
      case 4: scaled<false, false>(t, i0, n, f); break;
      case 5: scaled<true, false>(t, i0, n, f); break;
      case 6: scaled<false, true>(t, i0, n, f); break;
      case 7: scaled<true, true>(t, i0, n, f); break;
      default:
        for (int64_t i = i0 + threadIdx.x; i < n; i += kThreads)
          store_one(t.out, i, t.kind, load_one(t.data, i, t.kind) * f);
    }
  }
}

bool misaligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kMaxCount = int64_t{1} << 40;

int size_of(int type) { return type == TG_TYPE_F32 ? 4 : 2; }

tg_status check(const tg_gradient* list, int64_t n, bool outs) {
  std::vector<std::pair<uintptr_t, uintptr_t>> written;  // address ranges of the outputs
  std::vector<std::pair<uintptr_t, uintptr_t>> in_place;  // and those of inputs that are outputs
  for (int64_t i = 0; i < n; ++i) {
    const tg_gradient& g = list[i];
    if (g.count < 0 || g.count > kMaxCount) return TG_ERR_INVALID_ARG;
    if (g.type != TG_TYPE_F16 && g.type != TG_TYPE_F32) return TG_ERR_INVALID_ARG;
    if (outs && g.out_type != TG_TYPE_F16 && g.out_type != TG_TYPE_F32) return TG_ERR_INVALID_ARG;
    if (g.count == 0) continue;
    if (!g.data || (outs && !g.out)) return TG_ERR_INVALID_ARG;
    if (misaligned(g.data, size_of(g.type)) || (outs && misaligned(g.out, size_of(g.out_type))))
      return TG_ERR_MISALIGNED;
    if (!outs) continue;
    const uintptr_t o = reinterpret_cast<uintptr_t>(g.out);
    written.emplace_back(o, o + size_t(g.count) * size_of(g.out_type));
    if (g.out == g.data && g.type != g.out_type) return TG_ERR_INVALID_ARG;
  }
  if (!outs) return TG_OK;
  std::sort(written.begin(), written.end());
  for (size_t i = 1; i < written.size(); ++i)
    if (written[i].first < written[i - 1].second) return TG_ERR_INVALID_ARG;
  for (int64_t i = 0; i < n; ++i) {  // an input meets no output but its own, and that one exactly
    const tg_gradient& g = list[i];
    if (g.count == 0) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(g.data), b = a + size_t(g.count) * size_of(g.type);
    auto it = std::upper_bound(written.begin(), written.end(), std::make_pair(a, UINTPTR_MAX));
    if (it != written.end() && it->first < b) return TG_ERR_INVALID_ARG;
    if (it == written.begin()) continue;
    --it;
    if (it->second > a && !(g.out == g.data)) return TG_ERR_INVALID_ARG;
  }
  return TG_OK;
}

}  // namespace

extern "C" tg_status tg_clip_gradients(const tg_gradient* list, int64_t n, float scale, float max_norm,
                                       float* norm, tg_stream_t stream_) {
  try {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (n < 0 || n > (int64_t{1} << 24) || (n > 0 && !list) || !norm) return TG_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || !(scale <= 3.0e38f) || !(max_norm >= 0.0f)) return TG_ERR_INVALID_ARG;
    if (misaligned(norm, 4)) return TG_ERR_MISALIGNED;
    bool outs = false;
    for (int64_t i = 0; i < n; ++i) outs |= list[i].out != nullptr;
    tg_status st = check(list, n, outs);
    if (st != TG_OK) return st;
    int sms = 0;
    unsigned* err = nullptr;
    if ((st = tg::device_info(&sms, &err)) != TG_OK) return st;
    // launches of up to kTensors tensors, and of as many chunks as an unsigned counts
    std::vector<Table> tables(1);
    std::memset(tables.data(), 0, sizeof(Table));
    for (int64_t i = 0; i < n; ++i) {
      const tg_gradient& g = list[i];
      if (g.count == 0) continue;
      Table* tb = &tables.back();
      const int64_t chunks = cdiv(g.count, kChunk);
      if (tb->n == kTensors || tb->chunks + chunks > (int64_t{1} << 31)) {
        tables.emplace_back();
        tb = &tables.back();
        std::memset(tb, 0, sizeof(Table));
      }
      const bool vec = !misaligned(g.data, 16) && (!outs || !misaligned(g.out, 16));
      Tensor& t = tb->t[tb->n++];
      t.data = g.data;
      t.out = g.out;
      t.count = g.count;
      t.first = tb->chunks;
      t.kind = (g.type == TG_TYPE_F32 ? 1 : 0) | (outs && g.out_type == TG_TYPE_F32 ? 2 : 0) | (vec ? 4 : 0);
      tb->chunks += static_cast<unsigned>(chunks);
    }
    const int most = sms * kBlocksPerSm;
    int64_t parts = 0;
    for (const Table& tb : tables) parts += std::min<int64_t>(std::max(tb.chunks, 1u), most);
    float* part = nullptr;
    if ((st = tg::scratch_alloc(size_t(parts) * 4, stream, reinterpret_cast<void**>(&part))) != TG_OK)
      return st;
    cudaError_t e = cudaSuccess;
    int64_t at = 0;
    for (const Table& tb : tables) {
      const int grid = static_cast<int>(std::min<int64_t>(std::max(tb.chunks, 1u), most));
      tg_grad_squares_kernel<<<grid, kThreads, 0, stream>>>(tb, part + at);
      if ((e = cudaGetLastError()) != cudaSuccess) break;
      at += grid;
    }
    if (e == cudaSuccess && !outs) {
      tg_grad_norm_kernel<<<1, kThreads, 0, stream>>>(part, static_cast<int>(parts), scale, norm);
      e = cudaGetLastError();
    }
    for (const Table& tb : tables) {
      if (e != cudaSuccess || !outs) break;
      const int grid = static_cast<int>(std::min<int64_t>(std::max(tb.chunks, 1u), most));
      tg_grad_clip_kernel<<<grid, kThreads, 0, stream>>>(tb, part, static_cast<int>(parts), scale,
                                                         max_norm, norm);
      e = cudaGetLastError();
    }
    const cudaError_t fe = cudaFreeAsync(part, stream);
    if (e == cudaSuccess) e = fe;
    return e == cudaSuccess ? TG_OK : tg::record_cuda_error(e);
  } catch (...) {  // no host memory for the list
    return TG_ERR_NO_WORKSPACE;
  }
}
