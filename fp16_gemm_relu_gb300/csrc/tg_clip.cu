// tg_clip.cu — the global norm of many gradients, and the gradients unscaled and clipped by it.
//
//   norm = sqrt(sum over all tensors of g^2) / scale,   out = g * min(1, max_norm / norm) / scale
//
// Two passes: squares are summed by blocks over fixed chunks (so the result does not depend on
// timing), then every block adds the blocks' sums in the same order, and scales its chunks.  The table of tensors
// is the kernels' argument.  Bound by HBM, with a second read that the norm forces: 1.3 billion fp16 values to
// float32 in 375 us (7.1 TB/s) and 1275 (6.3); 11 tensors of 1 million values 13 us.
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
constexpr int kChunk = kThreads * 32;                   // elements of a chunk, 32 of them a thread's
constexpr int kTensors = 256;                           // tensors of a launch
constexpr int kBlocksPerSm = 4;

struct Tensor {
  const void* data;
  void* out;
  int64_t count;
  unsigned first;  // number of its first chunk in the launch
  int kind;        // bit 0: float32 input, bit 1: float32 output, bit 2: 16-byte vectors
};
struct Table {
  Tensor t[kTensors];
  int n;
  unsigned chunks;
};

// The tensor that chunk c is of: `at`, if it is still that one.
__device__ __forceinline__ int tensor_of(const Table& tb, unsigned c, int at) {
  if (tb.t[at].first <= c && (at + 1 == tb.n || c < tb.t[at + 1].first)) return at;
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

// E elements of one access: 8 fp16 or 4 float32 in 16 bytes, 4 fp16 in 8.
template <bool F32, int E>
struct Vec;
template <>
struct Vec<true, 4> {
  float4 v;
  __device__ __forceinline__ void load(const void* p) { v = *static_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w; }
  __device__ __forceinline__ static void store(void* p, const float (&f)[4]) {
    __stcs(static_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
  }
};
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  a = f.x;
  b = f.y;
}
template <>
struct Vec<false, 4> {
  uint2 v;
  __device__ __forceinline__ void load(const void* p) { v = *static_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    unpack2(v.x, f[0], f[1]);
    unpack2(v.y, f[2], f[3]);
  }
  __device__ __forceinline__ static void store(void* p, const float (&f)[4]) {
    __stcs(static_cast<uint2*>(p), make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3])));
  }
};
template <>
struct Vec<false, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const void* p) { v = *static_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    unpack2(v.x, f[0], f[1]);
    unpack2(v.y, f[2], f[3]);
    unpack2(v.z, f[4], f[5]);
    unpack2(v.w, f[6], f[7]);
  }
  __device__ __forceinline__ static void store(void* p, const float (&f)[8]) {
    __stcs(static_cast<uint4*>(p), make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]),
                                              pack2(f[6], f[7])));
  }
};

__device__ __forceinline__ float load_one(const void* p, int i, int kind) {
  return kind & 1 ? static_cast<const float*>(p)[i] : __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_one(void* p, int i, int kind, float v) {
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

// A thread's accesses of a chunk of n elements, E elements each and kThreads E apart: load(v, k) and then
// use(v) of each.  Those of a whole chunk are all in flight together.
template <int E, typename V, typename L, typename U>
__device__ __forceinline__ void accesses(int n, L load, U use) {
  if (n == kChunk) {
    V v[32 / E];
#pragma unroll
    for (int k = 0; k < 32 / E; ++k) load(v[k], k);
#pragma unroll
    for (int k = 0; k < 32 / E; ++k) use(v[k], k);
  } else {
    const int left = n / E - static_cast<int>(threadIdx.x);
#pragma unroll 1
    for (int k = 0; k * kThreads < left; ++k) {
      V v;
      load(v, k);
      use(v, k);
    }
  }
}

// A thread's sum of its part of n elements' squares, n <= kChunk.
template <bool F32>
__device__ __forceinline__ float squares(const void* p, int n) {
  constexpr int E = F32 ? 4 : 8, kSize = F32 ? 4 : 2;
  const uint8_t* base = static_cast<const uint8_t*>(p) + threadIdx.x * (E * kSize);
  using V = Vec<F32, E>;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  accesses<E, V>(n, [&](V& v, int k) { v.load(base + k * (kThreads * E * kSize)); }, [&](const V& v, int) {
    float f[E];
    v.get(f);
#pragma unroll
    for (int j = 0; j < E; ++j) s[j & 3] = fmaf(f[j], f[j], s[j & 3]);
  });
  const int i = n / E * E + static_cast<int>(threadIdx.x);
  if (i < n) {
    const float f = load_one(p, i, F32 ? 1 : 0);
    s[0] = fmaf(f, f, s[0]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// A thread's sums of chunks meet with what each addition rounds off carried along (Kahan, 1965): added up one
// by one, 2150 squares of fp16 values come out 1.5e-6 of their sum too large.
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    tg_grad_squares_kernel(const __grid_constant__ Table tb, float* part) {
  __shared__ float slots[kThreads / 32];
  float sum = 0.0f, off = 0.0f;
  tg::chain_wait();
  tg::chain_release();
  int at = 0;
  for (unsigned c = blockIdx.x; c < tb.chunks; c += gridDim.x) {
    at = tensor_of(tb, c, at);
    const Tensor& t = tb.t[at];
    const int64_t i0 = int64_t(c - t.first) * kChunk;
    const int n = static_cast<int>(min(t.count - i0, int64_t(kChunk)));
    const void* p = static_cast<const uint8_t*>(t.data) + i0 * (t.kind & 1 ? 4 : 2);
    float s = 0.0f;
    if (!(t.kind & 4)) {
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const float v = load_one(p, i, t.kind);
        s = fmaf(v, v, s);
      }
    } else if (t.kind & 1) {
      s = squares<true>(p, n);
    } else {
      s = squares<false>(p, n);
    }
    const float y = s - off, next = sum + y;
    off = next < INFINITY ? (next - sum) - y : 0.0f;  // an infinite sum stays one
    sum = next;
  }
  const float w = warp_sum(sum - off);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = w;
  __syncthreads();
  if (threadIdx.x != 0) return;
  sum = 0.0f;
  for (int i = 0; i < kThreads / 32; ++i) sum += slots[i];
  part[blockIdx.x] = sum;
}

// The norm from the blocks' sums, added in float64, and the gradients' factor: by every block alike, in one
// warp of it (float64 is slow here: in every thread it took 16 us).  A norm that is not finite clips nothing.
__device__ __forceinline__ float factor_of(const float* part, int parts, float scale, float max_norm,
                                           float* norm) {
  __shared__ float factor;
  if (threadIdx.x < 32) {
    double s = 0.0;
#pragma unroll 4
    for (int i = threadIdx.x; i < parts; i += 32) s += __ldcg(part + i);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (threadIdx.x == 0) {
      const double r = sqrt(s) / scale;
      if (norm && blockIdx.x == 0) *norm = static_cast<float>(r);
      const double c = r > max_norm && r < INFINITY ? max_norm / r : 1.0;
      factor = static_cast<float>(c / scale);
    }
  }
  __syncthreads();
  return factor;
}

__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    tg_grad_norm_kernel(const float* part, int parts, float scale, float* norm) {
  tg::chain_wait();
  factor_of(part, parts, scale, INFINITY, norm);
}

// n elements times f, n <= kChunk.  An access is as wide as lets the lanes of a warp write one contiguous
// piece: 8-byte loads of fp16 for 16-byte stores of float32 (with 16-byte loads, whose 32 bytes of output a
// lane writes in two stores, 1.3 billion values took 1717 us, so 1300).
template <bool F32, bool OUT32>
__device__ __forceinline__ void scaled(const void* p, void* o, int n, float f) {
  constexpr int E = F32 || OUT32 ? 4 : 8, kSize = F32 ? 4 : 2, kOutSize = OUT32 ? 4 : 2;
  const uint8_t* base = static_cast<const uint8_t*>(p) + threadIdx.x * (E * kSize);
  uint8_t* out = static_cast<uint8_t*>(o) + threadIdx.x * (E * kOutSize);
  using V = Vec<F32, E>;
  accesses<E, V>(n, [&](V& v, int k) { v.load(base + k * (kThreads * E * kSize)); }, [&](const V& v, int k) {
    float x[E];
    v.get(x);
#pragma unroll
    for (int j = 0; j < E; ++j) x[j] *= f;
    Vec<OUT32, E>::store(out + k * (kThreads * E * kOutSize), x);
  });
  const int i = n / E * E + static_cast<int>(threadIdx.x);
  if (i < n) store_one(o, i, OUT32 ? 2 : 0, load_one(p, i, F32 ? 1 : 0) * f);
}

// The chunks are taken from the last one back: what the pass before read last is still in L2.
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    tg_grad_clip_kernel(const __grid_constant__ Table tb, const float* part, int parts, float scale,
                        float max_norm, float* norm) {
  tg::chain_wait();
  tg::chain_release();
  const float f = factor_of(part, parts, scale, max_norm, norm);
  int at = tb.n - 1;
  for (unsigned b = blockIdx.x; b < tb.chunks; b += gridDim.x) {
    const unsigned c = tb.chunks - 1 - b;
    at = tensor_of(tb, c, at);
    const Tensor& t = tb.t[at];
    const int64_t i0 = int64_t(c - t.first) * kChunk;
    const int n = static_cast<int>(min(t.count - i0, int64_t(kChunk)));
    const void* p = static_cast<const uint8_t*>(t.data) + i0 * (t.kind & 1 ? 4 : 2);
    void* o = static_cast<uint8_t*>(t.out) + i0 * (t.kind & 2 ? 4 : 2);
    switch (t.kind) {
      case 4: scaled<false, false>(p, o, n, f); break;
      case 5: scaled<true, false>(p, o, n, f); break;
      case 6: scaled<false, true>(p, o, n, f); break;
      case 7: scaled<true, true>(p, o, n, f); break;
      default:
        for (int i = threadIdx.x; i < n; i += kThreads)
          store_one(o, i, t.kind, load_one(p, i, t.kind) * f);
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
    if (it->second > a && g.out != g.data) return TG_ERR_INVALID_ARG;
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
      e = tg::launch_chained(tg_grad_norm_kernel, true, dim3(1), kThreads, 0, stream, part,
                             static_cast<int>(parts), scale, norm);
    }
    for (const Table& tb : tables) {
      if (e != cudaSuccess || !outs) break;
      const int grid = static_cast<int>(std::min<int64_t>(std::max(tb.chunks, 1u), most));
      e = tg::launch_chained(tg_grad_clip_kernel, true, dim3(grid), kThreads, 0, stream, tb, part,
                             static_cast<int>(parts), scale, max_norm, norm);
    }
    const cudaError_t fe = cudaFreeAsync(part, stream);
    if (e == cudaSuccess) e = fe;
    return e == cudaSuccess ? TG_OK : tg::record_cuda_error(e);
  } catch (...) {  // no host memory for the list
    return TG_ERR_NO_WORKSPACE;
  }
}
