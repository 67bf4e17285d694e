// tg_head.cu — losses of a linear head over a large vocabulary, with their gradients, without
// keeping the logits: softmax cross entropy, and distillation from a teacher's top logits.
//
//   z = s X W^T  (T x V, float32; s the logit scale or 1 / temperature)
//   lse_t = log sum_v exp z_tv,  p_tv = exp(z_tv - lse_t)
//   cross entropy of target y:        loss_t = lse_t - z_ty
//   distillation from entries (i, u): q = softmax over the row's entries of s u,
//                                     loss_t = sum_e q_e (log q_e - (z_t,i_e - lse_t))
//   with the rows' weights w_t (d total / d loss_t), both have
//     d total / d (X W^T)_tv = s w_t (p_tv - [the row's target distribution]_v) = alpha G_tv
//     dX = alpha G W,  dW = alpha G^T X
//
// The three products are the work (2 T V D each), so they run on the tensor cores: the logits
// through tg_head_kernel.cuh, whose epilogue also leaves each tile's row maximum and sum of
// exponentials (so lse needs no pass over the logits, and cross entropy alone does not store
// them); dX and dW through the ordinary GEMMs on G.  Tokens go in pieces that bound the logits'
// scratch; dW is summed over the pieces in float32.
//
// G is rounded to fp16 once, the operand type of the products (kFineTokens: in two parts).  So that the many small
// probabilities stay normal fp16 numbers, G carries the factor 2^15 / max|w| (|p - q| <= 1, so
// nothing overflows) and alpha = s max|w| / 2^15 is applied to the float32 sums: a row of the
// largest weight keeps 11 bits of every p above 2^-29.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "tg_gemm_relu.h"
#include "tg_internal.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kGScale = 32768.0f;
// exp2f's results are 5.1e-8 of themselves too small on average (over [-24, 0], weighted by their size; measured with
// CUDA 13.0), and a row's sum goes through it twice: what that takes from lse, for losses whose log probabilities
// are added up.  The largest term, 1 of the row's sum s, is exact: 1 - 1 / s of it is owed.
constexpr float kExpLift = 1.0e-7f;

// What the passes after the logits know of a row.
struct alignas(16) RowInfo {
  float lse2;    // log2 of the sum of 2^(c logit), c = s log2(e)
  float gs;      // factor of the row of G: w_t 2^15 / max|w|, 0 for a row that does not count
  int target;    // cross entropy: the row's target in [0, V); -1 otherwise
  int pad;
};

enum class RowKind { kCounts, kIgnored, kBad };

// Cross entropy's target y: counted in [0, V), left out when it is ignore_index, anything else
// is an error of the caller's that shows as NaN.
__device__ __forceinline__ RowKind target_kind(int64_t y, int64_t vocab, int64_t ignore) {
  if (y == ignore) return RowKind::kIgnored;
  return y >= 0 && y < vocab ? RowKind::kCounts : RowKind::kBad;
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

// Elements [k, k + 8) of a 16-byte aligned row of n, zeros from n on.
__device__ __forceinline__ void load8(const uint16_t* row, int k, int n, float (&f)[8]) {
  if (k + 8 <= n) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(row + k)), f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = k + i < n ? __half2float(__ushort_as_half(row[k + i])) : 0.0f;
  }
}

// max |w_t| over the rows that count and have a finite w_t, as the bits of a non-negative float (an
// infinite one as the common factor would turn every row's 0 times it into NaN; so only its own row of
// G is not finite).  top == 0: cross
// entropy; else a row counts when one of its `top` entries does.  One block writes the maximum; with
// several it is zero before and the largest of theirs wins (the order of the atomics does not
// matter).
__global__ void __launch_bounds__(1024)
    tg_head_weight_kernel(const float* __restrict__ dloss, const int64_t* __restrict__ index,
                          int64_t ld, int top, int64_t ignore, int64_t rows, unsigned* wmax) {
  __shared__ float part[32];
  tg::chain_release();
  float m = 0.0f;
  for (int64_t r = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; r < rows;
       r += int64_t(gridDim.x) * blockDim.x) {
    bool live = top == 0 && index[r] != ignore;
    for (int j = 0; j < top && !live; ++j) live = index[r * ld + j] >= 0;
    const float w = live ? fabsf(dloss[r]) : 0.0f;
    if (w < INFINITY) m = fmaxf(m, w);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) m = fmaxf(m, part[w]);
  if (gridDim.x == 1)
    *wmax = __float_as_uint(m);
  else if (m > 0.0f)
    atomicMax(wmax, __float_as_uint(m));
}

__device__ __forceinline__ float row_factor(float w, float wmax) {
  return (wmax > 0.0f ? w / wmax : 0.0f * w) * kGScale;  // 0 * w keeps a NaN
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

constexpr int kRowThreads = 128;  // of a row in tg_head_rows_kernel

// Maximum and sum over the block; slots is used again only after the next meeting of the block.
__device__ __forceinline__ float block_max(float v, float* slots) {
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  return fmaxf(fmaxf(slots[0], slots[1]), fmaxf(slots[2], slots[3]));
}
__device__ __forceinline__ float block_sum(float v, float* slots) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  return (slots[0] + slots[1]) + (slots[2] + slots[3]);
}

// Where the logits of a row's targets are: in z, or (z NULL) in picked, [rows] or [rows][top].
struct Logits {
  const float* z;
  int64_t ldz;
  const float* picked;
};

// Entry e's teacher logit.
__device__ __forceinline__ float teacher_at(const void* t, int64_t at, int is_f32) {
  return is_f32 ? static_cast<const float*>(t)[at] : __half2float(static_cast<const __half*>(t)[at]);
}

// A block a row: lse from the row's statistics, then its loss and what the gradient needs of it.
// Distillation (top > 0): entries with a negative index are not there; q is the softmax of the
// others (one at -inf has q = 0), kept for the gradient when `q` is given (0 for what is not
// there).  A row without entries, or whose entries are all at -inf, has no teacher: loss 0 and no
// gradient.  Logits are scaled after the row's largest is taken off, so that those at the type's lowest
// value stay finite: a row of nothing else has a flat teacher.  alpha (one float): s max|w| / 2^15 (0 without wmax), written by the first block.  Bound by latency: 4096
// rows of 65537 classes (2 KB of statistics each) and 64 entries 18 us, one row 5 us.
__global__ void __launch_bounds__(kRowThreads)
    tg_head_rows_kernel(const float2* stats, int tiles, Logits lg, float scale,
                        int64_t vocab, const int64_t* __restrict__ index, int64_t ignore,
                        const void* __restrict__ teacher, int teacher_f32, int64_t ldt, int top,
                        const float* __restrict__ dloss, const unsigned* wmax,
                        float* loss, float* lse, RowInfo* info, float* q, float* alpha, float lift) {
  __shared__ float slots[6][4];
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  tg::chain_wait();
  tg::chain_release();
  const float w = wmax ? __uint_as_float(*wmax) : 0.0f;
  if (alpha && r == 0 && tid == 0) *alpha = scale * w / kGScale;
  // the first entries and their logits are on their way while the statistics are reduced
  int64_t i0 = -1;
  float u0 = 0.0f, z0 = 0.0f;
  if (tid < top) {
    i0 = index[r * ldt + tid];
    u0 = teacher_at(teacher, r * ldt + tid, teacher_f32);
    if (i0 >= 0 && i0 < vocab) z0 = lg.z ? lg.z[r * lg.ldz + i0] : lg.picked[r * top + tid];
  }
  float m = -INFINITY, s = 0.0f;
  const float2* parts = stats + r * tiles;
  if (lift > 0.0f) {  // with the row's maximum before any sum, so that each of them takes one power of two
#pragma unroll 4
    for (int t = tid; t < tiles; t += kRowThreads) m = fmaxf(m, __ldcg(&parts[t].x));
    m = block_max(m, slots[5]);
#pragma unroll 4
    for (int t = tid; t < tiles; t += kRowThreads) {
      const float2 v = __ldcg(parts + t);
      s += m > -INFINITY ? v.y * exp2f(v.x - m) : v.y;
    }
  }
#pragma unroll 4
  for (int t = lift > 0.0f ? tiles : tid; t < tiles; t += kRowThreads) {
    const float2 v = __ldcg(parts + t);
    const float m1 = fmaxf(m, v.x);
    if (m1 == -INFINITY) {
      s += v.y;  // zero or NaN
    } else {
      s = s * exp2f(m - m1) + v.y * exp2f(v.x - m1);
      m = m1;
    }
  }
  const float row_m = block_max(m, slots[0]);
  if (row_m > -INFINITY) s *= exp2f(m - row_m);
  const float sum = block_sum(s, slots[1]), lse2 = row_m + log2f(sum);
  const float lse_r = fmaf(lse2, kLn2, sum > 1.0f ? fmaf(-lift, 1.0f / sum, lift) : 0.0f);
  RowInfo ri;
  ri.lse2 = lse2;
  ri.gs = 0.0f;
  ri.target = -1;
  ri.pad = 0;
  float l = 0.0f;
  if (top == 0) {
    if (tid != 0) return;
    const int64_t y = index[r];
    const RowKind kind = target_kind(y, vocab, ignore);
    if (kind == RowKind::kCounts) {
      ri.target = static_cast<int>(y);
      l = lse_r - scale * (lg.z ? lg.z[r * lg.ldz + y] : lg.picked[r]);
      if (dloss) ri.gs = row_factor(dloss[r], w);
    } else if (kind == RowKind::kBad) {
      l = ri.gs = NAN;
    }
  } else {
    const float c = scale * kLog2e;
    float mt = -INFINITY;
    bool bad = false;
    for (int e = tid; e < top; e += kRowThreads) {
      const int64_t i = e == tid ? i0 : index[r * ldt + e];
      if (i < 0) continue;
      const float u = e == tid ? u0 : teacher_at(teacher, r * ldt + e, teacher_f32);
      bad |= i >= vocab || !(u < INFINITY);  // NaN or +inf
      mt = fmaxf(mt, u);
    }
    mt = block_max(mt, slots[2]);
    bad = __syncthreads_or(bad);
    float st = 0.0f;
    for (int e = tid; e < top && mt > -INFINITY; e += kRowThreads)
      if ((e == tid ? i0 : index[r * ldt + e]) >= 0)
        st += exp2f(((e == tid ? u0 : teacher_at(teacher, r * ldt + e, teacher_f32)) - mt) * c);
    const float lq = log2f(block_sum(st, slots[3]));
    for (int e = tid; e < top; e += kRowThreads) {
      float qe = 0.0f;
      const int64_t i = e == tid ? i0 : index[r * ldt + e];
      if (i >= 0 && mt > -INFINITY) {
        const float u = e == tid ? u0 : teacher_at(teacher, r * ldt + e, teacher_f32);
        const float t2 = fmaf(u - mt, c, -lq);
        qe = exp2f(t2);
        if (qe > 0.0f && i < vocab) {
          const float z = e == tid ? z0 : lg.z ? lg.z[r * lg.ldz + i] : lg.picked[r * top + e];
          l += qe * (t2 * kLn2 - (scale * z - lse_r));
        }
      }
      if (q) q[r * top + e] = qe;
    }
    l = block_sum(l, slots[4]);
    if (bad) l = ri.gs = NAN;
    else if (dloss && mt > -INFINITY) ri.gs = row_factor(dloss[r], w);
  }
  if (tid != 0) return;
  if (loss) loss[r] = l;
  if (lse) lse[r] = lse_r;
  info[r] = ri;
}

// The logits of a row's entries without the logits' matrix: one dot product of X and a row of W
// (V x D, 16-byte aligned rows) an entry, in float32.  A warp takes kPickRows entries at a time, whose
// loads go out together: bound by the latency of rows all over W (1024 tokens of 32 entries of 1024
// columns 19 us, 3.5 TB/s; with one entry a warp 21, two 20 to 24).
constexpr int kPickRows = 4;
__global__ void __launch_bounds__(256)
    tg_head_pick_kernel(const uint16_t* __restrict__ x, int64_t ldx, const uint16_t* __restrict__ w,
                        int64_t ldw, const int64_t* __restrict__ index, int64_t ldt, int top,
                        int64_t rows, int64_t vocab, int width, float* __restrict__ picked) {
  const int lane = threadIdx.x & 31;
  tg::chain_wait();
  tg::chain_release();
  const int64_t groups = (top + kPickRows - 1) / kPickRows;
  const int64_t step = int64_t(gridDim.x) * (blockDim.x >> 5);
  for (int64_t it = blockIdx.x * int64_t(blockDim.x >> 5) + (threadIdx.x >> 5); it < rows * groups;
       it += step) {
    const int64_t r = it / groups;
    const int e0 = static_cast<int>(it - r * groups) * kPickRows;
    const uint16_t* xr = x + r * ldx;
    const uint16_t* wr[kPickRows];
    float s[kPickRows];
#pragma unroll
    for (int j = 0; j < kPickRows; ++j) {  // an entry that is not there reads W's first row
      const int64_t i = e0 + j < top ? index[r * ldt + e0 + j] : 0;
      wr[j] = w + (i >= 0 && i < vocab ? i : 0) * ldw;
      s[j] = 0.0f;
    }
#pragma unroll 4
    for (int k = lane * 8; k < width; k += 256) {
      float a[8], b[kPickRows][8];
      load8(xr, k, width, a);
#pragma unroll
      for (int j = 0; j < kPickRows; ++j) load8(wr[j], k, width, b[j]);
#pragma unroll
      for (int j = 0; j < kPickRows; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j] = fmaf(a[i], b[j][i], s[j]);
    }
#pragma unroll
    for (int j = 0; j < kPickRows; ++j) {
      const float v = warp_sum(s[j]);
      if (lane == 0 && e0 + j < top) picked[r * top + e0 + j] = v;
    }
  }
}

// One value of G: gs (p - q).
__device__ __forceinline__ float grad_value(float z, float c, float lse2, float gs, float q) {
  return gs == 0.0f ? 0.0f : gs * (exp2f(fmaf(z, c, -lse2)) - q);
}

// G (fp16, rows of ldg) from the logits, eight columns of a row a thread; cross entropy's target with
// it.  Bound by HBM: 6 bytes an element, 4096 x 131072 in 456 us, 7.0 TB/s.
// FINE (few tokens): each value in two parts, G and `lo` elements further what its rounding left; and
// X's rows (16-byte aligned, of `width`) twice over, for the product with both parts.
// RAW: the rows hold their weights, whose largest is *wmax; alpha is written here (s: its scale).
template <bool FINE, bool RAW>
__global__ void __launch_bounds__(256)
    tg_head_grad_kernel(const float* z, int64_t ldz, float c, const RowInfo* info, int64_t rows,
                        int64_t vocab, uint16_t* __restrict__ g, int64_t ldg, int64_t lo,
                        const uint16_t* __restrict__ x, int64_t ldx, uint16_t* __restrict__ x2,
                        int64_t ldx2, int width, const unsigned* wmax, float s, float* alpha) {
  const int64_t v0 = (blockIdx.x * int64_t(blockDim.x) + threadIdx.x) << 3;
  tg::chain_wait();
  tg::chain_release();
  // RAW: the rows' common factor takes the largest weight to 2^15 (as row_factor: the large entries of rows of that
  // weight, near -1 times it, then lie just below a power of two, where fp16 rounds them by 2^-12 of themselves)
  const float most = RAW ? __uint_as_float(*wmax) : 0.0f;
  const float least = fmaxf(most, 0x1p-100f);  // (a NaN gives the other)
  const float up = kGScale / least;
  if (RAW && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    *alpha = s * least / kGScale;  // (not NaN: rows that do not count stay 0)
  if (FINE && x2 != nullptr && blockIdx.x == 0) {
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
      const uint16_t* from = x + r * ldx;
      uint16_t *to = x2 + r * ldx2, *again = x2 + (r + rows) * ldx2;
      const int whole = width & ~7;
      for (int k = threadIdx.x * 8; k < whole; k += blockDim.x * 8)
        *reinterpret_cast<uint4*>(to + k) = *reinterpret_cast<uint4*>(again + k) =
            __ldg(reinterpret_cast<const uint4*>(from + k));
      for (int k = whole + threadIdx.x; k < width; k += blockDim.x) to[k] = again[k] = from[k];
    }
  }
  if (v0 >= vocab) return;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    RowInfo ri = info[r];
    const float4* src = reinterpret_cast<const float4*>(z + r * ldz + v0);
    const float4 a = __ldcs(src), b = __ldcs(src + 1);  // ldz and ldg are multiples of 8
    if (RAW && ri.target >= 0) ri.gs = most == most ? ri.gs * up : most;
    const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t w[4], u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p0 = grad_value(f[2 * i], c, ri.lse2, ri.gs, v0 + 2 * i == ri.target ? 1.0f : 0.0f);
      const float p1 =
          grad_value(f[2 * i + 1], c, ri.lse2, ri.gs, v0 + 2 * i + 1 == ri.target ? 1.0f : 0.0f);
      const __half2 h = __floats2half2_rn(p0, p1);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
      if constexpr (FINE) {
        const float2 back = __half22float2(h);
        const __half2 rest = __floats2half2_rn(p0 - back.x, p1 - back.y);
        u[i] = *reinterpret_cast<const uint32_t*>(&rest);
      }
    }
    *reinterpret_cast<uint4*>(g + r * ldg + v0) = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (FINE)
      *reinterpret_cast<uint4*>(g + lo + r * ldg + v0) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// Distillation: G again at the teacher's entries, a warp a row.  Entries of one token add up; each of
// them then writes the same value.  Within the pass above the entries' reads would be on every
// block's way: 4096 x 65537 with 64 entries took 325 to 380 us so, 235 and 17 apart.
__global__ void __launch_bounds__(128)
    tg_head_teacher_grad_kernel(const int64_t* __restrict__ index, int64_t ldt, int top,
                                const float* q, const float* z, int64_t ldz, float c,
                                const RowInfo* info, int64_t rows, int64_t vocab,
                                __half* __restrict__ g, int64_t ldg, int64_t lo) {
  const int64_t r = (blockIdx.x * int64_t(blockDim.x) + threadIdx.x) >> 5;
  if (r >= rows) return;
  tg::chain_wait();
  tg::chain_release();
  const RowInfo ri = info[r];
  for (int e = threadIdx.x & 31; e < top; e += 32) {
    const int64_t i = index[r * ldt + e];
    if (i < 0 || i >= vocab) continue;
    float sum = 0.0f;
    for (int k = 0; k < top; ++k)
      if (index[r * ldt + k] == i) sum += q[r * top + k];
    const float v = grad_value(z[r * ldz + i], c, ri.lse2, ri.gs, sum);
    const __half h = __float2half_rn(v);
    g[r * ldg + i] = h;
    if (lo) g[lo + r * ldg + i] = __float2half_rn(v - __half2float(h));
  }
}

// A preference's or a policy's loss is a function of the targets' log probabilities logp_t = -nll_t, nll
// the cross entropy of tg_head_rows_kernel: the kernels below take those to the losses and to each row's
// weight w_t = d total / d nll_t, from which G follows as for cross entropy.
struct Objective {
  int kind;                  // 0: none, else kPreference or kPolicy
  const float* dloss;        // [pairs] or [T]: d total / d loss (NULL: no gradient)
  float* loss;               // [pairs] or [T], NULL: not wanted
  const float* reference;    // [T] log probabilities; NULL: 0 (preference), no penalty (policy)
  // preference: pair p is the rows [offsets[2p], offsets[2p + 1]) and from there to offsets[2p + 2]
  const int64_t* offsets;
  int64_t pairs;
  float beta, smooth;
  int average;
  float* ratios;             // [pairs][2], NULL: not wanted
  // policy
  const float *old, *advantage;
  float low, high, kl;       // the ratio's borders, and the penalty's weight
  float* logp;               // [T], NULL: not wanted
};
enum : int { kPreference = 1, kPolicy = 2 };

// Where an objective's weights go: max|w| over the rows as for cross entropy, NaN if any pair's offsets are
// wrong; and each row's, into its RowInfo::gs (the factor 2^15 / max|w| is taken in the pass over the logits) or
// into w, which is zero before.
struct Weights {
  unsigned* wmax;
  RowInfo* info;
  float* w;
  __device__ __forceinline__ void put(int64_t row, float v) const {
    if (info)
      info[row].gs = v;
    else
      w[row] = v;
  }
};
constexpr unsigned kNanBits = 0x7fc00000u;  // above all finite numbers' bits

// Bits of |w| where it is finite, else 0: see tg_head_weight_kernel.
__device__ __forceinline__ unsigned weight_bits(float w) {
  return fabsf(w) < INFINITY ? __float_as_uint(fabsf(w)) : 0u;
}

constexpr int kPairThreads = 256;

// A block a pair (Rafailov et al., 2023, with smoothed labels):
//   r_s = sum over a sequence's counted rows of logp - reference (average: their mean; none: 0)
//   m = beta (r_chosen - r_rejected),   loss = -(1 - e) log sigma(m) - e log sigma(-m)
// The sums are float64: those of a long answer are large and nearly the same in both.  Bound by latency:
// one pass over the rows of both sequences and one meeting of the block (16 pairs of 256 rows 6.5 us; with a meeting
// a sum 10).
__global__ void __launch_bounds__(kPairThreads)
    tg_head_pairs_kernel(Objective ob, const float* nll, const int64_t* __restrict__ index,
                         int64_t ignore, int64_t rows, Weights wt) {
  __shared__ double sums[2][kPairThreads / 32];
  __shared__ int counts[2][kPairThreads / 32];
  const int64_t p = blockIdx.x;
  const int64_t o[3] = {ob.offsets[2 * p], ob.offsets[2 * p + 1], ob.offsets[2 * p + 2]};
  const bool fits = o[0] >= 0 && o[0] <= o[1] && o[1] <= o[2] && o[2] <= rows;
  tg::chain_wait();
  tg::chain_release();
  double r[2] = {0.0, 0.0}, n[2];
  int count[2] = {0, 0};
  for (int64_t t = o[0] + threadIdx.x; fits && t < o[2]; t += kPairThreads) {
    if (index[t] == ignore) continue;
    const double d = -static_cast<double>(nll[t]) - (ob.reference ? ob.reference[t] : 0.0f);
    if (t < o[1]) {
      r[0] += d;
      ++count[0];
    } else {
      r[1] += d;
      ++count[1];
    }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) r[s] += __shfl_xor_sync(0xffffffffu, r[s], d);
    count[s] = __reduce_add_sync(0xffffffffu, count[s]);
    if ((threadIdx.x & 31) == 0) {
      sums[s][threadIdx.x >> 5] = r[s];
      counts[s][threadIdx.x >> 5] = count[s];
    }
  }
  __syncthreads();
  __shared__ float weight[2];
  if (threadIdx.x == 0) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      r[s] = 0.0;
      count[s] = 0;
      for (int i = 0; i < kPairThreads / 32; ++i) {
        r[s] += sums[s][i];
        count[s] += counts[s][i];
      }
      n[s] = ob.average && count[s] > 0 ? count[s] : 1;
      r[s] /= n[s];
    }
    const float m = static_cast<float>(ob.beta * (r[0] - r[1]));
    const float away = expf(-fabsf(m)), soft = log1pf(away);       // log(1 + e^-|m|)
    const float sigma = (m > 0.0f ? away : 1.0f) / (1.0f + away);  // sigma(-m)
    float loss = (1.0f - ob.smooth) * (soft + fmaxf(-m, 0.0f));
    if (ob.smooth > 0.0f) loss += ob.smooth * (soft + fmaxf(m, 0.0f));  // (not 0 times an infinite margin)
    if (!fits || m != m) loss = NAN;
    if (ob.loss) ob.loss[p] = loss;
    if (ob.ratios) {
      ob.ratios[2 * p] = fits ? static_cast<float>(r[0]) : NAN;
      ob.ratios[2 * p + 1] = fits ? static_cast<float>(r[1]) : NAN;
    }
    if (ob.dloss) {
      // d loss / d m = e - sigma(-m), and w is the slope along nll
      const float slope = ob.beta * (sigma - ob.smooth) * ob.dloss[p];
      weight[0] = static_cast<float>(slope / n[0]);
      weight[1] = static_cast<float>(-slope / n[1]);
      const unsigned most = max(count[0] > 0 ? weight_bits(weight[0]) : 0u,
                                count[1] > 0 ? weight_bits(weight[1]) : 0u);
      atomicMax(wt.wmax, fits ? most : kNanBits);
    }
  }
  if (!ob.dloss) return;
  __syncthreads();
  for (int64_t t = o[0] + threadIdx.x; fits && t < o[2]; t += kPairThreads)
    if (index[t] != ignore) wt.put(t, weight[t >= o[1]]);
}

// A thread a row (Schulman et al., 2017; the penalty's unbiased, never negative estimate is Schulman's
// of 2020):
//   r = exp(logp - old),   loss = -min(r A, clip(r, low, high) A) + kl (e^d - d - 1),  d = reference - logp
// The slope along logp is -r A where the first is the smaller, else 0, and kl (1 - e^d).  Comparisons
// are such that a NaN goes through.
__global__ void __launch_bounds__(256)
    tg_head_policy_kernel(Objective ob, const float* nll, const int64_t* __restrict__ index,
                          int64_t ignore, int64_t rows, Weights wt) {
  const int64_t r = blockIdx.x * int64_t(blockDim.x) + threadIdx.x;
  tg::chain_wait();
  tg::chain_release();
  unsigned most = 0;
  if (r < rows) {
    float loss = 0.0f, logp = 0.0f, slope = 0.0f;
    if (index[r] != ignore) {
      logp = -nll[r];
      const float ratio = expf(logp - ob.old[r]), adv = ob.advantage[r];
      const float kept = ratio < ob.low ? ob.low : ratio > ob.high ? ob.high : ratio;
      // (a ratio beyond float32's range times an advantage of 0 is 0; a NaN stays one)
      const float a = adv == 0.0f && ratio == INFINITY ? 0.0f : ratio * adv, b = kept * adv;
      const bool clipped = a > b;
      loss = clipped ? -b : -a;
      slope = clipped ? 0.0f : -a;
      if (ob.kl > 0.0f) {
        const float d = ob.reference[r] - logp, e = expm1f(d);
        loss += ob.kl * (d < 100.0f ? e - d : e);  // (not infinity less itself; a NaN is e's)
        slope -= ob.kl * e;
      }
    }
    if (ob.loss) ob.loss[r] = loss;
    if (ob.logp) ob.logp[r] = logp;
    if (ob.dloss && index[r] != ignore) {
      const float w = -slope * ob.dloss[r];
      wt.put(r, w);
      most = weight_bits(w);
    }
  }
  if (!ob.dloss) return;
  most = __reduce_max_sync(0xffffffffu, most);
  if ((threadIdx.x & 31) == 0 && most) atomicMax(wt.wmax, most);
}

// Every row's weight NaN if any pair's offsets are wrong.
__global__ void __launch_bounds__(256)
    tg_head_spoil_kernel(const unsigned* wmax, float* w, int64_t rows) {
  const int64_t r = blockIdx.x * int64_t(blockDim.x) + threadIdx.x;
  if (r < rows && *wmax == kNanBits) w[r] = NAN;
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
bool misaligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1024;
constexpr int64_t kMaxLd = int64_t{1} << 36;
constexpr int64_t kMaxElements = int64_t{1} << 44;
// Logits of a piece by default: 2 GiB of float32, 1 GiB of G.  Fewer, longer pieces cost less: a
// piece adds one pass of reads and writes over dW in float32.
constexpr int64_t kPieceLogits = int64_t{1} << 29;
// A TMA box of 128 rows of a matrix of fewer than eight (the rows of a swizzle atom) takes longer at
// some addresses: one token against 28672 x 8192, memory-bound, took 87 or 112 us by where the token
// lay, and never more than 88 from eight rows on.  So small operands lie in scratch of that many
// rows; what the others hold does not matter, an MMA's rows have nothing to do with each other.
constexpr int64_t kLeastRows = 8;
// Up to so many tokens the products are bound by W's and dW's bytes, not by the tensor cores, and G is
// kept in two fp16 parts (22 bits), as twice the rows of one product: with few rows its largest entries
// may all round badly (the gradients' error 0.00032 of their size, with two parts 0.00021, which is
// their own rounding to fp16; more tokens average to 0.0003).  It costs up to 3% of a step (64 tokens,
// 28672 classes of 4096: 160 against 155 us).
constexpr int64_t kFineTokens = 64;
// Columns of V that one accumulator sums for dX, tokens for dW.  The tensor core cuts off where it adds
// (tg_head_kernel.cuh), so a long sum shrinks: dX over 65536 columns in one accumulator by 1.2e-4 of
// itself, over 120000 by 2.2e-4, as much as its rounding to fp16, and by 2e-5 in accumulators of this
// length.  More splits (or, for dW, pieces) are added in float32: 1 to 2% of a step (2048 tokens of 28672 x
// 8192 in two splits 1862 us, in one 1830).
constexpr int64_t kSumLength = 16384;
// Without logits a token's scratch is its statistics: 1 GiB of them.
constexpr int64_t kPieceStats = int64_t{1} << 27;

// A stream beside the caller's, one a device, and the events that fork to it and join from it; held by
// one call at a time while that enqueues.
struct Side {
  bool ready = false;
  cudaStream_t stream = nullptr;
  cudaEvent_t start = nullptr, done = nullptr;
  std::mutex mu;
};
cudaError_t side_stream(Side** out) {
  static Side sides[64];  // device_info has refused devices past 63
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  Side& s = sides[dev & 63];
  std::lock_guard<std::mutex> lock(s.mu);
  if (!s.ready) {
    if ((e = cudaStreamCreateWithFlags(&s.stream, cudaStreamNonBlocking)) != cudaSuccess ||
        (e = cudaEventCreateWithFlags(&s.start, cudaEventDisableTiming)) != cudaSuccess ||
        (e = cudaEventCreateWithFlags(&s.done, cudaEventDisableTiming)) != cudaSuccess)
      return e;
    s.ready = true;
  }
  *out = &s;
  return cudaSuccess;
}

bool capturing(cudaStream_t stream) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusActive;
  if (cudaStreamIsCapturing(stream, &status) == cudaSuccess)
    return status != cudaStreamCaptureStatusNone;
  cudaGetLastError();  // the legacy stream while another one is captured
  return true;
}
// Elements of W from which dX and dW run side by side.
constexpr int64_t kSideWork = int64_t{12} << 20;

// One call's arguments beside the sizes; `top` > 0 makes it distillation.
struct Head {
  const void* X;
  const void* W;
  const int64_t* index;  // targets, or rows of ldt entries
  const void* teacher;
  int teacher_f32, top;
  int64_t ldt, ignore;
  const float* dloss;
  float *loss, *lse;
  void *dX, *dW;
  int64_t T, V, D, ldx, ldw, lddx, lddw;
  float scale;
  tg_head_options o;
  Objective ob;          // kind 0: the losses themselves
  bool precise;          // logits of an objective, or for one
};

// Parts of one scratch block, each 256-byte aligned.
struct Layout {
  int64_t bytes = 0;
  int64_t add(int64_t n) {
    const int64_t at = bytes;
    bytes += round_up(std::max<int64_t>(n, 1), 256);
    return at;
  }
};

tg_status check(const Head& h) {
  if (h.T < 0 || h.V < 1 || h.D < 1 || h.T > kMaxRows || h.V > kMaxRows || h.D > kMaxRows)
    return TG_ERR_INVALID_ARG;
  if (h.o.layout != TG_HEAD_VOCAB_MAJOR && h.o.layout != TG_HEAD_WIDTH_MAJOR)
    return TG_ERR_INVALID_ARG;
  // sizes whose products leave 64 bits could only come with pointers to nothing
  if (h.T > kMaxElements / h.D || h.V > kMaxElements / h.D) return TG_ERR_INVALID_ARG;
  if (h.o.piece_rows < 0 || h.o.timeout_ms < 0) return TG_ERR_INVALID_ARG;
  if (!(h.scale > 0.0f) || !(h.scale <= 3.0e38f)) return TG_ERR_INVALID_ARG;
  const int64_t w_cols = h.o.layout == TG_HEAD_VOCAB_MAJOR ? h.D : h.V;
  auto bad = [](int64_t ld, int64_t n) { return ld < n || ld > kMaxLd; };
  if (bad(h.ldx, h.D) || bad(h.ldw, w_cols)) return TG_ERR_INVALID_ARG;
  if ((h.dX && bad(h.lddx, h.D)) || (h.dW && bad(h.lddw, w_cols))) return TG_ERR_INVALID_ARG;
  if (h.top < 0 || h.top > TG_HEAD_MAX_TOP || (h.top > 0 && bad(h.ldt, h.top)))
    return TG_ERR_INVALID_ARG;
  if (h.T > 0) {
    if (!h.X || !h.W || !h.index || (h.top > 0 && !h.teacher)) return TG_ERR_INVALID_ARG;
    if ((h.dX || h.dW) && h.ob.kind == 0 && !h.dloss) return TG_ERR_INVALID_ARG;
  }
  if (misaligned(h.X, 2) || misaligned(h.W, 2) || misaligned(h.dX, 2) || misaligned(h.dW, 2) ||
      misaligned(h.index, 8) || misaligned(h.teacher, h.teacher_f32 ? 4 : 2) ||
      misaligned(h.dloss, 4) || misaligned(h.loss, 4) || misaligned(h.lse, 4))
    return TG_ERR_MISALIGNED;
  return TG_OK;
}

// Tokens whose logits (or statistics, per_row of either) are in scratch at a time.
int64_t piece_of(const Head& h, int64_t per_row, int64_t budget) {
  if (h.o.piece_rows)
    return std::min({h.o.piece_rows, h.T, std::max<int64_t>(kMaxElements / per_row, 1)});
  if (h.T <= budget / per_row) return h.T;
  const int64_t most = std::max<int64_t>(budget / per_row / 256 * 256, 256);
  return std::min(h.T, round_up(cdiv(h.T, cdiv(h.T, most)), 256));
}

// An objective's losses and weights from nll (chained: the launch before it is a kernel).
cudaError_t launch_objective(const Head& h, const float* nll, const Weights& wt, bool chained,
                             cudaStream_t stream) {
  const Objective& ob = h.ob;
  if (ob.kind == kPolicy)
    return tg::launch_chained(tg_head_policy_kernel, chained, dim3(static_cast<unsigned>(cdiv(h.T, 256))),
                              256, 0, stream, ob, nll, h.index, h.ignore, h.T, wt);
  if (ob.pairs == 0) return cudaSuccess;
  return tg::launch_chained(tg_head_pairs_kernel, chained, dim3(static_cast<unsigned>(ob.pairs)),
                            kPairThreads, 0, stream, ob, nll, h.index, h.ignore, h.T, wt);
}

tg_status run_head(const Head& h, cudaStream_t stream) {
  tg_status st = check(h);
  if (st != TG_OK) return st;
  int sms = 0;
  unsigned* err = nullptr;
  cudaError_t e;
  const bool by_vocab = h.o.layout == TG_HEAD_VOCAB_MAJOR;
  const int64_t w_rows = by_vocab ? h.V : h.D, w_cols = by_vocab ? h.D : h.V;
  if (h.T == 0 && !h.dW) return TG_OK;
  if ((st = tg::device_info(&sms, &err)) != TG_OK) return st;
  if (h.T == 0) {  // the sum over no rows
    e = cudaMemset2DAsync(h.dW, size_t(h.lddw) * 2, 0, size_t(w_cols) * 2, size_t(w_rows), stream);
    return e == cudaSuccess ? TG_OK : tg::record_cuda_error(e);
  }
  const bool grad = h.dX || h.dW;
  // The logits are needed again for a gradient, and for a teacher's entries, which without a
  // gradient are also had as dot products of their own: 2 top D bytes a token against 4 V to store
  // its logits (1024 tokens, V = 131072, D = 1024, 32 entries: 208 against 251 us).  A row of W is
  // contiguous only in a head stored V x D.
  const bool pick = h.top > 0 && !grad && by_vocab && h.top * h.D <= 2 * h.V;
  const bool store = grad || (h.top > 0 && !pick);
  const int64_t ldz = round_up(h.V, 32), ldg = round_up(h.V, 64);
  const int64_t tiles = 2 * cdiv(h.V, 128);  // statistics of a row, at most
  int64_t piece = piece_of(h, store ? ldz : tiles, store ? kPieceLogits : kPieceStats);
  if (h.dW && piece < h.T) piece = std::min(piece, kSumLength);
  const bool sum_w = h.dW && piece < h.T;  // dW is summed over pieces in float32
  const bool fine = grad && h.T <= kFineTokens && piece == h.T;
  const bool objective = h.ob.kind != 0;  // with a gradient and in one piece (run_objective)
  const int64_t parts = fine ? 2 : 1;  // of G

  Layout lay;
  // Rows that TMA cannot read in place are copied once for all pieces and products, and so are the
  // tokens where there are fewer than kLeastRows.
  const bool copy_x = misaligned(h.X, 16) || h.ldx % 8 != 0 || h.T < kLeastRows;
  const bool copy_w = misaligned(h.W, 16) || h.ldw % 8 != 0;
  const int64_t ldxp = round_up(h.D, 64), ldwp = round_up(w_cols, 64), ldw32 = round_up(w_cols, 32);
  const int64_t at_z = lay.add(store ? piece * ldz * 4 : 0);
  const int64_t at_stats = lay.add(tiles * piece * int64_t(sizeof(float2)));
  const int64_t at_picked = lay.add(store ? 0 : piece * std::max(h.top, 1) * 4);
  const int64_t at_info = lay.add(piece * int64_t(sizeof(RowInfo)));
  const int64_t at_small = lay.add(2 * 4);
  const int64_t at_nll = lay.add(objective ? h.T * 4 : 0);
  const int64_t at_g = lay.add(grad ? std::max(parts * piece, kLeastRows) * ldg * 2 : 0);
  const int64_t at_x2 = lay.add(fine && h.dW ? 2 * h.T * ldxp * 2 : 0);
  const int64_t at_q = lay.add(grad && h.top ? piece * h.top * 4 : 0);
  const int64_t at_x = lay.add(copy_x ? std::max(h.T, kLeastRows) * ldxp * 2 : 0);
  const int64_t at_w = lay.add(copy_w ? w_rows * ldwp * 2 : 0);
  const int64_t at_w32 = lay.add(sum_w ? w_rows * ldw32 * 4 : 0);
  uint8_t* mem = nullptr;
  if ((st = tg::scratch_alloc(size_t(lay.bytes), stream, reinterpret_cast<void**>(&mem))) != TG_OK)
    return st;
  auto done = [&](tg_status s) {
    const cudaError_t fe = cudaFreeAsync(mem, stream);
    return s == TG_OK && fe != cudaSuccess ? tg::record_cuda_error(fe) : s;
  };
  float* z = store ? reinterpret_cast<float*>(mem + at_z) : nullptr;
  float* picked = reinterpret_cast<float*>(mem + at_picked);
  float2* stats = reinterpret_cast<float2*>(mem + at_stats);
  RowInfo* info = reinterpret_cast<RowInfo*>(mem + at_info);
  unsigned* wmax = grad ? reinterpret_cast<unsigned*>(mem + at_small) : nullptr;
  float* alpha = grad ? reinterpret_cast<float*>(mem + at_small) + 1 : nullptr;
  uint16_t* g = reinterpret_cast<uint16_t*>(mem + at_g);
  float* q = grad && h.top ? reinterpret_cast<float*>(mem + at_q) : nullptr;
  float* w32 = reinterpret_cast<float*>(mem + at_w32);

  const uint16_t* X = static_cast<const uint16_t*>(h.X);
  const void* W = h.W;
  int64_t ldx = h.ldx, ldw = h.ldw;
  if (copy_x) {
    uint16_t* xp = reinterpret_cast<uint16_t*>(mem + at_x);
    if ((e = tg::launch_pack_rows(X, ldx, xp, ldxp, h.T, h.D, sms, stream)) != cudaSuccess)
      return done(tg::record_cuda_error(e));
    X = xp;
    ldx = ldxp;
  }
  if (copy_w) {
    if ((e = tg::launch_pack_rows(W, ldw, mem + at_w, ldwp, w_rows, w_cols, sms, stream)) !=
        cudaSuccess)
      return done(tg::record_cuda_error(e));
    W = mem + at_w;
    ldw = ldwp;
  }
  if (grad && !objective) {
    // one block for what it can read in a few microseconds, else several on a zeroed maximum
    const int64_t reads = h.T * std::max(h.top, 1);
    const int blocks = reads <= 4096 ? 1 : static_cast<int>(std::min<int64_t>(cdiv(h.T, 256), sms));
    const int threads = blocks == 1 ? static_cast<int>(std::min<int64_t>(round_up(h.T, 32), 1024)) : 256;
    if (blocks > 1 && (e = cudaMemsetAsync(wmax, 0, 4, stream)) != cudaSuccess)
      return done(tg::record_cuda_error(e));
    tg_head_weight_kernel<<<blocks, threads, 0, stream>>>(h.dloss, h.index, h.ldt, h.top, h.ignore,
                                                          h.T, wmax);
    if ((e = cudaGetLastError()) != cudaSuccess) return done(tg::record_cuda_error(e));
  }

  tg_options gemm_opt;
  std::memset(&gemm_opt, 0, sizeof(gemm_opt));
  gemm_opt.timeout_ms = h.o.timeout_ms;
  gemm_opt.debug_flags = h.o.debug_flags;
  const float c = h.scale * kLog2e;
  // the kernels between the products, each chained to the launch before it; the first error stays
  e = cudaSuccess;
  auto chain = [&](auto kern, dim3 grid, int threads, const auto&... args) {
    const cudaError_t le = tg::launch_chained(kern, true, grid, threads, 0, stream, args...);
    if (e == cudaSuccess) e = le;
  };
  for (int64_t t0 = 0; t0 < h.T; t0 += piece) {
    const int64_t n = std::min(piece, h.T - t0);
    const uint16_t* x = X + t0 * ldx;
    const int64_t* index = h.index + t0 * (h.top ? h.ldt : 1);
    const void* teacher = h.teacher == nullptr ? nullptr
                                               : static_cast<const uint8_t*>(h.teacher) +
                                                     t0 * h.ldt * (h.teacher_f32 ? 4 : 2);
    const float* dloss = grad && !objective ? h.dloss + t0 : nullptr;
    float* nll = reinterpret_cast<float*>(mem + at_nll);
    float* loss = objective ? nll : h.loss ? h.loss + t0 : nullptr;
    tg::GemmExtra ex;
    int block_n = 0;
    tg::LogitsExtra lx;
    lx.z = z;
    lx.ldz = ldz;
    lx.stats = stats;
    lx.stat_c = c;
    lx.target = store || h.top ? nullptr : reinterpret_cast<const long long*>(index);
    lx.picked = picked;
    lx.block_n = &block_n;
    lx.precise = h.precise;
    lx.width = h.D;
    std::memset(&ex, 0, sizeof(ex));
    ex.logits = &lx;
    if (h.T < kLeastRows) ex.a_rows = kLeastRows - t0;
    ex.chained = (grad && !objective) || copy_x || copy_w || t0 > 0;
    st = tg::gemm_extra(0, by_vocab, x, W, nullptr, n, h.V, h.D, ldx, ldw, h.V, ex, &gemm_opt,
                        stream);
    if (st != TG_OK) return done(st);
    if (pick)
      chain(tg_head_pick_kernel,
            dim3(static_cast<unsigned>(
                std::min<int64_t>(cdiv(n * cdiv(h.top, kPickRows), 8), 16 * int64_t(sms)))),
            256, x, ldx, static_cast<const uint16_t*>(W), ldw, index, h.ldt, h.top, n, h.V,
            static_cast<int>(h.D), picked);
    chain(tg_head_rows_kernel, dim3(static_cast<unsigned>(n)), kRowThreads,
        stats, static_cast<int>(2 * cdiv(h.V, block_n)), Logits{z, ldz, picked}, h.scale, h.V, index, h.ignore,
        teacher, h.teacher_f32, h.ldt, h.top, dloss, objective ? nullptr : wmax, loss,
        h.lse ? h.lse + t0 : nullptr, info, q,
        objective ? reinterpret_cast<float*>(wmax) : alpha,  // objective: zeroes the maximum
        h.precise ? kExpLift : 0.0f);
    if (e != cudaSuccess) return done(tg::record_cuda_error(e));
    if (objective) {
      e = launch_objective(h, nll, Weights{wmax, info, nullptr}, true, stream);
      if (e != cudaSuccess) return done(tg::record_cuda_error(e));
    }
    if (!grad) continue;
    const int64_t lo = fine ? n * ldg : 0;
    uint16_t* x2 = fine && h.dW ? reinterpret_cast<uint16_t*>(mem + at_x2) : nullptr;
    auto grad_kernel = objective ? (fine ? tg_head_grad_kernel<true, true> : tg_head_grad_kernel<false, true>)
                                 : (fine ? tg_head_grad_kernel<true, false> : tg_head_grad_kernel<false, false>);
    chain(grad_kernel,
          dim3(static_cast<unsigned>(cdiv(h.V, 2048)),
               static_cast<unsigned>(std::min<int64_t>(n, 65535))),
          256, z, ldz, c, info, n, h.V, g, ldg, lo, x, ldx, x2, ldxp, static_cast<int>(h.D), wmax, h.scale,
          alpha);
    if (h.top)
      chain(tg_head_teacher_grad_kernel, dim3(static_cast<unsigned>(cdiv(n, 4))), 128, index, h.ldt,
            h.top, q, z, ldz, c, info, n, h.V, reinterpret_cast<__half*>(g), ldg, lo);
    if (e != cudaSuccess) return done(tg::record_cuda_error(e));
    // Few tokens: dX reads W and dW writes as much, each bound by HBM, where writes alone run at 3.9 TB/s
    // and reads and writes together at up to 6.8.  So the two run side by side, dX on a third of the
    // SMs, where the work is worth a second stream.  dX's splits of V are then whole waves both on that
    // third and on all SMs, and the same in a graph that is being captured, where the two run one after
    // the other (the stream would belong to the graph until its end).  28672 x 4096: one token 157 us, one
    // after the other 175, 16 tokens 153 and 160, 64 tokens 160 and 169; 32 tokens of 28672 x 8192 287 and
    // 285, 128 of 131072 x 2048 367 and 358, with one wave of splits over the third 322 and 388.
    const int64_t width = h.D <= 2048 ? 128 : 256;  // narrow W: narrow tiles
    const int sms_x = sms / 3;
    const bool beside = h.dX && h.dW && n == h.T && n <= 128 && h.V * h.D >= kSideWork &&
                        2 * cdiv(h.D, width) <= 3 * sms_x;
    const bool both = beside && !capturing(stream);
    Side* side = nullptr;
    std::unique_lock<std::mutex> lock;
    cudaStream_t stream_w = stream;
    if (both) {
      if ((e = side_stream(&side)) != cudaSuccess) return done(tg::record_cuda_error(e));
      lock = std::unique_lock<std::mutex>(side->mu);
      if ((e = cudaEventRecord(side->start, stream)) != cudaSuccess ||
          (e = cudaStreamWaitEvent(side->stream, side->start, 0)) != cudaSuccess)
        return done(tg::record_cuda_error(e));
      stream_w = side->stream;
    }
    st = TG_OK;
    if (h.dW) {  // G^T X (V x D), or X^T G (D x V)
      std::memset(&ex, 0, sizeof(ex));
      ex.alpha = alpha;
      ex.chained = !both;
      ex.max_k = kSumLength;
      ex.rows = h.precise;
      if (sum_w) {  // the first piece writes the sums, the last takes them into its epilogue
        ex.ld32 = ldw32;
        if (t0 + piece < h.T) {
          ex.out32 = w32;
          ex.add = t0 > 0;
        } else {
          ex.addend = w32;
        }
      }
      // With few tokens dW's epilogue is the work: a tile of one CTA is better at it than a pair's
      // (28672 x 1024 from 128 tokens 20.5 against 26.7 us, 131072 x 2048 from 64 135 against 173; at
      // 512 tokens they are even).
      tg_options opt = gemm_opt;
      const uint16_t* xs = fine ? x2 : x;
      const int64_t ldxs = fine ? ldxp : ldx;
      if (n <= 256 && !(ex.out32 && ex.add)) opt.pair = -1;
      if (beside) opt.split_k = 1;  // of two k-blocks at most: the same sums on any number of SMs
      if (both) opt.max_ctas = sms - sms_x;
      st = by_vocab
               ? tg::gemm_extra(1, 0, g, xs, h.dW, h.V, h.D, parts * n, ldg, ldxs, h.lddw, ex, &opt,
                                stream_w)
               : tg::gemm_extra(1, 0, xs, g, h.dW, h.D, h.V, parts * n, ldxs, ldg, h.lddw, ex, &opt,
                                stream_w);
    }
    if (h.dX && st == TG_OK) {  // G (n x V) times W (V x D, or stored D x V)
      std::memset(&ex, 0, sizeof(ex));
      ex.alpha = alpha;
      ex.chained = !both;
      ex.a_rows = std::max(parts * n, kLeastRows);
      ex.fold = fine;
      ex.max_k = kSumLength;
      // One row of tiles reads W once at the memory's rate, if the splits of V make one wave of
      // blocks over the SMs (28672 x 1024 for one token 17 against 25 us as planned from the
      // products' costs and for 128 tokens 20.4 against 20.7, 131072 x 4096 166 against 203, 28672 x
      // 8192 for one token 77 against 119; two rows of tiles gain at some widths and lose at others).
      // Beside dW they make three waves over a third of the SMs.
      tg_options opt = gemm_opt;
      const int64_t splits = std::max(
          std::min({(beside ? 3 * sms_x : sms) / cdiv(h.D, width), cdiv(h.V, 128), int64_t(32)}),
          cdiv(h.V, kSumLength));
      if (n <= 128 && splits > 1) {
        opt.pair = -1;
        opt.block_n = static_cast<int>(width);
        opt.split_k = static_cast<int>(splits);
      }
      if (both) opt.max_ctas = sms_x;
      opt.force_workspace = fine ? 1 : 0;  // the sum of the parts is taken there
      st = tg::gemm_extra(0, !by_vocab, g, W, static_cast<uint16_t*>(h.dX) + t0 * h.lddx, parts * n,
                          h.D, h.V, ldg, ldw, h.lddx, ex, &opt, stream);
    }
    if (both) {  // joined on success and on error alike: the scratch is freed on `stream`
      if ((e = cudaEventRecord(side->done, side->stream)) == cudaSuccess)
        e = cudaStreamWaitEvent(stream, side->done, 0);
      if (e != cudaSuccess) {
        cudaStreamSynchronize(side->stream);
        if (st == TG_OK) st = tg::record_cuda_error(e);
      }
    }
    if (st != TG_OK) return done(st);
  }
  return done(TG_OK);
}

// A preference or policy loss.  The logits of all tokens fit into one piece: one product, the losses,
// and the gradient from the kept logits.  Else (and without a gradient) the log probabilities first,
// which keep no logits, then the losses, then cross entropy's gradient with the weights found: one
// product more.
tg_status run_objective(const Head& h, cudaStream_t stream) {
  tg_status st = check(h);
  if (st != TG_OK) return st;
  const Objective& ob = h.ob;
  const bool grad = h.dX || h.dW;
  if (ob.kind == kPreference) {
    if (ob.pairs < 0 || ob.pairs > kMaxRows / 2 || (ob.pairs > 0 && !ob.offsets)) return TG_ERR_INVALID_ARG;
    if (!(ob.beta > 0.0f) || !(ob.beta <= 3.0e38f) || !(ob.smooth >= 0.0f) || !(ob.smooth < 1.0f))
      return TG_ERR_INVALID_ARG;
    if (ob.pairs > 0 && grad && !ob.dloss) return TG_ERR_INVALID_ARG;
  } else {
    if (!(ob.low >= 0.0f) || !(ob.low <= 1.0f) || !(ob.high >= 1.0f) || !(ob.high <= 3.0e38f) ||
        !(ob.kl >= 0.0f) || !(ob.kl <= 3.0e38f))
      return TG_ERR_INVALID_ARG;
    if (h.T > 0 && (!ob.old || !ob.advantage || (ob.kl > 0.0f && !ob.reference) || (grad && !ob.dloss)))
      return TG_ERR_INVALID_ARG;
  }
  if (misaligned(ob.dloss, 4) || misaligned(ob.loss, 4) || misaligned(ob.reference, 4) ||
      misaligned(ob.offsets, 8) || misaligned(ob.ratios, 4) || misaligned(ob.old, 4) ||
      misaligned(ob.advantage, 4) || misaligned(ob.logp, 4))
    return TG_ERR_MISALIGNED;
  if (grad && h.T > 0 && piece_of(h, round_up(h.V, 32), kPieceLogits) == h.T) return run_head(h, stream);
  if (h.T == 0 && ob.kind == kPolicy) return run_head(h, stream);
  int sms = 0;
  unsigned* err = nullptr;
  if ((st = tg::device_info(&sms, &err)) != TG_OK) return st;
  Layout lay;
  // (the weights are zeroed together with their maximum; a policy's log probabilities are computed in place)
  const bool own_nll = !(ob.kind == kPolicy && ob.logp);
  const int64_t at_nll = lay.add(own_nll ? h.T * 4 : 0);
  const int64_t at_small = lay.add(grad ? 4 : 0), at_w = lay.add(grad ? h.T * 4 : 0);
  uint8_t* mem = nullptr;
  if (lay.bytes > 0 &&  // (none without rows and a gradient)
      (st = tg::scratch_alloc(size_t(lay.bytes), stream, reinterpret_cast<void**>(&mem))) != TG_OK)
    return st;
  float* nll = own_nll ? reinterpret_cast<float*>(mem + at_nll) : ob.logp;
  float* w = reinterpret_cast<float*>(mem + at_w);
  const Weights wt{reinterpret_cast<unsigned*>(mem + at_small), nullptr, w};
  cudaError_t e = grad ? cudaMemsetAsync(mem + at_small, 0, size_t(lay.bytes - at_small), stream) : cudaSuccess;
  if (e != cudaSuccess) st = tg::record_cuda_error(e);
  Head inner = h;
  inner.ob.kind = 0;
  inner.loss = nll;
  inner.dX = inner.dW = nullptr;
  if (st == TG_OK) st = run_head(inner, stream);
  if (st == TG_OK) {
    e = launch_objective(h, nll, wt, false, stream);
    if (e == cudaSuccess && grad && ob.kind == kPreference && h.T > 0) {
      tg_head_spoil_kernel<<<static_cast<unsigned>(cdiv(h.T, 256)), 256, 0, stream>>>(wt.wmax, w, h.T);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) st = tg::record_cuda_error(e);
  }
  if (st == TG_OK && grad) {
    inner = h;
    inner.ob.kind = 0;
    inner.loss = nullptr;
    inner.dloss = w;
    st = run_head(inner, stream);
  }
  e = mem ? cudaFreeAsync(mem, stream) : cudaSuccess;
  return st == TG_OK && e != cudaSuccess ? tg::record_cuda_error(e) : st;
}

tg_head_options options_or_default(const tg_head_options* opt) {
  tg_head_options o;
  std::memset(&o, 0, sizeof(o));
  if (opt) o = *opt;
  return o;
}

}  // namespace

extern "C" {

tg_status tg_linear_cross_entropy_f16(const void* X, const void* W, const int64_t* target,
                                      int64_t ignore_index, float logit_scale, const float* dloss,
                                      float* loss, float* lse, void* dX, void* dW, int64_t T,
                                      int64_t V, int64_t D, int64_t ldx, int64_t ldw, int64_t lddx,
                                      int64_t lddw, const tg_head_options* opt,
                                      tg_stream_t stream) {
  Head h;
  std::memset(&h, 0, sizeof(h));
  h.X = X;
  h.W = W;
  h.index = target;
  h.ignore = ignore_index;
  h.dloss = dloss;
  h.loss = loss;
  h.lse = lse;
  h.dX = dX;
  h.dW = dW;
  h.T = T, h.V = V, h.D = D;
  h.ldx = ldx, h.ldw = ldw, h.lddx = lddx, h.lddw = lddw;
  h.scale = logit_scale;
  h.o = options_or_default(opt);
  return run_head(h, reinterpret_cast<cudaStream_t>(stream));
}

tg_status tg_linear_distill_f16(const void* X, const void* W, const int64_t* teacher_index,
                                const void* teacher_logits, int teacher_type, int top, int64_t ldt,
                                float temperature, const float* dloss, float* loss, float* lse,
                                void* dX, void* dW, int64_t T, int64_t V, int64_t D, int64_t ldx,
                                int64_t ldw, int64_t lddx, int64_t lddw,
                                const tg_head_options* opt, tg_stream_t stream) {
  if (top < 1 || !(temperature > 0.0f) || !(temperature <= 3.0e38f)) return TG_ERR_INVALID_ARG;
  if (teacher_type != TG_TYPE_F16 && teacher_type != TG_TYPE_F32) return TG_ERR_INVALID_ARG;
  Head h;
  std::memset(&h, 0, sizeof(h));
  h.X = X;
  h.W = W;
  h.index = teacher_index;
  h.teacher = teacher_logits;
  h.teacher_f32 = teacher_type == TG_TYPE_F32;
  h.top = top;
  h.ldt = ldt;
  h.dloss = dloss;
  h.loss = loss;
  h.lse = lse;
  h.dX = dX;
  h.dW = dW;
  h.T = T, h.V = V, h.D = D;
  h.ldx = ldx, h.ldw = ldw, h.lddx = lddx, h.lddw = lddw;
  h.scale = 1.0f / temperature;
  h.o = options_or_default(opt);
  return run_head(h, reinterpret_cast<cudaStream_t>(stream));
}

tg_status tg_linear_preference_f16(const void* X, const void* W, const int64_t* target,
                                   int64_t ignore_index, float logit_scale, const int64_t* offsets,
                                   int64_t pairs, const float* reference, float beta,
                                   float label_smoothing, int average, const float* dloss, float* loss,
                                   float* ratios, void* dX, void* dW, int64_t T, int64_t V, int64_t D,
                                   int64_t ldx, int64_t ldw, int64_t lddx, int64_t lddw,
                                   const tg_head_options* opt, tg_stream_t stream) {
  Head h;
  std::memset(&h, 0, sizeof(h));
  h.X = X;
  h.W = W;
  h.index = target;
  h.ignore = ignore_index;
  h.dX = dX;
  h.dW = dW;
  h.T = T, h.V = V, h.D = D;
  h.ldx = ldx, h.ldw = ldw, h.lddx = lddx, h.lddw = lddw;
  h.scale = logit_scale;
  h.o = options_or_default(opt);
  h.ob.kind = kPreference;
  h.precise = true;
  h.ob.dloss = dX || dW ? dloss : nullptr;
  h.ob.loss = loss;
  h.ob.reference = reference;
  h.ob.offsets = offsets;
  h.ob.pairs = pairs;
  h.ob.beta = beta;
  h.ob.smooth = label_smoothing;
  h.ob.average = average != 0;
  h.ob.ratios = ratios;
  return run_objective(h, reinterpret_cast<cudaStream_t>(stream));
}

tg_status tg_linear_policy_f16(const void* X, const void* W, const int64_t* target,
                               int64_t ignore_index, float logit_scale, const float* old_logp,
                               const float* advantage, const float* reference, float clip_low,
                               float clip_high, float kl_weight, const float* dloss, float* loss,
                               float* logp, void* dX, void* dW, int64_t T, int64_t V, int64_t D,
                               int64_t ldx, int64_t ldw, int64_t lddx, int64_t lddw,
                               const tg_head_options* opt, tg_stream_t stream) {
  Head h;
  std::memset(&h, 0, sizeof(h));
  h.X = X;
  h.W = W;
  h.index = target;
  h.ignore = ignore_index;
  h.dX = dX;
  h.dW = dW;
  h.T = T, h.V = V, h.D = D;
  h.ldx = ldx, h.ldw = ldw, h.lddx = lddx, h.lddw = lddw;
  h.scale = logit_scale;
  h.o = options_or_default(opt);
  h.ob.kind = kPolicy;
  h.precise = true;
  h.ob.dloss = dX || dW ? dloss : nullptr;
  h.ob.loss = loss;
  h.ob.reference = kl_weight > 0.0f ? reference : nullptr;
  h.ob.old = old_logp;
  h.ob.advantage = advantage;
  h.ob.low = 1.0f - clip_low;
  h.ob.high = 1.0f + clip_high;
  h.ob.kl = kl_weight;
  h.ob.logp = logp;
  return run_objective(h, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
