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
// G is rounded to fp16 once, the operand type of the products.  So that the many small
// probabilities stay normal fp16 numbers, G carries the factor 2^15 / max|w| (|p - q| <= 1, so
// nothing overflows) and alpha = s max|w| / 2^15 is applied to the float32 sums: a row of the
// largest weight keeps 11 bits of every p above 2^-29.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "tg_gemm_relu.h"
#include "tg_internal.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kGScale = 32768.0f;

// What the passes after the logits know of a row.
struct RowInfo {
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

// max |w_t| over the rows that count, as the bits of a non-negative float (the maximum does not
// depend on the order of the atomics).  top == 0: cross entropy; else a row counts when one of
// its `top` entries does.
__global__ void tg_head_weight_kernel(const float* __restrict__ dloss,
                                      const int64_t* __restrict__ index, int64_t ld, int top,
                                      int64_t ignore, int64_t rows, unsigned* wmax) {
  float m = 0.0f;
  for (int64_t r = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; r < rows;
       r += int64_t(gridDim.x) * blockDim.x) {
    bool live = top == 0 && index[r] != ignore;
    for (int j = 0; j < top && !live; ++j) live = index[r * ld + j] >= 0;
    if (live) m = fmaxf(m, fabsf(dloss[r]));
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((threadIdx.x & 31) == 0 && m > 0.0f) atomicMax(wmax, __float_as_uint(m));
}

__device__ __forceinline__ float row_factor(float w, float wmax) {
  return (wmax > 0.0f ? w / wmax : 0.0f * w) * kGScale;  // 0 * w keeps a NaN
}

// lse of 32 rows a block from their tiles' statistics; cross entropy's loss and RowInfo too (the
// targets' logits from z, or picked where z is not stored).
// alpha (one float): s max|w| / 2^15, written by the first block.
constexpr int kRowLanes = 16;
__global__ void __launch_bounds__(32 * kRowLanes)
    tg_head_rows_kernel(const float2* __restrict__ stats, int tiles, int64_t rows,
                        const float* __restrict__ z, int64_t ldz,
                        const float* __restrict__ picked, float scale, int64_t vocab,
                        const int64_t* __restrict__ target, int64_t ignore,
                        const float* __restrict__ dloss, const unsigned* __restrict__ wmax,
                        float* loss, float* lse, RowInfo* info, float* alpha) {
  __shared__ float2 part[kRowLanes][32];
  const int64_t r = blockIdx.x * int64_t(32) + threadIdx.x;
  float m = -INFINITY, s = 0.0f;
  if (r < rows) {
    for (int t = threadIdx.y; t < tiles; t += kRowLanes) {
      const float2 v = stats[t * rows + r];
      const float m1 = fmaxf(m, v.x);
      if (m1 == -INFINITY) {
        s += v.y;  // zero or NaN
      } else {
        s = s * exp2f(m - m1) + v.y * exp2f(v.x - m1);
        m = m1;
      }
    }
  }
  part[threadIdx.y][threadIdx.x] = make_float2(m, s);
  __syncthreads();
  const float w = wmax ? __uint_as_float(*wmax) : 0.0f;
  if (alpha && blockIdx.x == 0 && threadIdx.x == 0 && threadIdx.y == 0) *alpha = scale * w / kGScale;
  if (threadIdx.y != 0 || r >= rows) return;
  m = -INFINITY;
  for (int y = 0; y < kRowLanes; ++y) m = fmaxf(m, part[y][threadIdx.x].x);
  s = 0.0f;
  for (int y = 0; y < kRowLanes; ++y) {
    const float2 v = part[y][threadIdx.x];
    s += m == -INFINITY ? v.y : v.y * exp2f(v.x - m);
  }
  const float lse2 = m + log2f(s);
  if (lse) lse[r] = lse2 * kLn2;
  RowInfo ri;
  ri.lse2 = lse2;
  ri.gs = 0.0f;
  ri.target = -1;
  ri.pad = 0;
  if (target) {
    const int64_t y = target[r];
    const RowKind kind = target_kind(y, vocab, ignore);
    float l = 0.0f;
    if (kind == RowKind::kCounts) {
      ri.target = static_cast<int>(y);
      l = lse2 * kLn2 - scale * (z ? z[r * ldz + y] : picked[r]);
      if (dloss) ri.gs = row_factor(dloss[r], w);
    } else if (kind == RowKind::kBad) {
      l = ri.gs = NAN;
    }
    if (loss) loss[r] = l;
  }
  info[r] = ri;
}

// Entry e's teacher logit.
__device__ __forceinline__ float teacher_at(const void* t, int64_t at, int is_f32) {
  return is_f32 ? static_cast<const float*>(t)[at] : __half2float(static_cast<const __half*>(t)[at]);
}

// Distillation: a warp a row.  Entries with a negative index are not there; q is the softmax of
// the others (one at -inf has q = 0).  A row without entries, or whose entries are all -inf, has
// no teacher: loss 0 and no gradient.  q (float32, 0 for what is not there) is kept for the
// gradient when `q` is given.
__global__ void tg_head_distil_rows_kernel(const int64_t* __restrict__ index,
                                           const void* __restrict__ teacher, int teacher_f32,
                                           int64_t ldt, int top, int64_t rows,
                                           const float* __restrict__ z, int64_t ldz, float scale,
                                           int64_t vocab, const float* __restrict__ dloss,
                                           const unsigned* __restrict__ wmax, float* loss,
                                           RowInfo* info, float* q) {
  const int64_t r = (blockIdx.x * int64_t(blockDim.x) + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (r >= rows) return;
  const float c = scale * kLog2e;
  float m = -INFINITY;
  bool bad = false;
  for (int e = lane; e < top; e += 32) {
    const int64_t i = index[r * ldt + e];
    if (i < 0) continue;
    bad |= i >= vocab;
    const float u = teacher_at(teacher, r * ldt + e, teacher_f32);
    bad |= !(u < INFINITY);  // NaN or +inf
    m = fmaxf(m, u * c);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  bad = __any_sync(0xffffffffu, bad);
  float s = 0.0f;
  for (int e = lane; e < top && m > -INFINITY; e += 32)
    if (index[r * ldt + e] >= 0)
      s += exp2f(fmaf(teacher_at(teacher, r * ldt + e, teacher_f32), c, -m));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  const float lq = m + log2f(s), lse = info[r].lse2 * kLn2;
  float l = 0.0f;
  for (int e = lane; e < top; e += 32) {
    float qe = 0.0f;
    const int64_t i = index[r * ldt + e];
    if (i >= 0 && m > -INFINITY) {
      const float t2 = fmaf(teacher_at(teacher, r * ldt + e, teacher_f32), c, -lq);
      qe = exp2f(t2);
      if (qe > 0.0f && i < vocab) l += qe * (t2 * kLn2 - (scale * z[r * ldz + i] - lse));
    }
    if (q) q[r * top + e] = qe;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  if (lane == 0) {
    if (bad) l = NAN;
    if (loss) loss[r] = l;
    float gs = 0.0f;
    if (bad) gs = NAN;
    else if (dloss && m > -INFINITY) gs = row_factor(dloss[r], __uint_as_float(*wmax));
    info[r].gs = gs;
  }
}

// One value of G: gs (p - q).
__device__ __forceinline__ float grad_value(float z, float c, float lse2, float gs, float q) {
  return gs == 0.0f ? 0.0f : gs * (exp2f(fmaf(z, c, -lse2)) - q);
}

// G (fp16, rows of ldg) from the logits, eight columns of a row a thread; the target's -1 with it.
__global__ void __launch_bounds__(256)
    tg_head_grad_kernel(const float* __restrict__ z, int64_t ldz, float c,
                        const RowInfo* __restrict__ info, int64_t rows, int64_t vocab,
                        uint16_t* __restrict__ g, int64_t ldg) {
  const int64_t v0 = (blockIdx.x * int64_t(blockDim.x) + threadIdx.x) << 3;
  if (v0 >= vocab) return;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const RowInfo ri = info[r];
    const float4* src = reinterpret_cast<const float4*>(z + r * ldz + v0);
    const float4 a = __ldcs(src), b = __ldcs(src + 1);  // ldz and ldg are multiples of 8
    const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = grad_value(f[2 * i], c, ri.lse2, ri.gs, v0 + 2 * i == ri.target ? 1.0f : 0.0f);
      const float hi =
          grad_value(f[2 * i + 1], c, ri.lse2, ri.gs, v0 + 2 * i + 1 == ri.target ? 1.0f : 0.0f);
      const __half2 h = __floats2half2_rn(lo, hi);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(g + r * ldg + v0) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Distillation: G at the teacher's entries, a warp a row.  Entries of one token add up; each of
// them then writes the same value.
__global__ void tg_head_distil_grad_kernel(const int64_t* __restrict__ index, int64_t ldt, int top,
                                           const float* __restrict__ q, const float* __restrict__ z,
                                           int64_t ldz, float c, const RowInfo* __restrict__ info,
                                           int64_t rows, int64_t vocab, __half* __restrict__ g,
                                           int64_t ldg) {
  const int64_t r = (blockIdx.x * int64_t(blockDim.x) + threadIdx.x) >> 5;
  if (r >= rows) return;
  const RowInfo ri = info[r];
  for (int e = threadIdx.x & 31; e < top; e += 32) {
    const int64_t i = index[r * ldt + e];
    if (i < 0 || i >= vocab) continue;
    float sum = 0.0f;
    for (int k = 0; k < top; ++k)
      if (index[r * ldt + k] == i) sum += q[r * top + k];
    g[r * ldg + i] = __float2half_rn(grad_value(z[r * ldz + i], c, ri.lse2, ri.gs, sum));
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
bool misaligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1024;
constexpr int64_t kMaxLd = int64_t{1} << 36;
// Logits of a piece by default: 2 GiB of float32, 1 GiB of G.  Fewer, longer pieces cost less: a
// piece adds one pass of reads and writes over dW in float32.
constexpr int64_t kPieceLogits = int64_t{1} << 29;
// Without logits a token's scratch is its statistics: 1 GiB of them.
constexpr int64_t kPieceStats = int64_t{1} << 27;

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
    if ((h.dX || h.dW) && !h.dloss) return TG_ERR_INVALID_ARG;
  }
  if (misaligned(h.X, 2) || misaligned(h.W, 2) || misaligned(h.dX, 2) || misaligned(h.dW, 2) ||
      misaligned(h.index, 8) || misaligned(h.teacher, h.teacher_f32 ? 4 : 2) ||
      misaligned(h.dloss, 4) || misaligned(h.loss, 4) || misaligned(h.lse, 4))
    return TG_ERR_MISALIGNED;
  return TG_OK;
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
  const bool store = grad || h.top > 0;  // the logits are needed again
  const int64_t ldz = round_up(h.V, 32), ldg = round_up(h.V, 64);
  const int64_t tiles = 2 * cdiv(h.V, 128);  // statistics of a row, at most
  const int64_t per_row = store ? ldz : tiles, budget = store ? kPieceLogits : kPieceStats;
  int64_t piece = h.o.piece_rows ? std::min(h.o.piece_rows, h.T) : h.T;
  if (!h.o.piece_rows && h.T > budget / per_row) {
    const int64_t most = std::max<int64_t>(budget / per_row / 256 * 256, 256);
    piece = std::min(h.T, round_up(cdiv(h.T, cdiv(h.T, most)), 256));
  }
  const bool sum_w = h.dW && piece < h.T;  // dW is summed over pieces in float32

  Layout lay;
  // rows that TMA cannot read in place are copied once for all pieces and products
  const bool copy_x = misaligned(h.X, 16) || h.ldx % 8 != 0;
  const bool copy_w = misaligned(h.W, 16) || h.ldw % 8 != 0;
  const int64_t ldxp = round_up(h.D, 64), ldwp = round_up(w_cols, 64), ldw32 = round_up(w_cols, 32);
  const int64_t at_z = lay.add(store ? piece * ldz * 4 : 0);
  const int64_t at_stats = lay.add(tiles * piece * int64_t(sizeof(float2)));
  const int64_t at_picked = lay.add(store ? 0 : piece * 4);
  const int64_t at_info = lay.add(piece * int64_t(sizeof(RowInfo)));
  const int64_t at_small = lay.add(2 * 4);
  const int64_t at_g = lay.add(grad ? piece * ldg * 2 : 0);
  const int64_t at_q = lay.add(grad && h.top ? piece * h.top * 4 : 0);
  const int64_t at_x = lay.add(copy_x ? h.T * ldxp * 2 : 0);
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
  if (grad) {
    if ((e = cudaMemsetAsync(wmax, 0, 4, stream)) != cudaSuccess)
      return done(tg::record_cuda_error(e));
    tg_head_weight_kernel<<<static_cast<unsigned>(std::min<int64_t>(cdiv(h.T, 128), 4 * sms)), 128, 0,
                            stream>>>(h.dloss, h.index, h.ldt, h.top, h.ignore, h.T, wmax);
    if ((e = cudaGetLastError()) != cudaSuccess) return done(tg::record_cuda_error(e));
  }

  tg_options opt;
  std::memset(&opt, 0, sizeof(opt));
  opt.timeout_ms = h.o.timeout_ms;
  opt.debug_flags = h.o.debug_flags;
  const float c = h.scale * kLog2e;
  for (int64_t t0 = 0; t0 < h.T; t0 += piece) {
    const int64_t n = std::min(piece, h.T - t0);
    const uint16_t* x = X + t0 * ldx;
    const int64_t* index = h.index + t0 * (h.top ? h.ldt : 1);
    const void* teacher = h.teacher == nullptr ? nullptr
                                               : static_cast<const uint8_t*>(h.teacher) +
                                                     t0 * h.ldt * (h.teacher_f32 ? 4 : 2);
    const float* dloss = grad ? h.dloss + t0 : nullptr;
    float* loss = h.loss ? h.loss + t0 : nullptr;
    int block_n = 0;
    tg::LogitsExtra lx;
    lx.z = z;
    lx.ldz = ldz;
    lx.stats = stats;
    lx.stat_c = c;
    lx.target = store ? nullptr : reinterpret_cast<const long long*>(index);
    lx.picked = picked;
    lx.block_n = &block_n;
    tg::GemmExtra ex;
    std::memset(&ex, 0, sizeof(ex));
    ex.logits = &lx;
    st = tg::gemm_extra(0, by_vocab, x, W, nullptr, n, h.V, h.D, ldx, ldw, h.V, ex, &opt, stream);
    if (st != TG_OK) return done(st);
    tg_head_rows_kernel<<<static_cast<unsigned>(cdiv(n, 32)), dim3(32, kRowLanes), 0, stream>>>(
        stats, static_cast<int>(2 * cdiv(h.V, block_n)), n, z, ldz, picked, h.scale, h.V,
        h.top ? nullptr : index, h.ignore, dloss, wmax, loss, h.lse ? h.lse + t0 : nullptr, info,
        alpha);
    if (h.top)
      tg_head_distil_rows_kernel<<<static_cast<unsigned>(cdiv(n, 4)), 128, 0, stream>>>(
          index, teacher, h.teacher_f32, h.ldt, h.top, n, z, ldz, h.scale, h.V, dloss, wmax, loss,
          info, q);
    if ((e = cudaGetLastError()) != cudaSuccess) return done(tg::record_cuda_error(e));
    if (!grad) continue;
    tg_head_grad_kernel<<<dim3(static_cast<unsigned>(cdiv(h.V, 2048)),
                               static_cast<unsigned>(std::min<int64_t>(n, 65535))),
                          256, 0, stream>>>(z, ldz, c, info, n, h.V, g, ldg);
    if (h.top)
      tg_head_distil_grad_kernel<<<static_cast<unsigned>(cdiv(n, 4)), 128, 0, stream>>>(
          index, h.ldt, h.top, q, z, ldz, c, info, n, h.V, reinterpret_cast<__half*>(g), ldg);
    if ((e = cudaGetLastError()) != cudaSuccess) return done(tg::record_cuda_error(e));
    if (h.dX) {  // G (n x V) times W (V x D, or stored D x V)
      std::memset(&ex, 0, sizeof(ex));
      ex.alpha = alpha;
      st = tg::gemm_extra(0, !by_vocab, g, W, static_cast<uint16_t*>(h.dX) + t0 * h.lddx, n, h.D,
                          h.V, ldg, ldw, h.lddx, ex, &opt, stream);
      if (st != TG_OK) return done(st);
    }
    if (h.dW) {  // G^T X (V x D), or X^T G (D x V)
      std::memset(&ex, 0, sizeof(ex));
      ex.alpha = alpha;
      if (sum_w) {  // the first piece writes the sums, the last takes them into its epilogue
        ex.ld32 = ldw32;
        if (t0 + piece < h.T) {
          ex.out32 = w32;
          ex.add = t0 > 0;
        } else {
          ex.addend = w32;
        }
      }
      st = by_vocab ? tg::gemm_extra(1, 0, g, x, h.dW, h.V, h.D, n, ldg, ldx, h.lddw, ex, &opt, stream)
                    : tg::gemm_extra(1, 0, x, g, h.dW, h.D, h.V, n, ldx, ldg, h.lddw, ex, &opt, stream);
      if (st != TG_OK) return done(st);
    }
  }
  return done(TG_OK);
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

}  // extern "C"
