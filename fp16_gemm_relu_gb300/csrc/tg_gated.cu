// tg_gated.cu — the gated feed-forward product and its backward pass.
//
//   gate = X Wg,  up = X Wu  (M x N, float32),   H = act(gate) * up
//   dG = dH * up * act'(gate),  dU = dH * act(gate)
//   dX = dG Wg^T + dU Wu^T,  dWg = X^T dG,  dWu = X^T dU
//
// Forward is one kernel (tg_gated_kernel.cuh), with K splits and a reduction where few tokens leave SMs idle.
// Backward is a pass over the M x N matrices that leaves [dG | dU] in scratch, and the products: both weights'
// gradients as one launch with two outputs, dX as one sum over both gradients with two right operands, and up
// to 256 tokens all three as one launch (tg_gemm_kernel.cuh: kModeTwo, kModeDual, tg_gemm_beside_kernel).  At 8192 x
// 4096 x 14336 the pass takes 183 us, the products 2100 (1.83 PFLOP/s); with dX as two products through float32
// and the weights' one by one the step took 2749, so 2290.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "tg_gemm_relu.h"
#include "tg_internal.h"

namespace {

using tg::gated_activation;
using tg::gated_slope;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
bool misaligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

constexpr int64_t kMaxSize = int64_t{1} << 29;  // twice N is a TMA coordinate
constexpr int64_t kMaxElements = int64_t{1} << 44;
constexpr int64_t kMaxLd = int64_t{1} << 36;
// A TMA box of many rows of a matrix of fewer than eight (the rows of a swizzle atom) takes longer at some
// addresses, so operands of the gradients' products lie in scratch of that many rows, the others zero.
constexpr int64_t kLeastRows = 8;
// Elements of each weight from which it counts how dX and dW share the SMs.
constexpr int64_t kBesideWork = int64_t{4} << 20;
constexpr int64_t kBesideTokens = 256;
// Elements of each weight and token from which gradients are taken without copies of the weights.
constexpr int64_t kStraightWork = int64_t{2} << 20;
// Terms that one accumulator adds up.  The tensor core cuts off where it adds, so a long sum shrinks: terms of one
// sign by 4.0e-4 of themselves over 65536 terms, nearly all that its rounding to fp16 may take (4.9e-4), and by 2.0e-4 at
// this length; terms of either sign lose several times less.  Longer sums are taken in splits that are added in
// float32.
constexpr int64_t kSumLength = 32768;

// H (and gate, up) from the K splits' float32 partial sums, added in order; four columns a thread and the
// loads of kAhead splits in flight.  A split's rows hold the gates and, nw columns further, the ups.
constexpr int kAhead = 4;
__device__ __forceinline__ void store4(__half* row, int64_t col, int64_t n, const float (&v)[4]) {
  __half* d = row + col;
  if (col + 4 <= n && (reinterpret_cast<uintptr_t>(d) & 7u) == 0) {
    const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(d) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < n) d[i] = __float2half_rn(v[i]);
  }
}
__global__ void __launch_bounds__(128)
    tg_gated_reduce_kernel(const float* ws, int64_t nw, int64_t stride, int splits, int act,
                           __half* h, int64_t ldh, __half* gate, int64_t ldg, __half* up, int64_t ldu,
                           int64_t M, int64_t N) {
  const int64_t c = (blockIdx.x * int64_t(blockDim.x) + threadIdx.x) << 2;
  if (c >= N) return;
  tg::chain_wait();
  for (int64_t r = blockIdx.y; r < M; r += gridDim.y) {
    const float* w = ws + r * 2 * nw + c;
    float g[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f}, v[4];
    for (int s0 = 0; s0 < splits; s0 += kAhead) {
      float4 a[kAhead], b[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (s0 + i >= splits) break;
        a[i] = __ldcg(reinterpret_cast<const float4*>(w + (s0 + i) * stride));
        b[i] = __ldcg(reinterpret_cast<const float4*>(w + (s0 + i) * stride + nw));
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (s0 + i >= splits) break;
        g[0] += a[i].x, g[1] += a[i].y, g[2] += a[i].z, g[3] += a[i].w;
        u[0] += b[i].x, u[1] += b[i].y, u[2] += b[i].z, u[3] += b[i].w;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = gated_activation(g[i], act) * u[i];
    store4(h + r * ldh, c, N, v);
    if (gate) store4(gate + r * ldg, c, N, g);
    if (up) store4(up + r * ldu, c, N, u);
  }
}

// Eight packed values of a row from column `col` on, zeros past n; 16 bytes at once where the row allows it.
__device__ __forceinline__ uint4 load8(const __half* row, int64_t col, int64_t n) {
  const __half* s = row + col;
  if (col + 8 <= n && (reinterpret_cast<uintptr_t>(s) & 15u) == 0)
    return __ldcs(reinterpret_cast<const uint4*>(s));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col + i < n) w[i >> 1] |= static_cast<uint32_t>(__half_as_ushort(s[i])) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float2 half2_of(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// dG and dU (fp16, rows x np each, rows of ld; zeros from column N and row M on), eight columns of kGradRows
// rows a thread, whose loads go out together.  Bound by HBM: 8192 x 14336 183 us, 6.4 TB/s (four rows a thread, at half
// the occupancy, 253).
constexpr int kGradRows = 2;
template <int ACT>
__global__ void __launch_bounds__(256, 4)
    tg_gated_grad_kernel(const __half* __restrict__ dh, int64_t lddh, const __half* __restrict__ gate,
                         int64_t ldg, const __half* __restrict__ up, int64_t ldu, __half* out, int64_t ld,
                         int64_t np, int64_t M, int64_t N, int64_t rows) {
  tg::chain_release();
  const int64_t c = (blockIdx.x * int64_t(blockDim.x) + threadIdx.x) << 3;
  if (c >= np) return;
  for (int64_t r0 = int64_t(blockIdx.y) * kGradRows; r0 < rows; r0 += int64_t(gridDim.y) * kGradRows) {
    uint4 d[kGradRows], g[kGradRows], u[kGradRows];
#pragma unroll
    for (int i = 0; i < kGradRows; ++i) {
      d[i] = g[i] = u[i] = make_uint4(0, 0, 0, 0);  // (a gate of 0 has a finite slope)
      if (r0 + i >= M) continue;
      d[i] = load8(dh + (r0 + i) * lddh, c, N);
      g[i] = load8(gate + (r0 + i) * ldg, c, N);
      u[i] = load8(up + (r0 + i) * ldu, c, N);
    }
#pragma unroll
    for (int i = 0; i < kGradRows; ++i) {
      if (r0 + i >= rows) break;
      const uint32_t dw[4] = {d[i].x, d[i].y, d[i].z, d[i].w}, gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w},
                     uw[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      uint32_t a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 dv = half2_of(dw[j]), gv = half2_of(gw[j]), uv = half2_of(uw[j]);
        a[j] = pack2(dv.x * (uv.x * gated_slope(gv.x, ACT)), dv.y * (uv.y * gated_slope(gv.y, ACT)));
        b[j] = pack2(dv.x * gated_activation(gv.x, ACT), dv.y * gated_activation(gv.y, ACT));
      }
      *reinterpret_cast<uint4*>(out + (r0 + i) * ld + c) = make_uint4(a[0], a[1], a[2], a[3]);
      *reinterpret_cast<uint4*>(out + (r0 + i) * ld + np + c) = make_uint4(b[0], b[1], b[2], b[3]);
    }
  }
}

cudaError_t launch_grad(int act, const __half* dh, int64_t lddh, const __half* gate, int64_t ldg,
                        const __half* up, int64_t ldu, __half* out, int64_t ld, int64_t np, int64_t M,
                        int64_t N, int64_t rows, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(cdiv(np, 2048)),
                  static_cast<unsigned>(std::min<int64_t>(cdiv(rows, kGradRows), 65535)));
  auto go = [&](auto kern) {
    kern<<<grid, 256, 0, stream>>>(dh, lddh, gate, ldg, up, ldu, out, ld, np, M, N, rows);
    return cudaGetLastError();
  };
  switch (act) {
    case TG_ACT_SILU: return go(tg_gated_grad_kernel<TG_ACT_SILU>);
    case TG_ACT_RELU: return go(tg_gated_grad_kernel<TG_ACT_RELU>);
    case TG_ACT_GELU: return go(tg_gated_grad_kernel<TG_ACT_GELU>);
    case TG_ACT_GELU_TANH: return go(tg_gated_grad_kernel<TG_ACT_GELU_TANH>);
    default: return go(tg_gated_grad_kernel<TG_ACT_NONE>);
  }
}

struct Gated {
  const void *X, *Wg, *Wu;
  int act, trans;
  int64_t M, N, K, ldx, ldwg, ldwu;
};

bool bad_ld(int64_t ld, int64_t n) { return ld < n || ld > kMaxLd; }

tg_status check(const Gated& a) {
  if (a.M < 0 || a.N < 1 || a.K < 1 || a.M > kMaxSize || a.N > kMaxSize || a.K > kMaxSize)
    return TG_ERR_INVALID_ARG;
  // sizes whose products leave 64 bits could only come with pointers to nothing
  if (a.M > kMaxElements / a.N || a.M > kMaxElements / a.K || a.N > kMaxElements / a.K)
    return TG_ERR_INVALID_ARG;
  if (a.act < TG_ACT_NONE || a.act > TG_ACT_SILU || (a.trans != 0 && a.trans != 1))
    return TG_ERR_INVALID_ARG;
  const int64_t row = a.trans ? a.K : a.N;
  if (bad_ld(a.ldx, a.K) || bad_ld(a.ldwg, row) || bad_ld(a.ldwu, row)) return TG_ERR_INVALID_ARG;
  if (a.M > 0 && (!a.X || !a.Wg || !a.Wu)) return TG_ERR_INVALID_ARG;
  if (misaligned(a.X, 2) || misaligned(a.Wg, 2) || misaligned(a.Wu, 2)) return TG_ERR_MISALIGNED;
  return TG_OK;
}

// Parts of one scratch block, each 256-byte aligned.
struct Layout {
  int64_t bytes = 0;
  int64_t add(int64_t n) {
    const int64_t at = bytes;
    bytes += round_up(n, 256);
    return at;
  }
};

bool tma_cannot(const void* p, int64_t ld) { return misaligned(p, 16) || ld % 8 != 0; }

// X and the weights as TMA reads them: in place, or as copies with rows of whole 128-byte lines where
// the caller's are not 16-byte aligned with leading dimensions that are multiples of 8.
struct Operands {
  const void *x, *wg, *wu;
  int64_t ldx, ldwg, ldwu;
  int64_t at[3];  // of the copies in scratch, or -1
  int64_t zeros;  // rows of zeros behind a copy of X

  // Of what is read (x, both weights); X of fewer than least_rows rows is copied too, with zeros behind it.
  void plan(const Gated& a, bool need_x, bool need_w, int64_t least_rows, Layout* lay) {
    zeros = std::max<int64_t>(least_rows - a.M, 0);
    auto one = [&](const void* p, int64_t ld, int64_t rows, int64_t cols, bool copy = false) -> int64_t {
      return copy || tma_cannot(p, ld) ? lay->add(rows * round_up(cols, 64) * 2) : -1;
    };
    const int64_t w_rows = a.trans ? a.N : a.K, w_cols = a.trans ? a.K : a.N;
    at[0] = need_x ? one(a.X, a.ldx, a.M + zeros, a.K, zeros > 0) : -1;
    at[1] = need_w ? one(a.Wg, a.ldwg, w_rows, w_cols) : -1;
    at[2] = need_w ? one(a.Wu, a.ldwu, w_rows, w_cols) : -1;
  }
  // The copies, in one launch; whether there are any.
  cudaError_t copy(const Gated& a, uint8_t* mem, int sms, bool chained, cudaStream_t stream, bool* any) {
    tg::PackJob jobs[3];
    int n = 0;
    auto one = [&](int i, const void* p, int64_t ld, int64_t rows, int64_t cols, const void** out,
                   int64_t* ldo, int64_t more = 0) {
      *out = p;
      *ldo = ld;
      if (at[i] < 0) return;
      *out = mem + at[i];
      *ldo = round_up(cols, 64);
      jobs[n++] = tg::PackJob{p, mem + at[i], ld, *ldo, rows, cols, more};
    };
    const int64_t w_rows = a.trans ? a.N : a.K, w_cols = a.trans ? a.K : a.N;
    one(0, a.X, a.ldx, a.M, a.K, &x, &ldx, zeros);
    one(1, a.Wg, a.ldwg, w_rows, w_cols, &wg, &ldwg);
    one(2, a.Wu, a.ldwu, w_rows, w_cols, &wu, &ldwu);
    *any = n > 0;
    return tg::launch_pack_jobs(jobs, n, sms, chained, stream);
  }
};

// Up to four tokens over weights that would be copied for TMA: read where they are (1 x 4096 x 14333: K x N 48 us,
// with the copies 133; N x K, 4095 x 14336, 51 and 135; two tokens 63 and 57, four 77 and 88; eight would be about as
// long as the copies).  Weights that TMA reads are faster through it (43).
bool straight(const Gated& a) { return a.M <= 4 && (tma_cannot(a.Wg, a.ldwg) || tma_cannot(a.Wu, a.ldwu)); }

// Whether TMA can store whole rows of n fp16 columns.
bool whole_rows(const void* p, int64_t ld, int64_t n) {
  return !misaligned(p, 16) && ld % 8 == 0 && n % 8 == 0;
}

// The plan of one row of tiles, M <= 128: bound by the weights' 4 K N bytes from memory.  A row of tiles reads
// them at 6.6 TB/s where its units fill whole waves of blocks, and a third slower at worst where they do not
// (the blocks that are left share the bandwidth); tiles of 128 columns read K x N weights 128 bytes of a
// row at a time, which costs 12%; splits cost a second kernel and their float32 sums through L2.  Measured
// (us) against the alternatives: 1 x 8192 x 28672, K x N: two splits of 256 columns 149, one 155, 128 columns 165, a
// pair's tiles 242; N x K: 128 columns 146, 256 in two splits 149; 16 x 8192 x 22016: four splits 122, one 137;
// 1 x 4096 x 14336: one split of 256 columns 44, four 45, 128 columns 51.  One block alone waits for its stages: a
// k-block takes it 0.40 us at 256 columns and 0.27 at 128, so narrow weights are split by that: 64 x 8192 x 1000 in
// 16 splits 19, whole 70; 1 x 28672 x 512 in 16 of 128 columns 22, whole 127; 1 x 4096 x 4096 in four 20, whole 31.
tg::TilePlan few_rows_plan(const Gated& a, int sms) {
  tg::TilePlan best;
  std::memset(&best, 0, sizeof(best));
  best.num_kb = static_cast<int>(cdiv(a.K, tg::kBK));
  best.units_cap = sms;
  const double bytes = 4.0 * double(a.K) * double(a.N);
  const int least = static_cast<int>(cdiv(a.K, kSumLength));
  double best_t = 0.0;
  for (int bn = 256; bn >= 128; bn -= 128) {
    const int64_t tiles = cdiv(a.N, bn / 2);
    for (int s = least; s <= std::max(least, 32); ++s) {
      const int kbps = static_cast<int>(cdiv(best.num_kb, s));
      if (cdiv(best.num_kb, kbps) != s || (s > least && kbps < 4)) continue;
      const int64_t units = tiles * s;
      const double full = double(units) / double(cdiv(units, sms) * sms);
      double t = bytes / 6.6e12 / (0.65 + 0.35 * full);
      if (bn == 128 && !a.trans) t *= 1.12;
      t = std::max(t, double(cdiv(units, sms)) * kbps * (bn == 128 ? 0.27e-6 : 0.40e-6));
      if (s > 1) t += 4e-6 + 16.0 * s * double(a.M) * double(a.N) / 1e13;
      if (best.block_n && t >= best_t) continue;
      best_t = t;
      best.block_n = bn;
      best.splits = s;
      best.kb_per_split = kbps;
    }
  }
  return best;
}

int timeout_of(const tg_options* opt) { return opt && opt->timeout_ms > 0 ? opt->timeout_ms : 2000; }

// What a launch of the gradients' products has in common.
void common_params(tg::GemmParams* p, const tg_options* opt, unsigned* err) {
  p->debug_flags = opt ? opt->debug_flags : 0;
  p->timeout_ns = 1000000ull * static_cast<unsigned long long>(timeout_of(opt));
  p->err = err;
}

// dWg and dWu in one launch: X^T [dG | dU] (trans 0; the second output's tiles follow the first's along N)
// or [dG | dU]^T X (trans 1; along M), g holding dU np columns after dG.  TG_ERR_NO_WORKSPACE: the planner
// splits the sum, or an option asks for what this launch has not; nothing is launched.
tg_status weight_grads(const Gated& a, const Operands& ops, const __half* g, int64_t np, void* dWg,
                       int64_t lddwg, void* dWu, int64_t lddwu, const tg_options* opt, unsigned* err,
                       bool beside, int sms, cudaStream_t stream, tg::GemmLaunch* out, int* block_n) {
  const int64_t rows = a.trans ? a.N : a.K, cols = a.trans ? a.K : a.N;  // of each output
  tg::TilePlan plan;
  tg_options o;
  std::memset(&o, 0, sizeof(o));
  if (opt) o = *opt;
  // Few tokens: a tile is all epilogue, which one CTA with 16 epilogue warps does faster than a pair with eight
  // each (4096 x 14336 from 64 tokens 49 against 65 us, 54 in tiles of 128 columns; from 256 tokens 86 against 79).
  if ((a.M <= 128 || beside) && !o.pair) {
    o.pair = -1;
    if (!o.block_n && (beside || cdiv(rows, 128) * cdiv(cols, 256) >= sms / 2)) o.block_n = 256;
  }
  tg_status st = tg::plan_tiles(a.trans ? 2 * rows : rows, a.trans ? cols : 2 * cols, a.M, kSumLength, true,
                                &o, &plan);
  if (st != TG_OK) return st;
  if (plan.splits > 1) return TG_ERR_NO_WORKSPACE;
  const int bm = plan.pair ? 256 : 128, bn = plan.block_n;
  const int64_t tm = cdiv(rows, bm), tn = cdiv(cols, bn);
  if (2 * tm * tn >= (int64_t{1} << 31)) return TG_ERR_NO_WORKSPACE;
  tg::GemmLaunch& l = *out;
  std::memset(&l, 0, sizeof(l));
  tg::GemmParams& p = l.p;
  p.tiles_m = static_cast<int>(a.trans ? 2 * tm : tm);
  p.tiles_n = static_cast<int>(a.trans ? tn : 2 * tn);
  p.num_kb = p.kb_per_split = plan.num_kb;
  p.splits = 1;
  p.units = p.tiles_m * p.tiles_n;
  p.panel_m = std::min(opt && opt->panel_m ? opt->panel_m : 8, p.tiles_m);
  p.a_mn = 1;
  common_params(&p, opt, err);
  p.c = static_cast<__half*>(dWg), p.ldc = lddwg;
  p.M = static_cast<int>(rows), p.N = static_cast<int>(cols);
  const bool tma = whole_rows(dWg, lddwg, cols) && whole_rows(dWu, lddwu, cols);
  p.n_tma = tma ? p.N : 0;
  l.two.m_first = a.trans ? static_cast<int>(tm) : INT32_MAX;
  l.two.n_first = a.trans ? INT32_MAX : static_cast<int>(tn);
  l.two.off = static_cast<int>(np);
  l.two.c = static_cast<__half*>(dWu), l.two.ldc = lddwu;
  l.grid = static_cast<int>(std::min<int64_t>(p.units, plan.units_cap)) * (plan.pair ? 2 : 1);
  l.chained = true;
  l.stream = stream;
  const int kbox = plan.pair ? 128 : 64;
  bool ok;
  const int64_t tokens = std::max(a.M, kLeastRows);  // zeros from a.M on
  if (a.trans)
    ok = tg::half_map(&l.a, g, 2 * np, tokens, 2 * np, 64, kbox) &&
         tg::half_map(&l.b, ops.x, a.K, tokens, ops.ldx, 64, kbox);
  else
    ok = tg::half_map(&l.a, ops.x, a.K, tokens, ops.ldx, 64, kbox) &&
         tg::half_map(&l.b, g, 2 * np, tokens, 2 * np, 64, kbox);
  if (tma)
    ok = ok && tg::half_map(&l.out, dWg, cols, rows, lddwg, 64, 32) &&
         tg::half_map(&l.out2, dWu, cols, rows, lddwu, 64, 32);
  *block_n = plan.pair ? 0 : bn;
  return ok ? TG_OK : tg::record_cuda_error(cudaErrorInvalidValue);
}

// Few tokens: dX, which reads the weights, beside dWg and dWu, which are as many bytes to write, in one launch
// where each has its share of the SMs: dX up to half of them, as many as its tiles of `width` columns in some number
// of splits make, one unit a block.  The splits, or 0 where the calls go one after the other (tiles of large
// weights that make less than three eighths).  64 tokens of 4096 x 14336 90 against 104 us one after the other (with two fifths
// of the SMs 103), 37 of 1112 x 4448 24 and 30, 128 of 4096 x 14336 102 and 118, 256 of it 150 and 167; 64 of 8192 x 28672
// 322 and 314, 512 of 4096 x 14336 231 and 201.  Small weights gain by the launch that is saved, 16 of 256 x 512 17 and 21,
// with no more splits than the sum's length pays for.
int beside_splits(const Gated& a, int64_t ld, int64_t width, int sms) {
  const int64_t tiles = cdiv(a.K, width) * cdiv(a.M, tg::kBM), least = cdiv(ld, kSumLength);
  const bool small = a.K * a.N < kBesideWork;
  const int64_t splits = std::min({sms / 2 / tiles, ld / 128, small ? std::max<int64_t>(8, ld / 1024) : ld});
  if (a.M > kBesideTokens || splits < std::max<int64_t>(least, 1) || (!small && tiles * splits * 8 < 3 * sms))
    return 0;
  const int64_t kbps = round_up(cdiv(ld / tg::kBK, splits), 2);  // (a stage never has both weights' k-blocks)
  return static_cast<int>(cdiv(ld / tg::kBK, kbps));
}

// dX's launch for that, its partial sums in ws.
bool beside_input(const Gated& a, const Operands& ops, const __half* g, int64_t ld, int64_t width, int splits,
                  float* ws, int64_t ldw, const tg_options* opt, unsigned* err, tg::GemmLaunch* l) {
  std::memset(l, 0, sizeof(*l));
  tg::GemmParams& p = l->p;
  p.tiles_m = static_cast<int>(cdiv(a.M, tg::kBM));
  p.tiles_n = static_cast<int>(cdiv(a.K, width));
  p.num_kb = static_cast<int>(ld / tg::kBK);
  p.kb_per_split = static_cast<int>(round_up(cdiv(p.num_kb, splits), 2));
  p.splits = splits;
  p.units = p.tiles_m * p.tiles_n * splits;
  p.panel_m = p.tiles_m;
  p.b_k = !a.trans;
  common_params(&p, opt, err);
  p.M = static_cast<int>(a.M), p.N = static_cast<int>(a.K);
  p.kb_switch = p.num_kb / 2;
  l->grid = p.units;
  auto right = [&](CUtensorMap* m, const void* w, int64_t ldwt) {
    return a.trans ? tg::half_map(m, w, a.K, a.N, ldwt, 64, 64)
                   : tg::half_map(m, w, a.N, a.K, ldwt, 64, static_cast<int>(width));
  };
  return tg::half_map(&l->a, g, ld, std::max(a.M, kLeastRows), ld, 64, tg::kBM) && right(&l->b, ops.wg, ops.ldwg) &&
         right(&l->b2, ops.wu, ops.ldwu) && tg::partial_map(&l->out, ws, a.K, a.M, splits, ldw);
}

}  // namespace

extern "C" {

tg_status tg_gated_f16(const void* X, const void* Wg, const void* Wu, void* H, void* gate, void* up,
                       int activation, int trans_w, int64_t M, int64_t N, int64_t K, int64_t ldx,
                       int64_t ldwg, int64_t ldwu, int64_t ldh, int64_t ldgate, int64_t ldup,
                       const tg_options* opt, tg_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const Gated a{X, Wg, Wu, activation, trans_w, M, N, K, ldx, ldwg, ldwu};
  tg_status st = check(a);
  if (st != TG_OK) return st;
  if (bad_ld(ldh, N) || (gate && bad_ld(ldgate, N)) || (up && bad_ld(ldup, N)))
    return TG_ERR_INVALID_ARG;
  if (M == 0) return TG_OK;
  if (!H) return TG_ERR_INVALID_ARG;
  if (misaligned(H, 2) || misaligned(gate, 2) || misaligned(up, 2)) return TG_ERR_MISALIGNED;
  int sms = 0;
  unsigned* err = nullptr;
  if ((st = tg::device_info(&sms, &err)) != TG_OK) return st;
  tg::TilePlan plan;
  const bool choose = !opt || (!opt->block_n && !opt->split_k && !opt->pair && !opt->max_ctas);
  // (a row of tiles of BN columns covers BN / 2 of each weight; the call refuses what no plan has)
  if ((st = tg::plan_tiles(M, 2 * round_up(N, 128), K, kSumLength, true, opt, &plan)) != TG_OK) return st;
  if (M <= 128 && choose) {
    plan = few_rows_plan(a, sms);
  } else if (choose && !plan.pair && plan.block_n == 128 && cdiv(M, 256) * cdiv(N, 128) >= sms / 2) {
    // a last wave that narrow tiles fill better is no gain where they read X four times as often: from 136 to 1024
    // tokens of six weights (2048 x 8192 to 8192 x 28672) they took 1.08 to 1.7 times as long as pairs (256 x 4096 x
    // 14336 61 us, on pairs 57, 320 of it 95 and 75, 160 x 4096 x 11008 60 and 54, 640 x 2048 x 8192 52 and 39); below a
    // wave of pairs the planner stands
    tg_options o;
    std::memset(&o, 0, sizeof(o));
    if (opt) o = *opt;
    o.pair = 1;
    if ((st = tg::plan_tiles(M, 2 * round_up(N, 128), K, kSumLength, true, &o, &plan)) != TG_OK) return st;
  }
  const int64_t nw = round_up(N, 32), stride = M * 2 * nw;
  auto launch_reduce = [&](const float* sums, int splits) {
    const dim3 grid(static_cast<unsigned>(cdiv(N, 512)), static_cast<unsigned>(std::min<int64_t>(M, 65535)));
    return tg::launch_chained(tg_gated_reduce_kernel, true, grid, 128, 0, stream, sums, nw, stride, splits,
                              activation, static_cast<__half*>(H), ldh, static_cast<__half*>(gate), ldgate,
                              static_cast<__half*>(up), ldup, M, N);
  };
  if (choose && straight(a)) {
    tg::GatedRows r;
    std::memset(&r, 0, sizeof(r));
    r.x = static_cast<const __half*>(X), r.ldx = ldx;
    r.wg = static_cast<const __half*>(Wg), r.ldwg = ldwg;
    r.wu = static_cast<const __half*>(Wu), r.ldwu = ldwu;
    r.h = static_cast<__half*>(H), r.ldh = ldh;
    r.gate = static_cast<__half*>(gate), r.ldgate = ldgate;
    r.up = static_cast<__half*>(up), r.ldup = ldup;
    r.N = N, r.L = K, r.M = static_cast<int>(M), r.act = activation, r.nw = nw;
    const int splits = tg::plan_gated_rows(&r, trans_w, false, sms);
    if (splits > 1 && (st = tg::scratch_alloc(size_t(splits * stride) * 4, stream,
                                              reinterpret_cast<void**>(&r.ws))) != TG_OK)
      return st;
    cudaError_t e = tg::launch_gated_rows(r, trans_w, splits, stream);
    if (r.ws) {
      if (e == cudaSuccess) e = launch_reduce(r.ws, splits);
      const cudaError_t fe = cudaFreeAsync(r.ws, stream);
      if (e == cudaSuccess) e = fe;
    }
    return e == cudaSuccess ? TG_OK : tg::record_cuda_error(e);
  }
  Operands ops;
  Layout lay;
  ops.plan(a, true, true, 0, &lay);
  const bool f32 = plan.splits > 1;
  const int64_t at_ws = lay.add(f32 ? plan.splits * stride * 4 : 0);
  uint8_t* mem = nullptr;
  if (lay.bytes > 0 &&
      (st = tg::scratch_alloc(size_t(lay.bytes), stream, reinterpret_cast<void**>(&mem))) != TG_OK)
    return st;
  auto done = [&](tg_status s) {
    const cudaError_t fe = mem ? cudaFreeAsync(mem, stream) : cudaSuccess;
    return s == TG_OK && fe != cudaSuccess ? tg::record_cuda_error(fe) : s;
  };
  bool copied = false;
  cudaError_t e = ops.copy(a, mem, sms, false, stream, &copied);
  if (e != cudaSuccess) return done(tg::record_cuda_error(e));

  const int hn = plan.pair ? 128 : plan.block_n / 2, bm = plan.pair ? 256 : 128;
  tg::GatedLaunch l;
  std::memset(&l, 0, sizeof(l));
  tg::GemmParams& p = l.p.g;
  p.tiles_m = static_cast<int>(cdiv(M, bm));
  p.tiles_n = static_cast<int>(cdiv(N, hn));
  p.num_kb = plan.num_kb;
  p.kb_per_split = plan.kb_per_split;
  p.splits = plan.splits;
  const int64_t units = int64_t(p.tiles_m) * p.tiles_n * p.splits;
  if (units >= (int64_t{1} << 31)) return done(TG_ERR_INVALID_ARG);
  p.units = static_cast<int>(units);
  // Panels of 16 rows of tiles: the weights, the larger operand, are read half as often from memory as with the
  // GEMM's 8, and 4096 rows of X still stay in L2 (8192 x 4096 x 14336 in a power-capped loop 1186 against 1222 us;
  // 32 rows 1227).
  p.panel_m = std::min(opt && opt->panel_m ? opt->panel_m : 16, p.tiles_m);
  p.act = activation;
  p.b_k = trans_w;
  p.debug_flags = opt ? opt->debug_flags : 0;
  p.timeout_ns = 1000000ull * static_cast<unsigned long long>(timeout_of(opt));
  p.err = err;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  l.p.h = static_cast<__half*>(H), l.p.ldh = ldh;
  l.p.gate = static_cast<__half*>(gate), l.p.ldgate = ldgate;
  l.p.up = static_cast<__half*>(up), l.p.ldup = ldup;
  l.p.a_rows = static_cast<int>(M < 128 && !plan.pair ? round_up(M, 8) : 128);
  l.p.nw = static_cast<int>(nw);
  l.p.rotate = p.tiles_m == 1;
  l.p.tma = whole_rows(H, ldh, N) && (!gate || whole_rows(gate, ldgate, N)) && (!up || whole_rows(up, ldup, N));
  l.grid = static_cast<int>(std::min<int64_t>(units, plan.units_cap)) * (plan.pair ? 2 : 1);
  l.block_n = plan.pair ? 0 : plan.block_n;
  l.out_f32 = f32;
  l.chained = copied;
  l.stream = stream;
  bool ok = tg::half_map(&l.x, ops.x, K, M, ops.ldx, 64, l.p.a_rows);
  const int kbox = plan.pair ? 128 : 64;
  if (trans_w)
    ok = ok && tg::half_map(&l.g, ops.wg, K, N, ops.ldwg, 64, plan.pair ? 128 : hn) &&
         tg::half_map(&l.u, ops.wu, K, N, ops.ldwu, 64, plan.pair ? 128 : hn);
  else
    ok = ok && tg::half_map(&l.g, ops.wg, N, K, ops.ldwg, 64, kbox) &&
         tg::half_map(&l.u, ops.wu, N, K, ops.ldwu, 64, kbox);
  float* ws = reinterpret_cast<float*>(mem + at_ws);
  if (f32)
    ok = ok && tg::partial_map(&l.h, ws, 2 * nw, M, p.splits, 2 * nw);
  else if (l.p.tma)
    ok = ok && tg::half_map(&l.h, H, N, M, ldh, 64, 32) &&
         (!gate || tg::half_map(&l.gate, gate, N, M, ldgate, 64, 32)) &&
         (!up || tg::half_map(&l.up, up, N, M, ldup, 64, 32));
  if (!ok) return done(tg::record_cuda_error(cudaErrorInvalidValue));
  if ((e = tg::launch_gated(l)) != cudaSuccess) return done(tg::record_cuda_error(e));
  if (f32) {
    e = launch_reduce(ws, p.splits);
    if (e != cudaSuccess) return done(tg::record_cuda_error(e));
  }
  return done(TG_OK);
}

tg_status tg_gated_backward_f16(const void* dH, const void* X, const void* Wg, const void* Wu,
                                const void* gate, const void* up, void* dX, void* dWg, void* dWu,
                                int activation, int trans_w, int64_t M, int64_t N, int64_t K,
                                int64_t lddh, int64_t ldx, int64_t ldwg, int64_t ldwu, int64_t ldgate,
                                int64_t ldup, int64_t lddx, int64_t lddwg, int64_t lddwu,
                                const tg_options* opt, tg_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const Gated a{X, Wg, Wu, activation, trans_w, M, N, K, ldx, ldwg, ldwu};
  tg_status st = check(a);
  if (st != TG_OK) return st;
  const int64_t w_rows = trans_w ? N : K, w_cols = trans_w ? K : N;
  if (bad_ld(lddh, N) || bad_ld(ldgate, N) || bad_ld(ldup, N) || (dX && bad_ld(lddx, K)) ||
      (dWg && bad_ld(lddwg, w_cols)) || (dWu && bad_ld(lddwu, w_cols)))
    return TG_ERR_INVALID_ARG;
  if (M > 0 && (!dH || !gate || !up)) return TG_ERR_INVALID_ARG;
  if (misaligned(dH, 2) || misaligned(gate, 2) || misaligned(up, 2) || misaligned(dX, 2) ||
      misaligned(dWg, 2) || misaligned(dWu, 2))
    return TG_ERR_MISALIGNED;
  if (!dX && !dWg && !dWu) return TG_OK;
  cudaError_t e;
  if (M == 0) {  // the sum over no rows
    int sms = 0;
    unsigned* err = nullptr;
    if ((st = tg::device_info(&sms, &err)) != TG_OK) return st;
    for (int i = 0; i < 2; ++i) {
      void* d = i ? dWu : dWg;
      if (!d) continue;
      e = cudaMemset2DAsync(d, size_t(i ? lddwu : lddwg) * 2, 0, size_t(w_cols) * 2, size_t(w_rows), stream);
      if (e != cudaSuccess) return tg::record_cuda_error(e);
    }
    return TG_OK;
  }
  int sms = 0;
  unsigned* err = nullptr;
  if ((st = tg::device_info(&sms, &err)) != TG_OK) return st;
  const int64_t np = round_up(N, 128), ld = 2 * np;
  tg::TilePlan asked;  // options that no plan has are refused before anything is launched
  if (opt && (st = tg::plan_tiles(M, K, ld, kSumLength, true, opt, &asked)) != TG_OK) return st;
  Layout lay;
  Operands ops;
  const int64_t rows = std::max(M, kLeastRows);
  const int64_t at_g = lay.add(rows * ld * 2);
  const int64_t width = K <= 2048 ? 128 : 256;  // few tokens: dX's tiles
  const bool choose = !opt || (!opt->block_n && !opt->split_k && !opt->pair && !opt->max_ctas && !opt->panel_m);
  // Its gradients: one token of 4096 x 14333 114 us, with the copies 220, two 129, four 166 and 222; smaller weights
  // pay more for two more launches than their copies cost (four of 1023 x 4091 42 to 45 and 40, one 28 to 34 and 38).
  const bool direct = choose && straight(a) && K * N >= M * kStraightWork;
  const int beside = dX && dWg && dWu && choose && !direct ? beside_splits(a, ld, width, sms) : 0;
  tg::GatedRows r;
  std::memset(&r, 0, sizeof(r));
  r.N = K, r.L = N, r.M = static_cast<int>(std::min<int64_t>(M, 4));
  const int apart = direct && dX ? tg::plan_gated_rows(&r, !trans_w, true, sms) : 1;  // dX's sum
  const int64_t ldw = round_up(K, 32), at_ws = lay.add((apart > 1 ? apart : beside) * M * ldw * 4);
  if (!direct) ops.plan(a, dWg || dWu, dX, dWg || dWu ? kLeastRows : 0, &lay);
  uint8_t* mem = nullptr;
  if ((st = tg::scratch_alloc(size_t(lay.bytes), stream, reinterpret_cast<void**>(&mem))) != TG_OK)
    return st;
  auto done = [&](tg_status s) {
    const cudaError_t fe = cudaFreeAsync(mem, stream);
    return s == TG_OK && fe != cudaSuccess ? tg::record_cuda_error(fe) : s;
  };
  __half* g = reinterpret_cast<__half*>(mem + at_g);
  e = launch_grad(activation, static_cast<const __half*>(dH), lddh, static_cast<const __half*>(gate), ldgate,
                  static_cast<const __half*>(up), ldup, g, ld, np, M, N, direct ? M : rows, stream);
  if (e != cudaSuccess) return done(tg::record_cuda_error(e));
  if (direct) {
    const __half* x = static_cast<const __half*>(X);
    if (dWg || dWu) {
      tg::GatedOuter w;
      std::memset(&w, 0, sizeof(w));
      w.rows = trans_w ? g : x, w.rows2 = trans_w ? g + np : x, w.ld_rows = trans_w ? ld : ldx;
      w.cols = trans_w ? x : g, w.cols2 = trans_w ? x : g + np, w.ld_cols = trans_w ? ldx : ld;
      w.out = static_cast<__half*>(dWg), w.ld = lddwg;
      w.out2 = static_cast<__half*>(dWu), w.ld2 = lddwu;
      w.n_rows = w_rows, w.n_cols = w_cols, w.M = static_cast<int>(M);
      e = tg::launch_gated_outer(w, stream);
    }
    if (dX && e == cudaSuccess) {
      r.x = g, r.x2 = g + np, r.ldx = ld;
      r.wg = static_cast<const __half*>(Wg), r.ldwg = ldwg;
      r.wu = static_cast<const __half*>(Wu), r.ldwu = ldwu;
      r.h = static_cast<__half*>(dX), r.ldh = lddx;
      r.ws = apart > 1 ? reinterpret_cast<float*>(mem + at_ws) : nullptr, r.nw = ldw;
      e = tg::launch_gated_rows(r, !trans_w, apart, stream);
      if (r.ws && e == cudaSuccess) {
        tg::GemmParams p;
        std::memset(&p, 0, sizeof(p));
        p.M = static_cast<int>(M), p.N = static_cast<int>(K);
        e = tg::launch_splitk_reduce(r.ws, ldw, M * ldw, apart, dX, lddx, p, sms, stream);
      }
    }
    return done(e == cudaSuccess ? TG_OK : tg::record_cuda_error(e));
  }
  bool copied = false;
  if ((e = ops.copy(a, mem, sms, true, stream, &copied)) != cudaSuccess) return done(tg::record_cuda_error(e));
  tg::GemmExtra ex;
  std::memset(&ex, 0, sizeof(ex));
  ex.max_k = kSumLength;
  bool one_by_one = !dWg || !dWu;
  if (!one_by_one) {
    tg::GemmLaunch w;
    int block_n = 0;
    st = weight_grads(a, ops, g, np, dWg, lddwg, dWu, lddwu, opt, err, beside > 0, sms, stream, &w, &block_n);
    if (st != TG_OK && st != TG_ERR_NO_WORKSPACE) return done(st);
    one_by_one = st == TG_ERR_NO_WORKSPACE;
    if (beside && !one_by_one && block_n == 256) {
      tg::GemmLaunch x;
      float* ws = reinterpret_cast<float*>(mem + at_ws);
      if (!beside_input(a, ops, g, ld, width, beside, ws, ldw, opt, err, &x))
        return done(tg::record_cuda_error(cudaErrorInvalidValue));
      w.grid = std::min(w.p.units, sms - x.grid);
      if ((e = tg::launch_gemm_beside(x, static_cast<int>(width), w)) == cudaSuccess)
        e = tg::launch_splitk_reduce(ws, ldw, M * ldw, beside, dX, lddx, x.p, sms, stream);
      return done(e == cudaSuccess ? TG_OK : tg::record_cuda_error(e));
    }
    if (!one_by_one && (e = tg::launch_gemm_two(w, block_n)) != cudaSuccess)
      return done(tg::record_cuda_error(e));
  }
  for (int i = 0; i < 2 && one_by_one; ++i) {
    void* d = i ? dWu : dWg;
    if (!d) continue;
    const void* gi = g + i * np;
    const int64_t ldd = i ? lddwu : lddwg;
    st = trans_w ? tg::gemm_extra(1, 0, gi, ops.x, d, N, K, M, ld, ops.ldx, ldd, ex, opt, stream)
                 : tg::gemm_extra(1, 0, ops.x, gi, d, K, N, M, ops.ldx, ld, ldd, ex, opt, stream);
    if (st != TG_OK) return done(st);
  }
  if (dX) {  // one sum over dG's columns with Wg, then dU's with Wu
    ex.chained = true;
    ex.B2 = ops.wu;
    ex.ldb2 = ops.ldwu;
    ex.b_k = N;
    ex.a_rows = rows;
    // Few tokens: one row of tiles reads the weights once, at the memory's rate if its splits make one wave of
    // blocks over the SMs.
    tg_options o;
    std::memset(&o, 0, sizeof(o));
    if (opt) o = *opt;
    const int64_t splits = std::max(std::min({sms / cdiv(K, width), ld / 128, int64_t(32)}), cdiv(ld, kSumLength));
    if (M <= 128 && splits > 1 && !o.pair && !o.block_n && !o.split_k) {
      o.pair = -1;
      o.block_n = static_cast<int>(width);
      o.split_k = static_cast<int>(splits);
    }
    st = tg::gemm_extra(0, !trans_w, g, ops.wg, dX, M, K, ld, ld, ops.ldwg, lddx, ex, &o, stream);
    if (st != TG_OK) return done(st);
  }
  return done(TG_OK);
}

}  // extern "C"
