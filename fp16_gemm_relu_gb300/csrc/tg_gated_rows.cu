// tg_gated_rows.cu — the gated product of a few tokens over weights that TMA cannot read (rows that start
// off 16-byte boundaries), straight from memory.
//
//   H[m, n] = act(sum_l X[m, l] Wg(l, n)) * sum_l X[m, l] Wu(l, n)
//
// A copy for TMA costs 4 bytes read and written for each 2 that the product needs, and few tokens need every
// weight once: the float32 units, with a multiply for an element and token, keep up with the memory.
// Weights are loaded in aligned words of two, 128 contiguous bytes a warp, wherever a row starts: a row that
// starts inside a word is read from half a word before it, and its sums (or its tokens' elements) are those of one
// column further left.  32 loads of a thread are under way at once, around the L1.  A word at a row's end may hold
// an element beside it, which is masked; at the matrix's own ends words are put together from their halves, so
// nothing outside of it is read.  Sums are float32, added in an order that the sizes alone decide; the tokens'
// elements lie in shared memory in float32.
//
// The gradients of such a call likewise: dX = dG Wg^T + dU Wu^T by the same two kernels with each weight's own
// left operand (DUAL: the sums are added instead), and dWg and dWu, whose rows start anywhere as well, in
// aligned words from a kernel that only writes.
//
// One token of 4096 x 14333: K x N 48 us with the splits' sums joined (the kernel 44, 5.3 TB/s; in 2-byte loads 61, the
// splits as clusters' blocks 80, which left SMs idle), 4095 x 14336 stored N x K 51; with the copies 133 and 135;
// 8192 x 28671 160 and 146, 480.  Bound by the loads under way for one token, and by instructions from two on (two 63 and
// 57, with 160 bytes a thread spilled: 80 registers for three blocks an SM; four 77 and 88).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "tg_internal.h"

namespace tg {
namespace {

constexpr int kWarps = 8;

// A half's bits, or 0; without a branch, so that many are under way at once.
__device__ __forceinline__ uint32_t half_bits(const __half* p, bool in) {
  uint32_t v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .u16 h;\n\tsetp.ne.s32 p, %2, 0;\n\tmov.u16 h, 0;\n\t"
      "@p ld.global.nc.L1::no_allocate.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}"
      : "=r"(v)
      : "l"(p), "r"(static_cast<int>(in)));
  return v;
}
// Elements [at, at + 2) of a row of n, a word.  kInside: all are.  kRim: one or both may not be, and are zeros; the
// word loaded is one of the row's, but may reach into the gap or the row beside it, so this is for rows with one on
// either side.  kEdge: for all others, by halves; zeros if !in.
enum : int { kInside, kRim, kEdge };
template <int MODE>
__device__ __forceinline__ uint32_t word(const __half* row, int64_t at, int64_t n, bool in) {
  if constexpr (MODE == kEdge)
    return half_bits(row + at, in && at >= 0 && at < n) | half_bits(row + at + 1, in && at >= -1 && at + 1 < n) << 16;
  uint32_t w, keep = ~0u;
  if constexpr (MODE == kRim) {
    keep = at < 0 ? 0xffff0000u : at + 1 < n ? ~0u : at < n ? 0xffffu : 0u;
    at = min(at, n - 1 - ((n - 1 - at) & 1));
  }
  asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(w) : "l"(row + at));
  return w & keep;
}
__device__ __forceinline__ float2 floats(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// Element l < end of a token, or 0.
__device__ __forceinline__ float token_at(const __half* x, int m, const GatedRows& p, int64_t l, int64_t end) {
  return m < p.M && l >= 0 && l < end ? __half2float(__ldg(x + m * p.ldx + l)) : 0.0f;
}
template <int MODE>
using Mode = std::integral_constant<int, MODE>;
// Whether a row starts in the middle of a word.
__device__ __forceinline__ int odd(const __half* p) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 1) & 1;
}

// A block's sums for one element of H: that element, or where the grid's y has splits, their sums as
// tg_gated_reduce_kernel takes them (DUAL: as a product's).
template <bool DUAL>
__device__ __forceinline__ void finish(const GatedRows& p, int m, int64_t n, float g, float u) {
  const int64_t row = int64_t(blockIdx.y) * p.M + m;
  if constexpr (DUAL) {
    if (p.ws)
      p.ws[row * p.nw + n] = g + u;
    else
      p.h[m * p.ldh + n] = __float2half_rn(g + u);
    return;
  }
  if (p.ws) {
    p.ws[row * 2 * p.nw + n] = g;
    p.ws[(row * 2 + 1) * p.nw + n] = u;
    return;
  }
  p.h[m * p.ldh + n] = __float2half_rn(gated_activation(g, p.act) * u);
  if (p.gate) p.gate[m * p.ldgate + n] = __float2half_rn(g);
  if (p.up) p.up[m * p.ldup + n] = __float2half_rn(u);
}

// Weights stored L x N.  A block has kColumns columns of H; the blocks along y share the rows, p.span each, and a
// block's warps take kTurn of them in turn.  A lane's two words of a row are columns n0 - odd + 2 lane and 64 further:
// an odd row's lack the last column of 128 and an even one's have none before n0, so a block's columns are 126.  The
// sums of even and odd rows stay apart until the end.
constexpr int kColumns = 126, kTurn = 8, kChunk = 1024, kSlots = 130;
template <int MM, bool DUAL>
__global__ void __launch_bounds__(kWarps * 32, MM > 2 ? 2 : 3) tg_gated_columns_kernel(const GatedRows p) {
  __shared__ __align__(16) float mem[MM * kWarps * 2 * kSlots];  // tokens' elements; then each warp's sums
  __shared__ float sum[MM][2 * kSlots];
  constexpr int kX = DUAL ? 2 * MM : MM;  // elements of a row's operands
  static_assert(kWarps * 2 * kSlots >= 2 * kChunk, "the elements fit");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n0 = blockIdx.x * int64_t(kColumns);
  const int64_t first = blockIdx.y * int64_t(p.span), last = min(p.L, first + p.span);
  const int og[2] = {odd(p.wg), odd(p.wg + p.ldwg)}, ou[2] = {odd(p.wu), odd(p.wu + p.ldwu)};
  float2 g[MM][2][2] = {}, u[MM][2][2] = {};  // by token, the row's parity, and 64 columns
  const bool inside = n0 > 0 && n0 + 128 <= p.N;
  auto turn = [&](auto mode, int64_t l, const float* x) {  // rows l to l + kTurn; l is even
    constexpr int kMode = decltype(mode)::value;
    uint32_t wg[kTurn][2], wu[kTurn][2];
#pragma unroll
    for (int i = 0; i < kTurn; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bool in = l + i < last;
        const int64_t at = n0 + 64 * c + 2 * lane;
        wg[i][c] = word<kMode>(p.wg + (l + i) * p.ldwg, at - og[i & 1], p.N, in);
        wu[i][c] = word<kMode>(p.wu + (l + i) * p.ldwu, at - ou[i & 1], p.N, in);
      }
#pragma unroll
    for (int i = 0; i < kTurn; ++i) {
      float xg[MM], xu[MM];
#pragma unroll
      for (int m = 0; m < MM; ++m) {
        xg[m] = x[i * kX + m];
        xu[m] = x[i * kX + m + (kX - MM)];
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float2 a = floats(wg[i][c]), b = floats(wu[i][c]);
#pragma unroll
        for (int m = 0; m < MM; ++m) {
          float2 &s = g[m][i & 1][c], &t = u[m][i & 1][c];
          s.x = fmaf(xg[m], a.x, s.x), s.y = fmaf(xg[m], a.y, s.y);
          t.x = fmaf(xu[m], b.x, t.x), t.y = fmaf(xu[m], b.y, t.y);
        }
      }
    }
  };
  for (int64_t c0 = first; c0 < last; c0 += kChunk) {
    __syncthreads();
    for (int i = threadIdx.x; i < kChunk * kX; i += kWarps * 32) {
      const int m = i / kChunk, l = i % kChunk;
      mem[l * kX + m] = token_at(m < MM ? p.x : p.x2, m % MM, p, c0 + l, last);
    }
    __syncthreads();
    const int rows = static_cast<int>(min(int64_t(kChunk), last - c0));
    for (int l = warp * kTurn; l < rows; l += kWarps * kTurn) {
      if (c0 + l == 0 || l + kTurn > rows || c0 + l + kTurn >= p.L)
        turn(Mode<kEdge>{}, c0 + l, mem + l * kX);
      else if (inside)
        turn(Mode<kInside>{}, c0 + l, mem + l * kX);
      else
        turn(Mode<kRim>{}, c0 + l, mem + l * kX);
    }
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MM; ++m) {
    float* mine = mem + (m * kWarps + warp) * 2 * kSlots + 1;  // slot 0 is column n0 - 1
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float *s = mine + 64 * c + 2 * lane - og[q], *t = mine + kSlots + 64 * c + 2 * lane - ou[q];
        const float2 a = g[m][q][c], b = u[m][q][c];
        s[0] = q ? s[0] + a.x : a.x, s[1] = q ? s[1] + a.y : a.y;
        t[0] = q ? t[0] + b.x : b.x, t[1] = q ? t[1] + b.y : b.y;
      }
      __syncwarp();
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < MM * 2 * kColumns; i += kWarps * 32) {  // over the warps, in order
    const int m = i / (2 * kColumns), w = i / kColumns % 2, c = i % kColumns;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) s += mem[(m * kWarps + k) * 2 * kSlots + w * kSlots + c + 1];
    sum[m][w * kSlots + c] = s;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < MM * kColumns; i += kWarps * 32) {
    const int m = i / kColumns, c = i % kColumns;
    if (m >= p.M || n0 + c >= p.N) continue;
    const float gs = sum[m][c], us = sum[m][kSlots + c];
    finish<DUAL>(p, m, n0 + c, gs, us);
  }
}

// Weights stored N x L.  A warp has four rows of each weight, and kReach words of each at once; p.parts of a
// block's warps share their length.  A lane's word of a row that starts inside a word meets the tokens' elements one
// further left, which it has too.
constexpr int kRows = 4, kReach = 4;
template <int MM, bool DUAL>
constexpr int kLength = MM > 2 && DUAL ? 1024 : 2048;  // elements of a turn in shared memory
template <int MM, bool DUAL>
__global__ void __launch_bounds__(kWarps * 32, MM > 2 ? 2 : 3) tg_gated_rows_kernel(const GatedRows p) {
  constexpr int kLen = kLength<MM, DUAL>, kX = DUAL ? 2 * MM : MM;
  __shared__ __align__(16) float x[kX][kLen + 2];  // from element c0 - 2 on
  __shared__ float red[kWarps][MM][2 * kRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / p.parts, part = warp % p.parts, groups = kWarps / p.parts;
  const int64_t n0 = (blockIdx.x * int64_t(groups) + group) * kRows;
  const __half *pg = p.wg + n0 * p.ldwg, *pu = p.wu + n0 * p.ldwu;  // (n0 is even: the parity of row 0 and row 1)
  const int og[2] = {odd(p.wg), odd(p.wg + p.ldwg)}, ou[2] = {odd(p.wu), odd(p.wu + p.ldwu)};
  float g[MM][kRows] = {}, u[MM][kRows] = {};
  auto reach = [&](auto mode, int64_t l, const float* x0) {
    constexpr int kMode = decltype(mode)::value;
    uint32_t wg[kReach][kRows], wu[kReach][kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int j = 0; j < kReach; ++j) {
        const bool in = n0 + r < p.N;
        const int64_t at = l + 64 * j + 2 * lane;
        wg[j][r] = word<kMode>(pg + r * p.ldwg, at - og[r & 1], p.L, in);
        wu[j][r] = word<kMode>(pu + r * p.ldwu, at - ou[r & 1], p.L, in);
      }
#pragma unroll
    for (int j = 0; j < kReach; ++j) {
      float xs[kX][3];
#pragma unroll
      for (int m = 0; m < kX; ++m) {
        const float* s = x0 + m * (kLen + 2) + 64 * j + 2 * lane;
        const float2 v = *reinterpret_cast<const float2*>(s);
        xs[m][0] = s[-1], xs[m][1] = v.x, xs[m][2] = v.y;
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float2 a = floats(wg[j][r]), b = floats(wu[j][r]);
        const bool sg = og[r & 1], su = ou[r & 1];
#pragma unroll
        for (int m = 0; m < MM; ++m) {
          g[m][r] = fmaf(sg ? xs[m][0] : xs[m][1], a.x, fmaf(sg ? xs[m][1] : xs[m][2], a.y, g[m][r]));
          const float* v = xs[m + kX - MM];
          u[m][r] = fmaf(su ? v[0] : v[1], b.x, fmaf(su ? v[1] : v[2], b.y, u[m][r]));
        }
      }
    }
  };
  const int step = 64 * kReach;
  const int64_t first = blockIdx.y * p.span, stop = min(first + p.span, p.L + 1);
  for (int64_t c0 = first; c0 < stop; c0 += kLen) {  // (element L - 1 may be the first of the word at L)
    __syncthreads();
    for (int i = threadIdx.x; i < kX * (kLen + 2); i += kWarps * 32) {
      const int m = i / (kLen + 2), l = i % (kLen + 2);
      x[m][l] = token_at(m < MM ? p.x : p.x2, m % MM, p, c0 + l - 2, p.L);
    }
    __syncthreads();
    const int64_t end = min(c0 + kLen, stop);
    for (int64_t l = c0 + part * step; l < end; l += p.parts * step) {
      if (l > 0 && l + step <= p.L && n0 + kRows <= p.N)
        reach(Mode<kInside>{}, l, &x[0][2] + (l - c0));
      else if (n0 > 0 && n0 + kRows < p.N)
        reach(Mode<kRim>{}, l, &x[0][2] + (l - c0));
      else
        reach(Mode<kEdge>{}, l, &x[0][2] + (l - c0));
    }
  }
#pragma unroll
  for (int m = 0; m < MM; ++m)
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        g[m][r] += __shfl_xor_sync(~0u, g[m][r], o);
        u[m][r] += __shfl_xor_sync(~0u, u[m][r], o);
      }
      if (lane == 0) {
        red[warp][m][r] = g[m][r];
        red[warp][m][kRows + r] = u[m][r];
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < groups * MM * kRows; i += kWarps * 32) {
    const int r = i % kRows, gr = i / kRows % groups, m = i / (kRows * groups);
    const int64_t n = (blockIdx.x * int64_t(groups) + gr) * kRows + r;
    if (m >= p.M || n >= p.N) continue;
    float gs = 0.0f, us = 0.0f;
    for (int q = 0; q < p.parts; ++q) {
      gs += red[gr * p.parts + q][m][r];
      us += red[gr * p.parts + q][m][kRows + r];
    }
    finish<DUAL>(p, m, n, gs, us);
  }
}

// dWg and dWu: element (r, c) is sum_m rows[m, r] cols[m, c].  A warp has 256 columns, four words a lane, of every
// eighth of kOuterRows rows, which all start at the same half of a word; an odd row's words lie one column further
// left.  Bound by writing for one token (4096 x 14333 49 us with dG's and dU's pass, 4.8 TB/s; four 72).
constexpr int kOuterRows = 128, kWords = 4, kStep = 4;
template <int MM>
__global__ void __launch_bounds__(kWarps * 32) tg_gated_outer_kernel(const GatedOuter p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const __half *rows = blockIdx.z ? p.rows2 : p.rows, *cols = blockIdx.z ? p.cols2 : p.cols;
  const int64_t ld = blockIdx.z ? p.ld2 : p.ld;
  const int64_t first = blockIdx.y * int64_t(kOuterRows) + warp, last = min(p.n_rows, first - warp + kOuterRows);
  if (first >= last) return;
  __half* out = (blockIdx.z ? p.out2 : p.out) + first * ld;
  const int64_t c0 = blockIdx.x * int64_t(64 * kWords) + 2 * lane - odd(out);
  out += c0;
  float b[MM][kWords][2];
  bool in[kWords][2];
#pragma unroll
  for (int j = 0; j < kWords; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t c = c0 + 64 * j + i;
      in[j][i] = c >= 0 && c < p.n_cols;
#pragma unroll
      for (int m = 0; m < MM; ++m)
        b[m][j][i] = m < p.M && in[j][i] ? __half2float(__ldg(cols + m * p.ld_cols + c)) : 0.0f;
    }
  const int64_t strip = blockIdx.x * int64_t(64 * kWords);
  const bool whole = strip > 0 && strip + 64 * kWords <= p.n_cols;
  for (int64_t r0 = first; r0 < last; r0 += kStep * kWarps) {
    float a[kStep][MM];
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int m = 0; m < MM; ++m)
        a[k][m] = m < p.M && r0 + k * kWarps < last ? __half2float(__ldg(rows + m * p.ld_rows + r0 + k * kWarps)) : 0.0f;
#pragma unroll
    for (int k = 0; k < kStep; ++k, out += kWarps * ld) {
      if (r0 + k * kWarps >= last) break;
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        float x = 0.0f, y = 0.0f;
#pragma unroll
        for (int m = 0; m < MM; ++m) {
          x = fmaf(a[k][m], b[m][j][0], x);
          y = fmaf(a[k][m], b[m][j][1], y);
        }
        const __half2 w = __floats2half2_rn(x, y);
        if (whole || (in[j][0] && in[j][1]))
          *reinterpret_cast<__half2*>(out + 64 * j) = w;
        else if (in[j][0])
          out[64 * j] = __low2half(w);
        else if (in[j][1])
          out[64 * j + 1] = __high2half(w);
      }
    }
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

int plan_gated_rows(GatedRows* p, bool trans, bool dual, int sms) {
  const int64_t at_once = int64_t(sms) * (p->M > 2 ? 2 : 3);
  int64_t best = 0;
  int splits = 1;
  p->parts = 1;
  if (!trans) {  // the rows of the longest turn of blocks
    const int64_t blocks = cdiv(p->N, kColumns);
    for (int s = 1; s <= 32 && (s == 1 || p->L >= int64_t(s) * kWarps * kTurn); ++s) {
      const int64_t t = cdiv(blocks * s, at_once) * cdiv(p->L, s) + 8 * s;
      if (s > 1 && t >= best) continue;
      best = t;
      splits = s;
    }
    p->span = cdiv(cdiv(p->L, splits), kTurn) * kTurn;
    return splits;
  }
  // the loads of the longest turn, with one's time for each filling of shared memory and four's for the splits' kernel
  const int64_t sets = cdiv(p->N, kRows), len = p->M > 2 && dual ? kLength<4, true> : kLength<1, false>;
  const int64_t fills = cdiv(p->L + 1, len), reaches = cdiv(std::min(p->L + 1, len), 64 * kReach);
  p->span = fills * len;
  for (int n = 1; n <= std::min<int64_t>(kWarps, len / (64 * kReach)); n *= 2)
    for (int64_t s = 1; s <= std::min<int64_t>(fills, 32); ++s) {
      const int64_t each = cdiv(fills, s), used = cdiv(fills, each);
      const int64_t t = cdiv(cdiv(sets * n, kWarps) * used, at_once) * each * (cdiv(reaches, n) + 1) + (s > 1 ? 4 : 0);
      if (best && t >= best) continue;
      best = t;
      splits = static_cast<int>(used);
      p->parts = n;
      p->span = each * len;
    }
  return splits;
}

cudaError_t launch_gated_rows(const GatedRows& p, bool trans, int splits, cudaStream_t stream) {
  auto go = [&](auto columns, auto rows) {
    const int64_t blocks = trans ? cdiv(cdiv(p.N, kRows) * p.parts, kWarps) : cdiv(p.N, kColumns);
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(splits));
    if (trans)
      rows<<<grid, kWarps * 32, 0, stream>>>(p);
    else
      columns<<<grid, kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
  };
  auto choose = [&](auto tokens) {
    constexpr int MM = decltype(tokens)::value;
    return p.x2 ? go(tg_gated_columns_kernel<MM, true>, tg_gated_rows_kernel<MM, true>)
                : go(tg_gated_columns_kernel<MM, false>, tg_gated_rows_kernel<MM, false>);
  };
  if (p.M == 1) return choose(Mode<1>{});
  if (p.M == 2) return choose(Mode<2>{});
  return choose(Mode<4>{});
}

cudaError_t launch_gated_outer(const GatedOuter& p, cudaStream_t stream) {
  const int outputs = (p.out ? 1 : 0) + (p.out2 ? 1 : 0);
  GatedOuter q = p;
  if (!q.out) q.out = q.out2, q.rows = q.rows2, q.cols = q.cols2, q.ld = q.ld2;
  // (an odd row's words reach one column less far)
  const int64_t strips = cdiv(p.n_cols + 1, 64 * kWords), blocks = cdiv(p.n_rows, kOuterRows);
  for (int64_t y = 0; y < blocks; y += 65535) {  // (the grid's y)
    GatedOuter part = q;
    const int64_t r0 = y * kOuterRows;
    part.rows += r0, part.rows2 += r0;
    part.out += r0 * q.ld;
    if (part.out2) part.out2 += r0 * q.ld2;
    part.n_rows = std::min<int64_t>(q.n_rows - r0, int64_t(65535) * kOuterRows);
    const dim3 grid(static_cast<unsigned>(strips), static_cast<unsigned>(cdiv(part.n_rows, kOuterRows)), outputs);
    if (p.M == 1)
      tg_gated_outer_kernel<1><<<grid, kWarps * 32, 0, stream>>>(part);
    else if (p.M == 2)
      tg_gated_outer_kernel<2><<<grid, kWarps * 32, 0, stream>>>(part);
    else
      tg_gated_outer_kernel<4><<<grid, kWarps * 32, 0, stream>>>(part);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace tg
