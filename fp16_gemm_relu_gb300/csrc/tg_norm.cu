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
#include <atomic>
#include <cstdint>

#include "tg_gemm_relu.h"
#include "tg_internal.h"

namespace {

// How a matrix's rows lie.  Whole: every row starts on a 16-byte boundary and its width is a multiple
// of 8 elements.  Alike: a call's matrices miss the boundaries by the same bytes, row by row
// (contiguous rows of any width do).  Any: each matrix in its own way.
//
// Alike rows r and r + 8 start equally far from a boundary (8 rows are a multiple of 16 bytes
// apart), so a block that takes every eighth row can work on aligned 16-byte blocks, `off` elements to
// the left of the row's own chunks of eight, and keeps the same columns for all of them: nothing is
// shifted, and only a row's first and last block need care.  4095 x 3073 forward 20 us, shifted 32,
// backward 39 and 47; 4096 x 12287 60 and 100, 133 and 199.
enum : int { kRowsAny = 0, kRowsAlike = 1, kRowsWhole = 2 };

// 16 bytes of the 32 in (lo, hi), from byte s on (even, below 16).  s is the same for a row's
// threads, so this branches on it, where selects by its bits would be 20 instructions.
template <int WORD, bool HALF>
__device__ __forceinline__ uint4 shifted(const uint32_t (&w)[8]) {
  if constexpr (HALF)
    return make_uint4(__funnelshift_r(w[WORD], w[WORD + 1], 16),
                      __funnelshift_r(w[WORD + 1], w[WORD + 2], 16),
                      __funnelshift_r(w[WORD + 2], w[WORD + 3], 16),
                      __funnelshift_r(w[WORD + 3], w[WORD + 4], 16));
  return make_uint4(w[WORD], w[WORD + 1], w[WORD + 2], w[WORD + 3]);
}
__device__ __forceinline__ uint4 shift16(const uint4& lo, const uint4& hi, uint32_t s) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  switch (s) {
    case 0: return lo;
    case 2: return shifted<0, true>(w);
    case 4: return shifted<1, false>(w);
    case 6: return shifted<1, true>(w);
    case 8: return shifted<2, false>(w);
    case 10: return shifted<2, true>(w);
    case 12: return shifted<3, false>(w);
    default: return shifted<3, true>(w);
  }
}

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
    return shift16(__ldg(blk), __ldg(blk + 1), b);
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
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint4 before;
  before.x = __shfl_up_sync(0xffffffffu, v.x, 1);
  before.y = __shfl_up_sync(0xffffffffu, v.y, 1);
  before.z = __shfl_up_sync(0xffffffffu, v.z, 1);
  before.w = __shfl_up_sync(0xffffffffu, v.w, 1);
  const bool whole = lane > 0 && e0 + own <= n;
  const bool next_whole = lane < 31 && e0 + 8 + own <= n;
  const uint4 o = shift16(before, v, 16u - b);
  if (whole) *reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(row + e0) - b) = o;
  if (whole && next_whole) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool covered = i < own ? whole : next_whole;
    if (!covered && e0 + i < n) row[e0 + i] = static_cast<uint16_t>(w[i >> 1] >> ((i & 1) << 4));
  }
}

// The same in a ring kernel.  Alike rows: chunk c begins off elements before 8c, on a 16-byte boundary.
template <int A>
__device__ __forceinline__ void store_row_chunk(uint16_t* row, int c, int off, int n, uint4 v, int lane) {
  if constexpr (A != kRowsAlike) {
    store_chunk<A == kRowsWhole>(row, c, n, v, lane);
    return;
  }
  const int e0 = (c << 3) - off;
  if (e0 >= 0 && e0 + 8 <= n) {
    *reinterpret_cast<uint4*>(row + e0) = v;
  } else if (e0 < n) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e0 + i >= 0 && e0 + i < n) row[e0 + i] = static_cast<uint16_t>(w[i >> 1] >> ((i & 1) << 4));
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

// Eight parameters from column 8c - off on (`none` where there are none: a null pointer, before 0 or
// past n).  VEC: the pointer is 16-byte aligned, n a multiple of 8 and off 0.
template <bool VEC, typename P>
__device__ __forceinline__ void load_param(const P* p, int c, int n, float none, f32x2 (&f)[4],
                                           int off = 0) {
  const int e0 = VEC ? c << 3 : (c << 3) - off;
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
    g[i] = (!VEC && p != nullptr && e0 + i >= 0 && e0 + i < n) ? as_float(p + e0 + i) : none;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pair(g[2 * i], g[2 * i + 1]);
}

// Eight columns from e0 on of a partial row of dgamma and dbeta (16-byte aligned rows; WHOLE: e0 is a
// multiple of 8).
template <bool WHOLE>
__device__ __forceinline__ void put_part(float* to_g, float* to_b, int e0, int n, const f32x2 (&g)[4],
                                         const f32x2 (&b)[4]) {
  if (WHOLE && e0 + 8 <= n) {
    ulonglong2* pg = reinterpret_cast<ulonglong2*>(to_g + e0);
    ulonglong2* pb = reinterpret_cast<ulonglong2*>(to_b + e0);
    pg[0] = make_ulonglong2(g[0], g[1]);
    pg[1] = make_ulonglong2(g[2], g[3]);
    pb[0] = make_ulonglong2(b[0], b[1]);
    pb[1] = make_ulonglong2(b[2], b[3]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = e0 + 2 * j;
    const float2 fg = halves(g[j]), fb = halves(b[j]);
    if (e >= 0 && e < n) to_g[e] = fg.x, to_b[e] = fb.x;
    if (e + 1 >= 0 && e + 1 < n) to_g[e + 1] = fg.y, to_b[e + 1] = fb.y;
  }
}

// ---------------------------------------------------------------------------------------
// Rows through shared memory.  A group of threads (a warp, or several) works on one row at a time;
// its first thread fetches rows ahead into a ring of slots with bulk copies, so the next rows'
// latency passes under the current one's arithmetic without holding registers, and a row costs
// one copy instruction instead of a load and its addresses a thread.
// ---------------------------------------------------------------------------------------

// 16-byte blocks that hold elements of a matrix's rows, from `lo` on and before `hi`: blocks in
// between may hold other elements of the same rows' buffer, never anything outside it.
struct Span {
  uintptr_t lo, hi;
};
__device__ __forceinline__ Span span_of(const uint16_t* p, int64_t ld, int64_t rows, int n) {
  return {(reinterpret_cast<uintptr_t>(p) + 15) & ~uintptr_t{15},
          reinterpret_cast<uintptr_t>(p + (rows - 1) * ld + n) & ~uintptr_t{15}};
}

// What one thread copies of a row into a slot (the row starts (row mod 16) bytes in): its aligned
// blocks [from, to), which the barrier is told of; elements of the matrix's first and last block,
// where those are not whole, one by one.
struct Fetch {
  uintptr_t from, to, start;
};
template <bool VEC>
__device__ __forceinline__ Fetch plan_fetch(const uint16_t* row, int n, const Span& sp) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(row), z = reinterpret_cast<uintptr_t>(row + n);
  if constexpr (VEC) return {a, z, a};
  const uintptr_t start = a & ~uintptr_t{15}, end = (z + 15) & ~uintptr_t{15};
  const uintptr_t from = start > sp.lo ? start : sp.lo, to = end < sp.hi ? end : sp.hi;
  return {from, to > from ? to : from, start};
}
// The elements that no whole block has; before the barrier's arrive, which releases them.  Only the
// matrix's first row (among a group's first fetches) and its last (after which its slot gets no other)
// have any: a ring's rows are longer than a block, so every other row lies inside the span.
template <bool VEC>
__device__ __forceinline__ void fetch_edges(const Fetch& f, uint8_t* slot, const uint16_t* row, int n) {
  if constexpr (!VEC) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(row), z = reinterpret_cast<uintptr_t>(row + n);
    for (uintptr_t p = a; p < z && p < f.from; p += 2)
      *reinterpret_cast<uint16_t*>(slot + (p - f.start)) = *reinterpret_cast<const uint16_t*>(p);
    for (uintptr_t p = f.to > a ? f.to : a; p < z; p += 2)
      *reinterpret_cast<uint16_t*>(slot + (p - f.start)) = *reinterpret_cast<const uint16_t*>(p);
  }
}
__device__ __forceinline__ void fetch_blocks(const Fetch& f, uint8_t* slot, uint32_t bar) {
  if (f.to == f.from) return;
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          tg::smem_u32(slot + (f.from - f.start))),
      "l"(f.from), "r"(static_cast<uint32_t>(f.to - f.from)), "r"(bar)
      : "memory");
}

// Waits for a slot: true when it is filled.  A wait that runs out (2 s) is recorded as a timeout and
// ends all later waits of the block, which then runs to its end on what is there.
__device__ __forceinline__ bool slot_wait(uint32_t bar, uint32_t parity, volatile int* late,
                                          unsigned* err) {
  if (tg::mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = tg::global_timer_ns();
  for (uint32_t it = 1; !tg::mbar_try_wait(bar, parity); ++it) {
    if ((it & 63u) != 0) continue;
    if (*late) return false;
    if (tg::global_timer_ns() - t0 > 2000000000ull) {
      *late = 1;
      atomicOr(err, 1u | (tg::kRoleProducer << 8));
      return false;
    }
  }
  return true;
}
// After a wait that ran out, by the thread that fetches, which then fetches nothing more: copies may
// still be on their way, and shared memory may be another block's once this one is gone.  So it waits
// for the last of its `fetched` fetches in each slot, with the same limit.
template <int S>
__device__ __forceinline__ void slots_drain(uint64_t* bars, int fetched) {
  const unsigned long long t0 = tg::global_timer_ns();
  for (int s = 0; s < S && s < fetched; ++s) {
    const uint32_t parity = static_cast<uint32_t>((fetched - 1 - s) / S) & 1u;
    while (!tg::mbar_try_wait(tg::smem_u32(&bars[s]), parity))
      if (tg::global_timer_ns() - t0 > 2000000000ull) return;
  }
}

// 1 for the columns `col` and `col` + 1 that a row of n has, 0 for the others.
__device__ __forceinline__ f32x2 there(int col, int n) {
  return pair(col >= 0 && col < n ? 1.0f : 0.0f, col + 1 >= 0 && col + 1 < n ? 1.0f : 0.0f);
}

// A row's first and last chunk may have elements that are not the row's: which of the eight are, as
// bits for them as fp16 and as factors for them as pairs.  In shared memory, the same for all rows of
// a block (8192 x 5001 backward 99 us; worked out at each read 106).
struct Edges {
  uint4 bits[2];
  f32x2 in[2][4];
};
__device__ __forceinline__ void set_edges(Edges* e, int off, int n) {
  const int i = threadIdx.x;
  if (i >= 16) return;
  const int last = ((n + off - 1) & ~7) - off;  // the last chunk's first column
  const int which = i >> 3, col = (which == 0 ? -off : last) + (i & 7);
  const bool in = col >= 0 && col < n;
  reinterpret_cast<uint16_t*>(&e->bits[which])[i & 7] = in ? 0xFFFFu : 0u;
  reinterpret_cast<float*>(&e->in[which][0])[i & 7] = in ? 1.0f : 0.0f;
}

// Chunk c of the row in a slot, zeros where the row has no element; b: bytes from the slot's start to
// the row's.  Whole and alike rows: block c of the slot, of which an alike row may have only a part (b
// is 2 off then).  Else elements [8c, 8c + 8), shifted together from the two blocks that hold them: with
// 4-byte reads at the row's own offset, a warp's pairs contiguous, 8192 x 4096 forward took 63 us, not 37.
template <int A>
__device__ __forceinline__ uint4 slot_chunk(const uint8_t* slot, uint32_t b, int c, int n,
                                            const Edges& edges) {
  uint4 v = make_uint4(0, 0, 0, 0);
  const int e0 = (c << 3) - (A == kRowsAlike ? static_cast<int>(b >> 1) : 0);
  if (e0 < n) {
    const uint4* blk = reinterpret_cast<const uint4*>(slot) + c;
    v = blk[0];
    if constexpr (A == kRowsAny) v = shift16(v, blk[1], b);
    if (A != kRowsWhole && ((A == kRowsAlike && e0 < 0) || e0 + 8 > n)) {
      const uint4 m = edges.bits[A == kRowsAlike && e0 < 0 ? 0 : 1];
      v = make_uint4(v.x & m.x, v.y & m.y, v.z & m.z, v.w & m.w);
    }
  }
  return v;
}

// The threads of a group meet (id: the group's number in the block).  barrier.sync, not bar.sync:
// the latter counts a whole warp each time that any of its threads comes by, and a warp's threads
// may come apart (waits, row ends, the first lane's fetch).
__device__ __forceinline__ void group_sync(int tpr, int id) {
  __syncwarp();
  if (tpr > 32) asm volatile("barrier.sync %0, %1;" ::"r"(id + 1), "r"(tpr) : "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Sum over a group; slots: a float for each of its warps, not in use by the call before.
__device__ __forceinline__ float group_sum(float v, int tpr, int id, float* slots) {
  v = warp_sum(v);
  if (tpr == 32) return v;
  const int wpr = tpr >> 5, lane = threadIdx.x & 31;
  if (lane == 0) slots[(threadIdx.x >> 5) - id * wpr] = v;
  group_sync(tpr, id);
  return warp_sum(lane < wpr ? slots[lane] : 0.0f);
}

// gamma (or beta) as float32 in shared memory, `chunks` of eight columns, `none` where there is no
// value: the chunks' first halves, then their second halves, so that a warp's 16-byte reads of
// either are contiguous (side by side they would meet in the same banks two by two).
template <bool VEC, typename P>
__device__ __forceinline__ void stage_param(float* dst, const P* p, int n, int chunks, float none,
                                            int off) {
  ulonglong2* q = reinterpret_cast<ulonglong2*>(dst);
#pragma unroll 4
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    f32x2 f[4];
    load_param<VEC>(p, c, n, none, f, off);
    q[c] = make_ulonglong2(f[0], f[1]);
    q[chunks + c] = make_ulonglong2(f[2], f[3]);
  }
}
__device__ __forceinline__ void staged(const float* src, int c, int chunks, f32x2 (&f)[4]) {
  const ulonglong2* q = reinterpret_cast<const ulonglong2*>(src) + c;
  const ulonglong2 a = q[0], b = q[chunks];
  f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}

// Bytes by which a row's start misses a 16-byte boundary.
__device__ __forceinline__ uint32_t row_shift(const uint16_t* p, int64_t ld, int64_t row) {
  return (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) +
          2u * static_cast<uint32_t>(ld) * static_cast<uint32_t>(row)) & 15u;
}

// The first row of a group; its others follow in steps of the grid's groups.  Alike rows: a block's
// rows are all in the class blockIdx.x mod 8 (the grid is a multiple of 8).
template <int A>
__device__ __forceinline__ int first_row(int per_block, int group) {
  if constexpr (A == kRowsAlike)
    return (blockIdx.x & 7) + 8 * ((blockIdx.x >> 3) * per_block + group);
  return blockIdx.x * per_block + group;
}

constexpr int kFwdChunks = 4, kFwdSlots = 2;

// Forward, kFwdChunks chunks a thread: 32 elements share the reductions' and the loop's cost.
// 16384 x 4096 takes 46 us, 0.86 of the copy rate (a row a warp in registers 59, two chunks a thread
// from global memory 59).
template <int THREADS, int BLOCKS, int A, typename P>
__global__ void __launch_bounds__(THREADS, BLOCKS)
    tg_layernorm_kernel(const uint16_t* __restrict__ x, int64_t ldx, const P* __restrict__ gamma,
                        const P* __restrict__ beta, uint16_t* __restrict__ y, int64_t ldy,
                        float* __restrict__ mean, float* __restrict__ rstd, int rows, int n,
                        float eps, unsigned* err, int tpr, int slot_bytes) {
  constexpr int CH = kFwdChunks, S = kFwdSlots;
  constexpr bool VEC = A == kRowsWhole;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t bars[8][S];
  __shared__ float sums[8][2][16];
  __shared__ __align__(16) Edges edges;
  __shared__ volatile int late;
  const int group = threadIdx.x / tpr, t = threadIdx.x - group * tpr, lane = threadIdx.x & 31;
  const int per_block = blockDim.x / tpr, chunks = CH * tpr;
  float* sg = reinterpret_cast<float*>(smem);
  float* so = sg + chunks * 8;
  uint8_t* ring = reinterpret_cast<uint8_t*>(so + chunks * 8) + group * S * slot_bytes;
  const Span sp = span_of(x, ldx, rows, n);
  const int step = gridDim.x * per_block, first = first_row<A>(per_block, group);
  const int count = first < rows ? (rows - 1 - first) / step + 1 : 0;  // rows of this group
  auto fetch = [&](int k, int s) {
    const uint16_t* src = x + (first + int64_t(k) * step) * ldx;
    const uint32_t bar = tg::smem_u32(&bars[group][s]);
    const Fetch f = plan_fetch<VEC>(src, n, sp);
    uint8_t* slot = ring + s * slot_bytes;
    fetch_edges<VEC>(f, slot, src, n);
    tg::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(f.to - f.from));
    fetch_blocks(f, slot, bar);
  };
  if (threadIdx.x == 0) late = 0;
  if (t == 0) {
    for (int s = 0; s < S; ++s) tg::mbar_init(tg::smem_u32(&bars[group][s]), 1);
    tg::fence_mbar_init();
    for (int s = 0; s < S && s < count; ++s) fetch(s, s);
    // a later row's copy may write what fetch_edges has written of the first
    if constexpr (!VEC) tg::fence_async_smem();
  }
  const uint32_t shift = A == kRowsAlike ? row_shift(x, ldx, first) : 0u;  // of all the group's rows
  const int off = static_cast<int>(shift >> 1);
  stage_param<VEC>(sg, gamma, n, chunks, 1.0f, off);
  stage_param<VEC>(so, beta, n, chunks, 0.0f, off);
  if constexpr (!VEC) set_edges(&edges, off, n);
  __syncthreads();
  const float inv_n = 1.0f / static_cast<float>(n);
  bool fetcher = t == 0;
  for (int k = 0; k < count; ++k) {
    const int s = k & 1;
    const int64_t r = first + int64_t(k) * step;
    if (!slot_wait(tg::smem_u32(&bars[group][s]), (k >> 1) & 1, &late, err) && fetcher) {
      slots_drain<S>(bars[group], min(count, k + S));
      fetcher = false;
    }
    const uint32_t b = A == kRowsAny ? row_shift(x, ldx, r) : shift;
    f32x2 v[CH][4], acc = pair(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      unpack8(slot_chunk<A>(ring + s * slot_bytes, b, i * tpr + t, n, edges), v[i]);
      acc = add2(acc, add2(add2(v[i][0], v[i][1]), add2(v[i][2], v[i][3])));
    }
    const float mu = group_sum(sum2(acc), tpr, group, sums[group][0]) * inv_n;
    if (fetcher && k + S < count) fetch(k + S, s);  // everyone has read this slot
    const f32x2 less = pair(-mu, -mu);
    f32x2 q = pair(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int e0 = ((i * tpr + t) << 3) - off;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = add2(v[i][j], less);
      if (VEC ? e0 < n : e0 >= 0 && e0 + 8 <= n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) q = fma2(v[i][j], v[i][j], q);
      } else if (!VEC && e0 < n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x2 d = mul2(v[i][j], edges.in[A == kRowsAlike && e0 < 0 ? 0 : 1][j]);
          q = fma2(d, d, q);
        }
      }
    }
    const float rs = rsqrtf(group_sum(sum2(q), tpr, group, sums[group][1]) * inv_n + eps);
    if (t == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
    const f32x2 times = pair(rs, rs);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      f32x2 g[4], o[4];
      staged(sg, i * tpr + t, chunks, g);
      staged(so, i * tpr + t, chunks, o);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = fma2(mul2(v[i][j], times), g[j], o[j]);
      store_row_chunk<A>(y + r * ldy, i * tpr + t, off, n, pack8(o), lane);
    }
  }
}

// Sums over a warp of R rows' pairs of values, all at once: each halving of the lanes also halves the
// values that a lane has left.  Value (which, row) ends in the lanes [16 which + 16 / R row, + 16 / R).
template <int R>
__device__ __forceinline__ float warp_sums(const float (&a)[R], const float (&b)[R], int lane) {
  const bool up = lane & 16;
  float v[R];
#pragma unroll
  for (int j = 0; j < R; ++j)
    v[j] = (up ? b[j] : a[j]) + __shfl_xor_sync(0xffffffffu, up ? a[j] : b[j], 16);
  float r = v[0];
  if constexpr (R == 2) {
    const bool second = lane & 8;
    r = (second ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, second ? v[0] : v[1], 8);
  }
#pragma unroll
  for (int d = 8 / R; d > 0; d >>= 1) r += __shfl_xor_sync(0xffffffffu, r, d);
  return r;
}

// Backward, CH chunks a thread, R adjacent rows at a time.  A thread keeps the same columns for all
// of its rows, so its part of dgamma and dbeta stays in registers, and each block writes one partial
// row of both (of np floats): part[0][block], part[1][block].  A row's two sums are needed before
// its dx, so the loop works on two turns: it sums the rows of turn k + 1 while it writes dx of turn
// k, and meets once a turn.  CARRY: rows stay in registers in between; otherwise they are read
// from their slots again.
template <int CH, int R, int S, bool CARRY, int A, typename P>
__global__ void __launch_bounds__(512)
    tg_layernorm_backward_kernel(const uint16_t* __restrict__ dy, int64_t lddy,
                                 const uint16_t* __restrict__ x, int64_t ldx,
                                 const P* __restrict__ gamma, const float* __restrict__ mean,
                                 const float* __restrict__ rstd, uint16_t* __restrict__ dx,
                                 int64_t lddx, float* __restrict__ part, int64_t np, int rows,
                                 int n, unsigned* err, int tpr, int slot_bytes) {
  static_assert(R == 1 || (R == 2 && A == kRowsWhole), "one row, or two whole ones");
  constexpr bool VEC = A == kRowsWhole;
  constexpr int V = 2 * R;             // sums of a turn
  constexpr int kLanes = 32 / V;       // lanes that read one of them back
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t bars[8][S];
  __shared__ __align__(16) Edges edges;
  __shared__ float sums[2][V][16];  // [turn mod 2][(which, row)][warp of the block]
  __shared__ volatile int late;
  const int group = threadIdx.x / tpr, t = threadIdx.x - group * tpr, lane = threadIdx.x & 31;
  const int per_block = blockDim.x / tpr, chunks = CH * tpr, wpr = tpr >> 5;
  float* sg = reinterpret_cast<float*>(smem);
  const int stage_bytes = 2 * R * slot_bytes;  // x and dy of each row in turn
  uint8_t* ring = reinterpret_cast<uint8_t*>(sg + chunks * 8) + group * S * stage_bytes;
  const Span sx = span_of(x, ldx, rows, n), sd = span_of(dy, lddy, rows, n);
  const int turns = (rows - 1) / R + 1;
  const int step = gridDim.x * per_block, first = first_row<A>(per_block, group);
  const int count = first < turns ? (turns - 1 - first) / step + 1 : 0;  // turns of this group
  auto row_of = [&](int k) { return (first + int64_t(k) * step) * R; };
  auto fetch = [&](int k, int s) {
    const uint32_t bar = tg::smem_u32(&bars[group][s]);
    Fetch fx[R], fd[R];
    uint32_t bytes = 0;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t row = row_of(k) + j;
      fx[j] = fd[j] = Fetch{0, 0, 0};
      if (row >= rows) continue;
      uint8_t* slot = ring + s * stage_bytes + 2 * j * slot_bytes;
      fx[j] = plan_fetch<VEC>(x + row * ldx, n, sx);
      fd[j] = plan_fetch<VEC>(dy + row * lddy, n, sd);
      fetch_edges<VEC>(fx[j], slot, x + row * ldx, n);
      fetch_edges<VEC>(fd[j], slot + slot_bytes, dy + row * lddy, n);
      bytes += static_cast<uint32_t>((fx[j].to - fx[j].from) + (fd[j].to - fd[j].from));
    }
    tg::mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      uint8_t* slot = ring + s * stage_bytes + 2 * j * slot_bytes;
      fetch_blocks(fx[j], slot, bar);
      fetch_blocks(fd[j], slot + slot_bytes, bar);
    }
  };
  if (threadIdx.x == 0) late = 0;
  if (t == 0) {
    for (int s = 0; s < S; ++s) tg::mbar_init(tg::smem_u32(&bars[group][s]), 1);
    tg::fence_mbar_init();
    for (int s = 0; s < S && s < count; ++s) fetch(s, s);
    // a later row's copy may write what fetch_edges has written of the first
    if constexpr (!VEC) tg::fence_async_smem();
  }
  const uint32_t shift = A == kRowsAlike ? row_shift(x, ldx, first) : 0u;  // of all the group's rows
  const int off = static_cast<int>(shift >> 1);
  stage_param<VEC>(sg, gamma, n, chunks, 1.0f, off);
  if constexpr (!VEC) set_edges(&edges, off, n);
  __syncthreads();
  const float inv_n = 1.0f / static_cast<float>(n);
  f32x2 dg[CH][4], db[CH][4];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dg[i][j] = db[i][j] = pair(0.0f, 0.0f);
  struct Stats {  // of a turn's rows; 0 for a row past the last, whose x and dy count as 0 too
    float mu[R], rs[R];
  };
  auto stats_of = [&](int k) {
    Stats st;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t row = row_of(k) + j;
      const bool live = k < count && row < rows;
      st.mu[j] = live ? __ldg(mean + row) : 0.0f;
      st.rs[j] = live ? __ldg(rstd + row) : 0.0f;
    }
    return st;
  };
  // x and dy of chunk i of a row in its slot; past the row's end, and the last row, 0
  auto read = [&](int s, int64_t row, int j, int i, uint4& xv, uint4& dv) {
    const uint8_t* slot = ring + s * stage_bytes + 2 * j * slot_bytes;
    const int c = i * tpr + t, width = R == 1 || row < rows ? n : 0;
    xv = slot_chunk<A>(slot, A == kRowsAny ? row_shift(x, ldx, row) : shift, c, width, edges);
    dv = slot_chunk<A>(slot + slot_bytes, A == kRowsAny ? row_shift(dy, lddy, row) : shift, c, width, edges);
  };
  constexpr int kHold = CARRY ? CH : 1;
  uint4 cx[R][kHold], cd[R][kHold];  // of turn k
  uint4 nx[R][kHold], nd[R][kHold];  // of turn k + 1
  // With u = x - mean, h = u rstd and g = d gamma: this thread's part of the sums of g and of g u
  // (= g h / rstd) of a turn's rows, and the rows' part of dgamma (d u, times rstd) and dbeta
  auto sum_rows = [&](int k, int s, const Stats& st) {
    f32x2 a2[R], b2[R];
#pragma unroll
    for (int j = 0; j < R; ++j) a2[j] = b2[j] = pair(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      f32x2 g[4];
      staged(sg, i * tpr + t, chunks, g);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int h = CARRY ? i : 0;
        const f32x2 less = pair(-st.mu[j], -st.mu[j]), times = pair(st.rs[j], st.rs[j]);
        f32x2 v[4], d[4];
        read(s, row_of(k) + j, j, i, nx[j][h], nd[j][h]);
        unpack8(nx[j][h], v);
        unpack8(nd[j][h], d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f32x2 du = mul2(d[e], add2(v[e], less));
          a2[j] = fma2(d[e], g[e], a2[j]);
          b2[j] = fma2(du, g[e], b2[j]);
          dg[i][e] = fma2(du, times, dg[i][e]);
          db[i][e] = add2(db[i][e], d[e]);
        }
      }
    }
    float a[R], b[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      a[j] = sum2(a2[j]);
      b[j] = sum2(b2[j]);
    }
    const float v = warp_sums<R>(a, b, lane);
    if (lane % kLanes == 0) sums[k & 1][lane / kLanes][threadIdx.x >> 5] = v;
  };
  auto carry = [&]() {
    if constexpr (CARRY) {
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          cx[j][i] = nx[j][i];
          cd[j][i] = nd[j][i];
        }
    }
  };
  // where this lane reads its value's parts: of one warp, or (R == 2) of two, eight apart
  const int first_warp = lane % kLanes;
  const float* mine = &sums[0][0][0] + lane / kLanes * 16 + group * wpr + first_warp;
  Stats now = stats_of(0), next = stats_of(1);
  bool fetcher = t == 0;
  auto wait = [&](int k, int s, uint32_t phase) {
    if (!slot_wait(tg::smem_u32(&bars[group][s]), phase, &late, err) && fetcher) {
      slots_drain<S>(bars[group], min(count, max(k - 1, 0) + S));
      fetcher = false;
    }
  };
  if (count > 0) {
    wait(0, 0, 0);
    sum_rows(0, 0, now);
  }
  carry();
  group_sync(tpr, group);
  int s = 0, s1 = 1;     // the stages of turns k and k + 1
  uint32_t phase1 = 0;   // of stage s1
  for (int k = 0; k < count; ++k) {
    const Stats ahead = stats_of(k + 2);
    if (k + 1 < count) {
      wait(k + 1, s1, phase1);
      sum_rows(k + 1, s1, next);
    }
    if (dx != nullptr) {
      // dx = rstd (g - mean(g) - h mean(g h)) = d (gamma rstd) + u c1 + c0 with
      // c1 = -rstd^3 mean(g u) and c0 = -rstd mean(g).  Centred: with x for u, and mean c1 taken off
      // c0, a row is off by 2^-24 |mean| / spread of h mean(g h), which dx may cancel to far less
      // (x = 1000 +- 0.5 and dy = h: dx off by a quarter).
      const float* from = mine + (k & 1) * (V * 16);
      float v = first_warp < wpr ? from[0] : 0.0f;
      if (R == 2 && first_warp + 8 < wpr) v += from[8];
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
      f32x2 less[R], of_u[R], plus[R], times[R];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const float a = __shfl_sync(0xffffffffu, v, j * kLanes);
        const float b = __shfl_sync(0xffffffffu, v, 16 + j * kLanes);
        const float rs = now.rs[j], c1 = -rs * (rs * (rs * (b * inv_n))), c0 = -rs * (a * inv_n);
        less[j] = pair(-now.mu[j], -now.mu[j]);
        of_u[j] = pair(c1, c1);
        plus[j] = pair(c0, c0);
        times[j] = pair(rs, rs);
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        f32x2 g[4];
        staged(sg, i * tpr + t, chunks, g);
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const int64_t row = row_of(k) + j;
          if (R > 1 && row >= rows) continue;  // the same for the whole group
          const int h = CARRY ? i : 0;
          if constexpr (!CARRY) read(s, row, j, i, cx[j][0], cd[j][0]);
          f32x2 w[4], d[4], o[4];
          unpack8(cx[j][h], w);
          unpack8(cd[j][h], d);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = fma2(d[e], mul2(g[e], times[j]), fma2(add2(w[e], less[j]), of_u[j], plus[j]));
          store_row_chunk<A>(dx + row * lddx, i * tpr + t, off, n, pack8(o), lane);
        }
      }
    }
    now = next;
    next = ahead;
    carry();
    group_sync(tpr, group);  // stage s and sums[k & 1] are free, sums[(k + 1) & 1] is written
    if (fetcher && k + S < count) fetch(k + S, s);
    s = s1;
    if (++s1 == S) {
      s1 = 0;
      phase1 ^= 1;
    }
  }
  if (part == nullptr) return;
  tg::chain_release();
  // the block's groups are added in their order; the ring is empty by now
  __syncthreads();
  float* groups = sg + chunks * 8;  // [groups][2][np], over the ring
  float* out_g = part + int64_t(blockIdx.x) * np;
  float* out_b = part + (int64_t(gridDim.x) + blockIdx.x) * np;
  float* to_g = per_block == 1 ? out_g : groups + int64_t(group) * 2 * np;
  float* to_b = per_block == 1 ? out_b : to_g + np;
#pragma unroll
  for (int i = 0; i < CH; ++i) 
    put_part<A != kRowsAlike>(to_g, to_b, ((i * tpr + t) << 3) - off, n, dg[i], db[i]);
  if (per_block == 1) return;
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    float g = 0.0f, b = 0.0f;
    for (int k = 0; k < per_block; ++k) {
      g += groups[int64_t(k) * 2 * np + e];
      b += groups[(int64_t(k) * 2 + 1) * np + e];
    }
    out_g[e] = g;
    out_b[e] = b;
  }
}

// ---------------------------------------------------------------------------------------
// Up to 512 columns: a row a warp, straight from global memory (the ring's waits and copies cost more
// than so short a row: 100000 x 128 forward 63 against 20 us, 32768 x 512 backward 36 against 32).
// The next row is loaded before the current one is worked on; the parameters stay in registers.
// ---------------------------------------------------------------------------------------
constexpr int kNarrowThreads = 256;

template <int CH, bool VEC, int THREADS, typename P>
__global__ void __launch_bounds__(THREADS)
    tg_layernorm_direct_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                               const P* __restrict__ gamma, const P* __restrict__ beta,
                               uint16_t* __restrict__ y, int64_t ldy, float* __restrict__ mean,
                               float* __restrict__ rstd, int64_t rows, int n, float eps) {
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * (THREADS >> 5);
  int64_t r = blockIdx.x * int64_t(THREADS >> 5) + (threadIdx.x >> 5);
  const float inv_n = 1.0f / static_cast<float>(n);
  uint4 next[CH];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < CH; ++i) next[i] = load_chunk<VEC>(x + row * ldx, i * 32 + lane, n);
  };
  if (r < rows) load(r);
  f32x2 g[CH][4], o[CH][4];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    load_param<VEC>(gamma, i * 32 + lane, n, 1.0f, g[i]);
    load_param<VEC>(beta, i * 32 + lane, n, 0.0f, o[i]);
  }
  for (; r < rows; r += step) {
    uint4 now[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) now[i] = next[i];
    if (r + step < rows) load(r + step);
    f32x2 s = pair(0.0f, 0.0f), q = s;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      f32x2 v[4];
      unpack8(now[i], v);
      s = add2(s, add2(add2(v[0], v[1]), add2(v[2], v[3])));
    }
    const float mu = warp_sum(sum2(s)) * inv_n;
    const f32x2 less = pair(-mu, -mu);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      f32x2 v[4];
      unpack8(now[i], v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 d = mul2(add2(v[j], less), there(((i * 32 + lane) << 3) + 2 * j, n));
        q = fma2(d, d, q);
      }
    }
    const float rs = rsqrtf(warp_sum(sum2(q)) * inv_n + eps);
    if (lane == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
    const f32x2 times = pair(rs, rs);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      f32x2 v[4];
      unpack8(now[i], v);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = fma2(mul2(add2(v[j], less), times), g[i][j], o[i][j]);
      store_chunk<VEC>(y + r * ldy, i * 32 + lane, n, pack8(v), lane);
    }
  }
}

// Backward, up to 512 columns.
template <int CH, bool VEC, int THREADS, typename P>
__global__ void __launch_bounds__(THREADS)
    tg_layernorm_backward_direct_kernel(const uint16_t* __restrict__ dy, int64_t lddy,
                                        const uint16_t* __restrict__ x, int64_t ldx,
                                        const P* __restrict__ gamma,
                                        const float* __restrict__ mean,
                                        const float* __restrict__ rstd, uint16_t* __restrict__ dx,
                                        int64_t lddx, float* __restrict__ part, int64_t np,
                                        int64_t rows, int n) {
  extern __shared__ float groups[];  // [warps][2][np]
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * (THREADS >> 5);
  int64_t r = blockIdx.x * int64_t(THREADS >> 5) + (threadIdx.x >> 5);
  const float inv_n = 1.0f / static_cast<float>(n);
  f32x2 dg[CH][4], db[CH][4];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dg[i][j] = db[i][j] = pair(0.0f, 0.0f);
  uint4 next_x[CH], next_dy[CH];
  float next_mu = 0.0f, next_rs = 0.0f;
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      next_x[i] = load_chunk<VEC>(x + row * ldx, i * 32 + lane, n);
      next_dy[i] = load_chunk<VEC>(dy + row * lddy, i * 32 + lane, n);
    }
    next_mu = __ldg(mean + row);
    next_rs = __ldg(rstd + row);
  };
  if (r < rows) load(r);
  f32x2 gm[CH][4];
#pragma unroll
  for (int i = 0; i < CH; ++i) load_param<VEC>(gamma, i * 32 + lane, n, 1.0f, gm[i]);
  for (; r < rows; r += step) {
    const float rs = next_rs;
    const f32x2 less = pair(-next_mu, -next_mu), times = pair(rs, rs);
    f32x2 h[CH][4], g[CH][4], a2 = pair(0.0f, 0.0f), b2 = pair(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      f32x2 d[4];  // past the row's end d, and with it g, is 0
      unpack8(next_x[i], h[i]);
      unpack8(next_dy[i], d);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[i][j] = mul2(add2(h[i][j], less), times);
        g[i][j] = mul2(d[j], gm[i][j]);
        a2 = add2(a2, g[i][j]);
        b2 = fma2(g[i][j], h[i][j], b2);
        dg[i][j] = fma2(d[j], h[i][j], dg[i][j]);
        db[i][j] = add2(db[i][j], d[j]);
      }
    }
    if (r + step < rows) load(r + step);
    if (dx != nullptr) {
      const float a = warp_sum(sum2(a2)) * inv_n, b = warp_sum(sum2(b2)) * inv_n;
      const f32x2 less_a = pair(-a, -a), less_b = pair(-b, -b);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        f32x2 out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          out[j] = mul2(times, fma2(h[i][j], less_b, add2(g[i][j], less_a)));
        store_chunk<VEC>(dx + r * lddx, i * 32 + lane, n, pack8(out), lane);
      }
    }
  }
  if (part == nullptr) return;
  tg::chain_release();
  float* mine = groups + int64_t(threadIdx.x >> 5) * 2 * np;
#pragma unroll
  for (int i = 0; i < CH; ++i) put_part<true>(mine, mine + np, (i * 32 + lane) << 3, n, dg[i], db[i]);
  __syncthreads();  // the block's warps are added in their order
  for (int e = threadIdx.x; e < n; e += THREADS) {
    float sg = 0.0f, sb = 0.0f;
    for (int k = 0; k < (THREADS >> 5); ++k) {
      sg += groups[int64_t(k) * 2 * np + e];
      sb += groups[(int64_t(k) * 2 + 1) * np + e];
    }
    part[int64_t(blockIdx.x) * np + e] = sg;
    part[(int64_t(gridDim.x) + blockIdx.x) * np + e] = sb;
  }
}

// ---------------------------------------------------------------------------------------
// More than 16384 columns: a row a block of T threads, as fp16 in registers between the passes over
// it.  A thread's i-th eight elements: whole rows, chunk i T + t.  Others, the columns 8 i T + t,
// T further and so on, each read and written alone: a warp's accesses are contiguous at any alignment,
// and nothing is shifted (4096 x 20001 forward 221 against 247 us with shifted chunks; 4096 x 20000 128).
// ---------------------------------------------------------------------------------------
template <bool VEC, int T>
__device__ __forceinline__ int long_column(int i, int e) {
  return VEC ? ((i * T + static_cast<int>(threadIdx.x)) << 3) + e
             : (8 * i + e) * T + static_cast<int>(threadIdx.x);
}
template <bool VEC, int T>
__device__ __forceinline__ uint4 long_load(const uint16_t* row, int i, int n) {
  if constexpr (VEC) return load_chunk<true>(row, i * T + threadIdx.x, n);
  uint32_t o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int col = long_column<VEC, T>(i, e);
    o[e] = col < n ? __ldg(row + col) : 0u;
  }
  return make_uint4(o[0] | (o[1] << 16), o[2] | (o[3] << 16), o[4] | (o[5] << 16), o[6] | (o[7] << 16));
}
template <bool VEC, int T>
__device__ __forceinline__ void long_store(uint16_t* row, int i, int n, uint4 v) {
  if constexpr (VEC) {
    store_chunk<true>(row, i * T + threadIdx.x, n, v, 0);
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int col = long_column<VEC, T>(i, e);
    if (col < n) row[col] = static_cast<uint16_t>(w[e >> 1] >> ((e & 1) << 4));
  }
}
template <bool VEC, int T, typename P>
__device__ __forceinline__ void long_param(const P* p, int i, int n, float none, f32x2 (&f)[4]) {
  if constexpr (VEC) {
    load_param<true>(p, i * T + threadIdx.x, n, none, f);
    return;
  }
  float g[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int col = long_column<VEC, T>(i, e);
    g[e] = p != nullptr && col < n ? as_float(p + col) : none;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = pair(g[2 * j], g[2 * j + 1]);
}

constexpr int kLongThreads = 1024, kLongChunks = 4;
template <bool VEC, typename P>
__global__ void __launch_bounds__(kLongThreads)
    tg_layernorm_long_kernel(const uint16_t* __restrict__ x, int64_t ldx, const P* __restrict__ gamma,
                             const P* __restrict__ beta, uint16_t* __restrict__ y, int64_t ldy,
                             float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int n,
                             float eps) {
  constexpr int CH = kLongChunks, T = kLongThreads;
  __shared__ float slots[2][32];
  const float inv_n = 1.0f / static_cast<float>(n);
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    uint4 now[CH];
    f32x2 s = pair(0.0f, 0.0f), q = s;
#pragma unroll
    for (int i = 0; i < CH; ++i) now[i] = long_load<VEC, T>(x + r * ldx, i, n);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      f32x2 v[4];
      unpack8(now[i], v);
      s = add2(s, add2(add2(v[0], v[1]), add2(v[2], v[3])));
    }
    const float mu = group_sum(sum2(s), T, 0, slots[0]) * inv_n;
    const f32x2 less = pair(-mu, -mu);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      f32x2 v[4];
      unpack8(now[i], v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 in = pair(long_column<VEC, T>(i, 2 * j) < n ? 1.0f : 0.0f,
                              long_column<VEC, T>(i, 2 * j + 1) < n ? 1.0f : 0.0f);
        const f32x2 d = mul2(add2(v[j], less), in);
        q = fma2(d, d, q);
      }
    }
    const float rs = rsqrtf(group_sum(sum2(q), T, 0, slots[1]) * inv_n + eps);
    if (threadIdx.x == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
    const f32x2 times = pair(rs, rs);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      f32x2 v[4], g[4], o[4];
      long_param<VEC, T>(gamma, i, n, 1.0f, g);
      long_param<VEC, T>(beta, i, n, 0.0f, o);
      unpack8(now[i], v);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = fma2(mul2(add2(v[j], less), times), g[j], o[j]);
      long_store<VEC, T>(y + r * ldy, i, n, pack8(v));
    }
  }
}

// Backward: a thread's part of dgamma and dbeta beside its elements does not fit its registers
// (4096 x 20000 took 630 us so, spilling, against 187), and so these two have a pass of their own.
// A chunk of eight columns a thread (shifted where rows are not whole: element by element 315 us
// against 106 for 4096 x 20001), a split of the rows a block; each split writes one partial row of
// both.  It reads what the pass for dx also reads: 10 bytes an element in all, not 6.
constexpr int kColumnThreads = 128;
template <bool VEC>
__global__ void __launch_bounds__(kColumnThreads)
    tg_layernorm_columns_kernel(const uint16_t* __restrict__ dy, int64_t lddy,
                                const uint16_t* __restrict__ x, int64_t ldx,
                                const float* __restrict__ mean, const float* __restrict__ rstd,
                                float* __restrict__ part, int64_t np, int64_t rows, int n) {
  const int c = blockIdx.x * kColumnThreads + threadIdx.x;
  const int64_t per = (rows + gridDim.y - 1) / gridDim.y;
  const int64_t from = blockIdx.y * per, to = from + per < rows ? from + per : rows;
  f32x2 dg[4], db[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) dg[j] = db[j] = pair(0.0f, 0.0f);
#pragma unroll(VEC ? 4 : 2)
  for (int64_t r = from; r < to; ++r) {
    const float mu = __ldg(mean + r), rs = __ldg(rstd + r);
    const f32x2 less = pair(-mu, -mu), times = pair(rs, rs);
    f32x2 h[4], d[4];
    unpack8(load_chunk<VEC>(x + r * ldx, c, n), h);
    unpack8(load_chunk<VEC>(dy + r * lddy, c, n), d);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      dg[j] = fma2(d[j], mul2(add2(h[j], less), times), dg[j]);
      db[j] = add2(db[j], d[j]);
    }
  }
  put_part<true>(part + blockIdx.y * np, part + (int64_t(gridDim.y) + blockIdx.y) * np, c << 3, n, dg,
                 db);
}

constexpr int kLongDxThreads = 512, kLongDxChunks = 8;
template <bool VEC, typename P>
__global__ void __launch_bounds__(kLongDxThreads)
    tg_layernorm_long_dx_kernel(const uint16_t* __restrict__ dy, int64_t lddy,
                                const uint16_t* __restrict__ x, int64_t ldx,
                                const P* __restrict__ gamma, const float* __restrict__ mean,
                                const float* __restrict__ rstd, uint16_t* __restrict__ dx,
                                int64_t lddx, int64_t rows, int n) {
  constexpr int CH = kLongDxChunks, T = kLongDxThreads;
  __shared__ float slots[2][2][32];
  const float inv_n = 1.0f / static_cast<float>(n);
  int turn = 0;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, turn ^= 1) {
    const float mu = __ldg(mean + r), rs = __ldg(rstd + r);
    uint4 xv[CH], dv[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      xv[i] = long_load<VEC, T>(x + r * ldx, i, n);
      dv[i] = long_load<VEC, T>(dy + r * lddy, i, n);
    }
    const f32x2 less = pair(-mu, -mu);
    f32x2 a2 = pair(0.0f, 0.0f), b2 = a2;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      f32x2 w[4], d[4], g[4];
      long_param<VEC, T>(gamma, i, n, 1.0f, g);
      unpack8(xv[i], w);
      unpack8(dv[i], d);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a2 = fma2(d[j], g[j], a2);
        b2 = fma2(mul2(d[j], add2(w[j], less)), g[j], b2);
      }
    }
    const float a = group_sum(sum2(a2), T, 0, slots[turn][0]);
    const float b = group_sum(sum2(b2), T, 0, slots[turn][1]);
    // as in the ring's kernel: dx = d (gamma rstd) + u c1 + c0
    const float c1 = -rs * (rs * (rs * (b * inv_n))), c0 = -rs * (a * inv_n);
    const f32x2 of_u = pair(c1, c1), plus = pair(c0, c0), times = pair(rs, rs);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      f32x2 w[4], d[4], g[4];
      long_param<VEC, T>(gamma, i, n, 1.0f, g);
      unpack8(xv[i], w);
      unpack8(dv[i], d);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = fma2(d[j], mul2(g[j], times), fma2(add2(w[j], less), of_u, plus));
      long_store<VEC, T>(dx + r * lddx, i, n, pack8(w));
    }
  }
}

// dgamma (blockIdx.y 0) or dbeta (1) from the blocks' partial rows, in a fixed order: 32 columns a
// block, four a thread; each of the 32 thread rows adds every 32nd partial row, eight loads in
// flight, then the thread rows are added in order.  The partial rows (304 of 4096 columns: 10 MB)
// are in L2; the latency of the few loads bounds it.  Chained to the kernel that writes them.
constexpr int kPartRows = 32;
template <typename P>
__global__ void __launch_bounds__(8 * kPartRows)
    tg_layernorm_params_kernel(const float* part, int parts, int64_t np, int n,
                               P* dgamma, P* dbeta) {
  __shared__ float4 sum[kPartRows][8];
  P* out = blockIdx.y == 0 ? dgamma : dbeta;
  if (out == nullptr) return;
  tg::chain_wait();
  const int row = threadIdx.x >> 3, quad = threadIdx.x & 7;
  const int j = blockIdx.x * 32 + quad * 4;  // np is a multiple of 4
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (j < n) {
    const float* src = part + int64_t(blockIdx.y) * parts * np + j;
#pragma unroll 8
    for (int p = row; p < parts; p += kPartRows) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src + p * np));
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
  }
  sum[row][quad] = acc;
  __syncthreads();
  const int e = threadIdx.x;
  if (e >= 32 || blockIdx.x * 32 + e >= n) return;
  float s = 0.0f;
#pragma unroll
  for (int p = 0; p < kPartRows; ++p) s += reinterpret_cast<const float*>(&sum[p][0])[e];
  put(out + blockIdx.x * 32 + e, s);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up4(int64_t n) { return (n + 3) & ~int64_t{3}; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kNarrowWidth = 512, kRingWidth = 16384;  // the ring's rows lie between

// Columns that a group's threads have to have.
int64_t room(int64_t n, int align) { return align == kRowsAlike ? n + 7 : n; }

// `same`: the same pitch and the same base address but for multiples of 16 bytes.  For the ring, and
// unless a power of two lies between the row and its seven more columns: there the warp more that
// they take costs resident warps or does not fit (8192 x 4095 backward 102 against 87 us).
int rows_lie(bool whole, bool same, int64_t n) {
  if (whole) return kRowsWhole;
  const bool fits = n > kNarrowWidth && n <= kRingWidth && ((n - 1) ^ (n + 6)) < n - 1;
  return same && fits ? kRowsAlike : kRowsAny;
}
bool same_pitch(const void* p, int64_t ldp, const void* q, int64_t ldq) {
  return ((reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(q)) & 15u) == 0 &&
         (ldp - ldq) % 8 == 0;
}

// Threads of a group, groups of a block, shared memory and blocks for n columns: ch chunks a
// thread, `slots` slots of `arrays` rows a group, `params` parameters staged.  An alike row may take
// seven columns more, and its grid is a multiple of 8.
struct Shape {
  int tpr, threads, slot_bytes, blocks;
  size_t smem;
};
Shape ring_shape(int64_t rows, int64_t n, int ch, int slots, int arrays, int params, int regs,
                 int align, int sms) {
  Shape s;
  const int64_t chunks = cdiv(room(n, align), 8);
  s.tpr = static_cast<int>(cdiv(chunks, 32 * ch) * 32);
  const int groups = std::max(1, 256 / s.tpr);  // at most 8
  s.threads = groups * s.tpr;
  s.slot_bytes = static_cast<int>((chunks + (align == kRowsAny ? 1 : 0)) * 16);
  s.smem = size_t(params) * ch * s.tpr * 8 * 4 + size_t(groups) * slots * arrays * s.slot_bytes;
  const int by_smem = static_cast<int>(size_t(tg::kSmemLimit) / (s.smem + 2048));
  const int per_sm = std::max(1, std::min(by_smem, 65536 / (regs * s.threads)));
  s.blocks = static_cast<int>(std::min<int64_t>(cdiv(rows, groups), int64_t(sms) * per_sm));
  if (align == kRowsAlike)
    s.blocks = static_cast<int>(std::min<int64_t>(cdiv(s.blocks, 8), std::max(1, sms * per_sm / 8)) * 8);
  return s;
}

Shape forward_shape(int64_t rows, int64_t n, int align, int sms) {
  return ring_shape(rows, n, kFwdChunks, kFwdSlots, 1, 2,
                    align != kRowsAny && n <= 8192 ? 80 : 128, align, sms);
}
// Which backward kernel.  Up to 8192 columns two chunks a thread and three stages; beyond, a block
// has threads for four chunks and shared memory for two stages.  Two rows a turn halve the meetings
// and the reductions' latency where one block fills an SM (8192 x 8192 80 us, one row a turn 90; 8192 x
// 5000 62 and 74); with blocks to spare (16384 x 4096 97 against 86 us), rows to shift (4095 x 3073 62
// against 49) or their end chunks (8192 x 5001 102 against 98), one row that stays in registers is better.
int backward_chunks(int64_t n) { return n <= 8192 ? 2 : 4; }
bool two_rows(int64_t n, int align) { return align == kRowsWhole && n > 4096 && n <= 8192; }
Shape backward_shape(int64_t rows, int64_t n, int align, int sms) {
  Shape s = {};
  if (n <= kNarrowWidth) {
    s.blocks = static_cast<int>(std::min<int64_t>(cdiv(rows, kNarrowThreads / 32), 2 * sms));
    return s;
  }
  if (n > kRingWidth) {  // the splits of the columns' pass: eight blocks an SM, eight rows each
    const int64_t most = 8 * int64_t(sms) / cdiv(n, 8 * kColumnThreads);
    s.blocks = static_cast<int>(std::max<int64_t>(1, std::min(most, cdiv(rows, 8))));
    return s;
  }
  if (two_rows(n, align)) return ring_shape((rows - 1) / 2 + 1, n, 2, 3, 4, 1, 128, align, sms);
  const int ch = backward_chunks(n);
  return ch == 2 ? ring_shape(rows, n, ch, 3, 2, 1, 120, align, sms)
                 : ring_shape(rows, n, ch, 2, 2, 1, 128, align, sms);
}

template <auto KERNEL>
struct Kernel {
  static constexpr auto value = KERNEL;
};

// Launches a ring kernel.  That it may have more than 48 KB of shared memory is said once for each
// device: said again at every launch it is a fifth of a small call's time.
constexpr int kRingSmem = tg::kSmemLimit - 1280;  // beside the kernels' static shared memory
template <auto KERNEL, typename... Args>
cudaError_t launch_ring(const Shape& s, cudaStream_t st, Args... args) {
  static std::atomic<uint64_t> told{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);  // device_info has refused devices past 63
  if ((told.load(std::memory_order_relaxed) & bit) == 0) {
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
    if (e != cudaSuccess) return e;
    told.fetch_or(bit, std::memory_order_relaxed);
  }
  KERNEL<<<s.blocks, s.threads, s.smem, st>>>(args..., s.tpr, s.slot_bytes);
  return cudaGetLastError();
}

template <int A, typename P>
cudaError_t forward(const void* x, const void* gamma, const void* beta, void* y, float* mean,
                    float* rstd, int64_t rows, int64_t n, int64_t ldx, int64_t ldy, float eps,
                    int sms, unsigned* err, cudaStream_t st) {
  constexpr bool VEC = A == kRowsWhole;
  const uint16_t* px = static_cast<const uint16_t*>(x);
  const P *g = static_cast<const P*>(gamma), *b = static_cast<const P*>(beta);
  uint16_t* py = static_cast<uint16_t*>(y);
  auto direct = [&](auto kern, int threads, int64_t blocks) {
    kern<<<static_cast<unsigned>(blocks), threads, 0, st>>>(px, ldx, g, b, py, ldy, mean, rstd, rows,
                                                            static_cast<int>(n), eps);
    return cudaGetLastError();
  };
  if constexpr (A != kRowsAlike) {
    if (n <= kNarrowWidth) {
      constexpr int kT = kNarrowThreads;
      const int64_t blocks = std::min<int64_t>(cdiv(rows, kT / 32), int64_t(sms) * 4);
      return n <= 256 ? direct(tg_layernorm_direct_kernel<1, VEC, kT, P>, kT, blocks)
                      : direct(tg_layernorm_direct_kernel<2, VEC, kT, P>, kT, blocks);
    }
    if (n > kRingWidth)
      return direct(tg_layernorm_long_kernel<VEC, P>, kLongThreads,
                    std::min<int64_t>(rows, sms));
  }
  const Shape s = forward_shape(rows, n, A, sms);
  const int width = static_cast<int>(n), count = static_cast<int>(rows);
  // up to 8192 columns a block has 256 threads at most: three of them an SM where registers allow
  if (n <= 8192)
    return launch_ring<tg_layernorm_kernel<256, A == kRowsAny ? 2 : 3, A, P>>(
        s, st, px, ldx, g, b, py, ldy, mean, rstd, count, width, eps, err);
  return launch_ring<tg_layernorm_kernel<512, 1, A, P>>(s, st, px, ldx, g, b, py, ldy, mean, rstd,
                                                          count, width, eps, err);
}

template <int A, typename P>
cudaError_t backward(const void* dy, const void* x, const void* gamma, const float* mean,
                     const float* rstd, void* dx, void* dgamma, void* dbeta, float* part,
                     int64_t rows, int64_t n, int64_t lddy, int64_t ldx, int64_t lddx,
                     const Shape& s, int sms, unsigned* err, cudaStream_t st) {
  constexpr bool VEC = A == kRowsWhole;
  const uint16_t *pd = static_cast<const uint16_t*>(dy), *px = static_cast<const uint16_t*>(x);
  const P* g = static_cast<const P*>(gamma);
  uint16_t* out = static_cast<uint16_t*>(dx);
  const int width = static_cast<int>(n);
  const int64_t np = round_up4(n);
  cudaError_t e;
  auto ring = [&]() {
    auto go = [&](auto which) {
      return launch_ring<which.value>(s, st, pd, lddy, px, ldx, g, mean, rstd, out, lddx, part, np,
                                      static_cast<int>(rows), width, err);
    };
    if (n > 8192) return go(Kernel<tg_layernorm_backward_kernel<4, 1, 2, false, A, P>>{});
    if (!two_rows(n, A)) return go(Kernel<tg_layernorm_backward_kernel<2, 1, 3, true, A, P>>{});
    return go(Kernel<tg_layernorm_backward_kernel<2, 2, 3, false, kRowsWhole, P>>{});
  };
  auto params = [&]() {
    return tg::launch_chained(tg_layernorm_params_kernel<P>, true,
                              dim3(static_cast<unsigned>(cdiv(n, 32)), 2), 8 * kPartRows, 0, st, part,
                              s.blocks, np, width, static_cast<P*>(dgamma), static_cast<P*>(dbeta));
  };
  if constexpr (A == kRowsAlike) {
    e = ring();
  } else if (n <= kNarrowWidth) {
    constexpr int kT = kNarrowThreads;
    const size_t smem = part ? size_t(kT / 32) * 2 * np * 4 : 0;  // at most 32 KB
    auto direct = [&](auto kern) {
      kern<<<s.blocks, kT, smem, st>>>(pd, lddy, px, ldx, g, mean, rstd, out, lddx, part, np, rows, width);
      return cudaGetLastError();
    };
    e = n <= 256 ? direct(tg_layernorm_backward_direct_kernel<1, VEC, kT, P>)
                 : direct(tg_layernorm_backward_direct_kernel<2, VEC, kT, P>);
  } else if (n > kRingWidth) {
    if (part != nullptr) {  // before dx, which may take dy's or x's place
      tg_layernorm_columns_kernel<VEC>
          <<<dim3(static_cast<unsigned>(cdiv(n, 8 * kColumnThreads)), static_cast<unsigned>(s.blocks)),
             kColumnThreads, 0, st>>>(pd, lddy, px, ldx, mean, rstd, part, np, rows, width);
      if ((e = cudaGetLastError()) != cudaSuccess || (e = params()) != cudaSuccess) return e;
    }
    if (out == nullptr) return cudaSuccess;
    tg_layernorm_long_dx_kernel<VEC, P>
        <<<static_cast<unsigned>(std::min<int64_t>(rows, sms)), kLongDxThreads, 0, st>>>(
            pd, lddy, px, ldx, g, mean, rstd, out, lddx, rows, width);
    return cudaGetLastError();
  } else {
    e = ring();
  }
  if (e != cudaSuccess || part == nullptr) return e;
  return params();
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
  const bool whole = aligned16(X) && aligned16(Y) && aligned16(gamma) && aligned16(beta) &&
                     ldx % 8 == 0 && ldy % 8 == 0 && N % 8 == 0;
  const int align = rows_lie(whole, same_pitch(X, ldx, Y, ldy), N);
  auto run = [&](auto f) { return f(X, gamma, beta, Y, mean, rstd, M, N, ldx, ldy, eps, sms, err, s); };
  auto with = [&](auto type) {
    using P = decltype(type);
    return align == kRowsWhole   ? run(forward<kRowsWhole, P>)
           : align == kRowsAlike ? run(forward<kRowsAlike, P>)
                                 : run(forward<kRowsAny, P>);
  };
  const cudaError_t e = param_type == TG_TYPE_F16 ? with(__half()) : with(0.0f);
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
  const bool whole = aligned16(dY) && aligned16(X) && aligned16(dX) && aligned16(gamma) &&
                     lddy % 8 == 0 && ldx % 8 == 0 && (!dX || lddx % 8 == 0) && N % 8 == 0;
  const bool same = same_pitch(X, ldx, dY, lddy) && (!dX || same_pitch(X, ldx, dX, lddx));
  const int align = rows_lie(whole, same, N);
  const Shape shape = backward_shape(M, N, align, sms);
  float* part = nullptr;
  if (dgamma || dbeta) {
    st = tg::scratch_alloc(size_t(2) * shape.blocks * round_up4(N) * 4, s, reinterpret_cast<void**>(&part));
    if (st != TG_OK) return st;
  }
  auto run = [&](auto f) {
    return f(dY, X, gamma, mean, rstd, dX, dgamma, dbeta, part, M, N, lddy, ldx, lddx, shape, sms, err, s);
  };
  auto with = [&](auto type) {
    using P = decltype(type);
    return align == kRowsWhole   ? run(backward<kRowsWhole, P>)
           : align == kRowsAlike ? run(backward<kRowsAlike, P>)
                                 : run(backward<kRowsAny, P>);
  };
  e = param_type == TG_TYPE_F16 ? with(__half()) : with(0.0f);
  if (part) {
    const cudaError_t fe = cudaFreeAsync(part, s);
    if (e == cudaSuccess) e = fe;
  }
  return e == cudaSuccess ? TG_OK : tg::record_cuda_error(e);
}

}  // extern "C"
