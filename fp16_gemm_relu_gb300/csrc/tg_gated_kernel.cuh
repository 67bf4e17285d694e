// tg_gated_kernel.cuh — the gated product H = act(X Wg) * (X Wu) on the tensor cores of sm_103a, and the
// activations' derivatives.
//
// The roles are those of tg_gemm_kernel.cuh (TMA producer, tcgen05 issuer, epilogue; one CTA a tile of 128
// rows, or a pair of CTAs a tile of 256).  What differs is the right operand: of the tile's BN columns the
// first half are Wg's and the second half Wu's, the same ones, so that the accumulator of a row holds a
// gate and its up BN / 2 columns apart, in the same TMEM lanes.  One product of twice the width then reads
// X once, and its epilogue has both factors of H in registers: neither leaves the chip in float32.  In a
// pair, CTA 0 loads the tile's columns of Wg and CTA 1 those of Wu, each as an ordinary half of the
// pair's right operand.  Eight epilogue warps, each with 32 rows and 64 columns of H: an activation costs up to 20
// instructions, and kept pre-activations are two more tiles to store, read from tensor memory again rather
// than held in registers.
//
// Bound by the tensor cores at training sizes: 8192 x 4096 x 14336 1051 us with gate and up kept, 1.83 PFLOP/s (as
// two float32 products and a pass over them 1474); 1.55 in a power-capped loop.  Bound by the weights' bytes for
// few tokens: 64 x 8192 x 28672 147 us, 6.4 TB/s; one token of 4096 x 14336 42 us, 5.5 TB/s.
#pragma once

#include "tg_gemm_kernel.cuh"

namespace tg {

enum : int { kActSilu = 4 };

// 1 / (1 + e^-x): 0 and 1 at the infinities.
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// x times this logistic is gelu's tanh form: (1 + tanh u) / 2 = 1 / (1 + e^-2u).
__device__ __forceinline__ float gelu_logistic(float x) {
  return logistic(1.5957691216057308f * (x + 0.044715f * x * x * x));
}

// The activation of a gate, in float32.  silu(x) = x / (1 + e^-x) (Elfwing et al., 2018); the others
// are the fused epilogue's (the tanh form as a logistic: half the instructions, and no cancellation far
// below zero).
__device__ __forceinline__ float gated_activation(float x, int act) {
  if (act == kActSilu) return x * logistic(x);
  if (act == kActGeluTanh) return x * gelu_logistic(x);
  return activation(x, act);
}

// Its derivative.  Where the derivative is 0 or 1 to float32's precision it is taken as that, so that
// an infinite gate does not become infinity times 0; a NaN stays one (but in relu, as in its value).
__device__ __forceinline__ float gated_slope(float x, int act) {
  switch (act) {
    case kActRelu: return x > 0.0f ? 1.0f : 0.0f;
    case kActGelu: {
      if (fabsf(x) > 16.0f) return x > 0.0f ? 1.0f : 0.0f;
      return 0.5f * (1.0f + erff(x * 0.70710678118654752f)) +
             x * 0.39894228040143268f * __expf(-0.5f * x * x);
    }
    case kActGeluTanh: {
      if (fabsf(x) > 16.0f) return x > 0.0f ? 1.0f : 0.0f;
      const float s = gelu_logistic(x);
      return s * (1.0f + (1.0f - s) * x * 1.5957691216057308f * (1.0f + 0.134145f * x * x));
    }
    case kActSilu: {
      if (fabsf(x) > 100.0f) return x > 0.0f ? 1.0f : 0.0f;
      const float s = logistic(x);
      return s * (1.0f + x * (1.0f - s));
    }
    default: return 1.0f;
  }
}

// CG CTAs a tile; BN columns of the accumulator, BN / 2 of H.
template <int CG, int BN>
struct GatedCfg {
  static_assert(BN == 256 || (CG == 1 && BN == 128), "tiles of 256 columns, or of 128 in one CTA");
  static constexpr int kKB = CG;                          // k-blocks of a stage
  static constexpr int kHN = BN / 2;                      // columns of H
  static constexpr int kEpiWarps = BN / 32;               // each 32 rows and 64 columns of H
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kBRows = BN / CG;                  // rows (or columns) of the weights in this CTA
  static constexpr int kAStage = kKB * kBM * kBK * 2;
  static constexpr int kBStage = kKB * kBK * kBRows * 2;
  static constexpr int kStageBytes = kAStage + kBStage;
  static constexpr int kStagingBytes = kEpiWarps * kStagingBuf;
  static constexpr int kStagesFit = (kSmemLimit - kSmemReserve - kStagingBytes) / kStageBytes;
  static constexpr int kStages = kStagesFit > 8 ? 8 : kStagesFit;
  static constexpr int kAccStride = BN;
  static constexpr int kTmemCols = 2 * kAccStride;
  static constexpr int kSmemBytes = kSmemReserve + kStages * kStageBytes + kStagingBytes;
  static_assert(kSmemBytes <= kSmemLimit, "shared memory budget exceeded");
};

struct GatedParams {
  GemmParams g;              // tiles (of BN / 2 columns of H), k-blocks, M and N, act, time limit, error word
  __half *h, *gate, *up;     // gate and up may be NULL
  long long ldh, ldgate, ldup;
  int tma;                   // the outputs take TMA stores (16-byte rows); else plain ones
  int a_rows;                // rows of X's box: 128, or (one row of tiles) M rounded up to 8
  int nw;                    // float32 partial sums: column of the first up
  int rotate;                // tiles start at different k-blocks (CG == 1)
};

// v = act(g) * v, both float32 bits.  The activation's branch is outside of the loop.
__device__ __forceinline__ void gated_values(const uint32_t (&g)[32], uint32_t (&v)[32], int act) {
  auto all = [&](auto f) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      v[i] = __float_as_uint(f(__uint_as_float(g[i])) * __uint_as_float(v[i]));
  };
  switch (act) {
    case kActSilu: all([](float x) { return x * logistic(x); }); break;
    case kActRelu: all([](float x) { return activation(x, kActRelu); }); break;
    case kActGelu: all([](float x) { return activation(x, kActGelu); }); break;
    case kActGeluTanh: all([](float x) { return x * gelu_logistic(x); }); break;
    default: all([](float x) { return x; });
  }
}

// 32 columns (the c-th 32 of 64) of the lane's row as fp16 into the warp's staging buffer.
__device__ __forceinline__ void stage_half(uint8_t* stg, const uint32_t (&v)[32], int c, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(__uint_as_float(v[8 * j + 2 * i]), __uint_as_float(v[8 * j + 2 * i + 1]));
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(stg + lane * 128 + (((4 * c + j) ^ (lane & 7)) << 4)) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The warp's 32 rows x 64 columns of fp16 in its staging buffer (128B-swizzled rows) to rows row0 and
// columns col0 on of an output.
__device__ __forceinline__ void gated_store(const CUtensorMap* tm, bool tma, __half* out, long long ld,
                                            const uint8_t* stg, int row0, int col0, int M, int N,
                                            int lane, uint64_t policy) {
  if (tma) {
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d_hint(tm, smem_u32(stg), col0, row0, policy);
      bulk_commit();
    }
    return;
  }
  store_rows(out, ld, stg, row0, col0, M, N, lane);
}

// tmX: fp16 X, dims {K, M}, box {64, a_rows};  tmG, tmU: the weights, B_K (stored N x K): dims {K, N}, box
// {64, 128 in a pair, else BN / 2};  else (K x N): dims {N, K}, box {64, 64 CG};  tmH, tmGate, tmUp: fp16
// outputs, dims {N, M}, box {64, 32};  OUT_F32: tmH is the float32 partial sums, dims {2 nw, M, splits},
// box {32, 32, 1}.  All with 128B swizzle.
template <int CG, int BN, bool B_K, bool OUT_F32>
__device__ __forceinline__ void gated_body(const CUtensorMap& tmX, const CUtensorMap& tmG,
                                           const CUtensorMap& tmU, const CUtensorMap& tmH,
                                           const CUtensorMap& tmGate, const CUtensorMap& tmUp,
                                           const GatedParams& gp) {
  using Cfg = GatedCfg<CG, BN>;
  constexpr int S = Cfg::kStages, KB = Cfg::kKB, HN = Cfg::kHN;
  constexpr int kAtom = kBM * kBK * 2;             // 128 rows x 64 k, K-major
  constexpr int kBAtom = Cfg::kBRows * kBK * 2;    // this CTA's rows of the weights x 64 k, K-major
  constexpr int kMNBox = KB * kBK * 64 * 2;        // 64 columns x KB 64 k, MN-major
  const GemmParams& p = gp.g;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + S * Cfg::kAStage;
  uint8_t* sStg = sB + S * Cfg::kBStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sStg + Cfg::kStagingBytes);
  uint64_t* full = bars;        // pairs: used in the leader
  uint64_t* empty = bars + S;   // in both CTAs
  uint64_t* tfull = bars + 2 * S;
  uint64_t* tempty = tfull + 2; // pairs: used in the leader
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile uint32_t* abort_flag = tmem_holder + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0;
  const int first = static_cast<int>(blockIdx.x) / CG;
  const int step = static_cast<int>(gridDim.x) / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), CG * Cfg::kEpiWarps);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmG);
    prefetch_tmap(&tmU);
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(smem_u32(tmem_holder), Cfg::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_holder), Cfg::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (CG == 2)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  chain_wait();
  chain_release();

  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t armed = 0, armed_parity = 0;
      bool dropped = false;
      const uint32_t bytes = CG == 2 ? 2 * Cfg::kStageBytes : gp.a_rows * kBK * 2 + Cfg::kBStage;
      for (int u = first; u < p.units; u += step) {
        const Unit w = unit_of(p, u);
        const int xrow = (w.m_blk * CG + static_cast<int>(rank)) * kBM;
        const int col = w.n_blk * HN;
        // few rows of X: the weights stream from memory once, and tiles that all walk the same rows of
        // them at the same time would meet in the same memory channels: each starts elsewhere
        const int span = w.kb_end - w.kb_begin;
        int at = CG == 1 && gp.rotate ? static_cast<int>(static_cast<unsigned>(u) * 7u % static_cast<unsigned>(span)) : 0;
        for (int kb = 0; kb < span; kb += KB) {
          if (!wait_phase(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, p, kRoleProducer))
            goto producer_done;
          if ((p.debug_flags & kDebugDropFirstStage) && first == 0 && rank == 0 && !dropped) {
            dropped = true;  // injected fault: this stage is never filled
          } else {
            const uint32_t fb_local = smem_u32(&full[stage]);
            if (rank == 0) {
              mbar_arrive_expect_tx(fb_local, bytes);
              armed |= 1u << stage;
              armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
            }
            const uint32_t fb = CG == 2 ? mapa_shared(fb_local, 0) : fb_local;
            const uint32_t a_dst = smem_u32(sA + stage * Cfg::kAStage);
            const uint32_t b_dst = smem_u32(sB + stage * Cfg::kBStage);
            auto load = [&](uint32_t dst, const CUtensorMap* m, int c0, int c1) {
              if constexpr (CG == 2)
                tma_load_2d_pair(dst, m, fb, c0, c1);
              else
                tma_load_2d(dst, m, fb, c0, c1);
            };
            const int k0 = w.kb_begin + at;
            // all k-blocks of a stage load (past K as zeros), so its byte count is fixed
#pragma unroll
            for (int h = 0; h < KB; ++h) load(a_dst + h * kAtom, &tmX, (k0 + h) * kBK, xrow);
            if constexpr (CG == 2) {
              const CUtensorMap* m = rank ? &tmU : &tmG;
              if constexpr (B_K) {
#pragma unroll
                for (int h = 0; h < KB; ++h) load(b_dst + h * kBAtom, m, (k0 + h) * kBK, col);
              } else {
#pragma unroll
                for (int j = 0; j < Cfg::kBRows / 64; ++j)
                  load(b_dst + j * kMNBox, m, col + j * 64, k0 * kBK);
              }
            } else if constexpr (B_K) {
              load(b_dst, &tmG, k0 * kBK, col);
              load(b_dst + HN * kBK * 2, &tmU, k0 * kBK, col);
            } else {
#pragma unroll
              for (int j = 0; j < HN / 64; ++j) {
                load(b_dst + j * kMNBox, &tmG, col + j * 64, k0 * kBK);
                load(b_dst + (HN / 64 + j) * kMNBox, &tmU, col + j * 64, k0 * kBK);
              }
            }
          }
          at += KB;
          if (CG == 1 && at == span) at = 0;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    producer_done:
      // no load may still be writing shared memory when the CTA exits (pairs: the leader's full
      // barriers count both CTAs' bytes)
      for (int s = 0; s < S; ++s)
        if (armed & (1u << s)) wait_phase_drain(smem_u32(&full[s]), (armed_parity >> s) & 1u, p);
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer (pairs: the leader) ------------------------------
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_f16_f32(CG * kBM, BN, 0, !B_K);
      int stage = 0;
      uint32_t phase = 0;
      int t = 0;
      for (int u = first; u < p.units; u += step, ++t) {
        const Unit w = unit_of(p, u);
        const int buf = t & 1;
        const uint32_t use = static_cast<uint32_t>(t >> 1) & 1u;
        if (!wait_phase(smem_u32(&tempty[buf]), use ^ 1u, abort_flag, p, kRoleMma)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * Cfg::kAccStride);
        bool ok = true;
        for (int kb = w.kb_begin; kb < w.kb_end; kb += KB) {
          if (!wait_phase(smem_u32(&full[stage]), phase, abort_flag, p, kRoleMma)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(sA + stage * Cfg::kAStage);
          const uint32_t b_addr = smem_u32(sB + stage * Cfg::kBStage);
          const uint64_t ad = desc_kmajor(a_addr);
          const uint64_t bd = B_K ? desc_kmajor(b_addr) : sw128_desc(b_addr, kMNBox, 1024);
          const int nk = (w.kb_end - kb >= KB ? KB : w.kb_end - kb) * (kBK / kUmmaK);
#pragma unroll
          for (int k = 0; k < KB * (kBK / kUmmaK); ++k) {
            const uint64_t a_off = static_cast<uint64_t>((k >> 2) * (kAtom >> 4) + 2 * (k & 3));
            const uint64_t b_off = B_K ? static_cast<uint64_t>((k >> 2) * (kBAtom >> 4) + 2 * (k & 3))
                                       : static_cast<uint64_t>(128 * k);
            if (k < nk) {
              const uint32_t acc = (kb > w.kb_begin || k > 0) ? 1u : 0u;
              if constexpr (CG == 2)
                umma_f16_pair(d_tmem, ad + a_off, bd + b_off, idesc, acc);
              else
                umma_f16(d_tmem, ad + a_off, bd + b_off, idesc, acc);
            }
          }
          if constexpr (CG == 2)
            umma_commit_pair_mc(smem_u32(&empty[stage]), 0x3);
          else
            umma_commit(smem_u32(&empty[stage]));
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if constexpr (CG == 2)
          umma_commit_pair_mc(smem_u32(&tfull[buf]), 0x3);
        else
          umma_commit(smem_u32(&tfull[buf]));
      }
      // every MMA issued by this thread has finished before TMEM can be released
      if constexpr (CG == 2)
        umma_commit_pair(smem_u32(drain));
      else
        umma_commit(smem_u32(drain));
      wait_phase_drain(smem_u32(drain), 0u, p);
    }
  } else {
    // ------------------------------ epilogue ------------------------------
    const int q = warp & 3;             // TMEM lane quarter this warp may access
    const int ew = warp - 2, part = ew >> 2;
    uint8_t* stg = sStg + ew * kStagingBuf;
    // the outputs are not read here again: they need not push the operands, which other tiles read, out of L2
    const uint64_t policy = evict_first_policy();
    int t = 0;
    for (int u = first; u < p.units; u += step, ++t) {
      const Unit w = unit_of(p, u);
      const int row0 = (w.m_blk * CG + static_cast<int>(rank)) * kBM + q * 32;
      const int col0 = w.n_blk * HN + part * 64;
      const int buf = t & 1;
      const uint32_t use = static_cast<uint32_t>(t >> 1) & 1u;
      int ok = 0;
      if (lane == 0) ok = wait_phase(smem_u32(&tfull[buf]), use, abort_flag, p, kRoleEpilogue);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2)
            mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[buf]), 0));
          else
            mbar_arrive(smem_u32(&tempty[buf]));
        }
      };
      if (row0 >= p.M || col0 >= p.N) {  // nothing of this warp's is in the outputs
        release();
        continue;
      }
      const uint32_t gates = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                          static_cast<uint32_t>(buf * Cfg::kAccStride + part * 64);
      const uint32_t ups = gates + HN;
      // the staging buffer is free when the last store has read it
      auto stage_free = [&]() {
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
      };
      if constexpr (OUT_F32) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {  // 32 columns of the gate, 32 more, and of the up
          uint32_t r[32];
          tmem_ld_x32((c < 2 ? gates : ups) + (c & 1) * 32, r);
          tmem_wait_ld(r);
          if (c == 3) release();
          const int at = col0 + (c & 1) * 32;
          if (at >= gp.nw) continue;
          stage_free();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tmH, smem_u32(stg), (c < 2 ? 0 : gp.nw) + at, row0, w.split);
            bulk_commit();
          }
        }
      } else {
        // 32 columns of H from their gates and ups
        stage_free();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t g[32], v[32];
          tmem_ld_x32(gates + c * 32, g);
          tmem_ld_x32(ups + c * 32, v);
          tmem_wait_ld(g);
          tmem_wait_ld(v);
          if (c == 1 && !gp.gate && !gp.up) release();
          gated_values(g, v, p.act);
          stage_half(stg, v, c, lane);
        }
        gated_store(&tmH, gp.tma, gp.h, gp.ldh, stg, row0, col0, p.M, p.N, lane, policy);
        if (gp.gate || gp.up) {
#pragma unroll 1
          for (int o = 0; o < 2; ++o) {  // the pre-activations, read from TMEM again
            stage_free();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t v[32];
              tmem_ld_x32((o ? ups : gates) + c * 32, v);
              tmem_wait_ld(v);
              if (o == 1 && c == 1) release();
              stage_half(stg, v, c, lane);
            }
            if (o ? gp.up != nullptr : gp.gate != nullptr)
              gated_store(o ? &tmUp : &tmGate, gp.tma, o ? gp.up : gp.gate, o ? gp.ldup : gp.ldgate,
                          stg, row0, col0, p.M, p.N, lane, policy);
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all<0>();
    __syncwarp();
  }

  if (CG == 2 && rank != 0 && *abort_flag && threadIdx.x == 0) __nanosleep(200000);
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // all MMAs into either CTA's TMEM and remote arrivals are done
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (CG == 2)
      tmem_dealloc_pair(tmem_base, Cfg::kTmemCols);
    else
      tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

template <int BN, bool B_K, bool OUT_F32>
__global__ void __launch_bounds__(GatedCfg<1, BN>::kThreads, 1)
    tg_gated_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmG,
                    const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmH,
                    const __grid_constant__ CUtensorMap tmGate,
                    const __grid_constant__ CUtensorMap tmUp, const __grid_constant__ GatedParams gp) {
  gated_body<1, BN, B_K, OUT_F32>(tmX, tmG, tmU, tmH, tmGate, tmUp, gp);
}

template <bool B_K, bool OUT_F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GatedCfg<2, 256>::kThreads, 1)
    tg_gated_pair_kernel(const __grid_constant__ CUtensorMap tmX,
                         const __grid_constant__ CUtensorMap tmG,
                         const __grid_constant__ CUtensorMap tmU,
                         const __grid_constant__ CUtensorMap tmH,
                         const __grid_constant__ CUtensorMap tmGate,
                         const __grid_constant__ CUtensorMap tmUp,
                         const __grid_constant__ GatedParams gp) {
  gated_body<2, 256, B_K, OUT_F32>(tmX, tmG, tmU, tmH, tmGate, tmUp, gp);
}

}  // namespace tg
