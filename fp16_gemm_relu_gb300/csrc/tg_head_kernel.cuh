// tg_head_kernel.cuh — the head's logits Z = X W^T (float32) with each row's softmax statistics, on
// the tensor cores of sm_103a.
//
// The roles are those of tg_gemm_kernel.cuh (TMA producer, tcgen05 issuer, epilogue; one CTA a tile
// of 128 x BN, or a pair of CTAs a tile of 256 x 256).  Two things differ:
//
//  - A tile's sum over the width is cut into segments of kSegK k-blocks (1024 columns).  The tensor
//    core adds each instruction's 16 products to the float32 accumulator by cutting off, not by
//    rounding, so a sum's error grows with its length and always towards zero: 8192 columns in one
//    piece put 4.5e-6 on a loss, in segments of 1024 columns 4e-7, which is also the error at 1024 or
//    2048 columns in all (float32 sums by other means are off by about 1e-7).  So each segment starts
//    from zero in one of the two TMEM accumulators, and the epilogue warps add it to running sums
//    in registers, rounding to nearest, while the next segment runs in the other.  Segments of 512
//    cost 1-3% more time than of 1024, those of 2048 save nothing further.
//    PRECISE, for losses of differences of log probabilities, where what every token's log probability is
//    off in one direction adds up over a sequence: segments of 768 columns, and what the cutting off takes from a
//    segment's sum v on average is put back as it is added.  Each of n instructions cuts half a unit of the partial
//    sum's last place (16 products of one sign: up to 2.5 units).  Of sums that are large beside their row's, whose partial sums go there straight, that is up to
//    0.3 n 2^-24, of others 0.27 n, whose partial sums stay below v or change sign; measured over normal logits of
//    spread 1 to 4, n = 5 to 48, it is (0.266 n + 0.38 + n min(0.0036 (v / s)^2, 0.035)) 2^-24 of v within 1% of n, s being the
//    row's root mean square (of a warp's first 32 columns).  An instruction past the last column cuts nothing.
//    A log probability is then off by less than 5e-8 on average (30666 classes of 768 1e-8; with 0.276 n for all 1.4e-7, with
//    nothing put back in segments of 1024 4.4e-6), root mean square 1.1e-6 (2.6e-6 in segments of 1024).  That is for
//    entries of about one size and logits up to 8: normal, uniform, one-sided and quantised ones within 1e-7, targets whose
//    weights point along x within 3e-7; logits up to 25 lean by 0.2 to 1.5e-6 (with nothing put back 14 to 26e-6).  What is
//    put back depends on n and v alone, so it is wrong where the cut is another: with eight columns 30 times the others it
//    takes the lean from 18 to 38e-6 down to 5 to 17e-6, with 5% of x not zero from 1.8e-6 to -1.9e-6, and sums of which nothing is cut (one-hot rows, small integers) come
//    out up to (0.301 n + 0.38) 2^-24, 8.9e-7, of themselves too large.
//    4096 tokens, 65537 classes of 2048: the whole step 2280 us, 2230 with 0.276 n for all; segments of 512 would cost 35 more.
//  - The running sums take 128 registers a thread, so there are eight epilogue warps, each with 32
//    rows and half of the tile's columns.  With the whole row segment in registers they take its
//    maximum and sum of exponentials, and then store it, or only look up the rows' targets.
//
// Bound by the tensor cores: 4096 tokens, 65537 classes of 2048 alone 605 us, 1817 TFLOP/s, 0.94 of
// the rate measured with large bf16 products, 674 with the logits stored; in a long run the power
// limit lowers the clock (695 us).  One token, 28672 classes of 8192: bound by HBM, 78 us, 6.0 TB/s.
#pragma once

#include "tg_gemm_kernel.cuh"

namespace tg {

constexpr int kSegK = 16;            // k-blocks of a segment
constexpr int kSegKPrecise = 12;     // those of PRECISE
constexpr int kHeadEpiWarps = 8;
constexpr int kHeadThreads = 64 + 32 * kHeadEpiWarps;

// CG CTAs a tile; BN columns.
template <int CG, int BN>
struct HeadCfg {
  static_assert(CG == 1 || (CG == 2 && BN == 256), "pairs have 256 x 256 tiles");
  static constexpr int kKB = CG;                          // k-blocks of a stage
  static constexpr int kBRows = BN / CG;                  // W rows (or columns) of this CTA
  static constexpr int kAStage = kKB * kBM * kBK * 2;
  static constexpr int kBStage = kKB * kBK * kBRows * 2;
  static constexpr int kStageBytes = kAStage + kBStage;
  static constexpr int kStagingBytes = kHeadEpiWarps * kStagingBuf;
  static constexpr int kStagesFit = (kSmemLimit - kSmemReserve - kStagingBytes) / kStageBytes;
  static constexpr int kStages = kStagesFit > 8 ? 8 : kStagesFit;
  static constexpr int kAccStride = BN <= 128 ? 128 : 256;
  static constexpr int kTmemCols = 2 * kAccStride;
  static constexpr int kSmemBytes = kSmemReserve + kStages * kStageBytes + kStagingBytes;
  static_assert(kSmemBytes <= kSmemLimit, "shared memory budget exceeded");
};

struct HeadParams {
  GemmParams g;             // tiles, k-blocks, M and N, time limit and error word
  float2* stats;            // [M][2 tiles_n]: of BN / 2 columns each
  float stat_c;             // scale of the statistics' logits, log2(e) included
  const long long* target;  // !STORE, or NULL: [M], the column whose logit goes to picked
  float* picked;
  int rotate;               // 1: tiles start at different k-blocks (CG == 1)
  int spare;                // instructions of the last k-block that add nothing
};

// The k-block that a tile begins with.
template <int CG>
__device__ __forceinline__ int first_kb(const HeadParams& hp, int u) {
  return CG == 1 && hp.rotate ? static_cast<int>(static_cast<unsigned>(u) * 7u % static_cast<unsigned>(hp.g.num_kb)) : 0;
}

// Softmax statistics of NC columns of one row (cnt: how many of them the matrix has): m = the largest
// of the scaled sums, s = the sum of 2^(scaled sum - m), with log2(e) in the scale c.  A row's
// statistics over several tiles combine as 2^(m - M) s.  m = -inf (every sum -inf, or no column)
// comes with s = 0, or NaN if there is a NaN among the sums.
template <int NC>
__device__ __forceinline__ float row_max(const float (&v)[NC], int cnt) {
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  if (cnt >= NC) {
#pragma unroll
    for (int i = 0; i < NC; ++i) top[i & 3] = fmaxf(top[i & 3], v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (i < cnt) top[i & 3] = fmaxf(top[i & 3], v[i]);
  }
  return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
}
// The part of s of 32 columns from `v` on.
__device__ __forceinline__ float row_sum32(const float* v, int cnt, float c, float m) {
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (m == -INFINITY) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < cnt && v[i] != v[i]) s[0] = v[i];
  } else if (cnt >= 32) {
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i & 3] += exp2f(fmaf(v[i], c, -m));
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < cnt) s[i & 3] += exp2f(fmaf(v[i], c, -m));
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// v[at mod 16] by selects: an index at run time would put the array into memory.
__device__ __forceinline__ float pick16(const float* v, int at) {
  float a[8], b[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = (at & 8) ? v[i + 8] : v[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = (at & 4) ? a[i + 4] : a[i];
  const float c0 = (at & 2) ? b[2] : b[0], c1 = (at & 2) ? b[3] : b[1];
  return (at & 1) ? c1 : c0;
}

// tmX: fp16 X, dims {D, T}, box {64, 128};  tmW: fp16 W, B_K (stored V x D): dims {D, V}, box
// {64, BN / CG};  else (D x V): dims {V, D}, box {64, 64 CG};  tmZ (STORE): float32 logits, dims
// {V, T, 1}, box {32, 32, 1}.  All with 128B swizzle.
template <int CG, int BN, bool B_K, bool STORE, bool PRECISE>
__device__ __forceinline__ void head_logits_body(const CUtensorMap& tmX, const CUtensorMap& tmW,
                                                 const CUtensorMap& tmZ, const HeadParams& hp) {
  using Cfg = HeadCfg<CG, BN>;
  constexpr int S = Cfg::kStages, KB = Cfg::kKB, SEG = PRECISE ? kSegKPrecise : kSegK;
  constexpr int kAtom = kBM * kBK * 2;             // 128 rows x 64 k, K-major
  constexpr int kBAtom = Cfg::kBRows * kBK * 2;    // this CTA's rows of W x 64 k, K-major
  constexpr int kMNBox = KB * kBK * 64 * 2;        // 64 columns x KB 64 k, MN-major
  const GemmParams& p = hp.g;

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
      mbar_init(smem_u32(&tempty[b]), CG * kHeadEpiWarps);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmW);
    if (STORE) prefetch_tmap(&tmZ);
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
      for (int u = first; u < p.units; u += step) {
        const Unit w = unit_of(p, u);
        const int xrow = (w.m_blk * CG + static_cast<int>(rank)) * kBM;
        const int wrow = w.n_blk * BN + static_cast<int>(rank) * Cfg::kBRows;
        // Where W's rows stream from memory once (few tokens), tiles that all walk the same
        // columns at the same time meet in the same memory channels: each starts elsewhere.
        int at = first_kb<CG>(hp, u);
        for (int kb = 0; kb < p.num_kb; kb += KB) {
          if (!wait_phase(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, p, kRoleProducer))
            goto producer_done;
          if ((p.debug_flags & kDebugDropFirstStage) && first == 0 && rank == 0 && !dropped) {
            dropped = true;  // injected fault: this stage is never filled
          } else {
            const uint32_t fb_local = smem_u32(&full[stage]);
            if (rank == 0) {
              mbar_arrive_expect_tx(fb_local, CG * Cfg::kStageBytes);
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
            // all k-blocks of a stage load (past D as zeros), so its byte count is fixed
#pragma unroll
            for (int h = 0; h < KB; ++h) load(a_dst + h * kAtom, &tmX, (at + h) * kBK, xrow);
            if constexpr (B_K) {
#pragma unroll
              for (int h = 0; h < KB; ++h) load(b_dst + h * kBAtom, &tmW, (at + h) * kBK, wrow);
            } else {
#pragma unroll
              for (int j = 0; j < Cfg::kBRows / 64; ++j)
                load(b_dst + j * kMNBox, &tmW, wrow + j * 64, at * kBK);
            }
          }
          at += KB;
          if (CG == 1 && at == p.num_kb) at = 0;
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
      bool ok = true;
      for (int u = first; ok && u < p.units; u += step) {
        for (int k0 = 0; ok && k0 < p.num_kb; k0 += SEG, ++t) {
          const int buf = t & 1;
          const uint32_t use = static_cast<uint32_t>(t >> 1) & 1u;
          if (!wait_phase(smem_u32(&tempty[buf]), use ^ 1u, abort_flag, p, kRoleMma)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * Cfg::kAccStride);
          const int k1 = min(k0 + SEG, p.num_kb);
          for (int kb = k0; kb < k1; kb += KB) {
            if (!wait_phase(smem_u32(&full[stage]), phase, abort_flag, p, kRoleMma)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_addr = smem_u32(sA + stage * Cfg::kAStage);
            const uint32_t b_addr = smem_u32(sB + stage * Cfg::kBStage);
            const uint64_t ad = desc_kmajor(a_addr);
            const uint64_t bd = B_K ? desc_kmajor(b_addr) : sw128_desc(b_addr, kMNBox, 1024);
            const int nk = (k1 - kb >= KB ? KB : k1 - kb) * (kBK / kUmmaK);
#pragma unroll
            for (int k = 0; k < KB * (kBK / kUmmaK); ++k) {
              const uint64_t a_off = static_cast<uint64_t>((k >> 2) * (kAtom >> 4) + 2 * (k & 3));
              const uint64_t b_off =
                  B_K ? static_cast<uint64_t>((k >> 2) * (kBAtom >> 4) + 2 * (k & 3))
                      : static_cast<uint64_t>(128 * k);
              if (k < nk) {
                const uint32_t acc = (kb > k0 || k > 0) ? 1u : 0u;
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
    constexpr int NC = BN / 2;          // columns of a warp
    const int q = warp & 3;             // TMEM lane quarter this warp may access
    const int ew = warp - 2, half = ew >> 2;
    uint8_t* stg = sStg + ew * kStagingBuf;
    // the logits are read again only after all of them are written: they need not push the operands,
    // which other tiles read, out of L2
    const uint64_t policy = evict_first_policy();
    int t = 0;
    bool ok = true;
    for (int u = first; ok && u < p.units; u += step) {
      const Unit w = unit_of(p, u);
      const int row0 = (w.m_blk * CG + static_cast<int>(rank)) * kBM + q * 32;
      const int col0 = w.n_blk * BN + half * NC;
      const bool live = row0 < p.M;     // a warp without rows only hands the accumulators back
      const int last_kb = p.num_kb - 1 - first_kb<CG>(hp, u);  // when the last k-block's turn is
      float acc[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) acc[i] = 0.0f;
      for (int k0 = 0; k0 < p.num_kb; k0 += SEG, ++t) {
        const int buf = t & 1;
        const uint32_t use = static_cast<uint32_t>(t >> 1) & 1u;
        int got = 0;
        if (lane == 0) got = wait_phase(smem_u32(&tfull[buf]), use, abort_flag, p, kRoleEpilogue);
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (live) {
          const uint32_t tl = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                              static_cast<uint32_t>(buf * Cfg::kAccStride + half * NC);
          // what the segment's instructions cut off, of its sum (PRECISE); 1 + back would be rounded to 2^-23
          const bool tail = last_kb >= k0 && last_kb < k0 + SEG;
          const int n = min(SEG, p.num_kb - k0) * (kBK / kUmmaK) - (tail ? hp.spare : 0);
          const float unit = 0x1p-24f * n, back = fmaf(0.266f, unit, 0.38f * 0x1p-24f), top = back + 0.035f * unit;
          float squares = 1e-30f, slope = 0.0f;
#pragma unroll
          for (int c = 0; c < NC / 16; ++c) {  // 16 at a time: NC registers are taken already
            uint32_t r[16];
            tmem_ld_x16(tl + c * 16, r);
            tmem_wait_ld(r);
            if constexpr (PRECISE)
              if (c < 2) {  // the spread of the row's sums, from its first columns
#pragma unroll
                for (int i = 0; i < 16; ++i) squares = fmaf(__uint_as_float(r[i]), __uint_as_float(r[i]), squares);
                slope = __fdividef(0.0036f * unit * (16 * c + 16), squares);
              }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float v = __uint_as_float(r[i]);
              if constexpr (PRECISE)
                acc[c * 16 + i] = fmaf(v, fminf(fmaf(v * v, slope, back), top), acc[c * 16 + i] + v);
              else
                acc[c * 16 + i] += v;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2)
            mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[buf]), 0));
          else
            mbar_arrive(smem_u32(&tempty[buf]));
        }
      }
      if (!ok || !live) continue;
      const int row = row0 + lane;
      const int cnt = p.N - col0;
      const float m = row_max<NC>(acc, cnt) * hp.stat_c;
      float sum = 0.0f;
#pragma unroll
      for (int c = 0; c < NC / 32; ++c) {
        if constexpr (STORE) {
          if (c * 32 < cnt) {  // this chunk's exponentials run while the store reads its buffer
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 v = make_float4(acc[c * 32 + 4 * j], acc[c * 32 + 4 * j + 1],
                                           acc[c * 32 + 4 * j + 2], acc[c * 32 + 4 * j + 3]);
              *reinterpret_cast<float4*>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) = v;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d_hint(&tmZ, smem_u32(stg), col0 + c * 32, row0, 0, policy);
              bulk_commit();
            }
          }
        }
        sum += row_sum32(acc + c * 32, cnt - c * 32, hp.stat_c, m);
      }
      if (row < p.M)
        hp.stats[static_cast<long long>(row) * (2 * p.tiles_n) + 2 * w.n_blk + half] =
            make_float2(m, sum);
      if constexpr (!STORE) {
        const long long y = hp.target && row < p.M ? hp.target[row] - col0 : -1;
        const bool mine = y >= 0 && y < NC && y < cnt;
        if (__any_sync(0xffffffffu, mine)) {
          const int at = static_cast<int>(y);
          float z = 0.0f;
#pragma unroll
          for (int c = 0; c < NC / 16; ++c) {
            const float v = pick16(acc + 16 * c, at);
            if ((at >> 4) == c) z = v;
          }
          if (mine) hp.picked[row] = z;
        }
      }
    }
    if (STORE && lane == 0) bulk_wait_all<0>();
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

template <int BN, bool B_K, bool STORE, bool PRECISE>
__global__ void __launch_bounds__(kHeadThreads, 1)
    tg_head_logits_kernel(const __grid_constant__ CUtensorMap tmX,
                          const __grid_constant__ CUtensorMap tmW,
                          const __grid_constant__ CUtensorMap tmZ,
                          const __grid_constant__ HeadParams hp) {
  head_logits_body<1, BN, B_K, STORE, PRECISE>(tmX, tmW, tmZ, hp);
}

template <bool B_K, bool STORE, bool PRECISE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kHeadThreads, 1)
    tg_head_logits_pair_kernel(const __grid_constant__ CUtensorMap tmX,
                               const __grid_constant__ CUtensorMap tmW,
                               const __grid_constant__ CUtensorMap tmZ,
                               const __grid_constant__ HeadParams hp) {
  head_logits_body<2, 256, B_K, STORE, PRECISE>(tmX, tmW, tmZ, hp);
}

// Launch of a tile width (block_n 0: CTA pairs).
template <bool B_K, bool STORE, bool PRECISE, typename L>
cudaError_t launch_logits_tile(L launch, int grid, int block_n) {
  switch (block_n) {
    case 0:
      if (grid <= 0 || (grid & 1)) return cudaErrorInvalidConfiguration;
      return launch(tg_head_logits_pair_kernel<B_K, STORE, PRECISE>, HeadCfg<2, 256>::kSmemBytes);
    case 256: return launch(tg_head_logits_kernel<256, B_K, STORE, PRECISE>, HeadCfg<1, 256>::kSmemBytes);
    case 192: return launch(tg_head_logits_kernel<192, B_K, STORE, PRECISE>, HeadCfg<1, 192>::kSmemBytes);
    default: return launch(tg_head_logits_kernel<128, B_K, STORE, PRECISE>, HeadCfg<1, 128>::kSmemBytes);
  }
}

}  // namespace tg
