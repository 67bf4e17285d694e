// Instantiations of the tensor-core kernels whose right operand is two matrices (kModeDual), and of those
// with two outputs (kModeTwo).
#include "tg_internal.h"

namespace tg {

namespace {
template <typename K, typename... Q>
cudaError_t launch(K kern, int threads, int smem, const GemmLaunch& l, const Q&... args) {
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, l.chained, dim3(static_cast<unsigned>(l.grid)), threads, smem, l.stream,
                        args...);
}

template <typename K>
cudaError_t launch_dual(K kern, int smem, const GemmLaunch& l) {
  return launch(kern, kThreads, smem, l, l.a, l.b, l.b2, l.out, l.p);
}
template <int BN>
cudaError_t launch_two(const GemmLaunch& l) {
  using Cfg = TileCfg<BN, BN / 64>;
  return launch(tg_gemm_tc_two_kernel<BN>, Cfg::kThreadsEG, Cfg::kSmemBytes, l, l.a, l.b, l.out, l.out2, l.p,
                l.two);
}

template <bool OUT_F32>
cudaError_t launch_tile(const GemmLaunch& l, int block_n) {
  switch (block_n) {
    case 256: return launch_dual(tg_gemm_tc_dual_kernel<256, OUT_F32>, TileCfg<256>::kSmemBytes, l);
    case 192: return launch_dual(tg_gemm_tc_dual_kernel<192, OUT_F32>, TileCfg<192>::kSmemBytes, l);
    case 128: return launch_dual(tg_gemm_tc_dual_kernel<128, OUT_F32>, TileCfg<128>::kSmemBytes, l);
    default: break;
  }
  if (l.grid <= 0 || (l.grid & 1)) return cudaErrorInvalidConfiguration;
  return l.p.b_k ? launch_dual(tg_gemm_pair_dual_kernel<OUT_F32, true>, PairCfgFwd::kSmemBytes, l)
                 : launch_dual(tg_gemm_pair_dual_kernel<OUT_F32, false>, PairCfgFwd::kSmemBytes, l);
}
}  // namespace

cudaError_t launch_gemm_dual(const GemmLaunch& l, bool out_f32, int block_n) {
  return out_f32 ? launch_tile<true>(l, block_n) : launch_tile<false>(l, block_n);
}

cudaError_t launch_gemm_two(const GemmLaunch& l, int block_n) {
  if (block_n) return block_n == 256 ? launch_two<256>(l) : launch_two<128>(l);
  if (l.grid <= 0 || (l.grid & 1)) return cudaErrorInvalidConfiguration;
  return launch(tg_gemm_pair_two_kernel<2>, 64 + 2 * 32 * kEpiWarps, PairCfgFwd::kSmemBytes, l, l.a, l.b,
                l.out, l.out2, l.p, l.two);
}

namespace {
template <int BN>
cudaError_t launch_beside(const GemmLaunch& x, const GemmLaunch& w) {
  using W = TileCfg<256, 4>;
  constexpr int smem = W::kSmemBytes > TileCfg<BN>::kSmemBytes ? W::kSmemBytes : TileCfg<BN>::kSmemBytes;
  const BesideMaps m{x.a, x.b, x.b2, x.out, w.a, w.b, w.out, w.out2};
  GemmLaunch l = w;
  l.grid = x.grid + w.grid;
  return launch(tg_gemm_beside_kernel<BN>, W::kThreadsEG, smem, l, m, x.p, w.p, w.two, x.grid);
}
}  // namespace

cudaError_t launch_gemm_beside(const GemmLaunch& x, int block_n, const GemmLaunch& w) {
  return block_n == 256 ? launch_beside<256>(x, w) : launch_beside<128>(x, w);
}

}  // namespace tg
