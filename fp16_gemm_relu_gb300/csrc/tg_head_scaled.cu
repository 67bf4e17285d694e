// Instantiations of the tensor-core kernels for the head's gradients: fp16(alpha (sum + addend)).
#include "tg_internal.h"

namespace tg {

namespace {
template <typename K>
cudaError_t launch(K kern, int smem, const GemmLaunch& l, int threads = kThreads) {
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, l.chained, dim3(static_cast<unsigned>(l.grid)), threads, smem, l.stream,
                        l.a, l.b, l.out, l.p);
}

// A^T B is dW.  Up to two k-blocks, 128 tokens, a tile is all epilogue: the kernel with more epilogue warps.  From
// four on the one with more stages (28672 x 1024 from 256 tokens 20 against 23 us).
template <int BN>
cudaError_t launch_tc(const GemmLaunch& l) {
  constexpr int smem = TileCfg<BN>::kSmemBytes;
  using Wide = TileCfg<BN, BN / 64>;
  if (l.p.a_mn && (l.rows || l.p.num_kb <= 2))
    return launch(tg_gemm_tc_scaled_kernel<BN>, Wide::kSmemBytes, l, Wide::kThreadsEG);
  return l.p.a_mn || l.p.b_k ? launch(tg_gemm_tc_kernel<BN, false, true, kModeScaled>, smem, l)
                             : launch(tg_gemm_tc_kernel<BN, false, false, kModeScaled>, smem, l);
}
}  // namespace

cudaError_t launch_gemm_scaled(const GemmLaunch& l, int block_n) {
  if (l.p.a_mn && l.p.b_k) return cudaErrorInvalidConfiguration;
  switch (block_n) {
    case 256: return launch_tc<256>(l);
    case 192: return launch_tc<192>(l);
    case 128: return launch_tc<128>(l);
    default: break;
  }
  if (l.grid <= 0 || (l.grid & 1)) return cudaErrorInvalidConfiguration;
  constexpr int smem = PairCfgFwd::kSmemBytes;
  if (l.rows) return launch(tg_gemm_pair_scaled_kernel<2>, smem, l, 64 + 2 * 32 * kEpiWarps);
  if (l.p.a_mn) return launch(tg_gemm_pair_kernel<false, true, false, kModeScaled>, smem, l);
  return l.p.b_k ? launch(tg_gemm_pair_kernel<false, false, true, kModeScaled>, smem, l)
                 : launch(tg_gemm_pair_kernel<false, false, false, kModeScaled>, smem, l);
}

}  // namespace tg
