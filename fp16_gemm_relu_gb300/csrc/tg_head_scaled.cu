// Instantiations of the tensor-core kernels for the head's gradients: fp16(alpha (sum + addend)).
#include "tg_internal.h"

namespace tg {

namespace {
template <typename K>
cudaError_t launch(K kern, int smem, const GemmLaunch& l) {
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, l.chained, dim3(static_cast<unsigned>(l.grid)), kThreads, smem, l.stream,
                        l.a, l.b, l.out, l.p);
}

template <int BN>
cudaError_t launch_tc(const GemmLaunch& l) {
  constexpr int smem = TileCfg<BN>::kSmemBytes;
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
  if (l.p.a_mn) return launch(tg_gemm_pair_kernel<false, true, false, kModeScaled>, smem, l);
  return l.p.b_k ? launch(tg_gemm_pair_kernel<false, false, true, kModeScaled>, smem, l)
                 : launch(tg_gemm_pair_kernel<false, false, false, kModeScaled>, smem, l);
}

}  // namespace tg
