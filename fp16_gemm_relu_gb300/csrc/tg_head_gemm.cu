// Instantiations of the tcgen05 kernels for the loss head: float32 logits with the rows' softmax
// statistics (kModeLogits), and the float32 sum over pieces of tokens (kModeAdd).
#include "tg_internal.h"

namespace tg {

namespace {
template <bool B_K>
cudaError_t launch_pair(const GemmLaunch& l) {
  auto kern = tg_gemm_pair_kernel<true, false, B_K, kModeLogits>;
  constexpr int smem = PairCfgFwd::kSmemBytes;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<l.grid, kThreads, smem, l.stream>>>(l.a, l.b, l.out, l.p);
  return cudaGetLastError();
}

template <int BN>
cudaError_t launch_single(const GemmLaunch& l) {
  auto kern = tg_gemm_tc_kernel<BN, true, true, kModeLogits>;
  constexpr int smem = TileCfg<BN>::kSmemBytes;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<l.grid, kThreads, smem, l.stream>>>(l.a, l.b, l.out, l.p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_head_logits(const GemmLaunch& l, int block_n) {
  switch (block_n) {
    case 0:
      if (l.grid <= 0 || (l.grid & 1)) return cudaErrorInvalidConfiguration;
      return l.p.b_k ? launch_pair<true>(l) : launch_pair<false>(l);
    case 256: return launch_single<256>(l);
    case 192: return launch_single<192>(l);
    default: return launch_single<128>(l);
  }
}

cudaError_t launch_head_add(const GemmLaunch& l) {
  if (l.grid <= 0 || (l.grid & 1)) return cudaErrorInvalidConfiguration;
  auto kern = tg_gemm_pair_kernel<true, true, false, kModeAdd>;
  constexpr int smem = PairCfgFwd::kSmemBytes;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<l.grid, kThreads, smem, l.stream>>>(l.a, l.b, l.out, l.p);
  return cudaGetLastError();
}

}  // namespace tg
