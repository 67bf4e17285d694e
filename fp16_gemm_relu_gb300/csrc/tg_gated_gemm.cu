// Instantiations and launches of the gated product's kernels.
#include "tg_internal.h"

namespace tg {

namespace {
template <typename K>
cudaError_t launch(K kern, int threads, int smem, const GatedLaunch& l) {
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, l.chained, dim3(static_cast<unsigned>(l.grid)), threads, smem, l.stream,
                        l.x, l.g, l.u, l.h, l.gate, l.up, l.p);
}

template <bool B_K, bool OUT_F32>
cudaError_t launch_tile(const GatedLaunch& l) {
  switch (l.block_n) {
    case 0:
      if (l.grid <= 0 || (l.grid & 1)) return cudaErrorInvalidConfiguration;
      return launch(tg_gated_pair_kernel<B_K, OUT_F32>, GatedCfg<2, 256>::kThreads,
                    GatedCfg<2, 256>::kSmemBytes, l);
    case 256:
      return launch(tg_gated_kernel<256, B_K, OUT_F32>, GatedCfg<1, 256>::kThreads,
                    GatedCfg<1, 256>::kSmemBytes, l);
    default:
      return launch(tg_gated_kernel<128, B_K, OUT_F32>, GatedCfg<1, 128>::kThreads,
                    GatedCfg<1, 128>::kSmemBytes, l);
  }
}
}  // namespace

cudaError_t launch_gated(const GatedLaunch& l) {
  if (l.p.g.b_k) return l.out_f32 ? launch_tile<true, true>(l) : launch_tile<true, false>(l);
  return l.out_f32 ? launch_tile<false, true>(l) : launch_tile<false, false>(l);
}

}  // namespace tg
