// Instantiations of the head's logits kernels whose sums are put right (PRECISE), in a unit of their own so
// that both kinds compile in parallel.
#include "tg_head_kernel.cuh"
#include "tg_internal.h"

namespace tg {

namespace {
template <bool B_K, bool STORE>
cudaError_t launch_logits(const GemmLaunch& l, const HeadParams& hp, int block_n) {
  return launch_logits_tile<B_K, STORE, true>(
      [&](auto kern, int smem) {
        const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
        if (e != cudaSuccess) return e;
        return launch_chained(kern, l.chained, dim3(static_cast<unsigned>(l.grid)), kHeadThreads, smem,
                              l.stream, l.a, l.b, l.out, hp);
      },
      l.grid, block_n);
}
}  // namespace

cudaError_t launch_head_logits_precise(const GemmLaunch& l, const HeadParams& hp, bool store,
                                       int block_n) {
  if (l.p.b_k) return store ? launch_logits<true, true>(l, hp, block_n) : launch_logits<true, false>(l, hp, block_n);
  return store ? launch_logits<false, true>(l, hp, block_n) : launch_logits<false, false>(l, hp, block_n);
}

}  // namespace tg
