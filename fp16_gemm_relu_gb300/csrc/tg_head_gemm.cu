// Instantiations of the head's tensor-core kernels: logits with the rows' softmax statistics, and
// the float32 sum of dW over pieces of tokens (kModeAdd).
#include "tg_head_kernel.cuh"
#include "tg_internal.h"

namespace tg {

namespace {
template <typename K, typename P>
cudaError_t launch(K kern, int threads, int smem, const GemmLaunch& l, const P& p) {
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, l.chained, dim3(static_cast<unsigned>(l.grid)), threads, smem, l.stream,
                        l.a, l.b, l.out, p);
}

template <bool B_K, bool STORE>
cudaError_t launch_logits(const GemmLaunch& l, const HeadParams& hp, int block_n) {
  return launch_logits_tile<B_K, STORE, false>(
      [&](auto kern, int smem) { return launch(kern, kHeadThreads, smem, l, hp); }, l.grid, block_n);
}
}  // namespace

cudaError_t launch_head_logits(const GemmLaunch& l, const LogitsExtra& x, int block_n) {
  HeadParams hp;
  hp.g = l.p;
  hp.stats = x.stats;
  hp.stat_c = x.stat_c;
  hp.target = x.target;
  hp.picked = x.picked;
  hp.rotate = l.p.tiles_m == 1 ? 1 : 0;
  hp.spare = static_cast<int>((int64_t(l.p.num_kb) * kBK - x.width) / kUmmaK);
  if (x.precise) return launch_head_logits_precise(l, hp, x.z != nullptr, block_n);
  if (l.p.b_k)
    return x.z ? launch_logits<true, true>(l, hp, block_n) : launch_logits<true, false>(l, hp, block_n);
  return x.z ? launch_logits<false, true>(l, hp, block_n) : launch_logits<false, false>(l, hp, block_n);
}

cudaError_t launch_head_add(const GemmLaunch& l) {
  if (l.grid <= 0 || (l.grid & 1)) return cudaErrorInvalidConfiguration;
  auto kern = tg_gemm_pair_kernel<true, true, false, kModeAdd>;
  constexpr int smem = PairCfgFwd::kSmemBytes;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  kern<<<l.grid, kThreads, smem, l.stream>>>(l.a, l.b, l.out, l.p);
  return cudaGetLastError();
}

}  // namespace tg
