// tg_internal.h — launchers shared between the C-ABI translation unit and the kernel units.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tg_gemm_kernel.cuh"
#include "tg_gemm_relu.h"

namespace tg {

struct GemmLaunch {
  CUtensorMap a, b, out;  // see tg_gemm_tc_kernel for the layouts each map describes
  GemmParams p;
  int grid;
  cudaStream_t stream;
  bool chained;  // logits and scaled kernels: the launch before it on the stream is the library's
};

// A launch that may begin while the kernel before it on the stream still runs: its blocks are made
// and set up early, and chain_wait (tg_gemm_kernel.cuh) in the kernel holds each thread until all
// of the kernel before has finished and its writes are visible.  A distillation step's eight kernels
// (128 tokens, 28672 classes of 1024) take 70 us so and 85 one after the other.
template <typename... P, typename... Q>
cudaError_t launch_chained(void (*kern)(P...), bool chained, dim3 grid, int threads, size_t smem,
                           cudaStream_t stream, const Q&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = chained ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// Shared-memory bytes and stage count of the kernel for a tile width.
int gemm_smem_bytes(int block_n);
int gemm_stages(int block_n);

// Launch tg_gemm_tc_kernel<block_n, out_f32>; returns the launch error (cudaSuccess if queued).
cudaError_t launch_gemm_bn256(const GemmLaunch& l, bool out_f32);
cudaError_t launch_gemm_bn192(const GemmLaunch& l, bool out_f32);
cudaError_t launch_gemm_bn128(const GemmLaunch& l, bool out_f32);

// CTA-pair kernel (256 x 256 tiles; l.grid must be even, l.p counts pair tiles).
cudaError_t launch_gemm_pair(const GemmLaunch& l, bool out_f32);
// The CTA-pair kernel with A read in place through row classes (float32 output only; l.a is
// unused, l.p.cls_* describe the classes).
cudaError_t launch_gemm_pair_cls(const AClassMaps& cls, const GemmLaunch& l);
// What the head's logits pass gives beside, or instead of, the logits.
struct LogitsExtra {
  float* z;                 // float32 logits, rows of ldz (a multiple of 32); NULL: not stored
  int64_t ldz;
  float2* stats;            // [M][2 ceil(N / *block_n)]: each row's softmax statistics over
  float stat_c;             // *block_n / 2 columns, of stat_c times the logits
  const long long* target;  // without z: [M], and the targets' logits [M]
  float* picked;
  int* block_n;             // out: the tiles' width
};
// Logits kernel (block_n 0: CTA pairs), X row-major, W in either layout (l.p.b_k).
cudaError_t launch_head_logits(const GemmLaunch& l, const LogitsExtra& x, int block_n);
// The CTA-pair kernel that adds A^T B to its float32 output (kModeAdd; A stored K x M).
cudaError_t launch_head_add(const GemmLaunch& l);
// The fp16-output kernels whose epilogue is the scaled sum (kModeScaled; block_n 0: CTA pairs).
// A^T B^T is not among the head's products and not a launch.
cudaError_t launch_gemm_scaled(const GemmLaunch& l, int block_n);
// Clusters of two that can be resident at once on the current device.
cudaError_t gemm_pair_max_clusters(int* out);

// Makes the runtime's context for `dev` current in the calling thread (once per thread), so that
// driver-API calls (tensor-map encoding) work from any host thread.
cudaError_t bind_thread_context(int dev);

// Records `e` as the calling thread's last CUDA error (what tg_last_cuda_error reports) and
// returns TG_ERR_CUDA, for entry points defined outside tg_api.cu.
tg_status record_cuda_error(cudaError_t e);

// Current device's SM count and error word (checks the device; sets up library state).
tg_status device_info(int* sm_count, unsigned int** err);

// Address of the device error word that kernels set when a pipeline wait runs out.
cudaError_t error_word_address(unsigned int** out);

// Stream-ordered scratch of `bytes` from the library's pool on the current device; give it back
// with cudaFreeAsync on the same stream.  TG_ERR_NO_WORKSPACE if the pool cannot supply it.
tg_status scratch_alloc(size_t bytes, cudaStream_t stream, void** out);

// cuTensorMapEncodeTiled from the driver (false if the driver does not provide it).
bool tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* fn);

// The GEMM behind every entry point, with what the head's passes need beside the public ones.
// With `logits` or out32 there are no K splits and no fp16 output (C is not used).
struct GemmExtra {
  const LogitsExtra* logits;
  const float* alpha;   // fp16 output, device float32: C = fp16(alpha (A B + addend)) (NULL: the
  const float* addend;  // plain product); addend, device float32, rows of ld32 (NULL: 0)
  float* out32;         // float32 output, rows of ld32 floats (a multiple of 32)
  int64_t ld32;
  bool add;             // add to out32 (A stored K x M, B stored K x N) instead of writing it
  bool chained;         // logits or alpha: see GemmLaunch
  bool fold;            // fp16 output: M even, C has M / 2 rows, row r the sum of rows r and r + M / 2
  int64_t max_k;        // 0, or the K columns that one split may have (without logits and out32)
  int64_t a_rows;       // 0, or the rows (>= M) that A, stored M x K and not copied, has in memory
};
tg_status gemm_extra(int ta, int tb, const void* A, const void* B, void* C, int64_t M, int64_t N,
                     int64_t K, int64_t lda, int64_t ldb, int64_t ldc, const GemmExtra& x,
                     const tg_options* opt, cudaStream_t stream);

// dst (rows x ld_dst, 16-byte aligned rows, columns up to a multiple of 8 written as zero) <- src.
cudaError_t launch_pack_rows(const void* src, int64_t ld_src, void* dst, int64_t ld_dst,
                             int64_t rows, int64_t cols, int num_sms, cudaStream_t stream);

// Deterministic split-K reduction: C = fp16(epi(sum_s W[s])) (see tg_splitk_reduce_kernel).
// p supplies the epilogue (act, bias, residual, ldr) and the shape (M, N).
cudaError_t launch_splitk_reduce(const float* ws, int64_t ldw, int64_t split_stride, int splits,
                                 void* C, int64_t ldc, const GemmParams& p, int num_sms,
                                 cudaStream_t stream);

}  // namespace tg
