"""GB300-native C = relu(A·B): fp16 A (M,K) and B (K,N) row-major, float32 accumulation in
tensor memory, fp16 C.  The computation is the matmul_relu example of the TileLang
paper-reading page (section 2).

The work runs in hand-written sm_103a kernels behind a C ABI (``include/tg_gemm_relu.h``);
this package is a thin binding over that library.  There is no CPU fallback: every entry point
raises if the compiled library is missing.
"""

from .binding import (  # noqa: F401
    TG_ACT_GELU,
    TG_ACT_GELU_TANH,
    TG_ACT_NONE,
    TG_ACT_RELU,
    TG_ACT_SILU,
    TG_EPILOGUE_NONE,
    TG_EPILOGUE_RELU,
    TG_HEAD_VOCAB_MAJOR,
    TG_HEAD_WIDTH_MAJOR,
    TgError,
    gemm_relu,
    gemm_relu_host,
    library_path,
    load_library,
    plan,
    tg_gemm_relu_f16,
    tg_gemm_relu_f16_ex,
    tg_gemm_relu_f16_host,
    tg_last_cuda_error,
    tg_release_workspace,
    tg_status_string,
)
from .clip import clip_gradients, gradient_norm  # noqa: F401
from .gated import gated_linear, gated_linear_backward  # noqa: F401
from .head import (  # noqa: F401
    linear_cross_entropy,
    linear_cross_entropy_step,
    linear_distillation,
    linear_distillation_step,
    linear_policy,
    linear_policy_step,
    linear_preference,
    linear_preference_step,
)
from .norm import layer_norm, layer_norm_backward  # noqa: F401
