// tg_gated_kernel.cuh — the activations of the gated product and their derivatives.
#pragma once

#include "tg_gemm_kernel.cuh"

namespace tg {

enum : int { kActSilu = 4 };

// 1 / (1 + e^-x): 0 and 1 at the infinities.
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// The activation of a gate, in float32.  silu(x) = x / (1 + e^-x) (Elfwing et al., 2018); the others
// are the fused epilogue's.
__device__ __forceinline__ float gated_activation(float x, int act) {
  return act == kActSilu ? x * logistic(x) : activation(x, act);
}

// Its derivative.  Where the derivative is 0 or 1 to float32's precision it is taken as that, so that
// an infinite gate does not become infinity times 0; a NaN stays one (but in relu, as in its value).
__device__ __forceinline__ float gated_slope(float x, int act) {
  switch (act) {
    case kActRelu: return x > 0.0f ? 1.0f : 0.0f;
    case kActGelu: {
      if (fabsf(x) > 16.0f) return x > 0.0f ? 1.0f : 0.0f;
      return 0.5f * (1.0f + erff(x * 0.70710678118654752f)) +
             x * 0.39894228040143268f * __expf(-0.5f * x * x);
    }
    case kActGeluTanh: {
      if (fabsf(x) > 16.0f) return x > 0.0f ? 1.0f : 0.0f;
      const float c = 0.79788456080286536f, t = tanhf(c * (x + 0.044715f * x * x * x));
      return 0.5f * (1.0f + t) + 0.5f * x * (1.0f - t * t) * c * (1.0f + 0.134145f * x * x);
    }
    case kActSilu: {
      if (fabsf(x) > 100.0f) return x > 0.0f ? 1.0f : 0.0f;
      const float s = logistic(x);
      return s * (1.0f + x * (1.0f - s));
    }
    default: return 1.0f;
  }
}

}  // namespace tg
