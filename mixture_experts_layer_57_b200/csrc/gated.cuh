// Gate activations of the gated expert FFN and their derivatives.
#pragma once

#include "common.cuh"

namespace moe {

// a = act(z), da = act'(z).
//   SiLU: act = z s, act' = s (1 + z (1 - s)) with s = 1 / (1 + e^-z)
//   GeLU (erf form): act = z Phi(z), act' = Phi(z) + z phi(z)
// e^-z overflowing to infinity gives s = 0, the limit. FAST uses the approximate exponential and
// division (a few units in the last place of fp32), far below the bf16 rounding that follows.
template <bool FAST = false>
__device__ __forceinline__ void gate_act(float z, int act, float& a, float& da) {
  if (act == MOE_GATE_SILU) {
    const float s = FAST ? __fdividef(1.0f, 1.0f + __expf(-z)) : 1.0f / (1.0f + expf(-z));
    a = z * s;
    da = s * (1.0f + z * (1.0f - s));
  } else {
    const float cdf = 0.5f * (1.0f + erff(z * 0.70710678118654752440f));
    a = z * cdf;
    da = cdf + z * 0.39894228040143267794f * (FAST ? __expf(-0.5f * z * z) : expf(-0.5f * z * z));
  }
}

// 3D tiled bulk tensor copy global -> shared, completion counted on `bar` in bytes.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int32_t x, int32_t y,
                                            int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

}  // namespace moe
