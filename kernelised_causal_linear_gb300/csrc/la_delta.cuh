// la_delta.cuh -- what the CUDA-core and the tensor-core delta-rule kernels share.
#pragma once

#include "la_internal.cuh"

namespace la {
namespace delta {

// LA_FM_L2: x / sqrt(|x|^2 + kL2Eps); a zero row stays zero.
constexpr float kL2Eps = 1e-6f;

// exp(-128) is below the smallest fp32 number: a log gate under it, -inf among
// them, is a full reset, and running sums stay finite.  NaN passes through.
__device__ __forceinline__ float clamp_gate(float g) { return g < -128.0f ? -128.0f : g; }

}  // namespace delta
}  // namespace la
