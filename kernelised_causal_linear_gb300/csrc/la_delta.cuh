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

// Pairs of fp32 in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Eight sums over lanes of the same t = lane & 3: halves are traded so that lane
// 4 g + t ends with the sum of y[g], seven shuffles instead of 24.
__device__ __forceinline__ float sum8(const float (&y)[8], int lane)
{
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a[i] = (lane & 16 ? y[i + 4] : y[i]) + __shfl_xor_sync(0xffffffffu, lane & 16 ? y[i] : y[i + 4], 16);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        b[i] = (lane & 8 ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, lane & 8 ? a[i] : a[i + 2], 8);
    return (lane & 4 ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, lane & 4 ? b[0] : b[1], 4);
}

// From segments' ends to their starts: S_{i+1} = M_i S_i + B_i from S_0 (mcount M and B
// per head), or with rev dS_{i-1} = M_i^T dS_i + C_i from the last (B: n - 1 C per head).
cudaError_t join_segments(const DeltaArgs& a, bool rev, const float* from, const float* B, const float* M, float* start,
                          int n, int mcount);

}  // namespace delta
}  // namespace la
