// la_rows.cuh -- what the convolution and the selective scan share: vectors of
// channels as they lie in memory, activations, strided token rows.
#pragma once

#include "la_internal.cuh"

namespace la {
namespace rows {

// V neighbouring channels as they lie in memory.
template <typename T, int V> struct Raw;
template <> struct Raw<float, 4> {
    float4 w;
};
template <> struct Raw<__nv_bfloat16, 4> {
    uint2 w;
};
template <> struct Raw<float, 2> {
    float2 w;
};
template <> struct Raw<__nv_bfloat16, 2> {
    uint32_t w;
};
template <> struct Raw<float, 1> {
    float w;
};
template <> struct Raw<__nv_bfloat16, 1> {
    __nv_bfloat16 w;
};

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> fetch(const T* p)
{
    Raw<T, V> r;
    r.w = __ldcs(reinterpret_cast<const decltype(r.w)*>(p));
    return r;
}

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> none()
{
    Raw<T, V> r;
    memset(&r, 0, sizeof r);
    return r;
}

template <int V>
struct Vec {
    float f[V];
};

__device__ __forceinline__ Vec<4> wide(const Raw<float, 4>& x) { return {{x.w.x, x.w.y, x.w.z, x.w.w}}; }
__device__ __forceinline__ Vec<1> wide(const Raw<float, 1>& x) { return {{x.w}}; }
__device__ __forceinline__ Vec<1> wide(const Raw<__nv_bfloat16, 1>& x) { return {{__bfloat162float(x.w)}}; }
__device__ __forceinline__ Vec<4> wide(const Raw<__nv_bfloat16, 4>& x)
{
    return {{__uint_as_float(x.w.x << 16), __uint_as_float(x.w.x & 0xffff0000u), __uint_as_float(x.w.y << 16),
             __uint_as_float(x.w.y & 0xffff0000u)}};
}

__device__ __forceinline__ Vec<2> wide(const Raw<float, 2>& x) { return {{x.w.x, x.w.y}}; }
__device__ __forceinline__ Vec<2> wide(const Raw<__nv_bfloat16, 2>& x)
{
    return {{__uint_as_float(x.w << 16), __uint_as_float(x.w & 0xffff0000u)}};
}

__device__ __forceinline__ void store(float* p, const Vec<4>& r)
{
    *reinterpret_cast<float4*>(p) = make_float4(r.f[0], r.f[1], r.f[2], r.f[3]);
}
__device__ __forceinline__ void store(float* p, const Vec<2>& r)
{
    *reinterpret_cast<float2*>(p) = make_float2(r.f[0], r.f[1]);
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const Vec<2>& r)
{
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(r.f[0], r.f[1]);
}
__device__ __forceinline__ void store(float* p, const Vec<1>& r) { *p = r.f[0]; }
__device__ __forceinline__ void store(__nv_bfloat16* p, const Vec<1>& r) { *p = __float2bfloat16_rn(r.f[0]); }
__device__ __forceinline__ void store(__nv_bfloat16* p, const Vec<4>& r)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(r.f[0], r.f[1]), b = __floats2bfloat162_rn(r.f[2], r.f[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Pairs of fp32 in one instruction, and the same for one.
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
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

constexpr float kLog2e = 1.4426950408889634f;

// 2^x and 1/x in hardware, a few 2^-24 off; what is under the smallest normal number is zero.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The larger one, and a NaN where either is one (fmaxf takes the other).
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// sigmoid(u) = 1 / (1 + e), e = exp(-u), and 1 - sigmoid(u) = e sigmoid(u), which keeps its
// digits where the difference would not.  u is held above -87, where e is still finite: what
// lies under it has results under 1e-35.  A NaN stays one.
struct Sigmoid {
    float2 u, s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid(float2 u)
{
    u = make_float2(max_nan(u.x, -87.0f), max_nan(u.y, -87.0f));
    const float2 t = mul2(u, both(-kLog2e)), e = make_float2(ex2(t.x), ex2(t.y)), q = add2(e, both(1.0f));
    const float2 s = make_float2(rcp(q.x), rcp(q.y));
    return {u, s, mul2(e, s)};
}

// act(u), and act'(u)
template <int ACT>
__device__ __forceinline__ float2 value(float2 u)
{
    if (ACT == LA_ACT_NONE)
        return u;
    // exp(-u) may be infinite here: its quotient is zero
    const float2 t = mul2(u, both(-kLog2e)), q = add2(make_float2(ex2(t.x), ex2(t.y)), both(1.0f));
    const float2 s = make_float2(rcp(q.x), rcp(q.y));
    return ACT == LA_ACT_SIGMOID ? s : mul2(u, s);
}
template <int ACT>
__device__ __forceinline__ float2 slope(float2 u)
{
    if (ACT == LA_ACT_NONE)
        return both(1.0f);
    const Sigmoid g = sigmoid(u);
    return mul2(g.s, ACT == LA_ACT_SIGMOID ? g.rest : fma2(g.u, g.rest, both(1.0f)));
}

// Tokens of row b: lengths clamped to 0 .. N, or N.
__device__ __forceinline__ int64_t row_length(const int* lengths, int64_t b, int64_t N)
{
    if (!lengths)
        return N;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n < N ? n : N;
}

// Whether pointer and strides (in elements of es bytes) put every row on a boundary of
// `bytes` (a power of two).
inline bool rows_on(const void* p, int64_t batch, int64_t token, int es, unsigned bytes)
{
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(batch * es) | (uintptr_t)(token * es)) & (bytes - 1)) == 0;
}

}  // namespace rows
}  // namespace la
