// la_rows.cuh -- what the convolution and the selective scan share: vectors of
// channels as they lie in memory, activations, strided token rows.
#pragma once

#include "la_internal.cuh"

namespace la {
namespace rows {

// V neighbouring channels: 16 bytes where every row starts on a 16-byte boundary,
// else one element.
template <typename T, int V> struct Raw;
template <> struct Raw<float, 4> {
    float4 w;
};
template <> struct Raw<__nv_bfloat16, 8> {
    uint4 w;
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
    r.w = __ldg(reinterpret_cast<const decltype(r.w)*>(p));
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
__device__ __forceinline__ Vec<8> wide(const Raw<__nv_bfloat16, 8>& x)
{
    Vec<8> r;
    const uint32_t u[4] = {x.w.x, x.w.y, x.w.z, x.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.f[2 * i] = __uint_as_float(u[i] << 16);
        r.f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
    return r;
}

__device__ __forceinline__ void store(float* p, const Vec<4>& r)
{
    *reinterpret_cast<float4*>(p) = make_float4(r.f[0], r.f[1], r.f[2], r.f[3]);
}
__device__ __forceinline__ void store(float* p, const Vec<1>& r) { *p = r.f[0]; }
__device__ __forceinline__ void store(__nv_bfloat16* p, const Vec<1>& r) { *p = __float2bfloat16_rn(r.f[0]); }
__device__ __forceinline__ void store(__nv_bfloat16* p, const Vec<8>& r)
{
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(r.f[2 * i], r.f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// sigmoid(g) and its slope from e = exp(-|g|), so that neither 1 - s nor the
// exponential of a large number is formed.
__device__ __forceinline__ float2 sigmoid_slope(float g)
{
    const float e = __expf(-fabsf(g)), r = __fdividef(1.0f, 1.0f + e);
    return make_float2(g >= 0.0f ? r : e * r, e * r * r);
}

// act(u) and act'(u)
__device__ __forceinline__ float2 activate(float u, int act)
{
    if (act == LA_ACT_NONE)
        return make_float2(u, 1.0f);
    const float2 s = sigmoid_slope(u);
    return act == LA_ACT_SIGMOID ? s : make_float2(u * s.x, fmaf(u, s.y, s.x));
}

// act(u) alone.  The exponential of a large -u is infinite and its quotient zero: under
// u = -87 the result is 0 in place of less than 1e-36.
__device__ __forceinline__ float activated(float u, int act)
{
    if (act == LA_ACT_NONE)
        return u;
    const float s = __fdividef(1.0f, 1.0f + __expf(-u));
    return act == LA_ACT_SIGMOID ? s : u * s;
}

// Tokens of row b: lengths clamped to 0 .. N, or N.
__device__ __forceinline__ int64_t row_length(const int* lengths, int64_t b, int64_t N)
{
    if (!lengths)
        return N;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n < N ? n : N;
}

// Whether pointer and strides (in elements) put every row on a 16-byte boundary.
inline bool rows16(const void* p, int64_t batch, int64_t token, int es)
{
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(batch * es) | (uintptr_t)(token * es)) & 15u) == 0;
}

}  // namespace rows
}  // namespace la
