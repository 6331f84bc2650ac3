// la_ssm.cuh -- what the forward and the gradient of the selective scan share: tiles of
// tokens in shared memory, steps and decays, where a block works.
//
//   dt_t = softplus(delta_t + delta_bias),  a_t = exp(dt_t A[c,s]),
//   S_t = a_t S_{t-1} + dt_t x_t B_t,       y_t = sum_s C_t S_t + D x_t
#pragma once

#include "la_rows.cuh"

namespace la {
namespace ssm {

// Where a block works: channels c0 .. c0 + valid - 1 of group g, row b, segment.
struct Place {
    int64_t b;
    int seg, g, c0, valid, tile;
};

struct Grid {
    int64_t B, N;
    int C, G, per_group;  // channel tiles of a group
    int segs, seg_len;    // seg_len a multiple of the tile
};

__device__ __forceinline__ Place place_of(const Grid& q, int64_t block, int width)
{
    const int tiles = q.G * q.per_group;
    const int64_t rest = block / tiles;
    Place p;
    p.tile = (int)(block - rest * tiles);
    p.b = rest / q.segs, p.seg = (int)(rest - p.b * q.segs);
    p.g = p.tile / q.per_group;
    const int in = (p.tile - p.g * q.per_group) * width, cg = q.C / q.G;
    p.c0 = p.g * cg + in, p.valid = min(width, cg - in);
    return p;
}

// Strided rows of one input.
struct Rows {
    const void* p;
    int64_t batch, token;
};

using rows::add2;
using rows::both;
using rows::ex2;
using rows::fma2;
using rows::kLog2e;
using rows::mul2;

// The decay 2^(dt A2), A2 = A log2(e).  The hardware exponential is low by 0.1 (arguments
// above -2^-9) to 0.46 * 2^-24 in the mean, which a state that remembers a thousand tokens
// adds up a thousand times; a quarter of 2^-24 more in the argument, in the same
// instruction as the product, brings that to within 0.09 above -2^-9 and 0.29 elsewhere
// above -1/4.  2^kLift itself is exactly 1: dt = 0 leaves a state as it was.
constexpr float kLift = 0.25f / 16777216.0f;
__device__ __forceinline__ float2 decay(float2 dt, float2 A2)
{
    const float2 t = fma2(dt, A2, both(kLift));
    return make_float2(ex2(t.x), ex2(t.y));
}

// log(1 + e^u) = max(u, 0) + log1p(e), e = exp(-|u|) in (0, 1].  log1p(e) = 2 atanh(w),
// w = e / (2 + e) <= 1/3, atanh(w) / w = 1 + q p(q) with q = w^2 and p the cubic through
// (atanh(w) / w - 1) / q at the Chebyshev points of [0, 1/9]: 1.6e-8 of the result.  A small
// step keeps all its digits, which log(1 + e) would not.
__device__ __forceinline__ float2 softplus(float2 u)
{
    const float2 e = make_float2(ex2(-fabsf(u.x) * kLog2e), ex2(-fabsf(u.y) * kLog2e));
    const float2 f = add2(e, both(2.0f)), w = mul2(e, make_float2(rows::rcp(f.x), rows::rcp(f.y))), q = mul2(w, w);
    float2 s = fma2(q, both(0.134257495f), both(0.141183093f));
    s = fma2(s, q, both(0.200037807f));
    s = fma2(s, q, both(0.333333194f));
    s = fma2(s, q, both(1.0f));
    return fma2(add2(w, w), s, make_float2(fmaxf(u.x, 0.0f), fmaxf(u.y, 0.0f)));
}

// Steps and inputs of V channels of one token from what lies in memory: dt and u = dt x,
// zero behind the row's last token.
template <int V>
__device__ __forceinline__ void steps(const rows::Vec<V>& raw, const rows::Vec<V>& x, const float (&bias)[V],
                                      int plus, bool on, float* dt, float* u)
{
#pragma unroll
    for (int j = 0; j < V; j += 4) {
        float2 d[2], v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = j + 2 * k;
            float2 r = add2(make_float2(raw.f[i], raw.f[i + 1]), make_float2(bias[i], bias[i + 1]));
            if (plus)
                r = softplus(r);
            d[k] = on ? r : make_float2(0.f, 0.f);
            v[k] = mul2(d[k], make_float2(x.f[i], x.f[i + 1]));
        }
        *reinterpret_cast<float4*>(dt + j) = make_float4(d[0].x, d[0].y, d[1].x, d[1].y);
        *reinterpret_cast<float4*>(u + j) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    }
}

// BYTES (4 or 16) from memory, of which the first `have` are read and the rest zero.
template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src, int have)
{
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(have) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(src), "r"(have) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// A tile of `WIDE` columns into shared memory [TT][WIDE], `live` tokens and `cols` columns of it
// from memory, the rest zero (bytes behind either are not read).  BYTES: what every row starts
// and ends on a multiple of, 16 or 4, for copies of that size in flight; 0 for neither, element
// by element (forward of B4 N8192 C2048 n = 16 bf16: 486 us on 16 bytes, 568 off by two elements,
// 796 off by one; fp32 B2: 277 us, and 371 off by one).
template <typename T, int TT, int WIDE, int BYTES, int NT>
__device__ __forceinline__ void copy_tile(T* dst, const T* src, int64_t token, int live, int cols)
{
    if constexpr (BYTES > 0) {
        constexpr int V = BYTES / (int)sizeof(T), PER = WIDE / V;
#pragma unroll
        for (int k = 0; k < (TT * PER + NT - 1) / NT; ++k) {
            const int i = k * NT + threadIdx.x, t = i / PER, c = i % PER * V;
            if (TT * PER % NT && i >= TT * PER)
                break;
            const bool on = t < live && c < cols;
            cp_async<BYTES>(dst + t * WIDE + c, on ? src + t * token + c : src, on ? BYTES : 0);
        }
    } else {
        constexpr int kAhead = 16;  // loads in flight together
        for (int i0 = threadIdx.x; i0 < TT * WIDE; i0 += kAhead * NT) {
            T v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + k * NT, t = i / WIDE, c = i % WIDE;
                v[k] = t < live && c < cols ? __ldg(src + t * token + c) : from_f32<T>(0.0f);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i0 + k * NT < TT * WIDE)
                    dst[i0 + k * NT] = v[k];
        }
    }
}

}  // namespace ssm
}  // namespace la
