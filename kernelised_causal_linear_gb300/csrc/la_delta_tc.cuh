// la_delta_tc.cuh -- device helpers of the tensor-core delta-rule kernels:
// fp16 operands with power-of-two scales, warp-level MMAs and their fragments.
//
// Operands.  A bf16 row times a power of two that brings its largest entry to
// [2^8, 2^9) is exact in fp16 (entries under 2^-17 of the largest lose bits,
// at most 2^-33 of it).  An fp32 operand so scaled is the sum of two fp16
// parts to 2^-22 of each entry.  So products of inputs are exact, products
// with an fp32 value cost two MMAs and lose about as much as fp32 itself, and
// the scales (exact) come off the fp32 accumulators.
//
// Fragments of m16n8k16, lane = 4 g + t: A (16 x 16) {A[g][2t..]},
// {A[g+8][2t..]}, {A[g][2t+8..]}, {A[g+8][2t+8..]}; B (16 x 8) {B[2t..][g]},
// {B[2t+8..][g]}; C (16 x 8) C[g][2t], C[g][2t+1], C[g+8][2t], C[g+8][2t+1].
// Two neighbouring C tiles are an A fragment: what a product leaves in
// registers enters the next one without touching shared memory.
#pragma once

#include <cuda_fp16.h>

#include "la_delta.cuh"
#include "la_sm100.cuh"

namespace la {
namespace delta {

using sm100::smem_addr;

constexpr int kC = 64;  // tokens per chunk

__device__ __forceinline__ uint32_t h2(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// two fp32 -> packed fp16 parts, hi + lo = x to 2^-22 (scaled operands)
__device__ __forceinline__ void h2_split(float a, float b, uint32_t& hi, uint32_t& lo)
{
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = h2(a - f.x, b - f.y);
}

// bf16 pair -> two fp32
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float2 bf2(uint32_t w) { return make_float2(lo_f(w), hi_f(w)); }

// The two rows of a C tile: row g (registers 0, 1), row g + 8 (2, 3)
__device__ __forceinline__ float2 row_a(const float (&x)[4]) { return make_float2(x[0], x[1]); }
__device__ __forceinline__ float2 row_b(const float (&x)[4]) { return make_float2(x[2], x[3]); }
__device__ __forceinline__ void set_rows(float (&x)[4], float2 a, float2 b)
{
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
// x times a factor for each row, or for each column
__device__ __forceinline__ void scale_rows(float (&x)[4], float a, float b)
{
    set_rows(x, mul2(row_a(x), both(a)), mul2(row_b(x), both(b)));
}
__device__ __forceinline__ void scale_cols(float (&x)[4], float2 f)
{
    set_rows(x, mul2(row_a(x), f), mul2(row_b(x), f));
}

// x times a power of two -> packed fp16 parts
__device__ __forceinline__ void h2_split(float2 x, float to, uint32_t& hi, uint32_t& lo)
{
    const float2 y = mul2(x, both(to));
    const __half2 h = __floats2half2_rn(y.x, y.y);
    const float2 f = __half22float2(h);
    const float2 r = fma2(f, both(-1.0f), y);  // exact
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = h2(r.x, r.y);
}

// The power of two that brings m (>= 0) to [2^8, 2^9), and its inverse.  Zero
// and numbers under 2^-118 get the largest scale, 2^126: an operand's own factors
// are multiplied in before it, so that no product of scales overflows.
struct Pow2 {
    float to, from;
};
__device__ __forceinline__ Pow2 pow2_for(float m)
{
    const int e = min(max((int)(__float_as_uint(m) >> 23), 9), 254);
    Pow2 p;
    p.to = __uint_as_float((uint32_t)(262 - e) << 23);
    p.from = __uint_as_float((uint32_t)(e - 8) << 23);
    return p;
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, const uint32_t (&r)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

// Byte offset of 16-byte part c of row r in a tile of BYTES-byte rows; the
// parts are swapped so that eight rows of one column block hit eight bank
// groups (ldmatrix without conflicts).
template <int BYTES>
__device__ __forceinline__ uint32_t tile_off(int r, int c)
{
    if (BYTES >= 128)
        return (uint32_t)(r * BYTES + ((c ^ (r & 7)) << 4));
    if (BYTES == 64)
        return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    return (uint32_t)(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
}

// Lane address of ldsm4 for B tiles (n0 .. n0+15) x (k0 .. k0+15) of a
// row-major X[n][k] tile: r[0], r[1] belong to n0, r[2], r[3] to n0 + 8.
template <int BYTES>
__device__ __forceinline__ uint32_t addr_b(uint32_t base, int lane, int n0, int k0)
{
    return base + tile_off<BYTES>(n0 + ((lane >> 4) << 3) + (lane & 7), (k0 >> 3) + ((lane >> 3) & 1));
}
// The same from X[k][n] (ldsm4t).
template <int BYTES>
__device__ __forceinline__ uint32_t addr_bt(uint32_t base, int lane, int k0, int n0)
{
    return base + tile_off<BYTES>(k0 + (((lane >> 3) & 1) << 3) + (lane & 7), (n0 >> 3) + (lane >> 4));
}
// Lane address of ldsm4 for the A tile (m0 .. +15) x (k0 .. +15) of X[m][k].
template <int BYTES>
__device__ __forceinline__ uint32_t addr_a(uint32_t base, int lane, int m0, int k0)
{
    return base + tile_off<BYTES>(m0 + (((lane >> 3) & 1) << 3) + (lane & 7), (k0 >> 3) + (lane >> 4));
}
// Lane address of ldsm4t / stsm4t for 16 tokens x 16 columns of X[token][col]
// as C tiles of the transpose: r[0], r[1] rows g and g + 8 (columns) of token
// tile 0, r[2], r[3] of token tile 1.
template <int BYTES>
__device__ __forceinline__ uint32_t addr_ct(uint32_t base, int lane, int tok0, int col0)
{
    return base + tile_off<BYTES>(tok0 + ((lane >> 4) << 3) + (lane & 7), (col0 >> 3) + ((lane >> 3) & 1));
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// bulk copy global -> shared, completing on an mbarrier
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_addr(bar))
        : "memory");
}

// Wait for phase `parity` of a barrier, two seconds at most (the copies waited for are
// a few microseconds old): false then, and the caller records LA_ERR_TIMEOUT.
__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity)
{
    if (sm100::mbar_try_wait(bar, parity))
        return true;
    const uint64_t until = now_ns() + 2000000000ull;
    while (!sm100::mbar_try_wait(bar, parity))
        if (now_ns() > until)
            return false;
    return true;
}

// 2^x on the hardware (2 ulp, denormals to zero)
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float max_abs(float m, float x) { return fmaxf(m, fabsf(x)); }

template <int N_>
__device__ __forceinline__ void clear(float (&x)[N_][4])
{
#pragma unroll
    for (int i = 0; i < N_; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[i][e] = 0.f;
}

// largest over the four lanes of a fragment row
__device__ __forceinline__ float quad_max(float x)
{
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

}  // namespace delta
}  // namespace la
