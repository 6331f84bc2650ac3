// la_norm.cu -- per-head RMS norm with weight and gate behind the heads'
// outputs, and its gradient.
//
//   xh = x rsqrt(mean(x^2) + eps),   y = w xh act(gate)
//   c  = dy w act(gate),  dx = r (c - xh mean(c xh)),  r = rsqrt(mean(x^2) + eps)
//   dgate = dy w xh act'(gate),  dw = sum over rows of dy xh act(gate)
//
// x is head-major [B,H,N,dv] as the attention kernels write it; gate and y are
// token-major [B,N,H,dv] as the projections around them read it, so the
// transposition costs no pass of its own.  A row is dv / 8 lanes of eight
// elements (16 bytes of bf16): its sums are shuffles, and each tensor is read
// or written once.  Bound by HBM: 67 M fp32 elements with a bf16 gate 84 us (6.4
// TB/s), 33.5 M bf16 elements 37 us (5.4 TB/s) and their gradient 63 us (5.4 TB/s).
#include "la_internal.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;

struct Row8 {
    float f[8];
};

// Eight elements as they come, and as fp32: what is in flight stays as narrow as it is
// in memory, for more of it in a thread's registers.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
    float4 a, b;
};
template <> struct Raw8<__nv_bfloat16> {
    uint4 w;
};

__device__ __forceinline__ Raw8<float> fetch8(const float* p)
{
    return {__ldcs(reinterpret_cast<const float4*>(p)), __ldcs(reinterpret_cast<const float4*>(p) + 1)};
}

__device__ __forceinline__ Raw8<__nv_bfloat16> fetch8(const __nv_bfloat16* p)
{
    return {__ldcs(reinterpret_cast<const uint4*>(p))};
}

__device__ __forceinline__ Row8 wide(const Raw8<float>& x)
{
    return {{x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w}};
}

__device__ __forceinline__ Row8 wide(const Raw8<__nv_bfloat16>& x)
{
    Row8 r;
    const uint32_t u[4] = {x.w.x, x.w.y, x.w.z, x.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.f[2 * i] = __uint_as_float(u[i] << 16);
        r.f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
    return r;
}

__device__ __forceinline__ void store8(float* p, const Row8& r)
{
    __stcs(reinterpret_cast<float4*>(p), make_float4(r.f[0], r.f[1], r.f[2], r.f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(r.f[4], r.f[5], r.f[6], r.f[7]));
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const Row8& r)
{
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(r.f[2 * i], r.f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(u[0], u[1], u[2], u[3]));
}

// sum over the LPR lanes of a row (LPR a power of two, rows aligned in the warp)
template <int LPR>
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// act(g) and act'(g), from e = exp(-|g|) so that neither 1 - s nor the exponential of a
// large number is formed: the slope e / (1 + e)^2 keeps its digits for gates of either
// sign (s (1 - s) was 1% off at 12 and 0 from 17 on).  The hardware exponential and
// quotient: exp is off by at most 2 + 1.16 |g| ulp, the rest by a few, in fp32 under the
// rounding of what follows it for gates near 0; with the library forms this arithmetic,
// not memory, set the pace (69 against 43 us for 33.5 M bf16 elements together with 32-bit
// row indexes).
__device__ __forceinline__ float2 activate(float g, int act)
{
    if (act == LA_ACT_NONE)
        return make_float2(g, 1.0f);
    const float e = __expf(-fabsf(g)), r = __fdividef(1.0f, 1.0f + e);
    const float s = g >= 0.0f ? r : e * r, slope = e * r * r;
    return act == LA_ACT_SIGMOID ? make_float2(s, slope) : make_float2(g * s, fmaf(g, slope, s));
}

// eight weights of row `h` (1 without a weight)
__device__ __forceinline__ Row8 weights(const float* w, int at)
{
    Row8 r;
    if (w) {
        const float4 a = *reinterpret_cast<const float4*>(w + at);
        const float4 b = *reinterpret_cast<const float4*>(w + at + 4);
        r.f[0] = a.x, r.f[1] = a.y, r.f[2] = a.z, r.f[3] = a.w;
        r.f[4] = b.x, r.f[5] = b.y, r.f[6] = b.z, r.f[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r.f[j] = 1.0f;
    }
    return r;
}

// Rows in token-major order, some per lane group with every load issued first (33.5 M
// bf16 elements: one row 38.9 us, two 36.8, three 36.5, four 37.5; 67 M from fp32 to
// bf16 84.8, 88.0, 83.3 and 85.2 us; with an fp32 gate two, 51 against 53 us).
template <typename T>
constexpr int rows_at_once()
{
    return sizeof(T) == 2 ? 3 : 2;
}

template <int DV, typename TX, typename T>
__global__ void __launch_bounds__(kThreads)
    k_norm_gate(const TX* __restrict__ x, const T* __restrict__ gate, const float* __restrict__ w,
                T* __restrict__ y, uint32_t rows, uint32_t N, uint32_t H, int act, int weight_heads,
                float eps)
{
    constexpr uint32_t LPR = DV / 8, RPC = kThreads / LPR;
    constexpr int kRows = rows_at_once<T>();
    const uint32_t sub = threadIdx.x % LPR;
    Raw8<TX> xr[kRows];
    Raw8<T> gr[kRows];
    uint32_t row[kRows], head[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        row[i] = (blockIdx.x * kRows + i) * RPC + threadIdx.x / LPR;
        const uint32_t at = min(row[i], rows - 1);  // lanes past the end read the last row, write nothing
        const uint32_t bn = at / H, b = bn / N;
        head[i] = at - bn * H;
        xr[i] = fetch8(x + ((int64_t)(b * H + head[i]) * N + (bn - b * N)) * DV + sub * 8);
        if (gate)
            gr[i] = fetch8(gate + (int64_t)at * DV + sub * 8);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const Row8 xs = wide(xr[i]);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            ss = fmaf(xs.f[j], xs.f[j], ss);
        const float r = rsqrtf(row_sum<LPR>(ss) * (1.0f / DV) + eps);
        const Row8 wr = weights(w, (weight_heads ? head[i] * DV : 0) + sub * 8);
        Row8 o;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            o.f[j] = xs.f[j] * r * wr.f[j];
        if (gate) {
            const Row8 gs = wide(gr[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o.f[j] *= activate(gs.f[j], act).x;
        }
        if (row[i] < rows)
            store8(y + (int64_t)row[i] * DV + sub * 8, o);
    }
}

// Gradient.  Rows in token-major order as above (by head, a block read pieces of
// DV elements H DV apart: 93 against 66 us for 33.5 M bf16 elements); a lane
// group takes every GT-th row, GT = gridDim.x * RPC.  With a weight for each head GT
// is a multiple of H, so a group's part of dw belongs to one head.  A block leaves
// one part [DV], or one for each of its min(RPC, H) heads; k_norm_dw sums them in a
// fixed order (no atomics: repeat runs are bitwise equal).
// Blocks on an SM, as many as their registers leave room for: the grid is what the GPU
// holds at once.
constexpr int grad_per_sm(bool fp32_gate) { return fp32_gate ? 2 : 3; }

template <int DV, typename TX, typename T>
__global__ void __launch_bounds__(kThreads, grad_per_sm(sizeof(T) == 4))
    k_norm_gate_grad(const T* __restrict__ dy, const TX* __restrict__ x, const T* __restrict__ gate,
                     const float* __restrict__ w, TX* __restrict__ dx, T* __restrict__ dgate,
                     float* __restrict__ part, uint32_t rows, uint32_t N, uint32_t H, int act,
                     int weight_heads, float eps)
{
    constexpr uint32_t LPR = DV / 8, RPC = kThreads / LPR;
    __shared__ float sw[RPC][DV];
    const uint32_t sub = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const uint32_t first = blockIdx.x * RPC + grp, GT = gridDim.x * RPC;
    const Row8 wr = weights(w, (weight_heads ? first % H * DV : 0) + sub * 8);
    Row8 acc;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        acc.f[j] = 0.f;
    // where a row lies; groups past the end read the last row and write nothing
    auto x_row = [&](uint32_t at) {
        const uint32_t bn = at / H, b = bn / N, h = at - bn * H;
        return (b * H + h) * N + (bn - b * N);
    };
    auto place = [&](uint32_t row) { return (int64_t)row * DV + sub * 8; };
    uint32_t at = min(first, rows - 1), xa = x_row(at);
    Raw8<TX> xn = fetch8(x + place(xa));
    Raw8<T> dn = fetch8(dy + place(at)), gn;
    if (gate)
        gn = fetch8(gate + place(at));
    // whole warps stay in the loop together: the shuffles need every lane.  The next
    // row is in flight under this one's arithmetic
    for (uint32_t base = first; __any_sync(0xffffffffu, base < rows); base += GT) {
        const bool live = base < rows;
        const Row8 xr = wide(xn), dr = wide(dn);
        Row8 gr;
        if (gate)
            gr = wide(gn);
        const uint32_t next = min(base + GT, rows - 1), xb = x_row(next);
        xn = fetch8(x + place(xb)), dn = fetch8(dy + place(next));
        if (gate)
            gn = fetch8(gate + place(next));
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            ss = fmaf(xr.f[j], xr.f[j], ss);
        const float r = rsqrtf(row_sum<LPR>(ss) * (1.0f / DV) + eps);
        Row8 c, dg;
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float xh = xr.f[j] * r;
            const float2 a = gate ? activate(gr.f[j], act) : make_float2(1.0f, 0.0f);
            const float t = dr.f[j] * xh;
            if (live)
                acc.f[j] = fmaf(t, a.x, acc.f[j]);
            dg.f[j] = t * wr.f[j] * a.y;
            c.f[j] = dr.f[j] * wr.f[j] * a.x;
            dot = fmaf(c.f[j], xh, dot);
        }
        dot = row_sum<LPR>(dot) * (1.0f / DV);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            c.f[j] = r * (c.f[j] - xr.f[j] * r * dot);
        if (live) {
            store8(dx + place(xa), c);
            if (gate)
                store8(dgate + place(at), dg);
        }
        at = next, xa = xb;
    }
    if (part) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sw[grp][sub * 8 + j] = acc.f[j];
        __syncthreads();
        const uint32_t parts = weight_heads ? min(RPC, H) : 1;
        for (uint32_t i = threadIdx.x; i < parts * DV; i += kThreads) {
            float s = 0.f;
            for (uint32_t k = i / DV; k < RPC; k += weight_heads ? H : 1)  // groups of one head
                s += sw[k][i % DV];
            part[(int64_t)blockIdx.x * parts * DV + i] = s;
        }
    }
}

// dw[head or 0][c] = sum of the blocks' parts; 32 columns x 32 partial sums per
// block.  With a weight for each head, block b's part i is of head (b RPC + i) % H.
__global__ void __launch_bounds__(1024)
    k_norm_dw(const float* __restrict__ part, float* __restrict__ dw, uint32_t blocks, int DV, uint32_t RPC,
              uint32_t H, int weight_heads)
{
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int per = DV / 32;
    const uint32_t head = blockIdx.x / per, parts = weight_heads ? min(RPC, H) : 1;
    const int c = blockIdx.x % per * 32 + lane;
    float x = 0.f;
#pragma unroll 4
    for (uint32_t b = grp; b < blocks; b += 32) {
        const uint32_t i = weight_heads ? (head + H - b % H * (RPC % H) % H) % H : 0;
        if (i < parts)
            x += part[((int64_t)b * parts + i) * DV + c];
    }
    s[grp][lane] = x;
    __syncthreads();
    if (grp == 0) {
        x = 0.f;
        for (int i = 0; i < 32; ++i)
            x += s[i][lane];
        dw[(int64_t)head * DV + c] = x;
    }
}

uint32_t gcd(uint32_t a, uint32_t b) { return b ? gcd(b, a % b) : a; }

// Blocks of the gradient: what 152 SMs hold at once (one more per SM is a
// second round: bf16 77 us for four, 62 us for three), no more
// than there are row groups, a multiple of what keeps a group on one head.
int64_t grad_blocks(const NormGateArgs& a, bool heads, bool fp32_gate)
{
    const int64_t rpc = kThreads / (a.dv / 8), most = grad_per_sm(fp32_gate) * 152;
    const int64_t groups = (a.B * a.N * a.H + rpc - 1) / rpc;
    const int64_t want = most < groups ? most : groups;
    const int64_t unit = heads ? a.H / gcd((uint32_t)a.H, (uint32_t)rpc) : 1;
    return (want + unit - 1) / unit * unit;
}

template <int DV, typename TX, typename T>
cudaError_t run_norm(const NormGateArgs& a, bool grad)
{
    const TX* x = static_cast<const TX*>(a.x);
    const T* gate = static_cast<const T*>(a.gate);
    if (!grad) {
        const int64_t rows = a.B * a.N * a.H;
        const int64_t per = (int64_t)rows_at_once<T>() * (kThreads / (DV / 8));
        k_norm_gate<DV, TX, T><<<(unsigned)((rows + per - 1) / per), kThreads, 0, a.stream>>>(
            x, gate, a.weight, static_cast<T*>(a.y), (uint32_t)rows, (uint32_t)a.N, (uint32_t)a.H, a.act,
            a.weight_heads, a.eps);
        count_launches(1);
        return cudaGetLastError();
    }
    const bool heads = a.weight && a.weight_heads;
    const uint32_t blocks = (uint32_t)grad_blocks(a, heads, sizeof(T) == 4);
    float* part = a.dweight ? static_cast<float*>(a.ws) : nullptr;
    k_norm_gate_grad<DV, TX, T><<<blocks, kThreads, 0, a.stream>>>(
        static_cast<const T*>(a.dy), x, gate, a.weight, static_cast<TX*>(a.dx),
        static_cast<T*>(a.dgate), part, (uint32_t)(a.B * a.N * a.H), (uint32_t)a.N, (uint32_t)a.H, a.act,
        heads, a.eps);
    count_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !part)
        return e;
    k_norm_dw<<<(unsigned)((heads ? a.H : 1) * (DV / 32)), 1024, 0, a.stream>>>(
        part, a.dweight, blocks, DV, kThreads / (DV / 8), (uint32_t)a.H, heads);
    count_launches(1);
    return cudaGetLastError();
}

template <int DV>
cudaError_t norm_types(const NormGateArgs& a, bool grad)
{
    if (a.x_dtype == LA_BF16)
        return a.dtype == LA_BF16 ? run_norm<DV, __nv_bfloat16, __nv_bfloat16>(a, grad)
                                  : run_norm<DV, __nv_bfloat16, float>(a, grad);
    return a.dtype == LA_BF16 ? run_norm<DV, float, __nv_bfloat16>(a, grad)
                              : run_norm<DV, float, float>(a, grad);
}

cudaError_t norm_dims(const NormGateArgs& a, bool grad)
{
    switch (a.dv) {
    case 32: return norm_types<32>(a, grad);
    case 64: return norm_types<64>(a, grad);
    default: return norm_types<128>(a, grad);
    }
}

}  // namespace

// for either layout of the weight and any types
size_t norm_gate_backward_workspace(const NormGateArgs& a)
{
    const int64_t rpc = kThreads / (a.dv / 8);
    const int64_t p = grad_blocks(a, true, false) * (a.H < rpc ? a.H : rpc), q = grad_blocks(a, false, false);
    return sizeof(float) * (size_t)(p > q ? p : q) * a.dv;
}

cudaError_t norm_gate(const NormGateArgs& a) { return norm_dims(a, false); }
cudaError_t norm_gate_backward(const NormGateArgs& a) { return norm_dims(a, true); }

}  // namespace la
