// la_ssm_grad.cu -- gradients of the selective state-space scan.
//
// With dy = dout silu(z) and g_t the gradient of S_t,
//   g_t = C_t dy_t + a_{t+1} g_{t+1},      q_t = a_t g_t S_{t-1}   (gradient of dt A)
//   dB_t = sum_c g_t dt x,  dC_t = sum_c dy S_t,  dA = sum_t dt q_t
//   w_t = sum_s g_t B_t:    dx = dt w + D dy
//   ddelta = (sum_s A q_t + x w_t) sigmoid(delta + bias),  dbias = sum_t ddelta
//   dD = sum dy x,          dz = dout (y + D x) silu'(z)
// q is the product itself: a_t S_{t-1} as S_t - dt x B_t would lose the digits of a
// strong decay.
//
// Every row is cut into segments of 32 tokens.  k_ssm_ends gives each segment's end from a
// zero start, the sum of its steps, and what it adds to the gradient in front of it, all in
// one walk; k_ssm_join_grad walks the segments both ways; k_ssm_grad then has a true start
// and a true end for each.  It goes through its segment forwards, leaving a state in shared
// memory every four tokens, and back four tokens at a time, whose states are formed again and
// stay in registers.  Nothing is kept from the forward pass.
//
// A thread owns four neighbouring channels times four states (n = 8: two); the lanes that share
// a channel quad sum over states for four tokens together, so that a lane ends with
// neighbouring channels of one token and finishes them in pairs.
//
// Bound by arithmetic: k_ssm_grad has 15 fp32 operations and three exponentials an element and
// 400 instructions for 512 elements, at half of the issue slots with the two warps a
// sub-partition that 255 registers leave (B4 N2048 C2048 n = 16 bf16: 332 us, of 474 with the ends
// 99, the join 29 and the sums 15).  Two states per thread and twice the warps take a third
// more instructions for the same time (392 us); twelve warps with 168 registers spill (435 us);
// keeping the decays saves 2% and costs 64 registers; halves of 16 tokens, walked one and a half
// times, 390 us.
#include <type_traits>

#include "la_ssm.cuh"

namespace la {
namespace ssm {
namespace {

using namespace rows;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <int NS>
struct Lay {
    static constexpr int SPT = NS == 8 ? 2 : 4;      // states of a thread
    static constexpr int LPC = NS / SPT;             // lanes that share a channel quad
    static constexpr int QPW = 32 / LPC;             // quads of a warp
    static constexpr int CT = kWarps * QPW * 4;      // channels of a block
};

constexpr int LEN = 32;  // tokens of a segment
constexpr int BLK = 4;   // tokens in registers at a time
constexpr int SUB = 8;   // tokens whose dB and dC are joined at a time

// States of a thread's four channels, [channel pair][state].
template <int SPT>
struct Quad {
    float2 v[2][SPT];
    __device__ __forceinline__ float2 (&operator[](int p))[SPT] { return v[p]; }
    __device__ __forceinline__ const float2 (&operator[](int p) const)[SPT] { return v[p]; }
};

template <int SPT>
__device__ __forceinline__ Quad<SPT> quad_of(float x)
{
    Quad<SPT> h;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int s = 0; s < SPT; ++s)
            h[p][s] = both(x);
    return h;
}

// From and to memory [C][n]; channels behind the last are zero and are not written.
template <int NS, int SPT>
__device__ __forceinline__ void load_quad(const float* __restrict__ p, int have, Quad<SPT>& h)
{
    float f[4][SPT] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < have) {
            if constexpr (SPT == 4) {
                const float4 v = *reinterpret_cast<const float4*>(p + i * NS);
                f[i][0] = v.x, f[i][1] = v.y, f[i][2] = v.z, f[i][3] = v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2*>(p + i * NS);
                f[i][0] = v.x, f[i][1] = v.y;
            }
        }
#pragma unroll
    for (int s = 0; s < SPT; ++s)
        h[0][s] = make_float2(f[0][s], f[1][s]), h[1][s] = make_float2(f[2][s], f[3][s]);
}
template <int NS, int SPT>
__device__ __forceinline__ void store_quad(float* __restrict__ p, int have, const Quad<SPT>& h)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < have) {
            float f[SPT];
#pragma unroll
            for (int s = 0; s < SPT; ++s)
                f[s] = i & 1 ? h[i / 2][s].y : h[i / 2][s].x;
            if constexpr (SPT == 4)
                *reinterpret_cast<float4*>(p + i * NS) = make_float4(f[0], f[1], f[2], f[3]);
            else
                *reinterpret_cast<float2*>(p + i * NS) = make_float2(f[0], f[1]);
        }
}

// B or C of a thread's states, each twice (one register pair per product), as they lie in
// shared memory.
template <int SPT>
struct Twice {
    float2 s[SPT];
};
template <int SPT>
__device__ __forceinline__ Twice<SPT> twice(const float2* p)
{
    Twice<SPT> r;
#pragma unroll
    for (int i = 0; i < SPT; i += 2) {
        const float4 a = reinterpret_cast<const float4*>(p)[i / 2];
        r.s[i] = make_float2(a.x, a.y), r.s[i + 1] = make_float2(a.z, a.w);
    }
    return r;
}

struct GradIns {
    Rows x, delta, B, C, z, dout;
    const float *A, *D, *bias;
    const int* lengths;
    int softplus;
};

// Tokens of a segment in fp32, TOK at a time; B and C hold every number twice.
template <int NS, int TOK>
struct Wide {
    using L = Lay<NS>;
    float dt[TOK][L::CT], u[TOK][L::CT], dy[TOK][L::CT];
    float2 B[TOK][NS], C[TOK][NS];
};

template <int NS>
struct GradSmem {
    Wide<NS, LEN> w;
    float4 kept[LEN / BLK - 2][Lay<NS>::SPT][kThreads];  // states before every fourth token but the first and the last
    float sums[kWarps][SUB][2 * NS];                      // the warps' parts of dB and dC
};

// Four channels of one token; VEC: in one load, else one by one, `have` of them.
template <typename T, bool VEC>
__device__ __forceinline__ Raw<T, 4> four_at(const T* p, int have)
{
    Raw<T, 4> r;
    if constexpr (VEC) {
        memset(&r, 0, sizeof r);
        if (have > 0)
            r.w = __ldg(reinterpret_cast<const decltype(r.w)*>(p));
    } else {
        T v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = i < have ? __ldg(p + i) : from_f32<T>(0.0f);
        memcpy(&r, v, sizeof r);
    }
    return r;
}

// Two channels of one token as they lie in memory.
template <typename T, bool VEC>
__device__ __forceinline__ void raw_two(const T* p, int have, T (&v)[2])
{
    using Word = typename std::conditional<sizeof(T) == 2, uint32_t, uint2>::type;
    if constexpr (VEC) {
        Word w = {};
        if (have > 0)
            w = __ldg(reinterpret_cast<const Word*>(p));
        memcpy(v, &w, sizeof w);
    } else {
        v[0] = have > 0 ? __ldg(p) : from_f32<T>(0.0f);
        v[1] = have > 1 ? __ldg(p + 1) : from_f32<T>(0.0f);
    }
}

// Two channels of a parameter.
__device__ __forceinline__ float2 two_of(const float* p, int have)
{
    return make_float2(have > 0 ? __ldg(p) : 0.f, have > 1 ? __ldg(p + 1) : 0.f);
}
template <bool VEC>
__device__ __forceinline__ void put_two(float* p, float2 v, int have)
{
    if (VEC && have > 0) {
        *reinterpret_cast<float2*>(p) = v;
    } else {
        if (have > 0)
            p[0] = v.x;
        if (have > 1)
            p[1] = v.y;
    }
}
template <bool VEC>
__device__ __forceinline__ void put_two(__nv_bfloat16* p, float2 v, int have)
{
    if (VEC && have > 0) {
        *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
    } else {
        if (have > 0)
            p[0] = __float2bfloat16_rn(v.x);
        if (have > 1)
            p[1] = __float2bfloat16_rn(v.y);
    }
}

__device__ __forceinline__ void pair_up(const Vec<4>& v, float2 (&p)[2])
{
    p[0] = make_float2(v.f[0], v.f[1]), p[1] = make_float2(v.f[2], v.f[3]);
}

// TOK tokens from memory into `w`, of which `live` are the row's: dt, u = dt x, dy, B and C;
// the rest zero.  `from`: the first of them.
template <typename T, int NS, int TOK, bool VEC>
__device__ __forceinline__ void widen(Wide<NS, TOK>& w, const GradIns& in, const Place& at, int64_t from, int live)
{
    using L = Lay<NS>;
    constexpr int PER = L::CT / 4, STEP = kThreads / PER, EACH = TOK / STEP < 4 ? TOK / STEP : 4;
    auto base = [&](const Rows& r, int64_t col) {
        return static_cast<const T*>(r.p) + at.b * r.batch + from * r.token + col;
    };
    const int c = threadIdx.x % PER * 4, have = at.valid - c;
    const T *xs = base(in.x, at.c0 + c), *ds = base(in.delta, at.c0 + c), *os = base(in.dout, at.c0 + c);
    const T* zs = in.z.p ? base(in.z, at.c0 + c) : nullptr;
    const T *Bs = base(in.B, at.g * NS), *Cs = base(in.C, at.g * NS);
#pragma unroll 4
    for (int i = threadIdx.x; i < TOK * NS; i += kThreads) {
        const int t = i / NS, s = i % NS;
        w.B[0][i] = both(t < live ? to_f32(Bs[t * in.B.token + s]) : 0.0f);
        w.C[0][i] = both(t < live ? to_f32(Cs[t * in.C.token + s]) : 0.0f);
    }
    float bias[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        bias[j] = in.bias && j < have ? __ldg(in.bias + at.c0 + c + j) : 0.0f;
#pragma unroll 1
    for (int t0 = threadIdx.x / PER; t0 < TOK; t0 += EACH * STEP) {
        Raw<T, 4> x[EACH], d[EACH], o[EACH], z[EACH];  // in flight together
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int t = t0 + k * STEP, some = t < live ? have : 0;
            x[k] = four_at<T, VEC>(xs + t * in.x.token, some);
            d[k] = four_at<T, VEC>(ds + t * in.delta.token, some);
            o[k] = four_at<T, VEC>(os + t * in.dout.token, some);
            if (zs)
                z[k] = four_at<T, VEC>(zs + t * in.z.token, some);
        }
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int t = t0 + k * STEP;
            steps<4>(wide(d[k]), wide(x[k]), bias, in.softplus, t < live, &w.dt[t][c], &w.u[t][c]);
            float2 dy[2];
            pair_up(wide(o[k]), dy);
            if (zs) {
                float2 g[2];
                pair_up(wide(z[k]), g);
                dy[0] = mul2(dy[0], value<LA_ACT_SILU>(g[0])), dy[1] = mul2(dy[1], value<LA_ACT_SILU>(g[1]));
            }
            *reinterpret_cast<float4*>(&w.dy[t][c]) = make_float4(dy[0].x, dy[0].y, dy[1].x, dy[1].y);
        }
    }
}

__device__ __forceinline__ void pair_up(const float4& v, float2 (&p)[2])
{
    p[0] = make_float2(v.x, v.y), p[1] = make_float2(v.z, v.w);
}

// Per segment: end of the state from zero, sum of the steps, and sum over its tokens of (the
// decays up to t) C_t dy_t, the gradient in front of it.
template <typename T, int NS, bool VEC>
// (Blocks an SM, the whole gradient: bf16 B4 N2048 C2048 three 486 us, four 474; fp32 at four spills,
// B2 273 and 286, B3 N701 C600 47 and 51.  bf16 at four spills 112 bytes with n = 16 off rows of four
// elements, 4 to 8 in four other forms.)
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3)
    k_ssm_ends(GradIns in, float* __restrict__ ends, float* __restrict__ sums, float* __restrict__ fronts, Grid q)
{
    using L = Lay<NS>;
    constexpr int SPT = L::SPT, TOK = LEN / 2;
    extern __shared__ __align__(16) unsigned char smem[];
    auto& w = *reinterpret_cast<Wide<NS, TOK>*>(smem);
    const Place at = place_of(q, blockIdx.x, L::CT);
    const int64_t len = row_length(in.lengths, at.b, q.N), first = (int64_t)at.seg * q.seg_len;
    const int live = (int)max((int64_t)0, min((int64_t)q.seg_len, len - first));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c4 = (warp * L::QPW + lane / L::LPC) * 4, s4 = lane % L::LPC * SPT;
    const int have = max(0, min(4, at.valid - c4));
    Quad<SPT> A2, h = quad_of<SPT>(0.f), G = h, P = quad_of<SPT>(1.f);
    float2 sum[2] = {};
    load_quad<NS>(in.A + (at.c0 + c4) * (int64_t)NS + s4, have, A2);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int s = 0; s < SPT; ++s)
            A2[p][s] = mul2(A2[p][s], both(kLog2e));
    for (int from = 0; from < live; from += TOK) {
        if (from)
            __syncthreads();
        widen<T, NS, TOK, VEC>(w, in, at, first + from, live - from);
        __syncthreads();
#pragma unroll 4
        for (int t = 0; t < TOK; ++t) {
            float2 d[2], v[2], y[2];
            pair_up(*reinterpret_cast<const float4*>(&w.dt[t][c4]), d);
            pair_up(*reinterpret_cast<const float4*>(&w.u[t][c4]), v);
            pair_up(*reinterpret_cast<const float4*>(&w.dy[t][c4]), y);
            const Twice<SPT> B = twice<SPT>(&w.B[t][s4]), Cr = twice<SPT>(&w.C[t][s4]);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                sum[p] = add2(sum[p], d[p]);
#pragma unroll
                for (int s = 0; s < SPT; ++s) {
                    const float2 a = decay(d[p], A2[p][s]);
                    h[p][s] = fma2(a, h[p][s], mul2(v[p], B.s[s]));
                    P[p][s] = mul2(P[p][s], a);
                    G[p][s] = fma2(P[p][s], mul2(y[p], Cr.s[s]), G[p][s]);
                }
            }
        }
    }
    const int64_t seg = at.b * q.segs + at.seg, kept = (seg * q.C + at.c0 + c4) * NS + s4;
    store_quad<NS>(ends + kept, have, h);
    store_quad<NS>(fronts + kept, have, G);
    if (s4 == 0)
        for (int i = 0; i < have; ++i)
            sums[seg * q.C + at.c0 + c4 + i] = i == 0 ? sum[0].x : i == 1 ? sum[0].y : i == 2 ? sum[1].x : sum[1].y;
}

// In place, one thread per state: ends -> starts of the segments, fronts -> gradients at
// their ends; loads of eight segments ahead of the chain (the whole gradient, C2048 n = 16, four, eight
// and sixteen ahead: B16 N512 473, 477 and 503 us, B4 N2048 473, 474 and 481, B1 N8192 486, 484 and 481).
__global__ void __launch_bounds__(128)
    k_ssm_join_grad(const float* __restrict__ A, const float* __restrict__ S0, const float* __restrict__ dS_out,
                    float* __restrict__ ends, const float* __restrict__ sums, float* __restrict__ fronts,
                    float* __restrict__ dS0, int segs, int64_t C, int NS, int64_t items)
{
    const int64_t item = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (item >= items)
        return;
    const bool back = blockIdx.y;
    const int64_t row = C * NS, b = item / row, e = item - b * row;
    const float a = A[e] * kLog2e;
    const float* init = back ? dS_out : S0;
    float S = init ? init[item] : 0.0f;
    float* p = (back ? fronts : ends) + b * segs * row + e;
    const float* d = sums + b * segs * C + e / NS;
    constexpr int kAhead = 8;
    float E[2][kAhead], P[2][kAhead];
    auto at = [&](int i) { return (int64_t)(back ? segs - 1 - i : i); };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        E[0][k] = k < segs ? p[at(k) * row] : 0.0f;
        P[0][k] = k < segs ? d[at(k) * C] : 0.0f;
    }
    for (int i0 = 0; i0 < segs; i0 += 2 * kAhead)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = i0 + half * kAhead, n = i + kAhead;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                E[half ^ 1][k] = n + k < segs ? p[at(n + k) * row] : 0.0f;
                P[half ^ 1][k] = n + k < segs ? d[at(n + k) * C] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i + k < segs) {
                    p[at(i + k) * row] = S;
                    S = fmaf(ex2(a * P[half][k]), S, E[half][k]);
                }
        }
    if (back && dS0)
        dS0[item] = S;
}

// 2 SPT values summed over the warp's quads (lanes of equal lane % LPC): halves are
// traded, so that v[0 ..] ends with the sums of values first .. first + count - 1.
template <int LPC, int SPT>
__device__ __forceinline__ int sum_quads(float (&v)[2 * SPT], int lane)
{
    int first = 0, half = SPT;
#pragma unroll
    for (int o = 16; o >= LPC; o /= 2) {
        if (half == 0) {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
            continue;
        }
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < SPT; ++i)
            if (i < half) {
                const float give = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        first += up ? half : 0;
        half /= 2;
    }
    return first;
}

// Sums over the lanes of a quad for four tokens' channel pairs v[token][pair]: tokens are
// traded, then (LPC >= 8) pairs, so that a lane ends with both pairs v[0][0], v[0][1] of token
// lane & 3, or with its pair (lane >> 2) & 1 in v[0][0].
template <int LPC>
__device__ __forceinline__ void sum_tokens(float2 (&v)[4][2], int lane)
{
    auto trade = [&](float2 give, float2 keep, int o) {
        return add2(keep, make_float2(__shfl_xor_sync(0xffffffffu, give.x, o), __shfl_xor_sync(0xffffffffu, give.y, o)));
    };
    const bool up = lane & 2, odd = lane & 1, second = lane & 4;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int p = 0; p < 2; ++p)
            v[t][p] = trade(up ? v[t][p] : v[t + 2][p], up ? v[t + 2][p] : v[t][p], 2);
#pragma unroll
    for (int p = 0; p < 2; ++p)
        v[0][p] = trade(odd ? v[0][p] : v[1][p], odd ? v[1][p] : v[0][p], 1);
    if constexpr (LPC > 4)
        v[0][0] = trade(second ? v[0][0] : v[0][1], second ? v[0][1] : v[0][0], 4);
#pragma unroll
    for (int o = 8; o < LPC; o *= 2)
        v[0][0] = trade(v[0][0], v[0][0], o);
}

struct Outs {
    void *dx, *ddelta, *dz;
    float *rows;             // [channel tile of a group][B][N][G][2][n]: parts of dB and dC
    float *dA, *dD, *dbias;  // [B * segs][C][n], [B * segs][C], [B * segs][C]
};

template <typename T, int NS, bool VEC>
__global__ void __launch_bounds__(kThreads)
    k_ssm_grad(GradIns in, const float* __restrict__ starts, const float* __restrict__ finals, Outs out, Grid q)
{
    using L = Lay<NS>;
    constexpr int SPT = L::SPT;
    constexpr int PAIRS = L::LPC == 4 ? 2 : 1;  // channel pairs that a lane finishes
    extern __shared__ __align__(16) unsigned char smem[];
    auto& sm = *reinterpret_cast<GradSmem<NS>*>(smem);
    const Place at = place_of(q, blockIdx.x, L::CT);
    const int64_t len = row_length(in.lengths, at.b, q.N), first = (int64_t)at.seg * q.seg_len;
    const int here = (int)min((int64_t)q.seg_len, q.N - first);  // tokens of the segment
    const int live = (int)max((int64_t)0, min((int64_t)here, len - first));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c4 = (warp * L::QPW + lane / L::LPC) * 4, s4 = lane % L::LPC * SPT;
    const int have = max(0, min(4, at.valid - c4));
    const int64_t C = q.C;
    // the token of four and the channels that this lane finishes
    const int tok = lane & 3, cf = c4 + (PAIRS == 1 && (lane & 4) ? 2 : 0), fin = max(0, min(2 * PAIRS, at.valid - cf));
    const bool writes = lane % L::LPC < 8;
    const int64_t seg = at.b * q.segs + at.seg;
    const int64_t kept = (seg * C + at.c0 + c4) * NS + s4;
    Quad<SPT> A2, base, ag, dA = quad_of<SPT>(0.f);  // base: the state in front of the tokens at hand
    float2 D[PAIRS], bias[PAIRS], dD[PAIRS] = {}, dbias[PAIRS] = {};
    load_quad<NS>(in.A + (at.c0 + c4) * (int64_t)NS + s4, have, A2);
    load_quad<NS>(starts + kept, have, base);
    load_quad<NS>(finals + kept, have, ag);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int s = 0; s < SPT; ++s)
            A2[p][s] = mul2(A2[p][s], both(kLog2e));
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) {
        D[p] = in.D ? two_of(in.D + at.c0 + cf + 2 * p, fin - 2 * p) : both(0.f);
        bias[p] = in.bias ? two_of(in.bias + at.c0 + cf + 2 * p, fin - 2 * p) : both(0.f);
    }
    const int64_t row0 = at.b * q.N + first, wide_rows = (int64_t)q.G * 2 * NS;
    float* parts = out.rows + ((int64_t)(at.tile - at.g * q.per_group) * q.B * q.N + row0) * wide_rows + at.g * 2 * NS;

    auto state = [&](int slot) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int s = 0; s < SPT; s += 2) {
                const float4 v = sm.kept[slot][p * (SPT / 2) + s / 2][threadIdx.x];
                base[p][s] = make_float2(v.x, v.y), base[p][s + 1] = make_float2(v.z, v.w);
            }
    };
    const int blocks = (live + BLK - 1) / BLK;
    if (live > 0) {
        widen<T, NS, LEN, VEC>(sm.w, in, at, first, live);
        __syncthreads();
        // forwards to the last four tokens
#pragma unroll 1
        for (int blk = 0; blk < blocks - 1; ++blk) {
            if (blk > 0) {
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int s = 0; s < SPT; s += 2)
                        sm.kept[blk - 1][p * (SPT / 2) + s / 2][threadIdx.x] =
                            make_float4(base[p][s].x, base[p][s].y, base[p][s + 1].x, base[p][s + 1].y);
            }
#pragma unroll
            for (int j = 0; j < BLK; ++j) {
                const int t = blk * BLK + j;
                float2 d[2], v[2];
                pair_up(*reinterpret_cast<const float4*>(&sm.w.dt[t][c4]), d);
                pair_up(*reinterpret_cast<const float4*>(&sm.w.u[t][c4]), v);
                const Twice<SPT> B = twice<SPT>(&sm.w.B[t][s4]);
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int s = 0; s < SPT; ++s)
                        base[p][s] = fma2(decay(d[p], A2[p][s]), base[p][s], mul2(v[p], B.s[s]));
            }
        }
        // and back
#pragma unroll 1
        for (int blk = blocks - 1; blk >= 0; --blk) {
            // what this lane will finish is on its way meanwhile
            const int ts = blk * BLK + tok;
            const bool on = writes && ts < live;
            T xr[PAIRS][2], rr[PAIRS][2], zr[PAIRS][2], orr[PAIRS][2];
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) {
                const int some = on ? fin - 2 * p : 0;
                auto of = [&](const Rows& r, T (&v)[2]) {
                    raw_two<T, VEC>(static_cast<const T*>(r.p) + at.b * r.batch + (first + ts) * r.token + at.c0 + cf + 2 * p,
                                    some, v);
                };
                of(in.x, xr[p]);
                of(in.delta, rr[p]);
                if (in.z.p)
                    of(in.z, zr[p]), of(in.dout, orr[p]);
            }
            Quad<SPT> hs[BLK];
#pragma unroll
            for (int j = 0; j < BLK; ++j) {
                const int t = blk * BLK + j;
                float2 d[2], v[2];
                pair_up(*reinterpret_cast<const float4*>(&sm.w.dt[t][c4]), d);
                pair_up(*reinterpret_cast<const float4*>(&sm.w.u[t][c4]), v);
                const Twice<SPT> B = twice<SPT>(&sm.w.B[t][s4]);
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int s = 0; s < SPT; ++s)
                        hs[j][p][s] = fma2(decay(d[p], A2[p][s]), j ? hs[j ? j - 1 : 0][p][s] : base[p][s],
                                           mul2(v[p], B.s[s]));
            }
            float2 w[BLK][2], ddt[BLK][2], y[BLK][2];
#pragma unroll
            for (int j = BLK - 1; j >= 0; --j) {
                const int t = blk * BLK + j;
                float2 d[2], v[2], e[2], dB[SPT], dC[SPT];
                pair_up(*reinterpret_cast<const float4*>(&sm.w.dt[t][c4]), d);
                pair_up(*reinterpret_cast<const float4*>(&sm.w.u[t][c4]), v);
                pair_up(*reinterpret_cast<const float4*>(&sm.w.dy[t][c4]), e);
                const Twice<SPT> B = twice<SPT>(&sm.w.B[t][s4]), Cr = twice<SPT>(&sm.w.C[t][s4]);
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int s = 0; s < SPT; ++s) {
                        const float2 g = fma2(e[p], Cr.s[s], ag[p][s]);
                        w[j][p] = s ? fma2(g, B.s[s], w[j][p]) : mul2(g, B.s[s]);
                        dB[s] = p ? fma2(g, v[p], dB[s]) : mul2(g, v[p]);
                        dC[s] = p ? fma2(e[p], hs[j][p][s], dC[s]) : mul2(e[p], hs[j][p][s]);
                        y[j][p] = s ? fma2(hs[j][p][s], Cr.s[s], y[j][p]) : mul2(hs[j][p][s], Cr.s[s]);
                        ag[p][s] = mul2(decay(d[p], A2[p][s]), g);
                        const float2 qt = mul2(ag[p][s], j ? hs[j ? j - 1 : 0][p][s] : base[p][s]);
                        ddt[j][p] = s ? fma2(qt, A2[p][s], ddt[j][p]) : mul2(qt, A2[p][s]);
                        if (t < live)  // behind the row's last token perhaps infinity times zero
                            dA[p][s] = fma2(qt, d[p], dA[p][s]);
                    }
                float r[2 * SPT];
#pragma unroll
                for (int s = 0; s < SPT; ++s)
                    r[s] = dB[s].x + dB[s].y, r[SPT + s] = dC[s].x + dC[s].y;
                const int r0 = sum_quads<L::LPC, SPT>(r, lane);
                constexpr int count = L::QPW >= 2 * SPT ? 1 : 2 * SPT / L::QPW;
                if (L::QPW <= 2 * SPT || !(lane & L::LPC)) {
#pragma unroll
                    for (int i = 0; i < count; ++i) {
                        const int m = r0 + i;
                        sm.sums[warp][t % SUB][(m & SPT ? NS : 0) + s4 + (m & (SPT - 1))] = r[i];
                    }
                }
            }
            sum_tokens<L::LPC>(w, lane);
            sum_tokens<L::LPC>(ddt, lane);
            if (in.z.p)
                sum_tokens<L::LPC>(y, lane);
            if (writes && ts < here) {
                const int64_t dst = (row0 + ts) * C + at.c0 + cf;
#pragma unroll
                for (int p = 0; p < PAIRS; ++p) {
                    const int some = fin - 2 * p, col = cf + 2 * p;
                    const float2 x = make_float2(to_f32(xr[p][0]), to_f32(xr[p][1]));
                    const float2 raw = make_float2(to_f32(rr[p][0]), to_f32(rr[p][1]));
                    const float2 d = *reinterpret_cast<const float2*>(&sm.w.dt[ts][col]);
                    const float2 e = *reinterpret_cast<const float2*>(&sm.w.dy[ts][col]);
                    float2 vx = fma2(d, w[0][p], mul2(D[p], e));
                    float2 vd = fma2(x, w[0][p], mul2(ddt[0][p], both(0.6931471805599453f)));
                    if (in.softplus)
                        vd = mul2(vd, sigmoid(add2(raw, bias[p])).s);
                    if (!on)
                        vx = vd = both(0.f);
                    dD[p] = fma2(e, x, dD[p]);
                    dbias[p] = add2(dbias[p], vd);
                    put_two<VEC>(static_cast<T*>(out.dx) + dst + 2 * p, vx, some);
                    put_two<VEC>(static_cast<T*>(out.ddelta) + dst + 2 * p, vd, some);
                    if (in.z.p) {
                        const float2 z = make_float2(to_f32(zr[p][0]), to_f32(zr[p][1]));
                        const float2 o = make_float2(to_f32(orr[p][0]), to_f32(orr[p][1]));
                        float2 vz = mul2(mul2(o, fma2(D[p], x, y[0][p])), slope<LA_ACT_SILU>(z));
                        if (!on)  // zero times an infinite state
                            vz = both(0.f);
                        put_two<VEC>(static_cast<T*>(out.dz) + dst + 2 * p, vz, some);
                    }
                }
            }
            if (blk > 1)
                state(blk - 2);
            else if (blk == 1)
                load_quad<NS>(starts + kept, have, base);
            if (blk * BLK % SUB == 0) {
                // dB and dC of eight tokens, the warps' parts in order
                __syncthreads();
                for (int i = threadIdx.x; i < SUB * 2 * NS; i += kThreads) {
                    const int t = i / (2 * NS), m = i - t * 2 * NS;
                    if (blk * BLK + t < min(here, blocks * BLK)) {
                        float sum = sm.sums[0][t][m];  // behind the row's last token perhaps zero times infinity
#pragma unroll
                        for (int k = 1; k < kWarps; ++k)
                            sum += sm.sums[k][t][m];
                        parts[(blk * BLK + t) * wide_rows + m] = blk * BLK + t < live ? sum : 0.0f;
                    }
                }
                __syncthreads();
            }
        }
    }
    // fours behind the row's last token
    const int done = min(here, blocks * BLK);
    for (int i = threadIdx.x; i < (here - done) * at.valid; i += kThreads) {
        const int64_t o = (row0 + done + i / at.valid) * C + at.c0 + i % at.valid;
        static_cast<T*>(out.dx)[o] = from_f32<T>(0.0f);
        static_cast<T*>(out.ddelta)[o] = from_f32<T>(0.0f);
        if (in.z.p)
            static_cast<T*>(out.dz)[o] = from_f32<T>(0.0f);
    }
    for (int i = threadIdx.x; i < (here - done) * 2 * NS; i += kThreads)
        parts[(done + i / (2 * NS)) * wide_rows + i % (2 * NS)] = 0.0f;
    store_quad<NS>(out.dA + kept, have, dA);
    // dD and dbias over the four lanes that share channels, each of which holds its tokens'
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) {
#pragma unroll
        for (int o = 1; o < 4; o *= 2) {
            dD[p] = add2(dD[p], make_float2(__shfl_xor_sync(0xffffffffu, dD[p].x, o), __shfl_xor_sync(0xffffffffu, dD[p].y, o)));
            dbias[p] = add2(dbias[p], make_float2(__shfl_xor_sync(0xffffffffu, dbias[p].x, o),
                                                  __shfl_xor_sync(0xffffffffu, dbias[p].y, o)));
        }
        if (writes && tok == 0) {
            put_two<false>(out.dD + seg * C + at.c0 + cf + 2 * p, dD[p], fin - 2 * p);
            put_two<false>(out.dbias + seg * C + at.c0 + cf + 2 * p, dbias[p], fin - 2 * p);
        }
    }
}

// The sums over blocks, in a fixed order.  Blocks 0 .. row_blocks - 1: dB, dC [rows][G][n] from
// the channel tiles' parts [tile][rows][G][2][n].  Then columns x 8 partial sums a block:
// those of dA (128), dD and dbias (32) over the segments.
struct Sums {
    const float* rows;
    int64_t values;       // of a tile's parts
    int tiles, NS;
    unsigned row_blocks;
    unsigned dA_blocks;
    const float* part[3];
    float* out[3];
    int64_t cols[2], segs;
};

__device__ __forceinline__ float4 plus(float4 a, float4 b)
{
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

template <typename T>
__global__ void __launch_bounds__(256) k_ssm_sums(Sums q, T* __restrict__ dB, T* __restrict__ dC)
{
    if (blockIdx.x < q.row_blocks) {
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
        if (i >= q.values)
            return;
        float s = 0.f;
        for (int k0 = 0; k0 < q.tiles; k0 += 8) {
            float v[8];  // in flight together
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = k0 + k < q.tiles ? __ldg(q.rows + (k0 + k) * q.values + i) : 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                s += v[k];
        }
        const int64_t pair = i / q.NS;
        (pair & 1 ? dC : dB)[pair / 2 * q.NS + i % q.NS] = from_f32<T>(s);
        return;
    }
    __shared__ float4 sums[8][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    unsigned block = blockIdx.x - q.row_blocks;
    if (block < q.dA_blocks) {
        const int64_t c = (int64_t)block * 32 + lane, cols = q.cols[0] / 4;  // four columns a lane
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < cols) {
            const float4* p = reinterpret_cast<const float4*>(q.part[0]) + c;
            for (int64_t r = grp; r < q.segs; r += 64) {
                float4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = r + 8 * k < q.segs ? __ldg(p + (r + 8 * k) * cols) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    x = plus(x, v[k]);
            }
        }
        sums[grp][lane] = x;
        __syncthreads();
        if (grp == 0 && c < cols) {
            for (int i = 1; i < 8; ++i)
                x = plus(x, sums[i][lane]);
            reinterpret_cast<float4*>(q.out[0])[c] = x;
        }
        return;
    }
    block -= q.dA_blocks;
    const unsigned half = (unsigned)((q.cols[1] + 31) / 32);
    const int which = block < half ? 1 : 2;
    const int64_t cols = q.cols[1], c = (int64_t)(block - (which == 2 ? half : 0)) * 32 + lane;
    float x = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t r = grp; r < q.segs; r += 8)
            x += __ldg(q.part[which] + r * cols + c);
    }
    sums[grp][lane].x = x;
    __syncthreads();
    if (grp == 0 && c < cols && q.out[which]) {
        for (int i = 1; i < 8; ++i)
            x += sums[i][lane].x;
        q.out[which][c] = x;
    }
}

template <int NS>
Grid grid_of(const SsmArgs& a)
{
    Grid q;
    q.B = a.B, q.N = a.N, q.C = (int)a.C, q.G = (int)a.G;
    q.per_group = (int)((a.C / a.G + Lay<NS>::CT - 1) / Lay<NS>::CT);
    q.seg_len = LEN;
    q.segs = (int)((a.N + q.seg_len - 1) / q.seg_len);
    return q;
}

Grid grid_any(const SsmArgs& a)
{
    switch (a.n) {
    case 8: return grid_of<8>(a);
    case 16: return grid_of<16>(a);
    case 32: return grid_of<32>(a);
    default: return grid_of<64>(a);
    }
}

// The workspace, in floats: states at the segments' starts, gradients at their ends, parts of
// dA; sums of the segments' steps (later the parts of dD), parts of dbias; parts of dB and dC.
struct Space {
    int64_t state, chan, rows;
    Space(const SsmArgs& a, const Grid& q)
        : state(a.B * q.segs * a.C * a.n), chan(a.B * q.segs * a.C), rows(q.per_group * a.B * a.N * a.G * 2 * a.n)
    {
        chan = (chan + 3) / 4 * 4;
    }
    int64_t floats() const { return 3 * state + 2 * chan + rows; }
};

template <typename T, int NS, bool VEC>
cudaError_t run_grad(const SsmArgs& a, const GradIns& in, const Grid& q)
{
    const Space sp(a, q);
    float* ends = static_cast<float*>(a.ws);
    float *fronts = ends + sp.state, *dA = fronts + sp.state, *sums = dA + sp.state, *dbias = sums + sp.chan;
    float* rows = dbias + sp.chan;
    const unsigned blocks = (unsigned)(a.B * q.segs * q.G * q.per_group);
    static_assert(sizeof(Wide<NS, LEN / 2>) <= 48 * 1024, "shared memory of a launch without attributes");
    k_ssm_ends<T, NS, VEC><<<blocks, kThreads, sizeof(Wide<NS, LEN / 2>), a.stream>>>(in, ends, sums, fronts, q);
    count_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    const int64_t items = a.B * a.C * NS;
    k_ssm_join_grad<<<dim3((unsigned)((items + 127) / 128), 2), 128, 0, a.stream>>>(
        a.A, a.S0, a.dS_out, ends, sums, fronts, a.dS0, q.segs, a.C, NS, items);
    count_launches(1);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    e = cudaFuncSetAttribute(k_ssm_grad<T, NS, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(GradSmem<NS>));
    if (e != cudaSuccess)
        return e;
    k_ssm_grad<T, NS, VEC><<<blocks, kThreads, sizeof(GradSmem<NS>), a.stream>>>(
        in, ends, fronts, Outs{a.dx, a.ddelta, a.dz, rows, dA, sums, dbias}, q);
    count_launches(1);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    const int64_t values = a.B * a.N * a.G * 2 * NS;
    const int64_t row_blocks = (values + 255) / 256, dA_blocks = (a.C * NS + 127) / 128;
    const int64_t col_blocks = dA_blocks + 2 * ((a.C + 31) / 32);
    k_ssm_sums<T><<<(unsigned)(row_blocks + col_blocks), 256, 0, a.stream>>>(
        Sums{rows, values, q.per_group, NS, (unsigned)row_blocks, (unsigned)dA_blocks, {dA, sums, dbias},
             {a.dA, a.dD, a.dbias}, {a.C * NS, a.C}, a.B * q.segs},
        static_cast<T*>(a.dB), static_cast<T*>(a.dC));
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, int NS>
cudaError_t grad_rows(const SsmArgs& a)
{
    const GradIns in{{a.x, a.x_batch, a.x_token}, {a.delta, a.delta_batch, a.delta_token},
                     {a.Bm, a.B_batch, a.B_token}, {a.Cm, a.C_batch, a.C_token}, {a.z, a.z_batch, a.z_token},
                     {a.dout, a.dout_batch, a.dout_token}, a.A, a.D, a.bias, a.lengths, a.softplus};
    // four channels in a load where rows and groups allow it (B4 N2048 C2048 n = 16 bf16, rows a little
    // wider than their channels: 488 us, off by one element 597)
    bool vec = a.C / a.G % 4 == 0;
    for (const Rows& r : {in.x, in.delta, in.z, in.dout})
        vec = vec && (!r.p || rows_on(r.p, r.batch, r.token, (int)sizeof(T), 4 * sizeof(T)));
    const Grid q = grid_of<NS>(a);
    return vec ? run_grad<T, NS, true>(a, in, q) : run_grad<T, NS, false>(a, in, q);
}

template <typename T>
cudaError_t grad_states(const SsmArgs& a)
{
    switch (a.n) {
    case 8: return grad_rows<T, 8>(a);
    case 16: return grad_rows<T, 16>(a);
    case 32: return grad_rows<T, 32>(a);
    default: return grad_rows<T, 64>(a);
    }
}

}  // namespace
}  // namespace ssm

size_t ssm_backward_workspace(const SsmArgs& a)
{
    return sizeof(float) * (size_t)ssm::Space(a, ssm::grid_any(a)).floats();
}

cudaError_t ssm_backward(const SsmArgs& a)
{
    return a.dtype == LA_BF16 ? ssm::grad_states<__nv_bfloat16>(a) : ssm::grad_states<float>(a);
}

}  // namespace la
