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
// Every row is cut into short segments.  k_ssm_ends gives each segment's end from a
// zero start, its decays, and what it adds to the gradient in front of it, all in one
// walk; k_ssm_join_grad walks the segments both ways; k_ssm_grad then has a true start
// and a true end for each.  It walks its segment forwards, leaving a state in shared
// memory every four tokens, and back four tokens at a time, whose states and decays
// are formed again and stay in registers.  Nothing is kept from the forward pass.
#include "la_ssm.cuh"

namespace la {
namespace ssm {
namespace {

using namespace rows;

template <int NS>
struct Seg {
    static constexpr int LEN = NS == 8 ? 16 : 32;  // tokens of a segment
    static constexpr int SUB = 8;                  // tokens in fp32 at a time
    static constexpr int BLK = 4;                  // tokens in registers at a time
};

struct GradIns {
    Rows x, delta, B, C, z, dout;
    const float *A, *D, *bias;
    const int* lengths;
    int softplus;
};

template <typename T, int NS>
struct RawSeg {
    using L = Lay<NS>;
    static constexpr int LEN = Seg<NS>::LEN;
    T x[LEN][L::CT], delta[LEN][L::CT], z[LEN][L::CT], dout[LEN][L::CT];
    T B[LEN][NS], C[LEN][NS];
};

template <int NS>
struct Wide {
    using L = Lay<NS>;
    float dt[Seg<NS>::SUB][L::CT], u[Seg<NS>::SUB][L::CT], dy[Seg<NS>::SUB][L::CT];
    float2 B[Seg<NS>::SUB][NS], C[Seg<NS>::SUB][NS];  // every number twice
};

template <typename T, int NS>
struct EndsSmem {
    RawSeg<T, NS> raw;
    Wide<NS> w;
};

template <typename T, int NS>
struct GradSmem {
    using L = Lay<NS>;
    RawSeg<T, NS> raw;
    Wide<NS> w;
    float4 kept[Seg<NS>::LEN / Seg<NS>::BLK - 1][4][kThreads];  // states before every fourth token but the first
    float sums[kWarps][Seg<NS>::SUB][2 * NS];                // the warps' parts of dB and dC
};

// The whole segment on its way into shared memory.
template <typename T, int NS, bool ASYNC>
__device__ __forceinline__ void load_segment(RawSeg<T, NS>& raw, const GradIns& in, const Place& at, int64_t first,
                                             int live)
{
    using L = Lay<NS>;
    constexpr int LEN = Seg<NS>::LEN;
    auto rows_of = [&](const Rows& r, int64_t col) {
        return static_cast<const T*>(r.p) + at.b * r.batch + first * r.token + col;
    };
    copy_tile<T, LEN, L::CT, ASYNC>(raw.x[0], rows_of(in.x, at.c0), in.x.token, live, at.valid);
    copy_tile<T, LEN, L::CT, ASYNC>(raw.delta[0], rows_of(in.delta, at.c0), in.delta.token, live, at.valid);
    copy_tile<T, LEN, L::CT, ASYNC>(raw.dout[0], rows_of(in.dout, at.c0), in.dout.token, live, at.valid);
    if (in.z.p)
        copy_tile<T, LEN, L::CT, ASYNC>(raw.z[0], rows_of(in.z, at.c0), in.z.token, live, at.valid);
    copy_tile<T, LEN, NS, ASYNC>(raw.B[0], rows_of(in.B, at.g * NS), in.B.token, live, NS);
    copy_tile<T, LEN, NS, ASYNC>(raw.C[0], rows_of(in.C, at.g * NS), in.C.token, live, NS);
    cp_commit();
    cp_wait<0>();
    __syncthreads();
}

// Tokens t0 .. t0 + SUB - 1 of the segment in fp32: dt, u = dt x, B and, with GRAD,
// dy and C.  Tokens behind the row's last have dt = u = dy = 0.
template <typename T, int NS, bool GRAD>
__device__ __forceinline__ void widen(const RawSeg<T, NS>& raw, Wide<NS>& w, const GradIns& in, const Place& at, int t0,
                                      int live)
{
    using L = Lay<NS>;
    constexpr int SUB = Seg<NS>::SUB, CT = L::CT, V = 4;
    const int c = threadIdx.x % (CT / V) * V;
    float bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        bias[j] = in.bias && c + j < at.valid ? __ldg(in.bias + at.c0 + c + j) : 0.0f;
#pragma unroll
    for (int t = threadIdx.x / (CT / V); t < SUB; t += kThreads / (CT / V)) {
        auto vec = [&](const T* p) {
            Raw<T, V> r;
            r.w = *reinterpret_cast<const decltype(r.w)*>(p);
            return wide(r);
        };
        auto put = [&](float* p, const float (&f)[V]) {
#pragma unroll
            for (int j = 0; j < V; j += 4)
                *reinterpret_cast<float4*>(p + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
        };
        steps<V>(vec(&raw.delta[t0 + t][c]), vec(&raw.x[t0 + t][c]), bias, in.softplus, t0 + t < live, &w.dt[t][c],
                 &w.u[t][c]);
        if constexpr (GRAD) {
            const Vec<V> o = vec(&raw.dout[t0 + t][c]);
            float dy[V];
            if (in.z.p) {
                const Vec<V> z = vec(&raw.z[t0 + t][c]);
#pragma unroll
                for (int j = 0; j < V; j += 2) {
                    const float2 g = value<LA_ACT_SILU>(make_float2(z.f[j], z.f[j + 1]));
                    dy[j] = o.f[j] * g.x, dy[j + 1] = o.f[j + 1] * g.y;
                }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    dy[j] = o.f[j];
            }
            put(&w.dy[t][c], dy);
        }
    }
    for (int i = threadIdx.x; i < SUB * NS; i += kThreads) {
        w.B[0][i] = both(to_f32(raw.B[t0][i]));
        if constexpr (GRAD)
            w.C[0][i] = both(to_f32(raw.C[t0][i]));
    }
}

__device__ __forceinline__ void zero_quad(float2 (&h)[2][4])
{
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int s = 0; s < 4; ++s)
            h[p][s] = make_float2(0.f, 0.f);
}

// Per segment: end of the state from zero, product of the decays, and sum over its
// tokens of (the decays up to t) C_t dy_t, the gradient in front of it.
template <typename T, int NS, bool ASYNC>
__global__ void __launch_bounds__(kThreads)
    k_ssm_ends(GradIns in, float* __restrict__ ends, float* __restrict__ decays, float* __restrict__ fronts, Grid q)
{
    using L = Lay<NS>;
    extern __shared__ __align__(16) unsigned char smem[];
    auto& sm = *reinterpret_cast<EndsSmem<T, NS>*>(smem);
    const Place at = place_of(q, blockIdx.x, L::CT);
    const int64_t len = row_length(in.lengths, at.b, q.N), first = (int64_t)at.seg * q.seg_len;
    const int live = (int)max((int64_t)0, min((int64_t)q.seg_len, len - first));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c4 = (warp * L::QPW + lane / L::LPC) * 4, s4 = lane % L::LPC * 4;
    const int have = max(0, min(4, at.valid - c4));
    float2 A2[2][4], h[2][4], G[2][4], P[2][4];
    load_quad<NS>(in.A + (at.c0 + c4) * (int64_t)NS + s4, have, A2);
    zero_quad(h);
    zero_quad(G);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int s = 0; s < 4; ++s)
            A2[p][s] = mul2(A2[p][s], both(kLog2e)), P[p][s] = make_float2(1.f, 1.f);
    if (live > 0)
        load_segment<T, NS, ASYNC>(sm.raw, in, at, first, live);
    for (int t0 = 0; t0 < live; t0 += Seg<NS>::SUB) {
        if (t0)
            __syncthreads();
        widen<T, NS, true>(sm.raw, sm.w, in, at, t0, live);
        __syncthreads();
#pragma unroll 4
        for (int t = 0; t < Seg<NS>::SUB; ++t) {
            const float4 dt = *reinterpret_cast<const float4*>(&sm.w.dt[t][c4]);
            const float4 u = *reinterpret_cast<const float4*>(&sm.w.u[t][c4]);
            const float4 dy = *reinterpret_cast<const float4*>(&sm.w.dy[t][c4]);
            const Four B = twice(&sm.w.B[t][s4]), Cr = twice(&sm.w.C[t][s4]);
            const float2 d[2] = {{dt.x, dt.y}, {dt.z, dt.w}}, v[2] = {{u.x, u.y}, {u.z, u.w}};
            const float2 y[2] = {{dy.x, dy.y}, {dy.z, dy.w}};
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float2 a = decay(d[p], A2[p][s]);
                    h[p][s] = fma2(a, h[p][s], mul2(v[p], B.s[s]));
                    P[p][s] = mul2(P[p][s], a);
                    G[p][s] = fma2(P[p][s], mul2(y[p], Cr.s[s]), G[p][s]);
                }
        }
    }
    const int64_t kept = ((at.b * q.segs + at.seg) * (int64_t)q.C + at.c0 + c4) * NS + s4;
    store_quad<NS>(ends + kept, have, h);
    store_quad<NS>(decays + kept, have, P);
    store_quad<NS>(fronts + kept, have, G);
}

// In place: ends -> starts of the segments, fronts -> gradients at their ends.
__global__ void __launch_bounds__(256)
    k_ssm_join_grad(const float* __restrict__ S0, const float* __restrict__ dS_out, float* __restrict__ ends,
                    const float* __restrict__ decays, float* __restrict__ fronts, float* __restrict__ dS0, int segs,
                    int64_t row, int64_t items)
{
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (item >= items)
        return;
    constexpr int kAhead = 8;
    const bool back = blockIdx.y;
    const int64_t b = item / row, e = item - b * row;  // e: four states of [C][n]
    const float4* init = reinterpret_cast<const float4*>(back ? dS_out : S0);
    float4 S = init ? init[item] : make_float4(0.f, 0.f, 0.f, 0.f);
    float4* p = reinterpret_cast<float4*>(back ? fronts : ends) + b * segs * row + e;
    const float4* d = reinterpret_cast<const float4*>(decays) + b * segs * row + e;
    for (int i = 0; i < segs; i += kAhead) {
        float4 E[kAhead], P[kAhead];
        auto at = [&](int k) { return (int64_t)(back ? segs - 1 - i - k : i + k) * row; };
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k < segs)
                E[k] = p[at(k)], P[k] = d[at(k)];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k < segs) {
                p[at(k)] = S;
                S.x = fmaf(P[k].x, S.x, E[k].x);
                S.y = fmaf(P[k].y, S.y, E[k].y);
                S.z = fmaf(P[k].z, S.z, E[k].z);
                S.w = fmaf(P[k].w, S.w, E[k].w);
            }
    }
    if (back && dS0)
        reinterpret_cast<float4*>(dS0)[item] = S;
}

// Eight values summed over the warp's quads (lanes of equal lane % LPC): halves are
// traded, so that v[0 ..] ends with the sums of values first .. first + count - 1.
template <int LPC>
__device__ __forceinline__ int sum_quads(float (&v)[8], int lane)
{
    int first = 0, half = 4;
#pragma unroll
    for (int o = 16; o >= LPC; o /= 2) {
        if (half == 0) {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
            continue;
        }
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < half) {
                const float give = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        first += up ? half : 0;
        half /= 2;
    }
    return first;
}

struct Outs {
    void *dx, *ddelta, *dz;
    float *rows;           // [channel tile of a group][B][N][G][2][n]: parts of dB and dC
    float *dA, *dD, *dbias;  // [B * segs][C][n], [B * segs][C], [B * segs][C]
};

template <typename T, int NS, bool ASYNC>
__global__ void __launch_bounds__(kThreads)
    k_ssm_grad(GradIns in, const float* __restrict__ starts, const float* __restrict__ finals, Outs out, Grid q)
{
    using L = Lay<NS>;
    constexpr int SUB = Seg<NS>::SUB, BLK = Seg<NS>::BLK;
    extern __shared__ __align__(16) unsigned char smem[];
    auto& sm = *reinterpret_cast<GradSmem<T, NS>*>(smem);
    const Place at = place_of(q, blockIdx.x, L::CT);
    const int64_t len = row_length(in.lengths, at.b, q.N), first = (int64_t)at.seg * q.seg_len;
    const int here = (int)min((int64_t)q.seg_len, q.N - first);  // tokens of the segment
    const int live = (int)max((int64_t)0, min((int64_t)here, len - first));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c4 = (warp * L::QPW + lane / L::LPC) * 4, s4 = lane % L::LPC * 4;
    const int have = max(0, min(4, at.valid - c4));
    const int64_t C = q.C;
    const int co = L::LPC == 2 ? c4 + (lane & 1) * 2 : c4 + (lane & 3);  // the channels this lane finishes
    bool mine[L::OWN];
    float Dv[L::OWN], bias[L::OWN], dD[L::OWN], dbias[L::OWN];
#pragma unroll
    for (int i = 0; i < L::OWN; ++i) {
        mine[i] = co + i < at.valid && s4 < 16;
        Dv[i] = mine[i] && in.D ? in.D[at.c0 + co + i] : 0.0f;
        bias[i] = mine[i] && in.bias ? in.bias[at.c0 + co + i] : 0.0f;
        dD[i] = dbias[i] = 0.0f;
    }
    const int64_t seg = at.b * q.segs + at.seg;
    const int64_t kept = (seg * C + at.c0 + c4) * NS + s4;
    float2 A2[2][4], h[2][4], ag[2][4], dA[2][4];
    load_quad<NS>(in.A + (at.c0 + c4) * (int64_t)NS + s4, have, A2);
    load_quad<NS>(starts + kept, have, h);
    load_quad<NS>(finals + kept, have, ag);
    zero_quad(dA);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int s = 0; s < 4; ++s)
            A2[p][s] = mul2(A2[p][s], both(kLog2e));
    const int64_t row0 = at.b * q.N + first;
    T* dx = static_cast<T*>(out.dx) + row0 * C + at.c0;
    T* ddelta = static_cast<T*>(out.ddelta) + row0 * C + at.c0;
    T* dz = in.z.p ? static_cast<T*>(out.dz) + row0 * C + at.c0 : nullptr;
    const int64_t wide_rows = (int64_t)q.G * 2 * NS;
    float* parts = out.rows + ((int64_t)(at.tile - at.g * q.per_group) * q.B * q.N + row0) * wide_rows + at.g * 2 * NS;

    if (live > 0)
        load_segment<T, NS, ASYNC>(sm.raw, in, at, first, live);
    const int subs = (live + SUB - 1) / SUB;
    // forwards: the state before every fourth token
    for (int k = 0; k < subs; ++k) {
        if (k)
            __syncthreads();
        widen<T, NS, false>(sm.raw, sm.w, in, at, k * SUB, live);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < SUB; ++t) {
            if (t % BLK == 0 && k + t > 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sm.kept[(k * SUB + t) / BLK - 1][i][threadIdx.x] =
                        make_float4(h[i / 2][i % 2 * 2].x, h[i / 2][i % 2 * 2].y, h[i / 2][i % 2 * 2 + 1].x,
                                    h[i / 2][i % 2 * 2 + 1].y);
            }
            step(*reinterpret_cast<const float4*>(&sm.w.dt[t][c4]), *reinterpret_cast<const float4*>(&sm.w.u[t][c4]),
                 twice(&sm.w.B[t][s4]), A2, h);
        }
    }
    // and back
    for (int k = subs - 1; k >= 0; --k) {
        __syncthreads();
        widen<T, NS, true>(sm.raw, sm.w, in, at, k * SUB, live);
        __syncthreads();
#pragma unroll 1
        for (int blk = SUB / BLK - 1; blk >= 0; --blk) {
            float2 base[2][4], a[BLK][2][4], hs[BLK][2][4];
            if (k + blk > 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 v = sm.kept[k * (SUB / BLK) + blk - 1][i][threadIdx.x];
                    base[i / 2][i % 2 * 2] = make_float2(v.x, v.y), base[i / 2][i % 2 * 2 + 1] = make_float2(v.z, v.w);
                }
            } else {
                load_quad<NS>(starts + kept, have, base);
            }
#pragma unroll
            for (int j = 0; j < BLK; ++j) {
                const int t = blk * BLK + j;
                const float4 dt = *reinterpret_cast<const float4*>(&sm.w.dt[t][c4]);
                const float4 u = *reinterpret_cast<const float4*>(&sm.w.u[t][c4]);
                const Four B = twice(&sm.w.B[t][s4]);
                const float2 d[2] = {{dt.x, dt.y}, {dt.z, dt.w}}, v[2] = {{u.x, u.y}, {u.z, u.w}};
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        a[j][p][s] = decay(d[p], A2[p][s]);
                        hs[j][p][s] = fma2(a[j][p][s], j ? hs[j ? j - 1 : 0][p][s] : base[p][s], mul2(v[p], B.s[s]));
                    }
            }
#pragma unroll
            for (int j = BLK - 1; j >= 0; --j) {
                const int t = blk * BLK + j, ts = k * SUB + t;
                const float4 dt = *reinterpret_cast<const float4*>(&sm.w.dt[t][c4]);
                const float4 u = *reinterpret_cast<const float4*>(&sm.w.u[t][c4]);
                const float4 dy = *reinterpret_cast<const float4*>(&sm.w.dy[t][c4]);
                const Four B = twice(&sm.w.B[t][s4]), Cr = twice(&sm.w.C[t][s4]);
                const float2 d[2] = {{dt.x, dt.y}, {dt.z, dt.w}}, v[2] = {{u.x, u.y}, {u.z, u.w}};
                const float2 e[2] = {{dy.x, dy.y}, {dy.z, dy.w}};
                float2 y[2], w[2], ddt[2], dB[4], dC[4];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    y[p] = w[p] = ddt[p] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const float2 g = fma2(e[p], Cr.s[s], ag[p][s]);
                        w[p] = fma2(g, B.s[s], w[p]);
                        dB[s] = p ? fma2(g, v[p], dB[s]) : mul2(g, v[p]);
                        dC[s] = p ? fma2(e[p], hs[j][p][s], dC[s]) : mul2(e[p], hs[j][p][s]);
                        y[p] = fma2(hs[j][p][s], Cr.s[s], y[p]);
                        ag[p][s] = mul2(a[j][p][s], g);
                        const float2 qt = mul2(ag[p][s], j ? hs[j ? j - 1 : 0][p][s] : base[p][s]);
                        ddt[p] = fma2(qt, A2[p][s], ddt[p]);
                        dA[p][s] = fma2(qt, d[p], dA[p][s]);
                    }
                }
                float wo[L::OWN], to[L::OWN], yo[L::OWN];
                sum_states<L::LPC>(w, lane, wo);
                sum_states<L::LPC>(ddt, lane, to);
                if (dz)
                    sum_states<L::LPC>(y, lane, yo);
                float r[8];
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    r[s] = dB[s].x + dB[s].y, r[4 + s] = dC[s].x + dC[s].y;
                const int r0 = sum_quads<L::LPC>(r, lane);
                constexpr int count = L::QPW >= 8 ? 1 : 8 / L::QPW;
                if (L::QPW < 16 || !(lane & L::LPC)) {
#pragma unroll
                    for (int i = 0; i < count; ++i) {
                        const int n = r0 + i;
                        sm.sums[warp][t][(n & 4 ? NS : 0) + s4 + (n & 3)] = r[i];
                    }
                }
#pragma unroll
                for (int i = 0; i < L::OWN; ++i) {
                    if (!mine[i] || ts >= here)
                        continue;
                    const int64_t o = ts * C + co + i;
                    float vx = 0.f, vd = 0.f, vz = 0.f;
                    if (ts < live) {
                        const float x = to_f32(sm.raw.x[ts][co + i]), dyo = sm.w.dy[t][co + i];
                        // the slopes of the step and of the gate, side by side
                        const float zr = dz ? to_f32(sm.raw.z[ts][co + i]) : 0.f;
                        const Sigmoid sg = sigmoid(make_float2(to_f32(sm.raw.delta[ts][co + i]) + bias[i], zr));
                        const float slope = in.softplus ? sg.s.x : 1.0f;
                        vx = fmaf(sm.w.dt[t][co + i], wo[i], Dv[i] * dyo);
                        vd = fmaf(x, wo[i], to[i] * 0.6931471805599453f) * slope;
                        dD[i] = fmaf(dyo, x, dD[i]);
                        dbias[i] += vd;
                        if (dz)
                            vz = to_f32(sm.raw.dout[ts][co + i]) * fmaf(Dv[i], x, yo[i]) * sg.s.y *
                                 fmaf(sg.u.y, sg.rest.y, 1.0f);
                    }
                    dx[o] = from_f32<T>(vx);
                    ddelta[o] = from_f32<T>(vd);
                    if (dz)
                        dz[o] = from_f32<T>(vz);
                }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < SUB * 2 * NS; i += kThreads) {
            const int t = i / (2 * NS), n = i - t * 2 * NS;
            if (k * SUB + t < here) {
                float s = sm.sums[0][t][n];
#pragma unroll
                for (int w = 1; w < kWarps; ++w)
                    s += sm.sums[w][t][n];
                parts[(k * SUB + t) * wide_rows + n] = s;
            }
        }
    }
    // tokens behind the row's last, whole sub-tiles of them
    for (int i = threadIdx.x; i < (here - min(here, subs * SUB)) * at.valid; i += kThreads) {
        const int t = subs * SUB + i / at.valid;
        const int64_t o = t * C + i % at.valid;
        dx[o] = from_f32<T>(0.0f);
        ddelta[o] = from_f32<T>(0.0f);
        if (dz)
            dz[o] = from_f32<T>(0.0f);
    }
    for (int i = threadIdx.x; i < (here - min(here, subs * SUB)) * 2 * NS; i += kThreads)
        parts[(subs * SUB + i / (2 * NS)) * wide_rows + i % (2 * NS)] = 0.0f;
    store_quad<NS>(out.dA + kept, have, dA);
#pragma unroll
    for (int i = 0; i < L::OWN; ++i)
        if (mine[i]) {
            out.dD[seg * C + at.c0 + co + i] = dD[i];
            out.dbias[seg * C + at.c0 + co + i] = dbias[i];
        }
}

// dB, dC [rows][G][n] from the channel tiles' parts [tile][rows][G][2][n].
template <typename T>
__global__ void __launch_bounds__(256)
    k_ssm_rows(const float* __restrict__ parts, T* __restrict__ dB, T* __restrict__ dC, int tiles, int NS, int64_t items)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= items)
        return;
    float s = 0.f;
    for (int k = 0; k < tiles; ++k)
        s += parts[k * items + i];
    const int64_t pair = i / NS;
    (pair & 1 ? dC : dB)[pair / 2 * NS + i % NS] = from_f32<T>(s);
}

// out[col] = sum over the rows of part[row][col], 32 columns x 8 partial sums a block.
__global__ void __launch_bounds__(256)
    k_ssm_columns(const float* __restrict__ part, float* __restrict__ out, int64_t rows, int64_t cols)
{
    __shared__ float sums[8][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float x = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (int64_t r = grp; r < rows; r += 8)
            x += part[r * cols + c];
    }
    sums[grp][lane] = x;
    __syncthreads();
    if (grp == 0 && c < cols) {
        x = 0.f;
        for (int i = 0; i < 8; ++i)
            x += sums[i][lane];
        out[c] = x;
    }
}

template <int NS>
Grid grid_of(const SsmArgs& a)
{
    Grid q;
    q.B = a.B, q.N = a.N, q.C = (int)a.C, q.G = (int)a.G;
    q.per_group = (int)((a.C / a.G + Lay<NS>::CT - 1) / Lay<NS>::CT);
    q.seg_len = Seg<NS>::LEN;
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

// The workspace, in floats: states at the segments' starts, their decays (later the
// parts of dA), gradients at their ends, parts of dD and dbias, parts of dB and dC.
struct Space {
    int64_t state, chan, rows;
    Space(const SsmArgs& a, const Grid& q)
        : state(a.B * q.segs * a.C * a.n), chan(a.B * q.segs * a.C), rows(q.per_group * a.B * a.N * a.G * 2 * a.n)
    {
        chan = (chan + 3) / 4 * 4;
    }
    int64_t floats() const { return 3 * state + 2 * chan + rows; }
};

cudaError_t sum_columns(const float* part, float* out, int64_t rows, int64_t cols, cudaStream_t st)
{
    if (!out)
        return cudaSuccess;
    k_ssm_columns<<<(unsigned)((cols + 31) / 32), 256, 0, st>>>(part, out, rows, cols);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, int NS, bool ASYNC>
cudaError_t run_grad(const SsmArgs& a, const GradIns& in, const Grid& q)
{
    const Space sp(a, q);
    float* ends = static_cast<float*>(a.ws);
    float *decays = ends + sp.state, *fronts = decays + sp.state, *dD = fronts + sp.state, *dbias = dD + sp.chan;
    float* rows = dbias + sp.chan;
    const unsigned blocks = (unsigned)(a.B * q.segs * q.G * q.per_group);
    cudaError_t e = cudaFuncSetAttribute(k_ssm_ends<T, NS, ASYNC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(EndsSmem<T, NS>));
    if (e != cudaSuccess)
        return e;
    k_ssm_ends<T, NS, ASYNC>
        <<<blocks, kThreads, sizeof(EndsSmem<T, NS>), a.stream>>>(in, ends, decays, fronts, q);
    count_launches(1);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    const int64_t row = a.C * NS / 4, items = a.B * row;
    k_ssm_join_grad<<<dim3((unsigned)((items + 255) / 256), 2), 256, 0, a.stream>>>(
        a.S0, a.dS_out, ends, decays, fronts, a.dS0, q.segs, row, items);
    count_launches(1);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    e = cudaFuncSetAttribute(k_ssm_grad<T, NS, ASYNC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(GradSmem<T, NS>));
    if (e != cudaSuccess)
        return e;
    k_ssm_grad<T, NS, ASYNC><<<blocks, kThreads, sizeof(GradSmem<T, NS>), a.stream>>>(
        in, ends, fronts, Outs{a.dx, a.ddelta, a.dz, rows, decays, dD, dbias}, q);
    count_launches(1);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    const int64_t values = a.B * a.N * a.G * 2 * NS;
    k_ssm_rows<T><<<(unsigned)((values + 255) / 256), 256, 0, a.stream>>>(rows, static_cast<T*>(a.dB),
                                                                         static_cast<T*>(a.dC), q.per_group, NS, values);
    count_launches(1);
    if ((e = cudaGetLastError()) != cudaSuccess ||
        (e = sum_columns(decays, a.dA, a.B * q.segs, a.C * NS, a.stream)) != cudaSuccess ||
        (e = sum_columns(dD, a.dD, a.B * q.segs, a.C, a.stream)) != cudaSuccess)
        return e;
    return sum_columns(dbias, a.dbias, a.B * q.segs, a.C, a.stream);
}

template <typename T, int NS>
cudaError_t grad_rows(const SsmArgs& a)
{
    const GradIns in{{a.x, a.x_batch, a.x_token}, {a.delta, a.delta_batch, a.delta_token},
                     {a.Bm, a.B_batch, a.B_token}, {a.Cm, a.C_batch, a.C_token}, {a.z, a.z_batch, a.z_token},
                     {a.dout, a.dout_batch, a.dout_token}, a.A, a.D, a.bias, a.lengths, a.softplus};
    bool async = a.C / a.G * (int)sizeof(T) % 16 == 0;
    for (const Rows& r : {in.x, in.delta, in.B, in.C, in.z, in.dout})
        async = async && (!r.p || rows_on(r.p, r.batch, r.token, (int)sizeof(T), 16));
    const Grid q = grid_of<NS>(a);
    return async ? run_grad<T, NS, true>(a, in, q) : run_grad<T, NS, false>(a, in, q);
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
