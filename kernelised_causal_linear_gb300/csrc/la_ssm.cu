// la_ssm.cu -- the selective state-space scan: forward over whole sequences and one
// token for every sequence.
//
// The recurrence is exact, token after token in fp32, with no products of decays
// kept.  Few long sequences are cut into segments: k_ssm<END> runs each from a zero
// state for its end, k_ssm_join walks the ends (the decay of a segment is exp(A sum
// dt)), and k_ssm runs every segment again from its true start.
#include "la_ssm.cuh"

namespace la {
namespace ssm {
namespace {

using namespace rows;

template <typename T, int NS, bool END>
struct Tiles {
    using L = Lay<NS>;
    // raw tiles, two of each: the next one is on its way while this one is used
    T x[2][L::TT][L::CT], delta[2][L::TT][L::CT], z[END ? 1 : 2][END ? 1 : L::TT][END ? 8 : L::CT];
    T B[2][L::TT][NS], C[2][L::TT][NS];
    // in use, fp32
    float dt[L::TT][L::CT], u[L::TT][L::CT], Bf[L::TT][NS], Cf[END ? 1 : L::TT][NS];
};

struct Ins {
    Rows x, delta, B, C, z;
    const float *A, *D, *bias;
    const int* lengths;
    int softplus;
};

// END: the state after each segment from a zero start (ends) and the sum of its steps
// (sums).  Else the outputs, from S0 or (segments) from `ends`, which then holds starts.
template <typename T, int NS, bool END, bool ASYNC>
__global__ void __launch_bounds__(kThreads)
    k_ssm(Ins in, T* __restrict__ out, const float* S0, float* S_out, float* __restrict__ ends,
          float* __restrict__ sums, Grid q)
{
    using L = Lay<NS>;
    constexpr int TT = L::TT, CT = L::CT, V = 16 / (int)sizeof(T);
    extern __shared__ __align__(16) unsigned char smem[];
    auto& sm = *reinterpret_cast<Tiles<T, NS, END>*>(smem);
    const Place at = place_of<NS>(q, blockIdx.x);
    const int64_t len = row_length(in.lengths, at.b, q.N);
    const int64_t first = (int64_t)at.seg * q.seg_len, end = min(q.N, first + q.seg_len);
    const int live = (int)max((int64_t)0, min(end, len) - first);  // tokens of this segment that the row has
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c4 = (warp * L::QPW + lane / L::LPC) * 4, s4 = lane % L::LPC * 4;  // quad and states
    const int have = max(0, min(4, at.valid - c4));
    const int64_t C = q.C;

    float2 A2[2][4], h[2][4], sum[2] = {}, low[2] = {};
    load_quad<NS>(in.A + (at.c0 + c4) * (int64_t)NS + s4, have, A2);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int s = 0; s < 4; ++s)
            A2[p][s] = mul2(A2[p][s], both(kLog2e)), h[p][s] = make_float2(0.f, 0.f);
    const int64_t state = (at.b * C + at.c0 + c4) * NS + s4;
    const int64_t kept = ((at.b * q.segs + at.seg) * C + at.c0 + c4) * NS + s4;
    if (!END) {
        if (q.segs > 1)
            load_quad<NS>(ends + kept, have, h);
        else if (S0)
            load_quad<NS>(S0 + state, have, h);
    }
    // the channels whose sums end in this lane
    const int co = L::LPC == 2 ? c4 + (lane & 1) * 2 : c4 + (lane & 3);
    float Dv[L::OWN];
    bool mine[L::OWN];
#pragma unroll
    for (int i = 0; i < L::OWN; ++i) {
        mine[i] = !END && co + i < at.valid && s4 < 16;
        Dv[i] = mine[i] && in.D ? in.D[at.c0 + co + i] : 0.0f;
    }

    const T* xs = static_cast<const T*>(in.x.p) + at.b * in.x.batch + at.c0;
    const T* ds = static_cast<const T*>(in.delta.p) + at.b * in.delta.batch + at.c0;
    const T* zs = in.z.p && !END ? static_cast<const T*>(in.z.p) + at.b * in.z.batch + at.c0 : nullptr;
    const T* Bs = static_cast<const T*>(in.B.p) + at.b * in.B.batch + at.g * NS;
    const T* Cs = static_cast<const T*>(in.C.p) + at.b * in.C.batch + at.g * NS;
    auto load = [&](int tile) {
        const int k = tile & 1;
        const int64_t t0 = first + (int64_t)tile * TT;
        const int n = min(TT, live - tile * TT);
        copy_tile<T, TT, CT, ASYNC>(sm.x[k][0], xs + t0 * in.x.token, in.x.token, n, at.valid);
        copy_tile<T, TT, CT, ASYNC>(sm.delta[k][0], ds + t0 * in.delta.token, in.delta.token, n, at.valid);
        copy_tile<T, TT, NS, ASYNC>(sm.B[k][0], Bs + t0 * in.B.token, in.B.token, n, NS);
        if constexpr (!END) {
            copy_tile<T, TT, NS, ASYNC>(sm.C[k][0], Cs + t0 * in.C.token, in.C.token, n, NS);
            if (zs)
                copy_tile<T, TT, CT, ASYNC>(sm.z[k][0], zs + t0 * in.z.token, in.z.token, n, at.valid);
        }
        cp_commit();
    };

    const int tiles = (live + TT - 1) / TT;
    if (tiles > 0)
        load(0);
    for (int tile = 0; tile < tiles; ++tile) {
        const int k = tile & 1, n = min(TT, live - tile * TT);
        cp_wait<0>();
        __syncthreads();  // this tile is there, and the last one is no longer read
        if (tile + 1 < tiles)
            load(tile + 1);
        // dt and u = dt x in fp32; tokens behind the last have dt = 0
#pragma unroll
        for (int i = threadIdx.x; i < TT * CT / V; i += kThreads) {
            const int t = i / (CT / V), c = i % (CT / V) * V;
            Raw<T, V> rd, rx;
            rd.w = *reinterpret_cast<const decltype(rd.w)*>(&sm.delta[k][t][c]);
            rx.w = *reinterpret_cast<const decltype(rx.w)*>(&sm.x[k][t][c]);
            const Vec<V> d = wide(rd), x = wide(rx);
            float dt[V], u[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float raw = d.f[j] + (in.bias && c + j < at.valid ? __ldg(in.bias + at.c0 + c + j) : 0.0f);
                dt[j] = t < n ? (in.softplus ? softplus(raw) : raw) : 0.0f;
                u[j] = dt[j] * x.f[j];
            }
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                *reinterpret_cast<float4*>(&sm.dt[t][c + j]) = make_float4(dt[j], dt[j + 1], dt[j + 2], dt[j + 3]);
                *reinterpret_cast<float4*>(&sm.u[t][c + j]) = make_float4(u[j], u[j + 1], u[j + 2], u[j + 3]);
            }
        }
        for (int i = threadIdx.x; i < TT * NS; i += kThreads) {
            sm.Bf[0][i] = to_f32(sm.B[k][0][i]);
            if constexpr (!END)
                sm.Cf[0][i] = to_f32(sm.C[k][0][i]);
        }
        __syncthreads();
        T* po = out + (at.b * q.N + first + (int64_t)tile * TT) * C + at.c0 + co;
        float2 part[2] = {};
#pragma unroll 4
        for (int t = 0; t < TT; ++t) {
            const float4 dt = *reinterpret_cast<const float4*>(&sm.dt[t][c4]);
            const float4 u = *reinterpret_cast<const float4*>(&sm.u[t][c4]);
            const float4 B = *reinterpret_cast<const float4*>(&sm.Bf[t][s4]);
            step(dt, u, B, A2, h);
            if constexpr (END) {
                part[0] = add2(part[0], make_float2(dt.x, dt.y));
                part[1] = add2(part[1], make_float2(dt.z, dt.w));
            } else {
                const float4 Cr = *reinterpret_cast<const float4*>(&sm.Cf[t][s4]);
                float2 y[2];
                float own[L::OWN];
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    y[p] = fma2(h[p][3], both(Cr.w), fma2(h[p][2], both(Cr.z), fma2(h[p][1], both(Cr.y),
                                mul2(h[p][0], both(Cr.x)))));
                sum_states<L::LPC>(y, lane, own);
#pragma unroll
                for (int i = 0; i < L::OWN; ++i) {
                    float o = fmaf(Dv[i], to_f32(sm.x[k][t][co + i]), own[i]);
                    if (zs)
                        o *= activate(to_f32(sm.z[k][t][co + i]), LA_ACT_SILU).x;
                    if (mine[i] && t < n)
                        po[t * C + i] = from_f32<T>(o);
                }
            }
        }
        if constexpr (END) {
            // the tiles' sums with what their addition loses kept beside
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const float2 s = add2(sum[p], part[p]);
                low[p].x += (sum[p].x - s.x) + part[p].x;
                low[p].y += (sum[p].y - s.y) + part[p].y;
                sum[p] = s;
            }
        }
    }
    if constexpr (END) {
        store_quad<NS>(ends + kept, have, h);
        if (s4 == 0) {
            const float f[4] = {sum[0].x + low[0].x, sum[0].y + low[0].y, sum[1].x + low[1].x, sum[1].y + low[1].y};
            for (int i = 0; i < have; ++i)
                sums[(at.b * q.segs + at.seg) * C + at.c0 + c4 + i] = f[i];
        }
    } else {
        // outputs behind the row's last token
        for (int64_t i = threadIdx.x + (int64_t)live * at.valid; i < (end - first) * at.valid; i += kThreads) {
            const int64_t t = i / at.valid;
            out[(at.b * q.N + first + t) * C + at.c0 + (i - t * at.valid)] = from_f32<T>(0.0f);
        }
        if (S_out && at.seg == q.segs - 1)
            store_quad<NS>(S_out + state, have, h);
    }
}

// ends -> starts in place, one thread per four states; rows in flight ahead of the chain.
__global__ void __launch_bounds__(256)
    k_ssm_join(const float* __restrict__ A, const float* S0, float* __restrict__ ends, const float* __restrict__ sums,
               int segs, int64_t C, int NS, int64_t items)
{
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (item >= items)
        return;
    const int64_t row = C * NS / 4, b = item / row, e = item - b * row;  // e: four states of [C][n]
    const int64_t c = e * 4 / NS;
    const float4 a = reinterpret_cast<const float4*>(A)[e];
    float4 S = S0 ? reinterpret_cast<const float4*>(S0)[item] : make_float4(0.f, 0.f, 0.f, 0.f);
    float4* p = reinterpret_cast<float4*>(ends) + b * segs * row + e;
    const float* d = sums + b * segs * C + c;
    constexpr int kAhead = 8;
    for (int i = 0; i < segs; i += kAhead) {
        float4 E[kAhead];
        float sd[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k < segs)
                E[k] = p[(i + k) * row], sd[k] = d[(i + k) * C] * kLog2e;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k < segs) {
                p[(i + k) * row] = S;
                S.x = fmaf(ex2(a.x * sd[k]), S.x, E[k].x);
                S.y = fmaf(ex2(a.y * sd[k]), S.y, E[k].y);
                S.z = fmaf(ex2(a.z * sd[k]), S.z, E[k].z);
                S.w = fmaf(ex2(a.w * sd[k]), S.w, E[k].w);
            }
    }
}

// One token: n / 4 lanes per channel, four states each; bound by the state's bytes.
struct StepIns {
    Rows x, delta, B, C, z;  // .batch: from row to row
    const float *A, *D, *bias;
    int softplus;
};

template <typename T, int NS>
__global__ void __launch_bounds__(256)
    k_ssm_step(float* __restrict__ S, StepIns in, T* __restrict__ out, int64_t C, int64_t per_group, int64_t quads)
{
    constexpr int LPC = NS / 4;
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const bool on = item < quads;  // whole groups of lanes: the sums below need every one
    const int64_t ch = (on ? item : 0) / LPC, b = ch / C, c = ch - b * C, g = c / per_group;
    const int s4 = (int)(item % LPC) * 4;
    float4* sp = reinterpret_cast<float4*>(S + ch * NS + s4);
    float4 h = *sp;
    const float4 a = __ldg(reinterpret_cast<const float4*>(in.A + c * NS + s4));
    const float x = to_f32(static_cast<const T*>(in.x.p)[b * in.x.batch + c]);
    float dt = to_f32(static_cast<const T*>(in.delta.p)[b * in.delta.batch + c]) + (in.bias ? __ldg(in.bias + c) : 0.0f);
    if (in.softplus)
        dt = softplus(dt);
    const T* Bp = static_cast<const T*>(in.B.p) + b * in.B.batch + g * NS + s4;
    const T* Cp = static_cast<const T*>(in.C.p) + b * in.C.batch + g * NS + s4;
    const float u = dt * x, d2 = dt * kLog2e;
    h.x = fmaf(decay(d2, a.x), h.x, u * to_f32(Bp[0]));
    h.y = fmaf(decay(d2, a.y), h.y, u * to_f32(Bp[1]));
    h.z = fmaf(decay(d2, a.z), h.z, u * to_f32(Bp[2]));
    h.w = fmaf(decay(d2, a.w), h.w, u * to_f32(Bp[3]));
    float y = h.x * to_f32(Cp[0]);
    y = fmaf(h.y, to_f32(Cp[1]), y);
    y = fmaf(h.z, to_f32(Cp[2]), y);
    y = fmaf(h.w, to_f32(Cp[3]), y);
#pragma unroll
    for (int o = LPC / 2; o > 0; o >>= 1)
        y += __shfl_xor_sync(0xffffffffu, y, o);
    if (!on)
        return;
    *sp = h;
    if (s4 == 0) {
        if (in.D)
            y = fmaf(__ldg(in.D + c), x, y);
        if (in.z.p)
            y *= activate(to_f32(static_cast<const T*>(in.z.p)[b * in.z.batch + c]), LA_ACT_SILU).x;
        out[b * C + c] = from_f32<T>(y);
    }
}

template <int NS>
Grid grid_of(const SsmArgs& a)
{
    using L = Lay<NS>;
    Grid q;
    q.B = a.B, q.N = a.N, q.C = (int)a.C, q.G = (int)a.G;
    q.per_group = (int)((a.C / a.G + L::CT - 1) / L::CT);
    const int64_t blocks = a.B * q.G * q.per_group, tiles = (a.N + L::TT - 1) / L::TT;
    int64_t segs = 1;
    if (blocks < 152 * 2) {
        segs = (152 * 4 + blocks - 1) / blocks;
        const int64_t most = (tiles + 3) / 4;  // four tiles at least
        segs = segs < most ? segs : most;
    }
    const int64_t per = (tiles + segs - 1) / segs;
    q.seg_len = (int)(per * L::TT), q.segs = (int)((tiles + per - 1) / per);
    return q;
}

template <typename T, int NS>
cudaError_t run_ssm(const SsmArgs& a)
{
    const Grid q = grid_of<NS>(a);
    Ins in{{a.x, a.x_batch, a.x_token}, {a.delta, a.delta_batch, a.delta_token}, {a.Bm, a.B_batch, a.B_token},
           {a.Cm, a.C_batch, a.C_token}, {a.z, a.z_batch, a.z_token}, a.A, a.D, a.bias, a.lengths, a.softplus};
    const int es = (int)sizeof(T);
    const bool async = rows16(a.x, a.x_batch, a.x_token, es) && rows16(a.delta, a.delta_batch, a.delta_token, es) &&
                       rows16(a.Bm, a.B_batch, a.B_token, es) && rows16(a.Cm, a.C_batch, a.C_token, es) &&
                       (!a.z || rows16(a.z, a.z_batch, a.z_token, es)) && a.C / a.G * es % 16 == 0;
    const unsigned blocks = (unsigned)(a.B * q.segs * q.G * q.per_group);
    float* ends = static_cast<float*>(a.ws);
    float* sums = ends + a.B * q.segs * a.C * NS;
    auto launch = [&](auto kernel, size_t bytes) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != cudaSuccess)
            return e;
        kernel<<<blocks, kThreads, bytes, a.stream>>>(in, static_cast<T*>(a.out), a.S0, a.S_out, ends, sums, q);
        count_launches(1);
        return cudaGetLastError();
    };
    if (q.segs > 1) {
        const size_t bytes = sizeof(Tiles<T, NS, true>);
        cudaError_t e = async ? launch(k_ssm<T, NS, true, true>, bytes) : launch(k_ssm<T, NS, true, false>, bytes);
        if (e != cudaSuccess || (e = join_forward(a, q, ends, sums)) != cudaSuccess)
            return e;
    }
    const size_t bytes = sizeof(Tiles<T, NS, false>);
    return async ? launch(k_ssm<T, NS, false, true>, bytes) : launch(k_ssm<T, NS, false, false>, bytes);
}

template <typename T, int NS>
cudaError_t run_step(const SsmArgs& a)
{
    StepIns in{{a.x, a.x_batch, 0}, {a.delta, a.delta_batch, 0}, {a.Bm, a.B_batch, 0}, {a.Cm, a.C_batch, 0},
               {a.z, a.z_batch, 0}, a.A, a.D, a.bias, a.softplus};
    const int64_t quads = a.B * a.C * (NS / 4);
    k_ssm_step<T, NS><<<(unsigned)((quads + 255) / 256), 256, 0, a.stream>>>(a.S_out, in, static_cast<T*>(a.out), a.C,
                                                                            a.C / a.G, quads);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T>
cudaError_t states(const SsmArgs& a, bool step)
{
    switch (a.n) {
    case 8: return step ? run_step<T, 8>(a) : run_ssm<T, 8>(a);
    case 16: return step ? run_step<T, 16>(a) : run_ssm<T, 16>(a);
    case 32: return step ? run_step<T, 32>(a) : run_ssm<T, 32>(a);
    default: return step ? run_step<T, 64>(a) : run_ssm<T, 64>(a);
    }
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

}  // namespace

cudaError_t join_forward(const SsmArgs& a, const Grid& q, float* ends, const float* sums)
{
    const int64_t items = a.B * a.C * a.n / 4;
    k_ssm_join<<<(unsigned)((items + 255) / 256), 256, 0, a.stream>>>(a.A, a.S0, ends, sums, q.segs, a.C, a.n, items);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace ssm

size_t ssm_forward_workspace(const SsmArgs& a)
{
    const ssm::Grid q = ssm::grid_any(a);
    return q.segs == 1 ? 0 : sizeof(float) * (size_t)(a.B * q.segs) * a.C * (a.n + 1);
}

cudaError_t ssm_forward(const SsmArgs& a)
{
    return a.dtype == LA_BF16 ? ssm::states<__nv_bfloat16>(a, false) : ssm::states<float>(a, false);
}

cudaError_t ssm_step(const SsmArgs& a)
{
    return a.dtype == LA_BF16 ? ssm::states<__nv_bfloat16>(a, true) : ssm::states<float>(a, true);
}

}  // namespace la
