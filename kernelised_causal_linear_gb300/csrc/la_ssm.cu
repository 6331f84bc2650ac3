// la_ssm.cu -- the selective state-space scan: forward over whole sequences and one
// token for every sequence.
//
// The recurrence is exact, token after token in fp32, with no products of decays
// kept.  A thread owns two neighbouring channels with up to 16 states each, in pairs of
// states: B and C, the same for every lane, are eight 16-byte reads of shared memory for
// 32 elements, and the sum over the states stays in the thread (n = 32 and 64: two and
// four lanes per channel pair).  What bounds it is arithmetic: an element costs one
// hardware exponential (32 a clock and SM) and four fp32 operations in two-wide instructions,
// which reach some 90 a clock and SM, not 128, where all three operands differ.  Both overlap in
// part: 512 elements take about 150 clocks of a sub-partition, 80 of them of the exponentials'
// unit, those of the steps and the gate among them (B4 N8192 C2048 n = 16 bf16: 277 us, and 188
// us for the run for the ends).  (Four channels times four states per thread, with steps in
// shared memory and shuffles, took 198 clocks.)
//
// Few long sequences are cut into segments: k_ssm<END> runs each from a zero
// state for its end, k_ssm_join walks the ends (the decay of a segment is exp(A sum
// dt)), and k_ssm runs every segment again from its true start.
#include <type_traits>

#include "la_ssm.cuh"

namespace la {
namespace ssm {
namespace {

using namespace rows;

template <typename T, int NS>
struct Cut {
    static constexpr int NT = 64;                   // threads
    static constexpr int SPT = NS < 16 ? NS : 16;   // states of a thread
    static constexpr int LPC = NS / SPT;            // lanes that share a channel pair
    static constexpr int CT = NT / LPC * 2;         // channels of a block
    static constexpr int TT = sizeof(T) == 2 ? 16 : 8;  // tokens of a tile: 4 KB of 128 channels
};

template <typename T, int NS, bool END>
struct Tiles {
    using L = Cut<T, NS>;
    // as they lie in memory, two of each: the next tile is on its way while this one is used
    T x[2][L::TT][L::CT], delta[2][L::TT][L::CT], z[END ? 1 : 2][END ? 1 : L::TT][END ? 8 : L::CT];
    T B[2][L::TT][NS], C[2][L::TT][NS];
    float Bf[L::TT][NS], Cf[END ? 1 : L::TT][NS];
};

struct Ins {
    Rows x, delta, B, C, z;
    const float *A, *D, *bias;
    const int* lengths;
    int softplus;
};

__device__ __forceinline__ float2 two(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 two(const __nv_bfloat16* p)
{
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void put_two(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
__device__ __forceinline__ void put_two(__nv_bfloat16* p, float2 v)
{
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}

// States s0 .. of two channels, [channel][state pair]; channels behind the last are zero
// and not written.
template <int NS, int SPT>
__device__ __forceinline__ void load_pair(const float* p, int have, float2 (&h)[2][SPT / 2])
{
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int s = 0; s < SPT / 2; s += 2) {
            const float4 v = c < have ? *reinterpret_cast<const float4*>(p + c * NS + 2 * s)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
            h[c][s] = make_float2(v.x, v.y), h[c][s + 1] = make_float2(v.z, v.w);
        }
}

template <int NS, int SPT>
__device__ __forceinline__ void store_pair(float* p, int have, const float2 (&h)[2][SPT / 2])
{
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int s = 0; s < SPT / 2; s += 2)
            if (c < have)
                *reinterpret_cast<float4*>(p + c * NS + 2 * s) =
                    make_float4(h[c][s].x, h[c][s].y, h[c][s + 1].x, h[c][s + 1].y);
}

// Registers for eight blocks an SM (128 each): bounds of seven and eight blocks 485 and 484 us, of nine
// and ten 580 (B4 N8192 C2048 n = 16 bf16; fp32 B2 281, 276, 336; n = 8 326, 324, 316; n = 64 B1 508,
// 501, 572).  Shared memory admits eight too, but for the outputs with n = 16 in bf16: 28 KB, seven.
//
// END: the state after each segment but the last from a zero start (ends) and the sum of
// its steps (sums).  Else the outputs, from S0 or (segments) from `ends`, which then holds
// starts.
template <typename T, int NS, bool END, int BYTES>
__global__ void __launch_bounds__(Cut<T, NS>::NT, 8)
    k_ssm(Ins in, T* __restrict__ out, const float* S0, float* S_out, float* __restrict__ ends,
          float* __restrict__ sums, Grid q)
{
    using L = Cut<T, NS>;
    constexpr int NT = L::NT, TT = L::TT, CT = L::CT, SPT = L::SPT, LPC = L::LPC;
    extern __shared__ __align__(16) unsigned char smem[];
    auto& sm = *reinterpret_cast<Tiles<T, NS, END>*>(smem);
    const Place at = place_of(q, blockIdx.x, CT);
    if (END && at.seg == q.segs - 1)
        return;
    const int64_t len = row_length(in.lengths, at.b, q.N);
    const int64_t first = (int64_t)at.seg * q.seg_len, end = min(q.N, first + q.seg_len);
    const int live = (int)max((int64_t)0, min(end, len) - first);  // tokens of this segment that the row has
    const int part = threadIdx.x % LPC, s0 = part * SPT, c2 = threadIdx.x / LPC * 2;
    const int have = max(0, min(2, at.valid - c2));
    const int64_t C = q.C;

    float2 A2[2][SPT / 2], h[2][SPT / 2], sum = {}, low = {};
    load_pair<NS, SPT>(in.A + (at.c0 + c2) * (int64_t)NS + s0, have, A2);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int s = 0; s < SPT / 2; ++s)
            A2[c][s] = mul2(A2[c][s], both(kLog2e)), h[c][s] = make_float2(0.f, 0.f);
    const int64_t state = (at.b * C + at.c0 + c2) * NS + s0;
    const int64_t kept = ((at.b * q.segs + at.seg) * C + at.c0 + c2) * NS + s0;
    if (!END) {
        if (q.segs > 1)
            load_pair<NS, SPT>(ends + kept, have, h);
        else if (S0)
            load_pair<NS, SPT>(S0 + state, have, h);
    }
    auto channels = [&](const float* p) {
        return p ? make_float2(have > 0 ? p[at.c0 + c2] : 0.f, have > 1 ? p[at.c0 + c2 + 1] : 0.f)
                 : make_float2(0.f, 0.f);
    };
    const float2 bias = channels(in.bias), D = channels(in.D);

    const T* xs = static_cast<const T*>(in.x.p) + at.b * in.x.batch + at.c0;
    const T* ds = static_cast<const T*>(in.delta.p) + at.b * in.delta.batch + at.c0;
    const T* zs = in.z.p && !END ? static_cast<const T*>(in.z.p) + at.b * in.z.batch + at.c0 : nullptr;
    const T* Bs = static_cast<const T*>(in.B.p) + at.b * in.B.batch + at.g * NS;
    const T* Cs = static_cast<const T*>(in.C.p) + at.b * in.C.batch + at.g * NS;
    auto load = [&](int tile) {
        const int k = tile & 1;
        const int64_t t0 = first + (int64_t)tile * TT;
        const int n = min(TT, live - tile * TT);
        copy_tile<T, TT, CT, BYTES, NT>(sm.x[k][0], xs + t0 * in.x.token, in.x.token, n, at.valid);
        copy_tile<T, TT, CT, BYTES, NT>(sm.delta[k][0], ds + t0 * in.delta.token, in.delta.token, n, at.valid);
        copy_tile<T, TT, NS, BYTES, NT>(sm.B[k][0], Bs + t0 * in.B.token, in.B.token, n, NS);
        if constexpr (!END) {
            copy_tile<T, TT, NS, BYTES, NT>(sm.C[k][0], Cs + t0 * in.C.token, in.C.token, n, NS);
            if (zs)
                copy_tile<T, TT, CT, BYTES, NT>(sm.z[k][0], zs + t0 * in.z.token, in.z.token, n, at.valid);
        }
        cp_commit();
    };

    const int tiles = (live + TT - 1) / TT;
    if (tiles > 0)
        load(0);
    T* po = out + (at.b * q.N + first) * C + at.c0 + c2;
    for (int tile = 0; tile < tiles; ++tile) {
        const int k = tile & 1, n = min(TT, live - tile * TT);
        cp_wait<0>();
        __syncthreads();  // this tile is there, and the last one is no longer read
        if (tile + 1 < tiles)
            load(tile + 1);
        for (int i = threadIdx.x; i < TT * NS; i += NT) {
            sm.Bf[0][i] = to_f32(sm.B[k][0][i]);
            if constexpr (!END)
                sm.Cf[0][i] = to_f32(sm.C[k][0][i]);
        }
        __syncthreads();
        float2 added = {};
#pragma unroll 2
        for (int t = 0; t < n; ++t, po += C) {
            const float2 x = two(&sm.x[k][t][c2]);
            float2 dt = add2(two(&sm.delta[k][t][c2]), bias);
            if (in.softplus)
                dt = softplus(dt);
            const float2 u = mul2(dt, x);
            const float4* B4 = reinterpret_cast<const float4*>(&sm.Bf[t][s0]);
            const float4* C4 = reinterpret_cast<const float4*>(&sm.Cf[END ? 0 : t][s0]);
            float2 y[2];
#pragma unroll
            for (int s = 0; s < SPT / 2; s += 2) {
                const float4 b = B4[s / 2];
                float4 c;
                if constexpr (!END)
                    c = C4[s / 2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 bi = i ? make_float2(b.z, b.w) : make_float2(b.x, b.y);
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        float2& hs = h[p][s + i];
                        hs = fma2(decay(both(p ? dt.y : dt.x), A2[p][s + i]), hs, mul2(both(p ? u.y : u.x), bi));
                        if constexpr (!END) {
                            const float2 ci = i ? make_float2(c.z, c.w) : make_float2(c.x, c.y);
                            y[p] = s + i ? fma2(hs, ci, y[p]) : mul2(hs, ci);
                        }
                    }
                }
            }
            if constexpr (END) {
                added = add2(added, dt);
            } else if constexpr (LPC == 1) {
                float2 o = fma2(D, x, make_float2(y[0].x + y[0].y, y[1].x + y[1].y));
                if (zs) {
                    const float2 z = two(&sm.z[k][t][c2]);
                    o = mul2(o, value<LA_ACT_SILU>(z));
                }
                if (BYTES >= 2 * (int)sizeof(T) && have == 2) {  // rows of an even number of channels
                    put_two(po, o);
                } else {
                    if (have > 0)
                        po[0] = from_f32<T>(o.x);
                    if (have > 1)
                        po[1] = from_f32<T>(o.y);
                }
            } else {
                // halves are traded: an even lane ends with channel 0, an odd one with channel 1
                const bool odd = part & 1;
                const float y0 = y[0].x + y[0].y, y1 = y[1].x + y[1].y;
                float o = (odd ? y1 : y0) + __shfl_xor_sync(0xffffffffu, odd ? y0 : y1, 1);
                if constexpr (LPC == 4)
                    o += __shfl_xor_sync(0xffffffffu, o, 2);
                o = fmaf(odd ? D.y : D.x, odd ? x.y : x.x, o);
                if (zs)
                    o *= value<LA_ACT_SILU>(both(to_f32(sm.z[k][t][c2 + odd]))).x;
                if (part < 2 && have > odd)
                    po[odd] = from_f32<T>(o);
            }
        }
        if constexpr (END) {
            // the tiles' sums with what their addition loses kept beside
            const float2 s = add2(sum, added);
            low.x += (sum.x - s.x) + added.x;
            low.y += (sum.y - s.y) + added.y;
            sum = s;
        }
    }
    if constexpr (END) {
        store_pair<NS, SPT>(ends + kept, have, h);
        if (part == 0) {
            float* p = sums + (at.b * q.segs + at.seg) * C + at.c0 + c2;
            if (have > 0)
                p[0] = sum.x + low.x;
            if (have > 1)
                p[1] = sum.y + low.y;
        }
    } else {
        // outputs behind the row's last token
        for (int64_t i = threadIdx.x + (int64_t)live * at.valid; i < (end - first) * at.valid; i += NT) {
            const int64_t t = i / at.valid;
            out[(at.b * q.N + first + t) * C + at.c0 + (i - t * at.valid)] = from_f32<T>(0.0f);
        }
        if (S_out && at.seg == q.segs - 1)
            store_pair<NS, SPT>(S_out + state, have, h);
    }
}

// ends -> starts in place, one thread per state: a chain of one product and sum per
// segment, with the loads of sixteen segments ahead of it (18 us for 76 segments of B4 C2048 n = 16;
// eight ahead with four states per thread took 41).
__global__ void __launch_bounds__(128)
    k_ssm_join(const float* __restrict__ A, const float* S0, float* __restrict__ ends, const float* __restrict__ sums,
               int segs, int64_t C, int NS, int64_t items)
{
    const int64_t item = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (item >= items)
        return;
    const int64_t row = C * NS, b = item / row, e = item - b * row;
    const float a = A[e] * kLog2e;
    float S = S0 ? S0[item] : 0.0f;
    float* p = ends + b * segs * row + e;
    const float* d = sums + b * segs * C + e / NS;
    constexpr int kAhead = 16;
    float E[2][kAhead], P[2][kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {  // the last segment's end is not needed
        E[0][k] = k < segs - 1 ? p[k * row] : 0.0f;
        P[0][k] = k < segs - 1 ? d[k * C] : 0.0f;
    }
    for (int i0 = 0; i0 < segs; i0 += 2 * kAhead)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = i0 + half * kAhead;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const bool on = i + kAhead + k < segs - 1;
                E[half ^ 1][k] = on ? p[(i + kAhead + k) * row] : 0.0f;
                P[half ^ 1][k] = on ? d[(i + kAhead + k) * C] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (i + k < segs)
                    p[(i + k) * row] = S;
                S = fmaf(ex2(a * P[half][k]), S, E[half][k]);
            }
        }
}

// One token: n / 4 lanes per channel, four states each, for ROWS rows of the batch with A,
// bias and D loaded once; bound by the state's bytes.
struct StepIns {
    Rows x, delta, B, C, z;  // .batch: from row to row
    const float *A, *D, *bias;
    int softplus, four;      // four: B and C rows allow loads of four
};

template <typename T>
__device__ __forceinline__ Raw<T, 4> four_of(const T* p, bool four)
{
    Raw<T, 4> r;
    if (four) {
        r.w = __ldg(reinterpret_cast<const decltype(r.w)*>(p));
    } else {
        T v[4] = {p[0], p[1], p[2], p[3]};
        memcpy(&r, v, sizeof r);
    }
    return r;
}

// The lanes of a channel share its rows: each reads x, delta and z of one row and finishes that
// row (ROWS <= LPC), and the steps travel by shuffles.
template <typename T, int NS, int ROWS>
__global__ void __launch_bounds__(128)
    k_ssm_step(float* __restrict__ S, StepIns in, T* __restrict__ out, int64_t B, int C, int per_group,
               unsigned across)
{
    constexpr int LPC = NS / 4;
    constexpr unsigned full = 0xffffffffu;
    static_assert(ROWS <= LPC && (ROWS & (ROWS - 1)) == 0, "a row for a lane");
    const unsigned down = blockIdx.x / across;  // `across` blocks hold the channels of ROWS rows
    const int item = (int)(blockIdx.x - down * across) * 128 + threadIdx.x;
    const bool on = item / LPC < C;  // whole groups of lanes: the sums below need every one
    const int c = on ? item / LPC : 0, g = c / per_group, part = item % LPC, s4 = part * 4, mine = part & (ROWS - 1);
    const int64_t b0 = (int64_t)down * ROWS;
    const int live = on ? (int)min((int64_t)ROWS, B - b0) : 0;
    float4* Sp = reinterpret_cast<float4*>(S + (b0 * C + c) * NS + s4);
    const T* Bp = static_cast<const T*>(in.B.p) + b0 * in.B.batch + g * NS + s4;
    const T* Cp = static_cast<const T*>(in.C.p) + b0 * in.C.batch + g * NS + s4;
    float4 h[ROWS];
    Raw<T, 4> Br[ROWS], Cr[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (r < live) {
            h[r] = __ldcs(Sp + (int64_t)r * C * (NS / 4));
            Br[r] = four_of(Bp, in.four);
            Cr[r] = four_of(Cp, in.four);
        } else {
            h[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            Br[r] = Cr[r] = none<T, 4>();
        }
        Bp += in.B.batch, Cp += in.C.batch;
    }
    float x = 0.f, dt = 0.f, z = 0.f;
    if (mine < live) {
        const int64_t b = b0 + mine;
        x = to_f32(static_cast<const T*>(in.x.p)[b * in.x.batch + c]);
        dt = to_f32(static_cast<const T*>(in.delta.p)[b * in.delta.batch + c]);
        if (in.z.p)
            z = to_f32(static_cast<const T*>(in.z.p)[b * in.z.batch + c]);
    }
    const float4 A = __ldg(reinterpret_cast<const float4*>(in.A + (int64_t)c * NS + s4));
    const float2 A2[2] = {mul2(make_float2(A.x, A.y), both(kLog2e)), mul2(make_float2(A.z, A.w), both(kLog2e))};
    if (in.bias)
        dt += __ldg(in.bias + c);
    if (in.softplus)
        dt = softplus(both(dt)).x;
    const float u = dt * x;
    float y[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const float2 d = both(ROWS > 1 ? __shfl_sync(full, dt, r, LPC) : dt);
        const float2 v = both(ROWS > 1 ? __shfl_sync(full, u, r, LPC) : u);
        const Vec<4> Bv = wide(Br[r]), Cv = wide(Cr[r]);
        const float2 lo = fma2(decay(d, A2[0]), make_float2(h[r].x, h[r].y), mul2(v, make_float2(Bv.f[0], Bv.f[1])));
        const float2 hi = fma2(decay(d, A2[1]), make_float2(h[r].z, h[r].w), mul2(v, make_float2(Bv.f[2], Bv.f[3])));
        const float2 p = fma2(hi, make_float2(Cv.f[2], Cv.f[3]), mul2(lo, make_float2(Cv.f[0], Cv.f[1])));
        y[r] = p.x + p.y;
        if (r < live)
            __stcs(Sp + (int64_t)r * C * (NS / 4), make_float4(lo.x, lo.y, hi.x, hi.y));
    }
    // rows are traded, so that a lane ends with the sum of its own
#pragma unroll
    for (int o = ROWS / 2; o > 0; o /= 2) {
        const bool up = part & o;
#pragma unroll
        for (int r = 0; r < o; ++r)
            y[r] = (up ? y[r + o] : y[r]) + __shfl_xor_sync(full, up ? y[r] : y[r + o], o);
    }
#pragma unroll
    for (int o = ROWS; o < LPC; o *= 2)
        y[0] += __shfl_xor_sync(full, y[0], o);
    if (part < ROWS && mine < live) {
        float o = y[0];
        if (in.D)
            o = fmaf(__ldg(in.D + c), x, o);
        if (in.z.p)
            o *= value<LA_ACT_SILU>(both(z)).x;
        out[(b0 + mine) * C + c] = from_f32<T>(o);
    }
}

// Segments.  The run for the ends costs 0.7 of the one that counts, so rows stay whole where they
// alone are more than two and a half blocks an SM.  Whole and cut at N2048, us:
//               320 blocks    384 blocks    448 blocks
//   n = 8       562    411    562    477    562    544   bf16
//   n = 16      762    611    763    724    763    826   bf16     fp32 at 448: 815 and 846
//   n = 32      717    604    719    708    719    796   bf16     fp32        766     835
//   n = 64      802    631    803    746    803    848   bf16     fp32        838     882
// (n = 8 would be cut up to some 470 blocks: 3%.)  Else about four rounds of eight blocks an SM, a tile
// each at least (fp32 B2 N333 C197: whole 92 us, a tile each 18.5; B1 N64 bf16 23 and 18.5).  One,
// two, four and eight rounds, 64 blocks of N8192: n = 16 bf16 509, 497, 484, 485 us; n = 32 961, 894, 914,
// 900; n = 8 312, 322, 324, 320; 32 blocks in fp32 260, 269, 277, 287; 16 blocks 150, 145, 152, 186.
template <typename T, int NS>
Grid grid_of(const SsmArgs& a)
{
    using L = Cut<T, NS>;
    Grid q;
    q.B = a.B, q.N = a.N, q.C = (int)a.C, q.G = (int)a.G;
    q.per_group = (int)((a.C / a.G + L::CT - 1) / L::CT);
    const int64_t blocks = a.B * q.G * q.per_group, tiles = (a.N + L::TT - 1) / L::TT;
    int64_t segs = 1;
    if (blocks < 390) {
        segs = 152 * 8 * 4 / blocks;
        segs = segs < tiles ? segs : tiles;
    }
    const int64_t per = (tiles + segs - 1) / segs;
    q.seg_len = (int)(per * L::TT), q.segs = (int)((tiles + per - 1) / per);
    return q;
}

cudaError_t join_forward(const SsmArgs& a, const Grid& q, float* ends, const float* sums)
{
    const int64_t items = a.B * a.C * a.n;
    k_ssm_join<<<(unsigned)((items + 127) / 128), 128, 0, a.stream>>>(a.A, a.S0, ends, sums, q.segs, a.C, a.n, items);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, int NS>
cudaError_t run_ssm(const SsmArgs& a)
{
    using L = Cut<T, NS>;
    const Grid q = grid_of<T, NS>(a);
    Ins in{{a.x, a.x_batch, a.x_token}, {a.delta, a.delta_batch, a.delta_token}, {a.Bm, a.B_batch, a.B_token},
           {a.Cm, a.C_batch, a.C_token}, {a.z, a.z_batch, a.z_token}, a.A, a.D, a.bias, a.lengths, a.softplus};
    const int es = (int)sizeof(T);
    auto on = [&](unsigned bytes) {
        return rows_on(a.x, a.x_batch, a.x_token, es, bytes) && rows_on(a.delta, a.delta_batch, a.delta_token, es, bytes) &&
               rows_on(a.Bm, a.B_batch, a.B_token, es, bytes) && rows_on(a.Cm, a.C_batch, a.C_token, es, bytes) &&
               (!a.z || rows_on(a.z, a.z_batch, a.z_token, es, bytes)) && a.C / a.G * es % bytes == 0;
    };
    const int bytes = on(16) ? 16 : on(4) ? 4 : 0;
    const unsigned blocks = (unsigned)(a.B * q.segs * q.G * q.per_group);
    float* ends = static_cast<float*>(a.ws);
    float* sums = ends + a.B * q.segs * a.C * NS;
    static_assert(sizeof(Tiles<T, NS, false>) <= 48 * 1024, "shared memory of a launch without attributes");
    auto launch = [&](auto kernel, size_t shared) {
        kernel<<<blocks, L::NT, shared, a.stream>>>(in, static_cast<T*>(a.out), a.S0, a.S_out, ends, sums, q);
        count_launches(1);
        return cudaGetLastError();
    };
    auto run = [&](auto end) {
        constexpr bool END = decltype(end)::value;
        constexpr size_t shared = sizeof(Tiles<T, NS, END>);
        if (bytes == 16)
            return launch(k_ssm<T, NS, END, 16>, shared);
        if constexpr (sizeof(T) == 2)
            if (bytes == 0)
                return launch(k_ssm<T, NS, END, 0>, shared);
        return launch(k_ssm<T, NS, END, 4>, shared);
    };
    if (q.segs > 1) {
        cudaError_t e = run(std::true_type{});
        if (e != cudaSuccess || (e = join_forward(a, q, ends, sums)) != cudaSuccess)
            return e;
    }
    return run(std::false_type{});
}

template <typename T, int NS, int ROWS>
cudaError_t launch_step(const SsmArgs& a, const StepIns& in)
{
    const int64_t across = (a.C * (NS / 4) + 127) / 128;
    k_ssm_step<T, NS, ROWS><<<(unsigned)(across * ((a.B + ROWS - 1) / ROWS)), 128, 0, a.stream>>>(
        a.S_out, in, static_cast<T*>(a.out), a.B, (int)a.C, (int)(a.C / a.G), (unsigned)across);
    count_launches(1);
    return cudaGetLastError();
}

// Four rows a thread (n = 8: two) where that leaves a block for every SM, else one: latency counts.
// C4096 bf16, one row a thread and several: B256 n = 16 35 and 21 us, n = 8 19 and 14; B64 n = 64 35 and
// 21, n = 16 in fp32 12 and 10; B16 and B5 the same.  Right after a flush of L2 23 us, 6.3 TB/s.  (With
// every lane reading all four rows' x, delta and z it took 28 us, of instructions.)
template <typename T, int NS>
cudaError_t run_step(const SsmArgs& a)
{
    const int es = (int)sizeof(T);
    const StepIns in{{a.x, a.x_batch, 0}, {a.delta, a.delta_batch, 0}, {a.Bm, a.B_batch, 0}, {a.Cm, a.C_batch, 0},
                     {a.z, a.z_batch, 0}, a.A, a.D, a.bias, a.softplus,
                     rows_on(a.Bm, a.B_batch, 0, es, 4 * es) && rows_on(a.Cm, a.C_batch, 0, es, 4 * es)};
    return a.B * a.C * (NS / 4) >= 152 * 128 * 4 ? launch_step<T, NS, NS == 8 ? 2 : 4>(a, in) : launch_step<T, NS, 1>(a, in);
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

template <typename T>
Grid grid_any(const SsmArgs& a)
{
    switch (a.n) {
    case 8: return grid_of<T, 8>(a);
    case 16: return grid_of<T, 16>(a);
    case 32: return grid_of<T, 32>(a);
    default: return grid_of<T, 64>(a);
    }
}

}  // namespace

}  // namespace ssm

size_t ssm_forward_workspace(const SsmArgs& a)
{
    const ssm::Grid q = a.dtype == LA_BF16 ? ssm::grid_any<__nv_bfloat16>(a) : ssm::grid_any<float>(a);
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
