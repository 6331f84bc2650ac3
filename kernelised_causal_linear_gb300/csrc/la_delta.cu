// la_delta.cu -- gated delta rule on the CUDA cores: the token recurrence, the
// decode step, the chunked gradient, and the choice of path.
//
// Per value head, with a_t = exp(log_alpha_t), k_t and q_t the rows of the key
// head it reads (L2-normalised with LA_FM_L2):
//
//   e_t = v_t - a_t S_{t-1}^T k_t          what the decayed state gets wrong about v_t
//   S_t = a_t S_{t-1} + beta_t k_t e_t^T,  o_t = scale S_t^T q_t
//
// The columns of S (value channels) never mix: column c needs only v[:, c].
// So a column belongs to one warp for the whole sequence and no token step
// needs a barrier.  The recurrence takes four tokens at a time, with S the state
// before them, A_j = a_1 .. a_j and p_ji = a_{i+1} .. a_j:
//
//   e_j = v_j - A_j S^T k_j - sum_{i < j} p_ji (k_j . k_i) u_i,   u_i = beta_i e_i
//   o_j = scale (A_j S^T q_j + sum_{i <= j} p_ji (q_j . k_i) u_i)
//   S <- A_4 S + sum_j p_4j k_j u_j^T
//
// so that the products with the state do not wait for one another.
#include <math.h>

#include "la_delta.cuh"

namespace la {
namespace {

using delta::both;
using delta::fma2;
using delta::kL2Eps;
using delta::mul2;

// ------------------------------------------------------ token recurrence ----
// 8 warps of 4 columns each; lane = 4 r + c holds rows 4 r .. 4 r + 3 of every
// 32 for column c.  Tokens are staged in blocks of kRecTok, q and k already
// normalised and a group's four tokens by one warp, which leaves their products with
// each other.  A group's eight dots with the state come down in one exchange (sum8),
// and what is left in order is a triangular solve of four scalars.  Bound by the latency
// of that chain: 0.14 us per token at d = 64, 0.18 at 128, two warps per sub-partition
// and 45% of their issue slots used.  (Token by token 0.19 and 0.25; two columns per
// lane, half the reads for twice the exchange, 207 against 182 us at B3 H8 N1000 d = 128.)
constexpr int kGroup = 4;     // tokens taken together
constexpr int kRecThreads = 256;
constexpr int kRecCols = 32;  // columns per CTA
constexpr int kRecTok = 32;   // tokens per staged block

// Few long sequences are cut into segments of `len` tokens that run at once, each from
// its own state.  The state is affine in the one before, column by column: a run from
// zero gives a segment's constant part B, and d more columns without V that start as
// the unit matrix its matrix M (carry: only these ends are wanted).
struct Segments {
    int count, first;    // segments that run, the first of them
    int64_t len;         // a multiple of kRecTok
    const float* start;  // [BH][count][d][dv], or NULL: one segment from S0
    int carry;
    float *B, *M;        // carry: [BH][count][d][dv], [BH][count][d][d]
};

template <int D, typename T>
__global__ void __launch_bounds__(kRecThreads)
    k_delta_rec(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                const float* __restrict__ beta, const float* __restrict__ log_alpha,
                T* __restrict__ out, const float* S0, float* S_out, float* __restrict__ chk,
                float* __restrict__ err, int64_t N, int H, int Hk, int DV, int l2, float scale, Segments seg)
{
    __shared__ __align__(16) float sk[kRecTok][D];
    __shared__ __align__(16) float sq[kRecTok][D];
    __shared__ float sv[kRecTok][kRecCols];
    __shared__ float so[kRecTok][kRecCols];
    // a token's row: p_ji k_j.k_i (i < j) and A_j; p_ji q_j.k_i (i <= j)
    __shared__ __align__(16) float4 skk[kRecTok], sqk[kRecTok];
    __shared__ __align__(16) float sbeta[kRecTok], slast[kRecTok];  // slast: p_4j
    __shared__ float raw[kRecThreads / 32][2][kGroup * kGroup];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, col = warp * 4 + (lane & 3);
    const int64_t run = blockIdx.x, bh = run / seg.count;  // head and segment; head
    const int64_t lo = (run % seg.count + seg.first) * seg.len, hi = min(N, lo + seg.len);
    const int c0 = blockIdx.y * kRecCols;
    const bool unit = c0 >= DV;  // carry: columns of the unit matrix
    const int64_t kh = bh / H * Hk + (bh % H) / (H / Hk);
    const T* qp = q ? q + kh * N * D : nullptr;
    const T* kp = k + kh * N * D;
    const T* vp = unit ? nullptr : v + bh * N * DV + c0;
    const int64_t nblk = (N + kRecTok - 1) / kRecTok;

    float2 s[D / 16];  // rows 4 r + 2 (i % 2) and the next of the 32 from 32 (i / 2)
    const float* start = seg.start ? seg.start + run * D * DV : S0 ? S0 + bh * D * DV : nullptr;
    auto row_of = [&](int i) { return i / 2 * 32 + 4 * r + i % 2 * 2; };
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        const int row = row_of(i), at = row * DV + c0 + col, u = c0 + col - DV;
        s[i].x = seg.carry ? (row == u ? 1.0f : 0.0f) : start ? start[at] : 0.0f;
        s[i].y = seg.carry ? (row + 1 == u ? 1.0f : 0.0f) : start ? start[at + DV] : 0.0f;
    }

    // a warp stages a group of tokens
    constexpr int kRows = kGroup;
    static_assert(kRecTok == kGroup * (kRecThreads / 32), "a group per warp");
    T nk[kRows][D / 32], nq[kRows][D / 32], nv[kRows];
    float nb[kRows], na[kRows];
    auto fetch = [&](int64_t b) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t t = b * kRecTok + warp * kGroup + i;
            const bool live = t < hi;
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                nk[i][x] = live ? kp[t * D + lane + 32 * x] : from_f32<T>(0.f);
                nq[i][x] = live && qp ? qp[t * D + lane + 32 * x] : from_f32<T>(0.f);
            }
            nv[i] = live && !unit ? vp[t * DV + lane] : from_f32<T>(0.f);
            nb[i] = live ? beta[bh * N + t] : 0.f;
            na[i] = live && log_alpha ? log_alpha[bh * N + t] : 0.f;
        }
    };
    const int64_t b0 = lo / kRecTok, b1 = (hi + kRecTok - 1) / kRecTok;
    fetch(b0);
    for (int64_t b = b0; b < b1; ++b) {
        const int64_t t0 = b * kRecTok;
        const int n = (int)min((int64_t)kRecTok, hi - t0);
        __syncthreads();  // the previous block's tiles are read
        {
            const int g = lane >> 2, j = g & 3, i = lane & 3;
            float y[3][8] = {};
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                float kk[kRows], qq[kRows];
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    kk[r] = to_f32<T>(nk[r][x]), qq[r] = to_f32<T>(nq[r][x]);
                    y[0][r] = fmaf(kk[r], kk[r], y[0][r]);
                    y[0][4 + r] = fmaf(qq[r], qq[r], y[0][4 + r]);
                    y[1][r] = fmaf(qq[r], kk[r], y[1][r]);
                }
                y[1][4] = fmaf(kk[1], kk[0], y[1][4]), y[1][5] = fmaf(kk[2], kk[0], y[1][5]);
                y[1][6] = fmaf(kk[3], kk[0], y[1][6]), y[1][7] = fmaf(kk[2], kk[1], y[1][7]);
                y[2][0] = fmaf(kk[3], kk[1], y[2][0]), y[2][1] = fmaf(kk[3], kk[2], y[2][1]);
                y[2][2] = fmaf(qq[1], kk[0], y[2][2]), y[2][3] = fmaf(qq[2], kk[0], y[2][3]);
                y[2][4] = fmaf(qq[3], kk[0], y[2][4]), y[2][5] = fmaf(qq[2], kk[1], y[2][5]);
                y[2][6] = fmaf(qq[3], kk[1], y[2][6]), y[2][7] = fmaf(qq[3], kk[2], y[2][7]);
            }
            float z[3];  // lanes 4 g ..: sum g
#pragma unroll
            for (int m = 0; m < 3; ++m) {
                z[m] = delta::sum8(y[m], lane);
                z[m] += __shfl_xor_sync(0xffffffffu, z[m], 2);
                z[m] += __shfl_xor_sync(0xffffffffu, z[m], 1);
            }
            // 1 / norms, the queries' with the scale: lanes 4 r .. of k_r, 16 + 4 r .. of q_r
            const float inv = (l2 ? rsqrtf(z[0] + kL2Eps) : 1.0f) * (g < 4 ? 1.0f : scale);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float rk = __shfl_sync(0xffffffffu, inv, 4 * r), rq = __shfl_sync(0xffffffffu, inv, 16 + 4 * r);
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    sk[warp * kGroup + r][lane + 32 * x] = to_f32<T>(nk[r][x]) * rk;
                    sq[warp * kGroup + r][lane + 32 * x] = to_f32<T>(nq[r][x]) * rq;
                }
                sv[warp * kGroup + r][lane] = to_f32<T>(nv[r]);  // kRecCols lanes
            }
            if (i == 0) {  // the sums to their places, 4 j + i, a digit for each
                raw[warp][g < 4][0x9c84fa50u >> (4 * g) & 15] = z[1];
                raw[warp][g >= 2][0xed9c84edu >> (4 * g) & 15] = z[2];
            }
            __syncwarp();
            // entry (j, i): lanes < 16 of k.k, the others of q.k
            float a[kRows], p = 1.0f, A = 1.0f, last = 1.0f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                a[r] = expf(na[r]);
                p *= r > i && r <= j ? a[r] : 1.0f;
                A *= r <= j ? a[r] : 1.0f;
                last *= r > j ? a[r] : 1.0f;
            }
            const float rj = __shfl_sync(0xffffffffu, inv, g < 4 ? 4 * j : 16 + 4 * j);
            const float ri = __shfl_sync(0xffffffffu, inv, 4 * i);
            float* row = reinterpret_cast<float*>((g < 4 ? skk : sqk) + warp * kGroup + j);
            if (g < 4)
                row[i] = i == 3 ? A : i < j ? raw[warp][0][4 * j + i] * (rj * ri * p) : 0.0f;
            else
                row[i] = i <= j ? raw[warp][1][4 * j + i] * (rj * ri * p) : 0.0f;
            if (lane < 16 && i == 0) {
                float b = nb[0];
#pragma unroll
                for (int r = 1; r < kRows; ++r)
                    b = j == r ? nb[r] : b;
                sbeta[warp * kGroup + j] = b;
                slast[warp * kGroup + j] = last;
            }
        }
        if (b + 1 < b1)
            fetch(b + 1);
        if (chk) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                float* at = chk + ((bh * (nblk + 1) + b) * D + row_of(i)) * DV + c0 + col;
                at[0] = s[i].x, at[DV] = s[i].y;
            }
        }
        __syncthreads();
        for (int t = 0; t < n; t += kGroup) {  // past the end: zero rows, no decay
            float2 d[8] = {}, kf[kGroup][D / 16];
#pragma unroll
            for (int m = 0; m < D / 32; ++m) {
#pragma unroll
                for (int j = 0; j < kGroup; ++j) {
                    const float4 x = *reinterpret_cast<const float4*>(&sk[t + j][32 * m + 4 * r]);
                    const float4 w = *reinterpret_cast<const float4*>(&sq[t + j][32 * m + 4 * r]);
                    kf[j][2 * m] = make_float2(x.x, x.y), kf[j][2 * m + 1] = make_float2(x.z, x.w);
                    d[j] = fma2(kf[j][2 * m], s[2 * m], fma2(kf[j][2 * m + 1], s[2 * m + 1], d[j]));
                    d[4 + j] = fma2(make_float2(w.x, w.y), s[2 * m], fma2(make_float2(w.z, w.w), s[2 * m + 1], d[4 + j]));
                }
            }
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[j] = d[j].x + d[j].y;
            const float z = delta::sum8(y, lane);  // row r < 4: k_r, else q_{r - 4}
            const float4 be = *reinterpret_cast<const float4*>(sbeta + t), pl = *reinterpret_cast<const float4*>(slast + t);
            const float b[4] = {be.x, be.y, be.z, be.w}, p[4] = {pl.x, pl.y, pl.z, pl.w};
            float e[kGroup], u[kGroup], A = 1.0f;
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                const float4 g = skk[t + j];
                const float c[3] = {g.x, g.y, g.z};
                A = g.w;
                e[j] = fmaf(-A, __shfl_sync(0xffffffffu, z, 4 * j + (lane & 3)), sv[t + j][col]);
#pragma unroll
                for (int i = 0; i < j; ++i)
                    e[j] = fmaf(-c[i], u[i], e[j]);
                u[j] = b[j] * e[j];
            }
            const float2 w[kGroup] = {both(p[0] * u[0]), both(p[1] * u[1]), both(p[2] * u[2]), both(p[3] * u[3])};
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                s[i] = mul2(both(A), s[i]);
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    s[i] = fma2(kf[j][i], w[j], s[i]);
            }
            if (r >= 4) {
                const float4 h = sqk[t + r - 4];
                so[t + r - 4][col] = fmaf(skk[t + r - 4].w, z, fmaf(h.x, u[0], fmaf(h.y, u[1], fmaf(h.z, u[2], h.w * u[3]))));
            } else if (err && t + r < n) {
                err[(bh * N + t0 + t + r) * DV + c0 + col] = r == 0 ? e[0] : r == 1 ? e[1] : r == 2 ? e[2] : e[3];
            }
        }
        __syncwarp();
        // a warp stores its own 4 columns
        if (out) {
            for (int i = lane; i < n * 4; i += 32)
                out[(bh * N + t0 + i / 4) * DV + c0 + warp * 4 + i % 4] =
                    from_f32<T>(so[i / 4][warp * 4 + i % 4]);
        }
        __syncwarp();
    }
    float* end = nullptr;
    int ld = DV;
    if (seg.carry) {
        end = unit ? seg.M + run * D * D - DV : seg.B + run * D * DV;  // unit column c is M's c - DV
        ld = unit ? D : DV;
    } else if (S_out && hi == N) {
        end = S_out + bh * D * DV;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        if (end) {
            float* at = end + (int64_t)row_of(i) * ld + c0 + col;
            at[0] = s[i].x, at[ld] = s[i].y;
        }
        if (chk && hi == N) {
            float* at = chk + ((bh * (nblk + 1) + nblk) * D + row_of(i)) * DV + c0 + col;
            at[0] = s[i].x, at[DV] = s[i].y;
        }
    }
}

// ----------------------------------------------------------- decode step ----
// One token per head: the state is read once and written once (8 bytes per
// element) and everything else is small, so the step is bound by HBM.  A CTA
// owns D rows x CS columns; a thread keeps its rows of one 16-byte column
// group in registers between the two products and the update.  256 x 32 heads of
// 128 x 128: 162 us, 6.7 TB/s of the 1.09 GB it has to move, as fast as a copy.
constexpr int kDecThreads = 256;

template <int D, int CS, typename T>
__global__ void __launch_bounds__(kDecThreads)
    k_delta_decode(float* __restrict__ S, const T* __restrict__ q, const T* __restrict__ k,
                   const T* __restrict__ v, const float* __restrict__ beta,
                   const float* __restrict__ log_alpha, T* __restrict__ out, int H, int Hk, int DV,
                   int l2, float scale)
{
    constexpr int TJ = CS / 4, TI = kDecThreads / TJ, RI = D / TI > 0 ? D / TI : 1;
    static_assert(D % TI == 0, "tile");
    __shared__ float sk[D], sq[D], snorm[3];
    __shared__ float4 rk[kDecThreads], rq[kDecThreads];
    __shared__ __align__(16) float su[CS];

    const int64_t bh = blockIdx.x;
    const int c0 = blockIdx.y * CS;
    const int tid = threadIdx.x, tj = tid % TJ, ti = tid / TJ;
    float* Sb = S + bh * (int64_t)D * DV + c0;
    float4 s[RI];
#pragma unroll
    for (int i = 0; i < RI; ++i)
        s[i] = __ldcs(reinterpret_cast<const float4*>(Sb + (ti + i * TI) * DV + tj * 4));

    const int64_t kh = bh / H * Hk + (bh % H) / (H / Hk);
    if (tid < 32) {  // one warp: norms, k . q
        float kk[D / 32], qq[D / 32], k2 = 0.f, q2 = 0.f, kq = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            kk[i] = to_f32<T>(k[kh * D + tid + 32 * i]);
            qq[i] = to_f32<T>(q[kh * D + tid + 32 * i]);
            k2 = fmaf(kk[i], kk[i], k2);
            q2 = fmaf(qq[i], qq[i], q2);
            kq = fmaf(kk[i], qq[i], kq);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            k2 += __shfl_xor_sync(0xffffffffu, k2, o);
            q2 += __shfl_xor_sync(0xffffffffu, q2, o);
            kq += __shfl_xor_sync(0xffffffffu, kq, o);
        }
        const float fk = l2 ? rsqrtf(k2 + kL2Eps) : 1.0f;
        const float fq = (l2 ? rsqrtf(q2 + kL2Eps) : 1.0f) * scale;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            sk[tid + 32 * i] = kk[i] * fk;
            sq[tid + 32 * i] = qq[i] * fq;
        }
        if (tid == 0) {
            snorm[0] = kq * fk * fq;
            snorm[1] = beta[bh];
            snorm[2] = log_alpha ? expf(log_alpha[bh]) : 1.0f;
        }
    }
    __syncthreads();
    const float a = snorm[2];
    float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        const float x = sk[ti + i * TI], y = sq[ti + i * TI];
        s[i].x *= a, s[i].y *= a, s[i].z *= a, s[i].w *= a;
        pk.x = fmaf(x, s[i].x, pk.x), pk.y = fmaf(x, s[i].y, pk.y);
        pk.z = fmaf(x, s[i].z, pk.z), pk.w = fmaf(x, s[i].w, pk.w);
        pq.x = fmaf(y, s[i].x, pq.x), pq.y = fmaf(y, s[i].y, pq.y);
        pq.z = fmaf(y, s[i].z, pq.z), pq.w = fmaf(y, s[i].w, pq.w);
    }
    rk[tid] = pk;
    rq[tid] = pq;
    __syncthreads();
    if (tid < CS) {  // column tid: sum the TI partial products
        const float* fk = reinterpret_cast<const float*>(rk) + tid;
        const float* fq = reinterpret_cast<const float*>(rq) + tid;
        float dk = 0.f, dq = 0.f;
#pragma unroll 8
        for (int i = 0; i < TI; ++i)
            dk += fk[i * CS], dq += fq[i * CS];
        const float u = snorm[1] * (to_f32<T>(v[bh * DV + c0 + tid]) - dk);
        su[tid] = u;
        out[bh * DV + c0 + tid] = from_f32<T>(fmaf(snorm[0], u, dq));
    }
    __syncthreads();
    const float4 u = *reinterpret_cast<const float4*>(su + tj * 4);
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        const float x = sk[ti + i * TI];
        float4 y = s[i];
        y.x = fmaf(x, u.x, y.x), y.y = fmaf(x, u.y, y.y);
        y.z = fmaf(x, u.z, y.z), y.w = fmaf(x, u.w, y.w);
        __stcs(reinterpret_cast<float4*>(Sb + (ti + i * TI) * DV + tj * 4), y);
    }
}

// -------------------------------------------------------------- gradient ----
// Chunks of C = kRecTok tokens.  With G the running sum of log_alpha inside the
// chunk, D_ij = exp(G_i - G_j), U = beta E, S0 and S1 the states before and after
// the chunk, dS1 the gradient of S1:
//
//   P_ij = D_ij q_i.k_j (j <= i),  A_ij = D_ij k_i.k_j (j < i)
//   dU = P^T dO + diag(e^{G_C - G}) K dS1
//   Y  = (I + diag(beta) A)^{-T} dU      from the last token back
//   dV = beta Y,  dbeta_i = Y_i.E_i
//   dS0 = e^{G_C} dS1 + (diag(e^G) Q)^T dO - (diag(e^G) K)^T dV
//   dQ = (dO U^T o D) K + diag(e^G) dO S0^T
//   dK = (dO U^T o D)^T Q + M K + M^T K - diag(e^G) dV S0^T + diag(e^{G_C - G}) U dS1^T
//        with M_ij = -D_ij dV_i.U_j (j < i)
//   dlog_alpha_t = sum_{i >= t > j} W_ij + sum_{i >= t} h_i + sum_{j < t} l_j + e^{G_C} <S0, dS1>
//        with W_ij = D_ij (dO_i.U_j q_i.k_j - dV_i.U_j k_i.k_j), l_j = e^{G_C - G_j} k_j.(dS1 U_j)
//        and h_i = e^{G_i} (q_i.(S0 dO_i) - k_i.(S0 dV_i))
//
// (the last line: log_alpha_t enters every decay that spans t, and each term here has
// such a decay as a factor.  It can be had from the rows' dots alone, as <S1, dS1> +
// sum_{i >= t} (q_i.dQ_i - v_i.dV_i), but there the terms that do not span t cancel only
// up to their rounding: of a gate of -8 half of the digits are left, of -16 none).
// S0 and E come from the recurrence above, which stored them.  Two kernels: the
// columns of dS, Y and dV never mix, so k_delta_grad_rev runs the chunks in reverse
// for 32 columns per CTA and keeps dS1, dV, Y.E and <S0, dS1> over its columns (over
// segments like the recurrence: dS0 is affine in dS1, its matrix the transposed M);
// k_delta_grad_dqk then takes every chunk on its own.  fp32 in shared memory, bound
// by its reads: B2 H4 N201 d = 64 2 x 22 us and 24 us.
struct GradKept {
    float* dS;  // [BH][nblk][D][DV] gradient of the state after the chunk
    float* dV;  // [BH][N][DV]
    float* bb;  // [BH][DV / 32][N] Y.E over 32 columns
    float* cd;  // [BH][DV / 32][nblk] <S0, dS1>
};

constexpr int kRevThreads = 256;

// K and Q rows of a chunk (normalised, Q scaled; zero past n) by warps of a block
template <int D>
__device__ __forceinline__ void load_rows(float* sk, float* sq, int LK, const float* k, const float* q, int64_t row0, int n, int l2,
                                          float scale)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int t = warp; t < kRecTok; t += blockDim.x >> 5) {
        float kk[D / 32], qq[D / 32], k2 = 0.f, q2 = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const int64_t at = (row0 + t) * D + lane + 32 * i;
            kk[i] = t < n ? k[at] : 0.f;
            qq[i] = t < n ? q[at] : 0.f;
            k2 = fmaf(kk[i], kk[i], k2);
            q2 = fmaf(qq[i], qq[i], q2);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            k2 += __shfl_xor_sync(0xffffffffu, k2, o);
            q2 += __shfl_xor_sync(0xffffffffu, q2, o);
        }
        const float rk = l2 ? rsqrtf(k2 + kL2Eps) : 1.0f;
        const float rq = (l2 ? rsqrtf(q2 + kL2Eps) : 1.0f) * scale;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            sk[t * LK + lane + 32 * i] = kk[i] * rk;
            sq[t * LK + lane + 32 * i] = qq[i] * rq;
        }
    }
}

// Running sums of a chunk's gates by one warp: G (64 bits), e^G, e^{G_C - G}
__device__ __forceinline__ void load_gates(double* G, float* eg, float* ege, const float* log_alpha, int n)
{
    const int lane = threadIdx.x & 31;
    double g = log_alpha && lane < n ? (double)delta::clamp_gate(log_alpha[lane]) : 0.0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, g, o);
        if (lane >= o)
            g += x;
    }
    G[lane] = g;
    eg[lane] = expf((float)g);
    ege[lane] = expf((float)(__shfl_sync(0xffffffffu, g, 31) - g));
}

template <int D>
__global__ void __launch_bounds__(kRevThreads)
    k_delta_grad_rev(const float* __restrict__ q, const float* __restrict__ k,
                     const float* __restrict__ beta, const float* __restrict__ log_alpha,
                     const float* __restrict__ dout, const float* __restrict__ dS_out,
                     const float* __restrict__ chk, const float* __restrict__ err, float* __restrict__ dv,
                     float* __restrict__ dS0, GradKept kept, int64_t N, int H, int Hk, int DV, int l2,
                     float scale, Segments seg)
{
    constexpr int C = kRecTok, LK = D + 4, LC = C + 4, R = D / 8;  // R: state rows per thread
    extern __shared__ __align__(16) float smem[];
    float* dS = smem;           // [D][32]
    float* sk = dS + D * 32;    // [C][LK]
    float* sq = sk + C * LK;    // [C][LK], scaled
    float* sdo = sq + C * LK;   // [C][32]
    float* sy = sdo + C * 32;   // [C][32] dU, then Y, then dV
    float* P = sy + C * 32;     // [C][LC]
    float* A = P + C * LC;      // [C][LC] beta_i A_ij
    __shared__ double G[C];
    __shared__ float eg[C], ege[C], sb[C], red[8];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t run = blockIdx.x, bh = run / seg.count;
    const int64_t lo = (run % seg.count + seg.first) * seg.len, hi = min(N, lo + seg.len);
    const bool ends = seg.carry;  // a run from dS = 0 that leaves the constant part in seg.B
    const int c0 = blockIdx.y * 32, nsl = gridDim.y;
    const int64_t kh = bh / H * Hk + (bh % H) / (H / Hk);
    const int64_t nblk = (N + C - 1) / C;

    // a thread keeps rows warp R .. of column lane in registers too
    float ds[R];
    const float* end = ends ? nullptr : seg.start ? seg.start + run * D * DV : dS_out ? dS_out + bh * D * DV : nullptr;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        ds[i] = end ? end[(warp * R + i) * DV + c0 + lane] : 0.f;
        dS[(warp * R + i) * 32 + lane] = ds[i];
    }
    for (int64_t b = (hi - 1) / C; b >= lo / C; --b) {
        const int64_t t0 = b * C;
        const int n = (int)min((int64_t)C, N - t0);
        // dS1 out, <S0, dS1>
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < R && !ends; ++i) {
            const int64_t row = warp * R + i;
            kept.dS[((bh * nblk + b) * D + row) * DV + c0 + lane] = ds[i];
            if (log_alpha)
                dot = fmaf(chk[((bh * (nblk + 1) + b) * D + row) * DV + c0 + lane], ds[i], dot);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0)
            red[warp] = dot;
        // rows past the end stay zero and leave nothing behind (beta = 0, G constant)
        load_rows<D>(sk, sq, LK, k, q, kh * N + t0, n, l2, scale);
#pragma unroll
        for (int t = warp; t < C; t += 8)
            sdo[t * 32 + lane] = t < n ? dout[(bh * N + t0 + t) * DV + c0 + lane] : 0.f;
        if (warp == 0) {
            load_gates(G, eg, ege, log_alpha ? log_alpha + bh * N + t0 : nullptr, n);
            sb[lane] = lane < n ? beta[bh * N + t0 + lane] : 0.f;
        }
        __syncthreads();
        if (tid == 0 && !ends) {
            float x = 0.f;
            for (int w = 0; w < 8; ++w)
                x += red[w];
            kept.cd[(bh * nsl + blockIdx.y) * nblk + b] = x;
        }
        // P and beta A: 4 rows (warp) x a column (lane) per thread
        {
            float p[4] = {}, a[4] = {};
            for (int x = 0; x < D; x += 4) {
                const float4 kj = *reinterpret_cast<const float4*>(sk + lane * LK + x);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 qi = *reinterpret_cast<const float4*>(sq + (4 * warp + i) * LK + x);
                    const float4 ki = *reinterpret_cast<const float4*>(sk + (4 * warp + i) * LK + x);
                    p[i] = fmaf(qi.x, kj.x, fmaf(qi.y, kj.y, fmaf(qi.z, kj.z, fmaf(qi.w, kj.w, p[i]))));
                    a[i] = fmaf(ki.x, kj.x, fmaf(ki.y, kj.y, fmaf(ki.z, kj.z, fmaf(ki.w, kj.w, a[i]))));
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 4 * warp + r;
                const float dec = lane <= i ? expf((float)(G[i] - G[lane])) : 0.f;
                P[i * LC + lane] = lane <= i ? p[r] * dec : 0.f;
                A[i * LC + lane] = lane < i ? a[r] * dec * sb[i] : 0.f;
            }
        }
        __syncthreads();
        // dU: rows 4 warp .. + 3 of column lane
        {
            float u[4] = {}, w[4] = {};
            for (int x = 0; x < D; x += 4) {
                const float d0 = dS[x * 32 + lane], d1 = dS[(x + 1) * 32 + lane], d2 = dS[(x + 2) * 32 + lane],
                            d3 = dS[(x + 3) * 32 + lane];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 kj = *reinterpret_cast<const float4*>(sk + (4 * warp + r) * LK + x);
                    w[r] = fmaf(kj.x, d0, fmaf(kj.y, d1, fmaf(kj.z, d2, fmaf(kj.w, d3, w[r]))));
                }
            }
            for (int i = 4 * warp; i < C; ++i) {
                const float4 p = *reinterpret_cast<const float4*>(P + i * LC + 4 * warp);
                const float d = sdo[i * 32 + lane];
                u[0] = fmaf(p.x, d, u[0]), u[1] = fmaf(p.y, d, u[1]);
                u[2] = fmaf(p.z, d, u[2]), u[3] = fmaf(p.w, d, u[3]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
                sy[(4 * warp + r) * 32 + lane] = fmaf(ege[4 * warp + r], w[r], u[r]);
        }
        __syncthreads();
        // Y: one warp, a column per lane; each solved token leaves the earlier ones
        if (warp == 0) {
            float y[C];
#pragma unroll
            for (int j = 0; j < C; ++j)
                y[j] = sy[j * 32 + lane];
#pragma unroll
            for (int i = C - 1; i > 0; --i) {
#pragma unroll
                for (int j = 0; j < i; j += 4) {  // A is zero from the diagonal on
                    const float4 a = *reinterpret_cast<const float4*>(A + i * LC + j);
                    y[j] = fmaf(-a.x, y[i], y[j]);
                    if (j + 1 < i)
                        y[j + 1] = fmaf(-a.y, y[i], y[j + 1]);
                    if (j + 2 < i)
                        y[j + 2] = fmaf(-a.z, y[i], y[j + 2]);
                    if (j + 3 < i)
                        y[j + 3] = fmaf(-a.w, y[i], y[j + 3]);
                }
            }
#pragma unroll
            for (int j = 0; j < C; ++j)
                sy[j * 32 + lane] = y[j];
        }
        __syncthreads();
        // dV, the dots over the columns
#pragma unroll
        for (int t = warp; t < C; t += 8) {
            float y = sy[t * 32 + lane], db = 0.f;
            const float g = sb[t] * y;
            sy[t * 32 + lane] = g;
            if (t < n && !ends) {
                const int64_t at = (bh * N + t0 + t) * DV + c0 + lane;
                dv[at] = g;
                kept.dV[at] = g;
                db = y * err[at];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                db += __shfl_xor_sync(0xffffffffu, db, o);
            if (lane == 0 && t < n && !ends)
                kept.bb[(bh * nsl + blockIdx.y) * N + t0 + t] = db;
        }
        __syncthreads();
        // dS <- dS0
#pragma unroll
        for (int i = 0; i < R; ++i)
            ds[i] *= eg[C - 1];
        for (int i = 0; i < C; ++i) {
            const float o = eg[i] * sdo[i * 32 + lane], g = -eg[i] * sy[i * 32 + lane];
#pragma unroll
            for (int x = 0; x < R; x += 4) {
                const float4 a = *reinterpret_cast<const float4*>(sq + i * LK + warp * R + x);
                const float4 c = *reinterpret_cast<const float4*>(sk + i * LK + warp * R + x);
                ds[x] = fmaf(a.x, o, fmaf(c.x, g, ds[x]));
                ds[x + 1] = fmaf(a.y, o, fmaf(c.y, g, ds[x + 1]));
                ds[x + 2] = fmaf(a.z, o, fmaf(c.z, g, ds[x + 2]));
                ds[x + 3] = fmaf(a.w, o, fmaf(c.w, g, ds[x + 3]));
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < R; ++i)
            dS[(warp * R + i) * 32 + lane] = ds[i];
    }
    float* to = ends ? seg.B + run * D * DV : dS0 && lo == 0 ? dS0 + bh * D * DV : nullptr;
    if (to) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            to[(warp * R + i) * DV + c0 + lane] = ds[i];
    }
}

template <int D>
constexpr size_t rev_smem()
{
    return sizeof(float) * (D * 32 + 2 * kRecTok * (D + 4) + 2 * kRecTok * 32 + 2 * kRecTok * (kRecTok + 4));
}

constexpr int kGradThreads = 256;

template <int D, int DV>
struct GradSmem {
    static constexpr int C = kRecTok;
    static constexpr int LS = DV + 4, LK = D + 4, LV = DV + 4, LC = C + 4;
    static constexpr int floats = D * LS + 2 * C * LK + 3 * C * LV + 3 * C * LC;
    static constexpr size_t bytes = sizeof(float) * floats;
    static_assert(bytes <= 232448, "shared memory");
};

// 16 x 16 threads per 32 x D result: thread (ty, tx) owns rows 2 ty, 2 ty + 1 and
// columns tx, tx + 16, .. (stride: rows of S at 4 banks' distance from each other)
template <int D, int DV>
__global__ void __launch_bounds__(kGradThreads)
    k_delta_grad_dqk(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ beta,
                     const float* __restrict__ log_alpha, const float* __restrict__ dout,
                     const float* __restrict__ chk, const float* __restrict__ err, GradKept kept,
                     float* __restrict__ dq, float* __restrict__ dk, float* __restrict__ dbeta,
                     float* __restrict__ dlog_alpha, int64_t N, int H, int Hk, int l2, float scale)
{
    using SM = GradSmem<D, DV>;
    constexpr int C = SM::C, LS = SM::LS, LK = SM::LK, LV = SM::LV, LC = SM::LC, CX = D / 16;
    extern __shared__ __align__(16) float smem[];
    float* S = smem;           // [D][LS] S0, then dS1
    float* sk = S + D * LS;    // [C][LK]
    float* sq = sk + C * LK;   // [C][LK], scaled
    float* sdo = sq + C * LK;  // [C][LV]
    float* su = sdo + C * LV;  // [C][LV] U
    float* sg = su + C * LV;   // [C][LV] dV
    float* P = sg + C * LV;    // [i][j] dO_i.U_j D_ij
    float* Pt = P + C * LC;    // its transpose
    float* M = Pt + C * LC;    // [j][i] M_ij (i > j), M_ji (i < j): the matrix on K for dK
    __shared__ double G[C];
    // span: sum of W_ij over i >= t > j for four rows i; dH: h; dL: l
    __shared__ float eg[C], ege[C], sb[C], span[kGradThreads / 32][C], dH[C], dL[C];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, ty = tid >> 4, tx = tid & 15;
    const int64_t nblk = (N + C - 1) / C;
    const int64_t bh = blockIdx.x / nblk, b = blockIdx.x % nblk;
    const int64_t kh = bh / H * Hk + (bh % H) / (H / Hk);
    const int64_t t0 = b * C;
    const int n = (int)min((int64_t)C, N - t0);

    load_rows<D>(sk, sq, LK, k, q, kh * N + t0, n, l2, scale);
    if (warp == 0)
        load_gates(G, eg, ege, log_alpha ? log_alpha + bh * N + t0 : nullptr, n);
    if (tid < C)
        sb[tid] = tid < n ? beta[bh * N + t0 + tid] : 0.f;
    for (int i = tid; i < D * DV; i += kGradThreads)
        S[i / DV * LS + i % DV] = chk[(bh * (nblk + 1) + b) * (int64_t)(D * DV) + i];
    for (int i = tid; i < C * DV; i += kGradThreads) {
        const int t = i / DV, c = i % DV;
        const int64_t at = (bh * N + t0 + t) * DV + c;
        sdo[t * LV + c] = t < n ? dout[at] : 0.f;
        su[t * LV + c] = t < n ? beta[bh * N + t0 + t] * err[at] : 0.f;
        sg[t * LV + c] = t < n ? kept.dV[at] : 0.f;
    }
    __syncthreads();
    // dO_i.U_j and dV_i.U_j: 4 rows (warp) x a column (lane) per thread
    {
        float p[4] = {}, m[4] = {}, qk[4] = {}, kk[4] = {}, w = 0.f;
        for (int x = 0; x < DV; x += 4) {
            const float4 u = *reinterpret_cast<const float4*>(su + lane * LV + x);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float4 o = *reinterpret_cast<const float4*>(sdo + (4 * warp + r) * LV + x);
                const float4 g = *reinterpret_cast<const float4*>(sg + (4 * warp + r) * LV + x);
                p[r] = fmaf(o.x, u.x, fmaf(o.y, u.y, fmaf(o.z, u.z, fmaf(o.w, u.w, p[r]))));
                m[r] = fmaf(g.x, u.x, fmaf(g.y, u.y, fmaf(g.z, u.z, fmaf(g.w, u.w, m[r]))));
            }
        }
        for (int x = 0; dlog_alpha && x < D; x += 4) {
            const float4 y = *reinterpret_cast<const float4*>(sk + lane * LK + x);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float4 a = *reinterpret_cast<const float4*>(sq + (4 * warp + r) * LK + x);
                const float4 b = *reinterpret_cast<const float4*>(sk + (4 * warp + r) * LK + x);
                qk[r] = fmaf(a.x, y.x, fmaf(a.y, y.y, fmaf(a.z, y.z, fmaf(a.w, y.w, qk[r]))));
                kk[r] = fmaf(b.x, y.x, fmaf(b.y, y.y, fmaf(b.z, y.z, fmaf(b.w, y.w, kk[r]))));
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 4 * warp + r, j = lane;
            const float dec = j <= i ? expf((float)(G[i] - G[j])) : 0.f;
            const float x = j <= i ? p[r] * dec : 0.f;
            P[i * LC + j] = x;
            Pt[j * LC + i] = x;
            if (j < i)
                M[i * LC + j] = M[j * LC + i] = -m[r] * dec;
            else if (j == i)
                M[i * LC + i] = 0.f;
            // sum over j < t = lane, of the rows i >= t
            float z = j < i ? dec * fmaf(p[r], qk[r], -m[r] * kk[r]) : 0.f;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float y = __shfl_up_sync(0xffffffffu, z, o);
                if (lane >= o)
                    z += y;
            }
            z = __shfl_up_sync(0xffffffffu, z, 1);
            w += lane > 0 && lane <= i ? z : 0.f;
        }
        span[warp][lane] = w;
    }
    __syncthreads();
    // x[row][column] += a[row][0 .. C) b[0 .. C)[column], rows 2 ty, 2 ty + 1
    auto tokens = [&](float (&x)[2][CX], const float* a, const float* bm) {
#pragma unroll 2
        for (int j = 0; j < C; j += 4) {
            const float4 a0 = *reinterpret_cast<const float4*>(a + 2 * ty * LC + j);
            const float4 a1 = *reinterpret_cast<const float4*>(a + (2 * ty + 1) * LC + j);
#pragma unroll
            for (int i = 0; i < CX; ++i) {
                const float* at = bm + j * LK + tx + 16 * i;
                const float b0 = at[0], b1 = at[LK], b2 = at[2 * LK], b3 = at[3 * LK];
                x[0][i] = fmaf(a0.x, b0, fmaf(a0.y, b1, fmaf(a0.z, b2, fmaf(a0.w, b3, x[0][i]))));
                x[1][i] = fmaf(a1.x, b0, fmaf(a1.y, b1, fmaf(a1.z, b2, fmaf(a1.w, b3, x[1][i]))));
            }
        }
    };
    // x[row][column] += f[row] a[row] . S[column]
    auto states = [&](float (&x)[2][CX], const float* a, float f0, float f1) {
        float y[2][CX] = {};
#pragma unroll 2
        for (int c = 0; c < DV; c += 4) {
            const float4 a0 = *reinterpret_cast<const float4*>(a + 2 * ty * LV + c);
            const float4 a1 = *reinterpret_cast<const float4*>(a + (2 * ty + 1) * LV + c);
#pragma unroll
            for (int i = 0; i < CX; ++i) {
                const float4 s = *reinterpret_cast<const float4*>(S + (tx + 16 * i) * LS + c);
                y[0][i] = fmaf(a0.x, s.x, fmaf(a0.y, s.y, fmaf(a0.z, s.z, fmaf(a0.w, s.w, y[0][i]))));
                y[1][i] = fmaf(a1.x, s.x, fmaf(a1.y, s.y, fmaf(a1.z, s.z, fmaf(a1.w, s.w, y[1][i]))));
            }
        }
#pragma unroll
        for (int i = 0; i < CX; ++i)
            x[0][i] = fmaf(f0, y[0][i], x[0][i]), x[1][i] = fmaf(f1, y[1][i], x[1][i]);
    };
    const int i0 = 2 * ty, i1 = i0 + 1;
    auto put = [&](float* dst, const float (&x)[2][CX]) {
#pragma unroll
        for (int i = 0; i < CX; ++i) {
            if (i0 < n)
                dst[(bh * N + t0 + i0) * D + tx + 16 * i] = x[0][i];
            if (i1 < n)
                dst[(bh * N + t0 + i1) * D + tx + 16 * i] = x[1][i];
        }
    };
    // row i0's and i1's dots of x with a, by the threads of lane 0
    auto row_dots = [&](const float (&x)[2][CX], const float* a, float& d0, float& d1) {
        d0 = d1 = 0.f;
#pragma unroll
        for (int i = 0; i < CX; ++i) {
            d0 = fmaf(x[0][i], a[i0 * LK + tx + 16 * i], d0);
            d1 = fmaf(x[1][i], a[i1 * LK + tx + 16 * i], d1);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            d0 += __shfl_xor_sync(0xffffffffu, d0, o);
            d1 += __shfl_xor_sync(0xffffffffu, d1, o);
        }
    };
    float h0, h1, d0, d1;
    {  // dQ
        float x[2][CX] = {};
        states(x, sdo, eg[i0], eg[i1]);
        row_dots(x, sq, h0, h1);
        tokens(x, P, sk);
        put(dq, x);
    }
    float x[2][CX] = {};
    states(x, sg, -eg[i0], -eg[i1]);
    row_dots(x, sk, d0, d1);
    if (tx == 0)
        dH[i0] = h0 + d0, dH[i1] = h1 + d1;
    tokens(x, Pt, sq);
    tokens(x, M, sk);
    __syncthreads();  // S0 is read
    for (int i = tid; i < D * DV; i += kGradThreads)
        S[i / DV * LS + i % DV] = kept.dS[(bh * nblk + b) * (int64_t)(D * DV) + i];
    __syncthreads();
    {
        float y[2][CX] = {};
        states(y, su, ege[i0], ege[i1]);
        row_dots(y, sk, d0, d1);
        if (tx == 0)
            dL[i0] = d0, dL[i1] = d1;
#pragma unroll
        for (int i = 0; i < CX; ++i)
            x[0][i] += y[0][i], x[1][i] += y[1][i];
    }
    put(dk, x);
    __syncthreads();
    if (warp == 0) {  // the gates' gradients
        const int nsl = DV / 32;
        float y = dH[lane], z = dL[lane], db = 0.f, w = 0.f, after = 0.f;
        for (int s = 0; s < nsl; ++s) {
            if (lane < n)
                db += kept.bb[(bh * nsl + s) * N + t0 + lane];
            after += kept.cd[(bh * nsl + s) * nblk + b];
        }
#pragma unroll
        for (int i = 0; i < kGradThreads / 32; ++i)
            w += span[i][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float a = __shfl_down_sync(0xffffffffu, y, o), c = __shfl_up_sync(0xffffffffu, z, o);
            if (lane + o < 32)
                y += a;
            if (lane >= o)
                z += c;
        }
        z = __shfl_up_sync(0xffffffffu, z, 1);
        if (lane < n) {
            dbeta[bh * N + t0 + lane] = db;
            if (dlog_alpha)
                dlog_alpha[bh * N + t0 + lane] = w + y + (lane > 0 ? z : 0.f) + eg[C - 1] * after;
        }
    }
}

// Gradients of the key heads' rows from those of the value heads that read
// them: summed in head order, through the scale and the L2 norm
// (x = u / l, l^2 = |u|^2 + eps: du = (dx - x (x.dx)) / l), rounded once.  A
// warp per row.
template <int D>
__global__ void __launch_bounds__(256)
    k_delta_finish(const float* __restrict__ g, const float* __restrict__ u, float* __restrict__ du,
                   int64_t rows, int64_t N, int H, int Hk, int l2, float scale)
{
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= rows)
        return;
    const int64_t kh = row / N, t = row % N;
    const int per = H / Hk;
    const int64_t h0 = kh / Hk * H + (kh % Hk) * per;
    float x[D / 32], y[D / 32], n2 = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        x[i] = 0.f;
        for (int p = 0; p < per; ++p)
            x[i] += g[((h0 + p) * N + t) * D + lane + 32 * i];
        x[i] *= scale;
        y[i] = u[row * D + lane + 32 * i];
        n2 = fmaf(y[i], y[i], n2);
    }
    if (l2) {
        float dot = 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            n2 += __shfl_xor_sync(0xffffffffu, n2, o);
        const float r = rsqrtf(n2 + kL2Eps);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            y[i] *= r;
            dot = fmaf(y[i], x[i], dot);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            x[i] = r * (x[i] - y[i] * dot);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        du[row * D + lane + 32 * i] = x[i];
}

// ----------------------------------------------------------------- hosts ----
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

int64_t rec_blocks(int64_t N) { return (N + kRecTok - 1) / kRecTok; }

// Segments of a sequence on this path (1: whole), and their tokens: as many as give
// two CTAs per SM at 152 SMs, at most 32 (they are joined one after the other, about
// 1 us each), of at least 64 tokens, or 32 in a short sequence.  At least 4 pay for the
// second run; where heads are what limits them 6 at d = 128, whose CTAs have an SM each.
// Forward and gradient, whole against cut (us): B1 H4 d = 64 N128 20 and 92 against 17
// and 72, N1000 139 and 514 against 46 and 133, N16384 2228 and 9524 against 353 and
// 1135; B1 H4 N512 d = 128 93 and 380 against 58 and 179 (81 and 199 in segments of
// 32); in four, B1 H16 N4096 64 x 128 559 and 2917 against 429 and 2120, but B2 H8
// N1000 d = 128 179 and 943 against 243 and 857.  By sizes alone, as workspaces are
// sized without the GPU.
int rec_segments(const DeltaArgs& a, int64_t* len)
{
    const int64_t slices = a.B * a.H * (a.dv / kRecCols);
    const int64_t least = a.N > 256 ? 2 * kRecTok : kRecTok;
    int64_t n = 2 * 152 / slices;
    *len = (a.N + kRecTok - 1) / kRecTok * kRecTok;
    if (n < (a.d > 64 ? 6 : 4) || a.N < 4 * kRecTok)
        return 1;
    n = n < a.N / kRecTok ? n : a.N / kRecTok;
    n = n < 32 ? n : 32;
    *len = ((a.N + n - 1) / n + kRecTok - 1) / kRecTok * kRecTok;
    if (*len < least)
        *len = least;
    return (int)((a.N + *len - 1) / *len);
}

struct RecLayout {
    size_t start, B, M, total;
};
RecLayout rec_layout(const DeltaArgs& a)
{
    int64_t len;
    const size_t n = (size_t)rec_segments(a, &len), BH = (size_t)(a.B * a.H);
    RecLayout l = {};
    if (n > 1) {
        l.B = up256(BH * n * a.d * a.dv * 4);
        l.M = l.B + up256(BH * n * a.d * a.dv * 4);
        l.total = l.M + up256(BH * n * a.d * a.d * 4);
    }
    return l;
}

template <int D, typename T>
cudaError_t launch_rec(const DeltaArgs& a, float* chk, float* err, const Segments& seg)
{
    const dim3 grid((unsigned)(a.B * a.H * seg.count), (unsigned)((a.dv + (seg.carry ? a.d : 0)) / kRecCols));
    k_delta_rec<D, T><<<grid, kRecThreads, 0, a.stream>>>(
        static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.beta,
        a.log_alpha, static_cast<T*>(a.out), a.S0, a.S_out, chk, err, a.N, (int)a.H, (int)a.Hk,
        a.dv, a.fm == LA_FM_L2, a.scale, seg);
    count_launches(1);
    return cudaGetLastError();
}

// The recurrence, over segments (ws: rec_layout) where there are any; a gradient
// (chk) wants the last segment's M too.
template <int D, typename T>
cudaError_t run_rec(const DeltaArgs& a, float* chk, float* err, unsigned char* ws)
{
    Segments seg = {1, 0, 0, nullptr, 0, nullptr, nullptr};
    const int n = rec_segments(a, &seg.len);
    if (n > 1) {
        const RecLayout l = rec_layout(a);
        float* start = reinterpret_cast<float*>(ws + l.start);
        float* B = reinterpret_cast<float*>(ws + l.B);
        float* M = reinterpret_cast<float*>(ws + l.M);
        const int m = chk ? n : n - 1;
        const Segments ends = {m, 0, seg.len, nullptr, 1, B, M};
        DeltaArgs f = a;
        f.q = nullptr, f.out = nullptr, f.S_out = nullptr;
        cudaError_t e = launch_rec<D, T>(f, nullptr, nullptr, ends);
        if (e != cudaSuccess || (e = delta::join_segments(a, false, a.S0, B, M, start, n, m)) != cudaSuccess)
            return e;
        seg.count = n, seg.start = start;
    }
    return launch_rec<D, T>(a, chk, err, seg);
}

template <int D, int CS, typename T>
cudaError_t launch_decode(const DeltaArgs& a)
{
    const dim3 grid((unsigned)(a.B * a.H), (unsigned)(a.dv / CS));
    k_delta_decode<D, CS, T><<<grid, kDecThreads, 0, a.stream>>>(
        a.S_out, static_cast<const T*>(a.q), static_cast<const T*>(a.k),
        static_cast<const T*>(a.v), a.beta, a.log_alpha, static_cast<T*>(a.out), (int)a.H,
        (int)a.Hk, a.dv, a.fm == LA_FM_L2, a.scale);
    count_launches(1);
    return cudaGetLastError();
}

template <int D, typename T>
cudaError_t run_decode(const DeltaArgs& a)
{
    switch (a.dv) {
    case 32: return launch_decode<D, 32, T>(a);
    case 64: return launch_decode<D, 64, T>(a);
    default: return launch_decode<D, 128, T>(a);
    }
}

struct GradLayout {
    size_t chk, err, dq, dk, dS, dV, bb, cd, seg, total;
};
GradLayout grad_layout(const DeltaArgs& a)
{
    const size_t BH = (size_t)(a.B * a.H), N = (size_t)a.N, sl = (size_t)a.dv / 32, nb = (size_t)rec_blocks(a.N);
    GradLayout l;
    size_t at = 0;
    auto take = [&](size_t floats) {
        const size_t p = at;
        at += up256(4 * floats);
        return p;
    };
    l.chk = take(BH * (nb + 1) * a.d * a.dv);
    l.err = take(BH * N * a.dv);
    l.dq = take(BH * N * a.d);
    l.dk = take(BH * N * a.d);
    l.dS = take(BH * nb * a.d * a.dv);
    l.dV = take(BH * N * a.dv);
    l.bb = take(BH * sl * N);
    l.cd = take(BH * sl * nb);
    l.seg = at;
    l.total = at + rec_layout(a).total;
    return l;
}

// fp32 alone: every bf16 gradient is on the tensor cores
template <int D, int DV>
cudaError_t run_grad(const DeltaArgs& a)
{
    const GradLayout l = grad_layout(a);
    unsigned char* ws = static_cast<unsigned char*>(a.ws);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    const GradKept kept = {f32(l.dS), f32(l.dV), f32(l.bb), f32(l.cd)};
    DeltaArgs f = a;
    f.out = nullptr, f.S_out = nullptr;
    cudaError_t e = run_rec<D, float>(f, f32(l.chk), f32(l.err), ws + l.seg);
    if (e != cudaSuccess)
        return e;
    const size_t rev = rev_smem<D>(), dqk = GradSmem<D, DV>::bytes;
    e = cudaFuncSetAttribute(k_delta_grad_rev<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)rev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_delta_grad_dqk<D, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)dqk);
    if (e != cudaSuccess)
        return e;
    const float* q = static_cast<const float*>(a.q);
    const float* k = static_cast<const float*>(a.k);
    const float* dout = static_cast<const float*>(a.dout);
    const int l2 = a.fm == LA_FM_L2, H = (int)a.H, Hk = (int)a.Hk;
    const int64_t BH = a.B * a.H;
    Segments seg = {1, 0, 0, nullptr, 0, nullptr, nullptr};
    const int n = rec_segments(a, &seg.len);
    auto reverse = [&](const Segments& x) {
        k_delta_grad_rev<D><<<dim3((unsigned)(BH * x.count), DV / 32), kRevThreads, rev, a.stream>>>(
            q, k, a.beta, a.log_alpha, dout, a.dS_out, f32(l.chk), f32(l.err),
            static_cast<float*>(a.dv_), a.dS0, kept, a.N, H, Hk, DV, l2, a.scale, x);
        count_launches(1);
        return cudaGetLastError();
    };
    if (n > 1) {  // M is where the recurrence's run left it
        const RecLayout r = rec_layout(a);
        float* start = f32(l.seg + r.start);
        float* C = f32(l.seg + r.B);
        const Segments ends = {n - 1, 1, seg.len, nullptr, 1, C, nullptr};
        if ((e = reverse(ends)) != cudaSuccess ||
            (e = delta::join_segments(a, true, a.dS_out, C, f32(l.seg + r.M), start, n, n)) != cudaSuccess)
            return e;
        seg.count = n, seg.start = start;
    }
    if ((e = reverse(seg)) != cudaSuccess)
        return e;
    k_delta_grad_dqk<D, DV><<<(unsigned)(BH * rec_blocks(a.N)), kGradThreads, dqk, a.stream>>>(
        q, k, a.beta, a.log_alpha, dout, f32(l.chk), f32(l.err), kept, f32(l.dq), f32(l.dk), a.dbeta,
        a.dlog_alpha, a.N, H, Hk, l2, a.scale);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    const int64_t rows = a.B * a.Hk * a.N;
    const unsigned grid = (unsigned)((rows + 7) / 8);
    k_delta_finish<D><<<grid, 256, 0, a.stream>>>(f32(l.dq), q, static_cast<float*>(a.dq), rows, a.N, H, Hk, l2,
                                                     a.scale);
    k_delta_finish<D><<<grid, 256, 0, a.stream>>>(f32(l.dk), k, static_cast<float*>(a.dk), rows, a.N, H, Hk, l2,
                                                     1.0f);
    count_launches(2);
    return cudaGetLastError();
}

template <int D>
cudaError_t grad_dims(const DeltaArgs& a)
{
    switch (a.dv) {
    case 32: return run_grad<D, 32>(a);
    case 64: return run_grad<D, 64>(a);
    default: return run_grad<D, 128>(a);
    }
}

}  // namespace

// The launches index blocks by a 32-bit grid: sequences, chunks and rows.
bool delta_grid_ok(const DeltaArgs& a)
{
    const int64_t most = INT32_MAX;
    return a.N <= most && rec_blocks(a.N) + 1 <= most / (a.B * a.H) && a.B * a.Hk <= most / (a.N > 0 ? a.N : 1);
}

namespace {

// The tensor-core forward pays for whole chunks of 64 tokens and two launches; the
// recurrence for every token, in rounds where its CTAs are more than the GPU holds
// (one per SM at d = 128, two below).  They meet near 64 tokens times rounds (us,
// recurrence and tensor cores): B4 H8 d = 128 8.7 and 14.4 at 32 tokens, 14.6 and 14.9
// at 64, 17.7 and 16.9 at 80; B8 H16 d = 128 (four rounds) 18.5 and 19.1 at 12, 26 and
// 19 at 24; B8 H32 d = 64 (two) 17.7 and 18.9 at 32, 25 and 19 at 44.  For 152 SMs by
// sizes alone: a workspace sized without the GPU at hand serves there.
bool forward_on_tensor_cores(const DeltaArgs& a)
{
    if (a.dtype != LA_BF16)
        return false;
    const int64_t held = a.d > 64 ? 152 : 2 * 152, ctas = a.B * a.H * (a.dv / kRecCols);
    return a.N > 64 || a.N * ((ctas + held - 1) / held) > 64;
}

// Its gradient is ahead at every length (8 tokens: 37 against 63 us at 32 heads,
// 172 against 370 us at 512).
bool backward_on_tensor_cores(const DeltaArgs& a) { return a.dtype == LA_BF16; }

}  // namespace

size_t delta_forward_workspace(const DeltaArgs& a)
{
    return forward_on_tensor_cores(a) ? delta_tc_forward_workspace(a) : rec_layout(a).total;
}

size_t delta_backward_workspace(const DeltaArgs& a)
{
    return backward_on_tensor_cores(a) ? delta_tc_backward_workspace(a) : grad_layout(a).total;
}

cudaError_t delta_forward(const DeltaArgs& a)
{
    if (forward_on_tensor_cores(a))
        return delta_tc_forward(a);
    const bool bf = a.dtype == LA_BF16;  // short: one segment
    unsigned char* ws = static_cast<unsigned char*>(a.ws);
    switch (a.d) {
    case 32: return bf ? run_rec<32, __nv_bfloat16>(a, nullptr, nullptr, ws) : run_rec<32, float>(a, nullptr, nullptr, ws);
    case 64: return bf ? run_rec<64, __nv_bfloat16>(a, nullptr, nullptr, ws) : run_rec<64, float>(a, nullptr, nullptr, ws);
    default: return bf ? run_rec<128, __nv_bfloat16>(a, nullptr, nullptr, ws) : run_rec<128, float>(a, nullptr, nullptr, ws);
    }
}

cudaError_t delta_decode(const DeltaArgs& a)
{
    const bool bf = a.dtype == LA_BF16;
    switch (a.d) {
    case 32: return bf ? run_decode<32, __nv_bfloat16>(a) : run_decode<32, float>(a);
    case 64: return bf ? run_decode<64, __nv_bfloat16>(a) : run_decode<64, float>(a);
    default: return bf ? run_decode<128, __nv_bfloat16>(a) : run_decode<128, float>(a);
    }
}

cudaError_t delta_backward(const DeltaArgs& a)
{
    if (backward_on_tensor_cores(a))
        return delta_tc_backward(a);
    switch (a.d) {
    case 32: return grad_dims<32>(a);
    case 64: return grad_dims<64>(a);
    default: return grad_dims<128>(a);
    }
}

}  // namespace la
