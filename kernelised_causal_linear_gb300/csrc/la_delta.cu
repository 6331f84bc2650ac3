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
// needs a barrier.  With S' = a_t S_{t-1} the two products S'^T k_t and
// S'^T q_t are taken in one pass over the registers, and
// o_t = scale (S'^T q_t + (k_t . q_t) beta_t e_t).
#include <math.h>

#include "la_delta.cuh"

namespace la {
namespace {

using delta::kL2Eps;

// ------------------------------------------------------ token recurrence ----
// 8 warps of 4 columns each; lane = 4 r + c holds rows 4 r .. 4 r + 3 of every
// 32 for column c.  Tokens are staged in blocks of kRecTok, q and k already
// normalised, so the step itself is D / 8 FMAs four times and three shuffles
// of two values.  Bound by the latency of that chain, once per token.
constexpr int kRecThreads = 256;
constexpr int kRecCols = 32;  // columns per CTA
constexpr int kRecTok = 32;   // tokens per staged block

template <int D, typename T>
__global__ void __launch_bounds__(kRecThreads)
    k_delta_rec(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                const float* __restrict__ beta, const float* __restrict__ log_alpha,
                T* __restrict__ out, const float* S0, float* S_out, float* __restrict__ chk,
                float* __restrict__ err, int64_t N, int H, int Hk, int DV, int l2, float scale)
{
    __shared__ __align__(16) float sk[kRecTok][D];
    __shared__ __align__(16) float sq[kRecTok][D];
    __shared__ float sv[kRecTok][kRecCols];
    __shared__ float so[kRecTok][kRecCols];
    __shared__ float sbeta[kRecTok], salpha[kRecTok], skq[kRecTok];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, col = warp * 4 + (lane & 3);
    const int64_t bh = blockIdx.x;
    const int c0 = blockIdx.y * kRecCols;
    const int64_t kh = bh / H * Hk + (bh % H) / (H / Hk);
    const T* qp = q ? q + kh * N * D : nullptr;
    const T* kp = k + kh * N * D;
    const T* vp = v + bh * N * DV + c0;
    const int64_t nblk = (N + kRecTok - 1) / kRecTok;

    float s[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
        s[i] = S0 ? S0[(bh * D + (i / 4) * 32 + 4 * r + i % 4) * DV + c0 + col] : 0.0f;

    for (int64_t b = 0; b < nblk; ++b) {
        const int64_t t0 = b * kRecTok;
        const int n = (int)min((int64_t)kRecTok, N - t0);
        __syncthreads();  // the previous block's tiles are read
        for (int t = warp; t < n; t += kRecThreads / 32) {
            float kk[D / 32], qq[D / 32], k2 = 0.f, q2 = 0.f, kq = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                kk[i] = to_f32<T>(kp[(t0 + t) * D + lane + 32 * i]);
                qq[i] = qp ? to_f32<T>(qp[(t0 + t) * D + lane + 32 * i]) : 0.f;
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
            const float rk = l2 ? rsqrtf(k2 + kL2Eps) : 1.0f;
            const float rq = (l2 ? rsqrtf(q2 + kL2Eps) : 1.0f) * scale;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                sk[t][lane + 32 * i] = kk[i] * rk;
                sq[t][lane + 32 * i] = qq[i] * rq;
            }
            sv[t][lane] = to_f32<T>(vp[(t0 + t) * DV + lane]);
            if (lane == 0) {
                skq[t] = kq * rk * rq;
                sbeta[t] = beta[bh * N + t0 + t];
                salpha[t] = log_alpha ? expf(log_alpha[bh * N + t0 + t]) : 1.0f;
            }
        }
        if (chk) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                chk[((bh * (nblk + 1) + b) * D + (i / 4) * 32 + 4 * r + i % 4) * DV + c0 + col] = s[i];
        }
        __syncthreads();
        for (int t = 0; t < n; ++t) {
            const float a = salpha[t];
            float pk = 0.f, pq = 0.f, kf[D / 8];
#pragma unroll
            for (int m = 0; m < D / 32; ++m) {
                const float4 x = *reinterpret_cast<const float4*>(&sk[t][32 * m + 4 * r]);
                const float4 y = *reinterpret_cast<const float4*>(&sq[t][32 * m + 4 * r]);
                kf[4 * m] = x.x, kf[4 * m + 1] = x.y, kf[4 * m + 2] = x.z, kf[4 * m + 3] = x.w;
                const float yf[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[4 * m + j] *= a;
                    pk = fmaf(kf[4 * m + j], s[4 * m + j], pk);
                    pq = fmaf(yf[j], s[4 * m + j], pq);
                }
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                pk += __shfl_xor_sync(0xffffffffu, pk, o);
                pq += __shfl_xor_sync(0xffffffffu, pq, o);
            }
            const float e = sv[t][col] - pk;
            const float u = sbeta[t] * e;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                s[i] = fmaf(kf[i], u, s[i]);
            if (r == 0) {
                so[t][col] = fmaf(skq[t], u, pq);
                if (err)
                    err[(bh * N + t0 + t) * DV + c0 + col] = e;
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
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        const int row = (i / 4) * 32 + 4 * r + i % 4;
        if (S_out)
            S_out[(bh * D + row) * DV + c0 + col] = s[i];
        if (chk)
            chk[((bh * (nblk + 1) + nblk) * D + row) * DV + c0 + col] = s[i];
    }
}

// ----------------------------------------------------------- decode step ----
// One token per head: the state is read once and written once (8 bytes per
// element) and everything else is small, so the step is bound by HBM.  A CTA
// owns D rows x CS columns; a thread keeps its rows of one 16-byte column
// group in registers between the two products and the update.
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
// Chunks of C = kRecTok tokens in reverse, one CTA per value head.  With G the
// running sum of log_alpha inside the chunk, D_ij = exp(G_i - G_j), U = beta E,
// S0 and S1 the states before and after the chunk, dS1 the gradient of S1:
//
//   P_ij = D_ij q_i.k_j (j <= i),  A_ij = D_ij k_i.k_j (j < i)
//   dU = P^T dO + diag(e^{G_C - G}) K dS1
//   Y  = (I + diag(beta) A)^{-T} dU      from the last token back, a column per thread
//   dV = beta Y,  dbeta_i = Y_i.E_i
//   dQ = (dO U^T o D) K + diag(e^G) dO S0^T
//   dK = (dO U^T o D)^T Q + M K + M^T K - diag(beta e^G) Y S0^T + diag(e^{G_C - G}) U dS1^T
//        with M_ij = -beta_i D_ij Y_i.U_j (j < i)
//   dS0 = e^{G_C} dS1 + (diag(e^G) Q)^T dO - (diag(beta e^G) K)^T Y
//   dlog_alpha_t = <S1, dS1> + sum_{i >= t in the chunk} (q_i.dQ_i - v_i.dV_i)
//
// (the last line: every place where G_i enters is a factor of o_i's or of
// e_i's right-hand side, and those products are q_i.dQ_i and v_i.dV_i).
// S0 and E come from the recurrence above, which stored them.  Everything is
// fp32 in shared memory; the products are bound by shared-memory reads.
constexpr int kGradThreads = 512;

template <int D, int DV>
struct GradSmem {
    static constexpr int C = kRecTok;
    static constexpr int LS = DV + 1, LK = D + 1, LV = DV + 1, LC = C + 1;
    static constexpr int floats = 2 * D * LS + 2 * C * LK + 3 * C * LV + 3 * C * LC + 8 * C + 32;
    static constexpr size_t bytes = sizeof(float) * floats;
    static_assert(bytes <= 232448, "shared memory");
};

template <int D, int DV, typename T>
__global__ void __launch_bounds__(kGradThreads)
    k_delta_grad(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                 const float* __restrict__ beta, const float* __restrict__ log_alpha,
                 const T* __restrict__ dout, const float* __restrict__ dS_out,
                 const float* __restrict__ chk, const float* __restrict__ err,
                 float* __restrict__ dq, float* __restrict__ dk, T* __restrict__ dv,
                 float* __restrict__ dbeta, float* __restrict__ dlog_alpha, float* dS0, int64_t N,
                 int H, int Hk, int l2, float scale)
{
    using SM = GradSmem<D, DV>;
    constexpr int C = SM::C, LS = SM::LS, LK = SM::LK, LV = SM::LV, LC = SM::LC;
    extern __shared__ __align__(16) float smem[];
    float* S = smem;             // [D][LS] state before the chunk
    float* dS = S + D * LS;      // [D][LS] gradient of the state after the chunk
    float* sk = dS + D * LS;     // [C][LK]
    float* sq = sk + C * LK;     // [C][LK], scaled
    float* sdo = sq + C * LK;    // [C][LV]
    float* se = sdo + C * LV;    // [C][LV]
    float* sy = se + C * LV;     // [C][LV]
    float* P = sy + C * LV;      // [C][LC] P, then dO U^T o D
    float* A = P + C * LC;       // [C][LC] A, then M
    float* Dm = A + C * LC;      // [C][LC] decay
    float* sb = Dm + C * LC;     // beta
    float* eg = sb + C;          // e^G
    float* ege = eg + C;         // e^{G_C - G}
    float* dG = ege + C;
    float* vdv = dG + C;
    float* red = vdv + C;        // [32]
    __shared__ double G[C];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int W = kGradThreads / 32;
    const int64_t bh = blockIdx.x;
    const int64_t kh = bh / H * Hk + (bh % H) / (H / Hk);
    const int64_t nblk = (N + C - 1) / C;
    const float* ck = chk + bh * (nblk + 1) * (int64_t)(D * DV);

    for (int i = tid; i < D * DV; i += kGradThreads) {
        S[i / DV * LS + i % DV] = ck[nblk * D * DV + i];
        dS[i / DV * LS + i % DV] = dS_out ? dS_out[bh * D * DV + i] : 0.f;
    }
    for (int64_t b = nblk - 1; b >= 0; --b) {
        const int64_t t0 = b * C;
        const int n = (int)min((int64_t)C, N - t0);
        __syncthreads();
        // <S1, dS1>, then S <- S0
        float dot = 0.f;
        for (int i = tid; i < D * DV; i += kGradThreads) {
            const int at = i / DV * LS + i % DV;
            dot = fmaf(S[at], dS[at], dot);
            S[at] = ck[b * D * DV + i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0)
            red[warp] = dot;
        // rows past the end stay zero and leave nothing behind (beta = 0, G constant)
        for (int t = warp; t < C; t += W) {
            float kk[D / 32], qq[D / 32], k2 = 0.f, q2 = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int64_t at = (kh * N + t0 + t) * D + lane + 32 * i;
                kk[i] = t < n ? to_f32<T>(k[at]) : 0.f;
                qq[i] = t < n ? to_f32<T>(q[at]) : 0.f;
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
            for (int c = lane; c < DV; c += 32) {
                const int64_t at = (bh * N + t0 + t) * DV + c;
                sdo[t * LV + c] = t < n ? to_f32<T>(dout[at]) : 0.f;
                se[t * LV + c] = t < n ? err[at] : 0.f;
            }
            if (lane == 0)
                sb[t] = t < n ? beta[bh * N + t0 + t] : 0.f;
        }
        if (warp == 0) {
            double g = log_alpha && lane < n ? (double)delta::clamp_gate(log_alpha[bh * N + t0 + lane]) : 0.0;
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
        __syncthreads();
        // P, A, D: a row per warp pass, a column j per lane
        for (int i = warp; i < C; i += W) {
            float p = 0.f, a = 0.f;
            for (int x = 0; x < D; ++x) {
                const float kj = sk[lane * LK + x];
                p = fmaf(sq[i * LK + x], kj, p);
                a = fmaf(sk[i * LK + x], kj, a);
            }
            const float dec = lane <= i ? expf((float)(G[i] - G[lane])) : 0.f;
            Dm[i * LC + lane] = dec;
            P[i * LC + lane] = lane <= i ? p * dec : 0.f;
            A[i * LC + lane] = lane < i ? a * dec : 0.f;
        }
        __syncthreads();
        // dU
        for (int at = tid; at < C * DV; at += kGradThreads) {
            const int j = at / DV, c = at % DV;
            float x = 0.f, y = 0.f;
            for (int i = j; i < C; ++i)
                x = fmaf(P[i * LC + j], sdo[i * LV + c], x);
            for (int i = 0; i < D; ++i)
                y = fmaf(sk[j * LK + i], dS[i * LS + c], y);
            sy[j * LV + c] = fmaf(ege[j], y, x);
        }
        __syncthreads();
        // Y, a column per thread
        if (tid < DV) {
            for (int j = C - 2; j >= 0; --j) {
                float y = sy[j * LV + tid];
                for (int i = j + 1; i < C; ++i)
                    y = fmaf(-sb[i] * A[i * LC + j], sy[i * LV + tid], y);
                sy[j * LV + tid] = y;
            }
        }
        __syncthreads();
        // dV, dbeta, v.dV; E becomes U
        for (int t = warp; t < C; t += W) {
            float db = 0.f, x = 0.f;
            for (int c = lane; c < DV; c += 32) {
                const float y = sy[t * LV + c], e = se[t * LV + c];
                db = fmaf(y, e, db);
                se[t * LV + c] = sb[t] * e;
                if (t < n) {
                    const int64_t at = (bh * N + t0 + t) * DV + c;
                    const float g = sb[t] * y;
                    dv[at] = from_f32<T>(g);
                    x = fmaf(g, to_f32<T>(v[at]), x);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                db += __shfl_xor_sync(0xffffffffu, db, o);
                x += __shfl_xor_sync(0xffffffffu, x, o);
            }
            if (lane == 0) {
                vdv[t] = x;
                if (t < n)
                    dbeta[bh * N + t0 + t] = db;
            }
        }
        __syncthreads();
        // P <- dO U^T o D, A <- M
        for (int i = warp; i < C; i += W) {
            float p = 0.f, m = 0.f;
            for (int c = 0; c < DV; ++c) {
                const float uj = se[lane * LV + c];
                p = fmaf(sdo[i * LV + c], uj, p);
                m = fmaf(sy[i * LV + c], uj, m);
            }
            const float dec = Dm[i * LC + lane];
            P[i * LC + lane] = p * dec;
            A[i * LC + lane] = lane < i ? -sb[i] * m * dec : 0.f;
        }
        __syncthreads();
        // dQ, q.dQ
        for (int i = warp; i < n; i += W) {
            float dot_q = 0.f;
            for (int x = lane; x < D; x += 32) {
                float z = 0.f, w = 0.f;
                for (int j = 0; j <= i; ++j)
                    z = fmaf(P[i * LC + j], sk[j * LK + x], z);
                for (int c = 0; c < DV; ++c)
                    w = fmaf(sdo[i * LV + c], S[x * LS + c], w);
                z = fmaf(eg[i], w, z);
                dot_q = fmaf(z, sq[i * LK + x], dot_q);
                dq[(bh * N + t0 + i) * D + x] = z;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                dot_q += __shfl_xor_sync(0xffffffffu, dot_q, o);
            if (lane == 0)
                dG[i] = dot_q - vdv[i];
        }
        // dK
        for (int j = warp; j < n; j += W) {
            for (int x = lane; x < D; x += 32) {
                float z = 0.f, w = 0.f, u = 0.f;
                for (int i = j; i < C; ++i)
                    z = fmaf(P[i * LC + j], sq[i * LK + x], z);
                for (int i = 0; i < C; ++i)
                    z = fmaf(i < j ? A[j * LC + i] : A[i * LC + j], sk[i * LK + x], z);
                for (int c = 0; c < DV; ++c) {
                    w = fmaf(sy[j * LV + c], S[x * LS + c], w);
                    u = fmaf(se[j * LV + c], dS[x * LS + c], u);
                }
                dk[(bh * N + t0 + j) * D + x] = z - sb[j] * eg[j] * w + ege[j] * u;
            }
        }
        __syncthreads();
        if (dlog_alpha && tid < n) {
            float x = 0.f;
            for (int w = 0; w < W; ++w)
                x += red[w];
            for (int i = n - 1; i >= tid; --i)
                x += dG[i];
            dlog_alpha[bh * N + t0 + tid] = x;
        }
        // dS <- dS0; S keeps S0, the next chunk's S1
        for (int at = tid; at < D * DV; at += kGradThreads) {
            const int x = at / DV, c = at % DV;
            float z = eg[C - 1] * dS[x * LS + c];
            for (int i = 0; i < C; ++i) {
                z = fmaf(eg[i] * sq[i * LK + x], sdo[i * LV + c], z);
                z = fmaf(-sb[i] * eg[i] * sk[i * LK + x], sy[i * LV + c], z);
            }
            dS[x * LS + c] = z;
        }
    }
    __syncthreads();
    if (dS0) {
        for (int i = tid; i < D * DV; i += kGradThreads)
            dS0[bh * D * DV + i] = dS[i / DV * LS + i % DV];
    }
}

// Gradients of the key heads' rows from those of the value heads that read
// them: summed in head order, through the scale and the L2 norm
// (x = u / l, l^2 = |u|^2 + eps: du = (dx - x (x.dx)) / l), rounded once.  A
// warp per row.
template <int D, typename T>
__global__ void __launch_bounds__(256)
    k_delta_finish(const float* __restrict__ g, const T* __restrict__ u, T* __restrict__ du,
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
        y[i] = to_f32<T>(u[row * D + lane + 32 * i]);
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
        du[row * D + lane + 32 * i] = from_f32<T>(x[i]);
}

// ----------------------------------------------------------------- hosts ----
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

int64_t rec_blocks(int64_t N) { return (N + kRecTok - 1) / kRecTok; }

template <int D, typename T>
cudaError_t run_rec(const DeltaArgs& a, float* chk, float* err)
{
    const dim3 grid((unsigned)(a.B * a.H), (unsigned)(a.dv / kRecCols));
    k_delta_rec<D, T><<<grid, kRecThreads, 0, a.stream>>>(
        static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.beta,
        a.log_alpha, static_cast<T*>(a.out), a.S0, a.S_out, chk, err, a.N, (int)a.H, (int)a.Hk,
        a.dv, a.fm == LA_FM_L2, a.scale);
    count_launches(1);
    return cudaGetLastError();
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
    size_t chk, err, dq, dk, total;
};
GradLayout grad_layout(const DeltaArgs& a)
{
    const size_t BH = (size_t)(a.B * a.H), N = (size_t)a.N;
    GradLayout l;
    l.chk = 0;
    l.err = up256(4 * BH * ((size_t)rec_blocks(a.N) + 1) * a.d * a.dv);
    l.dq = l.err + up256(4 * BH * N * a.dv);
    l.dk = l.dq + up256(4 * BH * N * a.d);
    l.total = l.dk + up256(4 * BH * N * a.d);
    return l;
}

template <int D, int DV, typename T>
cudaError_t run_grad(const DeltaArgs& a)
{
    const GradLayout l = grad_layout(a);
    unsigned char* ws = static_cast<unsigned char*>(a.ws);
    float* chk = reinterpret_cast<float*>(ws + l.chk);
    float* err = reinterpret_cast<float*>(ws + l.err);
    float* dq = reinterpret_cast<float*>(ws + l.dq);
    float* dk = reinterpret_cast<float*>(ws + l.dk);
    DeltaArgs f = a;
    f.out = nullptr, f.S_out = nullptr;
    cudaError_t e = run_rec<D, T>(f, chk, err);
    if (e != cudaSuccess)
        return e;
    auto kern = k_delta_grad<D, DV, T>;
    const size_t smem = GradSmem<D, DV>::bytes;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    const T* q = static_cast<const T*>(a.q);
    const T* k = static_cast<const T*>(a.k);
    const int l2 = a.fm == LA_FM_L2;
    kern<<<(unsigned)(a.B * a.H), kGradThreads, smem, a.stream>>>(
        q, k, static_cast<const T*>(a.v), a.beta, a.log_alpha, static_cast<const T*>(a.dout),
        a.dS_out, chk, err, dq, dk, static_cast<T*>(a.dv_), a.dbeta, a.dlog_alpha, a.dS0, a.N,
        (int)a.H, (int)a.Hk, l2, a.scale);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    const int64_t rows = a.B * a.Hk * a.N;
    const unsigned grid = (unsigned)((rows + 7) / 8);
    k_delta_finish<D, T><<<grid, 256, 0, a.stream>>>(dq, q, static_cast<T*>(a.dq), rows, a.N,
                                                     (int)a.H, (int)a.Hk, l2, a.scale);
    k_delta_finish<D, T><<<grid, 256, 0, a.stream>>>(dk, k, static_cast<T*>(a.dk), rows, a.N,
                                                     (int)a.H, (int)a.Hk, l2, 1.0f);
    count_launches(2);
    return cudaGetLastError();
}

template <int D, int DV>
cudaError_t grad_type(const DeltaArgs& a)
{
    return a.dtype == LA_BF16 ? run_grad<D, DV, __nv_bfloat16>(a) : run_grad<D, DV, float>(a);
}
template <int D>
cudaError_t grad_dims(const DeltaArgs& a)
{
    switch (a.dv) {
    case 32: return grad_type<D, 32>(a);
    case 64: return grad_type<D, 64>(a);
    default: return grad_type<D, 128>(a);
    }
}

}  // namespace

// The launches index blocks by a 32-bit grid: sequences, chunks and rows.
bool delta_grid_ok(const DeltaArgs& a)
{
    const int64_t most = INT32_MAX;
    return a.N <= most && rec_blocks(a.N) + 1 <= most / (a.B * a.H) && a.B * a.Hk <= most / (a.N > 0 ? a.N : 1);
}

size_t delta_forward_workspace(const DeltaArgs& a)
{
    return delta_tc_eligible(a) ? delta_tc_forward_workspace(a) : 0;
}

size_t delta_backward_workspace(const DeltaArgs& a)
{
    return delta_tc_eligible(a) ? delta_tc_backward_workspace(a) : grad_layout(a).total;
}

cudaError_t delta_forward(const DeltaArgs& a)
{
    if (delta_tc_eligible(a))
        return delta_tc_forward(a);
    const bool bf = a.dtype == LA_BF16;
    switch (a.d) {
    case 32: return bf ? run_rec<32, __nv_bfloat16>(a, nullptr, nullptr) : run_rec<32, float>(a, nullptr, nullptr);
    case 64: return bf ? run_rec<64, __nv_bfloat16>(a, nullptr, nullptr) : run_rec<64, float>(a, nullptr, nullptr);
    default: return bf ? run_rec<128, __nv_bfloat16>(a, nullptr, nullptr) : run_rec<128, float>(a, nullptr, nullptr);
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
    if (delta_tc_eligible(a))
        return delta_tc_backward(a);
    switch (a.d) {
    case 32: return grad_dims<32>(a);
    case 64: return grad_dims<64>(a);
    default: return grad_dims<128>(a);
    }
}

}  // namespace la
