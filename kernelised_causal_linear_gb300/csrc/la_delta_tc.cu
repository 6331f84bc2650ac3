// la_delta_tc.cu -- gated delta rule on the tensor cores (bf16 inputs).
//
// Chunks of C = 64 tokens.  Inside a chunk, with G the running sum of
// log_alpha, D_ij = exp(G_i - G_j), A_ij = D_ij k_i.k_j (j < i) and S0 the state
// before it, the errors of all tokens solve one triangular system:
//
//   (I + A diag(beta)) E = R,   R = V - diag(e^G) K S0,   U = diag(beta) E
//   O  = scale (diag(e^G) Q S0 + P U),  P_ij = D_ij q_i.k_j (j <= i)
//   S1 = e^{G_C} S0 + (diag(e^{G_C - G}) K)^T U
//
// With F = -(I + A diag(beta))^{-1} A the solution is E = R + F (beta R): the
// large part R enters as it is, and only the correction is a product.
//
// Two launches.
//   k_delta_prep   every chunk and value head on its own: scaled fp16 images of
//                  K and Q, F, P and the factors of each token.  Nothing here
//                  depends on the state.
//   k_delta_chain  the chunks of a sequence in order.  The columns of S never
//                  mix, so a warp owns 16 value columns for the whole sequence
//                  and keeps S^T [16 x d] in registers as MMA accumulators.
//                  Everything is computed transposed: S^T K^T, E^T = R^T + ..,
//                  S^T += U^T K.  The accumulators of one product are the A
//                  fragments of the next (see la_delta_tc.cuh), so between a
//                  chunk's products nothing passes through shared memory and no
//                  other warp is waited for.
#include "la_delta_tc.cuh"

namespace la {
namespace {

using namespace delta;

// What k_delta_prep writes per chunk and value head: [F hi][F lo][P][factors],
// tiles of 64 x 64 fp16 in the layout the chain reads them from shared memory.
enum Factor {
    kFacA,   // e^G_i |k_i| scale: R = v - fac * (K16 S)
    kFacF,   // scale of F's row
    kFacB,   // beta
    kFacO,   // e^G_i, q's scale and norm: inter-chunk part of o
    kFacP,   // scale of P's row
    kFacW,   // e^{G_C - G_j} beta_j, k's scale and norm: the state update
    kFacEnd, // [0] = e^{G_C}
    kFactors
};
constexpr int kTile = kC * kC * 2;  // bytes of a 64 x 64 fp16 tile
constexpr int kFacBytes = kFactors * kC * 4;
constexpr int kBlob = 3 * kTile + kFacBytes;

template <int D>
constexpr int row_image()  // bytes of K16 or Q16 per chunk
{
    return kC * D * 2;
}

// ------------------------------------------------------------- k_delta_prep --
// 4 warps.  The Gram products are exact fp16 MMAs on the lower blocks; F is
// fp32 on the CUDA cores in 16 x 16 blocks: the diagonal ones by substitution
// (a column per lane), then by distance from the diagonal
//   X = A_IJ + sum_{J <= L < I} A_IL beta_L F_LJ,   F_IJ = -X - F_II beta_I X.
constexpr int kPrepThreads = 128;
constexpr int kLd = 68;  // row stride of the fp32 tiles (16-byte rows, spread over banks)

template <int D>
struct PrepSmem {
    static constexpr int img = 2 * row_image<D>() > 3 * kTile ? 2 * row_image<D>() : 3 * kTile;
    static constexpr int A = img;
    static constexpr int F = A + kC * kLd * 4;
    static constexpr int X = F + kC * kLd * 4;
    static constexpr int vec = X + 4 * 16 * 20 * 4;
    static constexpr int bytes = vec + 12 * kC * 4;
};

template <int D>
__global__ void __launch_bounds__(kPrepThreads)
    k_delta_prep(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                 const float* __restrict__ beta, const float* __restrict__ log_alpha,
                 unsigned char* __restrict__ rows, unsigned char* __restrict__ blobs, int64_t N,
                 int nchunk, int H, int Hk, int l2, float scale)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    using SM = PrepSmem<D>;
    constexpr int RB = 2 * D;  // bytes per row
    float* sA = reinterpret_cast<float*>(smem + SM::A);
    float* sF = reinterpret_cast<float*>(smem + SM::F);
    float* vec = reinterpret_cast<float*>(smem + SM::vec);
    float *fk = vec, *fq = vec + kC, *gh = vec + 2 * kC, *gl = vec + 3 * kC, *sb = vec + 4 * kC;
    float* fac = vec + 5 * kC;  // [kFactors][kC]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t bh = blockIdx.x / nchunk;
    const int c = blockIdx.x % nchunk;
    const int per = H / Hk;
    const int64_t kh = bh / H * Hk + (bh % H) / per;
    const int64_t t0 = (int64_t)c * kC;
    const int n = (int)min((int64_t)kC, N - t0);
    const uint32_t sK = smem_addr(smem), sQ = sK + row_image<D>();

    // rows: scaled fp16 images and factors
    constexpr int LPR = D / 8, RPP = kPrepThreads / LPR;
#pragma unroll 4
    for (int r0 = 0; r0 < kC; r0 += RPP) {
        const int r = r0 + tid / LPR, p = tid % LPR;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const __nv_bfloat16* src = which ? q : k;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (r < n && src)
                w = *reinterpret_cast<const uint4*>(src + (kh * N + t0 + r) * D + p * 8);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            float f[8], ss = 0.f, mx = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(u[i] << 16);
                f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = fmaf(f[i], f[i], ss);
                mx = max_abs(mx, f[i]);
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            }
            const Pow2 s = pow2_for(mx);
            uint4 h;
            h.x = h2(f[0] * s.to, f[1] * s.to);
            h.y = h2(f[2] * s.to, f[3] * s.to);
            h.z = h2(f[4] * s.to, f[5] * s.to);
            h.w = h2(f[6] * s.to, f[7] * s.to);
            *reinterpret_cast<uint4*>(smem + (which ? row_image<D>() : 0) + tile_off<RB>(r, p)) = h;
            if (p == 0)
                (which ? fq : fk)[r] = s.from * (l2 ? rsqrtf(ss + kL2Eps) : 1.0f) * (which ? scale : 1.0f);
        }
    }
    // running sums of the gates in base 2, as a multiple of 2^-6 (exact: below
    // 2^14) and a rest, so that differences of far sums keep their low bits
    if (warp == 0) {
        float h0 = 0.f, l0 = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = lane + 32 * half;
            float h = 0.f, l = 0.f;
            if (log_alpha && t < n) {
                const float g = clamp_gate(log_alpha[bh * N + t0 + t]);
                const float g2 = g * 1.44269504f;
                const float rest = fmaf(g, 1.44269504f, -g2) + g * 1.92596299e-8f;
                h = rintf(g2 * 64.0f) * 0.015625f;
                l = (g2 - h) + rest;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float x = __shfl_up_sync(0xffffffffu, h, o), y = __shfl_up_sync(0xffffffffu, l, o);
                if (lane >= o)
                    h += x, l += y;
            }
            h += h0, l += l0;
            h0 = __shfl_sync(0xffffffffu, h, 31), l0 = __shfl_sync(0xffffffffu, l, 31);
            gh[t] = h, gl[t] = l;
            sb[t] = t < n ? beta[bh * N + t0 + t] : 0.f;
        }
    }
    __syncthreads();

    // Gram products, row block `warp`, column blocks 0 .. warp
    const int g = lane >> 2, tq = lane & 3;
    float ak[8][4], aq[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            ak[i][j] = aq[i][j] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D; kk += 16) {
        uint32_t a[4], b[4], x[4];
        ldsm4(a, addr_a<RB>(sK, lane, 16 * warp, kk));
        ldsm4(x, addr_a<RB>(sQ, lane, 16 * warp, kk));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j <= warp) {
                ldsm4(b, addr_b<RB>(sK, lane, 16 * j, kk));
                mma(ak[2 * j], a, b[0], b[1]);
                mma(ak[2 * j + 1], a, b[2], b[3]);
                mma(aq[2 * j], x, b[0], b[1]);
                mma(aq[2 * j + 1], x, b[2], b[3]);
            }
        }
    }
    // the images go out; one value head of a key head writes them
    if ((bh % H) % per == 0) {
        uint4* dst = reinterpret_cast<uint4*>(rows + (kh * nchunk + c) * (int64_t)(2 * row_image<D>()));
        for (int i = tid; i < 2 * row_image<D>() / 16; i += kPrepThreads)
            dst[i] = reinterpret_cast<const uint4*>(smem)[i];
    }
    __syncthreads();  // the images are read: F and P take their place

    const int i0 = 16 * warp + g;
    float pm[2] = {0.f, 0.f};
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + (e >> 1) * 8, j = 8 * nt + 2 * tq + (e & 1);
            const float dec = j <= i ? exp2f((gh[i] - gh[j]) + (gl[i] - gl[j])) : 0.f;
            sA[i * kLd + j] = j < i ? ak[nt][e] * fk[i] * fk[j] * dec : 0.f;
            aq[nt][e] = j <= i ? aq[nt][e] * fq[i] * fk[j] * dec * sb[j] : 0.f;
            pm[e >> 1] = max_abs(pm[e >> 1], aq[nt][e]);
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const Pow2 s = pow2_for(quad_max(pm[r]));
        const int i = i0 + 8 * r;
        if (tq == 0)
            fac[kFacP * kC + i] = s.from;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
            *reinterpret_cast<uint32_t*>(smem + 2 * kTile + tile_off<128>(i, nt) + 4 * tq) =
                h2(aq[nt][2 * r] * s.to, aq[nt][2 * r + 1] * s.to);
    }
    if (tid < kC) {
        const float e = exp2f(gh[tid] + gl[tid]);
        const float w = exp2f((gh[kC - 1] - gh[tid]) + (gl[kC - 1] - gl[tid]));
        fac[kFacA * kC + tid] = e * fk[tid];
        fac[kFacB * kC + tid] = sb[tid];
        fac[kFacO * kC + tid] = e * fq[tid];
        fac[kFacW * kC + tid] = w * fk[tid] * sb[tid];
        fac[kFacEnd * kC + tid] = exp2f(gh[kC - 1] + gl[kC - 1]);
    }
    __syncthreads();

    // F, diagonal blocks: column `lane & 15` of block `warp`
    {
        const int b = 16 * warp, j = lane & 15;
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float x = -sA[(b + i) * kLd + b + j];
#pragma unroll
            for (int l = 0; l < i; ++l)
                x = fmaf(-sA[(b + i) * kLd + b + l] * sb[b + l], f[l], x);
            f[i] = x;
        }
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                sF[(b + i) * kLd + b + j] = f[i];
        }
    }
    __syncthreads();
    float* sX = reinterpret_cast<float*>(smem + SM::X) + warp * 16 * 20;
    for (int dist = 1; dist < 4; ++dist) {
        const int J = warp, I = J + dist;
        if (I < 4) {
            const int r = lane >> 1, c0 = (lane & 1) * 8;
            const float* arow = sA + (16 * I + r) * kLd;
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = arow[16 * J + c0 + i];
            for (int l = 16 * J; l < 16 * I; ++l) {
                const float a = arow[l] * sb[l];
                const float4 u = *reinterpret_cast<const float4*>(sF + l * kLd + 16 * J + c0);
                const float4 v = *reinterpret_cast<const float4*>(sF + l * kLd + 16 * J + c0 + 4);
                x[0] = fmaf(a, u.x, x[0]), x[1] = fmaf(a, u.y, x[1]);
                x[2] = fmaf(a, u.z, x[2]), x[3] = fmaf(a, u.w, x[3]);
                x[4] = fmaf(a, v.x, x[4]), x[5] = fmaf(a, v.y, x[5]);
                x[6] = fmaf(a, v.z, x[6]), x[7] = fmaf(a, v.w, x[7]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sX[r * 20 + c0 + i] = x[i];
            __syncwarp();
            const float* frow = sF + (16 * I + r) * kLd + 16 * I;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = -x[i];
            for (int l = 0; l < r; ++l) {
                const float a = -frow[l] * sb[16 * I + l];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] = fmaf(a, sX[l * 20 + c0 + i], x[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sF[(16 * I + r) * kLd + 16 * J + c0 + i] = x[i];
            __syncwarp();
        }
        __syncthreads();
    }
    // F to two fp16 parts, rows scaled; two threads per row
    {
        const int r = tid >> 1, half = (tid & 1) * 32;
        float f[32], m = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            f[i] = half + i < r ? sF[r * kLd + half + i] : 0.f;
            m = max_abs(m, f[i]);
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const Pow2 s = pow2_for(m);
        if (half == 0)
            fac[kFacF * kC + r] = s.from;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            uint4 hi, lo;
            h2_split(f[i] * s.to, f[i + 1] * s.to, hi.x, lo.x);
            h2_split(f[i + 2] * s.to, f[i + 3] * s.to, hi.y, lo.y);
            h2_split(f[i + 4] * s.to, f[i + 5] * s.to, hi.z, lo.z);
            h2_split(f[i + 6] * s.to, f[i + 7] * s.to, hi.w, lo.w);
            const uint32_t at = tile_off<128>(r, (half + i) >> 3);
            *reinterpret_cast<uint4*>(smem + at) = hi;
            *reinterpret_cast<uint4*>(smem + kTile + at) = lo;
        }
    }
    __syncthreads();
    uint4* blob = reinterpret_cast<uint4*>(blobs + (bh * nchunk + c) * (int64_t)kBlob);
    for (int i = tid; i < 3 * kTile / 16; i += kPrepThreads)
        blob[i] = reinterpret_cast<const uint4*>(smem)[i];
    for (int i = tid; i < kFacBytes / 16; i += kPrepThreads)
        blob[3 * kTile / 16 + i] = reinterpret_cast<const uint4*>(fac)[i];
}

// ------------------------------------------------------------ k_delta_chain --
// W warps of 16 value columns.  The tiles of a chunk are shared by the warps and
// arrive by bulk copies kStages chunks ahead; a warp's own columns of V come by
// cp.async one chunk ahead, and its outputs leave through its own tile, turned
// back to token-major by stmatrix.
constexpr int kStages = 2;
constexpr uint32_t kWaitPolls = 1u << 22;

template <int D>
struct ChainSmem {
    static constexpr int stage = 2 * row_image<D>() + kBlob;
    static constexpr int v = kStages * stage;  // per warp: V twice, O
    static constexpr int per_warp = 3 * kC * 32;
    static int bytes(int W) { return v + W * per_warp + 64; }
};

template <int D>
__global__ void __launch_bounds__(256, 1)
    k_delta_chain(const unsigned char* __restrict__ rows, const unsigned char* __restrict__ blobs,
                  const __nv_bfloat16* __restrict__ v, __nv_bfloat16* __restrict__ out,
                  const float* S0, float* S_out, int64_t N, int nchunk, int H, int Hk, int DV,
                  int* status)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    using SM = ChainSmem<D>;
    constexpr int RB = 2 * D, NT = D / 8;  // bytes per row; n tiles of S^T
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, W = blockDim.x >> 5;
    const int g = lane >> 2, tq = lane & 3;
    const int slices = DV / (16 * W);
    const int64_t bh = blockIdx.x / slices;
    const int col0 = (blockIdx.x % slices) * 16 * W + 16 * warp;
    const int64_t kh = bh / H * Hk + (bh % H) / (H / Hk);
    const uint32_t base = smem_addr(smem);
    const uint32_t sv = base + SM::v + warp * SM::per_warp, so = sv + 2 * kC * 32;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::v + W * SM::per_warp);
    const unsigned char* row_src = rows + kh * nchunk * (int64_t)(2 * row_image<D>());
    const unsigned char* blob_src = blobs + bh * nchunk * (int64_t)kBlob;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i)
            sm100::mbar_init(full + i, 1);
        sm100::fence_mbar_init();
    }
    __syncthreads();
    auto load_stage = [&](int c) {
        const uint32_t dst = base + (c % kStages) * SM::stage;
        uint64_t* bar = full + c % kStages;
        sm100::mbar_arrive_expect_tx(bar, SM::stage);
        delta::bulk_load(dst, row_src + c * (int64_t)(2 * row_image<D>()), 2 * row_image<D>(), bar);
        delta::bulk_load(dst + 2 * row_image<D>(), blob_src + c * (int64_t)kBlob, kBlob, bar);
    };
    auto load_v = [&](int c) {
        const int64_t t0 = (int64_t)c * kC;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = (lane >> 1) + 16 * i, p = lane & 1;
            const bool live = t0 + t < N;
            cp16(sv + (c & 1) * kC * 32 + tile_off<32>(t, p),
                 v + (bh * N + (live ? t0 + t : 0)) * DV + col0 + p * 8, live);
        }
    };
    if (tid == 0)
        for (int c = 0; c < kStages && c < nchunk; ++c)
            load_stage(c);
    load_v(0);
    cp_commit();

    float s[NT][4];  // S^T[col0 + g, + 8][8 nt + 2 tq, + 1]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s[nt][e] = S0 ? S0[(bh * D + 8 * nt + 2 * tq + (e & 1)) * DV + col0 + g + (e >> 1) * 8] : 0.f;

    bool ok = true;
    int c = 0;
    for (; c < nchunk; ++c) {
        const uint32_t st = base + (c % kStages) * SM::stage;
        const uint32_t sK = st, sQ = st + row_image<D>(), sFh = st + 2 * row_image<D>();
        const float* fac = reinterpret_cast<const float*>(smem + (c % kStages) * SM::stage +
                                                          2 * row_image<D>() + 3 * kTile);
        if (c + 1 < nchunk)
            load_v(c + 1);
        cp_commit();
        ok = ok && sm100::mbar_wait(full + c % kStages, (c / kStages) & 1, kWaitPolls);
        cp_wait<1>();
        __syncwarp();
        if (ok) {
            // S^T K^T and S^T Q^T, S split on the way
            float m0 = 0.f, m1 = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                m0 = max_abs(max_abs(m0, s[nt][0]), s[nt][1]);
                m1 = max_abs(max_abs(m1, s[nt][2]), s[nt][3]);
            }
            m0 = quad_max(m0), m1 = quad_max(m1);
            const Pow2 p0 = pow2_for(m0), p1 = pow2_for(m1);
            float r[8][4], o[8][4];
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    r[nt][e] = o[nt][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t hi[4], lo[4], b[4];
                h2_split(s[2 * kk][0] * p0.to, s[2 * kk][1] * p0.to, hi[0], lo[0]);
                h2_split(s[2 * kk][2] * p1.to, s[2 * kk][3] * p1.to, hi[1], lo[1]);
                h2_split(s[2 * kk + 1][0] * p0.to, s[2 * kk + 1][1] * p0.to, hi[2], lo[2]);
                h2_split(s[2 * kk + 1][2] * p1.to, s[2 * kk + 1][3] * p1.to, hi[3], lo[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ldsm4(b, addr_b<RB>(sK, lane, 16 * j, 16 * kk));
                    mma(r[2 * j], hi, b[0], b[1]);
                    mma(r[2 * j + 1], hi, b[2], b[3]);
                    mma(r[2 * j], lo, b[0], b[1]);
                    mma(r[2 * j + 1], lo, b[2], b[3]);
                    if (out) {
                        ldsm4(b, addr_b<RB>(sQ, lane, 16 * j, 16 * kk));
                        mma(o[2 * j], hi, b[0], b[1]);
                        mma(o[2 * j + 1], hi, b[2], b[3]);
                    }
                }
            }
            // R, and the largest |beta R| of a column
            float br0 = 0.f, br1 = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
                ldsm4t(w, addr_ct<32>(sv + (c & 1) * kC * 32, lane, 16 * j, 0));
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int nt = 2 * j + u;
                    const float2 a = *reinterpret_cast<const float2*>(fac + kFacA * kC + 8 * nt + 2 * tq);
                    const float2 be = *reinterpret_cast<const float2*>(fac + kFacB * kC + 8 * nt + 2 * tq);
                    r[nt][0] = __uint_as_float(w[2 * u] << 16) - a.x * (r[nt][0] * p0.from);
                    r[nt][1] = __uint_as_float(w[2 * u] & 0xffff0000u) - a.y * (r[nt][1] * p0.from);
                    r[nt][2] = __uint_as_float(w[2 * u + 1] << 16) - a.x * (r[nt][2] * p1.from);
                    r[nt][3] = __uint_as_float(w[2 * u + 1] & 0xffff0000u) - a.y * (r[nt][3] * p1.from);
                    br0 = max_abs(max_abs(br0, be.x * r[nt][0]), be.y * r[nt][1]);
                    br1 = max_abs(max_abs(br1, be.x * r[nt][2]), be.y * r[nt][3]);
                    if (out) {
                        const float2 fo = *reinterpret_cast<const float2*>(fac + kFacO * kC + 8 * nt + 2 * tq);
                        o[nt][0] *= fo.x * p0.from, o[nt][1] *= fo.y * p0.from;
                        o[nt][2] *= fo.x * p1.from, o[nt][3] *= fo.y * p1.from;
                    }
                }
            }
            // E = R + F (beta R)
            float x[8][4];
            const Pow2 b0 = pow2_for(quad_max(br0)), b1 = pow2_for(quad_max(br1));
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[nt][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t hi[4], lo[4], b[4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int nt = 2 * kk + u;
                    const float2 be = *reinterpret_cast<const float2*>(fac + kFacB * kC + 8 * nt + 2 * tq);
                    h2_split(be.x * r[nt][0] * b0.to, be.y * r[nt][1] * b0.to, hi[2 * u], lo[2 * u]);
                    h2_split(be.x * r[nt][2] * b1.to, be.y * r[nt][3] * b1.to, hi[2 * u + 1], lo[2 * u + 1]);
                }
#pragma unroll
                for (int j = kk; j < 4; ++j) {  // F is strictly lower
                    ldsm4(b, addr_b<128>(sFh, lane, 16 * j, 16 * kk));
                    mma(x[2 * j], hi, b[0], b[1]);
                    mma(x[2 * j + 1], hi, b[2], b[3]);
                    mma(x[2 * j], lo, b[0], b[1]);
                    mma(x[2 * j + 1], lo, b[2], b[3]);
                    ldsm4(b, addr_b<128>(sFh + kTile, lane, 16 * j, 16 * kk));
                    mma(x[2 * j], hi, b[0], b[1]);
                    mma(x[2 * j + 1], hi, b[2], b[3]);
                }
            }
            float e0 = 0.f, e1 = 0.f, w0 = 0.f, w1 = 0.f;
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float2 f = *reinterpret_cast<const float2*>(fac + kFacF * kC + 8 * nt + 2 * tq);
                const float2 w = *reinterpret_cast<const float2*>(fac + kFacW * kC + 8 * nt + 2 * tq);
                r[nt][0] = fmaf(f.x * b0.from, x[nt][0], r[nt][0]);
                r[nt][1] = fmaf(f.y * b0.from, x[nt][1], r[nt][1]);
                r[nt][2] = fmaf(f.x * b1.from, x[nt][2], r[nt][2]);
                r[nt][3] = fmaf(f.y * b1.from, x[nt][3], r[nt][3]);
                e0 = max_abs(max_abs(e0, r[nt][0]), r[nt][1]);
                e1 = max_abs(max_abs(e1, r[nt][2]), r[nt][3]);
                w0 = max_abs(max_abs(w0, w.x * r[nt][0]), w.y * r[nt][1]);
                w1 = max_abs(max_abs(w1, w.x * r[nt][2]), w.y * r[nt][3]);
            }
            // O: P carries beta; one fp16 part of E (2^-12 of a term, under the
            // output's own rounding)
            if (out) {
                const Pow2 q0 = pow2_for(quad_max(e0)), q1 = pow2_for(quad_max(e1));
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[nt][e] = 0.f;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t a[4] = {h2(r[2 * kk][0] * q0.to, r[2 * kk][1] * q0.to),
                                           h2(r[2 * kk][2] * q1.to, r[2 * kk][3] * q1.to),
                                           h2(r[2 * kk + 1][0] * q0.to, r[2 * kk + 1][1] * q0.to),
                                           h2(r[2 * kk + 1][2] * q1.to, r[2 * kk + 1][3] * q1.to)};
                    uint32_t b[4];
#pragma unroll
                    for (int j = kk; j < 4; ++j) {
                        ldsm4(b, addr_b<128>(sFh + 2 * kTile, lane, 16 * j, 16 * kk));
                        mma(x[2 * j], a, b[0], b[1]);
                        mma(x[2 * j + 1], a, b[2], b[3]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t w[4];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int nt = 2 * j + u;
                        const float2 fp = *reinterpret_cast<const float2*>(fac + kFacP * kC + 8 * nt + 2 * tq);
                        w[2 * u] = sm100::pack_bf16x2(fmaf(fp.x * q0.from, x[nt][0], o[nt][0]),
                                                      fmaf(fp.y * q0.from, x[nt][1], o[nt][1]));
                        w[2 * u + 1] = sm100::pack_bf16x2(fmaf(fp.x * q1.from, x[nt][2], o[nt][2]),
                                                          fmaf(fp.y * q1.from, x[nt][3], o[nt][3]));
                    }
                    stsm4t(addr_ct<32>(so, lane, 16 * j, 0), w);
                }
            }
            // S1 = e^{G_C} S0 + (W E)^T K16 on accumulators scaled with the operand:
            // both under one power of two, so neither overflows nor loses bits the
            // other does not drown
            const float gend = fac[kFacEnd * kC];
            const Pow2 u0 = pow2_for(fmaxf(quad_max(w0), m0 * gend * 0.00390625f));
            const Pow2 u1 = pow2_for(fmaxf(quad_max(w1), m1 * gend * 0.00390625f));
            const float g0 = gend * u0.to, g1 = gend * u1.to;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                s[nt][0] *= g0, s[nt][1] *= g0;
                s[nt][2] *= g1, s[nt][3] *= g1;
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t hi[4], lo[4], b[4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int nt = 2 * kk + u;
                    const float2 w = *reinterpret_cast<const float2*>(fac + kFacW * kC + 8 * nt + 2 * tq);
                    h2_split(w.x * r[nt][0] * u0.to, w.y * r[nt][1] * u0.to, hi[2 * u], lo[2 * u]);
                    h2_split(w.x * r[nt][2] * u1.to, w.y * r[nt][3] * u1.to, hi[2 * u + 1], lo[2 * u + 1]);
                }
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) {
                    ldsm4t(b, addr_bt<RB>(sK, lane, 16 * kk, 16 * j));
                    mma(s[2 * j], hi, b[0], b[1]);
                    mma(s[2 * j + 1], hi, b[2], b[3]);
                    mma(s[2 * j], lo, b[0], b[1]);
                    mma(s[2 * j + 1], lo, b[2], b[3]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                s[nt][0] *= u0.from, s[nt][1] *= u0.from;
                s[nt][2] *= u1.from, s[nt][3] *= u1.from;
            }
            if (out) {
                __syncwarp();
                const int64_t t0 = (int64_t)c * kC;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = (lane >> 1) + 16 * i, p = lane & 1;
                    if (t0 + t < N)
                        *reinterpret_cast<uint4*>(out + (bh * N + t0 + t) * DV + col0 + p * 8) =
                            *reinterpret_cast<const uint4*>(smem + (so - base) + tile_off<32>(t, p));
                }
            }
        }
        ok = __syncthreads_and(ok);  // every warp is done with the stage
        if (!ok)
            break;
        if (tid == 0 && c + kStages < nchunk)
            load_stage(c + kStages);
    }
    cp_wait<0>();
    if (!ok) {  // a copy never arrived: see the others home, report, leave
        if (tid == 0) {
            for (int i = c; i < c + kStages && i < nchunk; ++i)
                sm100::mbar_wait(full + i % kStages, (i / kStages) & 1, kWaitPolls);
            set_status(status, LA_ERR_TIMEOUT);
        }
        return;
    }
    if (S_out) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S_out[(bh * D + 8 * nt + 2 * tq + (e & 1)) * DV + col0 + g + (e >> 1) * 8] = s[nt][e];
    }
}

// ------------------------------------------------------------------- hosts --
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
int chunks_of(int64_t N) { return (int)((N + kC - 1) / kC); }

struct TcLayout {
    size_t rows, blobs, total;
};
TcLayout tc_layout(const DeltaArgs& a)
{
    TcLayout l;
    const size_t n = (size_t)chunks_of(a.N);
    l.rows = 0;
    l.blobs = up256((size_t)(a.B * a.Hk) * n * 2 * kC * a.d * 2);
    l.total = l.blobs + up256((size_t)(a.B * a.H) * n * kBlob);
    return l;
}

// Warps per CTA of the chain: as few as give no more CTAs than SMs (a warp alone
// on its sub-partition has that tensor core to itself), at most all columns.
int chain_warps(const DeltaArgs& a)
{
    const int most = a.dv / 16, sms = device_sm_count();
    int W = 1;
    while (W < most && a.B * a.H * (most / W) > sms)
        W *= 2;
    return W;
}

template <int D>
cudaError_t run_forward(const DeltaArgs& a, int* status)
{
    const TcLayout l = tc_layout(a);
    unsigned char* ws = static_cast<unsigned char*>(a.ws);
    const int n = chunks_of(a.N);
    const int64_t BH = a.B * a.H;
    cudaError_t e = cudaFuncSetAttribute(
        k_delta_prep<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, PrepSmem<D>::bytes);
    if (e != cudaSuccess)
        return e;
    k_delta_prep<D><<<(unsigned)(BH * n), kPrepThreads, PrepSmem<D>::bytes, a.stream>>>(
        static_cast<const __nv_bfloat16*>(a.q), static_cast<const __nv_bfloat16*>(a.k), a.beta,
        a.log_alpha, ws + l.rows, ws + l.blobs, a.N, n, (int)a.H, (int)a.Hk, a.fm == LA_FM_L2,
        a.scale);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    const int W = chain_warps(a);
    const int smem = ChainSmem<D>::bytes(W);
    e = cudaFuncSetAttribute(k_delta_chain<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    k_delta_chain<D><<<(unsigned)(BH * (a.dv / (16 * W))), 32 * W, smem, a.stream>>>(
        ws + l.rows, ws + l.blobs, static_cast<const __nv_bfloat16*>(a.v),
        static_cast<__nv_bfloat16*>(a.out), a.S0, a.S_out, a.N, n, (int)a.H, (int)a.Hk, a.dv, status);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

bool delta_tc_eligible(const DeltaArgs& a) { return a.dtype == LA_BF16 && a.N > 16; }

size_t delta_tc_forward_workspace(const DeltaArgs& a) { return tc_layout(a).total; }

cudaError_t delta_tc_forward(const DeltaArgs& a)
{
    switch (a.d) {
    case 32: return run_forward<32>(a, a.status);
    case 64: return run_forward<64>(a, a.status);
    default: return run_forward<128>(a, a.status);
    }
}

}  // namespace la
