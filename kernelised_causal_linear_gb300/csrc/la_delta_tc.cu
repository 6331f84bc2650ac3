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

// What k_delta_prep writes per chunk and value head: [F hi][F lo][P hi][P lo, for
// gradients][factors], tiles of 64 x 64 fp16 in the layout the chains read them
// from shared memory.  k^_i = fk_i K16_i and scale q^_i = fq_i Q16_i are the mapped
// rows, fk and fq holding the image's power of two, the L2 norm and the scale.
enum Factor {
    kFacA,    // e^{G_i} fk_i
    kFacF,    // scale of F's row (a power of two)
    kFacB,    // beta
    kFacO,    // e^{G_i} fq_i
    kFacP,    // scale of P's row (a power of two)
    kFacW,    // e^{G_C - G_i} fk_i
    kFacEnd,  // [0] = e^{G_C}
    kFactors,
    // gradients only
    kFacK = kFactors,  // fk
    kFacQ,             // fq without the scale
    kFacRk,            // 1 / |k|, or 1 without the norm
    kFacRq,
    kFacGh,  // G in base 2: a multiple of 2^-6 and the rest
    kFacGl,
    kGradFactors
};
constexpr int kTile = kC * kC * 2;  // bytes of a 64 x 64 fp16 tile
template <bool GRAD>
constexpr int n_factors()
{
    return GRAD ? (int)kGradFactors : (int)kFactors;
}
template <bool GRAD>
constexpr int fac_at()  // byte offset of the factors in a blob
{
    return (GRAD ? 4 : 3) * kTile;
}
template <bool GRAD>
constexpr int blob_bytes()
{
    return fac_at<GRAD>() + n_factors<GRAD>() * kC * 4;
}

template <int D>
constexpr int row_image()  // bytes of K16 or Q16 per chunk
{
    return kC * D * 2;
}

// ------------------------------------------------------------- k_delta_prep --
// 4 warps.  The Gram products are exact fp16 MMAs on the lower blocks; F is
// fp32 on the CUDA cores in 16 x 16 blocks: the diagonal ones by substitution
// (a column per lane), then by distance from the diagonal, all threads on each,
//   X = A_IJ + sum_{J <= L < I} A_IL beta_L F_LJ,   F_IJ = -X - F_II beta_I X.
constexpr int kPrepThreads = 128;
constexpr int kLd = 68;  // row stride of the fp32 tiles (16-byte rows, spread over banks)

template <int D, bool GRAD>
struct PrepSmem {
    static constexpr int img = 2 * row_image<D>() > fac_at<GRAD>() ? 2 * row_image<D>() : fac_at<GRAD>();
    static constexpr int A = img;
    static constexpr int F = A + kC * kLd * 4;
    static constexpr int X = F + kC * kLd * 4;
    static constexpr int vec = X + 3 * 16 * 20 * 4;
    static constexpr int bytes = vec + (8 + n_factors<GRAD>()) * kC * 4;
};

template <int D, bool GRAD>
__global__ void __launch_bounds__(kPrepThreads)
    k_delta_prep(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                 const float* __restrict__ beta, const float* __restrict__ log_alpha,
                 unsigned char* __restrict__ rows, unsigned char* __restrict__ blobs, int64_t N,
                 int nchunk, int H, int Hk, int l2, float scale)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    using SM = PrepSmem<D, GRAD>;
    constexpr int RB = 2 * D;  // bytes per row
    float* sA = reinterpret_cast<float*>(smem + SM::A);
    float* sF = reinterpret_cast<float*>(smem + SM::F);
    float* vec = reinterpret_cast<float*>(smem + SM::vec);
    float *fk = vec, *fq = vec + kC, *gh = vec + 2 * kC, *gl = vec + 3 * kC, *sb = vec + 4 * kC;
    float *rk = vec + 5 * kC, *rq = vec + 6 * kC, *uq = vec + 7 * kC;
    float* fac = vec + 8 * kC;  // [factors][kC]

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
            if (p == 0) {
                const float norm = l2 ? rsqrtf(ss + kL2Eps) : 1.0f;
                (which ? rq : rk)[r] = norm;
                (which ? fq : fk)[r] = s.from * norm * (which ? scale : 1.0f);
                if (which)
                    uq[r] = s.from * norm;
            }
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
            aq[nt][e] = j <= i ? aq[nt][e] * fq[i] * fk[j] * dec * (GRAD ? 1.0f : sb[j]) : 0.f;
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
        for (int nt = 0; nt < 8; ++nt) {
            uint32_t hi, lo;
            h2_split(aq[nt][2 * r] * s.to, aq[nt][2 * r + 1] * s.to, hi, lo);
            unsigned char* at = smem + 2 * kTile + tile_off<128>(i, nt) + 4 * tq;
            *reinterpret_cast<uint32_t*>(at) = hi;
            if (GRAD)
                *reinterpret_cast<uint32_t*>(at + kTile) = lo;
        }
    }
    if (tid < kC) {
        const float e = exp2f(gh[tid] + gl[tid]);
        const float w = exp2f((gh[kC - 1] - gh[tid]) + (gl[kC - 1] - gl[tid]));
        fac[kFacA * kC + tid] = e * fk[tid];
        fac[kFacB * kC + tid] = sb[tid];
        fac[kFacO * kC + tid] = e * fq[tid];
        fac[kFacW * kC + tid] = w * fk[tid];
        fac[kFacEnd * kC + tid] = exp2f(gh[kC - 1] + gl[kC - 1]);
        if (GRAD) {
            fac[kFacK * kC + tid] = fk[tid];
            fac[kFacQ * kC + tid] = uq[tid];
            fac[kFacRk * kC + tid] = rk[tid];
            fac[kFacRq * kC + tid] = rq[tid];
            fac[kFacGh * kC + tid] = gh[tid];
            fac[kFacGl * kC + tid] = gl[tid];
        }
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
    // off-diagonal blocks, all threads on the 4 - dist blocks of a distance: thread
    // -> row of a block and 2 (dist 1: 6, dist 2: 4) of its columns
    float* sX = reinterpret_cast<float*>(smem + SM::X);  // [block][16][20]
#pragma unroll
    for (int dist = 1; dist < 4; ++dist) {
        const int r = (tid >> 3) & 15, c0 = (tid & 7) * 2;
        float x[3][2];
#pragma unroll
        for (int J = 0; J < 4 - dist; ++J) {
            const float* arow = sA + (16 * (J + dist) + r) * kLd;
            x[J][0] = arow[16 * J + c0], x[J][1] = arow[16 * J + c0 + 1];
#pragma unroll 8
            for (int l = 16 * J; l < 16 * (J + dist); ++l) {
                const float a = arow[l] * sb[l];
                const float2 f = *reinterpret_cast<const float2*>(sF + l * kLd + 16 * J + c0);
                x[J][0] = fmaf(a, f.x, x[J][0]), x[J][1] = fmaf(a, f.y, x[J][1]);
            }
            *reinterpret_cast<float2*>(sX + (J * 16 + r) * 20 + c0) = make_float2(x[J][0], x[J][1]);
        }
        __syncthreads();
#pragma unroll
        for (int J = 0; J < 4 - dist; ++J) {
            const int I = J + dist;
            const float* frow = sF + (16 * I + r) * kLd + 16 * I;
            float y0 = -x[J][0], y1 = -x[J][1];
#pragma unroll
            for (int l = 0; l < 16; ++l) {  // F_II is zero from its diagonal on
                const float a = -frow[l] * sb[16 * I + l];
                const float2 f = *reinterpret_cast<const float2*>(sX + (J * 16 + l) * 20 + c0);
                y0 = fmaf(a, f.x, y0), y1 = fmaf(a, f.y, y1);
            }
            *reinterpret_cast<float2*>(sF + (16 * I + r) * kLd + 16 * J + c0) = make_float2(y0, y1);
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
    uint4* blob = reinterpret_cast<uint4*>(blobs + (bh * nchunk + c) * (int64_t)blob_bytes<GRAD>());
    for (int i = tid; i < fac_at<GRAD>() / 16; i += kPrepThreads)
        blob[i] = reinterpret_cast<const uint4*>(smem)[i];
    for (int i = tid; i < n_factors<GRAD>() * kC / 4; i += kPrepThreads)
        blob[fac_at<GRAD>() / 16 + i] = reinterpret_cast<const uint4*>(fac)[i];
}

// ------------------------------------------------------------ k_delta_chain --
// W warps of 16 value columns.  The tiles of a chunk are shared by the warps and
// arrive by bulk copies kStages chunks ahead; a warp's own columns of V come by
// cp.async one chunk ahead, and its outputs leave through its own tile, turned
// back to token-major by stmatrix.
constexpr int kStages = 2;
constexpr uint32_t kWaitPolls = 1u << 22;

template <int D, bool GRAD>
struct ChainSmem {
    static constexpr int stage = 2 * row_image<D>() + blob_bytes<GRAD>();
    static constexpr int v = kStages * stage;  // per warp: V twice, O (GRAD: dO)
    static constexpr int per_warp = 3 * kC * 32;
    static int bytes(int W) { return v + W * per_warp + 64; }
};

// What the forward pass of a gradient keeps per chunk, in the fragments' own
// order ([16 columns][16-step][register][lane], every store 128 bytes): the state
// before the chunk and E, as two fp16 parts with a scale per value column.  An
// 8 x 8 block is 128 bytes with its rows in order, so k_delta_dqk reads it with
// ldmatrix whichever way round it needs it.  Per value head and chunk, bytes:
struct Kept {
    unsigned char* S;  // [BH][nchunk + 1][2 parts][D DV] fp16
    float* sS;         // [BH][nchunk + 1][DV]
    unsigned char* E;  // [BH][nchunk][2 parts][64 DV] fp16
    float* sE;         // [BH][nchunk][DV]
    unsigned char* dS; // [BH][nchunk][D DV] fp16: gradient of the state after the chunk
    float* sD;         // [BH][nchunk][DV]
    unsigned char* dV; // [BH][nchunk][64 DV] fp16
    float* sV;         // [BH][nchunk][DV]
    float* oo;         // [BH][DV / 16][N] dO.O over 16 columns
    float* vv;         // [BH][DV / 16][N] v.dV
    float* bb;         // [BH][DV / 16][N] Y.E
    float* cd;         // [BH][DV / 16][nchunk] <S1, dS1>
};

// One fragment's registers of plane `plane` (part_bytes each part, block = 16 x 16)
__device__ __forceinline__ void keep_part(unsigned char* p, int64_t part, int64_t part_bytes, int block,
                                          int lane, const uint32_t (&x)[4])
{
    uint32_t* at = reinterpret_cast<uint32_t*>(p + part * part_bytes) + block * 128 + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        at[32 * i] = x[i];
}
__device__ __forceinline__ void keep_parts(unsigned char* p, int64_t plane, int64_t part_bytes, int block,
                                           int lane, const uint32_t (&hi)[4], const uint32_t (&lo)[4])
{
    keep_part(p, 2 * plane, part_bytes, block, lane, hi);
    keep_part(p, 2 * plane + 1, part_bytes, block, lane, lo);
}

// Two tokens' sums over the warp's 16 columns (the lanes' g) -> row[t], row[t + 1]
__device__ __forceinline__ void store_dot(float* row, int64_t t, int64_t N, int g, float y0, float y1)
{
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        y0 += __shfl_xor_sync(0xffffffffu, y0, o);
        y1 += __shfl_xor_sync(0xffffffffu, y1, o);
    }
    if (g == 0) {
        if (t < N)
            row[t] = y0;
        if (t + 1 < N)
            row[t + 1] = y1;
    }
}

template <int D, bool GRAD>
__global__ void __launch_bounds__(256, 1)
    k_delta_chain(const unsigned char* __restrict__ rows, const unsigned char* __restrict__ blobs,
                  const __nv_bfloat16* __restrict__ v, __nv_bfloat16* __restrict__ out,
                  const float* S0, float* S_out, int64_t N, int nchunk, int H, int Hk, int DV,
                  const __nv_bfloat16* __restrict__ dout, Kept kept, int* status)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    using SM = ChainSmem<D, GRAD>;
    constexpr int kBlob = blob_bytes<GRAD>();
    const bool reads = GRAD || out;  // o is wanted
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
            const int64_t at = (bh * N + (live ? t0 + t : 0)) * DV + col0 + p * 8;
            cp16(sv + (c & 1) * kC * 32 + tile_off<32>(t, p), v + at, live);
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
                                                          2 * row_image<D>() + fac_at<GRAD>());
        if (GRAD) {  // dO, wanted at the end of the chunk
            const int64_t t0 = (int64_t)c * kC;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = (lane >> 1) + 16 * i, p = lane & 1;
                const bool live = t0 + t < N;
                cp16(so + tile_off<32>(t, p),
                     dout + (bh * N + (live ? t0 + t : 0)) * DV + col0 + p * 8, live);
            }
            cp_commit();
        }
        if (c + 1 < nchunk)
            load_v(c + 1);
        cp_commit();
        ok = ok && sm100::mbar_wait(full + c % kStages, (c / kStages) & 1, kWaitPolls);
        cp_wait<GRAD ? 2 : 1>();
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
                if (GRAD)
                    keep_parts(kept.S, bh * (nchunk + 1) + c, D * DV * 2, (col0 / 16) * (D / 16) + kk, lane,
                               hi, lo);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ldsm4(b, addr_b<RB>(sK, lane, 16 * j, 16 * kk));
                    mma(r[2 * j], hi, b[0], b[1]);
                    mma(r[2 * j + 1], hi, b[2], b[3]);
                    mma(r[2 * j], lo, b[0], b[1]);
                    mma(r[2 * j + 1], lo, b[2], b[3]);
                    if (reads) {
                        ldsm4(b, addr_b<RB>(sQ, lane, 16 * j, 16 * kk));
                        mma(o[2 * j], hi, b[0], b[1]);
                        mma(o[2 * j + 1], hi, b[2], b[3]);
                        if (GRAD) {  // o enters an fp32 gradient
                            mma(o[2 * j], lo, b[0], b[1]);
                            mma(o[2 * j + 1], lo, b[2], b[3]);
                        }
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
                    if (reads) {
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
            float e0 = 0.f, e1 = 0.f;
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float2 f = *reinterpret_cast<const float2*>(fac + kFacF * kC + 8 * nt + 2 * tq);
                r[nt][0] = fmaf(f.x * b0.from, x[nt][0], r[nt][0]);
                r[nt][1] = fmaf(f.y * b0.from, x[nt][1], r[nt][1]);
                r[nt][2] = fmaf(f.x * b1.from, x[nt][2], r[nt][2]);
                r[nt][3] = fmaf(f.y * b1.from, x[nt][3], r[nt][3]);
                e0 = max_abs(max_abs(e0, r[nt][0]), r[nt][1]);
                e1 = max_abs(max_abs(e1, r[nt][2]), r[nt][3]);
            }
            if (GRAD) {
                const Pow2 q0 = pow2_for(quad_max(e0)), q1 = pow2_for(quad_max(e1));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int nt = 2 * kk + u;
                        h2_split(r[nt][0] * q0.to, r[nt][1] * q0.to, hi[2 * u], lo[2 * u]);
                        h2_split(r[nt][2] * q1.to, r[nt][3] * q1.to, hi[2 * u + 1], lo[2 * u + 1]);
                    }
                    keep_parts(kept.E, bh * nchunk + c, kC * DV * 2, (col0 / 16) * 4 + kk, lane, hi, lo);
                }
                if (tq == 0) {
                    float* se = kept.sE + (bh * nchunk + c) * DV + col0;
                    float* ss = kept.sS + (bh * (nchunk + 1) + c) * DV + col0;
                    se[g] = q0.from, se[g + 8] = q1.from;
                    ss[g] = p0.from, ss[g + 8] = p1.from;
                }
            }
            // U = beta E, and the largest of the state update's factor times it
            float w0 = 0.f, w1 = 0.f;
            auto to_u = [&]() {
                e0 = e1 = 0.f;
#pragma unroll
                for (int nt = 0; nt < 8; ++nt) {
                    const float2 be = *reinterpret_cast<const float2*>(fac + kFacB * kC + 8 * nt + 2 * tq);
                    const float2 w = *reinterpret_cast<const float2*>(fac + kFacW * kC + 8 * nt + 2 * tq);
                    r[nt][0] *= be.x, r[nt][1] *= be.y, r[nt][2] *= be.x, r[nt][3] *= be.y;
                    e0 = max_abs(max_abs(e0, r[nt][0]), r[nt][1]);
                    e1 = max_abs(max_abs(e1, r[nt][2]), r[nt][3]);
                    w0 = max_abs(max_abs(w0, w.x * r[nt][0]), w.y * r[nt][1]);
                    w1 = max_abs(max_abs(w1, w.x * r[nt][2]), w.y * r[nt][3]);
                }
            };
            if (GRAD)
                to_u();
            // O = inter + (P beta) E: with beta in P, a token that writes nothing does not
            // set the scale of its row.  For the output alone one fp16 part of each is
            // enough (2^-12 of a term, under the output's own rounding); a gradient
            // takes both, and P without beta and U for E, since it needs P itself
            if (reads) {
                const Pow2 q0 = pow2_for(quad_max(e0)), q1 = pow2_for(quad_max(e1));
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
                        h2_split(r[nt][0] * q0.to, r[nt][1] * q0.to, hi[2 * u], lo[2 * u]);
                        h2_split(r[nt][2] * q1.to, r[nt][3] * q1.to, hi[2 * u + 1], lo[2 * u + 1]);
                    }
#pragma unroll
                    for (int j = kk; j < 4; ++j) {
                        ldsm4(b, addr_b<128>(sFh + 2 * kTile, lane, 16 * j, 16 * kk));
                        mma(x[2 * j], hi, b[0], b[1]);
                        mma(x[2 * j + 1], hi, b[2], b[3]);
                        if (GRAD) {
                            mma(x[2 * j], lo, b[0], b[1]);
                            mma(x[2 * j + 1], lo, b[2], b[3]);
                            ldsm4(b, addr_b<128>(sFh + 3 * kTile, lane, 16 * j, 16 * kk));
                            mma(x[2 * j], hi, b[0], b[1]);
                            mma(x[2 * j + 1], hi, b[2], b[3]);
                        }
                    }
                }
                if (GRAD) {
                    cp_wait<1>();  // dO is in
                    __syncwarp();
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t w[4];
                    if (GRAD)
                        ldsm4t(w, addr_ct<32>(so, lane, 16 * j, 0));
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int nt = 2 * j + u;
                        const float2 fp = *reinterpret_cast<const float2*>(fac + kFacP * kC + 8 * nt + 2 * tq);
                        o[nt][0] = fmaf(fp.x * q0.from, x[nt][0], o[nt][0]);
                        o[nt][1] = fmaf(fp.y * q0.from, x[nt][1], o[nt][1]);
                        o[nt][2] = fmaf(fp.x * q1.from, x[nt][2], o[nt][2]);
                        o[nt][3] = fmaf(fp.y * q1.from, x[nt][3], o[nt][3]);
                        if (GRAD) {
                            const float y0 = o[nt][0] * __uint_as_float(w[2 * u] << 16) +
                                             o[nt][2] * __uint_as_float(w[2 * u + 1] << 16);
                            const float y1 = o[nt][1] * __uint_as_float(w[2 * u] & 0xffff0000u) +
                                             o[nt][3] * __uint_as_float(w[2 * u + 1] & 0xffff0000u);
                            store_dot(kept.oo + (bh * (DV / 16) + col0 / 16) * N, (int64_t)c * kC + 8 * nt + 2 * tq,
                                      N, g, y0, y1);
                        } else {
                            w[2 * u] = sm100::pack_bf16x2(o[nt][0], o[nt][1]);
                            w[2 * u + 1] = sm100::pack_bf16x2(o[nt][2], o[nt][3]);
                        }
                    }
                    if (!GRAD)
                        stsm4t(addr_ct<32>(so, lane, 16 * j, 0), w);
                }
            }
            if (!GRAD)
                to_u();
            // S1 = e^{G_C} S0 + (W U)^T K16 on accumulators scaled with the operand:
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
            if (!GRAD && out) {
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
    if (GRAD) {  // the final state, for <S1, dS1> of the last chunk
        float m0 = 0.f, m1 = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m0 = max_abs(max_abs(m0, s[nt][0]), s[nt][1]);
            m1 = max_abs(max_abs(m1, s[nt][2]), s[nt][3]);
        }
        const Pow2 p0 = pow2_for(quad_max(m0)), p1 = pow2_for(quad_max(m1));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t hi[4], lo[4];
            h2_split(s[2 * kk][0] * p0.to, s[2 * kk][1] * p0.to, hi[0], lo[0]);
            h2_split(s[2 * kk][2] * p1.to, s[2 * kk][3] * p1.to, hi[1], lo[1]);
            h2_split(s[2 * kk + 1][0] * p0.to, s[2 * kk + 1][1] * p0.to, hi[2], lo[2]);
            h2_split(s[2 * kk + 1][2] * p1.to, s[2 * kk + 1][3] * p1.to, hi[3], lo[3]);
            keep_parts(kept.S, bh * (nchunk + 1) + nchunk, D * DV * 2, (col0 / 16) * (D / 16) + kk, lane, hi, lo);
        }
        if (tq == 0) {
            float* ss = kept.sS + (bh * (nchunk + 1) + nchunk) * DV + col0;
            ss[g] = p0.from, ss[g + 8] = p1.from;
        }
    }
    if (S_out) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S_out[(bh * D + 8 * nt + 2 * tq + (e & 1)) * DV + col0 + g + (e >> 1) * 8] = s[nt][e];
    }
}

// -------------------------------------------------------------- k_delta_rev --
// The chunks from the last to the first, dS^T [16 x d] of a warp's columns in
// registers (dS1 entering a chunk, dS0 leaving it):
//
//   dU = P^T dO + diag(e^{G_C - G}) K dS1,  z = beta dU
//   Y  = dU + F^T z,  dV = beta Y          ((I + diag(beta) A)^{-T} = I + F^T beta)
//   dS0 = e^{G_C} dS1 + (diag(e^G) Q)^T dO - (diag(e^G) K)^T dV
//
// and the dot products that need both directions' fp32 values: v.dV, Y.E, and
// <S0, dS0> (which is <S1, dS1> of the chunk before).
constexpr int kRevWarps = 4;

template <int D>
struct RevSmem {
    static constexpr int stage = 2 * row_image<D>() + blob_bytes<true>();
    static constexpr int warp0 = kStages * stage;
    // per warp: dO twice, V (then dV), E hi and lo, S hi and lo
    static constexpr int dO = 0, v = 2 * kC * 32, e = v + kC * 32, s = e + 2 * kC * 32,
                         per_warp = s + 2 * D * 32;
    static int bytes(int W) { return warp0 + W * per_warp + 64; }
};

template <int D>
__global__ void __launch_bounds__(32 * kRevWarps, 1)
    k_delta_rev(const unsigned char* __restrict__ rows, const unsigned char* __restrict__ blobs,
                const __nv_bfloat16* __restrict__ v, const __nv_bfloat16* __restrict__ dout,
                const float* __restrict__ dS_out, __nv_bfloat16* __restrict__ dv,
                float* __restrict__ dS0, int64_t N, int nchunk, int H, int Hk, int DV, int gated,
                Kept kept, int* status)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    using SM = RevSmem<D>;
    constexpr int RB = 2 * D, NT = D / 8, kBlob = blob_bytes<true>();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, W = blockDim.x >> 5;
    const int g = lane >> 2, tq = lane & 3;
    const int slices = DV / (16 * W);
    const int64_t bh = blockIdx.x / slices;
    const int col0 = (blockIdx.x % slices) * 16 * W + 16 * warp, slice = col0 / 16;
    const int64_t kh = bh / H * Hk + (bh % H) / (H / Hk);
    const uint32_t base = smem_addr(smem);
    const uint32_t mine = SM::warp0 + warp * SM::per_warp;
    const uint32_t sdo = base + mine + SM::dO, sv = base + mine + SM::v;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::warp0 + W * SM::per_warp);
    const unsigned char* row_src = rows + kh * nchunk * (int64_t)(2 * row_image<D>());
    const unsigned char* blob_src = blobs + bh * nchunk * (int64_t)kBlob;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i)
            sm100::mbar_init(full + i, 1);
        sm100::fence_mbar_init();
    }
    __syncthreads();
    auto load_stage = [&](int it) {
        const int64_t c = nchunk - 1 - it;
        const uint32_t dst = base + (it % kStages) * SM::stage;
        uint64_t* bar = full + it % kStages;
        sm100::mbar_arrive_expect_tx(bar, SM::stage);
        delta::bulk_load(dst, row_src + c * (2 * row_image<D>()), 2 * row_image<D>(), bar);
        delta::bulk_load(dst + 2 * row_image<D>(), blob_src + c * kBlob, kBlob, bar);
    };
    auto load_cols = [&](uint32_t dst, const __nv_bfloat16* src, int c) {
        const int64_t t0 = (int64_t)c * kC;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = (lane >> 1) + 16 * i, p = lane & 1;
            const bool live = t0 + t < N;
            cp16(dst + tile_off<32>(t, p), src + (bh * N + (live ? t0 + t : 0)) * DV + col0 + p * 8, live);
        }
    };
    // a warp's part of a kept plane, `n` blocks of 512 bytes
    auto load_blocks = [&](uint32_t dst, const unsigned char* plane, int64_t part, int64_t part_bytes, int n) {
        const unsigned char* src = plane + part * part_bytes + (int64_t)slice * n * 512;
        for (int i = 0; i < n; ++i)
            cp16(dst + i * 512 + lane * 16, src + i * 512 + lane * 16, true);
    };
    auto load_S = [&](int64_t c) {
        load_blocks(base + mine + SM::s, kept.S, 2 * (bh * (nchunk + 1) + c), D * DV * 2, D / 16);
        load_blocks(base + mine + SM::s + D * 32, kept.S, 2 * (bh * (nchunk + 1) + c) + 1, D * DV * 2, D / 16);
    };
    float ds[NT][4];  // dS^T[col0 + g, + 8][8 nt + 2 tq, + 1]
    // <S of chunk c, dS> over the warp's columns -> kept.cd of the chunk before
    auto dot_state = [&](int64_t c) {
        const uint32_t* hi = reinterpret_cast<const uint32_t*>(smem + mine + SM::s) + lane;
        const uint32_t* lo = hi + D * 8;
        const float* sc = kept.sS + (bh * (nchunk + 1) + c) * DV + col0;
        float a0 = 0.f, a1 = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // register i: row g + 8 (i & 1), tile 2 kk + (i >> 1)
                const uint32_t x = hi[(kk * 4 + i) * 32], y = lo[(kk * 4 + i) * 32];
                const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&x));
                const float2 l = __half22float2(*reinterpret_cast<const __half2*>(&y));
                const float* d = ds[2 * kk + (i >> 1)] + 2 * (i & 1);
                float& a = i & 1 ? a1 : a0;
                a = fmaf(h.x + l.x, d[0], fmaf(h.y + l.y, d[1], a));
            }
        }
        float x = a0 * sc[g] + a1 * sc[g + 8];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0)
            kept.cd[(bh * (DV / 16) + slice) * nchunk + c - 1] = x;
    };

    if (tid == 0)
        for (int i = 0; i < kStages && i < nchunk; ++i)
            load_stage(i);
    load_cols(sdo + ((nchunk - 1) & 1) * kC * 32, dout, nchunk - 1);
    if (gated)
        load_S(nchunk);
    cp_commit();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            ds[nt][e] =
                dS_out ? dS_out[(bh * D + 8 * nt + 2 * tq + (e & 1)) * DV + col0 + g + (e >> 1) * 8] : 0.f;
    cp_wait<0>();
    __syncwarp();
    if (gated)
        dot_state(nchunk);
    __syncwarp();

    bool ok = true;
    int it = 0;
    for (; it < nchunk; ++it) {
        const int c = nchunk - 1 - it;
        const uint32_t st = base + (it % kStages) * SM::stage;
        const uint32_t sK = st, sQ = st + row_image<D>(), sF = st + 2 * row_image<D>(), sP = sF + 2 * kTile;
        const float* fac = reinterpret_cast<const float*>(smem + (it % kStages) * SM::stage +
                                                          2 * row_image<D>() + fac_at<true>());
        const uint32_t tdo = sdo + (c & 1) * kC * 32;
        // this chunk's V, E and S, wanted from the middle on, and the next dO
        load_cols(sv, v, c);
        load_blocks(base + mine + SM::e, kept.E, 2 * (bh * nchunk + c), kC * DV * 2, 4);
        load_blocks(base + mine + SM::e + kC * 32, kept.E, 2 * (bh * nchunk + c) + 1, kC * DV * 2, 4);
        if (gated && c > 0)
            load_S(c);
        if (c > 0)
            load_cols(sdo + ((c - 1) & 1) * kC * 32, dout, c - 1);
        cp_commit();
        const float* se = kept.sE + (bh * nchunk + c) * DV + col0;
        const float se0 = se[g], se1 = se[g + 8];
        ok = ok && sm100::mbar_wait(full + it % kStages, (it / kStages) & 1, kWaitPolls);
        if (ok) {
            // dS1^T K^T; dS1 is kept for k_delta_dqk
            float m0 = 0.f, m1 = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                m0 = max_abs(max_abs(m0, ds[nt][0]), ds[nt][1]);
                m1 = max_abs(max_abs(m1, ds[nt][2]), ds[nt][3]);
            }
            m0 = quad_max(m0), m1 = quad_max(m1);
            const Pow2 p0 = pow2_for(m0), p1 = pow2_for(m1);
            float u[8][4], x[8][4];
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    u[nt][e] = x[nt][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t hi[4], lo[4], b[4];
                h2_split(ds[2 * kk][0] * p0.to, ds[2 * kk][1] * p0.to, hi[0], lo[0]);
                h2_split(ds[2 * kk][2] * p1.to, ds[2 * kk][3] * p1.to, hi[1], lo[1]);
                h2_split(ds[2 * kk + 1][0] * p0.to, ds[2 * kk + 1][1] * p0.to, hi[2], lo[2]);
                h2_split(ds[2 * kk + 1][2] * p1.to, ds[2 * kk + 1][3] * p1.to, hi[3], lo[3]);
                keep_part(kept.dS, bh * nchunk + c, D * DV * 2, slice * (D / 16) + kk, lane, hi);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ldsm4(b, addr_b<RB>(sK, lane, 16 * j, 16 * kk));
                    mma(u[2 * j], hi, b[0], b[1]);
                    mma(u[2 * j + 1], hi, b[2], b[3]);
                    mma(u[2 * j], lo, b[0], b[1]);
                    mma(u[2 * j + 1], lo, b[2], b[3]);
                }
            }
            // dO^T P: the rows of P carry powers of two, which go to dO (exact)
            float d0 = 0.f, d1 = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
                ldsm4t(w, addr_ct<32>(tdo, lane, 16 * j, 0));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 fp = *reinterpret_cast<const float2*>(fac + kFacP * kC + 16 * j + 8 * h + 2 * tq);
                    d0 = max_abs(max_abs(d0, fp.x * __uint_as_float(w[2 * h] << 16)),
                                 fp.y * __uint_as_float(w[2 * h] & 0xffff0000u));
                    d1 = max_abs(max_abs(d1, fp.x * __uint_as_float(w[2 * h + 1] << 16)),
                                 fp.y * __uint_as_float(w[2 * h + 1] & 0xffff0000u));
                }
            }
            const Pow2 q0 = pow2_for(quad_max(d0)), q1 = pow2_for(quad_max(d1));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t w[4], a[4], b[4];
                ldsm4t(w, addr_ct<32>(tdo, lane, 16 * kk, 0));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 fp = *reinterpret_cast<const float2*>(fac + kFacP * kC + 16 * kk + 8 * h + 2 * tq);
                    a[2 * h] = h2(fp.x * __uint_as_float(w[2 * h] << 16) * q0.to,
                                  fp.y * __uint_as_float(w[2 * h] & 0xffff0000u) * q0.to);
                    a[2 * h + 1] = h2(fp.x * __uint_as_float(w[2 * h + 1] << 16) * q1.to,
                                      fp.y * __uint_as_float(w[2 * h + 1] & 0xffff0000u) * q1.to);
                }
#pragma unroll
                for (int j = 0; j <= kk; ++j) {  // P_ij, j <= i
                    ldsm4t(b, addr_bt<128>(sP, lane, 16 * kk, 16 * j));
                    mma(x[2 * j], a, b[0], b[1]);
                    mma(x[2 * j + 1], a, b[2], b[3]);
                    ldsm4t(b, addr_bt<128>(sP + kTile, lane, 16 * kk, 16 * j));
                    mma(x[2 * j], a, b[0], b[1]);
                    mma(x[2 * j + 1], a, b[2], b[3]);
                }
            }
            // dU, and the largest |z| with F's row scales
            float z0 = 0.f, z1 = 0.f;
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float2 w = *reinterpret_cast<const float2*>(fac + kFacW * kC + 8 * nt + 2 * tq);
                const float2 be = *reinterpret_cast<const float2*>(fac + kFacB * kC + 8 * nt + 2 * tq);
                const float2 ff = *reinterpret_cast<const float2*>(fac + kFacF * kC + 8 * nt + 2 * tq);
                u[nt][0] = fmaf(w.x * p0.from, u[nt][0], q0.from * x[nt][0]);
                u[nt][1] = fmaf(w.y * p0.from, u[nt][1], q0.from * x[nt][1]);
                u[nt][2] = fmaf(w.x * p1.from, u[nt][2], q1.from * x[nt][2]);
                u[nt][3] = fmaf(w.y * p1.from, u[nt][3], q1.from * x[nt][3]);
                z0 = max_abs(max_abs(z0, be.x * ff.x * u[nt][0]), be.y * ff.y * u[nt][1]);
                z1 = max_abs(max_abs(z1, be.x * ff.x * u[nt][2]), be.y * ff.y * u[nt][3]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[nt][e] = 0.f;
            }
            const Pow2 y0 = pow2_for(quad_max(z0)), y1 = pow2_for(quad_max(z1));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t hi[4], lo[4], b[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int nt = 2 * kk + h;
                    const float2 be = *reinterpret_cast<const float2*>(fac + kFacB * kC + 8 * nt + 2 * tq);
                    const float2 ff = *reinterpret_cast<const float2*>(fac + kFacF * kC + 8 * nt + 2 * tq);
                    const float fx = be.x * ff.x, fy = be.y * ff.y;
                    h2_split(fx * u[nt][0] * y0.to, fy * u[nt][1] * y0.to, hi[2 * h], lo[2 * h]);
                    h2_split(fx * u[nt][2] * y1.to, fy * u[nt][3] * y1.to, hi[2 * h + 1], lo[2 * h + 1]);
                }
#pragma unroll
                for (int j = 0; j <= kk; ++j) {
                    ldsm4t(b, addr_bt<128>(sF, lane, 16 * kk, 16 * j));
                    mma(x[2 * j], hi, b[0], b[1]);
                    mma(x[2 * j + 1], hi, b[2], b[3]);
                    mma(x[2 * j], lo, b[0], b[1]);
                    mma(x[2 * j + 1], lo, b[2], b[3]);
                    ldsm4t(b, addr_bt<128>(sF + kTile, lane, 16 * kk, 16 * j));
                    mma(x[2 * j], hi, b[0], b[1]);
                    mma(x[2 * j + 1], hi, b[2], b[3]);
                }
            }
            cp_wait<0>();
            __syncwarp();
            // Y, the dots, dV
            float v0 = 0.f, v1 = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
                ldsm4t(w, addr_ct<32>(sv, lane, 16 * j, 0));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int nt = 2 * j + h;
                    const float2 be = *reinterpret_cast<const float2*>(fac + kFacB * kC + 8 * nt + 2 * tq);
                    u[nt][0] = fmaf(y0.from, x[nt][0], u[nt][0]);
                    u[nt][1] = fmaf(y0.from, x[nt][1], u[nt][1]);
                    u[nt][2] = fmaf(y1.from, x[nt][2], u[nt][2]);
                    u[nt][3] = fmaf(y1.from, x[nt][3], u[nt][3]);
                    const uint32_t* eh = reinterpret_cast<const uint32_t*>(smem + mine + SM::e) +
                                         (j * 4 + 2 * h) * 32 + lane;
                    const uint32_t* el = eh + kC * 8;
                    const float2 a0 = __half22float2(*reinterpret_cast<const __half2*>(eh));
                    const float2 a1 = __half22float2(*reinterpret_cast<const __half2*>(eh + 32));
                    const float2 l0 = __half22float2(*reinterpret_cast<const __half2*>(el));
                    const float2 l1 = __half22float2(*reinterpret_cast<const __half2*>(el + 32));
                    const int64_t t = (int64_t)c * kC + 8 * nt + 2 * tq;
                    store_dot(kept.bb + (bh * (DV / 16) + slice) * N, t, N, g,
                              u[nt][0] * (se0 * (a0.x + l0.x)) + u[nt][2] * (se1 * (a1.x + l1.x)),
                              u[nt][1] * (se0 * (a0.y + l0.y)) + u[nt][3] * (se1 * (a1.y + l1.y)));
                    u[nt][0] *= be.x, u[nt][1] *= be.y, u[nt][2] *= be.x, u[nt][3] *= be.y;
                    if (gated)
                        store_dot(kept.vv + (bh * (DV / 16) + slice) * N, t, N, g,
                                  u[nt][0] * __uint_as_float(w[2 * h] << 16) +
                                      u[nt][2] * __uint_as_float(w[2 * h + 1] << 16),
                                  u[nt][1] * __uint_as_float(w[2 * h] & 0xffff0000u) +
                                      u[nt][3] * __uint_as_float(w[2 * h + 1] & 0xffff0000u));
                    v0 = max_abs(max_abs(v0, u[nt][0]), u[nt][1]);
                    v1 = max_abs(max_abs(v1, u[nt][2]), u[nt][3]);
                }
            }
            __syncwarp();  // V is read; dV takes its place
            v0 = quad_max(v0), v1 = quad_max(v1);
            {
                const Pow2 s0 = pow2_for(v0), s1 = pow2_for(v1);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t w[4], a[4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int nt = 2 * j + h;
                        w[2 * h] = sm100::pack_bf16x2(u[nt][0], u[nt][1]);
                        w[2 * h + 1] = sm100::pack_bf16x2(u[nt][2], u[nt][3]);
                        a[2 * h] = h2(u[nt][0] * s0.to, u[nt][1] * s0.to);
                        a[2 * h + 1] = h2(u[nt][2] * s1.to, u[nt][3] * s1.to);
                    }
                    stsm4t(addr_ct<32>(sv, lane, 16 * j, 0), w);
                    keep_part(kept.dV, bh * nchunk + c, kC * DV * 2, slice * 4 + j, lane, a);
                }
                if (tq == 0) {
                    float* sd = kept.sD + (bh * nchunk + c) * DV + col0;
                    float* sw = kept.sV + (bh * nchunk + c) * DV + col0;
                    sd[g] = p0.from, sd[g + 8] = p1.from;
                    sw[g] = s0.from, sw[g + 8] = s1.from;
                }
            }
            __syncwarp();
            {
                const int64_t t0 = (int64_t)c * kC;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = (lane >> 1) + 16 * i, p = lane & 1;
                    if (t0 + t < N)
                        *reinterpret_cast<uint4*>(dv + (bh * N + t0 + t) * DV + col0 + p * 8) =
                            *reinterpret_cast<const uint4*>(smem + mine + SM::v + tile_off<32>(t, p));
                }
            }
            // dS0: both products on accumulators under one power of two
            float w0 = 0.f, w1 = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
                ldsm4t(w, addr_ct<32>(tdo, lane, 16 * j, 0));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int nt = 2 * j + h;
                    const float2 fo = *reinterpret_cast<const float2*>(fac + kFacO * kC + 8 * nt + 2 * tq);
                    const float2 fa = *reinterpret_cast<const float2*>(fac + kFacA * kC + 8 * nt + 2 * tq);
                    w0 = max_abs(max_abs(w0, fo.x * __uint_as_float(w[2 * h] << 16)),
                                 fo.y * __uint_as_float(w[2 * h] & 0xffff0000u));
                    w1 = max_abs(max_abs(w1, fo.x * __uint_as_float(w[2 * h + 1] << 16)),
                                 fo.y * __uint_as_float(w[2 * h + 1] & 0xffff0000u));
                    u[nt][0] *= -fa.x, u[nt][1] *= -fa.y, u[nt][2] *= -fa.x, u[nt][3] *= -fa.y;
                    w0 = max_abs(max_abs(w0, u[nt][0]), u[nt][1]);
                    w1 = max_abs(max_abs(w1, u[nt][2]), u[nt][3]);
                }
            }
            const float gend = fac[kFacEnd * kC];
            const Pow2 r0 = pow2_for(fmaxf(quad_max(w0), m0 * gend * 0.00390625f));
            const Pow2 r1 = pow2_for(fmaxf(quad_max(w1), m1 * gend * 0.00390625f));
            const float g0 = gend * r0.to, g1 = gend * r1.to;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                ds[nt][0] *= g0, ds[nt][1] *= g0;
                ds[nt][2] *= g1, ds[nt][3] *= g1;
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t w[4], hi[4], lo[4], b[4];
                ldsm4t(w, addr_ct<32>(tdo, lane, 16 * kk, 0));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 fo = *reinterpret_cast<const float2*>(fac + kFacO * kC + 16 * kk + 8 * h + 2 * tq);
                    h2_split(fo.x * __uint_as_float(w[2 * h] << 16) * r0.to,
                             fo.y * __uint_as_float(w[2 * h] & 0xffff0000u) * r0.to, hi[2 * h], lo[2 * h]);
                    h2_split(fo.x * __uint_as_float(w[2 * h + 1] << 16) * r1.to,
                             fo.y * __uint_as_float(w[2 * h + 1] & 0xffff0000u) * r1.to, hi[2 * h + 1],
                             lo[2 * h + 1]);
                }
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) {
                    ldsm4t(b, addr_bt<RB>(sQ, lane, 16 * kk, 16 * j));
                    mma(ds[2 * j], hi, b[0], b[1]);
                    mma(ds[2 * j + 1], hi, b[2], b[3]);
                    mma(ds[2 * j], lo, b[0], b[1]);
                    mma(ds[2 * j + 1], lo, b[2], b[3]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int nt = 2 * kk + h;
                    h2_split(u[nt][0] * r0.to, u[nt][1] * r0.to, hi[2 * h], lo[2 * h]);
                    h2_split(u[nt][2] * r1.to, u[nt][3] * r1.to, hi[2 * h + 1], lo[2 * h + 1]);
                }
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) {
                    ldsm4t(b, addr_bt<RB>(sK, lane, 16 * kk, 16 * j));
                    mma(ds[2 * j], hi, b[0], b[1]);
                    mma(ds[2 * j + 1], hi, b[2], b[3]);
                    mma(ds[2 * j], lo, b[0], b[1]);
                    mma(ds[2 * j + 1], lo, b[2], b[3]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                ds[nt][0] *= r0.from, ds[nt][1] *= r0.from;
                ds[nt][2] *= r1.from, ds[nt][3] *= r1.from;
            }
            if (gated && c > 0)
                dot_state(c);
        }
        ok = __syncthreads_and(ok);
        if (!ok)
            break;
        if (tid == 0 && it + kStages < nchunk)
            load_stage(it + kStages);
    }
    cp_wait<0>();
    if (!ok) {  // a copy never arrived: see the others home, report, leave
        if (tid == 0) {
            for (int i = it; i < it + kStages && i < nchunk; ++i)
                sm100::mbar_wait(full + i % kStages, (i / kStages) & 1, kWaitPolls);
            set_status(status, LA_ERR_TIMEOUT);
        }
        return;
    }
    if (dS0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                dS0[(bh * D + 8 * nt + 2 * tq + (e & 1)) * DV + col0 + g + (e >> 1) * 8] = ds[nt][e];
    }
}

// -------------------------------------------------------------- k_delta_dqk --
// dQ and dK of one chunk and key head, the value heads that read it in turn;
// every chunk on its own.  With U = beta E:
//
//   dQ_i = sum_{j<=i} D_ij (dO_i.U_j) k_j + e^{G_i} S0 dO_i
//   dK_j = sum_{i>=j} D_ij (dO_i.U_j) q_i - sum_{i>j} D_ij (dV_i.U_j) k_i
//          - sum_{i<j} D_ji (dV_j.U_i) k_i - e^{G_j} S0 dV_j + e^{G_C-G_j} dS1 U_j
//
// then through scale and norm to the inputs.  Warps 0-3 own 16 tokens of dQ
// each, warps 4-7 of dK.  The kept planes arrive with a scale per value column,
// the contracted index here; they are brought under one scale each in shared
// memory (a power of two: exact but for columns under 2^-24 of the largest), so
// that fragments go from ldmatrix into the MMA as they are and every factor is
// one of a row, applied to fp32 accumulators.  The 64 x 64 matrices pass through a
// tile of the warp's own as fp16 rows under a power of two each.  One fp16 part
// throughout (2^-12 of a term, under the results' own rounding to bf16).
// Loops over fragments stay rolled: unrolled, the two roles' code overran the
// instruction cache and its misses were half of all stalls.
constexpr int kDqkThreads = 256;
constexpr int kLdD = 66;  // row stride of the decay matrix

template <int D, int DV>
struct DqkSmem {
    static constexpr int K = 0, Q = row_image<D>(), E = 2 * row_image<D>(), dV = E + kC * DV * 2,
                         dO = dV + kC * DV * 2, S = dO + kC * DV * 2, dS = S + D * DV * 2,
                         tile = dS + D * DV * 2, dm = tile + 8 * 16 * 128, vec = dm + kC * kLdD * 4,
                         cols = vec + 16 * kC * 4, bytes = cols + 4 * DV * 4 + 64;
};

// Kept blocks (16 value columns x 16) times their columns' factors c[col] / m
__device__ __forceinline__ void one_scale(unsigned char* plane, int blocks, int per_slice, const float* c, float inv_m)
{
    for (int u = threadIdx.x; u < blocks * 32; u += kDqkThreads) {
        const int block = u >> 5, col = block / per_slice * 16 + ((u >> 3) & 1) * 8 + (u & 7);
        const __half2 f = __float2half2_rn(c[col] * inv_m);
        uint4* at = reinterpret_cast<uint4*>(plane) + u;
        uint4 x = *at;
        __half2* h = reinterpret_cast<__half2*>(&x);
        h[0] = __hmul2(h[0], f), h[1] = __hmul2(h[1], f), h[2] = __hmul2(h[2], f), h[3] = __hmul2(h[3], f);
        *at = x;
    }
}

// largest of c[0 .. n), by every lane of a warp
__device__ __forceinline__ float warp_max(const float* c, int n)
{
    float m = 0.f;
    for (int i = threadIdx.x & 31; i < n; i += 32)
        m = fmaxf(m, c[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

template <int D, int DV>
__global__ void __launch_bounds__(kDqkThreads, 1)
    k_delta_dqk(const unsigned char* __restrict__ rows, const unsigned char* __restrict__ blobs,
                const __nv_bfloat16* __restrict__ dout, Kept kept, __nv_bfloat16* __restrict__ dq,
                __nv_bfloat16* __restrict__ dk, float* __restrict__ dbeta, float* __restrict__ dlog_alpha,
                int64_t N, int nchunk, int H, int Hk, int l2, float scale, int* status)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    using SM = DqkSmem<D, DV>;
    constexpr int RB = 2 * D, VB = 2 * DV, NT = D / 8, KS = DV / 16;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    const uint32_t base = smem_addr(smem);
    float* dm = reinterpret_cast<float*>(smem + SM::dm);    // [i][j], j <= i
    float* vec = reinterpret_cast<float*>(smem + SM::vec);  // [kGradFactors][kC], then
    float* sdo = vec + kGradFactors * kC;                   // dO's row scales
    float* eg = sdo + kC;                                   // e^G
    float* ege = eg + kC;                                   // e^{G_C - G}
    float* cE = reinterpret_cast<float*>(smem + SM::cols);
    float *cS = cE + DV, *cV = cS + DV, *cD = cV + DV;
    uint64_t* full = reinterpret_cast<uint64_t*>(cD + DV);
    const int64_t kh = blockIdx.x / nchunk;
    const int c = blockIdx.x % nchunk;
    const int per = H / Hk;
    const int64_t t0 = (int64_t)c * kC;
    const int n = (int)min((int64_t)kC, N - t0);
    const bool role_k = warp >= 4;
    const int rt = warp & 3, r0 = 16 * rt;
    const uint32_t mytile = base + SM::tile + warp * 16 * 128;

    if (tid == 0) {
        sm100::mbar_init(full, 1);
        sm100::fence_mbar_init();
    }
    float tot[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            tot[nt][e] = 0.f;

    bool ok = true;
    for (int p = 0; p < per; ++p) {
        const int64_t bh = kh / Hk * H + (kh % Hk) * per + p;
        const int64_t at = bh * nchunk + c;
        __syncthreads();  // the head before is done with the tiles
        if (tid == 0) {
            sm100::fence_proxy_async_smem();  // their rescaling was written by threads
            const uint32_t bytes = 2 * kC * DV * 2 + 2 * D * DV * 2 + (p == 0 ? 2 * row_image<D>() : 0);
            sm100::mbar_arrive_expect_tx(full, bytes);
            if (p == 0)
                delta::bulk_load(base + SM::K, rows + (kh * nchunk + c) * (int64_t)(2 * row_image<D>()),
                                 2 * row_image<D>(), full);
            delta::bulk_load(base + SM::E, kept.E + 2 * at * (kC * DV * 2), kC * DV * 2, full);
            delta::bulk_load(base + SM::dV, kept.dV + at * (kC * DV * 2), kC * DV * 2, full);
            delta::bulk_load(base + SM::S, kept.S + 2 * (bh * (nchunk + 1) + c) * (int64_t)(D * DV * 2),
                             D * DV * 2, full);
            delta::bulk_load(base + SM::dS, kept.dS + at * (D * DV * 2), D * DV * 2, full);
        }
        // dO as scaled fp16 rows, factors, column scales
        constexpr int LPR = DV / 8, RPP = kDqkThreads / LPR;
#pragma unroll
        for (int b = 0; b < kC; b += RPP) {
            const int r = b + tid / LPR, part = tid % LPR;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (r < n)
                w = *reinterpret_cast<const uint4*>(dout + (bh * N + t0 + r) * DV + part * 8);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            float f[8], mx = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(u[i] << 16);
                f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
                mx = max_abs(max_abs(mx, f[2 * i]), f[2 * i + 1]);
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const Pow2 s = pow2_for(mx);
            uint4 h;
            h.x = h2(f[0] * s.to, f[1] * s.to), h.y = h2(f[2] * s.to, f[3] * s.to);
            h.z = h2(f[4] * s.to, f[5] * s.to), h.w = h2(f[6] * s.to, f[7] * s.to);
            *reinterpret_cast<uint4*>(smem + SM::dO + tile_off<VB>(r, part)) = h;
            if (part == 0)
                sdo[r] = s.from;
        }
        const float* fac = reinterpret_cast<const float*>(blobs + at * (int64_t)blob_bytes<true>() + fac_at<true>());
        for (int i = tid; i < kGradFactors * kC; i += kDqkThreads)
            vec[i] = fac[i];
        for (int i = tid; i < DV; i += kDqkThreads) {
            cE[i] = kept.sE[at * DV + i];
            cV[i] = kept.sV[at * DV + i];
            cD[i] = kept.sD[at * DV + i];
            cS[i] = kept.sS[(bh * (nchunk + 1) + c) * DV + i];
        }
        __syncthreads();
        const float *fB = vec + kFacB * kC, *fK = vec + kFacK * kC, *fQ = vec + kFacQ * kC,
                    *gh = vec + kFacGh * kC, *gl = vec + kFacGl * kC;
        for (int i = tid; i < kC * kC; i += kDqkThreads) {
            const int y = i / kC, x = i % kC;
            if (x <= y)
                dm[y * kLdD + x] = exp2f((gh[y] - gh[x]) + (gl[y] - gl[x]));
        }
        if (tid < kC) {
            eg[tid] = exp2f(gh[tid] + gl[tid]);
            ege[tid] = exp2f((gh[kC - 1] - gh[tid]) + (gl[kC - 1] - gl[tid]));
        }
        const float mE = warp_max(cE, DV), mV = warp_max(cV, DV), mS = warp_max(cS, DV), mD = warp_max(cD, DV);
        ok = ok && sm100::mbar_wait(full, p & 1, kWaitPolls);
        if (ok) {  // 1 / m of a power of two is exact
            one_scale(smem + SM::E, KS * 4, 4, cE, 1.0f / mE);
            one_scale(smem + SM::dV, KS * 4, 4, cV, 1.0f / mV);
            one_scale(smem + SM::S, KS * (D / 16), D / 16, cS, 1.0f / mS);
            one_scale(smem + SM::dS, KS * (D / 16), D / 16, cD, 1.0f / mD);
        }
        ok = __syncthreads_and(ok);
        if (!ok)
            break;

        const int ia = r0 + g, ib = ia + 8;
        // A fragments of this warp's rows, 16 value columns ks: dO is row-major, kept
        // planes lie turned
        auto a_rows = [&](uint32_t (&x)[4], int plane, int ks) {
            if (plane == SM::dO) {
                ldsm4(x, addr_a<VB>(base + SM::dO, lane, r0, 16 * ks));
            } else {
                uint32_t y[4];
                ldsm4t(y, base + plane + (ks * 4 + rt) * 512 + lane * 16);
                x[0] = y[0], x[1] = y[2], x[2] = y[1], x[3] = y[3];
            }
        };
        // x[row][token] = this warp's rows of plane `a` dot the tokens of plane `b`,
        // token tiles lo .. hi
        auto dots = [&](float (&x)[8][4], int a_plane, int b_plane, int lo, int hi) {
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[nt][e] = 0.f;
#pragma unroll 2
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t a[4], b[4];
                a_rows(a, a_plane, ks);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j >= lo && j <= hi) {
                        if (b_plane == SM::dO)
                            ldsm4(b, addr_b<VB>(base + SM::dO, lane, 16 * j, 16 * ks));
                        else
                            ldsm4t(b, base + b_plane + (ks * 4 + j) * 512 + lane * 16);
                        mma(x[2 * j], a, b[0], b[1]);
                        mma(x[2 * j + 1], a, b[2], b[3]);
                    }
                }
            }
        };
        auto add = [&](const float (&acc)[NT][4], float fa, float fb) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                tot[nt][0] = fmaf(fa, acc[nt][0], tot[nt][0]), tot[nt][1] = fmaf(fa, acc[nt][1], tot[nt][1]);
                tot[nt][2] = fmaf(fb, acc[nt][2], tot[nt][2]), tot[nt][3] = fmaf(fb, acc[nt][3], tot[nt][3]);
            }
        };
        // tot += (fa, fb) o this warp's rows of plane `a` times a kept state plane
        auto state = [&](int a_plane, int b_plane, float fa, float fb) {
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[nt][e] = 0.f;
#pragma unroll 1
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t a[4], b[4];
                a_rows(a, a_plane, ks);
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) {
                    ldsm4t(b, base + b_plane + (ks * (D / 16) + j) * 512 + lane * 16);
                    mma(acc[2 * j], a, b[0], b[1]);
                    mma(acc[2 * j + 1], a, b[2], b[3]);
                }
            }
            add(acc, fa, fb);
        };
        // tot += x (64 tokens, zero outside tiles lo .. hi) times a row image
        auto rows_product = [&](const float (&x)[8][4], int image, int lo, int hi) {
            float ma = 0.f, mb = 0.f;
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                ma = max_abs(max_abs(ma, x[nt][0]), x[nt][1]);
                mb = max_abs(max_abs(mb, x[nt][2]), x[nt][3]);
            }
            const Pow2 pa = pow2_for(quad_max(ma)), pb = pow2_for(quad_max(mb));
            __syncwarp();
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                *reinterpret_cast<uint32_t*>(smem + (mytile - base) + tile_off<128>(g, nt) + 4 * tq) =
                    h2(x[nt][0] * pa.to, x[nt][1] * pa.to);
                *reinterpret_cast<uint32_t*>(smem + (mytile - base) + tile_off<128>(g + 8, nt) + 4 * tq) =
                    h2(x[nt][2] * pb.to, x[nt][3] * pb.to);
            }
            __syncwarp();
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[nt][e] = 0.f;
#pragma unroll 1
            for (int kk = lo; kk <= hi; ++kk) {
                uint32_t a[4], b[4];
                ldsm4(a, addr_a<128>(mytile, lane, 0, 16 * kk));
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) {
                    ldsm4t(b, addr_bt<RB>(base + image, lane, 16 * kk, 16 * j));
                    mma(acc[2 * j], a, b[0], b[1]);
                    mma(acc[2 * j + 1], a, b[2], b[3]);
                }
            }
            add(acc, pa.from, pb.from);
        };
        float x[8][4];
        if (!role_k) {
            dots(x, SM::dO, SM::E, 0, rt);
            const float fa = mE * sdo[ia], fb = mE * sdo[ib];
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = e >> 1 ? ib : ia, j = 8 * nt + 2 * tq + (e & 1);
                    x[nt][e] = j <= i ? x[nt][e] * (e >> 1 ? fb : fa) * dm[i * kLdD + j] * (fB[j] * fK[j]) : 0.f;
                }
            rows_product(x, SM::K, 0, rt);
            state(SM::dO, SM::S, eg[ia] * (sdo[ia] * mS), eg[ib] * (sdo[ib] * mS));
        } else {
            float y[8][4];
            const float fm = mE * mV;
            dots(x, SM::E, SM::dV, rt, 3);
            dots(y, SM::dV, SM::E, 0, rt);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = e >> 1 ? ib : ia, i = 8 * nt + 2 * tq + (e & 1);
                    y[nt][e] = i > j   ? -x[nt][e] * fm * dm[i * kLdD + j] * (fB[j] * fK[i])
                               : i < j ? -y[nt][e] * fm * dm[j * kLdD + i] * (fB[i] * fK[i])
                                       : 0.f;
                }
            rows_product(y, SM::K, 0, 3);
            dots(x, SM::E, SM::dO, rt, 3);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = e >> 1 ? ib : ia, i = 8 * nt + 2 * tq + (e & 1);
                    x[nt][e] = i >= j ? x[nt][e] * (mE * sdo[i]) * dm[i * kLdD + j] * (fB[j] * (fQ[i] * scale)) : 0.f;
                }
            rows_product(x, SM::Q, rt, 3);
            state(SM::dV, SM::S, -eg[ia] * (mV * mS), -eg[ib] * (mV * mS));
            state(SM::E, SM::dS, ege[ia] * fB[ia] * (mE * mD), ege[ib] * fB[ib] * (mE * mD));
        }
        // the gates' gradients from the dots over 16 columns each
        if (warp == 0) {
            float z[2], after = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = lane + 32 * h;
                float b = 0.f, y = 0.f;
                if (t < n) {
                    for (int s = 0; s < KS; ++s) {
                        const int64_t row = (bh * KS + s) * N + t0 + t;
                        b += kept.bb[row];
                        if (dlog_alpha)
                            y += kept.oo[row] - kept.vv[row];
                    }
                    dbeta[bh * N + t0 + t] = b;
                }
                z[h] = y;
            }
            if (dlog_alpha) {
                for (int s = 0; s < KS; ++s)
                    after += kept.cd[(bh * KS + s) * nchunk + c];
#pragma unroll
                for (int h = 1; h >= 0; --h) {
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const float y = __shfl_down_sync(0xffffffffu, z[h], o);
                        if (lane + o < 32)
                            z[h] += y;
                    }
                    const int t = lane + 32 * h;
                    if (t < n)
                        dlog_alpha[bh * N + t0 + t] = z[h] + after;
                    after += __shfl_sync(0xffffffffu, z[h], 0);
                }
            }
        }
    }
    if (!ok) {
        if (tid == 0)
            set_status(status, LA_ERR_TIMEOUT);
        return;
    }
    // through scale and norm: unit = f image, dx = r (x - unit (unit.x))
    const int image = role_k ? SM::K : SM::Q;
    const float* f = vec + (role_k ? kFacK : kFacQ) * kC;
    const float* rr = vec + (role_k ? kFacRk : kFacRq) * kC;
    __nv_bfloat16* dst = role_k ? dk : dq;
    const float mul = role_k ? 1.0f : scale;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = r0 + g + 8 * h;
        const float r = rr[i];
        float dot = 0.f;
        if (l2) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 u = __half22float2(
                    *reinterpret_cast<const __half2*>(smem + image + tile_off<RB>(i, nt) + 4 * tq));
                dot = fmaf(u.x, tot[nt][2 * h], fmaf(u.y, tot[nt][2 * h + 1], dot));
            }
            dot += __shfl_xor_sync(0xffffffffu, dot, 1);
            dot += __shfl_xor_sync(0xffffffffu, dot, 2);
        }
        dot *= f[i] * f[i];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x0 = tot[nt][2 * h], x1 = tot[nt][2 * h + 1];
            if (l2) {
                const float2 u = __half22float2(
                    *reinterpret_cast<const __half2*>(smem + image + tile_off<RB>(i, nt) + 4 * tq));
                x0 -= u.x * dot, x1 -= u.y * dot;
            }
            if (i < n)
                *reinterpret_cast<uint32_t*>(dst + (kh * N + t0 + i) * D + 8 * nt + 2 * tq) =
                    sm100::pack_bf16x2(r * mul * x0, r * mul * x1);
        }
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
    l.total = l.blobs + up256((size_t)(a.B * a.H) * n * blob_bytes<false>());
    return l;
}

struct GradTcLayout {
    size_t rows, blobs, S, sS, E, sE, dS, sD, dV, sV, oo, vv, bb, cd, total;
};
GradTcLayout grad_tc_layout(const DeltaArgs& a)
{
    const size_t n = (size_t)chunks_of(a.N), BH = (size_t)(a.B * a.H), sl = (size_t)a.dv / 16;
    const size_t state = (size_t)a.d * a.dv * 2, toks = (size_t)kC * a.dv * 2;
    GradTcLayout l;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at += up256(bytes);
        return p;
    };
    l.rows = take((size_t)(a.B * a.Hk) * n * 2 * kC * a.d * 2);
    l.blobs = take(BH * n * blob_bytes<true>());
    l.S = take(BH * (n + 1) * 2 * state);
    l.sS = take(BH * (n + 1) * a.dv * 4);
    l.E = take(BH * n * 2 * toks);
    l.sE = take(BH * n * a.dv * 4);
    l.dS = take(BH * n * state);
    l.sD = take(BH * n * a.dv * 4);
    l.dV = take(BH * n * toks);
    l.sV = take(BH * n * a.dv * 4);
    l.oo = take(BH * sl * (size_t)a.N * 4);
    l.vv = take(BH * sl * (size_t)a.N * 4);
    l.bb = take(BH * sl * (size_t)a.N * 4);
    l.cd = take(BH * sl * n * 4);
    l.total = at;
    return l;
}

// Warps per CTA of the chain: as few as give no more CTAs than SMs (a warp alone
// on its sub-partition has that tensor core to itself), at most all columns.
int chain_warps(const DeltaArgs& a, int cap)
{
    const int most = a.dv / 16 < cap ? a.dv / 16 : cap, sms = device_sm_count();
    int W = 1;
    while (W < most && a.B * a.H * (a.dv / (16 * W)) > sms)
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
        k_delta_prep<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, PrepSmem<D, false>::bytes);
    if (e != cudaSuccess)
        return e;
    k_delta_prep<D, false><<<(unsigned)(BH * n), kPrepThreads, PrepSmem<D, false>::bytes, a.stream>>>(
        static_cast<const __nv_bfloat16*>(a.q), static_cast<const __nv_bfloat16*>(a.k), a.beta,
        a.log_alpha, ws + l.rows, ws + l.blobs, a.N, n, (int)a.H, (int)a.Hk, a.fm == LA_FM_L2,
        a.scale);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    const int W = chain_warps(a, 8);
    const int smem = ChainSmem<D, false>::bytes(W);
    e = cudaFuncSetAttribute(k_delta_chain<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    k_delta_chain<D, false><<<(unsigned)(BH * (a.dv / (16 * W))), 32 * W, smem, a.stream>>>(
        ws + l.rows, ws + l.blobs, static_cast<const __nv_bfloat16*>(a.v),
        static_cast<__nv_bfloat16*>(a.out), a.S0, a.S_out, a.N, n, (int)a.H, (int)a.Hk, a.dv, nullptr, Kept{}, status);
    count_launches(1);
    return cudaGetLastError();
}

template <typename K>
cudaError_t allow_smem(K kern, int bytes)
{
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int D, int DV>
cudaError_t run_backward(const DeltaArgs& a)
{
    const GradTcLayout l = grad_tc_layout(a);
    unsigned char* ws = static_cast<unsigned char*>(a.ws);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    const Kept kept = {ws + l.S, f32(l.sS), ws + l.E, f32(l.sE), ws + l.dS, f32(l.sD),
                       ws + l.dV, f32(l.sV), f32(l.oo), f32(l.vv), f32(l.bb), f32(l.cd)};
    const int n = chunks_of(a.N), H = (int)a.H, Hk = (int)a.Hk, l2 = a.fm == LA_FM_L2;
    const int64_t BH = a.B * a.H;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v);
    const __nv_bfloat16* dout = static_cast<const __nv_bfloat16*>(a.dout);
    const int Wc = chain_warps(a, 8), Wr = chain_warps(a, kRevWarps);
    const int smem_c = ChainSmem<D, true>::bytes(Wc), smem_r = RevSmem<D>::bytes(Wr);
    cudaError_t e = allow_smem(k_delta_prep<D, true>, PrepSmem<D, true>::bytes);
    if (e == cudaSuccess)
        e = allow_smem(k_delta_chain<D, true>, smem_c);
    if (e == cudaSuccess)
        e = allow_smem(k_delta_rev<D>, smem_r);
    if (e == cudaSuccess)
        e = allow_smem(k_delta_dqk<D, DV>, DqkSmem<D, DV>::bytes);
    if (e != cudaSuccess)
        return e;
    k_delta_prep<D, true><<<(unsigned)(BH * n), kPrepThreads, PrepSmem<D, true>::bytes, a.stream>>>(
        static_cast<const __nv_bfloat16*>(a.q), static_cast<const __nv_bfloat16*>(a.k), a.beta,
        a.log_alpha, ws + l.rows, ws + l.blobs, a.N, n, H, Hk, l2, a.scale);
    count_launches(1);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    k_delta_chain<D, true><<<(unsigned)(BH * (DV / (16 * Wc))), 32 * Wc, smem_c, a.stream>>>(
        ws + l.rows, ws + l.blobs, v, nullptr, a.S0, nullptr, a.N, n, H, Hk, DV, dout, kept, a.status);
    count_launches(1);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    k_delta_rev<D><<<(unsigned)(BH * (DV / (16 * Wr))), 32 * Wr, smem_r, a.stream>>>(
        ws + l.rows, ws + l.blobs, v, dout, a.dS_out, static_cast<__nv_bfloat16*>(a.dv_), a.dS0, a.N, n,
        H, Hk, DV, a.log_alpha != nullptr, kept, a.status);
    count_launches(1);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    k_delta_dqk<D, DV><<<(unsigned)(a.B * a.Hk * n), kDqkThreads, DqkSmem<D, DV>::bytes, a.stream>>>(
        ws + l.rows, ws + l.blobs, dout, kept, static_cast<__nv_bfloat16*>(a.dq),
        static_cast<__nv_bfloat16*>(a.dk), a.dbeta, a.dlog_alpha, a.N, n, H, Hk, l2, a.scale, a.status);
    count_launches(1);
    return cudaGetLastError();
}

template <int D>
cudaError_t backward_dims(const DeltaArgs& a)
{
    switch (a.dv) {
    case 32: return run_backward<D, 32>(a);
    case 64: return run_backward<D, 64>(a);
    default: return run_backward<D, 128>(a);
    }
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

size_t delta_tc_backward_workspace(const DeltaArgs& a) { return grad_tc_layout(a).total; }

cudaError_t delta_tc_backward(const DeltaArgs& a)
{
    switch (a.d) {
    case 32: return backward_dims<32>(a);
    case 64: return backward_dims<64>(a);
    default: return backward_dims<128>(a);
    }
}

}  // namespace la
