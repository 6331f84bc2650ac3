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
//   k_delta_prep   every chunk and value head on its own: scaled fp16 images of
//                  K and Q, F, P and the factors of each token.  Nothing here
//                  depends on the state.
//   k_delta_chain  the chunks of a sequence in order.  The columns of S never
//                  mix, so a warp owns 16 value columns for the whole sequence
//                  and keeps S^T [16 x d] in registers as MMA accumulators.
//                  Everything is computed transposed: S^T K^T, E^T = R^T + ..,
//                  S^T += U^T K.  The accumulators of one product are the A
//                  fragments of the next (see la_delta_tc.cuh), so between a
//                  chunk's products nothing passes through shared memory.  Few
//                  slices are shared by two warps each.
//   k_delta_join   few long sequences are cut into segments: a first run of the
//                  chain gives each segment's map of the state, this walks them,
//                  a second run starts every segment from its own state.
//
// The gradient: k_delta_prep, the chain again keeping the states before the chunks
// and E (k_delta_chain<GRAD>), k_delta_rev for the chunks in reverse, k_delta_dqk for
// dQ and dK of every chunk on its own, k_delta_gates for dbeta and dlog_alpha.
//
// Why warp-level MMAs and not tcgen05: the chain is a string of small dependent
// products (64 tokens x 16 columns x d), whose operands are the fp32 results of the
// one before, split in two.  In registers a result is the next operand after a few
// conversions; in tensor memory each would be read out, split and written back
// between any two products, for M = 128 columns of one head on one SM, where a head
// here spreads over as many SMs as there are.
#include "la_delta_tc.cuh"

namespace la {
namespace {

using namespace delta;

// What k_delta_prep writes per chunk and value head: [F hi][F lo][P hi][P lo, for
// gradients][factors], tiles of 64 x 64 fp16 in the layout the chains read them
// from shared memory.  k^_i = fk_i K16_i and scale q^_i = fq_i Q16_i are the mapped
// rows, fk and fq holding the image's power of two, the L2 norm and the scale.  p_i is
// the power of two under |k^_i| (1 with LA_FM_L2): a gradient's P is P_ij / p_j (else P_ij
// beta_j), F's image F_ij / (p_i p_j r_i c_j) with powers of two r and c of 16 tokens each
// (r one for the chunk and c = 1 in a stable recurrence).
enum Factor {
    kFacA,    // e^{G_i} fk_i
    kFacF,    // p_i r_i
    kFacZ,    // beta_i p_i c_i
    kFacO,    // e^{G_i} fq_i
    kFacP,    // scale of P's row (a power of two)
    kFacW,    // e^{G_C - G_i} fk_i
    kFacEnd,  // [0] = e^{G_C}
    kFacB,    // beta
    kFactors,
    // gradients only; k_delta_dqk reads kFacB to kFacGl
    kFacK = kFactors,  // fk
    kFacQ,             // fq without the scale
    kFacRk,            // 1 / |k|, or 1 without the norm
    kFacRq,
    kFacPk,  // p
    kFacGh,  // G in base 2: a multiple of 2^-6 and the rest
    kFacGl,
    kFacC,   // p c
    kFacBF,  // beta p r
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
// 4 warps, a row block of 16 tokens each.  The Gram products are exact fp16 MMAs on
// the lower blocks and stay in the warp's registers as A and P.  F in 16 x 16 blocks:
// the diagonal ones by fp32 substitution (a column per lane), then by distance from
// the diagonal
//   X = A_IJ + sum_{J <= L < I} (A beta)_IL F_LJ,   F_IJ = -X - F_II beta X
// as MMAs on two-part operands: (A beta)_IL are warp I's own accumulators, F_LJ the
// image it is writing.  A stable recurrence has beta_i |k_i|^2 <= 2, so with keys as
// given beta may be as large as the key is short; everything here is therefore in units
// of p_i, keys of length 1 to 2 with beta_i p_i^2 for beta_i: |F_ij| and |X_ij| are at
// most |k_i| |k_j| < 4 there and beta X at most twice that, and keys of all lengths keep
// the same bits (with beta itself in F's place beta X left fp16 at beta = 4096, and keys
// of 1e-3 beside keys of 1 lost half of their digits).  F is under one power of two per
// chunk, with 2^10 to spare over the largest |A|; what grows past that, in a recurrence
// that is not stable, takes a power of two of its own per block, and at the end one per
// 16 rows and one per 16 columns (growth over i - j tokens is a product of the two).
// Decays of off-diagonal blocks are a row's factor to the column block's end times a
// column's from there, both at most 1, so only diagonal blocks take an exponential per
// element.
// Measured: 101 us for the 4096 chunks of B4 H8 N8192 d=128 (107 us for a gradient),
// 347 us for 16384 (two value heads per key head).  By counters on 16 x 32 heads of 512
// tokens 43% of the issue slots are used, DRAM moves 2 TB/s and the tensor cores are
// 19% busy: short stretches between barriers, with four blocks per SM.  (On the CUDA
// cores the off-diagonal blocks alone were a quarter of it.)
constexpr int kPrepThreads = 128;

template <int D, bool GRAD>
struct PrepSmem {
    static constexpr int img = 2 * row_image<D>() > fac_at<GRAD>() ? 2 * row_image<D>() : fac_at<GRAD>();
    static constexpr int diag = img;  // [4][2][16][20] fp32
    static constexpr int vec = diag + 4 * 2 * 16 * 20 * 4;
    // arrays beside the factors.  With four blocks on an SM a gradient stays under 196 KB
    // of shared memory, which leaves L1 twice of what more would (108 against 116 us)
    static constexpr int own = GRAD ? 4 : 9;
    static constexpr int bytes = vec + (own + n_factors<GRAD>()) * kC * 4 + 64;
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
    float* vec = reinterpret_cast<float*>(smem + SM::vec);
    float *fk = vec, *fq = vec + kC;  // fk: in units of p
    float* ck = vec + 2 * kC;         // fk_j times the decay from j to its block's end
    float* bp = vec + 3 * kC;         // beta p^2
    // fk and ck of P's columns: times p beta; a gradient's P stays in units of p as F does
    float *pk = GRAD ? fk : vec + 4 * kC, *pck = GRAD ? ck : vec + 5 * kC;
    float* fac = vec + SM::own * kC;  // [factors][kC]
    float *gh = GRAD ? fac + kFacGh * kC : vec + 6 * kC, *gl = GRAD ? fac + kFacGl * kC : vec + 7 * kC;
    float *pw = GRAD ? fac + kFacPk * kC : vec + 8 * kC, *sb = fac + kFacB * kC;
    float* top = fac + kFacEnd * kC + 8;  // [4] largest |A|, [4] largest |A beta| of the warps
    float* blk = top + 8;                 // [4][4] inverse scales of F's blocks beside the chunk's

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t bh = blockIdx.x / nchunk;
    const int c = blockIdx.x % nchunk;
    const int per = H / Hk;
    const int64_t kh = bh / H * Hk + (bh % H) / per;
    const int64_t t0 = (int64_t)c * kC;
    const int n = (int)min((int64_t)kC, N - t0);
    const uint32_t sK = smem_addr(smem), sQ = sK + row_image<D>();

    // rows: scaled fp16 images and factors; 16 elements per thread
    constexpr int LPR = D / 16, RPP = kPrepThreads / LPR;
#pragma unroll
    for (int r0 = 0; r0 < kC; r0 += RPP) {
        const int r = r0 + tid / LPR, p = tid % LPR;
        if (RPP > kC && r >= kC)
            break;  // whole warps
        uint4 w[2][2];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const __nv_bfloat16* src = which ? q : k;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[which][h] = r < n && src ? *reinterpret_cast<const uint4*>(src + (kh * N + t0 + r) * D + (2 * p + h) * 8)
                                           : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const uint32_t u[8] = {w[which][0].x, w[which][0].y, w[which][0].z, w[which][0].w,
                                   w[which][1].x, w[which][1].y, w[which][1].z, w[which][1].w};
            float2 s2 = both(0.f), f[8];
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] = bf2(u[i]);
                s2 = fma2(f[i], f[i], s2);
                mx = max_abs(max_abs(mx, f[i].x), f[i].y);
            }
            float ss = s2.x + s2.y;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            }
            const Pow2 s = pow2_for(mx);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 y = mul2(f[4 * h + i], both(s.to));
                    x[i] = h2(y.x, y.y);
                }
                *reinterpret_cast<uint4*>(smem + (which ? row_image<D>() : 0) + tile_off<RB>(r, 2 * p + h)) =
                    make_uint4(x[0], x[1], x[2], x[3]);
            }
            if (p == 0) {
                const float norm = l2 ? rsqrtf(ss + kL2Eps) : 1.0f;
                (which ? fq : fk)[r] = s.from * norm * (which ? scale : 1.0f);
                if (!which)
                    pw[r] = ss;  // for now
                if (GRAD)
                    fac[(which ? kFacRq : kFacRk) * kC + r] = norm;
                if (GRAD && which)
                    fac[kFacQ * kC + r] = s.from * norm;
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
#pragma unroll 4
        for (int i = tid; i < 2 * row_image<D>() / 16; i += kPrepThreads)
            dst[i] = reinterpret_cast<const uint4*>(smem)[i];
    }
    if (tid < kC) {
        const float h = gh[tid], l = gl[tid], hc = gh[kC - 1], lc = gl[kC - 1];
        // p = 2^x where |k|^2 is in [2^{2 x}, 2^{2 x + 2}), and fk in units of it
        const int x = l2 ? 0 : ((int)(__float_as_uint(pw[tid]) >> 23) - 127) >> 1;
        const float e = exp2f(h + l), f = fk[tid], p = __uint_as_float((uint32_t)(127 + x) << 23);
        pw[tid] = p;
        fk[tid] = f * __uint_as_float((uint32_t)(127 - x) << 23);
        bp[tid] = sb[tid] * p * p;
        const float to = exp2f((gh[tid | 15] - h) + (gl[tid | 15] - l));
        ck[tid] = fk[tid] * to;
        if (!GRAD)
            pk[tid] = f * sb[tid], pck[tid] = f * sb[tid] * to;
        fac[kFacA * kC + tid] = e * f;
        fac[kFacZ * kC + tid] = sb[tid] * p;
        fac[kFacO * kC + tid] = e * fq[tid];
        fac[kFacW * kC + tid] = exp2f((hc - h) + (lc - l)) * f;
        if (tid == 0)
            fac[kFacEnd * kC] = exp2f(hc + lc);
        if (GRAD) {
            fac[kFacK * kC + tid] = f;
            fac[kFacC * kC + tid] = p;
        }
    }
    __syncthreads();  // the images are read: F and P take their place

    // A and P, their largest entries; blocks right of the diagonal are never read
    const int i0 = 16 * warp + g;
    float pm[2] = {0.f, 0.f}, am = 0.f, abm = 0.f;
    const float fki[2] = {fk[i0], fk[i0 + 8]}, fqi[2] = {fq[i0], fq[i0 + 8]};
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        if (b <= warp) {
            float row[2];  // decay from block b's end to the row
#pragma unroll
            for (int r = 0; r < 2; ++r)
                row[r] = exp2f((gh[i0 + 8 * r] - gh[16 * b + 15]) + (gl[i0 + 8 * r] - gl[16 * b + 15]));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int nt = 2 * b + h, j = 8 * nt + 2 * tq;
                const float2 col = *reinterpret_cast<const float2*>((b < warp ? ck : fk) + j);
                const float2 be = *reinterpret_cast<const float2*>(bp + j);
                const float2 pcol = *reinterpret_cast<const float2*>((b < warp ? pck : pk) + j);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = i0 + (e >> 1) * 8, jj = j + (e & 1);
                    float dec = row[e >> 1];
                    if (b == warp)
                        dec = jj <= i ? exp2f((gh[i] - gh[jj]) + (gl[i] - gl[jj])) : 0.f;
                    const float bj = e & 1 ? be.y : be.x;
                    // a select, not a product with 0: nothing to the right of the diagonal counts
                    ak[nt][e] = b < warp || jj < i ? ak[nt][e] * fki[e >> 1] * (dec * (e & 1 ? col.y : col.x)) : 0.f;
                    aq[nt][e] = b < warp || jj <= i ? aq[nt][e] * fqi[e >> 1] * (dec * (e & 1 ? pcol.y : pcol.x)) : 0.f;
                    pm[e >> 1] = max_abs(pm[e >> 1], aq[nt][e]);
                    am = max_abs(am, ak[nt][e]);
                    abm = max_abs(abm, ak[nt][e] * bj);
                }
            }
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
            if (nt <= 2 * warp + 1) {
                uint32_t hi, lo;
                h2_split(aq[nt][2 * r] * s.to, aq[nt][2 * r + 1] * s.to, hi, lo);
                unsigned char* at = smem + 2 * kTile + tile_off<128>(i, nt) + 4 * tq;
                *reinterpret_cast<uint32_t*>(at) = hi;
                if (GRAD)
                    *reinterpret_cast<uint32_t*>(at + kTile) = lo;
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        abm = fmaxf(abm, __shfl_xor_sync(0xffffffffu, abm, o));
    }
    if (lane == 0)
        top[warp] = am, top[4 + warp] = abm;
    // the diagonal block, for the substitution
    float* sd = reinterpret_cast<float*>(smem + SM::diag) + warp * 2 * 16 * 20;
    float* sdb = sd + 16 * 20;  // -A beta
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        if (b == warp) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = g * 20 + 8 * h + 2 * tq;
                const float2 be = *reinterpret_cast<const float2*>(bp + 16 * b + 8 * h + 2 * tq);
                const float2 minus = make_float2(-be.x, -be.y);
                *reinterpret_cast<float2*>(sd + at) = row_a(ak[2 * b + h]);
                *reinterpret_cast<float2*>(sd + at + 160) = row_b(ak[2 * b + h]);
                *reinterpret_cast<float2*>(sdb + at) = mul2(minus, row_a(ak[2 * b + h]));
                *reinterpret_cast<float2*>(sdb + at + 160) = mul2(minus, row_b(ak[2 * b + h]));
            }
        }
    }
    __syncthreads();
    // F s for s = 2^4 / max |A| and (A beta) t, both powers of two
    const Pow2 s = pow2_for(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * 16.0f);
    const Pow2 t = pow2_for(fmaxf(fmaxf(top[4], top[5]), fmaxf(top[6], top[7])));
    // The first time round every block is under s, and what fp16 does not hold is only
    // noticed; then a block that leaves fp16 under s takes a scale of its own beside it
    bool careful = false;
    uint32_t bad = 0;  // not 0 once infinities have come
    // two elements of F's images, x and y of a row
    auto put2 = [&](int i, int j, float x, float y) {
        uint32_t hi, lo;
        h2_split(x, y, hi, lo);
        asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(bad) : "r"(hi), "r"(0));
        unsigned char* at = smem + tile_off<128>(i, j >> 3) + (j & 7) * 2;
        *reinterpret_cast<uint32_t*>(at) = hi;
        *reinterpret_cast<uint32_t*>(at + kTile) = lo;
    };
    // that scale for a block's 16 x 16 entries x, which are multiplied by it
    auto own_scale = [&](float* x, int n) {
        float m = 0.f;
        for (int i = 0; i < n; ++i)
            m = max_abs(m, x[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        Pow2 q = {1.0f, 1.0f};
        if (m > 32768.0f)
            q = pow2_for(m);
        for (int i = 0; i < n; ++i)
            x[i] *= q.to;
        return q.from;
    };
    {  // the diagonal block: column `lane & 15` of block `warp`
        const int j = lane & 15;
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float x = -sd[i * 20 + j];
#pragma unroll
            for (int l = 0; l < i; l += 4) {  // zero from the diagonal on
                const float4 a = *reinterpret_cast<const float4*>(sdb + i * 20 + l);
                x = fmaf(a.x, f[l], x);
                if (l + 1 < i)
                    x = fmaf(a.y, f[l + 1], x);
                if (l + 2 < i)
                    x = fmaf(a.z, f[l + 2], x);
                if (l + 3 < i)
                    x = fmaf(a.w, f[l + 3], x);
            }
            f[i] = x;
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                sd[i * 20 + j] = f[i];
        }
        __syncwarp();
    }
    auto keep_rows = [&](float r) {
        if (lane < 16) {
            const int i = 16 * warp + lane;
            fac[kFacF * kC + i] = r * pw[i];
            if (GRAD)
                fac[kFacBF * kC + i] = r * pw[i] * sb[i];
        }
    };
    keep_rows(s.from);
    const uint32_t sF = smem_addr(smem);
    for (;; careful = true) {
        {  // its images by row pairs
            const int i = 16 * warp + (lane >> 3), jj = (lane & 7) * 2;
            float f[8];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float2 x = mul2(*reinterpret_cast<const float2*>(sd + (i + 4 * m - 16 * warp) * 20 + jj), both(s.to));
                f[2 * m] = x.x, f[2 * m + 1] = x.y;
            }
            if (careful)
                blk[5 * warp] = own_scale(f, 8);
#pragma unroll
            for (int m = 0; m < 4; ++m)
                put2(i + 4 * m, 16 * warp + jj, f[2 * m], f[2 * m + 1]);
        }
        __syncthreads();
        // off-diagonal: at distance `dist` warp I computes block (I, I - dist)
#pragma unroll 1
        for (int dist = 1; dist < 4; ++dist) {
            if (warp >= dist) {
                const int J = warp - dist;
                float x[2][4];
                uint32_t hi[4], lo[4], b[4];
#pragma unroll
                for (int L = 0; L < 3; ++L) {
                    if (L == J) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[h][e] = ak[2 * L + h][e] * s.to;
                    }
                }
#pragma unroll
                for (int L = 0; L < 3; ++L) {
                    if (L >= J && L < warp) {
                        float z[2][4];
                        clear(z);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float2 be = *reinterpret_cast<const float2*>(bp + 16 * L + 8 * h + 2 * tq);
                            h2_split(ak[2 * L + h][0] * be.x * t.to, ak[2 * L + h][1] * be.y * t.to, hi[2 * h], lo[2 * h]);
                            h2_split(ak[2 * L + h][2] * be.x * t.to, ak[2 * L + h][3] * be.y * t.to, hi[2 * h + 1],
                                     lo[2 * h + 1]);
                        }
                        ldsm4t(b, addr_bt<128>(sF, lane, 16 * L, 16 * J));
                        mma(z[0], hi, b[0], b[1]);
                        mma(z[1], hi, b[2], b[3]);
                        mma(z[0], lo, b[0], b[1]);
                        mma(z[1], lo, b[2], b[3]);
                        ldsm4t(b, addr_bt<128>(sF + kTile, lane, 16 * L, 16 * J));
                        mma(z[0], hi, b[0], b[1]);
                        mma(z[1], hi, b[2], b[3]);
                        const float from = careful ? t.from * blk[4 * L + J] : t.from;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[h][e] = fmaf(z[h][e], from, x[h][e]);
                    }
                }
                // X s, then beta X in F's place as the second product's operand
                const int j0 = 16 * J + 2 * tq;
                const float be0 = bp[i0], be1 = bp[i0 + 8];
                float from = -s.from, y[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[h][e] = (e >> 1 ? be1 : be0) * x[h][e];
                if (careful)
                    from *= own_scale(y[0], 8) * blk[5 * warp];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    put2(i0, j0 + 8 * h, y[h][0], y[h][1]);
                    put2(i0 + 8, j0 + 8 * h, y[h][2], y[h][3]);
                }
                __syncwarp();
                clear(y);
                uint32_t bl[4];
                ldsm4(hi, addr_a<128>(sF, lane, 16 * warp, 16 * warp));
                ldsm4(lo, addr_a<128>(sF + kTile, lane, 16 * warp, 16 * warp));
                ldsm4t(b, addr_bt<128>(sF, lane, 16 * warp, 16 * J));
                ldsm4t(bl, addr_bt<128>(sF + kTile, lane, 16 * warp, 16 * J));
                mma(y[0], hi, b[0], b[1]);
                mma(y[1], hi, b[2], b[3]);
                mma(y[0], lo, b[0], b[1]);
                mma(y[1], lo, b[2], b[3]);
                mma(y[0], hi, bl[0], bl[1]);
                mma(y[1], hi, bl[2], bl[3]);
                __syncwarp();
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[h][e] = fmaf(from, y[h][e], -x[h][e]);
                if (careful)
                    blk[4 * warp + J] = own_scale(y[0], 8);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    put2(i0, j0 + 8 * h, y[h][0], y[h][1]);
                    put2(i0 + 8, j0 + 8 * h, y[h][2], y[h][3]);
                }
            }
            if (dist < 3)
                __syncthreads();
        }
        if (careful || !__syncthreads_or(bad))
            break;
    }
    if (careful) {  // blocks to rows and columns: c by the last rows, r what is left
        __syncthreads();
        const int last = (n - 1) >> 4;
        auto c = [&](int J) { return J <= last ? blk[4 * last + J] / blk[4 * last] : 1.0f; };
        float r = 0.f;
        for (int J = 0; J <= warp; ++J)
            r = fmaxf(r, blk[4 * warp + J] / c(J));
        for (int J = 0; J <= warp; ++J) {
            const __half2 f = __float2half2_rn(blk[4 * warp + J] / (r * c(J)));  // at most 1
            unsigned char* at = smem + tile_off<128>(16 * warp + (lane >> 1), 2 * J + (lane & 1));
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                uint4 x = *reinterpret_cast<const uint4*>(at + part * kTile);
                __half2* h = reinterpret_cast<__half2*>(&x);
                h[0] = __hmul2(h[0], f), h[1] = __hmul2(h[1], f), h[2] = __hmul2(h[2], f), h[3] = __hmul2(h[3], f);
                *reinterpret_cast<uint4*>(at + part * kTile) = x;
            }
        }
        keep_rows(s.from * r);
        if (lane < 16) {
            const int i = 16 * warp + lane;
            fac[kFacZ * kC + i] *= c(warp);
            if (GRAD)
                fac[kFacC * kC + i] *= c(warp);
        }
        __syncthreads();
    }
    uint4* blob = reinterpret_cast<uint4*>(blobs + (bh * nchunk + c) * (int64_t)blob_bytes<GRAD>());
#pragma unroll 4
    for (int i = tid; i < fac_at<GRAD>() / 16; i += kPrepThreads)
        blob[i] = reinterpret_cast<const uint4*>(smem)[i];
    for (int i = tid; i < n_factors<GRAD>() * kC / 4; i += kPrepThreads)
        blob[fac_at<GRAD>() / 16 + i] = reinterpret_cast<const uint4*>(fac)[i];
}

// ------------------------------------------------------------ k_delta_chain --
// Slices of 16 value columns; the tiles of a chunk are shared by a CTA's slices and
// arrive by bulk copies a ring of stages ahead; V comes by cp.async one chunk ahead,
// and outputs leave through the slice's own tile, turned back to token-major by
// stmatrix.
//
// SP = 1: a warp does all of a slice's chunk.  SP = 2: two warps share it, each with
// half of the state's rows (the contracted index of S^T K^T and of S^T Q^T, the
// columns of the update) and half of the chunk's token tiles (0 and 3, or 1 and 2:
// equal shares of the triangular products).  They exchange fp32 sums through shared
// memory three times a chunk.  A warp's products follow one another, each waiting
// for the last: with a slice per warp a chunk was 7100 cycles at d = 128 of which
// the tensor core works 3100, so two warps shorten it where there are SMs to spare.
// Measured: 283 us for the 128 chunks of B4 H8 N8192 d=128 (SP = 2: 4300 cycles per
// chunk, tensor cores 38% busy on an SM, bound by the latency of its dependent
// products and conversions), 639 us for B16 H32 N2011 (SP = 1: three rounds of 152
// CTAs, 518 us, the rest with SP = 2, 121 us; by counters at N = 512 the tensor cores
// work 58% of the first part's time).  The chain of a gradient 340 us.
//
// With two warps on a sub-partition (SP = 1, eight warps) no barrier spans the CTA
// inside the loop: the warp that is last to finish with a stage asks for the chunk
// that takes its place, so warps drift apart and one's products run under another's
// arithmetic (512 heads of 2011 tokens: 734 us in step, 690 us adrift).  Alone on
// their sub-partitions (SP = 2) warps only lose by it: in step they share what the
// instruction cache fetches (reverse chain, 32 heads of 8192 tokens: 529 us in step,
// 595 us adrift).
constexpr int kXch = 2048;  // bytes of one warp's exchange buffer: 16 floats per lane

template <int D, bool GRAD, int SP>
struct ChainSmem {
    static constexpr int stages = SP == 1 ? 3 : 2;  // what fits at d = 128
    // [K][Q][F hi][F lo][P, for outputs][factors]
    static constexpr int fac = 2 * row_image<D>() + (GRAD ? 2 : 3) * kTile, stage = fac + kFactors * kC * 4;
    static constexpr int v = stages * stage;
    // per slice: V twice, O (GRAD: dO), and for each of two warps four exchange buffers
    static constexpr int x = 3 * kC * 32, per_slice = x + (SP > 1 ? SP * 4 * kXch : 0);
    static int bytes(int W) { return v + W * per_slice + 128; }
};

// What the forward pass of a gradient keeps per chunk, in the fragments' own
// order ([16 columns][16-step][register][lane], every store 128 bytes): the state
// before the chunk and E, as two fp16 parts with a scale per value column (states:
// per column and half of their rows; E and dV: per column and 16 tokens, dV in units of
// 1 / p as beta goes with the square of that).  An 8 x 8 block is 128 bytes with its rows in
// order, so k_delta_dqk reads it with ldmatrix whichever way round it needs it.
struct Kept {
    unsigned char* S;   // [BH][nchunk][2 parts][D DV] fp16
    float* sS;          // [BH][nchunk][2][DV]
    unsigned char* E;   // [BH][nchunk][2 parts][64 DV] fp16
    float* sE;          // [BH][nchunk][4][DV]
    unsigned char* dS;  // [BH][nchunk][D DV] fp16: gradient of the state after the chunk
    float* sD;          // [BH][nchunk][2][DV]
    unsigned char* dV;  // [BH][nchunk][64 DV] fp16
    float* sV;          // [BH][nchunk][4][DV]
    float* bb;          // [BH][DV / 16][N] Y.E over 16 columns
    // with gates only
    unsigned char* dVl;  // [BH][nchunk][64 DV] the other part of dV
    float4* KS;          // [BH][nchunk][DV / 16][8][32] S0^T K16, C tiles of 8 tokens
    float* hq;           // [BH][DV / 16][N] e^{G_i} q_i.(S0 dO_i) over 16 columns
    float* hk;           // [BH][DV / 16][N] -e^{G_i} k_i.(S0 dV_i)
    float* ll;           // [BH][DV / 16][N] e^{G_C - G_j} k_j.(dS1 U_j)
    float* cd;           // [BH][DV / 16][2][nchunk] <S0, dS1> over half of the rows
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

// The ring of stages: barriers for filled and for read, and how many warps have read
// (STEP: a barrier of the CTA in their place).  A warp's reads are ordered before the
// refill by its arrival and the refiller's (satisfied) wait on the same barrier; the
// count only tells who is last.  A fence instead would also wait for the chunk's stores
// to global memory.
template <int STAGES, bool STEP>
struct Ring {
    uint64_t *full, *read;
    unsigned* done;
    unsigned warps;
    bool ok;  // false once a wait has run out: the warp leaves its loop, and no stage it has
              // not read is filled again (a barrier with a copy still pending is not armed)
    __device__ __forceinline__ Ring(void* at, unsigned w)
        : full(static_cast<uint64_t*>(at)), read(full + STAGES), done(reinterpret_cast<unsigned*>(read + STAGES)),
          warps(w), ok(true)
    {
        if (threadIdx.x == 0) {
            for (int i = 0; i < STAGES; ++i) {
                sm100::mbar_init(full + i, 1);
                sm100::mbar_init(read + i, w);
                done[i] = 0;
            }
            sm100::fence_mbar_init();
        }
        __syncthreads();
    }
    __device__ __forceinline__ void wait(int i)
    {
        ok = __all_sync(0xffffffffu, wait_for(full + i % STAGES, (i / STAGES) & 1));
    }
    // warps that meet in every chunk find out at its end, together
    __device__ __forceinline__ bool go_on() const { return STEP || ok; }
    // after a wait has run out: what is in flight gets as long again
    __device__ __forceinline__ void drain()
    {
        for (int i = 0; i < STAGES; ++i)
            for (int parity = 0; parity < 2; ++parity)
                wait_for(full + i, parity);
    }
    // this warp is done with chunk i; true in one thread once all are.  (A warp that has
    // left does not arrive, so the others' count never fills and they run out in turn.)
    __device__ __forceinline__ bool last(int i)
    {
        if (STEP) {
            ok = __syncthreads_and(ok);
            return threadIdx.x == 0;
        }
        __syncwarp();
        if ((threadIdx.x & 31) != 0)
            return false;
        sm100::mbar_arrive(read + i % STAGES);
        if (atomicAdd_block(done + i % STAGES, 1u) != warps - 1)
            return false;
        done[i % STAGES] = 0;
        return wait_for(read + i % STAGES, (i / STAGES) & 1);
    }
};

// One warp's place in a slice shared by SP warps.  Token tiles (16 tokens) are
// held in local order: this warp's own first, then the other's.
template <int SP>
struct Share {
    static constexpr int own = 4 / SP;  // token tiles of a warp
    int slice, half;
    unsigned char *mine, *other;  // exchange buffers
    int lane;
    __device__ __forceinline__ int tile(int i) const
    {
        return SP == 1 ? i : (i >> 1 ? !half : half) ? 1 + (i & 1) : 3 * (i & 1);
    }
    __device__ __forceinline__ void sync() const
    {
        if (SP > 1)
            asm volatile("bar.sync %0, %1;" ::"r"(1 + slice), "r"(32 * SP) : "memory");
        else
            __syncwarp();
    }
    // y[tile][C tile][token of a pair], local tiles 2 part and 2 part + 1, summed over
    // the columns -> row[first token of the chunk + ..]
    __device__ __forceinline__ void store_sums(float* row, const float (&y)[8], int part, int64_t t0, int64_t N) const
    {
        const float x = delta::sum8(y, lane);
        const int g = lane >> 2;
        const int64_t t = t0 + 16 * tile(2 * part + (g >> 2)) + 8 * ((g >> 1) & 1) + 2 * (lane & 3) + (g & 1);
        if (t < N)
            row[t] = x;
    }
    // two token tiles (C layout) to buffer b, and the partner's from it
    __device__ __forceinline__ void put(int b, const float (&x)[2][4], const float (&y)[2][4]) const
    {
        float4* at = reinterpret_cast<float4*>(mine + b * kXch) + lane;
        at[0] = make_float4(x[0][0], x[0][1], x[0][2], x[0][3]);
        at[32] = make_float4(x[1][0], x[1][1], x[1][2], x[1][3]);
        at[64] = make_float4(y[0][0], y[0][1], y[0][2], y[0][3]);
        at[96] = make_float4(y[1][0], y[1][1], y[1][2], y[1][3]);
    }
    template <bool ADD>
    __device__ __forceinline__ void get(int b, float (&x)[2][4], float (&y)[2][4]) const
    {
        const float4* at = reinterpret_cast<const float4*>(other + b * kXch) + lane;
        float(*to[2])[4] = {x, y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = at[32 * i];
            float* d = to[i >> 1][i & 1];
            d[0] = ADD ? d[0] + v.x : v.x, d[1] = ADD ? d[1] + v.y : v.y;
            d[2] = ADD ? d[2] + v.z : v.z, d[3] = ADD ? d[3] + v.w : v.w;
        }
    }
};

// factor pair of the tokens of C tile `nt` of token tile `t`
__device__ __forceinline__ float2 fac2(const float* fac, int which, int t, int nt, int tq)
{
    return *reinterpret_cast<const float2*>(fac + which * kC + 16 * t + 8 * nt + 2 * tq);
}

// the scale of one column (e = 0: g, 2: g + 8) over the 16 tokens of tile i of x
__device__ __forceinline__ Pow2 tile_scale(const float (&x)[8][4], int i, int e)
{
    const float *a = x[2 * i] + e, *b = x[2 * i + 1] + e;
    return pow2_for(quad_max(fmaxf(fmaxf(fabsf(a[0]), fabsf(a[1])), fmaxf(fabsf(b[0]), fabsf(b[1])))));
}

// acc[2 i], acc[2 i + 1] += a b[i].  A product on two parts goes over all tiles with
// the one, then with the other: MMAs on the same accumulator stay apart
template <int N_>
__device__ __forceinline__ void mma_tiles(float (*acc)[4], const uint32_t (&a)[4], const uint32_t (&b)[N_][4])
{
#pragma unroll
    for (int i = 0; i < N_; ++i) {
        mma(acc[2 * i], a, b[i][0], b[i][1]);
        mma(acc[2 * i + 1], a, b[i][2], b[i][3]);
    }
}

// x[tile i] += (hi + lo) (B hi + B lo) without lo lo, over the tiles that `want` names;
// load(b, i, part) fetches B
template <int N_, typename Want, typename Load>
__device__ __forceinline__ void three_products(float (&x)[2 * N_][4], const uint32_t (&hi)[4], const uint32_t (&lo)[4],
                                               Want want, Load load)
{
    uint32_t b[N_][4], c[N_][4];
#pragma unroll
    for (int i = 0; i < N_; ++i)
        if (want(i))
            load(b[i], i, 0), load(c[i], i, 1);
    auto all = [&](const uint32_t(&a)[4], const uint32_t(&t)[N_][4]) {
#pragma unroll
        for (int i = 0; i < N_; ++i)
            if (want(i)) {
                mma(x[2 * i], a, t[i][0], t[i][1]);
                mma(x[2 * i + 1], a, t[i][2], t[i][3]);
            }
    };
    all(hi, b);
    all(lo, b);
    all(hi, c);
}

// s += (hi + lo) times rows row0 .. + 15 of an image, columns d0 .. + 16 KK
template <int RB, int KK>
__device__ __forceinline__ void rows_update(float (&s)[2 * KK][4], const uint32_t (&hi)[4], const uint32_t (&lo)[4],
                                            uint32_t image, int lane, int row0, int d0)
{
    constexpr int G = KK < 4 ? KK : 4;
#pragma unroll
    for (int j = 0; j < KK; j += G) {
        uint32_t b[G][4];
#pragma unroll
        for (int i = 0; i < G; ++i)
            ldsm4t(b[i], addr_bt<RB>(image, lane, row0, d0 + 16 * (j + i)));
        mma_tiles<G>(s + 2 * j, hi, b);
        mma_tiles<G>(s + 2 * j, lo, b);
    }
}


// A sequence may be cut into segments of `len` chunks that run at once.  A chunk's
// map of the state is affine in it, S1 = M S0 + B with B from V, column by column.
// So with S0 = 0 a segment's columns give its B, and d more columns with V = 0 that
// start as the unit matrix give its M (carry: only these ends are wanted);
// k_delta_join then walks the segments, and the run that counts starts each from its
// own state.
struct Segments {
    int count, len;      // segments that run, chunks of one
    const float* start;  // [BH][count][d][dv] state before each, or NULL: one segment from S0
    int carry;
    float *B, *M;        // carry: [BH][count][d][dv], [BH][count][d][d]
    int first;           // the first segment that runs
    int blob, fac;       // bytes of a blob, where its factors lie
    int64_t skip;        // runs that another launch takes
};

// READS: outputs are wanted (a branch on the pointer instead cuts every stretch of
// products in two); in a gradient, S0^T K and the dots of S0^T Q with dO for the gates'
template <int D, bool GRAD, int SP, bool READS>
__global__ void __launch_bounds__(256, 1)
    k_delta_chain(const unsigned char* __restrict__ rows, const unsigned char* __restrict__ blobs,
                  const __nv_bfloat16* __restrict__ v, __nv_bfloat16* __restrict__ out,
                  const float* S0, float* S_out, int64_t N, int nchunk, int H, int Hk, int DV,
                  const __nv_bfloat16* __restrict__ dout, Kept kept, Segments seg, int* status)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    using SM = ChainSmem<D, GRAD, SP>;
    constexpr int RB = 2 * D;                    // bytes per row
    constexpr int NT = D / 8 / SP, KK = NT / 2;  // n tiles of this warp's part of S^T; its 16-steps
    constexpr int OWN = Share<SP>::own;
    const int tid = threadIdx.x, lane = tid & 31, W = blockDim.x / (32 * SP);
    const int g = lane >> 2, tq = lane & 3;
    Share<SP> sh;
    sh.slice = (tid >> 5) / SP, sh.half = (tid >> 5) % SP, sh.lane = lane;
    const int slices = (DV + (seg.carry ? D : 0)) / (16 * W);
    const int64_t run = blockIdx.x / slices + seg.skip;  // head and segment
    const int64_t bh = run / seg.count;
    const int lo = (int)(run % seg.count) * seg.len, len = min(seg.len, nchunk - lo);
    const int col0 = (blockIdx.x % slices) * 16 * W + 16 * sh.slice;
    const int64_t kh = bh / H * Hk + (bh % H) / (H / Hk);
    const uint32_t base = smem_addr(smem);
    const int my = SM::v + sh.slice * SM::per_slice;
    sh.mine = smem + my + SM::x + sh.half * 4 * kXch;
    sh.other = smem + my + SM::x + (SP - 1 - sh.half) * 4 * kXch;
    const uint32_t sv = base + my, so = sv + 2 * kC * 32;
    Ring<SM::stages, (SP > 1)> ring(smem + SM::v + W * SM::per_slice, blockDim.x >> 5);
    const unsigned char* row_src = rows + kh * nchunk * (int64_t)(2 * row_image<D>());
    const unsigned char* blob_src = blobs + bh * nchunk * (int64_t)seg.blob;
    const int d0 = sh.half * (D / SP);  // first state row of this warp

    auto load_stage = [&](int i) {
        const int64_t c = lo + i;
        const uint32_t dst = base + (i % SM::stages) * SM::stage;
        uint64_t* bar = ring.full + i % SM::stages;
        const unsigned char *r = row_src + c * (2 * row_image<D>()), *f = blob_src + c * seg.blob;
        if (READS && !GRAD) {
            sm100::mbar_arrive_expect_tx(bar, SM::stage);
            delta::bulk_load(dst, r, 2 * row_image<D>(), bar);
            delta::bulk_load(dst + 2 * row_image<D>(), f, blob_bytes<false>(), bar);
        } else {  // no P, and Q where it is wanted
            constexpr int img = (READS ? 2 : 1) * row_image<D>();
            sm100::mbar_arrive_expect_tx(bar, img + 2 * kTile + kFactors * kC * 4);
            delta::bulk_load(dst, r, img, bar);
            delta::bulk_load(dst + 2 * row_image<D>(), f, 2 * kTile, bar);
            delta::bulk_load(dst + SM::fac, f + seg.fac, kFactors * kC * 4, bar);
        }
    };
    // this warp's token tiles of the slice's columns
    auto load_cols = [&](uint32_t dst, const __nv_bfloat16* src, int c) {
        const int64_t t0 = (int64_t)c * kC;
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int t = 16 * sh.tile(i) + (lane >> 1), p = lane & 1;
            const bool live = t0 + t < N && col0 < DV;  // the unit columns have no V
            cp16(dst + tile_off<32>(t, p), src + (live ? (bh * N + t0 + t) * DV + col0 + p * 8 : 0), live);
        }
    };
    if (tid == 0)
        for (int i = 0; i < SM::stages && i < len; ++i)
            load_stage(i);
    load_cols(sv, v, lo);
    cp_commit();

    float s[NT][4];  // S^T[col0 + g, + 8][d0 + 8 nt + 2 tq, + 1]
    const float* start = seg.start ? seg.start + run * D * DV : S0 ? S0 + bh * D * DV : nullptr;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = d0 + 8 * nt + 2 * tq + (e & 1), col = col0 + g + (e >> 1) * 8;
            s[nt][e] = seg.carry ? (row == col - DV ? 1.f : 0.f) : start ? start[row * DV + col] : 0.f;
        }

    auto row_max = [&](float& m0, float& m1) {
        m0 = m1 = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m0 = max_abs(max_abs(m0, s[nt][0]), s[nt][1]);
            m1 = max_abs(max_abs(m1, s[nt][2]), s[nt][3]);
        }
        m0 = quad_max(m0), m1 = quad_max(m1);
    };
    auto split_state = [&](int kk, Pow2 p0, Pow2 p1, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
        h2_split(row_a(s[2 * kk]), p0.to, hi[0], lo[0]);
        h2_split(row_b(s[2 * kk]), p1.to, hi[1], lo[1]);
        h2_split(row_a(s[2 * kk + 1]), p0.to, hi[2], lo[2]);
        h2_split(row_b(s[2 * kk + 1]), p1.to, hi[3], lo[3]);
    };
    auto keep_state_scale = [&](int64_t c, Pow2 p0, Pow2 p1) {
        if (tq == 0) {
            float* ss = kept.sS + ((bh * nchunk + c) * 2 + sh.half) * DV + col0;
            ss[g] = p0.from, ss[g + 8] = p1.from;
            if (SP == 1)
                ss[DV + g] = p0.from, ss[DV + g + 8] = p1.from;
        }
    };

    ring.wait(0);
    for (int step = 0; step < len && ring.go_on(); ++step) {
        const int c = lo + step;
        const uint32_t st = base + (step % SM::stages) * SM::stage;
        const uint32_t sK = st, sQ = st + row_image<D>(), sF = st + 2 * row_image<D>(), sP = sF + 2 * kTile;
        const float* fac = reinterpret_cast<const float*>(smem + (step % SM::stages) * SM::stage + SM::fac);
        if (GRAD && READS) {  // dO, wanted after E
            load_cols(so, dout, c);
            cp_commit();
        }
        load_cols(sv + ((step + 1) & 1) * kC * 32, v, c + 1);  // nothing past the last chunk
        cp_commit();

        // S^T K^T and S^T Q^T over this warp's rows of S, split on the way
        float m0, m1;
        row_max(m0, m1);
        const Pow2 p0 = pow2_for(m0), p1 = pow2_for(m1);
        float r[8][4], o[8][4];  // local token order
        clear(r);
        clear(o);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            uint32_t hi[4], lo[4];
            split_state(kk, p0, p1, hi, lo);
            if (GRAD) {
                const int block = (col0 / 16) * (D / 16) + d0 / 16 + kk;
                keep_part(kept.S, 2 * (bh * nchunk + c), D * DV * 2, block, lane, hi);
                // the second part is read by k_delta_rev alone, fragment by fragment
                reinterpret_cast<uint4*>(kept.S + (2 * (bh * nchunk + c) + 1) * (int64_t)(D * DV * 2))[block * 32 + lane] =
                    make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                uint32_t bk[2][4], bq[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    ldsm4(bk[i], addr_b<RB>(sK, lane, 16 * sh.tile(j + i), d0 + 16 * kk));
                if (READS) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        ldsm4(bq[i], addr_b<RB>(sQ, lane, 16 * sh.tile(j + i), d0 + 16 * kk));
                }
                mma_tiles<2>(r + 2 * j, hi, bk);
                if (READS)
                    mma_tiles<2>(o + 2 * j, hi, bq);
                mma_tiles<2>(r + 2 * j, lo, bk);
                if (GRAD && READS)  // o enters an fp32 gradient
                    mma_tiles<2>(o + 2 * j, lo, bq);
            }
        }
        if (GRAD)
            keep_state_scale(c, p0, p1);
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            scale_rows(r[nt], p0.from, p1.from);
            if (READS)
                scale_rows(o[nt], p0.from, p1.from);
        }
        auto pair = [](float (&x)[8][4], int i) -> float(&)[2][4] {
            return *reinterpret_cast<float(*)[2][4]>(x + 2 * i);
        };
        if (SP > 1) {
            sh.put(0, pair(r, 2), pair(r, 3));
            if (READS)
                sh.put(1, pair(o, 2), pair(o, 3));
            sh.sync();
            sh.template get<true>(0, pair(r, 0), pair(r, 1));
            if (READS)
                sh.template get<true>(1, pair(o, 0), pair(o, 1));
        }
        if (GRAD && READS) {
#pragma unroll
            for (int nt = 0; nt < 2 * OWN; ++nt)
                kept.KS[(((bh * nchunk + c) * (DV / 16) + col0 / 16) * 8 + 2 * sh.tile(nt >> 1) + (nt & 1)) * 32 + lane] =
                    make_float4(r[nt][0], r[nt][1], r[nt][2], r[nt][3]);
        }
        cp_wait<GRAD && READS ? 2 : 1>();  // V
        __syncwarp();
        // R of the own tiles, z = beta p c R
        float z[8][4];
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            uint32_t w[4];
            ldsm4t(w, addr_ct<32>(sv + (step & 1) * kC * 32, lane, 16 * sh.tile(i), 0));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int nt = 2 * i + u;
                const float2 a = fac2(fac, kFacA, sh.tile(i), u, tq), be = fac2(fac, kFacZ, sh.tile(i), u, tq);
                const float2 minus = make_float2(-a.x, -a.y);
                set_rows(r[nt], fma2(minus, row_a(r[nt]), bf2(w[2 * u])), fma2(minus, row_b(r[nt]), bf2(w[2 * u + 1])));
                set_rows(z[nt], mul2(be, row_a(r[nt])), mul2(be, row_b(r[nt])));
                if (READS)
                    scale_cols(o[nt], fac2(fac, kFacO, sh.tile(i), u, tq));
            }
        }
        if (SP > 1) {
            sh.put(2, pair(z, 0), pair(z, 1));
            sh.sync();
            sh.template get<false>(2, pair(z, 2), pair(z, 3));
        }
        float e0 = 0.f, e1 = 0.f;
        auto max8 = [&](const float (&x)[8][4]) {
            e0 = e1 = 0.f;
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                e0 = max_abs(max_abs(e0, x[nt][0]), x[nt][1]);
                e1 = max_abs(max_abs(e1, x[nt][2]), x[nt][3]);
            }
            e0 = quad_max(e0), e1 = quad_max(e1);
        };
        auto split8 = [&](const float (&x)[8][4], int kk, Pow2 q0, Pow2 q1, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                h2_split(row_a(x[2 * kk + u]), q0.to, hi[2 * u], lo[2 * u]);
                h2_split(row_b(x[2 * kk + u]), q1.to, hi[2 * u + 1], lo[2 * u + 1]);
            }
        };
        // E = R + F z on the own tiles
        float x[2 * OWN][4];
        clear(x);
        max8(z);
        {
            const Pow2 q0 = pow2_for(e0), q1 = pow2_for(e1);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t hi[4], lo[4];
                split8(z, kk, q0, q1, hi, lo);
                // F is strictly lower
                three_products<OWN>(
                    x, hi, lo, [&](int i) { return sh.tile(kk) <= sh.tile(i); },
                    [&](uint32_t(&b)[4], int i, int part) {
                        ldsm4(b, addr_b<128>(sF + part * kTile, lane, 16 * sh.tile(i), 16 * sh.tile(kk)));
                    });
            }
#pragma unroll
            for (int i = 0; i < 2 * OWN; ++i) {
                const float2 f = fac2(fac, kFacF, sh.tile(i >> 1), i & 1, tq);
                set_rows(r[i], fma2(mul2(f, both(q0.from)), row_a(x[i]), row_a(r[i])),
                         fma2(mul2(f, both(q1.from)), row_b(x[i]), row_b(r[i])));
            }
        }
        if (SP > 1) {
            sh.put(3, pair(r, 0), pair(r, 1));
            sh.sync();
            sh.template get<false>(3, pair(r, 2), pair(r, 3));
        }
        if (GRAD) {  // r is E
#pragma unroll
            for (int i = 0; i < OWN; ++i) {
                const Pow2 q0 = tile_scale(r, i, 0), q1 = tile_scale(r, i, 2);
                uint32_t hi[4], lo[4];
                split8(r, i, q0, q1, hi, lo);
                keep_parts(kept.E, bh * nchunk + c, kC * DV * 2, (col0 / 16) * 4 + sh.tile(i), lane, hi, lo);
                if (tq == 0) {
                    float* se = kept.sE + ((bh * nchunk + c) * 4 + sh.tile(i)) * DV + col0;
                    se[g] = q0.from, se[g + 8] = q1.from;
                }
            }
        }
        if (GRAD && READS) {  // dO.(e^G scale S0^T q)
            cp_wait<1>();
            __syncwarp();
            float dots[OWN / 2][8];
#pragma unroll
            for (int i = 0; i < OWN; ++i) {
                uint32_t w[4];
                ldsm4t(w, addr_ct<32>(so, lane, 16 * sh.tile(i), 0));
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int nt = 2 * i + u;
                    dots[nt >> 2][2 * (nt & 3)] = o[nt][0] * lo_f(w[2 * u]) + o[nt][2] * lo_f(w[2 * u + 1]);
                    dots[nt >> 2][2 * (nt & 3) + 1] = o[nt][1] * hi_f(w[2 * u]) + o[nt][3] * hi_f(w[2 * u + 1]);
                }
            }
#pragma unroll
            for (int part = 0; part < OWN / 2; ++part)
                sh.store_sums(kept.hq + (bh * (DV / 16) + col0 / 16) * N, dots[part], part, (int64_t)c * kC, N);
        }
        // O = inter + (P beta) E: with beta in P, a token that writes nothing does not
        // set the scale of its row.  One fp16 part of each is enough (2^-12 of a term,
        // under the output's own rounding)
        if (READS && !GRAD) {
            max8(r);
            const Pow2 q0 = pow2_for(e0), q1 = pow2_for(e1);
            clear(x);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t hi[4], lo[4], b[4];
                split8(r, kk, q0, q1, hi, lo);
#pragma unroll
                for (int i = 0; i < OWN; ++i) {
                    if (sh.tile(kk) <= sh.tile(i)) {
                        ldsm4(b, addr_b<128>(sP, lane, 16 * sh.tile(i), 16 * sh.tile(kk)));
                        mma(x[2 * i], hi, b[0], b[1]);
                        mma(x[2 * i + 1], hi, b[2], b[3]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < OWN; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int nt = 2 * i + u;
                    const float2 fp = fac2(fac, kFacP, sh.tile(i), u, tq);
                    set_rows(o[nt], fma2(mul2(fp, both(q0.from)), row_a(x[nt]), row_a(o[nt])),
                             fma2(mul2(fp, both(q1.from)), row_b(x[nt]), row_b(o[nt])));
                    w[2 * u] = sm100::pack_bf16x2(o[nt][0], o[nt][1]);
                    w[2 * u + 1] = sm100::pack_bf16x2(o[nt][2], o[nt][3]);
                }
                stsm4t(addr_ct<32>(so, lane, 16 * sh.tile(i), 0), w);
            }
        }
        // W U, U = beta E: the state update's operand, and its largest
        float w0 = 0.f, w1 = 0.f;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            const float2 w = fac2(fac, kFacW, sh.tile(nt >> 1), nt & 1, tq);
            scale_cols(r[nt], fac2(fac, kFacB, sh.tile(nt >> 1), nt & 1, tq));
            scale_cols(r[nt], w);
            w0 = max_abs(max_abs(w0, r[nt][0]), r[nt][1]);
            w1 = max_abs(max_abs(w1, r[nt][2]), r[nt][3]);
        }
        // S1 = e^{G_C} S0 + (W U)^T K16 on accumulators scaled with the operand: both
        // under one power of two, so neither overflows nor loses bits the other does
        // not drown
        const float gend = fac[kFacEnd * kC];
        const Pow2 u0 = pow2_for(fmaxf(quad_max(w0), m0 * gend * 0.00390625f));
        const Pow2 u1 = pow2_for(fmaxf(quad_max(w1), m1 * gend * 0.00390625f));
        const float g0 = gend * u0.to, g1 = gend * u1.to;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            scale_rows(s[nt], g0, g1);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int nt = 2 * kk + u;
                h2_split(row_a(r[nt]), u0.to, hi[2 * u], lo[2 * u]);
                h2_split(row_b(r[nt]), u1.to, hi[2 * u + 1], lo[2 * u + 1]);
            }
            rows_update<RB, KK>(s, hi, lo, sK, lane, 16 * sh.tile(kk), d0);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            scale_rows(s[nt], u0.from, u1.from);
        if (!GRAD && READS) {
            __syncwarp();
            const int64_t t0 = (int64_t)c * kC;
#pragma unroll
            for (int i = 0; i < OWN; ++i) {
                const int t = 16 * sh.tile(i) + (lane >> 1), p = lane & 1;
                if (t0 + t < N)
                    *reinterpret_cast<uint4*>(out + (bh * N + t0 + t) * DV + col0 + p * 8) =
                        *reinterpret_cast<const uint4*>(smem + (so - base) + tile_off<32>(t, p));
            }
        }
        const bool refill = ring.last(step);
        if (!ring.ok)
            break;
        if (refill && step + SM::stages < len)
            load_stage(step + SM::stages);
        // here and not at the chunk's start: what is issued there (copies, addresses)
        // then shares a stretch without branches with the first products
        if (step + 1 < len)
            ring.wait(step + 1);
    }
    cp_wait<0>();
    if (!ring.ok && lane == 0) {  // a copy did not arrive in time: the results are void
        ring.drain();
        set_status(status, LA_ERR_TIMEOUT);
    }
    float* end = nullptr;
    int ld = DV;
    if (seg.carry) {
        end = col0 < DV ? seg.B + run * D * DV : seg.M + run * D * D - DV;  // unit column c is M's c - DV
        ld = col0 < DV ? DV : D;
    } else if (S_out && lo + len == nchunk) {
        end = S_out + bh * D * DV;
    }
    if (end) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                end[(int64_t)(d0 + 8 * nt + 2 * tq + (e & 1)) * ld + col0 + g + (e >> 1) * 8] = s[nt][e];
    }
}

// The states before the segments of a sequence from their ends, S_{i+1} = M_i S_i + B_i
// from S_0, or (REV) the gradients of the states after them, dS_{i-1} = M_i^T dS_i + C_i
// from that of the last.  The steps follow one another, so a step is cut as fine as it
// goes: a CTA owns 8 columns, a warp D / 8 rows of M, a lane D / 32 columns of M; lane
// 4 g + t of a warp holds the state's column g in rows t, t + 4, .. of the warp's.  The
// next M and B come into registers while a step runs, each row as the one before it is
// used up.
constexpr int kJoinCols = 8;

template <int D, bool REV>
__global__ void __launch_bounds__(256)
    k_delta_join(const float* __restrict__ S0, const float* __restrict__ B, const float* __restrict__ M,
                 float* __restrict__ start, int count, int mcount, int DV)
{
    constexpr int V = D / 32, RW = D / 8, LS = D + 4;  // M's columns per lane, rows per warp
    // the state by columns, twice; REV: the warps' parts of the next, and the state's rows
    __shared__ __align__(16) float sm[REV ? 8 * 8 * LS + 8 * D : 2 * 8 * LS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int64_t bh = blockIdx.x;
    const int c = blockIdx.y * kJoinCols + g, row0 = warp * RW + t;
    float x[RW / 4], next[RW / 4], m[RW][V];
    // step i leads out of segment `of`; M and B have mcount segments, C count - 1 (not
    // the first)
    auto matrix = [&](int i, int r) {
        const int of = REV ? count - 1 - i : i;
        const float* p = M + ((bh * mcount + of) * D + warp * RW + r) * D + V * lane;
        if constexpr (V == 4) {
            const float4 y = *reinterpret_cast<const float4*>(p);
            m[r][0] = y.x, m[r][1] = y.y, m[r][2] = y.z, m[r][3] = y.w;
        } else if constexpr (V == 2) {
            const float2 y = *reinterpret_cast<const float2*>(p);
            m[r][0] = y.x, m[r][1] = y.y;
        } else {
            m[r][0] = *p;
        }
    };
    auto constant = [&](int i) {
        const int of = REV ? count - 1 - i : i;
        const float* b = B + (REV ? bh * (count - 1) + of - 1 : bh * mcount + of) * D * DV;
#pragma unroll
        for (int r = 0; r < RW / 4; ++r)
            next[r] = b[(row0 + 4 * r) * DV + c];
    };
#pragma unroll
    for (int r = 0; r < RW / 4; ++r)
        x[r] = S0 ? S0[(bh * D + row0 + 4 * r) * DV + c] : 0.f;
    if (count > 1) {
#pragma unroll
        for (int r = 0; r < RW; ++r)
            matrix(0, r);
        constant(0);
    }
    for (int i = 0;; ++i) {
        const int of = REV ? count - 1 - i : i;
        const bool more = i + 2 < count;
#pragma unroll
        for (int r = 0; r < RW / 4; ++r)
            start[((bh * count + of) * D + row0 + 4 * r) * DV + c] = x[r];
        if (i + 1 == count)
            return;
        if constexpr (REV) {
            float* mine = sm + 64 * LS + warp * RW * 8;  // [row][column]
            __syncwarp();
#pragma unroll
            for (int r = 0; r < RW / 4; ++r)
                mine[(t + 4 * r) * 8 + g] = x[r];
            __syncwarp();
            float y[8][V] = {};
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                const float4 a = *reinterpret_cast<const float4*>(mine + r * 8);
                const float4 b = *reinterpret_cast<const float4*>(mine + r * 8 + 4);
                const float s[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        y[j][v] = fmaf(m[r][v], s[j], y[j][v]);
                if (more)
                    matrix(i + 1, r);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    sm[(warp * 8 + j) * LS + V * lane + v] = y[j][v];
            __syncthreads();
#pragma unroll
            for (int r = 0; r < RW / 4; ++r) {
                x[r] = next[r];
#pragma unroll
                for (int w = 0; w < 8; ++w)
                    x[r] += sm[(w * 8 + g) * LS + row0 + 4 * r];
            }
            __syncthreads();  // the parts are read
        } else {
            float* s = sm + (i & 1) * 8 * LS;  // [column][row]
#pragma unroll
            for (int r = 0; r < RW / 4; ++r)
                s[g * LS + row0 + 4 * r] = x[r];
            __syncthreads();
            float k[8][V];
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    k[j][v] = s[j * LS + V * lane + v];
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    y[j] = m[r][0] * k[j][0];
#pragma unroll
                    for (int v = 1; v < V; ++v)
                        y[j] = fmaf(m[r][v], k[j][v], y[j]);
                }
                if (more)
                    matrix(i + 1, r);
                float z = delta::sum8(y, lane);
                z += __shfl_xor_sync(0xffffffffu, z, 2);
                z += __shfl_xor_sync(0xffffffffu, z, 1);
                if ((r & 3) == t)
                    x[r / 4] = z + next[r / 4];
            }
        }
        if (more)
            constant(i + 1);
    }
}

// -------------------------------------------------------------- k_delta_rev --
// The chunks from the last to the first, dS^T [16 x d] of a slice's columns in
// registers (dS1 entering a chunk, dS0 leaving it), shared between warps as in
// k_delta_chain:
//
//   dU = P^T dO + diag(e^{G_C - G}) K dS1,  z = beta dU
//   Y  = dU + F^T z,  dV = beta Y          ((I + diag(beta) A)^{-T} = I + F^T beta)
//   dS0 = e^{G_C} dS1 + (diag(e^G) Q)^T dO - (diag(e^G) K)^T dV
//
// and the dot products that need both directions' fp32 values: Y.E, and for the gates
// k.(S0 dV), k.(dS1 U) and <S0, dS1>.
//
// Over segments as in k_delta_chain: dS0 is affine in dS1, and its matrix over a
// segment is the transpose of the M that the states' run gave.  ENDS: a run from
// dS = 0 that leaves each segment's constant part in seg.B and nothing else.
//
// Measured: 535 us at B4 H8 N8192 d=128 (8100 cycles per chunk; 1.9 times the
// forward chain's instructions), 340 us at B8 H32 N1037; bound like the chain.
template <int D, int SP>
struct RevSmem {
    static constexpr int stages = 2;
    static constexpr int stage = 2 * row_image<D>() + blob_bytes<true>();
    static constexpr int slice0 = stages * stage;
    // per slice: dO twice, dV on its way out, E hi and lo, three exchange buffers for
    // each of two warps
    static constexpr int dO = 0, v = 2 * kC * 32, e = v + kC * 32, x = e + 2 * kC * 32,
                         per_slice = x + (SP > 1 ? SP * 3 * kXch : 0);
    static int bytes(int W) { return slice0 + W * per_slice + 128; }
};

template <int D, int SP, bool GATED, bool ENDS>
__global__ void __launch_bounds__(256, 1)
    k_delta_rev(const unsigned char* __restrict__ rows, const unsigned char* __restrict__ blobs,
                const __nv_bfloat16* __restrict__ dout,
                const float* __restrict__ dS_out, __nv_bfloat16* __restrict__ dv,
                float* __restrict__ dS0, int64_t N, int nchunk, int H, int Hk, int DV, Kept kept,
                Segments seg, int* status)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    using SM = RevSmem<D, SP>;
    constexpr int RB = 2 * D, kBlob = blob_bytes<true>();
    constexpr int NT = D / 8 / SP, KK = NT / 2, OWN = Share<SP>::own;
    const int tid = threadIdx.x, lane = tid & 31, W = blockDim.x / (32 * SP);
    const int g = lane >> 2, tq = lane & 3;
    Share<SP> sh;
    sh.slice = (tid >> 5) / SP, sh.half = (tid >> 5) % SP, sh.lane = lane;
    const int slices = DV / (16 * W);
    const int64_t run = blockIdx.x / slices + seg.skip;  // head and segment
    const int64_t bh = run / seg.count;
    const int lo = ((int)(run % seg.count) + seg.first) * seg.len, len = min(seg.len, nchunk - lo);
    const int col0 = (blockIdx.x % slices) * 16 * W + 16 * sh.slice, slice = col0 / 16;
    const int64_t kh = bh / H * Hk + (bh % H) / (H / Hk);
    const uint32_t base = smem_addr(smem);
    const int mine = SM::slice0 + sh.slice * SM::per_slice;
    sh.mine = smem + mine + SM::x + sh.half * 3 * kXch;
    sh.other = smem + mine + SM::x + (SP - 1 - sh.half) * 3 * kXch;
    const uint32_t sdo = base + mine + SM::dO, sv = base + mine + SM::v;
    Ring<SM::stages, (SP > 1)> ring(smem + SM::slice0 + W * SM::per_slice, blockDim.x >> 5);
    const unsigned char* row_src = rows + kh * nchunk * (int64_t)(2 * row_image<D>());
    const unsigned char* blob_src = blobs + bh * nchunk * (int64_t)kBlob;
    const int d0 = sh.half * (D / SP);

    auto load_stage = [&](int it) {
        const int64_t c = lo + len - 1 - it;
        const uint32_t dst = base + (it % SM::stages) * SM::stage;
        uint64_t* bar = ring.full + it % SM::stages;
        sm100::mbar_arrive_expect_tx(bar, SM::stage);
        delta::bulk_load(dst, row_src + c * (2 * row_image<D>()), 2 * row_image<D>(), bar);
        delta::bulk_load(dst + 2 * row_image<D>(), blob_src + c * kBlob, kBlob, bar);
    };
    auto load_cols = [&](uint32_t dst, const __nv_bfloat16* src, int c) {
        const int64_t t0 = (int64_t)c * kC;  // c = -1: nothing
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int t = 16 * sh.tile(i) + (lane >> 1), p = lane & 1;
            const bool live = t0 >= 0 && t0 + t < N;
            cp16(dst + tile_off<32>(t, p), src + (bh * N + (live ? t0 + t : 0)) * DV + col0 + p * 8, live);
        }
    };
    auto load_E = [&](int c) {  // the own token tiles' blocks
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int i = 0; i < OWN; ++i)
                cp16(base + mine + SM::e + part * kC * 32 + sh.tile(i) * 512 + lane * 16,
                     kept.E + (2 * (bh * nchunk + c) + part) * (int64_t)(kC * DV * 2) +
                         (slice * 4 + sh.tile(i)) * 512 + lane * 16,
                     true);
    };
    float ds[NT][4];  // dS^T[col0 + g, + 8][d0 + 8 nt + 2 tq, + 1]
    // <S0, dS> of chunk c over the warp's part -> kept.cd.  S0 is read where it lies
    // (128 bytes per load; asked into L2 a chunk ahead): staging it took the shared memory
    // of half of the slices
    auto state_at = [&](int64_t c, int part) {
        return kept.S + (2 * (bh * nchunk + c) + part) * (int64_t)(D * DV * 2) + (slice * (D / 16) + d0 / 16) * 512;
    };
    auto ask_state = [&](int64_t c) {
#pragma unroll
        for (int i = lane; i < 2 * KK * 4; i += 32)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(state_at(c, i / (KK * 4)) + i % (KK * 4) * 128));
    };
    auto dot_state = [&](int64_t c, float sc0, float sc1, bool keep) {
        const uint32_t* part0 = reinterpret_cast<const uint32_t*>(state_at(c, 0)) + lane;
        const uint4* part1 = reinterpret_cast<const uint4*>(state_at(c, 1)) + lane;
        float a0 = 0.f, a1 = 0.f;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const uint4 z = __ldg(part1 + kk * 32);
            const uint32_t y[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // register i: row g + 8 (i & 1), tile 2 kk + (i >> 1)
                const uint32_t x = __ldg(part0 + (kk * 4 + i) * 32);
                const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&x));
                const float2 l = __half22float2(*reinterpret_cast<const __half2*>(&y[i]));
                const float* d = ds[2 * kk + (i >> 1)] + 2 * (i & 1);
                float& a = i & 1 ? a1 : a0;
                a = fmaf(h.x + l.x, d[0], fmaf(h.y + l.y, d[1], a));
            }
        }
        float x = a0 * sc0 + a1 * sc1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0 && keep) {
            float* cd = kept.cd + (bh * (DV / 16) + slice) * 2 * nchunk + c;
            cd[sh.half * nchunk] = x;
            if (SP == 1)
                cd[nchunk] = 0.f;
        }
    };
    // E and S0^T K16 of the own token tiles, a chunk ahead
    auto ask_tokens = [&](int64_t c) {
#pragma unroll
        for (int i = lane; i < OWN * 16; i += 32) {
            const int tile = sh.tile(i / 16), line = i % 16;  // 4 + 4 lines of E's parts, 8 of KS
            const unsigned char* e = kept.E + (2 * (bh * nchunk + c) + (line >> 2 & 1)) * (int64_t)(kC * DV * 2) +
                                     (slice * 4 + tile) * 512 + (line & 3) * 128;
            const unsigned char* ks = reinterpret_cast<const unsigned char*>(
                kept.KS + (((bh * nchunk + c) * (DV / 16) + slice) * 8 + 2 * tile) * 32) + (line & 7) * 128;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(line < 8 ? e : ks));
        }
    };
    // the scales of the kept state and of E; E's a chunk ahead where a warp is alone on its
    // sub-partition
    float sc[2] = {}, se[OWN][2] = {};
    auto read_S_scales = [&](int64_t c) {
        const float* at = kept.sS + ((bh * nchunk + c) * 2 + sh.half) * DV + col0;
        sc[0] = __ldg(at + g), sc[1] = __ldg(at + g + 8);
    };
    auto read_E_scales = [&](int64_t c, float (&x)[OWN][2]) {
        if (ENDS)
            return;
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const float* at = kept.sE + ((bh * nchunk + c) * 4 + sh.tile(i)) * DV + col0;
            x[i][0] = __ldg(at + g), x[i][1] = __ldg(at + g + 8);
        }
    };
    // S0^T K16 of the own C tile nt, as k_delta_chain left it
    auto read_KS = [&](int64_t c, int nt) {
        return __ldg(kept.KS + (((bh * nchunk + c) * (DV / 16) + slice) * 8 + 2 * sh.tile(nt >> 1) + (nt & 1)) * 32 + lane);
    };

    if (tid == 0)
        for (int i = 0; i < SM::stages && i < len; ++i)
            load_stage(i);
    load_cols(sdo + ((lo + len - 1) & 1) * kC * 32, dout, lo + len - 1);
    cp_commit();
    const float* end = ENDS ? nullptr : seg.start ? seg.start + run * D * DV : dS_out ? dS_out + bh * D * DV : nullptr;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            ds[nt][e] = end ? end[(d0 + 8 * nt + 2 * tq + (e & 1)) * DV + col0 + g + (e >> 1) * 8] : 0.f;
    if (SP > 1)
        read_E_scales(lo + len - 1, se);
    if (GATED) {
        read_S_scales(lo + len - 1);
        dot_state(lo + len - 1, sc[0], sc[1], true);
    }
    cp_wait<0>();
    sh.sync();
    ring.wait(0);
    for (int it = 0; it < len && ring.go_on(); ++it) {
        const int c = lo + len - 1 - it;
        const uint32_t st = base + (it % SM::stages) * SM::stage;
        const uint32_t sK = st, sQ = st + row_image<D>(), sF = st + 2 * row_image<D>(), sP = sF + 2 * kTile;
        const float* fac = reinterpret_cast<const float*>(smem + (it % SM::stages) * SM::stage +
                                                          2 * row_image<D>() + fac_at<true>());
        const uint32_t tdo = sdo + (c & 1) * kC * 32;
        // this chunk's E and S, wanted from the middle on; the next dO, each warp its
        // token tiles, which both await before they meet at the chunk's end
        if (!ENDS)
            load_E(c);
        cp_commit();
        load_cols(sdo + ((c - 1) & 1) * kC * 32, dout, c - 1);
        cp_commit();
        float se_next[OWN][2] = {};
        if (SP == 1)
            read_E_scales(c, se);
        const int before = max(c - 1, lo);  // the last chunk asks for its own once more
        if (GATED) {
            ask_state(before);
            read_S_scales(before);
            if (SP > 1)
                ask_tokens(before);
        }
        if (SP > 1)
            read_E_scales(before, se_next);
        auto pair = [](float (&x)[8][4], int i) -> float(&)[2][4] {
            return *reinterpret_cast<float(*)[2][4]>(x + 2 * i);
        };

        // dS1^T K^T over this warp's rows; dS1 is kept for k_delta_dqk
        float m0 = 0.f, m1 = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m0 = max_abs(max_abs(m0, ds[nt][0]), ds[nt][1]);
            m1 = max_abs(max_abs(m1, ds[nt][2]), ds[nt][3]);
        }
        m0 = quad_max(m0), m1 = quad_max(m1);
        const Pow2 p0 = pow2_for(m0), p1 = pow2_for(m1);
        float u[8][4], x[2 * OWN][4];  // u in local token order
        clear(u);
        clear(x);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            uint32_t hi[4], lo[4], b[4][4];
            h2_split(row_a(ds[2 * kk]), p0.to, hi[0], lo[0]);
            h2_split(row_b(ds[2 * kk]), p1.to, hi[1], lo[1]);
            h2_split(row_a(ds[2 * kk + 1]), p0.to, hi[2], lo[2]);
            h2_split(row_b(ds[2 * kk + 1]), p1.to, hi[3], lo[3]);
            if (!ENDS)
                keep_part(kept.dS, bh * nchunk + c, D * DV * 2, slice * (D / 16) + d0 / 16 + kk, lane, hi);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ldsm4(b[j], addr_b<RB>(sK, lane, 16 * sh.tile(j), d0 + 16 * kk));
            mma_tiles<4>(u, hi, b);
            mma_tiles<4>(u, lo, b);
        }
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
            scale_rows(u[nt], p0.from, p1.from);
        if (SP > 1)
            sh.put(0, pair(u, 2), pair(u, 3));
        // dO^T P on the own tiles: the rows of P carry powers of two, which go to dO
        // (exact)
        float q_0 = 0.f, q_1 = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
            ldsm4t(w, addr_ct<32>(tdo, lane, 16 * j, 0));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 fp = fac2(fac, kFacP, j, h, tq);
                const float2 a = mul2(fp, bf2(w[2 * h])), b = mul2(fp, bf2(w[2 * h + 1]));
                q_0 = max_abs(max_abs(q_0, a.x), a.y);
                q_1 = max_abs(max_abs(q_1, b.x), b.y);
            }
        }
        const Pow2 q0 = pow2_for(quad_max(q_0)), q1 = pow2_for(quad_max(q_1));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            uint32_t w[4], a[4], b[4];
            ldsm4t(w, addr_ct<32>(tdo, lane, 16 * kk, 0));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 fp = fac2(fac, kFacP, kk, h, tq);
                const float2 x0 = mul2(mul2(fp, bf2(w[2 * h])), both(q0.to));
                const float2 x1 = mul2(mul2(fp, bf2(w[2 * h + 1])), both(q1.to));
                a[2 * h] = h2(x0.x, x0.y), a[2 * h + 1] = h2(x1.x, x1.y);
            }
#pragma unroll
            for (int i = 0; i < OWN; ++i) {
                if (sh.tile(i) <= kk) {  // P_ij, j <= i
                    ldsm4t(b, addr_bt<128>(sP, lane, 16 * kk, 16 * sh.tile(i)));
                    mma(x[2 * i], a, b[0], b[1]);
                    mma(x[2 * i + 1], a, b[2], b[3]);
                    ldsm4t(b, addr_bt<128>(sP + kTile, lane, 16 * kk, 16 * sh.tile(i)));
                    mma(x[2 * i], a, b[0], b[1]);
                    mma(x[2 * i + 1], a, b[2], b[3]);
                }
            }
        }
        if (SP > 1) {
            sh.sync();
            sh.template get<true>(0, pair(u, 0), pair(u, 1));
        }
        // E of the own C tile nt
        auto read_E = [&](int nt, float (&y)[4]) {
            const uint32_t* at = reinterpret_cast<const uint32_t*>(smem + mine + SM::e) +
                                 (sh.tile(nt >> 1) * 4 + 2 * (nt & 1)) * 32 + lane;
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(at));
            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(at + 32));
            const float2 l = __half22float2(*reinterpret_cast<const __half2*>(at + kC * 8));
            const float2 m = __half22float2(*reinterpret_cast<const __half2*>(at + kC * 8 + 32));
            const float s0 = se[nt >> 1][0], s1 = se[nt >> 1][1];
            y[0] = s0 * (a.x + l.x), y[1] = s0 * (a.y + l.y), y[2] = s1 * (b.x + m.x), y[3] = s1 * (b.y + m.y);
        };
        // dU.  Its part from the state is dotted with U for the gates: two warps per slice
        // have the registers to keep it until E is read for the other dots (534 against 553
        // us), one does it at once (324 against 332 us)
        constexpr bool L_NOW = GATED && !ENDS && SP == 1, L_LATE = GATED && !ENDS && SP > 1;
        if (L_NOW) {
            cp_wait<1>();  // E
            __syncwarp();
        }
        float lsum[OWN / 2][8], us[L_LATE ? 2 * OWN : 1][4];
        auto dot_U = [&](int nt, const float (&x)[4], const float (&y)[4]) {
            const float2 be = fac2(fac, kFacB, sh.tile(nt >> 1), nt & 1, tq);
            lsum[nt >> 2][2 * (nt & 3)] = be.x * (x[0] * y[0] + x[2] * y[2]);
            lsum[nt >> 2][2 * (nt & 3) + 1] = be.y * (x[1] * y[1] + x[3] * y[3]);
        };
#pragma unroll
        for (int i = 0; i < 2 * OWN; ++i) {
            scale_cols(u[i], fac2(fac, kFacW, sh.tile(i >> 1), i & 1, tq));
            if (L_NOW) {
                float y[4];
                read_E(i, y);
                dot_U(i, u[i], y);
            }
            if (L_LATE)
                set_rows(us[i], row_a(u[i]), row_b(u[i]));
            scale_cols(x[i], fac2(fac, kFacPk, sh.tile(i >> 1), i & 1, tq));
            set_rows(u[i], fma2(row_a(x[i]), both(q0.from), row_a(u[i])), fma2(row_b(x[i]), both(q1.from), row_b(u[i])));
        }
        if (SP > 1) {
            sh.put(1, pair(u, 0), pair(u, 1));
            sh.sync();
            sh.template get<false>(1, pair(u, 2), pair(u, 3));
        }
        // F^T z on the own tiles: F's rows carry their factors, which go to z = beta dU
        float z0 = 0.f, z1 = 0.f, z[8][4];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            const float2 be = fac2(fac, kFacBF, sh.tile(nt >> 1), nt & 1, tq);
            set_rows(z[nt], mul2(be, row_a(u[nt])), mul2(be, row_b(u[nt])));
            z0 = max_abs(max_abs(z0, z[nt][0]), z[nt][1]);
            z1 = max_abs(max_abs(z1, z[nt][2]), z[nt][3]);
        }
        const Pow2 y0 = pow2_for(quad_max(z0)), y1 = pow2_for(quad_max(z1));
        clear(x);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                h2_split(row_a(z[2 * kk + h]), y0.to, hi[2 * h], lo[2 * h]);
                h2_split(row_b(z[2 * kk + h]), y1.to, hi[2 * h + 1], lo[2 * h + 1]);
            }
            three_products<OWN>(
                x, hi, lo, [&](int i) { return sh.tile(i) <= sh.tile(kk); },
                [&](uint32_t(&b)[4], int i, int part) {
                    ldsm4t(b, addr_bt<128>(sF + part * kTile, lane, 16 * sh.tile(kk), 16 * sh.tile(i)));
                });
        }
        auto back = [&](int nt, Pow2 y) { return mul2(fac2(fac, kFacC, sh.tile(nt >> 1), nt & 1, tq), both(y.from)); };
        if (ENDS) {  // dV alone
#pragma unroll
            for (int nt = 0; nt < 2 * OWN; ++nt) {
                set_rows(u[nt], fma2(back(nt, y0), row_a(x[nt]), row_a(u[nt])),
                         fma2(back(nt, y1), row_b(x[nt]), row_b(u[nt])));
                scale_cols(u[nt], fac2(fac, kFacB, sh.tile(nt >> 1), nt & 1, tq));
            }
        } else {
            if (!L_NOW) {
                cp_wait<1>();  // E
                __syncwarp();
            }
            // Y, the dots, dV on the own tiles
            float bsum[OWN / 2][8], hsum[OWN / 2][8];
#pragma unroll
            for (int nt = 0; nt < 2 * OWN; ++nt) {
                const float2 be = fac2(fac, kFacB, sh.tile(nt >> 1), nt & 1, tq);
                set_rows(u[nt], fma2(back(nt, y0), row_a(x[nt]), row_a(u[nt])),
                         fma2(back(nt, y1), row_b(x[nt]), row_b(u[nt])));
                const int part = nt >> 2, k = 2 * (nt & 3);
                float y[4];
                read_E(nt, y);
                if (L_LATE)
                    dot_U(nt, us[nt], y);
                bsum[part][k] = u[nt][0] * y[0] + u[nt][2] * y[2];
                bsum[part][k + 1] = u[nt][1] * y[1] + u[nt][3] * y[3];
                scale_cols(u[nt], be);
                if (GATED) {
                    const float2 fa = fac2(fac, kFacA, sh.tile(nt >> 1), nt & 1, tq);
                    const float4 a = read_KS(c, nt);
                    hsum[part][k] = -fa.x * (u[nt][0] * a.x + u[nt][2] * a.z);
                    hsum[part][k + 1] = -fa.y * (u[nt][1] * a.y + u[nt][3] * a.w);
                }
            }
#pragma unroll
            for (int part = 0; part < OWN / 2; ++part) {
                sh.store_sums(kept.bb + (bh * (DV / 16) + slice) * N, bsum[part], part, (int64_t)c * kC, N);
                if (GATED) {
                    sh.store_sums(kept.hk + (bh * (DV / 16) + slice) * N, hsum[part], part, (int64_t)c * kC, N);
                    sh.store_sums(kept.ll + (bh * (DV / 16) + slice) * N, lsum[part], part, (int64_t)c * kC, N);
                }
            }
        }
        if (SP > 1)
            sh.put(2, pair(u, 0), pair(u, 1));
        sh.sync();
        if (SP > 1)
            sh.template get<false>(2, pair(u, 2), pair(u, 3));
        if (!ENDS) {
            // dV leaves as bf16 and is kept, times p, as scaled fp16 (both parts for the gates)
#pragma unroll
            for (int i = 0; i < OWN; ++i) {
                uint32_t w[4], a[4], l[4];
                float y[8][4];  // the first two C tiles: p dV
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 p = fac2(fac, kFacPk, sh.tile(i), h, tq);
                    set_rows(y[h], mul2(p, row_a(u[2 * i + h])), mul2(p, row_b(u[2 * i + h])));
                }
                const Pow2 s0 = tile_scale(y, 0, 0), s1 = tile_scale(y, 0, 2);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int nt = 2 * i + h;
                    w[2 * h] = sm100::pack_bf16x2(u[nt][0], u[nt][1]);
                    w[2 * h + 1] = sm100::pack_bf16x2(u[nt][2], u[nt][3]);
                    h2_split(row_a(y[h]), s0.to, a[2 * h], l[2 * h]);
                    h2_split(row_b(y[h]), s1.to, a[2 * h + 1], l[2 * h + 1]);
                }
                stsm4t(addr_ct<32>(sv, lane, 16 * sh.tile(i), 0), w);
                keep_part(kept.dV, bh * nchunk + c, kC * DV * 2, slice * 4 + sh.tile(i), lane, a);
                if (GATED)
                    keep_part(kept.dVl, bh * nchunk + c, kC * DV * 2, slice * 4 + sh.tile(i), lane, l);
                if (tq == 0) {
                    float* sw = kept.sV + ((bh * nchunk + c) * 4 + sh.tile(i)) * DV + col0;
                    sw[g] = s0.from, sw[g + 8] = s1.from;
                }
            }
            if (tq == 0) {
                float* sd = kept.sD + ((bh * nchunk + c) * 2 + sh.half) * DV + col0;
                sd[g] = p0.from, sd[g + 8] = p1.from;
                if (SP == 1)
                    sd[DV + g] = p0.from, sd[DV + g + 8] = p1.from;
            }
            __syncwarp();
            {
                const int64_t t0 = (int64_t)c * kC;
#pragma unroll
                for (int i = 0; i < OWN; ++i) {
                    const int t = 16 * sh.tile(i) + (lane >> 1), p = lane & 1;
                    if (t0 + t < N)
                        *reinterpret_cast<uint4*>(dv + (bh * N + t0 + t) * DV + col0 + p * 8) =
                            *reinterpret_cast<const uint4*>(smem + mine + SM::v + tile_off<32>(t, p));
                }
            }
        }
        // dS0 on this warp's rows: both products on accumulators under one power of two
        float w0 = 0.f, w1 = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
            ldsm4t(w, addr_ct<32>(tdo, lane, 16 * sh.tile(j), 0));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int nt = 2 * j + h;
                const float2 fo = fac2(fac, kFacO, sh.tile(j), h, tq), fa = fac2(fac, kFacA, sh.tile(j), h, tq);
                const float2 a = mul2(fo, bf2(w[2 * h])), b = mul2(fo, bf2(w[2 * h + 1]));
                w0 = max_abs(max_abs(w0, a.x), a.y);
                w1 = max_abs(max_abs(w1, b.x), b.y);
                scale_cols(u[nt], make_float2(-fa.x, -fa.y));
                w0 = max_abs(max_abs(w0, u[nt][0]), u[nt][1]);
                w1 = max_abs(max_abs(w1, u[nt][2]), u[nt][3]);
            }
        }
        const float gend = fac[kFacEnd * kC];
        const Pow2 r0 = pow2_for(fmaxf(quad_max(w0), m0 * gend * 0.00390625f));
        const Pow2 r1 = pow2_for(fmaxf(quad_max(w1), m1 * gend * 0.00390625f));
        const float g0 = gend * r0.to, g1 = gend * r1.to;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            scale_rows(ds[nt], g0, g1);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            uint32_t w[4], hi[4], lo[4];
            ldsm4t(w, addr_ct<32>(tdo, lane, 16 * sh.tile(kk), 0));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 fo = fac2(fac, kFacO, sh.tile(kk), h, tq);
                h2_split(mul2(fo, bf2(w[2 * h])), r0.to, hi[2 * h], lo[2 * h]);
                h2_split(mul2(fo, bf2(w[2 * h + 1])), r1.to, hi[2 * h + 1], lo[2 * h + 1]);
            }
            rows_update<RB, KK>(ds, hi, lo, sQ, lane, 16 * sh.tile(kk), d0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int nt = 2 * kk + h;
                h2_split(row_a(u[nt]), r0.to, hi[2 * h], lo[2 * h]);
                h2_split(row_b(u[nt]), r1.to, hi[2 * h + 1], lo[2 * h + 1]);
            }
            rows_update<RB, KK>(ds, hi, lo, sK, lane, 16 * sh.tile(kk), d0);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            scale_rows(ds[nt], r0.from, r1.from);
        if (GATED)  // no branch at the last chunk: the loads can go up among the products
            dot_state(before, sc[0], sc[1], it + 1 < len);
        if (SP > 1) {
#pragma unroll
            for (int o = 0; o < OWN; ++o)
                se[o][0] = se_next[o][0], se[o][1] = se_next[o][1];
        }
        cp_wait<0>();
        sh.sync();
        const bool refill = ring.last(it);
        if (!ring.ok)
            break;
        if (refill && it + SM::stages < len)
            load_stage(it + SM::stages);
        if (it + 1 < len)
            ring.wait(it + 1);
    }
    cp_wait<0>();
    if (!ring.ok && lane == 0) {  // a copy did not arrive in time: the results are void
        ring.drain();
        set_status(status, LA_ERR_TIMEOUT);
    }
    float* to = ENDS ? seg.B + run * D * DV : dS0 && lo == 0 ? dS0 + bh * D * DV : nullptr;
    if (to) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                to[(d0 + 8 * nt + 2 * tq + (e & 1)) * DV + col0 + g + (e >> 1) * 8] = ds[nt][e];
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
// then through scale and norm to the inputs.  Two warps own 16 tokens of dQ or of
// dK, each half of the d columns and of the token tiles.  The kept planes arrive with a
// scale per value column, the contracted index here; they are brought under one scale
// each (E and dV: one for 16 tokens) in shared memory (a power of two: exact but for
// columns under 2^-24 of the largest), so that fragments go from ldmatrix into the MMA
// as they are and every factor is one of a row, applied to fp32 accumulators.  The
// 64 x 64 matrices pass through a tile of the two warps' own as fp16 rows, each half under a power of two.  One fp16 part
// throughout: 2^-12 of a term, a sixteenth of the bf16 rounding of the results.  (A result
// that cancels to less than a sixteenth of its terms shows it: one token, one key head
// and value heads whose gradients happen to oppose.)
// Loops over fragments stay rolled: unrolled, the two roles' code overran the
// instruction cache and its misses were half of all stalls.
//
// A CTA per SM takes every gridDim-th chunk.  Its loads run a step (one value head
// of one chunk) ahead: the token planes have two buffers; the state planes are used
// first in a step and refilled while the rest of it runs.  (One chunk per CTA, each
// waiting for its own 150 KB: 508 against 399 us at B4 H8 N8192 d=128.)  Measured there:
// 357 us for 4096 chunks, 1.7 TB/s of 5.9e8 bytes; the loads alone take 165 us, the
// rest is a step's dependent stretches between its barriers (42% of the issue slots
// used, a quarter of a warp's cycles per instruction at barriers).
constexpr int kDqkThreads = 512;

template <int D, int DV>
struct DqkSmem {
    // a step's token planes, factors and column scales, twice
    static constexpr int E = 0, dV = kC * DV * 2, dO = 2 * kC * DV * 2, fac = 3 * kC * DV * 2,
                         facs = (kFacC - kFacB) * kC * 4, cols = fac + facs, step = cols + 12 * DV * 4;
    static constexpr int S = 2 * step, dS = S + D * DV * 2, K = dS + D * DV * 2, Q = K + row_image<D>(),
                         tile = Q + row_image<D>(), vec = tile + 8 * 16 * 128, bar = vec + (6 * kC + 8 * 32) * 4,
                         bytes = bar + 64;
    static_assert(bytes <= 232448, "shared memory");
};

// Kept blocks (16 value columns x 16; `per` of them per slice, the factors of every
// `group` of those behind one another) times c[col] / m
__device__ __forceinline__ void one_scale(unsigned char* plane, int blocks, int per, int group, int DV, const float* c,
                                          float inv_m)
{
    for (int u = threadIdx.x; u < blocks * 32; u += kDqkThreads) {
        const int block = u >> 5, col = block / per * 16 + ((u >> 3) & 1) * 8 + (u & 7);
        const __half2 f = __float2half2_rn(c[col + block % per / group * DV] * inv_m);
        uint4* at = reinterpret_cast<uint4*>(plane) + u;
        uint4 x = *at;
        __half2* h = reinterpret_cast<__half2*>(&x);
        h[0] = __hmul2(h[0], f), h[1] = __hmul2(h[1], f), h[2] = __hmul2(h[2], f), h[3] = __hmul2(h[3], f);
        *at = x;
    }
}

// a warp's wait: one verdict for all lanes
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, wait_for(bar, parity));
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
                __nv_bfloat16* __restrict__ dk, int64_t N, int nchunk, int items, int H, int Hk, int l2, float scale,
                int* status)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    using SM = DqkSmem<D, DV>;
    constexpr int RB = 2 * D, VB = 2 * DV, NT = D / 16, KS = DV / 16;  // NT: n tiles of half a row
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    const uint32_t base = smem_addr(smem);
    float* sdo = reinterpret_cast<float*>(smem + SM::vec);  // dO's row scales
    float* eg = sdo + kC;                                   // e^G
    float* ege = eg + kC;                                   // e^{G_C - G}
    float* cd = ege + kC;                                   // decay from a token to its tile's end
    float* ip = cd + kC;                                    // 1 / p
    float* kp = ip + kC;                                    // fk / p
    float* prow = kp + kC + (warp >> 1) * 32;               // [half][16 rows], the two warps' own
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::bar);  // token planes (2), states, row images
    float *mE = reinterpret_cast<float*>(full + 4), *mV = mE + 4;  // E's and dV's scales, of 16 tokens each
    const int per = H / Hk;
    const bool role_k = warp >= 8;
    const int pr = warp >> 1, h = warp & 1, rt = pr & 3, r0 = 16 * rt;
    const int dg = h * (D / 32);  // first 16-column group
    const uint32_t mytile = base + SM::tile + pr * 16 * 128;
    auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + pr) : "memory"); };
    const int steps = (items - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x * per;

    if (tid == 0) {
        for (int i = 0; i < 4; ++i)
            sm100::mbar_init(full + i, 1);
        sm100::fence_mbar_init();
    }
    __syncthreads();
    struct Step {
        int64_t kh, bh, at, t0;
        int c, n;
    };
    auto step_of = [&](int s) {
        Step x;
        const int item = blockIdx.x + s / per * gridDim.x;
        x.kh = item / nchunk, x.c = item % nchunk;
        x.bh = x.kh / Hk * H + (x.kh % Hk) * per + s % per;
        x.at = x.bh * nchunk + x.c;
        x.t0 = (int64_t)x.c * kC;
        x.n = (int)min((int64_t)kC, N - x.t0);
        return x;
    };
    // loads, by one thread, after every thread's accesses to the buffer are fenced
    auto load_tokens = [&](int s) {
        const Step x = step_of(s);
        const uint32_t to = base + (s & 1) * SM::step;
        uint64_t* bar = full + (s & 1);
        sm100::mbar_arrive_expect_tx(bar, 2 * kC * DV * 2 + x.n * DV * 2 + SM::facs + 12 * DV * 4);
        delta::bulk_load(to + SM::E, kept.E + 2 * x.at * (kC * DV * 2), kC * DV * 2, bar);
        delta::bulk_load(to + SM::dV, kept.dV + x.at * (kC * DV * 2), kC * DV * 2, bar);
        delta::bulk_load(to + SM::dO, dout + (x.bh * N + x.t0) * DV, x.n * DV * 2, bar);
        delta::bulk_load(to + SM::fac, blobs + x.at * (int64_t)blob_bytes<true>() + fac_at<true>() + kFacB * kC * 4,
                         SM::facs, bar);
        delta::bulk_load(to + SM::cols, kept.sE + x.at * 4 * DV, 4 * DV * 4, bar);
        delta::bulk_load(to + SM::cols + 4 * DV * 4, kept.sV + x.at * 4 * DV, 4 * DV * 4, bar);
        delta::bulk_load(to + SM::cols + 8 * DV * 4, kept.sS + x.at * 2 * DV, 2 * DV * 4, bar);
        delta::bulk_load(to + SM::cols + 10 * DV * 4, kept.sD + x.at * 2 * DV, 2 * DV * 4, bar);
    };
    auto load_states = [&](int s) {
        const Step x = step_of(s);
        sm100::mbar_arrive_expect_tx(full + 2, 2 * D * DV * 2);
        delta::bulk_load(base + SM::S, kept.S + 2 * x.at * (int64_t)(D * DV * 2), D * DV * 2, full + 2);
        delta::bulk_load(base + SM::dS, kept.dS + x.at * (D * DV * 2), D * DV * 2, full + 2);
    };
    auto load_rows = [&](int s) {
        const Step x = step_of(s);
        sm100::mbar_arrive_expect_tx(full + 3, 2 * row_image<D>());
        delta::bulk_load(base + SM::K, rows + (x.kh * nchunk + x.c) * (int64_t)(2 * row_image<D>()),
                         2 * row_image<D>(), full + 3);
    };
    if (tid == 0 && steps > 0) {
        load_tokens(0);
        load_states(0);
        load_rows(0);
    }
    float tot[NT][4];
    bool ok = true;
    for (int s = 0; s < steps; ++s) {
        const int buf = (s & 1) * SM::step, p = s % per;
        if (p == 0)
            clear(tot);
        if (tid == 0 && s + 1 < steps)
            load_tokens(s + 1);
        const int oE = buf + SM::E, odV = buf + SM::dV, odO = buf + SM::dO;
        const float* fac = reinterpret_cast<const float*>(smem + buf + SM::fac) - kFacB * kC;
        const float *cE = reinterpret_cast<const float*>(smem + buf + SM::cols), *cV = cE + 4 * DV, *cS = cV + 4 * DV,
                    *cD = cS + 2 * DV;
        const float *fB = fac + kFacB * kC, *fK = fac + kFacK * kC, *fQ = fac + kFacQ * kC, *gh = fac + kFacGh * kC,
                    *gl = fac + kFacGl * kC;
        ok = ok && wait_warp(full + (s & 1), (s >> 1) & 1);
        float mS = 0.f, mD = 0.f;
        if (ok) {
            // dO to scaled fp16 rows in place, a row by the lanes of one warp
            constexpr int LPR = DV / 8, RPP = kDqkThreads / LPR;
            const int n = step_of(s).n;
#pragma unroll
            for (int b = 0; b < kC; b += RPP) {
                const int r = b + tid / LPR, part = tid % LPR;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (r < n)
                    w = *reinterpret_cast<const uint4*>(smem + odO + r * VB + part * 16);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                float f[8], mx = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[2 * i] = lo_f(u[i]), f[2 * i + 1] = hi_f(u[i]);
                    mx = max_abs(max_abs(mx, f[2 * i]), f[2 * i + 1]);
                }
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const Pow2 q = pow2_for(mx);
                uint4 h;
                h.x = h2(f[0] * q.to, f[1] * q.to), h.y = h2(f[2] * q.to, f[3] * q.to);
                h.z = h2(f[4] * q.to, f[5] * q.to), h.w = h2(f[6] * q.to, f[7] * q.to);
                __syncwarp();
                if (r < kC) {  // at DV = 32 half of the warps have no row
                    *reinterpret_cast<uint4*>(smem + odO + tile_off<VB>(r, part)) = h;
                    if (part == 0)
                        sdo[r] = q.from;
                }
            }
            if (tid < kC) {
                eg[tid] = exp2f(gh[tid] + gl[tid]);
                ege[tid] = exp2f((gh[kC - 1] - gh[tid]) + (gl[kC - 1] - gl[tid]));
                cd[tid] = exp2f((gh[tid | 15] - gh[tid]) + (gl[tid | 15] - gl[tid]));
                ip[tid] = 1.0f / fac[kFacPk * kC + tid];
                kp[tid] = fK[tid] / fac[kFacPk * kC + tid];
            }
            mS = warp_max(cS, 2 * DV), mD = warp_max(cD, 2 * DV);
            // 1 / m of a power of two is exact; the blocks of a warp are all of token tile warp % 4
            const float xE = warp_max(cE + (warp & 3) * DV, DV), xV = warp_max(cV + (warp & 3) * DV, DV);
            if (warp < 4 && lane == 0)
                mE[warp] = xE, mV[warp] = xV;
            one_scale(smem + oE, KS * 4, 4, 1, DV, cE, 1.0f / xE);
            one_scale(smem + odV, KS * 4, 4, 1, DV, cV, 1.0f / xV);
        }
        ok = ok && wait_warp(full + 2, s & 1);
        if (ok) {
            one_scale(smem + SM::S, KS * (D / 16), D / 16, D / 32, DV, cS, 1.0f / mS);
            one_scale(smem + SM::dS, KS * (D / 16), D / 16, D / 32, DV, cD, 1.0f / mD);
        }
        ok = __syncthreads_and(ok);
        if (!ok)
            break;

        const int ia = r0 + g, ib = ia + 8;
        // A fragments of this warp's rows, 16 value columns ks: dO is row-major, kept
        // planes lie turned
        auto a_rows = [&](uint32_t (&x)[4], int plane, int ks) {
            if (plane == odO) {
                ldsm4(x, addr_a<VB>(base + odO, lane, r0, 16 * ks));
            } else {
                uint32_t y[4];
                ldsm4t(y, base + plane + (ks * 4 + rt) * 512 + lane * 16);
                x[0] = y[0], x[1] = y[2], x[2] = y[1], x[3] = y[3];
            }
        };
        // x[row][token] = this warp's rows of plane `a` dot the tokens of plane `b`,
        // its token tiles h and h + 2 of lo .. hi
        auto dots = [&](float (&x)[4][4], int a_plane, int b_plane, int lo, int hi) {
            clear(x);
#pragma unroll 2
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t a[4], b[4];
                a_rows(a, a_plane, ks);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int j = h + 2 * u;
                    if (j >= lo && j <= hi) {
                        if (b_plane == odO)
                            ldsm4(b, addr_b<VB>(base + odO, lane, 16 * j, 16 * ks));
                        else
                            ldsm4t(b, base + b_plane + (ks * 4 + j) * 512 + lane * 16);
                        mma(x[2 * u], a, b[0], b[1]);
                        mma(x[2 * u + 1], a, b[2], b[3]);
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
            clear(acc);
#pragma unroll 2
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t a[4], b[4];
                a_rows(a, a_plane, ks);
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) {
                    ldsm4t(b, base + b_plane + (ks * (D / 16) + dg + j) * 512 + lane * 16);
                    mma(acc[2 * j], a, b[0], b[1]);
                    mma(acc[2 * j + 1], a, b[2], b[3]);
                }
            }
            add(acc, fa, fb);
        };
        // tot += x (64 tokens over the two warps, zero outside tiles lo .. hi) times a
        // row image
        auto rows_product = [&](const float (&x)[4][4], int image, int lo, int hi) {
            float ma = 0.f, mb = 0.f;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                ma = max_abs(max_abs(ma, x[nt][0]), x[nt][1]);
                mb = max_abs(max_abs(mb, x[nt][2]), x[nt][3]);
            }
            const Pow2 pa = pow2_for(quad_max(ma)), pb = pow2_for(quad_max(mb));
            pair_sync();  // the tile is read
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const int part = 2 * (h + (nt & 2)) + (nt & 1);  // 16-byte part of a row
                *reinterpret_cast<uint32_t*>(smem + (mytile - base) + tile_off<128>(g, part) + 4 * tq) =
                    h2(x[nt][0] * pa.to, x[nt][1] * pa.to);
                *reinterpret_cast<uint32_t*>(smem + (mytile - base) + tile_off<128>(g + 8, part) + 4 * tq) =
                    h2(x[nt][2] * pb.to, x[nt][3] * pb.to);
            }
            if (tq == 0)
                prow[16 * h + g] = pa.from, prow[16 * h + g + 8] = pb.from;
            pair_sync();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float acc[NT][4];
                clear(acc);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int kk = half + 2 * u;
                    if (kk >= lo && kk <= hi) {
                        uint32_t a[4], b[4];
                        ldsm4(a, addr_a<128>(mytile, lane, 0, 16 * kk));
#pragma unroll
                        for (int j = 0; j < NT / 2; ++j) {
                            ldsm4t(b, addr_bt<RB>(base + image, lane, 16 * kk, 16 * (dg + j)));
                            mma(acc[2 * j], a, b[0], b[1]);
                            mma(acc[2 * j + 1], a, b[2], b[3]);
                        }
                    }
                }
                add(acc, prow[16 * half + g], prow[16 * half + g + 8]);
            }
        };
        // decays in base 2: between two tokens, and from a tile's end to a later token
        auto gap = [&](int i, int j) { return (gh[i] - gh[j]) + (gl[i] - gl[j]); };
        auto since = [&](int i, int tile) { return ex2(gap(i, 16 * tile + 15)); };
        auto pair2 = [&](const float* f, int i) { return *reinterpret_cast<const float2*>(f + i); };
        // the products with the states first: their planes are refilled meanwhile
        if (!role_k) {
            state(odO, SM::S, eg[ia] * (sdo[ia] * mS), eg[ib] * (sdo[ib] * mS));
        } else {
            state(odV, SM::S, -eg[ia] * ip[ia] * (mV[rt] * mS), -eg[ib] * ip[ib] * (mV[rt] * mS));
            state(oE, SM::dS, ege[ia] * fB[ia] * (mE[rt] * mD), ege[ib] * fB[ib] * (mE[rt] * mD));
        }
        sm100::fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0 && s + 1 < steps)
            load_states(s + 1);
        if (p == 0) {
            ok = __syncthreads_and(wait_warp(full + 3, (s / per) & 1));
            if (!ok)
                break;
        }
        if (!role_k) {
            float x[4][4];
            dots(x, odO, oE, 0, rt);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int tile = h + 2 * u;
                const float fa = mE[tile] * sdo[ia], fb = mE[tile] * sdo[ib];
                if (tile < rt) {  // a row's decay from the tile's end, a column's to it
                    const float da = fa * since(ia, tile), db = fb * since(ib, tile);
#pragma unroll
                    for (int nt = 2 * u; nt < 2 * u + 2; ++nt) {
                        const int j = 16 * tile + 8 * (nt & 1) + 2 * tq;
                        const float2 f = mul2(mul2(pair2(fB, j), pair2(fK, j)), pair2(cd, j));
                        set_rows(x[nt], mul2(mul2(row_a(x[nt]), both(da)), f), mul2(mul2(row_b(x[nt]), both(db)), f));
                    }
                } else {
#pragma unroll
                    for (int nt = 2 * u; nt < 2 * u + 2; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = e >> 1 ? ib : ia, j = 16 * tile + 8 * (nt & 1) + 2 * tq + (e & 1);
                            x[nt][e] = j <= i ? x[nt][e] * (e >> 1 ? fb : fa) * ex2(gap(i, j)) * (fB[j] * fK[j]) : 0.f;
                        }
                }
            }
            rows_product(x, SM::K, 0, rt);
        } else {
            float x[4][4], y[4][4];
            {
                float z[4][4];
                dots(z, oE, odV, rt, 3);
                dots(y, odV, oE, 0, rt);
                dots(x, oE, odO, rt, 3);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int tile = h + 2 * u;
                    // dV's rows are the warp's (y) or tile's (z), E's the other's
                    if (tile > rt) {  // i > j: the columns' decay from the rows' tile's end
                        const float da = mE[rt] * fB[ia] * cd[ia], db = mE[rt] * fB[ib] * cd[ib], mv = -mV[tile];
#pragma unroll
                        for (int nt = 2 * u; nt < 2 * u + 2; ++nt) {
                            const int i = 16 * tile + 8 * (nt & 1) + 2 * tq;
                            const float2 dec = make_float2(since(i, rt), since(i + 1, rt));
                            const float2 fy = mul2(mul2(dec, pair2(kp, i)), both(mv));
                            set_rows(y[nt], mul2(mul2(row_a(z[nt]), both(da)), fy), mul2(mul2(row_b(z[nt]), both(db)), fy));
                            const float2 fx = mul2(mul2(mul2(dec, pair2(fQ, i)), pair2(sdo, i)), both(scale));
                            set_rows(x[nt], mul2(mul2(row_a(x[nt]), both(da)), fx), mul2(mul2(row_b(x[nt]), both(db)), fx));
                        }
                    } else if (tile < rt) {  // i < j: M alone, x is zero
                        const float fm = -mE[tile] * mV[rt];
                        const float da = fm * ip[ia] * since(ia, tile), db = fm * ip[ib] * since(ib, tile);
#pragma unroll
                        for (int nt = 2 * u; nt < 2 * u + 2; ++nt) {
                            const int i = 16 * tile + 8 * (nt & 1) + 2 * tq;
                            const float2 f = mul2(mul2(pair2(fB, i), pair2(fK, i)), pair2(cd, i));
                            set_rows(y[nt], mul2(mul2(row_a(y[nt]), both(da)), f), mul2(mul2(row_b(y[nt]), both(db)), f));
                        }
                    } else {
                        const float fm = mE[rt] * mV[rt], fx = mE[rt] * scale;
#pragma unroll
                        for (int nt = 2 * u; nt < 2 * u + 2; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int j = e >> 1 ? ib : ia, i = 16 * tile + 8 * (nt & 1) + 2 * tq + (e & 1);
                                const float d = gap(i, j), dec = ex2(i >= j ? d : -d);
                                y[nt][e] = i > j   ? -z[nt][e] * fm * dec * (fB[j] * kp[i])
                                           : i < j ? -y[nt][e] * fm * dec * (fB[i] * fK[i] * ip[j])
                                                   : 0.f;
                                x[nt][e] = i >= j ? x[nt][e] * (fx * sdo[i]) * dec * (fB[j] * fQ[i]) : 0.f;
                            }
                    }
                }
            }
            rows_product(y, SM::K, 0, 3);
            rows_product(x, SM::Q, rt, 3);
        }
        int again = s;  // the step's place is worked out anew, for registers
        asm volatile("" : "+r"(again));
        const Step me = step_of(again);
        const int64_t t0 = me.t0;
        const int n = me.n;
        if (p == per - 1) {
            // through scale and norm: unit = f image, dx = r (x - unit (unit.x))
            const int image = role_k ? SM::K : SM::Q;
            const float* f = fac + (role_k ? kFacK : kFacQ) * kC;
            const float* rr = fac + (role_k ? kFacRk : kFacRq) * kC;
            __nv_bfloat16* dst = role_k ? dk : dq;
            const float mul = role_k ? 1.0f : scale;
            auto unit = [&](int i, int nt) {
                return __half22float2(*reinterpret_cast<const __half2*>(
                    smem + image + tile_off<RB>(i, 2 * dg + nt) + 4 * tq));
            };
            float dot[2] = {0.f, 0.f};
            if (l2) {  // a row's dot over both warps' columns
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float2 u = unit(r0 + g + 8 * e, nt);
                        dot[e] = fmaf(u.x, tot[nt][2 * e], fmaf(u.y, tot[nt][2 * e + 1], dot[e]));
                    }
                    dot[e] += __shfl_xor_sync(0xffffffffu, dot[e], 1);
                    dot[e] += __shfl_xor_sync(0xffffffffu, dot[e], 2);
                }
                pair_sync();  // the products' factors are read
                if (tq == 0)
                    prow[16 * h + g] = dot[0], prow[16 * h + g + 8] = dot[1];
                pair_sync();
                dot[0] = prow[g] + prow[16 + g];
                dot[1] = prow[8 + g] + prow[24 + g];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = r0 + g + 8 * e;
                const float r = rr[i] * mul, d = dot[e] * f[i] * f[i];
                uint32_t w[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float2 x = make_float2(tot[nt][2 * e], tot[nt][2 * e + 1]);
                    if (l2)
                        x = fma2(unit(i, nt), both(-d), x);
                    w[nt] = sm100::pack_bf16x2(r * x.x, r * x.y);
                }
                __nv_bfloat16* row = dst + (me.kh * N + t0 + i) * D + 16 * dg;
                if (NT % 4 == 0) {
                    // lane tq of a quad gathers tile 4 m + tq of its row: 16 bytes
#pragma unroll
                    for (int m = 0; m < NT / 4; ++m) {
                        uint32_t v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            // round k: give the part of tile tq ^ k, get that of the own
                            const int want = tq ^ k;
                            const uint32_t give = want & 2 ? (want & 1 ? w[4 * m + 3] : w[4 * m + 2])
                                                           : (want & 1 ? w[4 * m + 1] : w[4 * m]);
                            v[k] = __shfl_xor_sync(0xffffffffu, give, k);
                        }
                        // v[k] came from lane tq ^ k: its columns are 2 (tq ^ k)
                        const uint32_t q0 = tq & 1 ? v[1] : v[0], q1 = tq & 1 ? v[0] : v[1],
                                       q2 = tq & 1 ? v[3] : v[2], q3 = tq & 1 ? v[2] : v[3];
                        const uint4 o = tq & 2 ? make_uint4(q2, q3, q0, q1) : make_uint4(q0, q1, q2, q3);
                        if (i < n)
                            *reinterpret_cast<uint4*>(row + 8 * (4 * m + tq)) = o;
                    }
                } else if (i < n) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        *reinterpret_cast<uint32_t*>(row + 8 * nt + 2 * tq) = w[nt];
                }
            }
        }
        sm100::fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0 && p == per - 1 && s + 1 < steps)
            load_rows(s + 1);
    }
    if (!ok && tid == 0) {
        // a copy did not arrive in time: the results are void.  Whatever else is in
        // flight gets as long again before its shared memory goes
        for (int i = 0; i < 4; ++i)
            for (int parity = 0; parity < 2; ++parity)
                if (!wait_for(full + i, parity))
                    break;
        set_status(status, LA_ERR_TIMEOUT);
    }
}

// ------------------------------------------------------------ k_delta_gates --
// dbeta and dlog_alpha of one chunk and value head.  log_alpha_t enters every decay
// that spans t, so its gradient is the sum of all terms with such a decay:
//
//   dlog_alpha_t = sum_{i >= t > j} W_ij + sum_{i >= t} h_i + sum_{j < t} l_j + e^{G_C} <S0, dS1>
//   W_ij = D_ij (dO_i.U_j scale q_i.k_j - dV_i.U_j k_i.k_j)
//
// with h, l and <S0, dS1> from the chains.  (By the rows' dots alone it is <S1, dS1> +
// sum_{i >= t} (q_i.dQ_i - v_i.dV_i), but there the terms that do not span t cancel only
// up to their rounding, which is all that is left of a strong gate's gradient.)
// A warp takes one or two 16 x 16 tiles of one of W's two parts: the Gram products from
// the row images, the dots over the value columns 32 at a time, from two fp16 parts (dO is
// exact), their column scales going to the fragments.  Then running sums along the rows,
// every entry added where it counts and nowhere taken off again.
// Measured: 137 us for the 4096 chunks of B4 H8 N8192 d=128, whose 480 MB alone take 94 us
// (5.1 TB/s); two blocks per SM, whose products (26 us), Gram products and sums are only
// partly under the other's loads.
constexpr int kGateThreads = 384;
constexpr int kGateCols = 32;

template <int D, int DV>
struct GateSmem {
    static constexpr int part = kC * kGateCols * 2, step = 4 * part, steps = DV / kGateCols;
    // the last two of four steps go where the row images were, once those are used
    static constexpr int late = steps == 4 && 2 * step <= 2 * row_image<D>() ? 2 : 0;
    static constexpr int K = 0, Q = row_image<D>(), buf = 2 * row_image<D>(), dO = buf + (steps - late) * step,
                         fac = dO + kC * DV * 2, facs = (kFacC - kFacB) * kC * 4,
                         cols = fac + facs,                            // [E, dV][4 tiles][DV] fp16 column scales
                         sums = cols + 8 * DV * 2,                     // [12 warps][32]
                         vec = sums + 12 * 32 * 4, bar = vec + 5 * kC * 4, bytes = bar + 128;
    static constexpr int at(int s) { return s < steps - late ? buf + s * step : (s - (steps - late)) * step; }
};

template <int D, int DV>
__global__ void __launch_bounds__(kGateThreads, 2)
    k_delta_gates(const unsigned char* __restrict__ rows, const unsigned char* __restrict__ blobs,
                  const __nv_bfloat16* __restrict__ dout, Kept kept, float* __restrict__ dbeta,
                  float* __restrict__ dlog_alpha, int64_t N, int nchunk, int H, int Hk, float scale, int* status)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    using SM = GateSmem<D, DV>;
    constexpr int RB = 2 * D, VB = 2 * DV, KS = DV / 16, STEPS = SM::steps;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    const bool of_k = warp >= 6;  // the part of k_i.k_j
    // tile of rows, the first tile of columns, the second there or not:
    // (3, 0 1) (3, 2 3) (2, 0 1) (1, 0 1) (2, 2) (0, 0)
    const int who = of_k ? warp - 6 : warp, I = 0x021233 >> 4 * who & 3, J = 0x020020 >> 4 * who & 3;
    const bool two = who < 4;
    const uint32_t base = smem_addr(smem);
    const int64_t at = blockIdx.x, bh = at / nchunk;
    const int c = (int)(at % nchunk);
    const int64_t kh = bh / H * Hk + (bh % H) / (H / Hk), t0 = (int64_t)c * kC;
    const int n = (int)min((int64_t)kC, N - t0);
    float* sdo = reinterpret_cast<float*>(smem + SM::vec);  // dO's row scales
    float *sh = sdo + kC, *sl = sh + 2 * kC;                // h in two parts, l
    float* rest = sl + kC;                                  // [2][32] row sums of the tiles (3, 0 1) and (2, 0 1)
    float* sums = reinterpret_cast<float*>(smem + SM::sums);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::bar);  // row images and factors, the steps
    float* top = reinterpret_cast<float*>(full + 5);               // [E, dV][4] largest column scale
    const float* fac = reinterpret_cast<const float*>(smem + SM::fac) - kFacB * kC;
    const float *fB = fac + kFacB * kC, *fK = fac + kFacK * kC, *fQ = fac + kFacQ * kC, *fP = fac + kFacPk * kC,
                *gh = fac + kFacGh * kC, *gl = fac + kFacGl * kC;

    auto load_step = [&](int s) {
        uint64_t* bar = full + 1 + s;
        const uint32_t to = base + SM::at(s);
        sm100::mbar_arrive_expect_tx(bar, SM::step);
        delta::bulk_load(to, kept.E + 2 * at * (kC * DV * 2) + s * SM::part, SM::part, bar);
        delta::bulk_load(to + SM::part, kept.E + (2 * at + 1) * (kC * DV * 2) + s * SM::part, SM::part, bar);
        delta::bulk_load(to + 2 * SM::part, kept.dV + at * (kC * DV * 2) + s * SM::part, SM::part, bar);
        delta::bulk_load(to + 3 * SM::part, kept.dVl + at * (kC * DV * 2) + s * SM::part, SM::part, bar);
    };
    if (tid == 0) {
        for (int i = 0; i < 1 + STEPS; ++i)
            sm100::mbar_init(full + i, 1);
        sm100::fence_mbar_init();
        sm100::mbar_arrive_expect_tx(full, 2 * row_image<D>() + SM::facs);
        delta::bulk_load(base + SM::K, rows + (kh * nchunk + c) * (int64_t)(2 * row_image<D>()), 2 * row_image<D>(), full);
        delta::bulk_load(base + SM::fac, blobs + at * blob_bytes<true>() + fac_at<true>() + kFacB * kC * 4, SM::facs, full);
        for (int s = 0; s < STEPS - SM::late; ++s)
            load_step(s);
    }
    // Meanwhile, every load first: dO, the column scales (E's by warps 0 to 3, dV's by the
    // others) and the chains' dots over 16 columns each
    constexpr int LPR = DV / 8, RPP = 256 / LPR;  // lanes per row of dO, rows of 256 threads
    uint4 w[kC / RPP];
#pragma unroll
    for (int b = 0; b < kC / RPP; ++b) {
        const int r = b * RPP + tid / LPR;
        w[b] = make_uint4(0, 0, 0, 0);
        if (r < n && tid < 256)
            w[b] = *reinterpret_cast<const uint4*>(dout + (bh * N + t0 + r) * DV + tid % LPR * 8);
    }
    float scales[DV / 32], dots[KS];
#pragma unroll
    for (int i = 0; i < DV / 32; ++i)
        scales[i] = (warp < 4 ? kept.sE : kept.sV)[(at * 4 + (warp & 3)) * DV + lane + 32 * i];  // again by warps 8 ..
    const float* sums_of = tid < kC ? kept.hq : tid < 2 * kC ? kept.hk : tid < 3 * kC ? kept.ll : kept.bb;
#pragma unroll
    for (int i = 0; i < KS; ++i)
        dots[i] = tid < 256 && tid % kC < n ? sums_of[(bh * KS + i) * N + t0 + tid % kC] : 0.f;
    float cd = tid < 2 * KS ? kept.cd[(bh * 2 * KS + tid) * nchunk + c] : 0.f;
    if (warp < 8) {
#pragma unroll
        for (int b = 0; b < kC / RPP; ++b) {  // dO to fp16 rows, a row by the lanes of one warp
            const int r = b * RPP + tid / LPR;
            const uint32_t u[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mx = max_abs(max_abs(mx, lo_f(u[i])), hi_f(u[i]));
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const Pow2 q = pow2_for(mx);
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[i] = h2(lo_f(u[i]) * q.to, hi_f(u[i]) * q.to);
            *reinterpret_cast<uint4*>(smem + SM::dO + tile_off<VB>(r, tid % LPR)) = make_uint4(h[0], h[1], h[2], h[3]);
            if (tid % LPR == 0)
                sdo[r] = q.from;
        }
        {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < DV / 32; ++i)
                m = fmaxf(m, scales[i]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            __half* dst = reinterpret_cast<__half*>(smem + SM::cols) + warp * DV;
#pragma unroll
            for (int i = 0; i < DV / 32; ++i)
                dst[lane + 32 * i] = __float2half_rn(scales[i] * (1.0f / m));  // powers of two
            if (lane == 0)
                top[warp] = m;
        }
        {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < KS; ++i)
                x += dots[i];
            if (tid < 3 * kC)
                sh[tid] = x;  // h's parts, l
            else if (tid % kC < n)
                dbeta[bh * N + t0 + tid % kC] = x;
        }
    }
    if (warp == 0) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            cd += __shfl_xor_sync(0xffffffffu, cd, o);
    }
    __syncthreads();
    bool ok = wait_warp(full, 0);
    // this warp's rows times its columns' tokens: Gram products, then dots over value columns
    float gm[4][4], x[4][4];
    clear(gm);
    clear(x);
    if (ok) {
#pragma unroll 4
        for (int kk = 0; kk < D; kk += 16) {
            uint32_t a[4], b[4];
            ldsm4(a, addr_a<RB>(base + (of_k ? SM::K : SM::Q), lane, 16 * I, kk));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (j == 0 || two) {
                    ldsm4(b, addr_b<RB>(base + SM::K, lane, 16 * (J + j), kk));
                    mma(gm[2 * j], a, b[0], b[1]);
                    mma(gm[2 * j + 1], a, b[2], b[3]);
                }
            }
        }
    }
    if (SM::late) {
        sm100::fence_proxy_async_smem();
        ok = __syncthreads_and(ok);  // the row images are read
        if (tid == 0 && ok)
            for (int s = STEPS - SM::late; s < STEPS; ++s)
                load_step(s);
    }
    auto times = [](uint32_t (&x)[4], uint32_t f0, uint32_t f1) {  // registers 0, 2 and 1, 3
        const uint32_t f[2] = {f0, f1};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&x[i]), *reinterpret_cast<const __half2*>(&f[i & 1]));
            x[i] = *reinterpret_cast<const uint32_t*>(&y);
        }
    };
    // column scales of tile `row` (E: 0 .. 3, dV: 4 ..), columns c0 + 2 tq and the next
    auto col = [&](int row, int c0) {
        return *reinterpret_cast<const uint32_t*>(smem + SM::cols + (row * DV + c0 + 2 * tq) * 2);
    };
#pragma unroll 1
    for (int s = 0; s < STEPS; ++s) {
        ok = ok && wait_warp(full + 1 + s, 0);
        const uint32_t buf = base + SM::at(s);
        if (ok) {
#pragma unroll
            for (int ks = 0; ks < kGateCols / 16; ++ks) {
                const int c0 = s * kGateCols + 16 * ks;
                uint32_t ah[4], al[4];
                if (of_k) {
                    uint32_t y[4], z[4];
                    ldsm4t(y, buf + 2 * SM::part + (ks * 4 + I) * 512 + lane * 16);
                    ldsm4t(z, buf + 3 * SM::part + (ks * 4 + I) * 512 + lane * 16);
                    times(y, col(4 + I, c0), col(4 + I, c0 + 8));
                    times(z, col(4 + I, c0), col(4 + I, c0 + 8));
                    ah[0] = y[0], ah[1] = y[2], ah[2] = y[1], ah[3] = y[3];
                    al[0] = z[0], al[1] = z[2], al[2] = z[1], al[3] = z[3];
                } else {
                    ldsm4(ah, addr_a<VB>(base + SM::dO, lane, 16 * I, c0));
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (j == 0 || two) {
                        uint32_t bh_[4], bl[4];
                        ldsm4t(bh_, buf + (ks * 4 + J + j) * 512 + lane * 16);
                        ldsm4t(bl, buf + SM::part + (ks * 4 + J + j) * 512 + lane * 16);
                        const uint32_t f0 = col(J + j, c0), f1 = col(J + j, c0 + 8);
                        times(bh_, f0, f1);
                        times(bl, f0, f1);
                        mma(x[2 * j], ah, bh_[0], bh_[1]);
                        mma(x[2 * j + 1], ah, bh_[2], bh_[3]);
                        mma(x[2 * j], ah, bl[0], bl[1]);
                        mma(x[2 * j + 1], ah, bl[2], bl[3]);
                        if (of_k) {
                            mma(x[2 * j], al, bh_[0], bh_[1]);
                            mma(x[2 * j + 1], al, bh_[2], bh_[3]);
                        }
                    }
                }
            }
        }
    }
    if (!__syncthreads_and(ok)) {
        // a copy did not arrive in time: the results are void.  What is in flight gets as
        // long again before its shared memory goes
        if (tid == 0) {
            for (int i = 0; i < 1 + STEPS; ++i)
                wait_for(full + i, 0);
            set_status(status, LA_ERR_TIMEOUT);
        }
        __syncthreads();
        return;
    }
    // W, its running sums along the rows up to column t, and those added up over rows i >= t
    const int ia = 16 * I + g, ib = ia + 8;
    const float ra = of_k ? -fK[ia] : fQ[ia] * scale, rb = of_k ? -fK[ib] : fQ[ib] * scale;
    const float va = of_k ? top[4 + I] / fP[ia] : sdo[ia], vb = of_k ? top[4 + I] / fP[ib] : sdo[ib];
    float y[8] = {}, suma = 0.f, sumb = 0.f;
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        if (nt < 2 || two) {
            const int j = 16 * J + 8 * nt + 2 * tq;
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = e >> 1 ? ib : ia, jj = j + (e & 1);
                const float d = ex2((gh[i] - gh[jj]) + (gl[i] - gl[jj]));
                const float a = gm[nt][e] * ((e >> 1 ? rb : ra) * fK[jj]);
                const float b = x[nt][e] * ((e >> 1 ? vb : va) * (fB[jj] * top[J + (nt >> 1)]));
                w[e] = jj < i ? a * b * d : 0.f;
            }
            float pa = w[0] + w[1], pb = w[2] + w[3];  // inclusive over the quad
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                const float qa = __shfl_up_sync(0xffffffffu, pa, o, 4), qb = __shfl_up_sync(0xffffffffu, pb, o, 4);
                if (tq >= o)
                    pa += qa, pb += qb;
            }
            float ea = __shfl_up_sync(0xffffffffu, pa, 1, 4), eb = __shfl_up_sync(0xffffffffu, pb, 1, 4);
            ea = suma + (tq ? ea : 0.f), eb = sumb + (tq ? eb : 0.f);  // of the columns before j
            y[2 * nt] = (ia >= j ? ea : 0.f) + (ib >= j ? eb : 0.f);
            y[2 * nt + 1] = (ia > j ? ea + w[0] : 0.f) + (ib > j ? eb + w[2] : 0.f);
            suma += __shfl_sync(0xffffffffu, pa, 3, 4), sumb += __shfl_sync(0xffffffffu, pb, 3, 4);
        }
    }
    // lane 4 g + tq: C tile g >> 1, column 2 tq + (g & 1)
    sums[warp * 32 + 8 * (g >> 1) + 2 * tq + (g & 1)] = delta::sum8(y, lane);
    if (tq == 0 && (who == 0 || who == 2)) {  // for the columns behind tiles 0 and 1
        float* to = rest + (of_k ? 32 : 0) + 16 * (I - 2) + g;
        to[0] = suma, to[8] = sumb;
    }
    __syncthreads();
    if (warp == 0) {
        float h[2], l[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            h[u] = sh[lane + 32 * u] + sh[kC + lane + 32 * u], l[u] = sl[lane + 32 * u];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float a = __shfl_down_sync(0xffffffffu, h[u], o), b = __shfl_up_sync(0xffffffffu, l[u], o);
                if (lane + o < 32)
                    h[u] += a;
                if (lane >= o)
                    l[u] += b;
            }
        }
        float r = rest[lane] + rest[32 + lane];  // of rows 32 + lane
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float a = __shfl_down_sync(0xffffffffu, r, o);
            if (lane + o < 32)
                r += a;
        }
        h[0] += __shfl_sync(0xffffffffu, h[1], 0);
        const float half = __shfl_sync(0xffffffffu, l[0], 31);
        cd *= exp2f(gh[kC - 1] + gl[kC - 1]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int t = lane + 32 * u;
            float z = 0.f, before = __shfl_up_sync(0xffffffffu, l[u], 1);
            before = (lane ? before : 0.f) + (u ? half : 0.f);
#pragma unroll
            for (int p = 0; p < 12; p += 6) {  // the tiles with this column: of both warps' halves, of the first
                if (u == 0)
                    z += sums[(p + 0) * 32 + lane] + sums[(p + 2) * 32 + lane] + sums[(p + 3) * 32 + lane];
                else
                    z += sums[(p + 1) * 32 + lane];
                if (lane < 16)
                    z += sums[(p + (u ? 4 : 5)) * 32 + lane];
            }
            if (u)
                z += r;
            if (t < n)
                dlog_alpha[bh * N + t0 + t] = z + h[u] + before + cd;
        }
    }
}

// dbeta alone, without gates
__global__ void __launch_bounds__(256)
    k_delta_dbeta(const float* __restrict__ bb, float* __restrict__ dbeta, int64_t N, int64_t count, int slices)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= count)
        return;
    const float* at = bb + i / N * slices * N + i % N;
    float x = 0.f;
    for (int s = 0; s < slices; ++s)
        x += at[s * N];
    dbeta[i] = x;
}

// ------------------------------------------------------------------- hosts --
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
int chunks_of(int64_t N) { return (int)((N + kC - 1) / kC); }

// Segments of a sequence.  Two runs over a segment and a walk over their ends take
// the place of one run over the whole, worth it from three segments on (forward and
// gradient, B1 H12 N4096 d = 128: 165 and 573 us whole, 153 and 450 us in three; B1 H16
// in two: 169 and 602 against 176 and 578 us); no more than give each warp of the
// second run a sub-partition of its own at 152 SMs, and no more than 32: the walk is
// serial, 0.7 us a step at d = 64, 1.9 us at 128.  So a segment is at least four chunks
// at d = 128 and two below (calls; B1 H4: N1000 d = 128 59 and 155 us in segments of
// eight chunks, 48 and 121 us of four, 54 and 120 us of two; N700 d = 64 34 and 98 us
// whole, 37 and 88 us of two or three; under eight chunks whole: N400 27 and 77 us, 36
// and 85 us in three).  By sizes alone, so that workspaces can be sized without the GPU.
int segments_of(const DeltaArgs& a)
{
    const int64_t slices = a.B * a.H * (a.dv / 16), most = chunks_of(a.N) / (a.d > 64 ? 4 : 2);
    int64_t n = 2 * 152 / slices;
    n = n < most ? n : most;
    n = n < 32 ? n : 32;
    if (n < 3 || chunks_of(a.N) < 8)
        return 1;
    const int64_t len = (chunks_of(a.N) + n - 1) / n;  // chunks of a segment; the last may be short
    return (int)((chunks_of(a.N) + len - 1) / len);
}

// Beginnings (or gradients of the ends), constant parts and matrices of the segments.
struct SegLayout {
    size_t start, B, M, total;  // relative to its own beginning
};
SegLayout seg_layout(const DeltaArgs& a)
{
    const size_t n = (size_t)segments_of(a), BH = (size_t)(a.B * a.H);
    SegLayout l = {};
    if (n > 1) {
        l.B = up256(BH * n * a.d * a.dv * 4);
        l.M = l.B + up256(BH * n * a.d * a.dv * 4);
        l.total = l.M + up256(BH * n * a.d * a.d * 4);
    }
    return l;
}

struct TcLayout {
    size_t rows, blobs, seg, total;
};
TcLayout tc_layout(const DeltaArgs& a)
{
    TcLayout l;
    const size_t n = (size_t)chunks_of(a.N);
    l.rows = 0;
    l.blobs = up256((size_t)(a.B * a.Hk) * n * 2 * kC * a.d * 2);
    l.seg = l.blobs + up256((size_t)(a.B * a.H) * n * blob_bytes<false>());
    l.total = l.seg + seg_layout(a).total;
    return l;
}

struct GradTcLayout {
    size_t rows, blobs, S, sS, E, sE, dS, sD, dV, sV, bb, dVl, KS, hq, hk, ll, cd, seg, total;
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
    l.S = take(BH * n * 2 * state);
    l.sS = take(BH * n * 2 * a.dv * 4);
    l.E = take(BH * n * 2 * toks);
    l.sE = take(BH * n * 4 * a.dv * 4);
    l.dS = take(BH * n * state);
    l.sD = take(BH * n * 2 * a.dv * 4);
    l.dV = take(BH * n * toks);
    l.sV = take(BH * n * 4 * a.dv * 4);
    l.bb = take(BH * sl * (size_t)a.N * 4);
    l.dVl = take(BH * n * toks);  // from here: with gates only, but the size is asked for without
    l.KS = take(BH * n * 2 * toks);
    l.hq = take(BH * sl * (size_t)a.N * 4);
    l.hk = take(BH * sl * (size_t)a.N * 4);
    l.ll = take(BH * sl * (size_t)a.N * 4);
    l.cd = take(BH * sl * 2 * n * 4);
    l.seg = take(seg_layout(a).total);
    l.total = at;
    return l;
}

// How a chain kernel is cut.  SP = 2 (two warps per slice) while that gives no
// more warps than the GPU has sub-partitions to give each a tensor core of its own;
// slices per CTA: as few as give no more CTAs than SMs, at most 8 warps.  Measured at
// d = 128: 32 heads of 8192 tokens 468 us with one warp per slice, 304 us with two;
// 512 heads of 2011 tokens 736 us with one, 886 us with two.  Two also where a head has
// two slices, which would be two warps on an SM (dv = 32, forward and gradient, one and
// two: 256 heads of 1024 tokens d = 128 213 and 813, 184 and 699 us; 512 of d = 64 317
// and 1227, 295 and 1090 us; not at d = 32, 272 and 923, 229 and 979 us).
struct Cut {
    int SP, W;
};
Cut cut_of(int64_t runs, int columns, int d)  // sequences or segments, value columns of each
{
    const int sms = device_sm_count();
    const int64_t slices = runs * (columns / 16);
    Cut c;
    c.SP = 2 * slices <= 4 * (int64_t)sms || (columns <= 32 && d > 32) ? 2 : 1;
    const int cap = 8 / c.SP;
    c.W = 1;
    while (2 * c.W <= cap && columns / 16 % (2 * c.W) == 0 && slices / c.W > sms)
        c.W *= 2;
    return c;
}

// The runs of the last round of CTAs, where they are few enough for two CTAs each:
// two warps per slice then end sooner than one would.  Forward and gradient, in one
// launch and in two (us): B5 H32 N1024 d = 128 248 and 922, 229 and 865; B16 H32 N2011
// 1070 and 4325, 1027 and 4265; B14 H16 N1024 64 x 128 201 and 839, 195 and 809.  Not
// for smaller states: B20 H16 N1024 64 x 64 214 and 754, 215 and 766; B10 H16 32 x 32
// 103 and 271, 101 and 348 (these four before the gates had a kernel of their own).
int64_t tail_of(const Cut& cut, int64_t runs, int columns, int d)
{
    const int sms = device_sm_count();
    if (cut.SP == 2 || columns != 16 * cut.W || d < 64 || d + columns <= 128 || runs <= sms)
        return 0;
    const int64_t tail = runs % sms;
    return 2 * tail <= sms ? tail : 0;
}

// launch(cut, first run, runs) for all runs
template <typename Launch>
cudaError_t in_rounds(int64_t runs, int columns, int d, Launch launch)
{
    const Cut cut = cut_of(runs, columns, d);
    const int64_t tail = tail_of(cut, runs, columns, d);
    const cudaError_t e = launch(cut, (int64_t)0, runs - tail);
    return e != cudaSuccess || !tail ? e : launch(Cut{2, cut.W / 2}, runs - tail, tail);
}

template <typename K>
cudaError_t allow_smem(K kern, int bytes)
{
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int D, bool GRAD, int SP, bool READS>
cudaError_t launch_chain(const DeltaArgs& a, int W, const unsigned char* rows, const unsigned char* blobs,
                         const Kept& kept, const Segments& seg, int64_t runs)
{
    const int smem = ChainSmem<D, GRAD, SP>::bytes(W);
    const cudaError_t e = allow_smem(k_delta_chain<D, GRAD, SP, READS>, smem);
    if (e != cudaSuccess)
        return e;
    const int columns = a.dv + (seg.carry ? a.d : 0);
    k_delta_chain<D, GRAD, SP, READS>
        <<<(unsigned)(runs * (columns / (16 * W))), 32 * SP * W, smem, a.stream>>>(
            rows, blobs, static_cast<const __nv_bfloat16*>(a.v),
            READS && !GRAD ? static_cast<__nv_bfloat16*>(a.out) : nullptr, a.S0,
            GRAD || seg.carry ? nullptr : a.S_out, a.N, chunks_of(a.N), (int)a.H, (int)a.Hk, a.dv,
            static_cast<const __nv_bfloat16*>(a.dout), kept, seg, a.status);
    count_launches(1);
    return cudaGetLastError();
}

template <int D, int SP, bool GATED, bool ENDS>
cudaError_t launch_rev(const DeltaArgs& a, int W, const unsigned char* rows, const unsigned char* blobs,
                       const Kept& kept, const Segments& seg, int64_t runs)
{
    const int smem = RevSmem<D, SP>::bytes(W);
    const cudaError_t e = allow_smem(k_delta_rev<D, SP, GATED, ENDS>, smem);
    if (e != cudaSuccess)
        return e;
    k_delta_rev<D, SP, GATED, ENDS>
        <<<(unsigned)(runs * (a.dv / (16 * W))), 32 * SP * W, smem, a.stream>>>(
            rows, blobs, static_cast<const __nv_bfloat16*>(a.dout), a.dS_out,
            static_cast<__nv_bfloat16*>(a.dv_), a.dS0, a.N, chunks_of(a.N), (int)a.H, (int)a.Hk, a.dv, kept, seg,
            a.status);
    count_launches(1);
    return cudaGetLastError();
}

template <int D, bool GATED, bool ENDS>
cudaError_t run_rev_cut(const DeltaArgs& a, const unsigned char* rows, const unsigned char* blobs, const Kept& kept,
                        const Segments& seg)
{
    return in_rounds(a.B * a.H * seg.count, a.dv, D, [&](Cut cut, int64_t first, int64_t runs) {
        Segments x = seg;
        x.skip = first;
        return cut.SP == 2 ? launch_rev<D, 2, GATED, ENDS>(a, cut.W, rows, blobs, kept, x, runs)
                           : launch_rev<D, 1, GATED, ENDS>(a, cut.W, rows, blobs, kept, x, runs);
    });
}

template <int D, bool REV>
cudaError_t launch_join(const DeltaArgs& a, const float* from, const float* B, const float* M, float* start, int n,
                        int mcount)
{
    k_delta_join<D, REV><<<dim3((unsigned)(a.B * a.H), a.dv / kJoinCols), 256, 0, a.stream>>>(from, B, M, start, n,
                                                                                             mcount, a.dv);
    count_launches(1);
    return cudaGetLastError();
}

// A chain over whole sequences, or over segments once their states are known.  A
// gradient's reverse chain wants the last segment's M too.
template <int D, bool GRAD, bool READS>
cudaError_t run_chain(const DeltaArgs& a, const unsigned char* rows, const unsigned char* blobs, const Kept& kept,
                      unsigned char* ws)
{
    const int n = segments_of(a);
    Segments seg = {1, chunks_of(a.N), nullptr, 0, nullptr, nullptr, 0, blob_bytes<GRAD>(), fac_at<GRAD>(), 0};
    if (n > 1) {
        const SegLayout l = seg_layout(a);
        float* start = reinterpret_cast<float*>(ws + l.start);
        float* B = reinterpret_cast<float*>(ws + l.B);
        float* M = reinterpret_cast<float*>(ws + l.M);
        seg.len = (chunks_of(a.N) + n - 1) / n;
        const int m = GRAD ? n : n - 1;
        const Segments ends = {m, seg.len, nullptr, 1, B, M, 0, seg.blob, seg.fac, 0};
        const int64_t runs = a.B * a.H * m;
        const Cut cut = cut_of(runs, a.dv + a.d, D);
        cudaError_t e = cut.SP == 2 ? launch_chain<D, false, 2, false>(a, cut.W, rows, blobs, Kept{}, ends, runs)
                                    : launch_chain<D, false, 1, false>(a, cut.W, rows, blobs, Kept{}, ends, runs);
        if (e != cudaSuccess || (e = launch_join<D, false>(a, a.S0, B, M, start, n, m)) != cudaSuccess)
            return e;
        seg.count = n, seg.start = start;
    }
    return in_rounds(a.B * a.H * n, a.dv, D, [&](Cut cut, int64_t first, int64_t runs) {
        Segments x = seg;
        x.skip = first;
        return cut.SP == 2 ? launch_chain<D, GRAD, 2, READS>(a, cut.W, rows, blobs, kept, x, runs)
                           : launch_chain<D, GRAD, 1, READS>(a, cut.W, rows, blobs, kept, x, runs);
    });
}

// The reverse chain, after run_chain<GRAD>: it finds the segments' M where that left
// them.
template <int D>
cudaError_t run_rev(const DeltaArgs& a, const unsigned char* rows, const unsigned char* blobs, const Kept& kept,
                    unsigned char* ws)
{
    const int n = segments_of(a);
    Segments seg = {1, chunks_of(a.N), nullptr, 0, nullptr, nullptr, 0, blob_bytes<true>(), fac_at<true>(), 0};
    if (n > 1) {
        const SegLayout l = seg_layout(a);
        float* start = reinterpret_cast<float*>(ws + l.start);
        float* C = reinterpret_cast<float*>(ws + l.B);
        const float* M = reinterpret_cast<const float*>(ws + l.M);
        seg.len = (chunks_of(a.N) + n - 1) / n;
        Segments ends = seg;
        ends.count = n - 1, ends.first = 1, ends.B = C;
        cudaError_t e = run_rev_cut<D, false, true>(a, rows, blobs, kept, ends);
        if (e != cudaSuccess || (e = launch_join<D, true>(a, a.dS_out, C, M, start, n, n)) != cudaSuccess)
            return e;
        seg.count = n, seg.start = start;
    }
    return a.log_alpha ? run_rev_cut<D, true, false>(a, rows, blobs, kept, seg)
                       : run_rev_cut<D, false, false>(a, rows, blobs, kept, seg);
}

template <int D>
cudaError_t run_forward(const DeltaArgs& a)
{
    const TcLayout l = tc_layout(a);
    unsigned char* ws = static_cast<unsigned char*>(a.ws);
    const int n = chunks_of(a.N);
    const int64_t BH = a.B * a.H;
    cudaError_t e = allow_smem(k_delta_prep<D, false>, PrepSmem<D, false>::bytes);
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
    const unsigned char *rows = ws + l.rows, *blobs = ws + l.blobs;
    return a.out ? run_chain<D, false, true>(a, rows, blobs, Kept{}, ws + l.seg)
                 : run_chain<D, false, false>(a, rows, blobs, Kept{}, ws + l.seg);
}

template <int D, int DV>
cudaError_t run_backward(const DeltaArgs& a)
{
    const GradTcLayout l = grad_tc_layout(a);
    unsigned char* ws = static_cast<unsigned char*>(a.ws);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    const Kept kept = {ws + l.S, f32(l.sS), ws + l.E, f32(l.sE), ws + l.dS, f32(l.sD),
                       ws + l.dV, f32(l.sV), f32(l.bb), ws + l.dVl, reinterpret_cast<float4*>(ws + l.KS),
                       f32(l.hq), f32(l.hk), f32(l.ll), f32(l.cd)};
    const int n = chunks_of(a.N), H = (int)a.H, Hk = (int)a.Hk, l2 = a.fm == LA_FM_L2;
    const int64_t BH = a.B * a.H;
    const __nv_bfloat16* dout = static_cast<const __nv_bfloat16*>(a.dout);
    cudaError_t e = allow_smem(k_delta_prep<D, true>, PrepSmem<D, true>::bytes);
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
    const unsigned char *rows = ws + l.rows, *blobs = ws + l.blobs;
    e = a.log_alpha ? run_chain<D, true, true>(a, rows, blobs, kept, ws + l.seg)
                    : run_chain<D, true, false>(a, rows, blobs, kept, ws + l.seg);
    if (e == cudaSuccess)
        e = run_rev<D>(a, rows, blobs, kept, ws + l.seg);
    if (e != cudaSuccess)
        return e;
    const int64_t items = a.B * a.Hk * n;
    const int sms = device_sm_count() > 0 ? device_sm_count() : 1;
    k_delta_dqk<D, DV><<<(unsigned)(items < sms ? items : sms), kDqkThreads, DqkSmem<D, DV>::bytes, a.stream>>>(
        ws + l.rows, ws + l.blobs, dout, kept, static_cast<__nv_bfloat16*>(a.dq),
        static_cast<__nv_bfloat16*>(a.dk), a.N, n, (int)items, H, Hk, l2, a.scale, a.status);
    count_launches(1);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    if (a.log_alpha) {
        if ((e = allow_smem(k_delta_gates<D, DV>, GateSmem<D, DV>::bytes)) != cudaSuccess)
            return e;
        k_delta_gates<D, DV><<<(unsigned)(BH * n), kGateThreads, GateSmem<D, DV>::bytes, a.stream>>>(
            rows, blobs, dout, kept, a.dbeta, a.dlog_alpha, a.N, n, H, Hk, a.scale, a.status);
    } else {
        const int64_t count = BH * a.N;
        k_delta_dbeta<<<(unsigned)((count + 255) / 256), 256, 0, a.stream>>>(kept.bb, a.dbeta, a.N, count, DV / 16);
    }
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


namespace delta {

cudaError_t join_segments(const DeltaArgs& a, bool rev, const float* from, const float* B, const float* M, float* start,
                          int n, int mcount)
{
    switch (a.d) {
    case 32: return rev ? launch_join<32, true>(a, from, B, M, start, n, mcount)
                        : launch_join<32, false>(a, from, B, M, start, n, mcount);
    case 64: return rev ? launch_join<64, true>(a, from, B, M, start, n, mcount)
                        : launch_join<64, false>(a, from, B, M, start, n, mcount);
    default: return rev ? launch_join<128, true>(a, from, B, M, start, n, mcount)
                        : launch_join<128, false>(a, from, B, M, start, n, mcount);
    }
}

}  // namespace delta

size_t delta_tc_forward_workspace(const DeltaArgs& a) { return tc_layout(a).total; }

cudaError_t delta_tc_forward(const DeltaArgs& a)
{
    switch (a.d) {
    case 32: return run_forward<32>(a);
    case 64: return run_forward<64>(a);
    default: return run_forward<128>(a);
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
