// la_conv.cu -- short causal convolution along the tokens, one filter per
// channel, with bias and activation: the mixing in front of the state-space scan
// and of the delta rule's queries, keys and values.
//
//   u_t = bias + sum_j w[c,j] x_{t-W+1+j},   y_t = act(u_t)
//   du_t = dy_t act'(u_t),  dx_t = sum_j w[c,j] du_{t+W-1-j},
//   dw[c,j] = sum_{b,t} du_t x_{t-W+1+j},    dbias = sum_{b,t} du_t
//
// x is token-major with any token and batch strides (a slice of a projection), y
// head-major [B,H,N,C/H] (H = 1: token-major), so the transposition in front of
// the attention calls costs no pass of its own.  A thread owns four neighbouring
// channels, as two pairs in two-wide instructions, and walks a run of tokens with the
// last W - 1 inputs in registers: each tensor crosses HBM once, plus W - 1 rows per run
// that come from L2.
#include "la_rows.cuh"

namespace la {
namespace {

using namespace rows;

constexpr int kThreads = 128;

struct ConvShape {
    int64_t N, xb, xt;  // x strides in elements
    int C, H;
    int64_t runs;
    int run;  // tokens per run
};

// V channels in pairs (V = 1: half a pair)
template <int V>
struct Pairs {
    static constexpr int P = (V + 1) / 2;
    float2 p[P];
};
template <typename T, int V>
__device__ __forceinline__ Pairs<V> pairs(const Raw<T, V>& r)
{
    const Vec<V> v = wide(r);
    Pairs<V> q;
    if constexpr (V == 1) {
        q.p[0] = make_float2(v.f[0], 0.0f);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            q.p[i] = make_float2(v.f[2 * i], v.f[2 * i + 1]);
    }
    return q;
}
template <typename T, int V>
__device__ __forceinline__ void store_pairs(T* p, const Pairs<V>& q)
{
    Vec<V> v;
    if constexpr (V == 1) {
        v.f[0] = q.p[0].x;
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            v.f[2 * i] = q.p[i].x, v.f[2 * i + 1] = q.p[i].y;
    }
    store(p, v);
}

// filters of V channels from weight [C][W], and their biases
template <int V, int W>
__device__ __forceinline__ void load_filter(const float* __restrict__ weight, const float* __restrict__ bias, int c,
                                            Pairs<V> (&w)[W], Pairs<V>& b)
{
    float flat[2 * Pairs<V>::P * W] = {};  // neighbouring filters are neighbours in memory
    if constexpr (V == 2) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float2 q = __ldg(reinterpret_cast<const float2*>(weight + (int64_t)c * W) + k);
            flat[2 * k] = q.x, flat[2 * k + 1] = q.y;
        }
    } else if constexpr (V == 4) {
#pragma unroll
        for (int k = 0; k < V * W / 4; ++k) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(weight + (int64_t)c * W) + k);
            flat[4 * k] = q.x, flat[4 * k + 1] = q.y, flat[4 * k + 2] = q.z, flat[4 * k + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
            flat[j] = __ldg(weight + (int64_t)c * W + j);
    }
#pragma unroll
    for (int i = 0; i < Pairs<V>::P; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            w[j].p[i] = make_float2(flat[2 * i * W + j], flat[(2 * i + 1) * W + j]);
        b.p[i] = make_float2(bias ? __ldg(bias + c + 2 * i) : 0.0f, bias && V > 1 ? __ldg(bias + c + 2 * i + 1) : 0.0f);
    }
}

// Input at position p of row b, before the first token from the window, as it lies
// in memory.
template <typename T, int V, int W>
__device__ __forceinline__ Raw<T, V> input(const T* __restrict__ x, const T* __restrict__ S0, int64_t b, int64_t p,
                                           int c, const ConvShape& s)
{
    if (p >= 0)
        return fetch<T, V>(x + b * s.xb + p * s.xt + c);
    if (S0)
        return fetch<T, V>(S0 + (b * (W - 1) + (p + W - 1)) * s.C + c);
    return none<T, V>();
}

// Where channels c .. c+V-1 of token t of row b lie in y.
__device__ __forceinline__ int64_t y_at(int64_t b, int64_t t, int c, const ConvShape& s)
{
    const int dh = s.C / s.H, h = c / dh;
    return ((b * s.H + h) * s.N + t) * dh + (c - h * dh);
}

// Tokens whose loads are issued together, one group ahead of the one in use (B4 N8192 C4096 bf16:
// four 109 us, eight 96, sixteen 111; the same bytes in fp32: four 95 us, sixteen 130).  Times in this
// file are of a call among others, device and no host; after a flush of L2, when no earlier call's
// lines wait to be written, the same kernel takes 87 us (fp32 82).
template <typename T>
constexpr int ahead()
{
    return sizeof(T) == 2 ? 8 : 4;
}

// Five blocks an SM, 96 registers: 96 us; as many registers as it likes 103, four blocks 111, six
// 106.  In three forms four or eight bytes a thread spill (fp32 with sigmoid W = 4 and silu W = 2, bf16
// with silu W = 3).
template <typename T, int V, int W, int ACT>
__global__ void __launch_bounds__(kThreads, 5)
    k_conv(const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
           T* __restrict__ y, const T* S0, T* S_out, const int* __restrict__ lengths, ConvShape s, int64_t items)
{
    constexpr int P = Pairs<V>::P, kAhead = ahead<T>();
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (item >= items)
        return;
    const int vecs = s.C / V;
    const int64_t br = item / vecs, b = br / s.runs, r = br - b * s.runs;
    const int c = (int)(item - br * vecs) * V;
    const int64_t len = row_length(lengths, b, s.N);
    Pairs<V> w[W], bs, win[W];  // win: the last W - 1 inputs, then the new one
    load_filter<V, W>(weight, bias, c, w, bs);
    const int64_t first = r * s.run, end = min(s.N, first + s.run), live = min(end, len);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t p = first - (W - 1) + j;  // not behind the row's last
        win[j] = pairs(p < len ? input<T, V, W>(x, S0, b, p, c, s) : none<T, V>());
    }
    if (r == 0 && S_out) {
        // the window after the last token; S_out may be S0, whose rows of these channels
        // this thread alone reads
        Raw<T, V> last[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            last[j] = input<T, V, W>(x, S0, b, len - (W - 1) + j, c, s);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            *reinterpret_cast<Raw<T, V>*>(S_out + (b * (W - 1) + j) * s.C + c) = last[j];
    }
    const int dh = s.C / s.H;
    const T* xp = x + b * s.xb + first * s.xt + c;
    T* yp = y + y_at(b, first, c, s);
    auto token = [&](const Raw<T, V>& in) {
        Pairs<V> o;
        win[W - 1] = pairs(in);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float2 u = bs.p[i];
#pragma unroll
            for (int j = 0; j < W; ++j)
                u = fma2(w[j].p[i], win[j].p[i], u);
            o.p[i] = value<ACT>(u);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            win[j] = win[j + 1];
        store_pairs(yp, o);
        yp += dh;
    };
    int left = (int)max((int64_t)0, live - first);
    // the next group is on its way while this one is used
    Raw<T, V> in[2][kAhead];
    auto group = [&](Raw<T, V> (&g)[kAhead]) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            g[k] = fetch<T, V>(xp + k * s.xt);
        xp += kAhead * s.xt;
    };
    if (left >= kAhead)
        group(in[0]);
    while (left >= kAhead) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (left < kAhead)
                break;
            left -= kAhead;
            if (left >= kAhead)
                group(in[half ^ 1]);
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                token(in[half][k]);
        }
    }
    for (; left > 0; --left, xp += s.xt)
        token(fetch<T, V>(xp));
    Pairs<V> zero = {};
    for (int64_t t = max(first, live); t < end; ++t, yp += dh)
        store_pairs(yp, zero);
}

// One token: y from the window and x, the window moved on in place.
template <typename T, int V, int W, int ACT>
__global__ void __launch_bounds__(kThreads)
    k_conv_step(T* __restrict__ S, const T* __restrict__ x, const float* __restrict__ weight,
                const float* __restrict__ bias, T* __restrict__ y, int64_t xb, int C, int64_t items)
{
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (item >= items)
        return;
    const int vecs = C / V;
    const int64_t b = item / vecs;
    const int c = (int)(item - b * vecs) * V;
    T* win = S + b * (W - 1) * C + c;
    Raw<T, V> in[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        in[j] = *reinterpret_cast<const Raw<T, V>*>(win + (int64_t)j * C);
    in[W - 1] = fetch<T, V>(x + b * xb + c);
    Pairs<V> w[W], u;
    load_filter<V, W>(weight, bias, c, w, u);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const Pairs<V> v = pairs(in[j]);
#pragma unroll
        for (int i = 0; i < Pairs<V>::P; ++i)
            u.p[i] = fma2(w[j].p[i], v.p[i], u.p[i]);
    }
#pragma unroll
    for (int i = 0; i < Pairs<V>::P; ++i)
        u.p[i] = value<ACT>(u.p[i]);
    store_pairs(y + b * C + c, u);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        *reinterpret_cast<Raw<T, V>*>(win + (int64_t)j * C) = in[j + 1];
}

// Gradients.  A thread walks its run forwards and holds the last W - 1 slopes du:
// dx lags W - 1 tokens behind, so a run reads that many tokens of the next one.
// dw and dbias stay in registers over all of a thread's runs; block row p leaves
// part [p][W+1][C], summed in a fixed order by k_conv_dw (no atomics).
// Bound by HBM's latency: four blocks an SM, which 128 registers allow, with two groups of
// tokens in flight (B4 N8192 C2048 bf16, sums included: three blocks 106 us, four 86, five with spills
// 120; groups of two, four and six tokens 102, 86 and 95 us; the same bytes in fp32: 81, 92 and 98).
// After a flush of L2 77 us and 4.4 for the sums.  One channel a load in bf16 spills 32 bytes, a
// few forms 4 to 12.
constexpr int kGradPerSm = 4;

template <typename T, int V, int W, int ACT>
__global__ void __launch_bounds__(kThreads, kGradPerSm)
    k_conv_grad(const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ weight,
                const float* __restrict__ bias, const T* __restrict__ S0, const T* __restrict__ dS_out,
                const int* __restrict__ lengths, T* __restrict__ dx, T* __restrict__ dS0, float* __restrict__ part,
                ConvShape s, int64_t jobs)
{
    constexpr int P = Pairs<V>::P, kAhead = sizeof(T) == 2 ? 4 : 2;
    const int c = (blockIdx.x * kThreads + threadIdx.x) * V;
    if (c >= s.C)
        return;
    Pairs<V> w[W], bs, dw[W] = {}, db = {};
    load_filter<V, W>(weight, bias, c, w, bs);
    const int dh = s.C / s.H;
    for (int64_t job = blockIdx.y; job < jobs; job += gridDim.y) {
        const int64_t b = job / s.runs, r = job - b * s.runs;
        const int64_t len = row_length(lengths, b, s.N);
        const int64_t first = r * s.run, end = min(s.N, first + s.run);
        Pairs<V> win[W], du[W] = {};  // inputs t-W+1 .. t; slopes of the same tokens
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int64_t p = first - (W - 1) + j;  // not behind the row's last: nothing is known of that
            win[j] = pairs(p < len ? input<T, V, W>(x, S0, b, p, c, s) : none<T, V>());
        }
        // From token t, its inputs x and dy, whether the row has it (behind its end the slope of
        // an infinite u would make 0 dy a NaN) and whether it is one of this run's, which alone
        // dw and dbias take (zero times an infinite input of the window would be a NaN): du_t, and
        // dx of the token W - 1 before.
        auto token = [&](const Raw<T, V>& xin, const Raw<T, V>& din, bool on, bool own) {
            win[W - 1] = pairs(xin);
            const Pairs<V> d = pairs(din);
            Pairs<V> o;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float2 u = bs.p[i];
#pragma unroll
                for (int j = 0; j < W; ++j)
                    u = fma2(w[j].p[i], win[j].p[i], u);
                const float2 g = on ? mul2(d.p[i], slope<ACT>(u)) : both(0.0f);
                if (on && own) {
                    db.p[i] = add2(db.p[i], g);
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        dw[j].p[i] = fma2(g, win[j].p[i], dw[j].p[i]);
                }
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    du[j].p[i] = du[j + 1].p[i], win[j].p[i] = win[j + 1].p[i];
                du[W - 1].p[i] = g;
                o.p[i] = mul2(w[W - 1].p[i], du[0].p[i]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    o.p[i] = fma2(w[j].p[i], du[W - 1 - j].p[i], o.p[i]);
            }
            return o;
        };
        const T* xp = x + b * s.xb + first * s.xt + c;
        const T* dp = dy + y_at(b, first, c, s);
        T* out = dx + (b * s.N + first) * s.C + c;
        // the edges: a run's first W - 1 tokens, of which the row's first run passes what lies
        // before them to the window, and its end, where tokens may be missing, dx may end and
        // the final window (positions len - W + 1 .. len - 1) adds its gradient
        auto edge = [&](int64_t t) {
            const bool on = t < len && t < s.N;
            Pairs<V> o = token(on ? fetch<T, V>(xp) : none<T, V>(), on ? fetch<T, V>(dp) : none<T, V>(), on, t < end);
            xp += s.xt, dp += dh;
            const int64_t at = t - (W - 1), row = at - (len - (W - 1));
            if (at < first && (r > 0 || !dS0))
                return;
            if (dS_out && row >= 0 && row < W - 1) {
                const Pairs<V> g = pairs(fetch<T, V>(dS_out + (b * (W - 1) + row) * s.C + c));
#pragma unroll
                for (int i = 0; i < P; ++i)
                    o.p[i] = add2(o.p[i], g.p[i]);
            }
            if (at >= first) {
                store_pairs(out, o);
                out += s.C;
            } else {
                store_pairs(dS0 + (b * (W - 1) + at + W - 1) * s.C + c, o);
            }
        };
        int64_t t = first;
        for (; t < first + W - 1; ++t)
            edge(t);
        // whole groups of tokens of this run, none of them near the row's end
        Raw<T, V> xin[2][kAhead], din[2][kAhead];
        auto group = [&](Raw<T, V> (&a)[kAhead], Raw<T, V> (&b)[kAhead]) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                a[k] = fetch<T, V>(xp), b[k] = fetch<T, V>(dp);
                xp += s.xt, dp += dh;
            }
        };
        int left = (int)(max(t, min(end, len)) - t);
        if (left >= kAhead)
            group(xin[0], din[0]);
        while (left >= kAhead) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (left < kAhead)
                    break;
                left -= kAhead, t += kAhead;
                if (left >= kAhead)
                    group(xin[half ^ 1], din[half ^ 1]);
#pragma unroll
                for (int k = 0; k < kAhead; ++k, out += s.C)
                    store_pairs(out, token(xin[half][k], din[half][k], true, true));
            }
        }
        for (; t < end + W - 1; ++t)
            edge(t);
    }
    float* p = part + (int64_t)blockIdx.y * (W + 1) * s.C + c;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        const Pairs<V>& q = j < W ? dw[j < W ? j : 0] : db;
        store_pairs(p + (int64_t)j * s.C, q);
    }
}

// dw [C][W] and dbias [C] from the parts: 32 channels x 32 partial sums per block.
__global__ void __launch_bounds__(1024)
    k_conv_dw(const float* __restrict__ part, float* __restrict__ dw, float* __restrict__ dbias, int parts, int W,
              int C)
{
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, j = blockIdx.y;
    float x = 0.f;
    if (c < C) {
#pragma unroll 4
        for (int p = grp; p < parts; p += 32)
            x += part[((int64_t)p * (W + 1) + j) * C + c];
    }
    sums[grp][lane] = x;
    __syncthreads();
    if (grp == 0 && c < C) {
        x = 0.f;
        for (int i = 0; i < 32; ++i)
            x += sums[i][lane];
        if (j < W)
            dw[(int64_t)c * W + j] = x;
        else if (dbias)
            dbias[c] = x;
    }
}

// Tokens per run of the forward: long enough that the W - 1 rows read twice are few (B4 N8192 C4096
// bf16: runs of 32 tokens 105 us, 64 97, 128 and 256 96), short enough that the GPU is full (B64 N256
// C4096: runs until there are 152 * 1024 threads 53 us, a quarter or half as many 58, twice 57).
// The other side: a call as small as B1 N1024 C2048 has runs of four tokens, which load one after the
// other, and takes 10 us where runs of eight would take 6.
int run_length(const ConvArgs& a, int vec)
{
    const int64_t vecs = a.C / vec * a.B;
    int run = 128;
    while (run > 4 && vecs * ((a.N + run - 1) / run) < 152 * 1024)
        run /= 2;
    return run;
}

// Block rows of the gradient, four blocks an SM in all, and their runs: one for each where
// there are no more sequences than block rows, eight tokens at least.
int64_t grad_rows(const ConvArgs& a, int vec)
{
    const int64_t wide = vec * kThreads, cols = (a.C + wide - 1) / wide, rows = kGradPerSm * 152 / cols;
    return rows > 1 ? rows : 1;
}
int grad_run(const ConvArgs& a, int64_t rows)
{
    const int64_t runs = rows > a.B ? rows / a.B : 1, run = (a.N + runs - 1) / runs;
    return (int)(run > 8 ? run : 8);
}

// Channels of a load, as many as rows and heads allow (bf16, forward of B4 N8192 C4096: four 96 us,
// two 129, one 148; gradient of C2048 86, 125 and 227 us; fp32 95, 93 and 95, gradient 81, 96 and 162).
int width(const ConvArgs& a, int es, bool step)
{
    for (int v = 4; v > 1; v /= 2)
        if (a.C / a.H % v == 0 && rows_on(a.x, a.xb, step ? 0 : a.xt, es, v * es))
            return v;
    return 1;
}

template <typename T, int V, int W, int ACT>
cudaError_t run_conv(const ConvArgs& a, int mode)
{
    const T *x = static_cast<const T*>(a.x), *S0 = static_cast<const T*>(a.S0);
    if (mode == 1) {
        const int64_t items = a.B * (a.C / V);
        k_conv_step<T, V, W, ACT><<<(unsigned)((items + kThreads - 1) / kThreads), kThreads, 0, a.stream>>>(
            static_cast<T*>(a.S_out), x, a.weight, a.bias, static_cast<T*>(a.y), a.xb, (int)a.C, items);
        count_launches(1);
        return cudaGetLastError();
    }
    ConvShape s;
    const int64_t rows = grad_rows(a, V);
    s.N = a.N, s.xb = a.xb, s.xt = a.xt, s.C = (int)a.C, s.H = (int)a.H;
    s.run = mode == 0 ? run_length(a, V) : grad_run(a, rows);
    s.runs = (a.N + s.run - 1) / s.run;
    const int64_t jobs = a.B * s.runs;
    if (mode == 0) {
        const int64_t items = jobs * (a.C / V);
        k_conv<T, V, W, ACT><<<(unsigned)((items + kThreads - 1) / kThreads), kThreads, 0, a.stream>>>(
            x, a.weight, a.bias, static_cast<T*>(a.y), S0, static_cast<T*>(a.S_out), a.lengths, s, items);
        count_launches(1);
        return cudaGetLastError();
    }
    const int parts = (int)(rows < jobs ? rows : jobs);
    const dim3 grid((unsigned)((a.C / V + kThreads - 1) / kThreads), (unsigned)parts);
    float* part = static_cast<float*>(a.ws);
    k_conv_grad<T, V, W, ACT><<<grid, kThreads, 0, a.stream>>>(
        static_cast<const T*>(a.dy), x, a.weight, a.bias, S0, static_cast<const T*>(a.dS_out), a.lengths,
        static_cast<T*>(a.dx), static_cast<T*>(a.dS0), part, s, jobs);
    count_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    k_conv_dw<<<dim3((unsigned)((a.C + 31) / 32), W + 1), 1024, 0, a.stream>>>(part, a.dweight, a.dbias, parts, W,
                                                                               (int)a.C);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, int V, int W>
cudaError_t conv_act(const ConvArgs& a, int mode)
{
    switch (a.act) {
    case LA_ACT_SILU: return run_conv<T, V, W, LA_ACT_SILU>(a, mode);
    case LA_ACT_SIGMOID: return run_conv<T, V, W, LA_ACT_SIGMOID>(a, mode);
    default: return run_conv<T, V, W, LA_ACT_NONE>(a, mode);
    }
}

template <typename T, int V>
cudaError_t conv_taps(const ConvArgs& a, int mode)
{
    switch (a.W) {
    case 2: return conv_act<T, V, 2>(a, mode);
    case 3: return conv_act<T, V, 3>(a, mode);
    default: return conv_act<T, V, 4>(a, mode);
    }
}

template <typename T>
cudaError_t conv_widths(const ConvArgs& a, int mode)
{
    switch (width(a, (int)sizeof(T), mode == 1)) {
    case 4: return conv_taps<T, 4>(a, mode);
    case 2: return conv_taps<T, 2>(a, mode);
    default: return conv_taps<T, 1>(a, mode);
    }
}

cudaError_t conv_types(const ConvArgs& a, int mode)
{
    return a.dtype == LA_BF16 ? conv_widths<__nv_bfloat16>(a, mode) : conv_widths<float>(a, mode);
}

}  // namespace

// A part for every block row of the launch.  Block rows are most with four channels a thread
// (fewest column blocks), whatever width the launch then takes.
size_t conv_backward_workspace(const ConvArgs& a)
{
    const int64_t rows = grad_rows(a, 4);
    return sizeof(float) * (size_t)rows * (a.W + 1) * a.C;
}

cudaError_t conv_forward(const ConvArgs& a) { return conv_types(a, 0); }
cudaError_t conv_step(const ConvArgs& a) { return conv_types(a, 1); }
cudaError_t conv_backward(const ConvArgs& a) { return conv_types(a, 2); }

}  // namespace la
