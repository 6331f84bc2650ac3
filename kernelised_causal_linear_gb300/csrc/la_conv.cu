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
// the attention calls costs no pass of its own.  A thread owns a vector of
// channels and walks a run of tokens with the last W - 1 inputs in registers: each
// tensor crosses HBM once, plus W - 1 rows per run that come from L2.
#include "la_rows.cuh"

namespace la {
namespace {

using namespace rows;

constexpr int kThreads = 128;
constexpr int kAhead = 4;  // tokens whose loads are in flight together

struct ConvShape {
    int64_t N, xb, xt;  // x strides in elements
    int C, H;
    int64_t runs;
    int run;  // tokens per run, a multiple of kAhead
    int act;
};

// filters of V channels from weight [C][W]
template <int V, int W>
__device__ __forceinline__ void load_filter(const float* __restrict__ weight, const float* __restrict__ bias, int c,
                                            float (&w)[W][V], float (&b)[V])
{
    if constexpr (V > 1) {
        float flat[V * W];  // neighbouring filters are neighbours in memory
#pragma unroll
        for (int k = 0; k < V * W / 4; ++k) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(weight + (int64_t)c * W) + k);
            flat[4 * k] = q.x, flat[4 * k + 1] = q.y, flat[4 * k + 2] = q.z, flat[4 * k + 3] = q.w;
        }
#pragma unroll
        for (int k = 0; k < V * W; ++k)
            w[k % W][k / W] = flat[k];
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
            w[j][0] = __ldg(weight + (int64_t)c * W + j);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        b[i] = bias ? __ldg(bias + c + i) : 0.0f;
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

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
    k_conv(const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
           T* __restrict__ y, const T* S0, T* S_out, const int* __restrict__ lengths, ConvShape s, int64_t items)
{
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (item >= items)
        return;
    const int vecs = s.C / V;
    const int64_t br = item / vecs, b = br / s.runs, r = br - b * s.runs;
    const int c = (int)(item - br * vecs) * V;
    const int64_t len = row_length(lengths, b, s.N);
    float w[W][V], bs[V];
    load_filter<V, W>(weight, bias, c, w, bs);
    int64_t t = r * s.run;
    const int64_t end = min(s.N, t + s.run), live = min(end, len);
    float win[W][V];  // the last W - 1 inputs, then the new one
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const Vec<V> v = wide(input<T, V, W>(x, S0, b, t - (W - 1) + j, c, s));
#pragma unroll
        for (int i = 0; i < V; ++i)
            win[j][i] = v.f[i];
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
    const T* xp = x + b * s.xb + t * s.xt + c;
    T* yp = y + y_at(b, t, c, s);
    const int dh = s.C / s.H;
    for (; t < live; t += kAhead, xp += kAhead * s.xt, yp += kAhead * dh) {
        Raw<T, V> in[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            in[k] = t + k < live ? fetch<T, V>(xp + k * s.xt) : none<T, V>();
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const Vec<V> v = wide(in[k]);
            Vec<V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                win[W - 1][i] = v.f[i];
                float u = bs[i];
#pragma unroll
                for (int j = 0; j < W; ++j)
                    u = fmaf(w[j][i], win[j][i], u);
                o.f[i] = t + k < live ? activated(u, s.act) : 0.0f;
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    win[j][i] = win[j + 1][i];
            }
            if (t + k < end)
                store(yp + k * dh, o);
        }
    }
    Vec<V> zero;
#pragma unroll
    for (int i = 0; i < V; ++i)
        zero.f[i] = 0.0f;
    for (; t < end; ++t, yp += dh)
        store(yp, zero);
}

// One token: y from the window and x, the window moved on in place.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
    k_conv_step(T* __restrict__ S, const T* __restrict__ x, const float* __restrict__ weight,
                const float* __restrict__ bias, T* __restrict__ y, int64_t xb, int C, int act, int64_t items)
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
    float w[W][V], u[V];
    load_filter<V, W>(weight, bias, c, w, u);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const Vec<V> v = wide(in[j]);
#pragma unroll
        for (int i = 0; i < V; ++i)
            u[i] = fmaf(w[j][i], v.f[i], u[i]);
    }
    Vec<V> o;
#pragma unroll
    for (int i = 0; i < V; ++i)
        o.f[i] = activated(u[i], act);
    store(y + b * C + c, o);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        *reinterpret_cast<Raw<T, V>*>(win + (int64_t)j * C) = in[j + 1];
}

// Gradients.  A thread walks its runs forwards and holds the last W - 1 slopes du:
// dx lags W - 1 tokens behind, so a run reads that many tokens of the next one.
// dw and dbias stay in registers over all of a thread's runs; block row p leaves
// part [p][W+1][C], summed in a fixed order by k_conv_dw (no atomics).
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
    k_conv_grad(const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ weight,
                const float* __restrict__ bias, const T* __restrict__ S0, const T* __restrict__ dS_out,
                const int* __restrict__ lengths, T* __restrict__ dx, T* __restrict__ dS0, float* __restrict__ part,
                ConvShape s, int64_t jobs)
{
    const int c = (blockIdx.x * kThreads + threadIdx.x) * V;
    if (c >= s.C)
        return;
    float w[W][V], bs[V], dw[W][V], db[V];
    load_filter<V, W>(weight, bias, c, w, bs);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j)
            dw[j][i] = 0.0f;
    }
    const int dh = s.C / s.H;
    for (int64_t job = blockIdx.y; job < jobs; job += gridDim.y) {
        const int64_t b = job / s.runs, r = job - b * s.runs;
        const int64_t len = row_length(lengths, b, s.N);
        const int64_t first = r * s.run, end = min(s.N, first + s.run);
        float win[W][V], du[W][V];  // inputs t-W+1 .. t; slopes of the same tokens
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int64_t p = first - (W - 1) + j;  // not behind the row's last: nothing is known of that
            const Vec<V> v = wide(p < len ? input<T, V, W>(x, S0, b, p, c, s) : none<T, V>());
#pragma unroll
            for (int i = 0; i < V; ++i)
                win[j][i] = v.f[i], du[j + 1][i] = 0.0f;
        }
        const T* xp = x + b * s.xb + c;
        const T* dp = dy + y_at(b, 0, c, s);
        T* out = dx + b * s.N * s.C + c;
        // token t gives du_t and, W - 1 behind, dx; the row's first run also walks back
        // into the window (positions before 0)
        for (int64_t t = first; t < end + W - 1; t += kAhead) {
            Raw<T, V> xin[kAhead], din[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const bool on = t + k < len && t + k < end + W - 1;
                xin[k] = on ? fetch<T, V>(xp + (t + k) * s.xt) : none<T, V>();
                din[k] = on ? fetch<T, V>(dp + (t + k) * dh) : none<T, V>();
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const Vec<V> v = wide(xin[k]), d = wide(din[k]);
                Vec<V> o;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    win[W - 1][i] = v.f[i];
                    float u = bs[i];
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        u = fmaf(w[j][i], win[j][i], u);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j)
                        du[j][i] = du[j + 1][i];
                    const float g = t + k < len ? d.f[i] * activate(u, s.act).y : 0.0f;
                    du[W - 1][i] = g;
                    if (t + k < end) {
                        db[i] += g;
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            dw[j][i] = fmaf(g, win[j][i], dw[j][i]);
                    }
                    o.f[i] = 0.0f;
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        o.f[i] = fmaf(w[j][i], du[W - 1 - j][i], o.f[i]);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j)
                        win[j][i] = win[j + 1][i];
                }
                const int64_t at = t + k - (W - 1);
                if (at >= end || (at < first && (r > 0 || !dS0)))
                    continue;
                // the final window holds positions len - W + 1 .. len - 1
                const int64_t row = at - (len - (W - 1));
                if (dS_out && row >= 0 && row < W - 1) {
                    const Vec<V> g = wide(fetch<T, V>(dS_out + (b * (W - 1) + row) * s.C + c));
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        o.f[i] += g.f[i];
                }
                if (at >= first)
                    store(out + at * s.C, o);
                else if (at >= -(W - 1))
                    store(dS0 + (b * (W - 1) + at + W - 1) * s.C + c, o);
            }
        }
    }
    float* p = part + (int64_t)blockIdx.y * (W + 1) * s.C + c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        p[(int64_t)W * s.C + i] = db[i];
#pragma unroll
        for (int j = 0; j < W; ++j)
            p[(int64_t)j * s.C + i] = dw[j][i];
    }
}

// dw [C][W] and dbias [C] from the parts: 32 channels x 8 partial sums per block.
__global__ void __launch_bounds__(256)
    k_conv_dw(const float* __restrict__ part, float* __restrict__ dw, float* __restrict__ dbias, int parts, int W,
              int C)
{
    __shared__ float sums[8][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, j = blockIdx.y;
    float x = 0.f;
    if (c < C) {
#pragma unroll 4
        for (int p = grp; p < parts; p += 8)
            x += part[((int64_t)p * (W + 1) + j) * C + c];
    }
    sums[grp][lane] = x;
    __syncthreads();
    if (grp == 0 && c < C) {
        x = 0.f;
        for (int i = 0; i < 8; ++i)
            x += sums[i][lane];
        if (j < W)
            dw[(int64_t)c * W + j] = x;
        else if (dbias)
            dbias[c] = x;
    }
}

// Tokens per run: long enough that the W - 1 rows read twice are few, short enough
// that the GPU is full.
int run_length(const ConvArgs& a, int vec)
{
    const int64_t vecs = a.C / vec * a.B;
    int run = 64;
    while (run > kAhead && vecs * ((a.N + run - 1) / run) < 152 * 1024)
        run /= 2;
    return run;
}

bool vectors(const ConvArgs& a, int es, bool step)
{
    const int v = 16 / es;
    return a.C % v == 0 && (a.C / a.H) % v == 0 && rows16(a.x, a.xb, step ? 0 : a.xt, es);
}

// Block rows of the gradient, for any vector width: the parts are sized by them.
int64_t grad_rows(const ConvArgs& a, int vec, int64_t jobs)
{
    const int64_t cols = (a.C / vec + kThreads - 1) / kThreads;
    const int64_t want = (152 * 4 + cols - 1) / cols;
    return want < jobs ? want : jobs;
}

ConvShape shape_of(const ConvArgs& a, int run)
{
    ConvShape s;
    s.N = a.N, s.xb = a.xb, s.xt = a.xt, s.C = (int)a.C, s.H = (int)a.H, s.run = run;
    s.runs = (a.N + run - 1) / run, s.act = a.act;
    return s;
}

template <typename T, int V, int W>
cudaError_t run_conv(const ConvArgs& a, int mode)
{
    const T *x = static_cast<const T*>(a.x), *S0 = static_cast<const T*>(a.S0);
    if (mode == 1) {
        const int64_t items = a.B * (a.C / V);
        k_conv_step<T, V, W><<<(unsigned)((items + kThreads - 1) / kThreads), kThreads, 0, a.stream>>>(
            static_cast<T*>(a.S_out), x, a.weight, a.bias, static_cast<T*>(a.y), a.xb, (int)a.C, a.act, items);
        count_launches(1);
        return cudaGetLastError();
    }
    const ConvShape s = shape_of(a, run_length(a, V));
    const int64_t jobs = a.B * s.runs;
    if (mode == 0) {
        const int64_t items = jobs * (a.C / V);
        k_conv<T, V, W><<<(unsigned)((items + kThreads - 1) / kThreads), kThreads, 0, a.stream>>>(
            x, a.weight, a.bias, static_cast<T*>(a.y), S0, static_cast<T*>(a.S_out), a.lengths, s, items);
        count_launches(1);
        return cudaGetLastError();
    }
    const int rows = (int)grad_rows(a, V, jobs);
    const dim3 grid((unsigned)((a.C / V + kThreads - 1) / kThreads), (unsigned)rows);
    float* part = static_cast<float*>(a.ws);
    k_conv_grad<T, V, W><<<grid, kThreads, 0, a.stream>>>(
        static_cast<const T*>(a.dy), x, a.weight, a.bias, S0, static_cast<const T*>(a.dS_out), a.lengths,
        static_cast<T*>(a.dx), static_cast<T*>(a.dS0), part, s, jobs);
    count_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    k_conv_dw<<<dim3((unsigned)((a.C + 31) / 32), W + 1), 256, 0, a.stream>>>(part, a.dweight, a.dbias, rows, W,
                                                                              (int)a.C);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t conv_taps(const ConvArgs& a, int mode)
{
    switch (a.W) {
    case 2: return run_conv<T, V, 2>(a, mode);
    case 3: return run_conv<T, V, 3>(a, mode);
    default: return run_conv<T, V, 4>(a, mode);
    }
}

cudaError_t conv_types(const ConvArgs& a, int mode)
{
    if (a.dtype == LA_BF16)
        return vectors(a, 2, mode == 1) ? conv_taps<__nv_bfloat16, 8>(a, mode) : conv_taps<__nv_bfloat16, 1>(a, mode);
    return vectors(a, 4, mode == 1) ? conv_taps<float, 4>(a, mode) : conv_taps<float, 1>(a, mode);
}

}  // namespace

// Block rows are most with the widest vectors (fewest column blocks).
size_t conv_backward_workspace(const ConvArgs& a)
{
    const int vec = a.dtype == LA_BF16 ? 8 : 4;
    const int64_t cols = (a.C / vec + kThreads - 1) / kThreads;
    const int64_t most = 152 * 4 / (cols > 0 ? cols : 1) + 1, jobs = a.B * ((a.N + kAhead - 1) / kAhead);
    return sizeof(float) * (size_t)(most < jobs ? most : jobs) * (a.W + 1) * a.C;
}

cudaError_t conv_forward(const ConvArgs& a) { return conv_types(a, 0); }
cudaError_t conv_step(const ConvArgs& a) { return conv_types(a, 1); }
cudaError_t conv_backward(const ConvArgs& a) { return conv_types(a, 2); }

}  // namespace la
