// la_api.cu -- the C ABI of liblinattn.so: argument checks, dispatch, status.
//
// Every entry point validates its arguments before anything is enqueued and
// never allocates: scratch is the caller's workspace, and the only
// library-owned device object is the per-device status word below, a static
// __device__ variable that exists as soon as the module is loaded.
#include <atomic>
#include <math.h>
#include <mutex>

#include "la_internal.cuh"

namespace la {
__device__ int g_device_status;  // LA_OK, or the first device-side error code

static std::atomic<uint64_t> g_launches{0};
void count_launches(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_status_mu;
int* g_status_ptr[kMaxDevices];

// Device address of the status word for the current device (looked up once).
int* status_ptr()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return nullptr;
    std::lock_guard<std::mutex> lk(g_status_mu);
    if (!g_status_ptr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess)
            return nullptr;
        g_status_ptr[dev] = static_cast<int*>(p);
    }
    return g_status_ptr[dev];
}

bool dim_ok(int x) { return x == 32 || x == 64 || x == 128; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Workspaces hold 128-byte lines that kernels drop from L2 and 1024-byte
// aligned TMA regions laid out from the base, so the base must be 256-aligned.
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

la_status check_sizes(int64_t B, int64_t H, int64_t N, int d, int dv, int fm, int dtype)
{
    if (B < 1 || H < 1 || N < 0 || d < 1 || dv < 1)
        return LA_ERR_INVALID_ARG;
    if (fm != LA_FM_ELU1 && fm != LA_FM_IDENTITY_NORM && fm != LA_FM_NONE)
        return LA_ERR_INVALID_ARG;
    if (dtype != LA_BF16 && dtype != LA_FP32)
        return LA_ERR_INVALID_ARG;
    if (!dim_ok(d) || !dim_ok(dv))
        return LA_ERR_UNSUPPORTED;
    if (B > INT32_MAX / H)
        return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

// Fill the by-value decay table; NULL gamma means no decay.
la_status make_gamma(const float* gamma, int64_t H, GammaTable* t)
{
    t->has_decay = 0;
    t->H = (int)(H < kMaxGammaHeads ? H : kMaxGammaHeads);
    if (!gamma)
        return LA_OK;
    if (H > kMaxGammaHeads)
        return LA_ERR_UNSUPPORTED;
    for (int64_t h = 0; h < H; ++h) {
        const float gm = gamma[h];
        if (!(gm > 0.0f && gm <= 1.0f))
            return LA_ERR_INVALID_ARG;
        t->g[h] = gm;
        t->log2g[h] = (float)log2((double)gm);
    }
    t->has_decay = 1;
    return LA_OK;
}

la_status from_cuda(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

int la_version(void) { return 100; }  // 0.1.0

const char* la_status_string(la_status s)
{
    switch (s) {
    case LA_OK: return "LA_OK: success";
    case LA_ERR_INVALID_ARG: return "LA_ERR_INVALID_ARG: invalid argument (pointer, size, enum or gamma)";
    case LA_ERR_UNSUPPORTED: return "LA_ERR_UNSUPPORTED: valid request outside what is implemented";
    case LA_ERR_CUDA: return "LA_ERR_CUDA: a CUDA runtime call or kernel launch failed";
    case LA_ERR_TIMEOUT: return "LA_ERR_TIMEOUT: a bounded device-side wait gave up";
    case LA_ERR_DEVICE_CHECK: return "LA_ERR_DEVICE_CHECK: a device-side consistency check failed";
    case LA_ERR_WORKSPACE: return "LA_ERR_WORKSPACE: workspace missing or too small";
    case LA_ERR_TOO_LARGE:
        return "LA_ERR_TOO_LARGE: sizes need more scratch than la_forward_noalloc's fixed array";
    }
    return "unknown la_status";
}

// The kernel paths, in order of preference: the single-pass tcgen05 kernel
// (bf16, d = dv = 64, causal, no decay, no state in or out), the chunked
// tcgen05 path (bf16, d and dv in {64, 128}), the CUDA-core path.
enum Path { PATH_TC = 0, PATH_TG = 1, PATH_SIMT = 2 };

static Path choose_path(const FwdArgs& a)
{
    if (a.out && !a.S0 && !a.S_out && tc_forward_eligible(a))
        return PATH_TC;
    if (tg_eligible(a))
        return PATH_TG;
    return PATH_SIMT;
}

static FwdArgs probe_args(int64_t B, int64_t H, int64_t N, int d, int dv, int causal, int fm,
                          int dtype, GammaTable* g, bool out, bool state)
{
    FwdArgs a{};
    a.B = B, a.H = H, a.N = N, a.d = d, a.dv = dv, a.causal = causal, a.fm = fm;
    a.dtype = dtype, a.gamma = g;
    // placeholders that only mark which results are wanted
    a.out = out ? reinterpret_cast<float*>(uintptr_t(256)) : nullptr;
    a.S_out = state ? reinterpret_cast<float*>(uintptr_t(256)) : nullptr;
    return a;
}

static size_t path_workspace(const FwdArgs& a, Path path)
{
    switch (path) {
    case PATH_TC: return tc_forward_workspace(a.B * a.H, a.N);
    case PATH_TG: return tg_workspace(a.B * a.H, a.N, a.d, a.dv, a.fm, a.causal);
    default:
        return a.out ? simt_forward_workspace(a.B * a.H, a.N, a.d, a.dv, a.causal)
                     : simt_state_workspace(a.B * a.H, a.N, a.d, a.dv);
    }
}

// Workspace that covers every path a call with these sizes may take (the
// feature map and the decay are not known here).
static size_t max_workspace(int64_t B, int64_t H, int64_t N, int d, int dv, int causal,
                            int dtype, bool out, bool state)
{
    size_t n = 0;
    for (int fm = 0; fm < 3; ++fm)
        for (int decay = 0; decay < 2; ++decay) {
            GammaTable g{};
            g.has_decay = decay;
            const FwdArgs a = probe_args(B, H, N, d, dv, causal, fm, dtype, &g, out, state);
            const size_t w = path_workspace(a, choose_path(a));
            n = w > n ? w : n;
        }
    return n;
}

size_t la_forward_workspace_size(int64_t B, int64_t H, int64_t N, int d, int dv, int causal,
                                 int dtype)
{
    if (check_sizes(B, H, N, d, dv, LA_FM_ELU1, dtype) != LA_OK || N == 0)
        return 0;
    // the forward alone, and with states in or out (causal only)
    size_t n = max_workspace(B, H, N, d, dv, causal, dtype, true, false);
    if (causal) {
        const size_t w = max_workspace(B, H, N, d, dv, causal, dtype, true, true);
        n = w > n ? w : n;
    }
    return n;
}

const char* la_forward_path(int64_t B, int64_t H, int64_t N, int d, int dv, int causal,
                            int feature_map, int has_decay, int dtype)
{
    if (check_sizes(B, H, N, d, dv, feature_map, dtype) != LA_OK)
        return "invalid";
    GammaTable g{};
    g.has_decay = has_decay;
    const FwdArgs a = probe_args(B, H, N, d, dv, causal, feature_map, dtype, &g, true, false);
    switch (choose_path(a)) {
    case PATH_TC: return "tcgen05";
    case PATH_TG: return "tcgen05_chunked";
    default: return "simt";
    }
}

size_t la_state_workspace_size(int64_t B, int64_t H, int64_t N, int d, int dv, int dtype)
{
    if (check_sizes(B, H, N, d, dv, LA_FM_ELU1, dtype) != LA_OK || N == 0)
        return 0;
    return max_workspace(B, H, N, d, dv, 1, dtype, false, true);
}

// Runs a validated forward and/or state request on its path.
static la_status run_path(const FwdArgs& a)
{
    const Path path = choose_path(a);
    const size_t need = path_workspace(a, path);
    if (!a.ws || a.ws_bytes < need || !aligned256(a.ws))
        return LA_ERR_WORKSPACE;
    switch (path) {
    case PATH_TC: return from_cuda(tc_forward(a));
    case PATH_TG: return from_cuda(tg_run(a));
    default: return from_cuda(a.out ? simt_forward(a) : simt_state(a));
    }
}

la_status la_forward(const void* q, const void* k, const void* v, float* out, int64_t B,
                     int64_t H, int64_t N, int d, int dv, int causal, int feature_map,
                     const float* gamma, int dtype, void* workspace, size_t workspace_bytes,
                     la_stream_t stream)
{
    la_status st = check_sizes(B, H, N, d, dv, feature_map, dtype);
    if (st != LA_OK)
        return st;
    if (causal != 0 && causal != 1)
        return LA_ERR_INVALID_ARG;
    if (!causal && gamma)
        return LA_ERR_UNSUPPORTED;  // decay is defined only for the causal form
    GammaTable gt;
    if ((st = make_gamma(gamma, H, &gt)) != LA_OK)
        return st;
    if (N == 0)
        return LA_OK;
    if (!q || !k || !v || !out)
        return LA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
        return LA_ERR_INVALID_ARG;
    FwdArgs a{};
    a.q = q, a.k = k, a.v = v, a.out = out;
    a.B = B, a.H = H, a.N = N, a.d = d, a.dv = dv;
    a.causal = causal, a.fm = feature_map, a.dtype = dtype;
    a.gamma = &gt;
    a.ws = workspace, a.ws_bytes = workspace_bytes;
    a.status = status_ptr();
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return run_path(a);
}

la_status la_forward_with_state(const void* q, const void* k, const void* v, float* out,
                                const float* S0, const float* z0, float* S_out, float* z_out,
                                int64_t B, int64_t H, int64_t N, int d, int dv, int feature_map,
                                const float* gamma, int dtype, void* workspace,
                                size_t workspace_bytes, la_stream_t stream)
{
    la_status st = check_sizes(B, H, N, d, dv, feature_map, dtype);
    if (st != LA_OK)
        return st;
    GammaTable gt;
    if ((st = make_gamma(gamma, H, &gt)) != LA_OK)
        return st;
    if (!S0 != !z0 || !S_out != !z_out || (!out && !S_out) || (!q != !out))
        return LA_ERR_INVALID_ARG;
    if ((S0 && (!aligned16(S0) || !aligned16(z0))) ||
        (S_out && (!aligned16(S_out) || !aligned16(z_out))))
        return LA_ERR_INVALID_ARG;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) {  // no tokens: the final state is the initial one
        if (!S_out)
            return LA_OK;
        const size_t sb = sizeof(float) * (size_t)(B * H) * d * dv;
        const size_t zb = sizeof(float) * (size_t)(B * H) * d;
        cudaError_t e;
        if (S0) {
            e = S0 == S_out ? cudaSuccess : cudaMemcpyAsync(S_out, S0, sb, cudaMemcpyDeviceToDevice, cs);
            if (e == cudaSuccess && z0 != z_out)
                e = cudaMemcpyAsync(z_out, z0, zb, cudaMemcpyDeviceToDevice, cs);
        } else {
            e = cudaMemsetAsync(S_out, 0, sb, cs);
            if (e == cudaSuccess)
                e = cudaMemsetAsync(z_out, 0, zb, cs);
        }
        return from_cuda(e);
    }
    if (!k || !v || !aligned16(k) || !aligned16(v))
        return LA_ERR_INVALID_ARG;
    if (out && (!aligned16(q) || !aligned16(out)))
        return LA_ERR_INVALID_ARG;
    FwdArgs a{};
    a.q = q, a.k = k, a.v = v, a.out = out;
    a.B = B, a.H = H, a.N = N, a.d = d, a.dv = dv;
    a.causal = 1, a.fm = feature_map, a.dtype = dtype;
    a.gamma = &gt;
    a.ws = workspace, a.ws_bytes = workspace_bytes;
    a.S0 = S0, a.z0 = z0, a.S_out = S_out, a.z_out = z_out;
    a.status = status_ptr();
    a.stream = cs;
    return run_path(a);
}

la_status la_state(const void* k, const void* v, float* S, float* z, int64_t B, int64_t H,
                   int64_t N, int d, int dv, int feature_map, const float* gamma, int dtype,
                   void* workspace, size_t workspace_bytes, la_stream_t stream)
{
    la_status st = check_sizes(B, H, N, d, dv, feature_map, dtype);
    if (st != LA_OK)
        return st;
    GammaTable gt;
    if ((st = make_gamma(gamma, H, &gt)) != LA_OK)
        return st;
    if (!S || !z || !aligned16(S) || !aligned16(z))
        return LA_ERR_INVALID_ARG;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) {
        cudaError_t e = cudaMemsetAsync(S, 0, sizeof(float) * (size_t)(B * H) * d * dv, cs);
        if (e == cudaSuccess)
            e = cudaMemsetAsync(z, 0, sizeof(float) * (size_t)(B * H) * d, cs);
        return from_cuda(e);
    }
    if (!k || !v || !aligned16(k) || !aligned16(v))
        return LA_ERR_INVALID_ARG;
    FwdArgs a{};
    a.k = k, a.v = v;
    a.B = B, a.H = H, a.N = N, a.d = d, a.dv = dv;
    a.causal = 1, a.fm = feature_map, a.dtype = dtype;
    a.gamma = &gt;
    a.ws = workspace, a.ws_bytes = workspace_bytes;
    a.S_out = S, a.z_out = z;
    a.status = status_ptr();
    a.stream = cs;
    return run_path(a);
}

la_status la_decode_step(float* S, float* z, const void* q, const void* k, const void* v,
                         float* out, int64_t B, int64_t H, int d, int dv, int feature_map,
                         const float* gamma, int dtype, la_stream_t stream)
{
    la_status st = check_sizes(B, H, 1, d, dv, feature_map, dtype);
    if (st != LA_OK)
        return st;
    GammaTable gt;
    if ((st = make_gamma(gamma, H, &gt)) != LA_OK)
        return st;
    if (!S || !z || !q || !k || !v || !out)
        return LA_ERR_INVALID_ARG;
    if (!aligned16(S) || !aligned16(z) || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
        !aligned16(out))
        return LA_ERR_INVALID_ARG;
    DecodeArgs a{};
    a.S = S, a.z = z, a.q = q, a.k = k, a.v = v, a.out = out;
    a.BH = B * H, a.H = H, a.d = d, a.dv = dv, a.fm = feature_map, a.dtype = dtype;
    a.gamma = &gt;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(decode_step(a));
}

size_t la_gla_workspace_size(int64_t B, int64_t H, int64_t N, int d, int dv)
{
    if (check_sizes(B, H, N, d, dv, LA_FM_ELU1, LA_FP32) != LA_OK)
        return 0;
    return gla_workspace(B * H, N, d, dv);
}

la_status la_forward_gla(const void* q, const void* k, const void* v, const float* alpha,
                         float* out, int64_t B, int64_t H, int64_t N, int d, int dv,
                         int feature_map, int dtype, void* workspace, size_t workspace_bytes,
                         la_stream_t stream)
{
    la_status st = check_sizes(B, H, N, d, dv, feature_map, dtype);
    if (st != LA_OK)
        return st;
    if (N == 0)
        return LA_OK;
    if (!q || !k || !v || !alpha || !out || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
        !aligned16(alpha) || !aligned16(out))
        return LA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < gla_workspace(B * H, N, d, dv) || !aligned256(workspace))
        return LA_ERR_WORKSPACE;
    GlaArgs a{};
    a.q = q, a.k = k, a.v = v, a.alpha = alpha, a.out = out;
    a.B = B, a.H = H, a.N = N, a.d = d, a.dv = dv, a.fm = feature_map, a.dtype = dtype;
    a.ws = workspace, a.ws_bytes = workspace_bytes;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(gla_forward(a));
}

la_status la_decode_step_gla(float* S, float* z, const void* q, const void* k, const void* v,
                             const float* alpha, float* out, int64_t B, int64_t H, int d, int dv,
                             int feature_map, int dtype, la_stream_t stream)
{
    if (!alpha || !aligned16(alpha))
        return LA_ERR_INVALID_ARG;
    la_status st = check_sizes(B, H, 1, d, dv, feature_map, dtype);
    if (st != LA_OK)
        return st;
    if (!S || !z || !q || !k || !v || !out)
        return LA_ERR_INVALID_ARG;
    if (!aligned16(S) || !aligned16(z) || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
        !aligned16(out))
        return LA_ERR_INVALID_ARG;
    GammaTable gt;
    make_gamma(nullptr, H, &gt);
    DecodeArgs a{};
    a.S = S, a.z = z, a.q = q, a.k = k, a.v = v, a.alpha = alpha, a.out = out;
    a.BH = B * H, a.H = H, a.d = d, a.dv = dv, a.fm = feature_map, a.dtype = dtype;
    a.gamma = &gt;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(decode_step(a));
}

// Sizes, enums and scale of the delta-rule calls.
static la_status check_delta(const DeltaArgs& a)
{
    if (a.B < 1 || a.H < 1 || a.Hk < 1 || a.N < 0 || a.d < 1 || a.dv < 1 || a.H % a.Hk)
        return LA_ERR_INVALID_ARG;
    if (a.fm != LA_FM_ELU1 && a.fm != LA_FM_IDENTITY_NORM && a.fm != LA_FM_NONE && a.fm != LA_FM_L2)
        return LA_ERR_INVALID_ARG;
    if ((a.dtype != LA_BF16 && a.dtype != LA_FP32) || !isfinite(a.scale))
        return LA_ERR_INVALID_ARG;
    if (!dim_ok(a.d) || !dim_ok(a.dv) || (a.fm != LA_FM_NONE && a.fm != LA_FM_L2))
        return LA_ERR_UNSUPPORTED;
    if (a.B > INT32_MAX / a.H || !delta_grid_ok(a))
        return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

// NULL where `need` is not set, else a 16-byte aligned pointer.
static bool ptr_ok(const void* p, bool need = true) { return p ? aligned16(p) : !need; }

static bool workspace_ok(const void* ws, size_t bytes, size_t need)
{
    return need == 0 || (ws && bytes >= need && aligned256(ws));
}

static DeltaArgs delta_sizes(int64_t B, int64_t H, int64_t Hk, int64_t N, int d, int dv, int fm,
                             float scale, int dtype)
{
    DeltaArgs a{};
    a.B = B, a.H = H, a.Hk = Hk, a.N = N, a.d = d, a.dv = dv;
    a.fm = fm, a.scale = scale, a.dtype = dtype;
    return a;
}

// dst <- src, or zero for a NULL src (the state of an empty sequence)
static la_status copy_state(float* dst, const float* src, const DeltaArgs& a)
{
    const size_t n = sizeof(float) * (size_t)(a.B * a.H) * a.d * a.dv;
    if (!dst || dst == src)
        return LA_OK;
    return from_cuda(src ? cudaMemcpyAsync(dst, src, n, cudaMemcpyDeviceToDevice, a.stream)
                         : cudaMemsetAsync(dst, 0, n, a.stream));
}

size_t la_delta_workspace_size(int64_t B, int64_t H, int64_t Hk, int64_t N, int d, int dv,
                               int dtype)
{
    const DeltaArgs a = delta_sizes(B, H, Hk, N, d, dv, LA_FM_L2, 1.0f, dtype);
    return check_delta(a) != LA_OK || N == 0 ? 0 : delta_forward_workspace(a);
}

la_status la_forward_delta(const void* q, const void* k, const void* v, const float* beta,
                           const float* log_alpha, void* out, const float* S0, float* S_out,
                           int64_t B, int64_t H, int64_t Hk, int64_t N, int d, int dv,
                           int feature_map, float scale, int dtype, void* workspace,
                           size_t workspace_bytes, la_stream_t stream)
{
    DeltaArgs a = delta_sizes(B, H, Hk, N, d, dv, feature_map, scale, dtype);
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    const la_status st = check_delta(a);
    if (st != LA_OK)
        return st;
    if (!ptr_ok(S0, false) || !ptr_ok(S_out, false))
        return LA_ERR_INVALID_ARG;
    if (N == 0)
        return copy_state(S_out, S0, a);
    if (!q != !out || (!out && !S_out) || !ptr_ok(q, false) || !ptr_ok(out, false) || !ptr_ok(k) || !ptr_ok(v) || !ptr_ok(beta) ||
        !ptr_ok(log_alpha, false))
        return LA_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, delta_forward_workspace(a)))
        return LA_ERR_WORKSPACE;
    a.q = q, a.k = k, a.v = v, a.beta = beta, a.log_alpha = log_alpha, a.out = out;
    a.S0 = S0, a.S_out = S_out, a.ws = workspace;
    a.status = status_ptr();
    return from_cuda(delta_forward(a));
}

la_status la_decode_step_delta(float* S, const void* q, const void* k, const void* v,
                               const float* beta, const float* log_alpha, void* out, int64_t B,
                               int64_t H, int64_t Hk, int d, int dv, int feature_map, float scale,
                               int dtype, la_stream_t stream)
{
    DeltaArgs a = delta_sizes(B, H, Hk, 1, d, dv, feature_map, scale, dtype);
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    const la_status st = check_delta(a);
    if (st != LA_OK)
        return st;
    if (!ptr_ok(S) || !ptr_ok(q) || !ptr_ok(k) || !ptr_ok(v) || !ptr_ok(beta) ||
        !ptr_ok(log_alpha, false) || !ptr_ok(out))
        return LA_ERR_INVALID_ARG;
    a.q = q, a.k = k, a.v = v, a.beta = beta, a.log_alpha = log_alpha, a.out = out, a.S_out = S;
    return from_cuda(delta_decode(a));
}

size_t la_delta_backward_workspace_size(int64_t B, int64_t H, int64_t Hk, int64_t N, int d, int dv,
                                        int dtype)
{
    const DeltaArgs a = delta_sizes(B, H, Hk, N, d, dv, LA_FM_L2, 1.0f, dtype);
    return check_delta(a) != LA_OK || N == 0 ? 0 : delta_backward_workspace(a);
}

la_status la_backward_delta(const void* dout, const float* dS_out, const void* q, const void* k,
                            const void* v, const float* beta, const float* log_alpha,
                            const float* S0, void* dq, void* dk, void* dv_out, float* dbeta,
                            float* dlog_alpha, float* dS0, int64_t B, int64_t H, int64_t Hk,
                            int64_t N, int d, int dv, int feature_map, float scale, int dtype,
                            void* workspace, size_t workspace_bytes, la_stream_t stream)
{
    DeltaArgs a = delta_sizes(B, H, Hk, N, d, dv, feature_map, scale, dtype);
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    const la_status st = check_delta(a);
    if (st != LA_OK)
        return st;
    if (!ptr_ok(S0, false) || !ptr_ok(dS_out, false) || !ptr_ok(dS0, false))
        return LA_ERR_INVALID_ARG;
    if (N == 0)
        return copy_state(dS0, dS_out, a);
    if (!log_alpha != !dlog_alpha || !ptr_ok(dout) || !ptr_ok(q) || !ptr_ok(k) || !ptr_ok(v) || !ptr_ok(beta) ||
        !ptr_ok(log_alpha, false) || !ptr_ok(dq) || !ptr_ok(dk) || !ptr_ok(dv_out) ||
        !ptr_ok(dbeta) || !ptr_ok(dlog_alpha, false))
        return LA_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, delta_backward_workspace(a)))
        return LA_ERR_WORKSPACE;
    a.q = q, a.k = k, a.v = v, a.beta = beta, a.log_alpha = log_alpha;
    a.S0 = S0, a.dout = dout, a.dS_out = dS_out, a.dq = dq, a.dk = dk, a.dv_ = dv_out;
    a.dbeta = dbeta, a.dlog_alpha = dlog_alpha, a.dS0 = dS0;
    a.ws = workspace;
    a.status = status_ptr();
    return from_cuda(delta_backward(a));
}

static la_status check_norm(const NormGateArgs& a)
{
    if (a.B < 1 || a.H < 1 || a.N < 0 || a.dv < 1 || !(a.eps > 0.0f) || !isfinite(a.eps))
        return LA_ERR_INVALID_ARG;
    if ((a.act != LA_ACT_SILU && a.act != LA_ACT_SIGMOID && a.act != LA_ACT_NONE) ||
        (a.weight_heads != 0 && a.weight_heads != 1) ||
        (a.x_dtype != LA_BF16 && a.x_dtype != LA_FP32) ||
        (a.dtype != LA_BF16 && a.dtype != LA_FP32))
        return LA_ERR_INVALID_ARG;
    // rows are counted in 32 bits; a gradient with a weight for each head keeps up to
    // H rows of partial sums per lane group
    if (!dim_ok(a.dv) || a.H > 16384 || a.B > INT32_MAX / a.H ||
        (a.N > 0 && a.B * a.H > INT32_MAX / a.N))
        return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

static NormGateArgs norm_sizes(int64_t B, int64_t H, int64_t N, int dv, int act, int weight_heads,
                               float eps, int x_dtype, int dtype, la_stream_t stream)
{
    NormGateArgs a{};
    a.B = B, a.H = H, a.N = N, a.dv = dv, a.act = act, a.weight_heads = weight_heads;
    a.eps = eps, a.x_dtype = x_dtype, a.dtype = dtype;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return a;
}

la_status la_norm_gate(const void* x, const void* gate, const float* weight, void* y, int64_t B,
                       int64_t H, int64_t N, int dv, int activation, int weight_heads, float eps,
                       int x_dtype, int dtype, la_stream_t stream)
{
    NormGateArgs a = norm_sizes(B, H, N, dv, activation, weight_heads, eps, x_dtype, dtype, stream);
    const la_status st = check_norm(a);
    if (st != LA_OK || N == 0)
        return st;
    if (!ptr_ok(x) || !ptr_ok(y) || !ptr_ok(gate, false) || !ptr_ok(weight, false))
        return LA_ERR_INVALID_ARG;
    a.x = x, a.gate = gate, a.weight = weight, a.y = y;
    return from_cuda(norm_gate(a));
}

size_t la_norm_gate_backward_workspace_size(int64_t B, int64_t H, int64_t N, int dv)
{
    const NormGateArgs a =
        norm_sizes(B, H, N, dv, LA_ACT_SILU, 0, 1.0f, LA_FP32, LA_FP32, nullptr);
    return check_norm(a) != LA_OK || N == 0 ? 0 : norm_gate_backward_workspace(a);
}

la_status la_norm_gate_backward(const void* dy, const void* x, const void* gate,
                                const float* weight, void* dx, void* dgate, float* dweight,
                                int64_t B, int64_t H, int64_t N, int dv, int activation,
                                int weight_heads, float eps, int x_dtype, int dtype,
                                void* workspace, size_t workspace_bytes, la_stream_t stream)
{
    NormGateArgs a = norm_sizes(B, H, N, dv, activation, weight_heads, eps, x_dtype, dtype, stream);
    const la_status st = check_norm(a);
    if (st != LA_OK)
        return st;
    if (!weight != !dweight || !ptr_ok(dweight, false))
        return LA_ERR_INVALID_ARG;
    if (N == 0)
        return !dweight ? LA_OK
                        : from_cuda(cudaMemsetAsync(
                              dweight, 0, sizeof(float) * (weight_heads ? H : 1) * dv, a.stream));
    if (!gate != !dgate || !ptr_ok(dy) || !ptr_ok(x) || !ptr_ok(dx) || !ptr_ok(gate, false) || !ptr_ok(dgate, false) ||
        !ptr_ok(weight, false))
        return LA_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, weight ? norm_gate_backward_workspace(a) : 0))
        return LA_ERR_WORKSPACE;
    a.dy = dy, a.x = x, a.gate = gate, a.weight = weight, a.dx = dx, a.dgate = dgate;
    a.dweight = dweight, a.ws = workspace;
    return from_cuda(norm_gate_backward(a));
}

// dst <- src, or zero for a NULL src
static la_status copy_bytes(void* dst, const void* src, size_t bytes, cudaStream_t st)
{
    if (!dst || dst == src)
        return LA_OK;
    return from_cuda(src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, st)
                         : cudaMemsetAsync(dst, 0, bytes, st));
}

static la_status clear(float* dst, int64_t count, cudaStream_t st)
{
    return dst ? from_cuda(cudaMemsetAsync(dst, 0, sizeof(float) * (size_t)count, st)) : LA_OK;
}

static int type_size(int dtype) { return dtype == LA_BF16 ? 2 : 4; }

// A strided input: aligned to its type.
static bool rows_ok(const void* p, int dtype, bool need = true)
{
    return p ? reinterpret_cast<uintptr_t>(p) % (unsigned)type_size(dtype) == 0 : !need;
}

static bool lengths_ok(const int32_t* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

constexpr int64_t kMaxChannels = 1 << 24;

static la_status check_conv(const ConvArgs& a)
{
    if (a.B < 1 || a.N < 0 || a.C < 1 || a.H < 1 || a.C % a.H || a.W < 1 || a.xb < 0 || a.xt < 0)
        return LA_ERR_INVALID_ARG;
    if ((a.act != LA_ACT_SILU && a.act != LA_ACT_SIGMOID && a.act != LA_ACT_NONE) ||
        (a.dtype != LA_BF16 && a.dtype != LA_FP32))
        return LA_ERR_INVALID_ARG;
    // blocks of 128 threads, each with four tokens at least
    if (a.W < 2 || a.W > 4 || a.C > kMaxChannels || a.N > INT32_MAX ||
        (double)a.B * ((double)a.N / 4 + 1) * ((double)a.C / 128 + 1) > INT32_MAX)
        return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

static ConvArgs conv_sizes(int64_t B, int64_t N, int64_t C, int64_t H, int W, int act, int dtype,
                           int64_t xb, int64_t xt, la_stream_t stream)
{
    ConvArgs a{};
    a.B = B, a.N = N, a.C = C, a.H = H, a.W = W, a.act = act, a.dtype = dtype;
    a.xb = xb, a.xt = xt;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return a;
}

static size_t window_bytes(const ConvArgs& a)
{
    return (size_t)(a.B * (a.W - 1) * a.C) * type_size(a.dtype);
}

la_status la_forward_conv(const void* x, int64_t x_batch, int64_t x_token, const float* weight,
                          const float* bias, void* y, const void* S0, void* S_out,
                          const int32_t* lengths, int64_t B, int64_t N, int64_t C, int64_t H, int W,
                          int activation, int dtype, la_stream_t stream)
{
    ConvArgs a = conv_sizes(B, N, C, H, W, activation, dtype, x_batch, x_token, stream);
    const la_status st = check_conv(a);
    if (st != LA_OK)
        return st;
    if (!ptr_ok(S0, false) || !ptr_ok(S_out, false) || !lengths_ok(lengths))
        return LA_ERR_INVALID_ARG;
    if (N == 0)
        return copy_bytes(S_out, S0, window_bytes(a), a.stream);
    if (!rows_ok(x, dtype) || !ptr_ok(weight) || !ptr_ok(bias, false) || !ptr_ok(y))
        return LA_ERR_INVALID_ARG;
    a.x = x, a.weight = weight, a.bias = bias, a.y = y, a.S0 = S0, a.S_out = S_out;
    a.lengths = lengths;
    return from_cuda(conv_forward(a));
}

la_status la_decode_step_conv(void* S, const void* x, int64_t x_batch, const float* weight,
                              const float* bias, void* y, int64_t B, int64_t C, int W,
                              int activation, int dtype, la_stream_t stream)
{
    ConvArgs a = conv_sizes(B, 1, C, 1, W, activation, dtype, x_batch, 0, stream);
    const la_status st = check_conv(a);
    if (st != LA_OK)
        return st;
    if (!ptr_ok(S) || !rows_ok(x, dtype) || !ptr_ok(weight) || !ptr_ok(bias, false) || !ptr_ok(y))
        return LA_ERR_INVALID_ARG;
    a.S_out = S, a.x = x, a.weight = weight, a.bias = bias, a.y = y;
    return from_cuda(conv_step(a));
}

size_t la_conv_backward_workspace_size(int64_t B, int64_t N, int64_t C, int W, int dtype)
{
    const ConvArgs a = conv_sizes(B, N, C, 1, W, LA_ACT_SILU, dtype, 0, 0, nullptr);
    return check_conv(a) != LA_OK || N == 0 ? 0 : conv_backward_workspace(a);
}

la_status la_backward_conv(const void* dy, const void* dS_out, const void* x, int64_t x_batch,
                           int64_t x_token, const float* weight, const float* bias, const void* S0,
                           const int32_t* lengths, void* dx, float* dweight, float* dbias,
                           void* dS0, int64_t B, int64_t N, int64_t C, int64_t H, int W,
                           int activation, int dtype, void* workspace, size_t workspace_bytes,
                           la_stream_t stream)
{
    ConvArgs a = conv_sizes(B, N, C, H, W, activation, dtype, x_batch, x_token, stream);
    la_status st = check_conv(a);
    if (st != LA_OK)
        return st;
    if (!ptr_ok(S0, false) || !ptr_ok(dS_out, false) || !ptr_ok(dS0, false) || !lengths_ok(lengths) ||
        !ptr_ok(dweight) || !ptr_ok(dbias, false) || !bias != !dbias)
        return LA_ERR_INVALID_ARG;
    if (N == 0) {
        if ((st = copy_bytes(dS0, dS_out, window_bytes(a), a.stream)) != LA_OK ||
            (st = clear(dweight, C * W, a.stream)) != LA_OK)
            return st;
        return clear(dbias, C, a.stream);
    }
    if (!ptr_ok(dy) || !rows_ok(x, dtype) || !ptr_ok(weight) || !ptr_ok(bias, false) || !ptr_ok(dx))
        return LA_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, conv_backward_workspace(a)))
        return LA_ERR_WORKSPACE;
    a.dy = dy, a.dS_out = dS_out, a.x = x, a.weight = weight, a.bias = bias, a.S0 = S0;
    a.lengths = lengths, a.dx = dx, a.dweight = dweight, a.dbias = dbias, a.dS0 = dS0;
    a.ws = workspace;
    return from_cuda(conv_backward(a));
}

static la_status check_ssm(const SsmArgs& a)
{
    if (a.B < 1 || a.N < 0 || a.C < 1 || a.G < 1 || a.C % a.G || a.n < 1 ||
        (a.softplus != 0 && a.softplus != 1) || (a.dtype != LA_BF16 && a.dtype != LA_FP32))
        return LA_ERR_INVALID_ARG;
    if ((a.n != 8 && a.n != 16 && a.n != 32 && a.n != 64) || a.C > kMaxChannels || a.N > INT32_MAX)
        return LA_ERR_UNSUPPORTED;
    // blocks: segments of at least 8 tokens times tiles of at least 16 channels of a
    // group; threads of the sums and of a step
    const double tiles = (double)a.G * ((double)(a.C / a.G) / 16 + 1);
    if ((double)a.B * ((double)a.N / 8 + 1) * tiles > INT32_MAX ||
        (double)a.B * ((double)a.C * a.n / 128 + 1) > INT32_MAX || (double)a.B * a.N * a.G * a.n / 128 + 1 > INT32_MAX)
        return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

// `s`: the caller's strides, or NULL.  A step has one stride for each input.
static bool ssm_strides(SsmArgs* a, const int64_t* s, bool step, bool grad)
{
    const int64_t row = a->C, shared = a->G * a->n, rows = step ? 1 : a->N;
    int64_t *const batch[6] = {&a->x_batch, &a->delta_batch, &a->B_batch, &a->C_batch, &a->z_batch, &a->dout_batch};
    int64_t *const token[6] = {&a->x_token, &a->delta_token, &a->B_token, &a->C_token, &a->z_token, &a->dout_token};
    for (int i = 0; i < (grad ? 6 : 5); ++i) {
        const int64_t width = i == 2 || i == 3 ? shared : row;
        *batch[i] = s ? s[step ? i : 2 * i] : width * rows;
        *token[i] = step ? 0 : s ? s[2 * i + 1] : width;
        if (*batch[i] < 0 || *token[i] < 0)
            return false;
    }
    return true;
}

static SsmArgs ssm_sizes(int64_t B, int64_t N, int64_t C, int64_t G, int n, int softplus, int dtype,
                         la_stream_t stream)
{
    SsmArgs a{};
    a.B = B, a.N = N, a.C = C, a.G = G, a.n = n, a.softplus = softplus, a.dtype = dtype;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return a;
}

static bool ssm_inputs_ok(const SsmArgs& a)
{
    return rows_ok(a.x, a.dtype) && rows_ok(a.delta, a.dtype) && ptr_ok(a.A) && rows_ok(a.Bm, a.dtype) &&
           rows_ok(a.Cm, a.dtype) && ptr_ok(a.D, false) && rows_ok(a.z, a.dtype, false) && ptr_ok(a.bias, false);
}

size_t la_ssm_workspace_size(int64_t B, int64_t N, int64_t C, int64_t G, int n, int dtype)
{
    const SsmArgs a = ssm_sizes(B, N, C, G, n, 1, dtype, nullptr);
    return check_ssm(a) != LA_OK || N == 0 ? 0 : ssm_forward_workspace(a);
}

la_status la_forward_ssm(const void* x, const void* delta, const float* A, const void* Bm,
                         const void* Cm, const float* D, const void* z, const float* delta_bias,
                         void* out, const float* S0, float* S_out, const int32_t* lengths,
                         const int64_t* strides, int64_t B, int64_t N, int64_t C, int64_t G, int n,
                         int softplus, int dtype, void* workspace, size_t workspace_bytes,
                         la_stream_t stream)
{
    SsmArgs a = ssm_sizes(B, N, C, G, n, softplus, dtype, stream);
    const la_status st = check_ssm(a);
    if (st != LA_OK)
        return st;
    if (!ssm_strides(&a, strides, false, false) || !ptr_ok(S0, false) || !ptr_ok(S_out, false) ||
        !lengths_ok(lengths))
        return LA_ERR_INVALID_ARG;
    if (N == 0)
        return copy_bytes(S_out, S0, sizeof(float) * (size_t)(B * C) * n, a.stream);
    a.x = x, a.delta = delta, a.A = A, a.Bm = Bm, a.Cm = Cm, a.D = D, a.z = z, a.bias = delta_bias;
    if (!ssm_inputs_ok(a) || !ptr_ok(out))
        return LA_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, ssm_forward_workspace(a)))
        return LA_ERR_WORKSPACE;
    a.out = out, a.S0 = S0, a.S_out = S_out, a.lengths = lengths, a.ws = workspace;
    return from_cuda(ssm_forward(a));
}

la_status la_decode_step_ssm(float* S, const void* x, const void* delta, const float* A,
                             const void* Bm, const void* Cm, const float* D, const void* z,
                             const float* delta_bias, void* out, const int64_t* strides, int64_t B,
                             int64_t C, int64_t G, int n, int softplus, int dtype,
                             la_stream_t stream)
{
    SsmArgs a = ssm_sizes(B, 1, C, G, n, softplus, dtype, stream);
    const la_status st = check_ssm(a);
    if (st != LA_OK)
        return st;
    a.x = x, a.delta = delta, a.A = A, a.Bm = Bm, a.Cm = Cm, a.D = D, a.z = z, a.bias = delta_bias;
    if (!ssm_strides(&a, strides, true, false) || !ptr_ok(S) || !ssm_inputs_ok(a) || !ptr_ok(out))
        return LA_ERR_INVALID_ARG;
    a.S_out = S, a.out = out;
    return from_cuda(ssm_step(a));
}

size_t la_ssm_backward_workspace_size(int64_t B, int64_t N, int64_t C, int64_t G, int n, int dtype)
{
    const SsmArgs a = ssm_sizes(B, N, C, G, n, 1, dtype, nullptr);
    return check_ssm(a) != LA_OK || N == 0 ? 0 : ssm_backward_workspace(a);
}

la_status la_backward_ssm(const void* dout, const float* dS_out, const void* x, const void* delta,
                          const float* A, const void* Bm, const void* Cm, const float* D,
                          const void* z, const float* delta_bias, const float* S0,
                          const int32_t* lengths, void* dx, void* ddelta, float* dA, void* dBm,
                          void* dCm, float* dD, void* dz, float* ddelta_bias, float* dS0,
                          const int64_t* strides, int64_t B, int64_t N, int64_t C, int64_t G, int n,
                          int softplus, int dtype, void* workspace, size_t workspace_bytes,
                          la_stream_t stream)
{
    SsmArgs a = ssm_sizes(B, N, C, G, n, softplus, dtype, stream);
    la_status st = check_ssm(a);
    if (st != LA_OK)
        return st;
    if (!ssm_strides(&a, strides, false, true) || !ptr_ok(S0, false) || !ptr_ok(dS_out, false) ||
        !ptr_ok(dS0, false) || !lengths_ok(lengths) || !ptr_ok(dA) || !ptr_ok(dD, false) ||
        !ptr_ok(ddelta_bias, false) || !D != !dD || !delta_bias != !ddelta_bias)
        return LA_ERR_INVALID_ARG;
    if (N == 0) {
        if ((st = copy_bytes(dS0, dS_out, sizeof(float) * (size_t)(B * C) * n, a.stream)) != LA_OK ||
            (st = clear(dA, C * n, a.stream)) != LA_OK || (st = clear(dD, C, a.stream)) != LA_OK)
            return st;
        return clear(ddelta_bias, C, a.stream);
    }
    a.x = x, a.delta = delta, a.A = A, a.Bm = Bm, a.Cm = Cm, a.D = D, a.z = z, a.bias = delta_bias;
    if (!ssm_inputs_ok(a) || !rows_ok(dout, dtype) || !ptr_ok(dx) || !ptr_ok(ddelta) || !ptr_ok(dBm) ||
        !ptr_ok(dCm) || !ptr_ok(dz, false) || !z != !dz)
        return LA_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, ssm_backward_workspace(a)))
        return LA_ERR_WORKSPACE;
    a.dout = dout, a.dS_out = dS_out, a.S0 = S0, a.lengths = lengths;
    a.dx = dx, a.ddelta = ddelta, a.dA = dA, a.dB = dBm, a.dC = dCm, a.dD = dD, a.dz = dz;
    a.dbias = ddelta_bias, a.dS0 = dS0, a.ws = workspace;
    return from_cuda(ssm_backward(a));
}

la_status la_state_prefix(const float* S_parts, const float* z_parts, int nparts,
                          const int64_t* part_len, int upto, float* S_out, float* z_out,
                          int64_t B, int64_t H, int d, int dv, const float* gamma,
                          la_stream_t stream)
{
    la_status st = check_sizes(B, H, 1, d, dv, LA_FM_ELU1, LA_FP32);
    if (st != LA_OK)
        return st;
    GammaTable gt;
    if ((st = make_gamma(gamma, H, &gt)) != LA_OK)
        return st;
    if (nparts < 1 || nparts > state_prefix_max_parts() || upto < 0 || upto > nparts || !part_len)
        return LA_ERR_INVALID_ARG;
    for (int q = 0; q < nparts; ++q)
        if (part_len[q] < 0)
            return LA_ERR_INVALID_ARG;
    if (!S_parts || !z_parts || !S_out || !z_out || !aligned16(S_parts) || !aligned16(z_parts) ||
        !aligned16(S_out) || !aligned16(z_out))
        return LA_ERR_INVALID_ARG;
    return from_cuda(state_prefix(S_parts, z_parts, nparts, part_len, upto, S_out, z_out, B * H,
                                  (int)H, d, dv, gt, reinterpret_cast<cudaStream_t>(stream)));
}

la_status la_favor_features(const void* x, const float* w, void* out, int64_t rows, int d, int r,
                            int in_dtype, int out_dtype, la_stream_t stream)
{
    if (rows < 0 || !favor_shape_ok(d, r))
        return rows < 0 || d < 1 || r < 1 ? LA_ERR_INVALID_ARG : LA_ERR_UNSUPPORTED;
    if ((in_dtype != LA_BF16 && in_dtype != LA_FP32) || (out_dtype != LA_BF16 && out_dtype != LA_FP32))
        return LA_ERR_INVALID_ARG;
    if (rows == 0)
        return LA_OK;
    if (!x || !w || !out || !aligned16(x) || !aligned16(w) || !aligned16(out))
        return LA_ERR_INVALID_ARG;
    return from_cuda(favor_features(x, w, out, rows, d, r, in_dtype, out_dtype, status_ptr(),
                                    reinterpret_cast<cudaStream_t>(stream)));
}

uint64_t la_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

la_status la_get_device_status(la_stream_t stream)
{
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return LA_ERR_CUDA;
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_status, sizeof(int)) != cudaSuccess)
        return LA_ERR_CUDA;
    if (v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int)) != cudaSuccess)
            return LA_ERR_CUDA;
    }
    return static_cast<la_status>(v);
}

}  // extern "C"
