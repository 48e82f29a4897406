// dense_api.cu — host side of the dense feed-forward calls of
// include/moe_mxfp4.h: argument checks, the per-GPU status word, launches.
// Nothing here allocates or synchronises except moe_dense_status.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "dense.cuh"
#include "host_checks.cuh"

namespace {

// One status word per GPU that loads the library (as the scratch of
// moe_forward_noalloc): the dense calls have no handle to keep one in.  A line
// further: what a read of it has taken out.
__device__ unsigned g_dense_status[64];
constexpr int kTaken = 32;

// Kernels on any stream may set bits meanwhile: each is taken here or stays.
__global__ void take_status_kernel(unsigned *status) { status[kTaken] = atomicExch(status, 0u); }

std::atomic<int> g_polls{moe::kDensePolls};

struct DeviceInfo {
    int rc = MOE_ERR_CUDA;
    int sms = 0;
    unsigned *status = nullptr;
};

// SM count and status word of the current device, looked up once per device.
int device_info(int *dev, DeviceInfo *out) {
    static DeviceInfo info[moe::PerDeviceOnce::kMaxDevices];
    static moe::PerDeviceOnce once;
    int d = -1;
    if (cudaGetDevice(&d) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    if (d < 0 || d >= moe::PerDeviceOnce::kMaxDevices) return MOE_ERR_UNSUPPORTED;
    int rc = MOE_OK;
    const cudaError_t e = moe::per_device_once(once, [&] {
        int sms = 0;
        rc = moe::current_device_ok(nullptr, &sms);
        if (rc != MOE_OK) return cudaErrorNotSupported;
        void *p = nullptr;
        const cudaError_t s = cudaGetSymbolAddress(&p, g_dense_status);
        if (s != cudaSuccess) return s;
        info[d].sms = sms;
        info[d].status = static_cast<unsigned *>(p);
        return cudaSuccess;
    });
    if (rc != MOE_OK) return rc;
    if (e != cudaSuccess) return moe::cuda_rc(e);
    *dev = d;
    *out = info[d];
    return MOE_OK;
}

// Row indices (with a tile's rows past the last one) stay inside an int.
constexpr int kMaxTokens = 1 << 30;
bool tokens_ok(int T) { return T >= 0 && T <= kMaxTokens; }
bool dim_ok(int v) { return v >= 8 && v <= 65536 && v % 8 == 0; }

struct Range {
    const void *p;
    size_t n;
};

bool overlap(const Range &a, const Range &b) {
    if (!a.p || !b.p || !a.n || !b.n) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + b.n && y < x + a.n;
}

// Every output against every input and every other output.
template <int NO, int NI>
bool outputs_clash(const Range (&out)[NO], const Range (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = i + 1; j < NO; ++j)
            if (overlap(out[i], out[j])) return true;
        for (int j = 0; j < NI; ++j)
            if (overlap(out[i], in[j])) return true;
    }
    return false;
}

size_t bf16_bytes(int64_t rows, int64_t cols) { return (size_t)rows * (size_t)cols * 2; }

}  // namespace

extern "C" {

int moe_gated_ffn(const uint16_t *x, int T, int H, int I, const uint16_t *w_gate,
                  const uint16_t *w_up, int act, unsigned flags, uint16_t *x_norm, uint16_t *h,
                  void *stream) {
    if (!tokens_ok(T) || !dim_ok(H) || !dim_ok(I)) return MOE_ERR_ARG;
    if (act < MOE_ACT_SILU || act > MOE_ACT_GELU_TANH || (flags & ~MOE_FFN_RMSNORM)) return MOE_ERR_ARG;
    const bool norm = flags & MOE_FFN_RMSNORM;
    if (norm != (x_norm != nullptr) && T > 0) return MOE_ERR_ARG;
    if (T == 0) return MOE_OK;
    const Range out[2] = {{h, bf16_bytes(T, I)}, {x_norm, bf16_bytes(T, H)}};
    const Range in[3] = {{x, bf16_bytes(T, H)}, {w_gate, bf16_bytes(I, H)}, {w_up, bf16_bytes(I, H)}};
    if (outputs_clash(out, in)) return MOE_ERR_ARG;
    int dev = 0, rc;
    DeviceInfo d;
    if ((rc = device_info(&dev, &d)) != MOE_OK) return rc;
    const void *ptrs[4] = {x, w_gate, w_up, h};
    for (const void *q : ptrs)
        if ((rc = moe::check_device_memory(dev, q, 16)) != MOE_OK) return rc;
    if (norm && (rc = moe::check_device_memory(dev, x_norm, 16)) != MOE_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (norm && (rc = moe::cuda_rc(moe::launch_rms_norm(x, T, H, x_norm, s))) != MOE_OK) return rc;
    moe::GatedParams p = {};
    p.x = norm ? x_norm : x;
    p.wg = w_gate;
    p.wu = w_up;
    p.h = h;
    p.status = d.status;
    p.polls = g_polls.load(std::memory_order_relaxed);
    p.T = T;
    p.H = H;
    p.I = I;
    p.act = act;
    return moe::cuda_rc(moe::launch_gated(p, d.sms, s));
}

int moe_gated_ffn_backward_workspace_bytes(int T, int H, int I, size_t *bytes) {
    if (!bytes || !tokens_ok(T) || !dim_ok(H) || !dim_ok(I)) return MOE_ERR_ARG;
    *bytes = moe::align_up(2 * bf16_bytes(T > 0 ? T : 1, I), 256);
    return MOE_OK;
}

int moe_gated_ffn_backward(const uint16_t *x, int T, int H, int I, const uint16_t *w_gate,
                           const uint16_t *w_up, int act, const uint16_t *dh, uint16_t *dx,
                           uint16_t *dw_gate, uint16_t *dw_up, void *workspace, size_t bytes,
                           void *stream) {
    if (!tokens_ok(T) || !dim_ok(H) || !dim_ok(I)) return MOE_ERR_ARG;
    if (act < MOE_ACT_SILU || act > MOE_ACT_GELU_TANH) return MOE_ERR_ARG;
    if ((dw_gate == nullptr) != (dw_up == nullptr)) return MOE_ERR_ARG;
    if (T > 0 && !dx && !dw_gate) return MOE_ERR_ARG;
    int dev = 0, rc;
    DeviceInfo d;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t wbytes = bf16_bytes(I, H);
    if (T == 0) {
        if (!dw_gate) return MOE_OK;
        const Range a = {dw_gate, wbytes}, b = {dw_up, wbytes};
        if (overlap(a, b)) return MOE_ERR_ARG;
        if ((rc = device_info(&dev, &d)) != MOE_OK) return rc;
        if ((rc = moe::check_device_memory(dev, dw_gate, 16)) != MOE_OK) return rc;
        if ((rc = moe::check_device_memory(dev, dw_up, 16)) != MOE_OK) return rc;
        if ((rc = moe::cuda_rc(cudaMemsetAsync(dw_gate, 0, wbytes, s))) != MOE_OK) return rc;
        return moe::cuda_rc(cudaMemsetAsync(dw_up, 0, wbytes, s));
    }
    const size_t need = moe::align_up(2 * bf16_bytes(T, I), 256);
    const Range out[4] = {{dx, bf16_bytes(T, H)}, {dw_gate, wbytes}, {dw_up, wbytes}, {workspace, need}};
    const Range in[4] = {{x, bf16_bytes(T, H)}, {w_gate, wbytes}, {w_up, wbytes}, {dh, bf16_bytes(T, I)}};
    if (outputs_clash(out, in)) return MOE_ERR_ARG;
    if ((rc = device_info(&dev, &d)) != MOE_OK) return rc;
    const void *ptrs[4] = {x, w_gate, w_up, dh};
    for (const void *q : ptrs)
        if ((rc = moe::check_device_memory(dev, q, 16)) != MOE_OK) return rc;
    const void *outs[3] = {dx, dw_gate, dw_up};
    for (const void *q : outs)
        if (q && (rc = moe::check_device_memory(dev, q, 16)) != MOE_OK) return rc;
    if ((rc = moe::check_device_memory(dev, workspace, 256)) != MOE_OK) return rc;
    if (bytes < need) return MOE_ERR_WORKSPACE;
    moe::GatedParams p = {};
    p.x = x;
    p.wg = w_gate;
    p.wu = w_up;
    p.dh = dh;
    p.dgu = static_cast<uint16_t *>(workspace);
    p.dx = dx;
    p.dwg = dw_gate;
    p.dwu = dw_up;
    p.status = d.status;
    p.polls = g_polls.load(std::memory_order_relaxed);
    p.T = T;
    p.H = H;
    p.I = I;
    p.act = act;
    return moe::cuda_rc(moe::launch_gated_backward(p, d.sms, s));
}

int moe_adapter_proj_workspace_bytes(int T, int K, int N, int n_adapters, int rank, size_t *bytes) {
    if (!bytes || !tokens_ok(T) || !dim_ok(K) || !dim_ok(N) || n_adapters < 0) return MOE_ERR_ARG;
    if (n_adapters > 0 && (rank < 8 || rank > 256 || rank % 8)) return MOE_ERR_ARG;
    *bytes = n_adapters > 0 ? moe::adapter_workspace(T > 0 ? T : 1, K, N, n_adapters, rank) : 0;
    return MOE_OK;
}

int moe_adapter_proj(const uint16_t *x, int T, int K, int N, const uint16_t *w,
                     const uint16_t *residual, int n_adapters, int rank, const uint16_t *lora_a,
                     const uint16_t *lora_b, const float *lora_scale, const int32_t *adapter_ids,
                     uint16_t *y, void *workspace, size_t bytes, void *stream) {
    size_t need = 0;
    int rc = moe_adapter_proj_workspace_bytes(T, K, N, n_adapters, rank, &need);
    if (rc != MOE_OK) return rc;
    if (n_adapters == 0 && (lora_a || lora_b || lora_scale || adapter_ids)) return MOE_ERR_ARG;
    if (T == 0) return MOE_OK;
    const size_t an = n_adapters;
    const size_t ybytes = bf16_bytes(T, N);
    const Range out[2] = {{y, ybytes}, {workspace, need}};
    const Range in[6] = {{x, bf16_bytes(T, K)},          {w, bf16_bytes(N, K)},
                         {lora_a, bf16_bytes(an * (size_t)rank, K)}, {lora_b, bf16_bytes(an * (size_t)N, rank)},
                         {lora_scale, an * 4},           {adapter_ids, an ? (size_t)T * 4 : 0}};
    if (outputs_clash(out, in)) return MOE_ERR_ARG;
    // the residual may be y itself (each element is read before it is
    // written, by the same thread), but not overlap it otherwise
    const Range res = {residual, ybytes};
    if ((residual != y && overlap(out[0], res)) || overlap(out[1], res)) return MOE_ERR_ARG;
    int dev = 0;
    DeviceInfo d;
    if ((rc = device_info(&dev, &d)) != MOE_OK) return rc;
    const void *ptrs[3] = {x, w, y};
    for (const void *q : ptrs)
        if ((rc = moe::check_device_memory(dev, q, 16)) != MOE_OK) return rc;
    if (residual && (rc = moe::check_device_memory(dev, residual, 16)) != MOE_OK) return rc;
    if (n_adapters > 0) {
        if ((rc = moe::check_device_memory(dev, lora_a, 16)) != MOE_OK) return rc;
        if ((rc = moe::check_device_memory(dev, lora_b, 16)) != MOE_OK) return rc;
        if ((rc = moe::check_device_memory(dev, lora_scale, 4)) != MOE_OK) return rc;
        if ((rc = moe::check_device_memory(dev, adapter_ids, 4)) != MOE_OK) return rc;
        if ((rc = moe::check_device_memory(dev, workspace, 256)) != MOE_OK) return rc;
        if (bytes < need) return MOE_ERR_WORKSPACE;
    }
    moe::AdapterParams p = {};
    p.x = x;
    p.w = w;
    p.residual = residual;
    p.a = lora_a;
    p.b = lora_b;
    p.scale = lora_scale;
    p.ids = adapter_ids;
    p.y = y;
    p.v = static_cast<float *>(workspace);
    p.status = d.status;
    p.polls = g_polls.load(std::memory_order_relaxed);
    p.T = T;
    p.K = K;
    p.N = N;
    p.n = n_adapters;
    p.rank = rank;
    return moe::cuda_rc(moe::launch_adapter_proj(p, d.sms, static_cast<cudaStream_t>(stream)));
}

int moe_adapter_proj_plan(int T, int K, int N, int n_adapters, int rank, int num_sms,
                          const int *cluster_ctas, int *plan) {
    size_t need = 0;
    int rc = moe_adapter_proj_workspace_bytes(T, K, N, n_adapters, rank, &need);
    if (rc != MOE_OK) return rc;
    if (!plan || T == 0 || num_sms < 0 || (num_sms > 0) != (cluster_ctas != nullptr)) return MOE_ERR_ARG;
    for (int l = 0; cluster_ctas && l < 3; ++l)  // one CTA per SM
        if (cluster_ctas[l] < 0 || cluster_ctas[l] > num_sms) return MOE_ERR_ARG;
    if (num_sms == 0) {
        int dev = 0;
        DeviceInfo d;
        if ((rc = device_info(&dev, &d)) != MOE_OK) return rc;
        num_sms = d.sms;
    }
    moe::AdapterPlan p;
    if ((rc = moe::cuda_rc(moe::adapter_plan(T, K, N, n_adapters, rank, num_sms, cluster_ctas, &p))) != MOE_OK)
        return rc;
    const int v[6] = {p.products, p.splits, p.inner, p.inner_splits, p.direct, p.groups};
    for (int i = 0; i < 6; ++i) plan[i] = v[i];
    return MOE_OK;
}

int moe_dense_status(void *stream, unsigned *device_status) {
    if (!device_status) return MOE_ERR_ARG;
    int dev = 0;
    DeviceInfo d;
    const int rc = device_info(&dev, &d);
    if (rc != MOE_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned v = 0;
    if (cudaStreamSynchronize(s) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    // one reader at a time has the taken word, for as long as the read itself takes
    static std::mutex reading;
    std::lock_guard<std::mutex> lock(reading);
    take_status_kernel<<<1, 1, 0, s>>>(d.status);
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyAsync(&v, d.status + kTaken, sizeof v, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    *device_status = v;
    return MOE_OK;
}

int moe_dense_set_spin_limit(int polls) {
    if (polls < 0) return MOE_ERR_ARG;
    g_polls.store(polls, std::memory_order_relaxed);
    return MOE_OK;
}

}  // extern "C"
