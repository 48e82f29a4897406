// dense.cu — order of the dense feed-forward launches, and the RMSNorm ahead
// of the gated block.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "dense.cuh"
#include "gemv.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

// One CTA per row: xn = BF16(r / sqrt(mean(r^2) + 1e-6)).
__global__ void __launch_bounds__(kThreads) rms_norm_kernel(const uint16_t *x, int H, uint16_t *xn) {
    __shared__ float red[kThreads / 32];
    const uint4 *row = reinterpret_cast<const uint4 *>(x + (size_t)blockIdx.x * H);
    uint4 *out = reinterpret_cast<uint4 *>(xn + (size_t)blockIdx.x * H);
    pdl_wait();
    pdl_launch_dependents();
    float ss = 0.f;
    for (int c = threadIdx.x; c < H / 8; c += kThreads) {
        const uint4 v = row[c];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float a = bf16_to_f32(w[q] & 0xFFFFu), b = bf16_to_f32(w[q] >> 16);
            ss = fmaf(a, a, fmaf(b, b, ss));
        }
    }
    ss = warp_sum(ss);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) ss += red[i];
    const float inv = 1.0f / sqrtf(ss / (float)H + 1e-6f);
    for (int c = threadIdx.x; c < H / 8; c += kThreads) {
        const uint4 v = row[c];
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
            w[q] = (uint32_t)f32_to_bf16(bf16_to_f32(w[q] & 0xFFFFu) * inv) |
                   ((uint32_t)f32_to_bf16(bf16_to_f32(w[q] >> 16) * inv) << 16);
        out[c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace

cudaError_t launch_rms_norm(const uint16_t *x, int T, int H, uint16_t *xn, cudaStream_t s) {
    return launch_ex(rms_norm_kernel, dim3(T), dim3(kThreads), 0, s, true, x, H, xn);
}

cudaError_t launch_gated(const GatedParams &p, int sms, cudaStream_t s) {
    return gemv_supported(p.T, p.H) ? launch_gated_gemv(p, sms, s) : launch_gated_tc(p, sms, s);
}

cudaError_t launch_gated_backward(const GatedParams &p, int sms, cudaStream_t s) {
    cudaError_t e = launch_gated_tc(p, sms, s);
    if (e == cudaSuccess && p.dx) e = launch_dx_tc(p, sms, s);
    if (e == cudaSuccess && p.dwg) e = launch_dw_tc(p, p.dx != nullptr, sms, s);
    return e;
}

size_t adapter_workspace(int T, int, int, int, int rank) {
    // v: FP32 of up to 8 tokens, else BF16
    const size_t n = (size_t)T * rank * (T <= 8 ? sizeof(float) : sizeof(uint16_t));
    return (n + 255) / 256 * 256;
}

cudaError_t launch_adapter_proj(const AdapterParams &p, int sms, cudaStream_t s) {
    return gemv_supported(p.T, p.K) ? launch_proj_gemv(p, sms, s) : launch_proj_tc(p, sms, s);
}

}  // namespace moe
