// dense.cu — the dense feed-forward products, plain form: one 64 x 64 output
// tile per CTA, BF16 operands staged in shared memory as FP32, FP32 sums.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "dense.cuh"
#include "dense_act.cuh"
#include "gemv.cuh"

namespace moe {

namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;

// acc[i][j] += sum_k A(m0 + ty + 16 i, k) B(n0 + tx + 16 j, k), k in [0, K).
template <class FA, class FB>
__device__ void tile_product(float (&acc)[4][4], int K, FA A, FB B) {
    __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int k0 = 0; k0 < K; k0 += kStep) {
        __syncthreads();
        for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
            const int k = i % kStep, r = i / kStep;
            sa[k][r] = k0 + k < K ? A(r, k0 + k) : 0.f;
            sb[k][r] = k0 + k < K ? B(r, k0 + k) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
    }
}

__device__ __forceinline__ float at(const uint16_t *p, int r, int rows, int c, int cols, size_t ld) {
    return r < rows && c < cols ? bf16_to_f32(p[(size_t)r * ld + c]) : 0.f;
}

__global__ void __launch_bounds__(kThreads) gated_kernel(const GatedParams p) {
    const int m0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile;
    float g[4][4] = {}, u[4][4] = {};
    auto X = [&](int r, int k) { return at(p.x, m0 + r, p.T, k, p.H, p.H); };
    tile_product(g, p.H, X, [&](int r, int k) { return at(p.wg, n0 + r, p.I, k, p.H, p.H); });
    tile_product(u, p.H, X, [&](int r, int k) { return at(p.wu, n0 + r, p.I, k, p.H, p.H); });
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= p.T || n >= p.I) continue;
            if (p.h) {
                p.h[(size_t)m * p.I + n] = f32_to_bf16(act_value(g[i][j], p.act) * u[i][j]);
            } else {
                float a, da;
                act_value_grad(g[i][j], p.act, a, da);
                const float d = bf16_to_f32(p.dh[(size_t)m * p.I + n]);
                uint16_t *row = p.dgu + (size_t)m * 2 * p.I;
                row[n] = f32_to_bf16(d * u[i][j] * da);
                row[p.I + n] = f32_to_bf16(d * a);
            }
        }
}

__global__ void __launch_bounds__(kThreads) dx_kernel(const GatedParams p) {
    const int m0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile;
    float acc[4][4] = {};
    for (int half = 0; half < 2; ++half) {
        const uint16_t *w = half ? p.wu : p.wg;
        tile_product(
            acc, p.I,
            [&](int r, int k) { return at(p.dgu + half * p.I, m0 + r, p.T, k, p.I, 2 * (size_t)p.I); },
            [&](int r, int k) { return at(w, k, p.I, n0 + r, p.H, p.H); });
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < p.T && n < p.H) p.dx[(size_t)m * p.H + n] = f32_to_bf16(acc[i][j]);
        }
}

__global__ void __launch_bounds__(kThreads) dw_kernel(const GatedParams p) {
    const int m0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile, half = blockIdx.z;
    float acc[4][4] = {};
    tile_product(
        acc, p.T,
        [&](int r, int k) { return at(p.dgu + half * p.I, k, p.T, m0 + r, p.I, 2 * (size_t)p.I); },
        [&](int r, int k) { return at(p.x, k, p.T, n0 + r, p.H, p.H); });
    uint16_t *dw = half ? p.dwu : p.dwg;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < p.I && n < p.H) dw[(size_t)m * p.H + n] = f32_to_bf16(acc[i][j]);
        }
}

// v[t][j] = scale[a] sum_k x[t][k] A[a][j][k], one warp per (t, j).
__global__ void __launch_bounds__(kThreads) adapter_inner_kernel(const AdapterParams p) {
    const int lane = threadIdx.x & 31;
    const size_t i = (size_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (i >= (size_t)p.T * p.rank) return;
    const int t = (int)(i / p.rank), j = (int)(i % p.rank), id = p.ids[t];
    if (id < 0 || id >= p.n) {
        if (lane == 0 && id != -1) atomicOr(p.status, kBadAdapterStatus);
        if (lane == 0) p.v[i] = 0.f;
        return;
    }
    const uint16_t *x = p.x + (size_t)t * p.K, *a = p.a + ((size_t)id * p.rank + j) * p.K;
    float s = 0.f;
    for (int k = lane; k < p.K; k += 32) s = fmaf(bf16_to_f32(x[k]), bf16_to_f32(a[k]), s);
    s = warp_sum(s);
    if (lane == 0) p.v[i] = s * p.scale[id];
}

__global__ void __launch_bounds__(kThreads) adapter_proj_kernel(const AdapterParams p) {
    const int m0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile;
    float acc[4][4] = {};
    tile_product(acc, p.K, [&](int r, int k) { return at(p.x, m0 + r, p.T, k, p.K, p.K); },
                 [&](int r, int k) { return at(p.w, n0 + r, p.N, k, p.K, p.K); });
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= p.T || n >= p.N) continue;
            float s = acc[i][j];
            const int id = p.n > 0 ? p.ids[m] : -1;
            if (id >= 0 && id < p.n) {
                const uint16_t *b = p.b + ((size_t)id * p.N + n) * p.rank;
                for (int q = 0; q < p.rank; ++q)
                    s = fmaf(p.v[(size_t)m * p.rank + q], bf16_to_f32(b[q]), s);
            }
            const size_t o = (size_t)m * p.N + n;
            if (p.residual) s += bf16_to_f32(p.residual[o]);
            p.y[o] = f32_to_bf16(s);
        }
}

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

unsigned tiles(int n) { return (unsigned)((n + kTile - 1) / kTile); }

}  // namespace

cudaError_t launch_rms_norm(const uint16_t *x, int T, int H, uint16_t *xn, cudaStream_t s) {
    return launch_ex(rms_norm_kernel, dim3(T), dim3(kThreads), 0, s, true, x, H, xn);
}

cudaError_t launch_gated(const GatedParams &p, int, cudaStream_t s) {
    return launch_ex(gated_kernel, dim3(tiles(p.T), tiles(p.I)), dim3(kThreads), 0, s, false, p);
}

cudaError_t launch_gated_backward(const GatedParams &p, int sms, cudaStream_t s) {
    cudaError_t e = launch_gated(p, sms, s);
    if (e == cudaSuccess && p.dx)
        e = launch_ex(dx_kernel, dim3(tiles(p.T), tiles(p.H)), dim3(kThreads), 0, s, false, p);
    if (e == cudaSuccess && p.dwg)
        e = launch_ex(dw_kernel, dim3(tiles(p.I), tiles(p.H), 2), dim3(kThreads), 0, s, false, p);
    return e;
}

size_t adapter_workspace(int T, int, int, int, int rank) {
    return ((size_t)T * rank * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_adapter_proj(const AdapterParams &p, int, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (p.n > 0) {
        const size_t warps = (size_t)p.T * p.rank;
        e = launch_ex(adapter_inner_kernel, dim3((unsigned)((warps + 7) / 8)), dim3(kThreads), 0, s,
                      false, p);
    }
    if (e == cudaSuccess)
        e = launch_ex(adapter_proj_kernel, dim3(tiles(p.T), tiles(p.N)), dim3(kThreads), 0, s, false, p);
    return e;
}

}  // namespace moe
