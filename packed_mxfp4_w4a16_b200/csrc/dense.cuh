// dense.cuh — launch parameters and entry points of the dense feed-forward
// kernels (gated block, its backward pass, projection with adapters).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.cuh"

namespace moe {

constexpr unsigned kBadAdapterStatus = 0x4u;  // MOE_DEVICE_BAD_ADAPTER_ID

// Polls of a wait before it gives up (about 6 s).  An accumulator is waited for
// over a whole K loop, so the bound is longer than a copy's.
constexpr int kDensePolls = 1 << 22;

struct GatedParams {
    const uint16_t *x;       // [T][H]
    const uint16_t *wg, *wu; // [I][H]
    const uint16_t *dh;      // [T][I], backward only
    uint16_t *h;             // [T][I], forward only
    uint16_t *dgu;           // backward: [T][2][I] dg and du (workspace)
    uint16_t *dx;            // [T][H] or null
    uint16_t *dwg, *dwu;     // [I][H] or both null
    unsigned *status;
    int polls;               // of a bounded wait
    int T, H, I, act;
};

struct AdapterParams {
    const uint16_t *x;         // [T][K]
    const uint16_t *w;         // [N][K]
    const uint16_t *residual;  // [T][N] or null
    const uint16_t *a;         // [n][rank][K]
    const uint16_t *b;         // [n][N][rank]
    const float *scale;        // [n]
    const int32_t *ids;        // [T]
    uint16_t *y;               // [T][N]
    float *v;                  // workspace
    unsigned *status;
    int polls;                 // of a bounded wait
    int T, K, N, n, rank;
};

cudaError_t launch_rms_norm(const uint16_t *x, int T, int H, uint16_t *xn, cudaStream_t s);
cudaError_t launch_gated(const GatedParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_gated_backward(const GatedParams &p, int num_sms, cudaStream_t s);
// up to 8 tokens (dense_gemv.cu)
bool gemv_supported(int T, int K);
cudaError_t launch_gated_gemv(const GatedParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_proj_gemv(const AdapterParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_inner(const AdapterParams &p, bool bf16, int num_sms, cudaStream_t s);
// tcgen05 products (dense_gemm.cu)
cudaError_t launch_gated_tc(const GatedParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_dx_tc(const GatedParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_dw_tc(const GatedParams &p, bool after_dx, int num_sms, cudaStream_t s);
cudaError_t launch_proj_tc(const AdapterParams &p, int num_sms, cudaStream_t s);

// What a projection of these sizes takes (see moe_adapter_proj_plan);
// cluster_ctas: [3], or null for the current device's.
struct AdapterPlan {
    int products, splits, inner, inner_splits, direct, groups;
};
cudaError_t adapter_plan(int T, int K, int N, int n, int rank, int num_sms, const int *cluster_ctas,
                         AdapterPlan *out);

size_t adapter_workspace(int T, int K, int N, int n, int rank);
cudaError_t launch_adapter_proj(const AdapterParams &p, int num_sms, cudaStream_t s);

}  // namespace moe
