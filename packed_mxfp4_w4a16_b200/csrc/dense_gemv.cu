// dense_gemv.cu — the dense feed-forward products of up to 8 tokens (decode):
// the weights' bytes, read once.
//
//   gated  h[t][i] = act(Wg[i] x[t]) * (Wu[i] x[t])
//   proj   y[t][n] = W[n] x[t] + sum_j v[t][j] B[id_t][n][j] (+ residual)
//   inner  v[t][j] = scale * (A[id_t][j] x[t])          (workspace; FP32, or BF16 for
//          the tensor-core projection of more tokens)
//
// One CTA per SM owns a contiguous range of output rows (ranges differ by at
// most one row, so every SM streams the same bytes) and walks it in tiles of
// 16 weight rows (gated: 8 of Wg and the same 8 of Wu) and K chunks of up to
// 2048.  A producer warp keeps a ring of chunks in flight with bulk copies, one
// per row and chunk: the copies' issue is what limits short ones (T 1, H 2048,
// I 7168: chunks of 512 took 23.1 us, 1024 13.1, 2048 11.1; floor 9.1).  Eight
// consumer warps take an eighth of each chunk as m16n8k16 products, weight
// rows as M and the tokens as N.  The K order inside 64 elements is permuted the same way for both operands: thread (g, q) of a warp
// holds 16 consecutive elements of weight rows g and g + 8 and of token g, so
// every fragment is two 16-byte shared-memory reads (row pitches of 16 bytes
// more than a multiple of 128 keep them free of bank conflicts).  FP32 sums;
// the eight warps' parts are added in warp order.
//
// Bound by HBM.  mma.sync is used for its register operands, not its rate: 16
// x 8 products per weight row would be 1/16 of a tcgen05 tile of 128 rows.
#include <cuda_runtime.h>
#include <stdint.h>

#include "dense.cuh"
#include "dense_act.cuh"
#include "gemv.cuh"
#include "tc.cuh"

namespace moe {

namespace {

constexpr int kMaxRing = 8;
constexpr int kWarps = 8;                       // consumers; warp 8 produces
constexpr int kThreads = 32 * (kWarps + 1);
constexpr size_t kRed = 2 * kWarps * 128 * sizeof(float);

struct GemvArgs {
    const uint16_t *x;         // [T][K]
    const uint16_t *w0, *w1;   // gated: Wg, Wu; proj: W
    uint16_t *out;             // [T][rows]
    const uint16_t *residual;  // proj, or null
    const uint16_t *b;         // proj: [n][rows][rank]
    const float *v;            // proj: [T][rank]
    const int32_t *ids;        // proj
    unsigned *status;
    int polls;                 // of a bounded wait
    int T, K, rows, n, rank;
    int ring, chunk;           // ring slots, K elements in each
};

__host__ __device__ inline uint32_t row_pitch(int chunk) { return (uint32_t)chunk * 2 + 16; }
__host__ __device__ inline uint32_t x_pitch(int K) { return (uint32_t)((K + 63) / 64 * 64) * 2 + 16; }

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

template <bool GATED, int ACT>
__global__ void __launch_bounds__(kThreads, 1) gemv_kernel(const GemvArgs p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_full[kMaxRing], s_empty[kMaxRing];
    __shared__ int s_abort;
    constexpr int tile = GATED ? 8 : 16;  // output rows per tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *red = reinterpret_cast<float *>(smem);
    uint8_t *xs = smem + kRed;
    const uint32_t xp = x_pitch(p.K);
    const uint32_t ring0 = smem_u32(xs) + (p.T * xp + 127) / 128 * 128;
    uint8_t *ringp = xs + (p.T * xp + 127) / 128 * 128;
    const int r0 = (int)((int64_t)p.rows * blockIdx.x / gridDim.x);
    const int r1 = (int)((int64_t)p.rows * (blockIdx.x + 1) / gridDim.x);
    const int chunks = (p.K + p.chunk - 1) / p.chunk, share = p.chunk / kWarps;
    const uint32_t pitch = row_pitch(p.chunk), slot = 16 * pitch;
    volatile int *abort = &s_abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.ring; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], kWarps);
        }
        s_abort = 0;
        mbar_fence_init();
    }
    // this lane's weight row of the tile that starts at r, or null
    auto row_of = [&](int r) -> const uint16_t * {
        const int i = r + (GATED ? lane & 7 : lane);
        if (lane >= 16 || i >= r1) return nullptr;
        return (GATED && lane >= 8 ? p.w1 : p.w0) + (size_t)i * p.K;
    };
    if (warp == kWarps) {
        // ahead of the wait for the previous kernel: the first ring of weights
        // into L2 (a hint that reads nothing, so it may run early)
        const uint16_t *row = row_of(r0);
        if (row) prefetch_l2_bulk(row, (uint32_t)min(p.K, p.ring * p.chunk) * 2);
    }
    // After inner_kernel, which lets this one start only once its own inputs
    // were complete, only v has to be waited for, where it is read.
    const bool late = !GATED && p.n > 0;
    if (!late) pdl_wait();
    pdl_launch_dependents();
    __syncthreads();  // barriers set up

    if (warp == kWarps) {
        bool ok = true;
        int it = 0;
#pragma unroll 1
        for (int r = r0; r < r1 && ok; r += tile) {
            const uint16_t *row = row_of(r);
            const uint32_t nrows = min(tile, r1 - r) * (GATED ? 2 : 1);
#pragma unroll 1
            for (int c = 0; c < chunks; ++c, ++it) {
                const int s = it % p.ring;
                if (it >= p.ring) {
                    ok = tc::wait(&s_empty[s], (it / p.ring - 1) & 1, abort, p.polls);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                const uint32_t bytes = (uint32_t)min(p.chunk, p.K - c * p.chunk) * 2;
                if (lane == 0) tc::arrive_tx(&s_full[s], nrows * bytes);
                __syncwarp();
                if (row) bulk_load(ring0 + s * slot + lane * pitch, row + c * p.chunk, bytes, &s_full[s]);
            }
        }
        // nothing in flight on the way out, whichever warp's wait gave up
        for (int j = it > p.ring ? it - p.ring : 0; j < it; ++j) mbar_wait(&s_full[j % p.ring], (j / p.ring) & 1);
    } else {
        // the tokens, zero-padded to a multiple of 64 elements
        const int per_row = (int)((xp - 16) / 16);
        for (int i = threadIdx.x; i < p.T * per_row; i += 32 * kWarps) {
            const int t = i / per_row, c = i % per_row;
            uint4 d = make_uint4(0, 0, 0, 0);
            if (c * 8 < p.K) d = *reinterpret_cast<const uint4 *>(p.x + (size_t)t * p.K + c * 8);
            *reinterpret_cast<uint4 *>(xs + t * xp + c * 16) = d;
        }
        const int i = threadIdx.x >> 3, t = threadIdx.x & 7;  // output row of a tile, token
        int id = -1;
        if (late && threadIdx.x < 128 && t < p.T) {
            id = p.ids[t];
            if (id < 0 || id >= p.n) id = -1;
            if (id >= 0 && r0 + i < r1)  // this thread's row of B, needed at the end
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.b + ((size_t)id * p.rows + r0 + i) * p.rank));
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
        const int g = lane >> 2, q = lane & 3;
        const bool token = g < p.T;
        int it = 0, buf = 0;
        bool ok = true;
#pragma unroll 1
        for (int r = r0; r < r1; r += tile, buf ^= 1) {
            float acc[4] = {};
#pragma unroll 1
            for (int c = 0; c < chunks; ++c, ++it) {
                const int s = it % p.ring;
                ok = ok && tc::wait(&s_full[s], (it / p.ring) & 1, abort, p.polls);
#pragma unroll 2
                for (int sub = 0; sub < share; sub += 64) {
                    const int kc = warp * share + sub + q * 16;  // this thread's 16 elements
                    const int k = c * p.chunk + kc;
                    const uint8_t *lo = ringp + s * slot + g * pitch + kc * 2;
                    const uint8_t *xr = xs + g * xp + (size_t)k * 2;
                    // past K nothing was copied: zeros in its place
                    const uint4 z = make_uint4(0, 0, 0, 0);
                    const bool v0 = k < p.K, v1 = k + 8 < p.K;
                    const uint4 a0 = v0 ? *reinterpret_cast<const uint4 *>(lo) : z;
                    const uint4 a1 = v1 ? *reinterpret_cast<const uint4 *>(lo + 16) : z;
                    const uint4 b0 = v0 ? *reinterpret_cast<const uint4 *>(lo + 8 * pitch) : z;
                    const uint4 b1 = v1 ? *reinterpret_cast<const uint4 *>(lo + 8 * pitch + 16) : z;
                    const uint4 x0 = token && v0 ? *reinterpret_cast<const uint4 *>(xr) : z;
                    const uint4 x1 = token && v1 ? *reinterpret_cast<const uint4 *>(xr + 16) : z;
                    mma_bf16(acc, a0.x, b0.x, a0.y, b0.y, x0.x, x0.y);
                    mma_bf16(acc, a0.z, b0.z, a0.w, b0.w, x0.z, x0.w);
                    mma_bf16(acc, a1.x, b1.x, a1.y, b1.y, x1.x, x1.y);
                    mma_bf16(acc, a1.z, b1.z, a1.w, b1.w, x1.z, x1.w);
                }
                __syncwarp();
                // (after a wait that gave up the slot may still be filled: not handed on)
                if (lane == 0 && ok) mbar_arrive(&s_empty[s]);
            }
            // rows g, g + 8 x tokens 2 q, 2 q + 1 of this warp's share of K
            float *mine = red + (buf * kWarps + warp) * 128;
            *reinterpret_cast<float2 *>(mine + g * 8 + 2 * q) = make_float2(acc[0], acc[1]);
            *reinterpret_cast<float2 *>(mine + (g + 8) * 8 + 2 * q) = make_float2(acc[2], acc[3]);
            asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
            if (threadIdx.x < tile * 8 && r + i < r1 && t < p.T && !s_abort) {
                float a = 0.f, u = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    a += red[(buf * kWarps + w) * 128 + threadIdx.x];
                    if (GATED) u += red[(buf * kWarps + w) * 128 + 64 + threadIdx.x];
                }
                const size_t o = (size_t)t * p.rows + r + i;
                if (GATED) {
                    p.out[o] = f32_to_bf16(act_value<ACT>(a) * u);
                } else {
                    if (late) pdl_wait();
                    if (id >= 0) {
                        const uint16_t *b = p.b + ((size_t)id * p.rows + r + i) * p.rank;
                        const float *v = p.v + t * p.rank;
                        for (int j = 0; j < p.rank; j += 8) {
                            const uint4 d = __ldg(reinterpret_cast<const uint4 *>(b + j));
                            const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                a = fmaf(v[j + 2 * h], bf16_to_f32(w[h] & 0xFFFFu), a);
                                a = fmaf(v[j + 2 * h + 1], bf16_to_f32(w[h] >> 16), a);
                            }
                        }
                    }
                    if (p.residual) a += bf16_to_f32(p.residual[o]);
                    p.out[o] = f32_to_bf16(a);
                }
            }
        }
    }
    // inner_kernel may still run where no token had an adapter: whatever waits
    // for this kernel relies on both being done
    if (late) pdl_wait();
    __syncthreads();
    if (threadIdx.x == 0 && s_abort) atomicOr(p.status, kTimeoutStatus);
}

// Inner products by plain loads: one CTA per TT tokens and RJ rank rows (x is
// read once for all RJ).  It takes the tokens in runs that name the same
// adapter, whose rows are read once for the run.
constexpr int kInnerThreads = 128;
template <int RJ, int TT, bool BF16>
__global__ void __launch_bounds__(kInnerThreads)
inner_kernel(const AdapterParams p) {
    __shared__ float red[kInnerThreads / 32][TT * RJ];
    pdl_wait();
    pdl_launch_dependents();
    const int groups = (p.rank + RJ - 1) / RJ;
    const int j0 = blockIdx.x % groups * RJ, t0 = blockIdx.x / groups * TT;
    int ids[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        ids[i] = t0 + i < p.T ? p.ids[t0 + i] : -1;
        if (ids[i] < -1 || ids[i] >= p.n) {
            if (threadIdx.x == 0 && j0 == 0) atomicOr(p.status, kBadAdapterStatus);
            ids[i] = -1;
        }
    }
    const int chunks = p.K / 8;  // per row
#pragma unroll 1
    for (int first = 0; first < TT;) {
        int id = -1, count = 0;  // the run that starts at `first`
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            if (i == first) id = ids[i];
            if (i == first + count && ids[i] == id) ++count;
        }
        const int t = t0 + first;
        first += count;
        if (id < 0) continue;  // v of a token without an adapter is not read
        const uint4 *a = reinterpret_cast<const uint4 *>(p.a + ((size_t)id * p.rank + j0) * p.K);
        // (tokens past the run repeat its last one; their sums are not written)
        const uint4 *x[TT];
#pragma unroll
        for (int i = 0; i < TT; ++i)
            x[i] = reinterpret_cast<const uint4 *>(p.x + (size_t)(t + min(i, count - 1)) * p.K);
        float s[TT][RJ] = {};
#pragma unroll 2
        for (int c = threadIdx.x; c < chunks; c += kInnerThreads) {
            uint4 av[RJ], xv[TT];
#pragma unroll
            for (int j = 0; j < RJ; ++j) av[j] = __ldg(a + (size_t)j * chunks + c);
#pragma unroll
            for (int i = 0; i < TT; ++i) xv[i] = __ldg(x[i] + c);
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                if (i >= count) break;
                const uint32_t xw[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
#pragma unroll
                for (int j = 0; j < RJ; ++j) {
                    const uint32_t aw[4] = {av[j].x, av[j].y, av[j].z, av[j].w};
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        s[i][j] = fmaf(bf16_to_f32(xw[h] & 0xFFFFu), bf16_to_f32(aw[h] & 0xFFFFu), s[i][j]);
                        s[i][j] = fmaf(bf16_to_f32(xw[h] >> 16), bf16_to_f32(aw[h] >> 16), s[i][j]);
                    }
                }
            }
        }
        __syncthreads();  // red[] of the run before has been read
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int j = 0; j < RJ; ++j) {
                s[i][j] = warp_sum(s[i][j]);
                if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5][i * RJ + j] = s[i][j];
            }
        __syncthreads();
        if (threadIdx.x < count * RJ) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kInnerThreads / 32; ++w) v += red[w][threadIdx.x];
            v *= p.scale[id];
            const size_t o = (size_t)(t + threadIdx.x / RJ) * p.rank + j0 + threadIdx.x % RJ;
            if (BF16)
                reinterpret_cast<uint16_t *>(p.v)[o] = f32_to_bf16(v);
            else
                p.v[o] = v;
        }
    }
}

template <int RJ, int TT, bool BF16>
cudaError_t launch_inner_v(const AdapterParams &p, cudaStream_t s) {
    static PerDeviceOnce once;
    const cudaError_t e = per_device_once(once, [] { return smem_attributes(inner_kernel<RJ, TT, BF16>, 0); });
    if (e != cudaSuccess) return e;
    return launch_ex(inner_kernel<RJ, TT, BF16>, dim3((p.T + TT - 1) / TT * ((p.rank + RJ - 1) / RJ)), dim3(kInnerThreads), 0, s, true, p);
}

constexpr size_t kSmemMost = 220 * 1024;

size_t before_ring(int T, int K) { return kRed + (T * (size_t)x_pitch(K) + 127) / 128 * 128; }

// The longest chunk (no longer than K needs) of which two or more fit beside
// the tokens; false: the tokens are too many for any.
bool ring_plan(int T, int K, int *ring, int *chunk) {
    const size_t base = before_ring(T, K);
    for (int c = 2048; c >= 512; c /= 2) {
        if (c > 512 && c / 2 >= K) continue;
        const size_t slot = 16 * (size_t)row_pitch(c);
        const size_t n = base < kSmemMost ? (kSmemMost - base) / slot : 0;
        if (n >= 2) {
            *ring = (int)(n > kMaxRing ? kMaxRing : n);
            *chunk = c;
            return true;
        }
    }
    return false;
}

template <bool GATED, int ACT>
cudaError_t launch_gemv(GemvArgs g, int num_sms, cudaStream_t s) {
    static PerDeviceOnce once;
    const cudaError_t e = per_device_once(once, [] {
        return smem_attributes(gemv_kernel<GATED, ACT>, kSmemMost);
    });
    if (e != cudaSuccess) return e;
    if (!ring_plan(g.T, g.K, &g.ring, &g.chunk)) return cudaErrorInvalidValue;
    const int grid = g.rows < num_sms ? g.rows : num_sms;
    // no more slots than a CTA has chunks
    const int tile = GATED ? 8 : 16;
    const int64_t most = (int64_t)(((g.rows + grid - 1) / grid + tile - 1) / tile) * ((g.K + g.chunk - 1) / g.chunk);
    if (g.ring > most) g.ring = (int)most;
    const size_t smem = before_ring(g.T, g.K) + (size_t)g.ring * 16 * row_pitch(g.chunk);
    return launch_ex(gemv_kernel<GATED, ACT>, dim3(grid), dim3(kThreads), smem, s, true, g);
}

}  // namespace

bool gemv_supported(int T, int K) {
    int ring, chunk;
    return T <= 8 && ring_plan(T, K, &ring, &chunk);
}

cudaError_t launch_gated_gemv(const GatedParams &p, int num_sms, cudaStream_t s) {
    GemvArgs g = {};
    g.x = p.x;
    g.w0 = p.wg;
    g.w1 = p.wu;
    g.out = p.h;
    g.status = p.status;
    g.polls = p.polls;
    g.T = p.T;
    g.K = p.H;
    g.rows = p.I;
    if (p.act == MOE_ACT_SILU) return launch_gemv<true, MOE_ACT_SILU>(g, num_sms, s);
    if (p.act == MOE_ACT_GELU) return launch_gemv<true, MOE_ACT_GELU>(g, num_sms, s);
    return launch_gemv<true, MOE_ACT_GELU_TANH>(g, num_sms, s);
}

// v in FP32 (read by gemv_kernel, up to 8 tokens) or BF16 (by the tensor-core
// projection).  rank is a multiple of 8: four rank rows per CTA, one where those
// leave SMs idle; four tokens where single ones would fill the SMs several
// times over.
cudaError_t launch_inner(const AdapterParams &p, bool bf16, int num_sms, cudaStream_t s) {
    const int64_t ctas = (int64_t)p.T * (p.rank / 4);
    if (!bf16) return ctas >= num_sms ? launch_inner_v<4, 1, false>(p, s) : launch_inner_v<1, 1, false>(p, s);
    if (ctas > 8 * num_sms) return launch_inner_v<4, 4, true>(p, s);
    return ctas >= num_sms ? launch_inner_v<4, 1, true>(p, s) : launch_inner_v<1, 1, true>(p, s);
}

cudaError_t launch_proj_gemv(const AdapterParams &p, int num_sms, cudaStream_t s) {
    if (p.n > 0) {
        const cudaError_t e = launch_inner(p, false, num_sms, s);
        if (e != cudaSuccess) return e;
    }
    GemvArgs g = {};
    g.x = p.x;
    g.w0 = p.w;
    g.out = p.y;
    g.residual = p.residual;
    g.b = p.b;
    g.v = p.v;
    g.ids = p.ids;
    g.status = p.status;
    g.polls = p.polls;
    g.T = p.T;
    g.K = p.K;
    g.rows = p.N;
    g.n = p.n;
    g.rank = p.rank;
    return launch_gemv<false, 0>(g, num_sms, s);
}

}  // namespace moe
