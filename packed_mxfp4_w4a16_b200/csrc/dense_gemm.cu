// dense_gemm.cu — the dense feed-forward products on tcgen05 (FP32
// accumulators in TMEM, operands brought in by TMA with the 128-byte swizzle).
//
// The products differ in where their operands come from and in their epilogue
// (M x N = sum over K):
//   kFwd   T x I    = x Wg^T and x Wu^T side by side; h = act(g) * u
//   kBwd   the same sums; dg and du from them and dh
//   kDx    T x H    = dg Wg + du Wu   (K runs over the halves of [dg | du])
//   kDw    2I x H   = [dg | du]^T x   (K = T; both operands MN-major)
//   kProj  T x N    = x W^T + v B^T (+ residual): the adapters' inner products
//          v and the rows of their B appended to K, one block of 64 at a time
//   kInner v = scale (x A^T) for the adapters that a tile's tokens name
//   kInnerAll the same as one product with every adapter's A, T x (n rank), of
//          which each row keeps its own adapter's columns
#include <cuda_runtime.h>
#include <stdint.h>

#include "dense.cuh"
#include "dense_act.cuh"
#include "gemv.cuh"
#include "tc.cuh"

namespace moe {

namespace {

enum Mode { kFwd, kBwd, kDx, kDw, kProj, kInner, kInnerAll };

struct GemmArgs {
    const uint16_t *dh;        // kBwd
    const uint16_t *residual;  // kProj, or null
    uint16_t *out0, *out1;     // kDw: dWg, dWu; else out0
    unsigned *status;
    int polls;                 // of a bounded wait
    int M, N;                  // rows of the output (kDw: of one half), its columns
    int kb, kb_half;           // K blocks of 64; kDx: of one half
    int mt, nt, mt_half;       // tiles along M and N; kDw: along M of one half
    int n_fast;                // consecutive tiles share M (else N)
    int wide;                  // outputs allow 32-byte stores
    int tail;                  // big_kernel: the last tiles, done as two of half the columns
    int width, cols;           // small_kernel: output columns per tile, columns of its products
    // adapters (kProj with n > 0, kInner)
    const int32_t *ids;        // [M]
    const float *scale;        // [n], kInner
    const uint16_t *lora_b;    // [n][N][rank], kProj
    uint16_t *v;               // [M][rank] BF16: written by kInner, read by kProj
    // Set for the second of two launches that both depend on the one before
    // them only (dx, then dW, after kBwd): it starts as the first leaves SMs
    // free, which lets it start only after its own wait, and waits for it at its end.
    int late;
    int n, rank;
    int direct;                // small_kernel: v B^T by plain products beside the K loop,
                               // left at this offset in shared memory (0: not)
    int per_tile, parts;       // kInner: adapters per 128 columns, or tiles per adapter
    int groups;                // kInner: CTAs (clusters) that share a row tile's adapters
};

constexpr bool gated(int mode) { return mode == kFwd || mode == kBwd; }
constexpr bool a_mn(int mode) { return mode == kDw; }
constexpr bool b_mn(int mode) { return mode == kDx || mode == kDw; }

// One K block of operand A from row `m` on: K-major in one box of all its
// lines, MN-major in `boxes` boxes of 64 rows.
template <int MODE, int CG>
__device__ __forceinline__ void load_a(uint32_t dst, const CUtensorMap *a, const GemmArgs &g, int kb, int m,
                                       int half, int boxes, uint32_t bar) {
    if (MODE == kDx) {
        const int h = kb >= g.kb_half;
        tc::load3<CG>(dst, a, (kb - h * g.kb_half) * 64, h, m, bar);
    } else if (MODE == kDw) {
        for (int i = 0; i < boxes; ++i) tc::load3<CG>(dst + i * tc::kBox, a, m + 64 * i, half, kb * 64, bar);
    } else {
        tc::load2<CG>(dst, a, kb * 64, m, bar);
    }
}

// One box (MN-major: 64 columns of the output; K-major: the map's lines of a
// weight) of operand B.
template <int MODE, int CG>
__device__ __forceinline__ void load_b(uint32_t dst, const CUtensorMap *b0, const CUtensorMap *b1,
                                       const GemmArgs &g, int kb, int n, int second, uint32_t bar) {
    if (MODE == kDx) {
        const int h = kb >= g.kb_half;
        tc::load2<CG>(dst, h ? b1 : b0, n, (kb - h * g.kb_half) * 64, bar);
    } else if (MODE == kDw) {
        tc::load2<CG>(dst, b0, n, kb * 64, bar);
    } else if (MODE == kInner) {  // n: the adapter, second: its first rank row
        tc::load3<CG>(dst, b0, kb * 64, second, n, bar);
    } else {
        tc::load2<CG>(dst, second ? b1 : b0, kb * 64, n, bar);
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float lo_f32(uint32_t w) { return bf16_to_f32(w & 0xFFFFu); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// W neighbouring BF16 (4: 8 bytes, 8: 16 bytes, 16: 32 bytes) as words.
template <int W>
struct Words {
    uint32_t w[W / 2];
};
template <int W>
__device__ __forceinline__ Words<W> load_words(const uint16_t *p) {
    Words<W> r;
    if (W == 4) {
        const uint2 d = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = d.x, r.w[1] = d.y;
    } else {
#pragma unroll
        for (int i = 0; i < W / 8; ++i) {
            const uint4 d = *reinterpret_cast<const uint4 *>(p + 8 * i);
            r.w[4 * i] = d.x, r.w[4 * i + 1] = d.y, r.w[(4 * i + 2) % (W / 2)] = d.z, r.w[(4 * i + 3) % (W / 2)] = d.w;
        }
    }
    return r;
}
// W = 16: one 32-byte store (p 32-byte aligned).  A lane that owns a row writes
// a whole sector that way (with two 16-byte stores the backward pass of T 2048,
// H 2048, I 1536 took 69.1 us instead of 65.2).
template <int W>
__device__ __forceinline__ void store_bf16(uint16_t *p, const float (&v)[W]) {
    uint32_t w[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) w[i] = pack2(v[2 * i], v[2 * i + 1]);
    if (W == 16)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1 % (W / 2)]),
                     "r"(w[2 % (W / 2)]), "r"(w[3 % (W / 2)]), "r"(w[4 % (W / 2)]), "r"(w[5 % (W / 2)]),
                     "r"(w[6 % (W / 2)]), "r"(w[7 % (W / 2)])
                     : "memory");
    else if (W == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2 % (W / 2)], w[3 % (W / 2)]);
    else
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

// What the outputs at (row, n ..) need besides the sums: dh or the residual.
template <int MODE, int W>
__device__ __forceinline__ Words<W> side_words(const GemmArgs &g, int64_t row, int n) {
    if (MODE == kBwd) return load_words<W>(g.dh + row * g.N + n);
    if (MODE == kProj && g.residual) return load_words<W>(g.residual + row * g.N + n);
    return Words<W>{};
}

// W neighbouring outputs of one row: columns n .. n + W - 1 (all inside the
// matrix: n and N are multiples of W).  v: the sums (gated: g), u: gated only.
// h, dg, du, dx, dW and y are rounded here, once, from FP32; dg and du are
// BF16 because they are operands of the next products.
template <int MODE, int ACT, int W>
__device__ __forceinline__ void finish(const GemmArgs &g, int64_t row, int half, int n, const float (&v)[W],
                                       const float (&u)[W], const Words<W> &side) {
    float o[W];
    if (MODE == kFwd) {
#pragma unroll
        for (int i = 0; i < W; ++i) o[i] = act_value<ACT>(v[i]) * u[i];
        store_bf16<W>(g.out0 + row * g.N + n, o);
    } else if (MODE == kBwd) {
        float p[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float dh = i & 1 ? hi_f32(side.w[i >> 1]) : lo_f32(side.w[i >> 1]);
            float a, da;
            act_value_grad<ACT>(v[i], a, da);
            o[i] = dh * u[i] * da;
            p[i] = dh * a;
        }
        uint16_t *r = g.out0 + row * 2 * g.N + n;
        store_bf16<W>(r, o);
        store_bf16<W>(r + g.N, p);
    } else if (MODE == kInnerAll) {
        // these columns are of one adapter (its rank is a multiple of 8)
        const int id = g.ids[row], a = n / g.rank;
        if (id == a) {
            const float sc = g.scale[id];
#pragma unroll
            for (int i = 0; i < W; ++i) o[i] = v[i] * sc;
            store_bf16<W>(g.v + row * g.rank + (n - a * g.rank), o);
        } else if (n == 0 && (id < -1 || id >= g.n)) {
            // (once per row; the projection may take plain products, which
            // pass over such ids)
            atomicOr(g.status, kBadAdapterStatus);
        }
    } else if (MODE == kDw) {
        store_bf16<W>((half ? g.out1 : g.out0) + row * g.N + n, v);
    } else {
        // without a residual the words are zero; -0 + 0 is +0, so they are not added
        if (MODE == kProj && g.residual) {
#pragma unroll
            for (int i = 0; i < W; ++i) o[i] = v[i] + (i & 1 ? hi_f32(side.w[i >> 1]) : lo_f32(side.w[i >> 1]));
            store_bf16<W>(g.out0 + row * g.N + n, o);
        } else {
            store_bf16<W>(g.out0 + row * g.N + n, v);
        }
    }
}

// ------------------------------------------------------------- adapters --
// The tokens of one tile name some set of adapters.  A group of 128 threads
// lists them, and appends to the tile's K loop blocks of 64 columns that hold
// several adapters side by side (64 / rank of them, or 64 of one adapter's
// columns): the A operand holds a token's v in the columns of its own adapter
// and zeros in the others', the B operand the adapters' B rows.  So one
// accumulator receives every token's own correction, for any mixture.
//
// Zeros do not hide infinities and NaN (0 * inf is NaN), and one request's
// broken adapter must not reach another's tokens: non-finite elements of B
// are left out of the operand, and noted; the epilogue of a tile with such a
// note adds v * b for exactly those elements to the rows that name the
// adapter.  Non-finite v stays in its own row.
struct __align__(16) AdapterSmem {
    int ids[256];    // of the tile's rows; -1: none
    int list[256];   // distinct ids
    union {
        int first[256];        // whether a row is the first of its adapter
        unsigned named[32];    // pools of up to 1024: a bit per adapter
    };
    int count;
    int cmd;         // to the MMA thread: 1 a block is in the buffer, 2 the tile's last
    int bad;         // a non-finite element of B was left out
};

constexpr int kGroup = 128;

// Barrier of the group that tells whether `ok` holds in all of it.
__device__ __forceinline__ bool group_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.red.and.pred q, 1, %2, p; selp.u32 %0, 1, 0, q; }"
        : "=r"(r)
        : "r"((uint32_t)ok), "n"(kGroup)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void group_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kGroup) : "memory"); }

// ids, list and count of rows m0 .. m0 + rows - 1 (rows 128 or 256; rows past
// M have none); tid: index in the group.  Pools of up to 1024 adapters are
// listed by id from a bitmap, larger ones in the order of first rows.
__device__ __forceinline__ void list_adapters(AdapterSmem &s, const GemmArgs &g, int m0, int rows, int tid) {
    const bool bits = g.n <= 1024;
    if (bits && tid < 32) s.named[tid] = 0;
    for (int i = tid; i < rows; i += kGroup) {
        int id = m0 + i < g.M ? g.ids[m0 + i] : -1;
        if (id < -1 || id >= g.n) {
            atomicOr(g.status, kBadAdapterStatus);
            id = -1;
        }
        s.ids[i] = id;
    }
    group_sync();
    if (bits) {
        for (int i = tid; i < rows; i += kGroup) {
            const int id = s.ids[i];
            // (one of a run of equal neighbours marks it)
            if (id >= 0 && (i == 0 || s.ids[i - 1] != id)) atomicOr(&s.named[id >> 5], 1u << (id & 31));
        }
        group_sync();
        if (tid < 32) {
            unsigned w = s.named[tid];
            const int mine = __popc(w);
            int before = mine;  // inclusive prefix sum over the words
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, before, o);
                if (tid >= o) before += v;
            }
            if (tid == 31) s.count = before;
            for (int at = before - mine; w; w &= w - 1) s.list[at++] = tid * 32 + __ffs(w) - 1;
        }
        group_sync();
        return;
    }
    for (int i = tid; i < rows; i += kGroup) {
        // compared with every earlier row, four per load and no early way out
        // (the loads of a scan that may stop wait for one another: 3 us)
        const int id = s.ids[i];
        bool seen = id < 0;
#pragma unroll 8
        for (int j = 0; j < rows; j += 4) {
            const int4 o = *reinterpret_cast<const int4 *>(s.ids + j);
            seen |= (o.x == id && j < i) | (o.y == id && j + 1 < i) | (o.z == id && j + 2 < i) |
                    (o.w == id && j + 3 < i);
        }
        s.first[i] = !seen;
    }
    group_sync();
    if (tid < 32) {
        int count = 0;
        for (int i = tid; i < rows; i += 32) {
            const bool f = s.first[i];
            const unsigned m = __ballot_sync(0xffffffffu, f);
            if (f) s.list[count + __popc(m & ((1u << tid) - 1))] = s.ids[i];
            count += __popc(m);
        }
        if (tid == 0) s.count = count;
    }
    group_sync();
}

__host__ __device__ __forceinline__ int adapter_blocks(int count, int rank) {
    if (rank > 64) return count * ((rank + 63) / 64);
    const int per = 64 / rank;
    return (count + per - 1) / per;
}

// The adapter (index in the list, or -1) and its rank column of chunk c (8
// columns) of appended block e.
__device__ __forceinline__ void chunk_of(int e, int c, int rank, int count, int &at, int &col) {
    if (rank > 64) {
        const int per = (rank + 63) / 64;
        at = e / per;
        col = (e - at * per) * 64 + c * 8;
        if (col >= rank) at = -1;
    } else {
        const int per = 64 / rank, slot = c * 8 / rank;
        at = e * per + slot;
        col = c * 8 - slot * rank;
        if (slot >= per || at >= count) at = -1;
    }
}

// Bits of the non-finite elements (all exponent bits set) of two BF16.
__device__ __forceinline__ uint32_t non_finite(uint32_t w) {
    return ((w & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}

// A thread's share of an appended block: chunk tid % 8 of every 16th row of the
// A operand (a token's v) and of the B operand (an output's row of the
// adapters' B).  Eight threads read a row's 128 bytes, and each has one chunk
// to find (a row per thread, 32 lines per load: T 400, rank 32, 16 adapters at
// random in 30.4 us instead of 24.8).  Fetched ahead of the buffer being free;
// kInner is waited for before the first v is read.
struct AppendRows {
    uint4 a[8], b[8];
};
__device__ __forceinline__ void fetch_block(AppendRows &f, const AdapterSmem &s, const GemmArgs &g, int e, int m,
                                            int row0, int n, int cols, int tid, bool first) {
    int at, col;
    chunk_of(e, tid & 7, g.rank, s.count, at, col);
    const int id = at < 0 ? -2 : s.list[at], r = tid >> 3;
    const uint16_t *b = g.lora_b + ((int64_t)id * g.N + n + r) * g.rank + col;
    const int last = id < 0 ? 0 : min(cols, g.N - n);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f.b[i] = make_uint4(0, 0, 0, 0);
        if (r + 16 * i < last) f.b[i] = __ldg(reinterpret_cast<const uint4 *>(b + (int64_t)16 * i * g.rank));
    }
    if (first) pdl_wait();
    const uint16_t *v = g.v + (int64_t)(m + r) * g.rank + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f.a[i] = make_uint4(0, 0, 0, 0);
        if (s.ids[row0 + r + 16 * i] == id) f.a[i] = *reinterpret_cast<const uint4 *>(v + (int64_t)16 * i * g.rank);
    }
}
// Into the operand tiles at `a` (room for `lines` rows) and `b` (`cols`),
// K-major with the 128-byte swizzle: 16-byte chunk c of row r lies at r * 128
// + 16 (c ^ (r & 7)).  True if a non-finite element of B was left out.
__device__ __forceinline__ bool append_block(const AppendRows &f, uint8_t *a, uint8_t *b, int lines, int cols,
                                             int tid) {
    bool bad = false;
    const int r = tid >> 3, off = r * 128 + 16 * ((tid ^ r) & 7);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t x = non_finite(f.b[i].x), y = non_finite(f.b[i].y), z = non_finite(f.b[i].z),
                       w = non_finite(f.b[i].w);
        bad |= (x | y | z | w) != 0;
        if (r + 16 * i < lines) *reinterpret_cast<uint4 *>(a + off + i * 2048) = f.a[i];
        if (r + 16 * i < cols)
            *reinterpret_cast<uint4 *>(b + off + i * 2048) =
                make_uint4(f.b[i].x & ~x, f.b[i].y & ~y, f.b[i].z & ~z, f.b[i].w & ~w);
    }
    tc::fence_async();  // before the tensor core reads them
    return bad;
}

// The terms that append_block left out, of row `row`, added to outputs n .. n +
// W - 1 (v: the row's, lora_b: the adapter's from row n on).  Out of line and by value: an array whose address
// leaves the kernel would live in local memory on the ordinary way too.
template <int W>
struct Sums {
    float v[W];
};
template <int W>
__device__ __noinline__ Sums<W> with_left_out(int id, const uint16_t *v, const uint16_t *lora_b, int rank,
                                              Sums<W> s) {
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll 1
        for (int j = 0; j < rank; ++j) {
            const uint16_t b = lora_b[(size_t)i * rank + j];
            if ((b & 0x7F80u) == 0x7F80u) s.v[i] += bf16_to_f32(v[j]) * bf16_to_f32(b);
        }
    return s;
}
template <int W>
__device__ __forceinline__ void add_left_out(const GemmArgs &g, int64_t row, int n, float (&v)[W]) {
    const int id = g.ids[row];
    if (id < 0 || id >= g.n) return;
    Sums<W> s;
#pragma unroll
    for (int i = 0; i < W; ++i) s.v[i] = v[i];
    s = with_left_out<W>(id, g.v + row * g.rank, g.lora_b + ((size_t)id * g.N + n) * g.rank, g.rank, s);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = s.v[i];
}

// v B^T by plain FP32 products, for few rows per CTA: each row reads the B rows
// of its own adapter only.  128 threads that are idle during the K loop take
// four outputs of a row at a time, two such groups together, and leave them in
// `delta` ([rows][width] in shared memory) for the finishing threads.
__device__ __forceinline__ void dot8(const uint4 &x, const uint4 &y, float &acc) {
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        acc = fmaf(lo_f32(xw[h]), lo_f32(yw[h]), acc);
        acc = fmaf(hi_f32(xw[h]), hi_f32(yw[h]), acc);
    }
}
__device__ __forceinline__ void direct_products(const GemmArgs &g, int m0, int r0, int r1, int n0, int tid,
                                                float *delta) {
    const int per_row = g.width / 4, items = (r1 - r0) * per_row, chunks = g.rank / 8;
    bool waited = false;
#pragma unroll 1
    for (int i0 = tid; i0 < items || !waited; i0 += 2 * kGroup) {
        const uint4 *v[2], *b[2];
        float acc[2][4] = {};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = i0 + k * kGroup, t = m0 + r0 + i / per_row, n = n0 + i % per_row * 4;
            const int id = i < items && n < g.N ? g.ids[t] : -1;
            v[k] = b[k] = nullptr;
            if (id >= 0 && id < g.n) {
                v[k] = reinterpret_cast<const uint4 *>(g.v + (size_t)t * g.rank);
                b[k] = reinterpret_cast<const uint4 *>(g.lora_b + ((size_t)id * g.N + n) * g.rank);
            }
        }
#pragma unroll 1
        for (int c0 = 0; c0 < chunks; c0 += 2) {
            uint4 vv[2][2], bv[2][2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (v[k] && c0 + c < chunks)
#pragma unroll
                        for (int j = 0; j < 4; ++j) bv[k][c][j] = __ldg(b[k] + j * chunks + c0 + c);
            if (!waited) pdl_wait();  // v; the first of B is on its way
            waited = true;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (v[k] && c0 + c < chunks) vv[k][c] = v[k][c0 + c];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (v[k] && c0 + c < chunks)
#pragma unroll
                        for (int j = 0; j < 4; ++j) dot8(vv[k][c], bv[k][c][j], acc[k][j]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (i0 + k * kGroup < items)
                *reinterpret_cast<float4 *>(delta + 4 * (i0 + k * kGroup)) =
                    make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
    }
}

// W neighbouring sums of a row, as read from TMEM, to the outputs.
template <int MODE, int ACT, int W>
__device__ __forceinline__ void finish_row(const GemmArgs &g, bool bad, int64_t row, int half, int n,
                                           const uint32_t (&v)[W], const uint32_t (&u)[W]) {
    float fv[W], fu[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        fv[i] = __uint_as_float(v[i]);
        fu[i] = gated(MODE) ? __uint_as_float(u[i]) : 0.f;
    }
    if (MODE == kProj && bad) add_left_out<W>(g, row, n, fv);
    finish<MODE, ACT, W>(g, row, half, n, fv, fu, side_words<MODE, W>(g, row, n));
}

// ------------------------------------------------------- large products --
// A pair of CTAs (cluster of 2, cta_group::2) owns 256 x `cols` accumulators
// (cols up to 256, fewer where that leaves fewer SMs without a tile at the end):
// each CTA loads and keeps its 128 rows of A and half of B's rows, the
// leader's MMAs read both CTAs' shared memory, and each CTA's TMEM receives
// its 128 rows.  Gated: one CTA brings cols / 2 rows of Wg, the other as many of Wu,
// so a row's g and u meet in one thread.  Persistent: pairs walk the tiles
// with a stride of the pair count; two accumulators of 256 columns, so the
// epilogue of one tile runs under the products of the next.
// The projection keeps one of the six stages for appended adapter blocks, which
// four more warps fill while the main K loop runs.
constexpr int kBigSlots = 6;
constexpr int kStrip = 8;
constexpr uint32_t kBigStage = 4 * tc::kBox;  // per CTA: A 128 x 64, B 128 x 64
constexpr size_t kBigSmem = kBigSlots * kBigStage + 1024;
// warp 0 TMA, 1 MMA, 2 TMEM, 4..7 epilogue; 8..11 adapters (kProj) or four
// more epilogue warps (gated: the activations of a 128-row tile took four
// warps longer than the products of a K of 2048)
constexpr int big_threads(int mode) { return mode == kProj || gated(mode) ? 384 : 256; }

template <int MODE, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(big_threads(MODE), 1)
big_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b0,
           const __grid_constant__ CUtensorMap map_b1, const GemmArgs g) {
    extern __shared__ uint8_t smem_raw[];
    constexpr int kEpi = gated(MODE) ? 8 : 4;
    constexpr int kBigStages = MODE == kProj ? kBigSlots - 1 : kBigSlots;
    __shared__ __align__(8) uint64_t s_full[kBigStages], s_empty[kBigStages], s_tfull[2], s_tempty[2];
    __shared__ __align__(8) uint64_t s_xfull, s_xempty;
    __shared__ AdapterSmem s_ad;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    // The last `tail` tiles are done as two of half the columns each.
    const int whole = g.mt * g.nt - g.tail, tiles = whole + 2 * g.tail;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBigStages; ++i) {
            mbar_init(&s_full[i], 2);  // both CTAs' producers
            mbar_init(&s_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_tfull[i], 1);
            mbar_init(&s_tempty[i], 2 * kEpi);  // the epilogue warps of both CTAs
        }
        mbar_init(&s_xfull, 2);
        mbar_init(&s_xempty, 1);
        s_abort = 0;
        s_ad.bad = 0;
        mbar_fence_init();
        tc::prefetch_map(&map_a);
        tc::prefetch_map(&map_b0);
        if (gated(MODE) || MODE == kDx) tc::prefetch_map(&map_b1);
    }
    if (warp == 2) tc::tmem_alloc<2>(&s_tmem, 512);
    tc::fence_before();
    tc::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = s_tmem;
    volatile int *abort = &s_abort;
    // With adapters this kernel follows kInner, which lets it start only
    // after its own inputs were complete: just v, which kInner writes, has to
    // be waited for.  Every warp does so before its first wait on a barrier
    // that needs v: those waits are bounded, kInner's run is not.
    const bool adapters = MODE == kProj && g.n > 0, late = adapters || g.late;
    if (!late) pdl_wait();
    pdl_launch_dependents();

    // tile -> first row of the pair's tile, half (kDw), first output column;
    // lines of B in each CTA
    auto place = [&](int t, int &m, int &half, int &n) {
        const int part = t >= whole ? (t - whole) & 1 : 0, split = t >= whole;
        if (split) t = whole + ((t - whole) >> 1);
        // strips of up to 8 tiles along the shorter dimension: the tiles of one
        // moment form a block that shares operands in L2
        const int fast = g.n_fast ? g.nt : g.mt, slow = g.n_fast ? g.mt : g.nt;
        const int strip = t / (kStrip * slow), at = t - strip * kStrip * slow;
        const int width = min(kStrip, fast - strip * kStrip);
        const int a = strip * kStrip + at % width, b = at / width;
        int mt = g.n_fast ? b : a;
        const int nt = g.n_fast ? a : b;
        half = MODE == kDw && mt >= g.mt_half;
        if (half) mt -= g.mt_half;
        m = mt * 256;
        n = nt * g.width + part * (g.width >> 1);
        return g.cols >> (1 + split);
    };

    if (warp == 0) {
        tc::Ring at;
        bool ok = true;
        const bool issue = tc::elect();
        const uint32_t bar0 = tc::map_rank(smem_u32(&s_full[0]), 0);
#pragma unroll 1
        for (int t = pair; t < tiles && ok; t += pairs) {
            int m, half, n;
            const int half_cols = place(t, m, half, n);
            const uint32_t bytes = 2 * tc::kBox + half_cols * 128;
            m += rank * 128;
            if (!gated(MODE)) n += rank * half_cols;
#pragma unroll 1
            for (int kb = 0; kb < g.kb; ++kb, at.next(kBigStages)) {
                if (at.pass > 0) {
                    ok = tc::wait(&s_empty[at.slot], (at.pass - 1) & 1, abort, g.polls);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                if (issue) {
                    const uint32_t bar = bar0 + 8 * at.slot, dst = smem + at.slot * kBigStage;
                    tc::arrive_tx_cluster(bar, bytes);
                    load_a<MODE, 2>(dst, &map_a, g, kb, m, half, 2, bar);
                    load_b<MODE, 2>(dst + 2 * tc::kBox, &map_b0, &map_b1, g, kb, n, rank, bar);
                    if ((b_mn(MODE) || g.tail) && half_cols > 64)
                        load_b<MODE, 2>(dst + 3 * tc::kBox, &map_b0, &map_b1, g, kb, n + 64, rank, bar);
                }
                __syncwarp();
            }
            if (adapters && t == pair) pdl_wait();
        }
        // Nothing in flight on the way out: once the products have used this
        // CTA's last block, every copy of the pair up to it has landed.  (After a
        // wait that gave up they may never: then the bound of this wait, 1.5 s,
        // is the time in which they land.)
        if (at.pass > 0 || at.slot > 0) {
            at.prev(kBigStages);
            mbar_wait(&s_empty[at.slot], at.pass & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint64_t a0 = tc::desc<a_mn(MODE)>(smem), b0 = tc::desc<b_mn(MODE)>(smem + 2 * tc::kBox);
            const bool issue = tc::elect();
            tc::Ring at;
            int j = 0, x = 0;
            bool ok = true, any = false;
#pragma unroll 1
            for (int t = pair; t < tiles && ok; t += pairs, ++j) {
                const uint32_t id = tc::idesc(256, g.cols >> (t >= whole), a_mn(MODE), b_mn(MODE));
                const int buf = j & 1;
                if (j >= 2) {
                    ok = __all_sync(0xffffffffu, tc::wait(&s_tempty[buf], ((j >> 1) - 1) & 1, abort, g.polls));
                    if (!ok) break;
                }
                tc::fence_after();
#pragma unroll 1
                for (int kb = 0; kb < g.kb; ++kb, at.next(kBigStages)) {
                    ok = __all_sync(0xffffffffu, tc::wait(&s_full[at.slot], at.pass & 1, abort, g.polls));
                    if (!ok) break;
                    tc::fence_after();
                    const uint64_t da = a0 + at.slot * (kBigStage >> 4), db = b0 + at.slot * (kBigStage >> 4);
                    if (issue) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma<2>(tmem + buf * 256, da + k * (tc::kstep<a_mn(MODE)>() >> 4),
                                       db + k * (tc::kstep<b_mn(MODE)>() >> 4), id, kb > 0 || k > 0);
                        tc::commit<2>(&s_empty[at.slot]);
                    }
                    __syncwarp();
                    any = true;
                }
                if (MODE == kProj && adapters) {
                    if (t == pair) pdl_wait();
                    for (bool last = false; ok && !last; ++x) {
                        ok = __all_sync(0xffffffffu, tc::wait<true>(&s_xfull, x & 1, abort, g.polls));
                        if (!ok) break;
                        tc::fence_after();
                        const int cmd = *(volatile int *)&s_ad.cmd;
                        last = cmd & 2;
                        const uint64_t da = a0 + kBigStages * (kBigStage >> 4), db = b0 + kBigStages * (kBigStage >> 4);
                        if (issue) {
                            if (cmd & 1)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    tc::mma<2>(tmem + buf * 256, da + 2 * k, db + 2 * k, id, true);
                            tc::commit<2>(&s_xempty);
                        }
                        __syncwarp();
                    }
                }
                if (ok && issue) tc::commit<2>(&s_tfull[buf]);
                __syncwarp();
            }
            // the products issued so far have finished, whichever wait gave up
            if (ok) {
                if (j > 0) mbar_wait(&s_tfull[(j - 1) & 1], ((j - 1) >> 1) & 1);
            } else {
                if (any) {
                    at.prev(kBigStages);
                    mbar_wait(&s_empty[at.slot], at.pass & 1);
                }
                if (x > 0) mbar_wait(&s_xempty, (x - 1) & 1);
            }
        }
        __syncwarp();
    } else if (MODE == kProj && warp >= 8) {
        if (adapters) {
            const int tid = threadIdx.x - 256;
            uint8_t *xa = smem_raw + (smem - smem_u32(smem_raw)) + kBigStages * kBigStage, *xb = xa + 2 * tc::kBox;
            const uint32_t xfull = tc::map_rank(smem_u32(&s_xfull), 0);
            const uint32_t peer_bad = tc::map_rank(smem_u32(&s_ad.bad), rank ^ 1);
            int x = 0;
            bool ok = true;
#pragma unroll 1
            for (int t = pair; t < tiles && ok; t += pairs) {
                int m, half, n;
                const int half_cols = place(t, m, half, n);
                list_adapters(s_ad, g, m, 256, tid);
                const int blocks = adapter_blocks(s_ad.count, g.rank);
                AppendRows f;
                if (blocks)
                    fetch_block(f, s_ad, g, 0, m + rank * 128, rank * 128, n + rank * half_cols, half_cols, tid, true);
                else if (t == pair)
                    pdl_wait();  // the buffer is handed back by a warp that waits for v
#pragma unroll 1
                for (int e = 0; e < (blocks ? blocks : 1); ++e, ++x) {
                    if (x > 0) {
                        ok = group_all(tc::wait(&s_xempty, (x - 1) & 1, abort, g.polls));  // the whole group goes on or leaves
                        if (!ok) break;
                    }
                    if (blocks && append_block(f, xa, xb, 128, half_cols, tid)) {
                        s_ad.bad = 1;
                        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_bad), "r"(1) : "memory");
                        asm volatile("fence.acq_rel.cluster;" ::: "memory");
                    }
                    if (tid == 0) s_ad.cmd = (blocks ? 1 : 0) | (e + 1 >= blocks ? 2 : 0);
                    group_sync();
                    // The tensor core reads each CTA's rows from that CTA's own
                    // shared memory, and every writer has ordered its writes before
                    // such reads; only the note above goes to the other CTA, with
                    // its own fence.  A release at cluster scope would wait for
                    // more: T 8192, K 2048, N 7168, rank 32, 24 adapters at random
                    // in 406 us instead of 353.
                    if (tid == 0) tc::arrive_cluster(xfull);
                    if (e + 1 < blocks)
                        fetch_block(f, s_ad, g, e + 1, m + rank * 128, rank * 128, n + rank * half_cols, half_cols, tid,
                                    false);
                }
                group_sync();  // the list is rebuilt for the next tile
            }
        }
    } else if (warp >= 4) {
        const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t empty0 = tc::map_rank(smem_u32(&s_tempty[0]), 0);
        const uint32_t empty1 = tc::map_rank(smem_u32(&s_tempty[1]), 0);
        int j = 0;
        if (adapters) pdl_wait();
#pragma unroll 1
        for (int t = pair; t < tiles; t += pairs, ++j) {
            const int buf = j & 1;
            const bool ok = tc::wait(&s_tfull[buf], (j >> 1) & 1, abort, g.polls);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc::fence_after();
            int m, half, n;
            const int half_cols = place(t, m, half, n), width = gated(MODE) ? half_cols : 2 * half_cols;
            m += rank * 128 + (warp & 3) * 32 + lane;
            const uint32_t acc = base + buf * 256;
            // gated: two warps share the rows, each finishes every other 16 columns
#pragma unroll 1
            for (int c = gated(MODE) && warp >= 8 ? 16 : 0; c < width && n + c < g.N; c += gated(MODE) ? 32 : 16) {
                uint32_t v[16], u[16];
                tc::tmem_ld16(acc + c, v);
                if (gated(MODE)) tc::tmem_ld16(acc + half_cols + c, u);
                tc::tmem_wait();
                if (m < g.M) {
                    if (g.wide && n + c + 16 <= g.N) {
                        finish_row<MODE, ACT, 16>(g, adapters && *(volatile int *)&s_ad.bad, m, half, n + c, v, u);
                    } else {
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            if (n + c + 8 * q < g.N)
                                finish_row<MODE, ACT, 8>(g, adapters && *(volatile int *)&s_ad.bad, m, half,
                                                         n + c + 8 * q, *reinterpret_cast<uint32_t(*)[8]>(v + 8 * q),
                                                         *reinterpret_cast<uint32_t(*)[8]>(u + 8 * q));
                    }
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::arrive_cluster(buf ? empty1 : empty0);
        }
    }
    // the launch before may still run: whatever waits for this one relies on
    // both being done
    if (late) pdl_wait();
    __syncthreads();
    if (threadIdx.x == 0 && s_abort) atomicOr(g.status, kTimeoutStatus);
    tc::fence_before();
    tc::cluster_sync();  // no CTA leaves while the other may still signal or read it
    if (warp == 2) {
        tc::fence_after();
        tc::tmem_free<2>(tmem, 512);
    }
}

// ------------------------------------------------------- small products --
// One CTA (cta_group::1) owns up to 128 x 128 accumulators (gated: `width`
// columns of g and the same of u; kInner: the A rows of the adapters that fit
// in 128 columns, one tile after the other while the row tile names more of
// them).  The width is chosen so that the tiles fill the SMs: a few hundred
// tokens or fewer are bound by streaming the weights, and every SM that
// streams adds its share.
// Where the tiles are too few for the SMs, a cluster of S CTAs splits K (and
// the appended adapter blocks): every CTA leaves its partial sums in shared
// memory, and each then finishes its share of the rows, adding the S parts in
// rank order through distributed shared memory (the same bits every time, and
// no workspace or counter that two calls could share).
// A K block takes `lines` (8 to 128) lines of 128 bytes of A and `cols` of B: the
// fewer the tokens, the more of the weights is in flight.  A stage holds two
// blocks where there is room for three such stages: a wait, a commit and the loop around them cost the issuing warp about
// 390 clocks, the four MMAs of a block 78.
constexpr int kSmallMaxStages = 8;
__host__ __device__ constexpr uint32_t small_stage(int lines, int cols) { return (lines + cols) * 128; }
constexpr int kSmallThreads = 256;  // warp 0 TMA, 1 MMA, 2 TMEM, 4..7 adapters; all finish rows
constexpr int kPartPitch = 132;     // floats per row of partial sums (528 bytes: spreads banks)
constexpr size_t kParts = 128 * kPartPitch * 4;

template <int MODE, int ACT>
__global__ void __launch_bounds__(kSmallThreads, 2)
small_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b0,
             const __grid_constant__ CUtensorMap map_b1, const GemmArgs g, const int stages, const int per,
             const int splits, const int a_lines) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[kSmallMaxStages], s_empty[kSmallMaxStages], s_done, s_xfull, s_xempty;
    __shared__ AdapterSmem s_ad;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t stage = small_stage(a_lines, g.cols), b_at = a_lines * 128;
    // first product column of u
    const int u_at = gated(MODE) ? g.cols / 2 : 0;
    uint8_t *const base = smem_raw + (smem - smem_u32(smem_raw));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % splits, t = blockIdx.x / splits;

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 1);
        }
        mbar_init(&s_done, 1);
        mbar_init(&s_xfull, 1);
        mbar_init(&s_xempty, 1);
        s_abort = 0;
        s_ad.bad = 0;
        mbar_fence_init();
        tc::prefetch_map(&map_a);
        tc::prefetch_map(&map_b0);
        if (gated(MODE) || MODE == kDx) tc::prefetch_map(&map_b1);
    }
    if (warp == 2) tc::tmem_alloc<1>(&s_tmem, 128);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s_tmem;
    volatile int *abort = &s_abort;

    int mt, nt = 0;
    if (MODE == kInner) {
        mt = t / g.groups;
    } else {
        const int fast = g.n_fast ? g.nt : g.mt;
        mt = g.n_fast ? t / fast : t % fast;
        nt = g.n_fast ? t % fast : t / fast;
    }
    const int half = MODE == kDw && mt >= g.mt_half;
    if (half) mt -= g.mt_half;
    const int m0 = mt * 128, n0 = nt * g.width;
    const int kb0 = (int)((int64_t)g.kb * rank / splits), kb1 = (int)((int64_t)g.kb * (rank + 1) / splits);
    // as in big_kernel, only v has to be waited for after kInner
    const bool adapters = MODE == kProj && g.n > 0, late = adapters || g.late;
    const bool append = adapters && !g.direct;
    if (!late) pdl_wait();
    pdl_launch_dependents();
    const int rows = min(128, g.M - m0);
    // kInner: this row tile's adapters, `per_tile` of them (or a part of one) at a time
    const int lines = MODE == kInner ? min(g.rank, 128) : 1;
    int w0 = 0, w1 = 1, wstep = 1;
    if (MODE == kInner) {
        if (warp >= 4) list_adapters(s_ad, g, m0, 128, threadIdx.x - 128);
        __syncthreads();
        w0 = t % g.groups;
        w1 = g.parts > 1 ? s_ad.count * g.parts : (s_ad.count + g.per_tile - 1) / g.per_tile;
        wstep = g.groups;
    }
    tc::Ring at;
    int round = 0;
    uint32_t issued = 0;  // stages of this round, in the lane that issues the copies
#pragma unroll 1
    for (int w = w0; w < w1; w += wstep, ++round) {
        const int part = MODE == kInner ? w % g.parts : 0;
        const int a0 = MODE == kInner ? w / g.parts * g.per_tile : 0;
        const int slots = MODE == kInner ? min(g.per_tile, s_ad.count - a0) : 0;
        issued = 0;
        if (warp == 0) {
            // (rows that the products read beyond a_lines are garbage that stays in
            // its rows)
            const uint32_t bytes = a_lines * 128 + (MODE == kInner  ? slots * lines * 128
                                                                    : gated(MODE) ? 2 * g.width * 128
                                                                                  : g.width * 128);
            const bool issue = tc::elect();
            bool ok = !*abort;
            // (a lane whose wait gives up goes on without issuing: the warp's
            // lanes keep the same way through the loop without a vote)
#pragma unroll 1
            for (int kb = kb0; kb < kb1; kb += per, at.next(stages)) {
                if (at.pass > 0) ok = ok && tc::wait(&s_empty[at.slot], (at.pass - 1) & 1, abort, g.polls);
                if (issue && ok) {
                    const uint32_t bar = smem_u32(&s_full[at.slot]);
                    uint32_t dst = smem + at.slot * per * stage;
                    const int two = per == 2 && kb + 1 < kb1;
                    tc::arrive_tx(&s_full[at.slot], bytes << two);
#pragma unroll
                    for (int j = 0; j < 2; ++j, dst += stage) {
                        if (j > two) break;
                        if (MODE == kInner) {
                            for (int i = 0; i < slots; ++i)
                                load_b<MODE, 1>(dst + b_at + i * lines * 128, &map_b0, &map_b1, g, kb + j,
                                                s_ad.list[a0 + i], part * 128, bar);
                        } else {
                            // K-major: `width` lines in one box; MN-major: boxes of 64 columns
                            load_b<MODE, 1>(dst + b_at, &map_b0, &map_b1, g, kb + j, n0, 0, bar);
                            if (gated(MODE))
                                load_b<MODE, 1>(dst + b_at + u_at * 128, &map_b0, &map_b1, g, kb + j, n0, 1, bar);
                            if (b_mn(MODE) && g.width > 64)
                                load_b<MODE, 1>(dst + b_at + tc::kBox, &map_b0, &map_b1, g, kb + j, n0 + 64, 0, bar);
                        }
                        load_a<MODE, 1>(dst, &map_a, g, kb + j, m0, half, a_lines / 64, bar);
                    }
                    ++issued;
                }
                __syncwarp();
            }
            __syncwarp();
        } else if (warp == 1) {
            const uint32_t id = tc::idesc(128, g.cols, a_mn(MODE), b_mn(MODE));
            const uint64_t da0 = tc::desc<a_mn(MODE)>(smem), db0 = tc::desc<b_mn(MODE)>(smem + b_at);
            const bool issue = tc::elect();
            bool ok = !*abort;
            int x = 0;
#pragma unroll 1
            for (int kb = kb0; kb < kb1; kb += per, at.next(stages)) {
                ok = ok && tc::wait(&s_full[at.slot], at.pass & 1, abort, g.polls);
                tc::fence_after();
                const uint64_t da = da0 + at.slot * per * (stage >> 4), db = db0 + at.slot * per * (stage >> 4);
                if (issue && ok) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc::mma<1>(tmem, da + k * (tc::kstep<a_mn(MODE)>() >> 4),
                                   db + k * (tc::kstep<b_mn(MODE)>() >> 4), id, kb > kb0 || k > 0);
                    if (per == 2 && kb + 1 < kb1)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma<1>(tmem, da + (stage >> 4) + k * (tc::kstep<a_mn(MODE)>() >> 4),
                                       db + (stage >> 4) + k * (tc::kstep<b_mn(MODE)>() >> 4), id, true);
                    tc::commit<1>(&s_empty[at.slot]);
                }
                __syncwarp();
            }
            if (MODE == kProj && append) {
                pdl_wait();
                for (bool last = false; !last; ++x) {
                    ok = __all_sync(0xffffffffu, ok && tc::wait(&s_xfull, x & 1, abort, g.polls));
                    if (!ok) break;
                    tc::fence_after();
                    const int cmd = *(volatile int *)&s_ad.cmd;
                    last = cmd & 2;
                    const uint64_t da = da0 + stages * per * (stage >> 4), db = db0 + stages * per * (stage >> 4);
                    if (issue) {
                        if (cmd & 1)
#pragma unroll
                            for (int k = 0; k < 4; ++k) tc::mma<1>(tmem, da + 2 * k, db + 2 * k, id, true);
                        tc::commit<1>(&s_xempty);
                    }
                    __syncwarp();
                }
            }
            if (issue) tc::commit<1>(&s_done);
            __syncwarp();
        } else if ((MODE == kBwd || MODE == kProj) && warp == 3) {
            // dh or the residual of the rows that this CTA finishes, into L2
            const uint16_t *side = MODE == kBwd ? g.dh : g.residual;
            const int share = (rows + splits - 1) / splits;
            if (side)
                for (int i = lane; i < share; i += 32) {
                    const int r = rank * share + i;
                    if (r < rows)
                        for (int c = 0; c < g.width && n0 + c < g.N; c += 32)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(side + (int64_t)(m0 + r) * g.N + n0 + c));
                }
        } else if (MODE == kProj && warp >= 4 && adapters && g.direct) {
            // B of the adapters of the rows that this CTA finishes, into L2: the
            // tile's outputs are consecutive in it
            const int share = (rows + splits - 1) / splits, r0 = rank * share;
            const int bytes = min(g.width, g.N - n0) * g.rank * 2;
            for (int i = threadIdx.x - 128; i < share * 32; i += 128) {
                const int r = r0 + i / 32, id = r < rows ? g.ids[m0 + r] : -1;
                if (id >= 0 && id < g.n)
                    for (int b = i % 32 * 128; b < bytes; b += 32 * 128)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(
                            reinterpret_cast<const uint8_t *>(g.lora_b + ((size_t)id * g.N + n0) * g.rank) + b));
            }
            direct_products(g, m0, r0, min(rows, r0 + share), n0, threadIdx.x - 128,
                            reinterpret_cast<float *>(base + g.direct));
        } else if (MODE == kProj && warp >= 4 && adapters) {
            const int tid = threadIdx.x - 128;
            list_adapters(s_ad, g, m0, 128, tid);
            const int blocks = adapter_blocks(s_ad.count, g.rank);
            const int e0 = blocks * rank / splits, e1 = blocks * (rank + 1) / splits;
            uint8_t *xa = base + stages * per * stage;
            AppendRows f;
            if (e0 < e1) fetch_block(f, s_ad, g, e0, m0, 0, n0, g.width, tid, true);
            int x = 0;
#pragma unroll 1
            for (int e = e0; e < max(e1, e0 + 1); ++e, ++x) {
                if (x > 0 && !group_all(tc::wait(&s_xempty, (x - 1) & 1, abort, g.polls))) break;
                if (e < e1 && append_block(f, xa, xa + b_at, a_lines, g.width, tid)) s_ad.bad = 1;
                if (tid == 0) s_ad.cmd = (e < e1 ? 1 : 0) | (e + 1 >= e1 ? 2 : 0);
                group_sync();
                if (tid == 0) mbar_arrive(&s_xfull);
                if (e + 1 < e1) fetch_block(f, s_ad, g, e + 1, m0, 0, n0, g.width, tid, false);
            }
        }
        // every warp: the sums are complete (so all copies have been used too);
        // with appended blocks not before v is
        if (append) pdl_wait();
        const bool ok = tc::wait(&s_done, round & 1, abort, g.polls);
        if (__syncthreads_and(ok && !*abort)) {
            tc::fence_after();
            // TMEM -> shared memory: warp w takes lanes 32 (w % 4) .., every other
            // 16 columns
            float *parts = reinterpret_cast<float *>(base);
            const int r = (warp & 3) * 32 + lane;
            const uint32_t acc = tmem + ((uint32_t)((warp & 3) * 32) << 16);
            if ((warp & 3) * 32 < rows)
#pragma unroll 2
                for (int c = (warp >> 2) * 16; c < g.cols; c += 32) {
                    uint32_t v[16];
                    tc::tmem_ld16(acc + c, v);
                    tc::tmem_wait();
#pragma unroll
                    for (int q = 0; q < 16; q += 4)
                        *reinterpret_cast<uint4 *>(parts + r * kPartPitch + c + q) =
                            make_uint4(v[q], v[q + 1], v[q + 2], v[q + 3]);
                }
        } else if (warp == 0) {
            // some warp's wait gave up: nothing stays in flight, neither copies ...
            const uint32_t total = (uint32_t)(kb1 - kb0 + per - 1) / per;
            tc::Ring back = at;  // to the slot behind the last one issued
            for (uint32_t i = issued; i < total; ++i) back.prev(stages);
            for (uint32_t i = 0; i < min(issued, (uint32_t)stages); ++i) {
                back.prev(stages);
                mbar_wait(&s_full[back.slot], back.pass & 1);
            }
        } else if (warp == 1) {
            mbar_wait(&s_done, round & 1);  // ... nor products
        }
        __syncwarp();
        tc::fence_before();
        if (splits > 1)
            tc::cluster_sync();
        else
            __syncthreads();
        if (!s_abort) {
            // Four outputs of a row at a time (a warp reads consecutive bytes of a
            // part), four such groups per thread together: all that they read is
            // requested before the first is added (a remote read takes about 0.4
            // us, dh or the residual more).
            const int per_row = MODE == kInner ? g.cols / 4 : g.width / 4;
            const int share = (rows + splits - 1) / splits;
            const int r0 = rank * share, r1 = min(rows, r0 + share);
            int bad = 0;
            if (MODE == kProj && append)
                for (int q = 0; q < splits; ++q)
                    bad |= tc::ld_cluster(splits > 1 ? tc::map_rank(smem_u32(&s_ad.bad), q) : smem_u32(&s_ad.bad));
            constexpr int U = 4;
#pragma unroll 1
            for (int i0 = threadIdx.x; i0 < (r1 - r0) * per_row; i0 += U * kSmallThreads) {
                int row[U], col[U];
                float scale[U];
                Words<4> side[U];
                float v[U][4] = {}, u[U][4] = {};
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int i = i0 + k * kSmallThreads;
                    bool on = i < (r1 - r0) * per_row;
                    const int r = r0 + i / per_row, c = (i % per_row) * 4;
                    if (MODE == kInner) {
                        const int slot = c / lines;
                        on = on && slot < slots && part * 128 + c - slot * lines < g.rank;
                        const int id = on ? s_ad.ids[r] : -1;
                        on = on && s_ad.list[a0 + slot] == id;
                        scale[k] = on ? g.scale[id] : 0.f;
                    } else {
                        on = on && n0 + c < g.N;
                        if (on) side[k] = side_words<MODE, 4>(g, (int64_t)m0 + r, n0 + c);
                    }
                    row[k] = on ? r : -1;
                    col[k] = c;
                }
#pragma unroll 2
                for (int q = 0; q < splits; ++q) {
                    const uint32_t from = splits > 1 ? tc::map_rank(smem, q) : smem;
                    float4 a[U], b[U];
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        if (row[k] < 0) continue;
                        const uint32_t at = from + (uint32_t)(row[k] * kPartPitch + col[k]) * 4;
                        a[k] = tc::ld_cluster16(at);
                        if (gated(MODE)) b[k] = tc::ld_cluster16(at + u_at * 4);
                    }
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        if (row[k] < 0) continue;
                        v[k][0] += a[k].x, v[k][1] += a[k].y, v[k][2] += a[k].z, v[k][3] += a[k].w;
                        if (gated(MODE)) u[k][0] += b[k].x, u[k][1] += b[k].y, u[k][2] += b[k].z, u[k][3] += b[k].w;
                    }
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    if (row[k] < 0) continue;
                    const int64_t m = (int64_t)m0 + row[k];
                    if (MODE == kInner) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[k][j] *= scale[k];
                        // rounded to BF16: an operand of the projection's appended blocks
                        store_bf16<4>(g.v + (size_t)m * g.rank + part * 128 + col[k] % lines, v[k]);
                        continue;
                    }
                    if (MODE == kProj && adapters && g.direct) {
                        const float4 d = *reinterpret_cast<const float4 *>(
                            base + g.direct + 4 * ((row[k] - r0) * g.width + col[k]));
                        v[k][0] += d.x, v[k][1] += d.y, v[k][2] += d.z, v[k][3] += d.w;
                    }
                    if (MODE == kProj && bad) add_left_out<4>(g, m, n0 + col[k], v[k]);
                    finish<MODE, ACT, 4>(g, m, half, n0 + col[k], v[k], u[k], side[k]);
                }
            }
        }
        if (MODE == kInner) tc::fence_async();  // the parts' space becomes stages again
        // no CTA goes on (or leaves) while another reads its parts
        if (splits > 1)
            tc::cluster_sync();
        else
            __syncthreads();
    }
    // the launch before may still run: whatever waits for this one relies on
    // both being done
    if (late) pdl_wait();
    if (threadIdx.x == 0 && s_abort) atomicOr(g.status, kTimeoutStatus);
    if (warp == 2) {
        tc::fence_after();
        tc::tmem_free<1>(tmem, 128);
    }
}

// ------------------------------------------------------------------- host --

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                           cudaStream_t s, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

struct Maps {
    CUtensorMap a, b0, b1;
};

constexpr int kMaxSplits = 8;  // portable cluster size
constexpr size_t kSmallSmem = 200 * 1024;  // of one CTA's stages
constexpr size_t kMaxDelta = 16 * 1024;    // of direct_products' outputs

// Lines of A in a CTA's stage: 128; in the single-CTA kernel the rows there are
// (8-line groups of the swizzle) where they are 64 or fewer.
int a_lines(int mode, int M, bool pairs = false) {
    return pairs || M > 64 ? 128 : a_mn(mode) ? 64 : (M + 7) / 8 * 8;
}

// How many clusters of 2, 4 and 8 CTAs that fill an SM each can run at the
// same time on the current device (GPCs have SMs that no cluster can use).
struct ClusterFill {
    int ctas[4];  // [log2 of the cluster's size]: CTAs
};
cudaError_t cluster_fill(int num_sms, ClusterFill *out);

// What a launch does and its estimated time.
struct Plan {
    double us;
    bool pairs;
    int splits, width, cols, nt;
    int tail;  // pairs: the tiles of the last wave that are halved
};

// Time of `ctas` CTAs that take `blocks` K blocks of `stage` bytes each, of
// matrices of `once` bytes.  Measured: an SM takes in 117 bytes per ns where
// the operands come from L2 (a pair's products keep up with that, 0.28 us per
// block), about 45 where every byte comes from HBM; the share between is the
// matrices' bytes over all that is loaded.  However few its bytes, a block
// takes 0.15 us of issue and waits.
double stream_us(int64_t ctas, int blocks, double stage, double once, int num_sms) {
    const double all = stage * blocks * (double)ctas, share = once < all ? once / all : 1.0;
    const double waves = (double)((ctas + num_sms - 1) / num_sms);
    const double block = stage * 1e-3 * (share / 45 + (1 - share) / 117);
    return waves * blocks * (block > 0.15 ? block : 0.15);
}

// Pairs of CTAs with 256-row tiles, or single ones with a tile width and a
// split of K; whichever the estimate prefers.
Plan make_plan(int mode, const GemmArgs &g, int num_sms, const ClusterFill &fill) {
    const int halves = mode == kDw ? 2 : 1, most = gated(mode) ? 64 : 128;
    const double once = 128.0 * g.kb * ((double)g.M * halves + (double)g.N * (gated(mode) ? 2 : 1));
    Plan best = {1e30, true, 1, 0, 0, 0};
    // narrower pair tiles only where every wave is full of work: a block's
    // products and its loads shrink with the columns, its rows of A do not
    for (int cols = 256; g.M > 128 && fill.ctas[1] >= 2 && cols >= 128; cols -= b_mn(mode) ? 128 : 32) {
        Plan p = {0, true, 1, gated(mode) ? cols / 2 : cols, cols, 0};
        p.nt = ceil_div(g.N, p.width);
        const int64_t tiles = (int64_t)ceil_div(g.M, 256) * halves * p.nt;
        const double stage = 2.0 * tc::kBox + cols * 64;
        p.us = stream_us(2 * tiles, g.kb, stage, once, num_sms / 2 * 2);
        // a last wave with work for half of the pairs at most is done as tiles of
        // half the columns, which take three quarters of the time (their rows of
        // A are the same).  Projection of T 8192, K 7168, N 2048 with adapters
        // 193.7 us instead of 200.3, backward pass of T 2048, H 2048, I 1536 62.9
        // instead of 64.8; many waves change by less than the noise.
        const int pairs = num_sms / 2, last = (int)(tiles % pairs);
        if (cols == 256 && tiles > pairs && last > 0 && 2 * last <= pairs) {
            const double part = (double)last / tiles;
            p.tail = last;
            p.us = stream_us(2 * (tiles - last), g.kb, stage, once * (1 - part), 2 * pairs) +
                   stream_us(4 * last, g.kb, stage - cols * 32, once * part, 2 * pairs);
        }
        if (p.us < 0.97 * best.us) best = p;
    }
    const int64_t mt = (int64_t)ceil_div(g.M, 128) * halves;
    for (int l = 0; l < 4; ++l) {
        const int splits = 1 << l;
        if (l > 0 && (g.kb / splits < 4 || fill.ctas[l] < splits)) break;
        const int64_t room = fill.ctas[l] / (mt * splits);  // tiles along N that run at once
        for (int narrow = 0; narrow < 2; ++narrow) {
            Plan p = {0, false, splits, most, 0, 0};
            if (narrow && b_mn(mode)) {
                p.width = 64;
            } else if (narrow) {
                if (room <= ceil_div(g.N, most)) break;
                p.width = (ceil_div(g.N, room) + 3) / 4 * 4;
                if (p.width < 8) p.width = 8;
            }
            p.cols = gated(mode) ? (p.width + 7) / 8 * 16 : (p.width + 15) / 16 * 16;
            p.nt = ceil_div(g.N, p.width);
            const double stage = small_stage(a_lines(mode, g.M), p.cols);
            p.us = stream_us(mt * p.nt * splits, ceil_div(g.kb, splits), stage, once, fill.ctas[l]);
            // joining the parts of a split K: the barriers, and about 20 bytes per
            // ns into a CTA through distributed shared memory
            if (l > 0) p.us += 1.2 + (g.M < 128 ? g.M : 128) * p.cols * 4 / 20e3;
            if (p.us < best.us) best = p;
        }
    }
    return best;
}

template <int MODE, int ACT>
cudaError_t small_attribute() {
    static PerDeviceOnce once;
    return per_device_once(once, [] {
        return smem_attributes(small_kernel<MODE, ACT>, kSmallSmem + kMaxDelta + 1024);
    });
}

cudaError_t cluster_fill(int num_sms, ClusterFill *out) {
    static PerDeviceOnce once;
    static ClusterFill found[PerDeviceOnce::kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = per_device_once(once, [&] {
        cudaError_t r = small_attribute<kDx, 0>();
        ClusterFill f = {{num_sms, 0, 0, 0}};
        for (int l = 1; l < 4 && r == cudaSuccess; ++l) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(1u << l);
            cfg.blockDim = dim3(kSmallThreads);
            cfg.dynamicSmemBytes = kSmallSmem + 1024;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1u << l;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            r = cudaOccupancyMaxActiveClusters(&n, small_kernel<kDx, 0>, &cfg);
            f.ctas[l] = n << l;
        }
        if (r == cudaSuccess) found[dev] = f;
        return r;
    });
    if (e == cudaSuccess) *out = found[dev];
    return e;
}

// Shared memory of the outputs that direct_products leaves.
size_t delta_bytes(int M, const Plan &plan) {
    return (size_t)ceil_div(M < 128 ? M : 128, plan.splits) * plan.width * 4;
}

// How the adapters' inner products v are computed.
enum Inner {
    kNone,   // no adapters
    kLoads,  // inner_kernel
    kNamed,  // kInner: the adapters that a tile's tokens name
    kEvery   // kInnerAll
};

struct ProjPlan {
    Plan proj;
    Inner inner;
    Plan v;                       // kNamed, kEvery
    bool direct;                  // v B^T by plain products
    int per_tile, parts, groups;  // kNamed, as in GemmArgs
};

ProjPlan plan_proj(int T, int K, int N, int n, int rank, int num_sms, const ClusterFill &fill) {
    GemmArgs g = {};
    g.M = T;
    g.N = N;
    g.kb = ceil_div(K, 64);
    ProjPlan p = {};
    // (the same plan with and without adapters: a token without one gets the
    // plain projection's bits)
    p.proj = make_plan(kProj, g, num_sms, fill);
    if (n == 0) return p;
    // Inner products by plain loads: x once per four ranks and A once per token
    // (2.5 T rank K bytes), or per up to four tokens of a run (1 to 2.5),
    // through L2 at about 6 TB/s, and 2 us for each time the SMs fill with
    // CTAs; or by kInner, 6.5 us and 0.4 per K block.
    const int mt = ceil_div(T, 128);
    int inner_splits = 1;
    for (int l = 1; l < 4 && fill.ctas[l] >= 1 << l; ++l) {
        if (2 * mt * inner_splits > num_sms || g.kb / (2 * inner_splits) < 4) break;
        inner_splits *= 2;
    }
    const int64_t ctas = (int64_t)T * rank / 4;
    const double inner_us = ctas > 8 * num_sms
                                ? 1.6 * T * (double)rank * K / 6e6 + 2.0 * ceil_div(ctas / 4, 4 * num_sms)
                                : 2.5 * T * (double)rank * K / 6e6 + 2.0;
    // v B^T by plain products: about 2.2 us for two groups of four outputs per
    // thread and 16 ranks, part of it beside the K loop; or by appended
    // blocks, 1.8 us each for the adapters that a tile may name (the tokens of
    // a long batch are taken to come in runs).
    const int rows = T < 128 ? T : 128;
    const int items = ceil_div(rows, p.proj.splits) * (p.proj.width / 4);
    const int distinct = T <= 64 ? (n < T ? n : T) : (n < 12 ? n : 12);
    const int blocks = ceil_div(adapter_blocks(distinct, rank), p.proj.splits);
    const double direct_us = 2.2 * ceil_div(items, 2 * kGroup) * ceil_div(rank, 16);
    p.direct = !p.proj.pairs && delta_bytes(T, p.proj) <= kMaxDelta &&
               direct_us < 0.3 * p.proj.us + 0.5 + 1.8 * blocks;
    const double list_us = 6.5 + 0.4 * ceil_div(g.kb, inner_splits);
    if (!p.proj.pairs && inner_us < list_us) {
        p.inner = kLoads;
        return p;
    }
    // Every adapter's A in one product (however the tokens name them), where
    // that is not much more than kInner takes for tokens that come in runs;
    // for tokens that name adapters at random kInner takes a pass over x for
    // every 128 columns of a tile's adapters.
    if (n <= 65536 / rank) {
        GemmArgs ga = g;
        ga.N = n * rank;
        p.v = make_plan(kInnerAll, ga, num_sms, fill);
        if (p.v.us < 1.5 * (p.proj.pairs ? 2.0 * T * K / 3.7e6 + 8 : list_us)) {
            p.inner = kEvery;
            return p;
        }
    }
    p.inner = kNamed;
    const int lines = rank < 128 ? rank : 128;
    p.per_tile = 128 / lines;
    p.parts = ceil_div(rank, 128);
    // SMs that K splits leave go to clusters that share a row tile's
    // adapters (a split always has work, such a cluster may find none),
    // fewer adapters at a time if that gives each of them some
    p.v = {0, false, inner_splits, 128, 128, 1};
    const int most = n < 128 ? n : 128;
    p.groups = num_sms / (mt * inner_splits);
    if (p.groups < 1) p.groups = 1;
    while (p.per_tile > 1 && ceil_div(most, p.per_tile) < p.groups) p.per_tile = (p.per_tile + 1) / 2;
    p.v.cols = (p.per_tile * lines + 15) / 16 * 16;
    const int tiles = p.parts > 1 ? most * p.parts : ceil_div(most, p.per_tile);
    if (p.groups > tiles) p.groups = tiles;
    return p;
}

// `beside`: the launch and one after it are to share the SMs (kInner and the
// single-CTA projection).
template <int MODE, int ACT>
cudaError_t launch_small(const Maps &m, GemmArgs g, const Plan &plan, int num_sms, bool beside, cudaStream_t s) {
    const cudaError_t e = small_attribute<MODE, ACT>();
    if (e != cudaSuccess) return e;
    g.mt_half = ceil_div(g.M, 128);
    g.mt = g.mt_half * (MODE == kDw ? 2 : 1);
    g.nt = plan.nt;
    g.width = plan.width;
    g.cols = plan.cols;
    g.n_fast = g.nt < g.mt;
    const int64_t ctas = (int64_t)g.mt * (MODE == kInner ? g.groups : g.nt) * plan.splits;
    const int lines = a_lines(MODE, g.M);
    const uint32_t stage = small_stage(lines, g.cols);
    // Shared memory: one CTA on an SM with all the stages, or two with half of
    // them where there are more CTAs than SMs; beside one another, 70 KB for
    // kInner and twice that for the projection, whose K loop then runs meanwhile.
    size_t budget = ctas > num_sms ? kSmallSmem / 2 : kSmallSmem;
    if (beside) budget = MODE == kInner ? 70 * 1024 : ctas > num_sms ? 70 * 1024 : 140 * 1024;
    // the products read 128 rows of A also where a stage holds fewer: room
    // behind the last stage keeps that inside the allocation
    const size_t tail = 2 * tc::kBox - lines * 128;
    // one block is for appended adapters
    const int extra = MODE == kProj && g.n > 0 && !g.direct ? 1 : 0;
    const int blocks = (int)((budget - tail) / stage) - extra;
    const int per = blocks >= 6 ? 2 : 1;  // K blocks per stage, three stages at least
    int stages = blocks / per;
    if (stages > kSmallMaxStages) stages = kSmallMaxStages;
    size_t smem = (size_t)(per * stages + extra) * stage + tail;
    if (smem < kParts) smem = kParts;
    if (MODE == kProj && g.direct) {
        g.direct = (int)smem;
        smem += delta_bytes(g.M, plan);
    }
    return launch_cluster(small_kernel<MODE, ACT>, (unsigned)ctas, kSmallThreads, smem + 1024,
                          plan.splits > 1 ? plan.splits : 0, s, m.a, m.b0, m.b1, g, stages, per, plan.splits, lines);
}

template <int MODE, int ACT>
cudaError_t launch_big(const Maps &m, GemmArgs g, const Plan &plan, int num_sms, cudaStream_t s) {
    static PerDeviceOnce once;
    const cudaError_t e = per_device_once(once, [] {
        return smem_attributes(big_kernel<MODE, ACT>, kBigSmem);
    });
    if (e != cudaSuccess) return e;
    g.mt_half = ceil_div(g.M, 256);
    g.mt = g.mt_half * (MODE == kDw ? 2 : 1);
    g.nt = plan.nt;
    g.width = plan.width;
    g.cols = plan.cols;
    g.tail = plan.tail;
    g.n_fast = g.nt < g.mt;
    g.wide = MODE != kInnerAll && g.N % 16 == 0 && ((uintptr_t)g.out0 | (uintptr_t)g.out1) % 32 == 0;
    const int64_t tiles = (int64_t)g.mt * g.nt + g.tail;
    const int pairs = (int)(tiles < num_sms / 2 ? tiles : num_sms / 2);
    return launch_cluster(big_kernel<MODE, ACT>, 2 * pairs, big_threads(MODE), kBigSmem, 0, s, m.a, m.b0, m.b1, g);
}

// Activations [rows][cols] as K-major operand A.
cudaError_t map_tokens(CUtensorMap *m, const uint16_t *x, int64_t rows, int64_t cols, bool pairs) {
    return tc::map_matrix(m, x, rows, cols, a_lines(kFwd, (int)rows, pairs));
}

// A weight [rows][cols] as K-major operand B: lines per box as the plan's kernel loads them.
cudaError_t map_weight(CUtensorMap *m, const uint16_t *w, int64_t rows, int64_t cols, const Plan &plan) {
    return tc::map_matrix(m, w, rows, cols, plan.pairs ? plan.cols / (plan.tail ? 4 : 2) : plan.width);
}

template <int MODE, int ACT>
cudaError_t launch_gemm(const Maps &m, const GemmArgs &g, const Plan &plan, int num_sms, cudaStream_t s,
                        bool beside = false) {
    if (plan.pairs) return launch_big<MODE, ACT>(m, g, plan, num_sms, s);
    return launch_small<MODE, ACT>(m, g, plan, num_sms, beside, s);
}

template <int MODE>
cudaError_t launch_act(int act, const Maps &m, const GemmArgs &g, const Plan &plan, int num_sms, cudaStream_t s) {
    if (act == MOE_ACT_SILU) return launch_gemm<MODE, MOE_ACT_SILU>(m, g, plan, num_sms, s);
    if (act == MOE_ACT_GELU) return launch_gemm<MODE, MOE_ACT_GELU>(m, g, plan, num_sms, s);
    return launch_gemm<MODE, MOE_ACT_GELU_TANH>(m, g, plan, num_sms, s);
}

}  // namespace

cudaError_t launch_gated_tc(const GatedParams &p, int num_sms, cudaStream_t s) {
    ClusterFill fill;
    cudaError_t e = cluster_fill(num_sms, &fill);
    if (e != cudaSuccess) return e;
    GemmArgs g = {};
    g.status = p.status;
    g.polls = p.polls;
    g.M = p.T;
    g.N = p.I;
    g.kb = ceil_div(p.H, 64);
    const Plan plan = make_plan(kFwd, g, num_sms, fill);
    Maps m;
    e = map_tokens(&m.a, p.x, p.T, p.H, plan.pairs);
    if (e == cudaSuccess) e = map_weight(&m.b0, p.wg, p.I, p.H, plan);
    if (e == cudaSuccess) e = map_weight(&m.b1, p.wu, p.I, p.H, plan);
    if (e != cudaSuccess) return e;
    if (p.h) {
        g.out0 = p.h;
        return launch_act<kFwd>(p.act, m, g, plan, num_sms, s);
    }
    g.dh = p.dh;
    g.out0 = p.dgu;
    return launch_act<kBwd>(p.act, m, g, plan, num_sms, s);
}

cudaError_t launch_dx_tc(const GatedParams &p, int num_sms, cudaStream_t s) {
    ClusterFill fill;
    cudaError_t e = cluster_fill(num_sms, &fill);
    if (e != cudaSuccess) return e;
    GemmArgs g = {};
    g.status = p.status;
    g.polls = p.polls;
    g.M = p.T;
    g.N = p.H;
    g.kb_half = ceil_div(p.I, 64);
    g.kb = 2 * g.kb_half;
    g.out0 = p.dx;
    const Plan plan = make_plan(kDx, g, num_sms, fill);
    Maps m;
    e = tc::map_halves(&m.a, p.dgu, p.T, p.I, a_lines(kDx, p.T, plan.pairs));
    if (e == cudaSuccess) e = tc::map_matrix(&m.b0, p.wg, p.I, p.H);
    if (e == cudaSuccess) e = tc::map_matrix(&m.b1, p.wu, p.I, p.H);
    if (e != cudaSuccess) return e;
    return launch_gemm<kDx, 0>(m, g, plan, num_sms, s);
}

cudaError_t launch_dw_tc(const GatedParams &p, bool after_dx, int num_sms, cudaStream_t s) {
    ClusterFill fill;
    cudaError_t e = cluster_fill(num_sms, &fill);
    if (e != cudaSuccess) return e;
    Maps m;
    e = tc::map_halves(&m.a, p.dgu, p.T, p.I);
    if (e == cudaSuccess) e = tc::map_matrix(&m.b0, p.x, p.T, p.H);
    if (e != cudaSuccess) return e;
    m.b1 = m.b0;
    GemmArgs g = {};
    g.status = p.status;
    g.polls = p.polls;
    g.M = p.I;
    g.N = p.H;
    g.kb = ceil_div(p.T, 64);
    g.out0 = p.dwg;
    g.out1 = p.dwu;
    g.late = after_dx;
    return launch_gemm<kDw, 0>(m, g, make_plan(kDw, g, num_sms, fill), num_sms, s);
}

cudaError_t launch_proj_tc(const AdapterParams &p, int num_sms, cudaStream_t s) {
    ClusterFill fill;
    cudaError_t e = cluster_fill(num_sms, &fill);
    if (e != cudaSuccess) return e;
    const ProjPlan plan = plan_proj(p.T, p.K, p.N, p.n, p.rank, num_sms, fill);
    GemmArgs g = {};
    g.status = p.status;
    g.polls = p.polls;
    g.M = p.T;
    g.N = p.N;
    g.kb = ceil_div(p.K, 64);
    Maps m;
    const bool beside = plan.inner == kNamed && !plan.proj.pairs;
    if (p.n > 0) {
        g.ids = p.ids;
        g.scale = p.scale;
        g.lora_b = p.b;
        g.v = reinterpret_cast<uint16_t *>(p.v);
        g.n = p.n;
        g.rank = p.rank;
        g.direct = plan.direct;
        g.per_tile = plan.per_tile;
        g.parts = plan.parts;
        g.groups = plan.groups;
        if (plan.inner == kLoads) {
            if ((e = launch_inner(p, true, num_sms, s)) != cudaSuccess) return e;
        } else if (plan.inner == kEvery) {
            GemmArgs ga = g;
            ga.N = p.n * p.rank;
            if ((e = map_tokens(&m.a, p.x, p.T, p.K, plan.v.pairs)) != cudaSuccess) return e;
            if ((e = map_weight(&m.b0, p.a, ga.N, p.K, plan.v)) != cudaSuccess) return e;
            m.b1 = m.b0;
            if ((e = launch_gemm<kInnerAll, 0>(m, ga, plan.v, num_sms, s)) != cudaSuccess) return e;
        } else {
            if ((e = map_tokens(&m.a, p.x, p.T, p.K, false)) != cudaSuccess) return e;
            if ((e = tc::map_stack(&m.b0, p.a, p.n, p.rank, p.K, p.rank < 128 ? p.rank : 128)) != cudaSuccess)
                return e;
            m.b1 = m.b0;
            if ((e = launch_small<kInner, 0>(m, g, plan.v, num_sms, beside, s)) != cudaSuccess) return e;
        }
    }
    if ((e = map_tokens(&m.a, p.x, p.T, p.K, plan.proj.pairs)) != cudaSuccess) return e;
    if ((e = map_weight(&m.b0, p.w, p.N, p.K, plan.proj)) != cudaSuccess) return e;
    m.b1 = m.b0;
    g.residual = p.residual;
    g.out0 = p.y;
    return launch_gemm<kProj, 0>(m, g, plan.proj, num_sms, s, beside);
}

cudaError_t adapter_plan(int T, int K, int N, int n, int rank, int num_sms, const int *cluster_ctas,
                         AdapterPlan *out) {
    *out = AdapterPlan{};
    if (gemv_supported(T, K)) {
        out->splits = 1;
        out->inner = n > 0 ? kLoads : kNone;
        out->inner_splits = n > 0;
        out->direct = n > 0;
        return cudaSuccess;
    }
    ClusterFill fill = {{num_sms, 0, 0, 0}};
    if (cluster_ctas) {
        for (int l = 1; l < 4; ++l) fill.ctas[l] = cluster_ctas[l - 1];
    } else {
        const cudaError_t e = cluster_fill(num_sms, &fill);
        if (e != cudaSuccess) return e;
    }
    const ProjPlan p = plan_proj(T, K, N, n, rank, num_sms, fill);
    out->products = p.proj.pairs ? 2 : 1;
    out->splits = p.proj.splits;
    out->inner = p.inner;
    out->inner_splits = p.inner == kNone ? 0 : p.inner == kLoads ? 1 : p.v.splits;
    out->direct = p.direct;
    out->groups = p.groups;
    return cudaSuccess;
}

}  // namespace moe
