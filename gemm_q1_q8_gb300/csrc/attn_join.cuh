// What the two attention kernels share: the cut of their work into runs of units, and the joining of tiles that runs share.
//
// A kernel's units (pieces of one tile's keys), in the order sequence, kv head, row tile, key, are cut into equal runs.  A run that begins and
// ends a tile writes its rows; of a tile that several runs share, each leaves partial sums, and attn_join_kernel adds them in the order of the
// runs: the result does not depend on timing.
#pragma once

#include "layer_ops.cuh"

namespace gq {
namespace {

constexpr float kNone = -3e38f;                    // running maximum of a row that has seen no key, below every finite score
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }    // -126 <= e <= 127

// A capped score times log2 e, cap * tanh(y), for 16-bit queries; x = 2 y log2 e.  1 - 2 / (e^2y + 1) is off by some 2^-22 absolutely, which a cap above
// kCapNear makes felt.  ANY takes every cap: below |y| = 1/4 the series of tanh (off by 2^-21 of itself).
constexpr float kCapNear = 512.f;
template <bool ANY>
__device__ __forceinline__ float capped16(float x, float cap) {
    const float far = fmaf(-2.f * cap, rcp(ex2(x) + 1.f), cap);
    if (!ANY) return far;
    const float y = x * 0.34657359f, z = y * y;
    const float series = cap * y * fmaf(z, fmaf(z, fmaf(z, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
    return fabsf(y) < 0.25f ? series : far;
}

// The query rows of sequence b.  q_start comes from device memory: rows outside [0, a.rows) are neither read nor written.
struct QueryRows {
    int q0, T;             // first row, query tokens
    int tokens;            // those that are computed: at most max_q of them, and their rows exist
};
__device__ __forceinline__ QueryRows query_rows(const AttnArgs& a, int b) {
    const int limit = a.rows >= 0 ? a.rows : a.q_start[a.seqs];
    QueryRows r;
    r.q0 = a.q_start[b];
    const int end = a.q_start[b + 1];
    if (r.q0 < 0 || end < r.q0 || end > limit) report_error(kErrIndex);
    if (r.q0 < 0 || end < r.q0 || r.q0 >= limit) {
        r.q0 = r.T = r.tokens = 0;
        return r;
    }
    r.T = end - r.q0;
    if (r.T > a.max_q) report_error(kErrIndex);
    r.tokens = min(min(r.T, a.max_q), limit - r.q0);
    return r;
}

// x / d and x % d, in 32 bits where x allows
__device__ __forceinline__ void div_mod(long long x, int d, int& quot, int& rest) {
    if (x < 0x7fffffffll) {
        quot = static_cast<int>(x) / d;
        rest = static_cast<int>(x) - quot * d;
    } else {
        quot = static_cast<int>(x / d);
        rest = static_cast<int>(x % d);
    }
}

// The workspace: partial sums [2][runs][rows][HD] (heads, tails) relative to 2^m, their m and l [2][runs][rows], and for each run the tile
// whose end it has after an earlier run began it.  (The row kernel's f32 sums that leave the registers stand in their own run's tail, until its
// block's open tiles meet.)
struct Head {
    int first;             // the run that began the tile; -1: none
    int q0, tile0, rows, hk;
};
struct Parts {
    float* o;
    float2* ml;
    Head* head;
};
inline size_t parts_bytes(size_t runs, size_t rows, size_t hd) { return runs * (2 * rows * (hd * 4 + 8) + sizeof(Head)); }
inline Parts parts_at(void* workspace, size_t runs, size_t rows, size_t hd) {
    Parts p;
    p.o = static_cast<float*>(workspace);
    p.ml = reinterpret_cast<float2*>(p.o + 2 * runs * rows * hd);
    p.head = reinterpret_cast<Head*>(p.ml + 2 * runs * rows);
    return p;
}

template <typename K, typename... A>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, int smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A block looks at GROUP neighbouring runs (the warps of a block of the first kernel) with the blocks of its column, a warp takes rows of their
// heads, a lane four columns (256: two times four).  The group has joined its tails already: the first of a tile's holds the sum.  Sixteen
// (eight) parts are requested at once, before their weights are known.  Rows of sequences without keys are written here too.
// It is bound by latency, three dependent loads: with a block for each run, most of them without a head, it was its own eleven waves of blocks.
template <typename T, int HD, int ROWS, int GROUP>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a, const Parts parts, int runs) {
    constexpr int kWarps = 8, kLanes = HD == 64 ? 16 : 32, kRuns = HD == 256 ? 2 : 1, kBatch = (ROWS > 8 ? 8 : 16) / kRuns;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = a.q_heads / a.kv_heads;
    const int run0 = blockIdx.x * GROUP;
    unsigned heads = __ballot_sync(0xffffffffu, lane < GROUP && run0 + lane < runs && parts.head[min(run0 + lane, runs - 1)].first >= 0);
    // the rows of the heads one after another: this warp's are warp + kWarps * blockIdx.y and every kWarps * gridDim.y further
    for (int at = warp + kWarps * blockIdx.y; heads; at -= ROWS, heads &= heads - 1) {
        const int run = run0 + __ffs(heads) - 1;
        if (at >= ROWS) continue;
        const Head head = parts.head[run];
        for (; at < ROWS; at += kWarps * gridDim.y) {
            const int r = at;
            if (r >= head.rows) continue;
            // parts: the tail of the run that began the tile, those of the groups between, the head
            const int group0 = head.first / GROUP, n = (run + GROUP - 1) / GROUP - group0 + 1;
            float top = kNone, l = 0.f;
            float4 v[kRuns];
#pragma unroll
            for (int c = 0; c < kRuns; ++c) v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int j0 = 0; j0 < n; j0 += kBatch) {
                auto slot = [&](int j) {
                    const size_t s = j >= n - 1 ? run : runs + (j == 0 ? head.first : (group0 + j) * GROUP);
                    return s * ROWS + r;
                };
                const int j = j0 + lane % kBatch;
                const float2 ml = j < n ? parts.ml[slot(j)] : make_float2(kNone, 0.f);
                float4 x[kBatch][kRuns];
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
#pragma unroll
                    for (int c = 0; c < kRuns; ++c)
                        if (j0 + k < n) x[k][c] = *reinterpret_cast<const float4*>(parts.o + slot(j0 + k) * HD + 128 * c + 4 * (lane % kLanes));
                float up = fmaxf(ml.x, top);
#pragma unroll
                for (int o = kBatch / 2; o > 0; o >>= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, o));
                const float f = ex2(ml.x - up), down = ex2(top - up);
                float sum = f * ml.y;
#pragma unroll
                for (int o = kBatch / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                l = fmaf(l, down, sum);
                top = up;
#pragma unroll
                for (int c = 0; c < kRuns; ++c) v[c] = make_float4(v[c].x * down, v[c].y * down, v[c].z * down, v[c].w * down);
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const float h = __shfl_sync(0xffffffffu, f, k);
                    if (j0 + k < n)
#pragma unroll
                        for (int c = 0; c < kRuns; ++c)
                            v[c] = make_float4(fmaf(h, x[k][c].x, v[c].x), fmaf(h, x[k][c].y, v[c].y), fmaf(h, x[k][c].z, v[c].z), fmaf(h, x[k][c].w, v[c].w));
                }
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            T* out = static_cast<T*>(a.out) + (head.q0 + (head.tile0 + r) / group) * a.out_stride + (head.hk * group + (head.tile0 + r) % group) * HD;
#pragma unroll
            for (int c = 0; c < kRuns; ++c)
                if (lane < kLanes) store4(out + 128 * c + 4 * lane, make_float4(v[c].x * inv, v[c].y * inv, v[c].z * inv, v[c].w * inv));
        }
    }
    if (blockIdx.y == 0)
        for (int b = blockIdx.x; b < a.seqs; b += gridDim.x) {
            if (a.kv_len[b] > 0) continue;
            const QueryRows rows = query_rows(a, b);
            for (int tok = warp; tok < rows.tokens; tok += kWarps)
                for (int d = lane * 4; d < a.q_heads * HD; d += 128)
                    store4(static_cast<T*>(a.out) + (rows.q0 + tok) * a.out_stride + d, make_float4(0.f, 0.f, 0.f, 0.f));
        }
}

template <typename T, int HD, int ROWS, int GROUP>
cudaError_t launch_join(const AttnArgs& a, const Parts& parts, int runs, cudaStream_t s) {
    constexpr int kBlocksUp = ROWS > 16 ? 8 : 4;
    return launch_dependent(attn_join_kernel<T, HD, ROWS, GROUP>, dim3((runs + GROUP - 1) / GROUP, kBlocksUp), 256, 0, s, a, parts, runs);
}

}  // namespace
}  // namespace gq
