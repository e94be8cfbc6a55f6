// Log probabilities of given tokens, the entropy and the best alternatives of rows of logits.
//
//   p = softmax(scale * x);  in powers of two, c = scale * log2(e), t = c (x - max x), s = sum 2^t:
//   logprob = scale (x[token] - max x) - log2(s) ln 2,  H = (log2 s - (sum 2^t t) / s) ln 2.
// A thread block takes a row, or a part of one where there are few rows: one pass over the logits keeps the largest and the two sums a
// thread (relative to one of its logits, exchanged where another is far above it).  The k best need no sorting: the k-th largest of the threads' own maxima bounds the
// k-th largest logit from below, and a search over the bits of an order-preserving key finds it by 16 block-wide counts.  Only the threads whose maximum
// reaches the bound (about k) have their logits read once more, from L2, by a warp together.  Equal values go by
// the lower index: where too many share the bound (masked rows), they are taken in the order of their index.
// Parts are joined in their order: within a cluster, or by a second kernel.  Bound by HBM for many rows, by round trips and the
// searches' barriers for one.
#include <algorithm>

#include "layer_ops.cuh"

namespace gq {
GQ_ERROR_ACCESSOR(logprobs)

namespace {

constexpr int kJoinThreads = 256;
constexpr int kMaxTop = 32, kMaxSplits = 64;
constexpr int kFound = 2048;                      // candidates
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float d;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
    return d;
}

// Values in the order of unsigned numbers: both zeros alike, NaN above all, 0 below all
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    if (x != x) return ~0u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    if (key == ~0u) return __uint_as_float(0x7fffffffu);
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ uint64_t entry(uint32_t key, uint32_t index) { return static_cast<uint64_t>(key) << 32 | (0xffffffffu - index); }

// s = sum 2^t, u = sum 2^t t, t = c (x - m) with m the largest logit.  A thread first sums relative to a logit near its largest (kRise below).  Near: t = c x - r with
// r = c m rounded, one fma, while |r| < 2^20 (r is then off by at most 1/32, the same in every term).  Far: t = c (x - m), for rows whose largest logit is further
// out, summed once more.
struct Sums { float m, s, u; };
// A thread's m stays until a logit is further above it.  Were it the running maximum, one of a warp's 32 would rise at almost every one of a row's few
// steps; but t is rounded relative to its size and u is a difference of what both signs of t give, so with m far below (60 here) what is left
// of log2 s and the entropy of a row with one likely token is off by 2^-19.  With 8, t of what counts is off by 2^-22 at most.
constexpr float kRise = 8.f;
constexpr float kNear = 1048576.f;
__device__ __forceinline__ bool is_far(float m, float c) { return !(fabsf(c * m) < kNear); }
__device__ __forceinline__ float floor_of(float c) { return -1.0001f * kNear / c; }            // a first m that is far

__device__ __forceinline__ float power(float x, float m, float c, bool far) { return max_nan(far ? c * (x - m) : fmaf(c, x, -(c * m)), -1e4f); }
__device__ __forceinline__ void rescale(Sums& a, float m, float c, bool far) {
    const float d = max_nan(far ? c * (a.m - m) : c * a.m - c * m, -1e4f), f = exp2_fast(d);
    a.u = fmaf(a.s, d, a.u) * f;
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ void add(Sums& a, float x, float c, bool far) {
    const float t = power(x, a.m, c, far), e = exp2_fast(t);                       // -inf: no weight, and no 0 * inf
    a.s += e;
    a.u = fmaf(e, t, a.u);
}
// A thread's sums relative to its largest logit `top`, whose own term is taken out as it was added and becomes exactly 1: with every t at most 0 then, log2 s is not below 0,
// and a row of one allowed token gives 0.  Where no logit is above `least`, m is that.
__device__ __forceinline__ void rebase(Sums& a, float top, float least, float c, bool far) {
    if (top <= least) return;
    const float t = power(top, a.m, c, far), e = exp2_fast(t), f = exp2_fast(-t);
    const float s = a.s - e, u = a.u - e * t;                                      // the product as add rounds it for a first term
    a.u = fmaf(-s, t, u) * f;
    a.s = fmaf(s, f, 1.f);
    a.m = top;
}
// The sums of a warp's lanes, or of a group's of N: the maximum first, so that each is rescaled once
template <int N>
__device__ __forceinline__ Sums of_lanes(Sums t, float c) {
    float m = t.m;
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    rescale(t, m, c, true);
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
        t.s += __shfl_xor_sync(0xffffffffu, t.s, o);
        t.u += __shfl_xor_sync(0xffffffffu, t.u, o);
    }
    return t;
}

// 16 bytes of logits
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int W = 4;
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&r)[N]) {
        float m = max_nan(max_nan(__uint_as_float(r[0].x), __uint_as_float(r[0].y)), max_nan(__uint_as_float(r[0].z), __uint_as_float(r[0].w)));
        if (N == 2) m = max_nan(m, max_nan(max_nan(__uint_as_float(r[N - 1].x), __uint_as_float(r[N - 1].y)), max_nan(__uint_as_float(r[N - 1].z), __uint_as_float(r[N - 1].w))));
        return m;
    }
    static __device__ __forceinline__ float one(const uint4& r, int j) { return __uint_as_float(j == 0 ? r.x : j == 1 ? r.y : j == 2 ? r.z : r.w); }
    static __device__ __forceinline__ void get(const uint4& r, float (&v)[4]) {
        v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y); v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int W = 8;
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t m;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
        return m;
    }
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&r)[N]) {        // in packed maxima
        uint32_t m = max2(max2(r[0].x, r[0].y), max2(r[0].z, r[0].w));
        if (N == 2) m = max2(m, max2(max2(r[N - 1].x, r[N - 1].y), max2(r[N - 1].z, r[N - 1].w)));
        return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
    static __device__ __forceinline__ float one(const uint4& r, int j) {
        const uint32_t w = j < 2 ? r.x : j < 4 ? r.y : j < 6 ? r.z : r.w;
        return __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
    }
    static __device__ __forceinline__ void get(const uint4& r, float (&v)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <> struct Vec<__half> {
    static constexpr int W = 8;
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t m;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
        return m;
    }
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&r)[N]) {        // in packed maxima
        uint32_t m = max2(max2(r[0].x, r[0].y), max2(r[0].z, r[0].w));
        if (N == 2) m = max2(m, max2(max2(r[N - 1].x, r[N - 1].y), max2(r[N - 1].z, r[N - 1].w)));
        return max_nan(__half2float(__ushort_as_half(static_cast<unsigned short>(m))), __half2float(__ushort_as_half(static_cast<unsigned short>(m >> 16))));
    }
    static __device__ __forceinline__ float one(const uint4& r, int j) {
        const uint32_t w = j < 2 ? r.x : j < 4 ? r.y : j < 6 ? r.z : r.w;
        return __half2float(__ushort_as_half(static_cast<unsigned short>(j & 1 ? w >> 16 : w)));
    }
    static __device__ __forceinline__ void get(const uint4& r, float (&v)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
};

__device__ __forceinline__ float logprob_of(float x, const Sums& a, float scale) {
    if (a.s == 0.f) return x != x ? x : __uint_as_float(0xff800000u);              // nothing has any weight
    return scale * (x - a.m) - log2f(a.s) * kLn2;
}
template <typename T>
__device__ __forceinline__ void finish_row(const LogprobArgs& a, size_t row, const Sums& t) {
    if (a.entropy) {
        const float h = t.s == 0.f ? 0.f : (log2f(t.s) - t.u / t.s) * kLn2;
        a.entropy[row] = h < 0.f ? 0.f : h;                                       // by its rounding; NaN stays
    }
    if (a.logprob) {
        const int64_t tok = a.tokens[row];
        float r = 0.f;
        if (tok >= a.vocab) {
            r = __uint_as_float(0x7fffffffu);
            report_error(kErrIndex);
        } else if (tok >= 0) r = logprob_of(to_f32(static_cast<const T*>(a.x)[row * a.stride + tok]), t, a.scale);
        a.logprob[row] = r;
    }
}

// The workspace of rows in parts: Sums (as float4) and `top` entries of each part
__host__ __device__ __forceinline__ float4* part_sums(void* w) { return static_cast<float4*>(w); }
__device__ __forceinline__ uint64_t* part_best(void* w, size_t parts) { return reinterpret_cast<uint64_t*>(static_cast<float4*>(w) + parts); }

// A row's parts: their sums in their order, and the best of the parts' best.  By a whole block; sums_of(i) and best_of(i) give part i's sums and the
// i-th of all parts' entries.
template <typename T, int kThreads, int kEntries, typename S, typename B>
__device__ __forceinline__ void join_row(const LogprobArgs& a, size_t row, int splits, float c, uint64_t* found, int* count, S sums_of, B best_of) {
    constexpr int PER = (kEntries + kThreads - 1) / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, k = a.top;
    float most = kLowest;
    for (int i = lane; i < splits; i += 32) most = max_nan(most, sums_of(i).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
    Sums t = {most, 0.f, 0.f};
    for (int i = lane; i < splits; i += 32) {
        const float4 v = sums_of(i);
        Sums p = {v.x, v.y, v.z};
        rescale(p, most, c, true);
        t.u += p.u;
        t.s += p.s;
    }
    t = of_lanes<32>(t, c);
    if (tid == 0) {
        finish_row<T>(a, row, t);
        *count = 0;
    }
    if (k == 0) return;
    uint64_t mine[PER], top = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        mine[i] = tid + i * kThreads < splits * k ? best_of(tid + i * kThreads) : 0;
        top = max(top, mine[i]);
    }
    // as for a part's threads, over entries, which are all different: with all their bits, k threads reach the bound
    uint64_t bound = 0;
    int reach = kThreads;
    for (int b = 63; b >= 0; --b) {
        if (b == 47 && reach <= 2 * k + 16) break;
        const uint64_t try_ = bound | 1ull << b;
        const int q = __syncthreads_count(top >= try_);
        if (q >= k) {
            bound = try_;
            reach = q;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (mine[i] && mine[i] >= bound) found[atomicAdd(count, 1)] = mine[i];
    __syncthreads();
    const int have = *count;
    for (int i = tid; i < have; i += kThreads) {
        const uint64_t e = found[i];
        int rank = 0;
        for (int j = 0; j < have; ++j) rank += found[j] > e;
        if (rank < k) {
            a.top_ids[row * k + rank] = 0xffffffffu - static_cast<uint32_t>(e);
            a.top_values[row * k + rank] = logprob_of(value_of(static_cast<uint32_t>(e >> 32)), t, a.scale);
        }
    }
}

// Shared memory of another block of the cluster
__device__ __forceinline__ uint32_t peer(const void* p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// CLUSTER > 1: so many blocks, the parts of a row, are a cluster, whose first joins them.  Blocks an SM of the small ones: f32 at ten would spill its
// sums' registers (4096 rows of 49152: nine 132 us, ten 140, eight 146).
template <typename T, int kThreads, int CLUSTER>
__global__ void __launch_bounds__(kThreads, kThreads == 128 ? (sizeof(T) == 4 ? 9 : 10) : CLUSTER > 1 ? 2 : 3) logprobs_kernel(const LogprobArgs a, int splits, int part) {
    constexpr int W = Vec<T>::W;
    __shared__ uint64_t found[kFound];
    __shared__ Sums warp_sums[kThreads / 32];
    __shared__ int count, warp_counts[kThreads / 32];
    __shared__ float4 own_sums;                                            // a cluster's part
    __shared__ uint64_t own_best[kMaxTop];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const unsigned row32 = splits == 1 ? blockIdx.x : blockIdx.x / splits;
    const size_t row = row32;
    const int split = blockIdx.x - row32 * splits, v0 = split * part, n = max(0, min(part, a.vocab - v0));
    const T* x = static_cast<const T*>(a.x) + row * a.stride + v0;
    const int k = a.top;
    const float c = a.scale * kLog2e;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // whole vectors, and up to 7 logits on either side of them, one a thread
    const int head = min(n, static_cast<int>((16 - reinterpret_cast<uintptr_t>(x) % 16) % 16 / sizeof(T)));
    const int vecs = (n - head) / W, tail = n - head - vecs * W;
    const int extra = tid < head ? tid : tid >= 32 && tid - 32 < tail ? head + vecs * W + tid - 32 : -1;
    const uint4* xv = reinterpret_cast<const uint4*>(x + head);
    const float none = __uint_as_float(0xff800000u);
    float top = none;                                                             // the thread's largest
    Sums t;
    auto stream = [&](bool far) {
        const float least = far ? kLowest : max_nan(floor_of(c), kLowest);
        t = {least, 0.f, 0.f};
        bool hidden = false;
        if (extra >= 0) {
            const float f = to_f32(x[extra]);
            top = max_nan(top, f);
            if (f > least) t.m = f;
            add(t, f, c, far);
        }
        auto step = [&](const auto& r) {                                   // one or two vectors
            constexpr int N = sizeof(r) / sizeof(uint4);
            const float m = Vec<T>::largest(r);
            top = max_nan(top, m);
            if ((far ? c * (m - t.m) : fmaf(c, m, -(c * t.m))) > kRise) rescale(t, m, c, far);
            if (far) {
#pragma unroll 1
                for (int i = 0; i < N; ++i)
#pragma unroll 1
                    for (int j = 0; j < W; ++j) add(t, Vec<T>::one(i ? r[N - 1] : r[0], j), c, true);
                return;
            }
            // two sums side by side, packed
            const float2 low = make_float2(-(c * t.m), -(c * t.m)), cc = make_float2(c, c);
            float2 s2 = make_float2(0.f, 0.f), u2 = s2;
            if (!hidden) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float f[W];
                    Vec<T>::get(r[i], f);
#pragma unroll
                    for (int j = 0; j < W; j += 2) {
                        const float2 d = ffma2(cc, make_float2(f[j], f[j + 1]), low);
                        const float2 e = make_float2(exp2_fast(d.x), exp2_fast(d.y));
                        s2 = fadd2(s2, e);
                        u2 = ffma2(e, d, u2);
                    }
                }
                hidden = u2.x + u2.y != u2.x + u2.y;                       // 0 * inf
            }
            if (hidden) {
                // a logit of -inf has no weight; rows with one take this way from there on
                s2 = u2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float f[W];
                    Vec<T>::get(r[i], f);
#pragma unroll
                    for (int j = 0; j < W; j += 2) {
                        float2 d = ffma2(cc, make_float2(f[j], f[j + 1]), low);
                        d = make_float2(max_nan(d.x, -1e4f), max_nan(d.y, -1e4f));
                        const float2 e = make_float2(exp2_fast(d.x), exp2_fast(d.y));
                        s2 = fadd2(s2, e);
                        u2 = ffma2(e, d, u2);
                    }
                }
            }
            t.s += s2.x + s2.y;
            t.u += u2.x + u2.y;
        };
        // two vectors a step, whose loads are ahead by one; at most one is left
        uint4 ahead[2];
        int v = tid;
        if (v < vecs) ahead[0] = xv[v];
        if (v + kThreads < vecs) ahead[1] = xv[v + kThreads];
#pragma unroll 2
        for (; v + kThreads < vecs; v += 2 * kThreads) {
            const uint4 r[2] = {ahead[0], ahead[1]};
            if (v + 2 * kThreads < vecs) ahead[0] = xv[v + 2 * kThreads];
            if (v + 3 * kThreads < vecs) ahead[1] = xv[v + 3 * kThreads];
            step(r);
        }
        if (v < vecs) {
            const uint4 r[1] = {ahead[0]};
            step(r);
        }
        rebase(t, top, least, c, far);
        t = of_lanes<32>(t, c);
        if (lane == 0) warp_sums[warp] = t;
        if (tid == 0) count = 0;
        __syncthreads();
        t = of_lanes<kThreads / 32>(warp_sums[lane % (kThreads / 32)], c);
    };
    stream(false);
    if (is_far(t.m, c)) {                                                  // the same in every thread
        __syncthreads();
        stream(true);
    }
    const uint32_t mine = key_of(top);
    if (tid == 0) {
        if (CLUSTER > 1) own_sums = make_float4(t.m, t.s, t.u, 0.f);
        else if (splits == 1) finish_row<T>(a, row, t);
        else part_sums(a.workspace)[blockIdx.x] = make_float4(t.m, t.s, t.u, 0.f);
    }
    auto join = [&] {
        if (CLUSTER == 1) return;
        cluster_sync();
        if (split == 0)
            join_row<T, kThreads, CLUSTER * kMaxTop>(a, row, CLUSTER, c, found, &count, [&](int i) {
                float4 v;
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(peer(&own_sums, i)));
                return v;
            }, [&](int i) {
                uint64_t v;
                asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer(own_best + i % k, i / k)));
                return v;
            });
        cluster_sync();                                                    // a block's shared memory is there until the first has read it
    };
    if (k == 0) {
        join();
        return;
    }

    // bound: the largest number that k threads' maxima reach, in its upper 16 bits, or exactly
    uint32_t bound = 0;
    auto search = [&](int from, int to, int q) {
        for (int b = from; b >= to; --b) {
            const uint32_t try_ = bound | 1u << b;
            const int reach = __syncthreads_count(mine >= try_);
            if (reach >= k) {
                bound = try_;
                q = reach;
            }
        }
        return q;
    };
    // entries of the threads that reach the bound, of logits at least `least`
    auto gather = [&](uint32_t least) {
        for (unsigned left = __ballot_sync(0xffffffffu, mine >= least); left; left &= left - 1) {
            const int other = warp * 32 + __ffs(left) - 1;
            for (int v = other + lane * kThreads; v < vecs; v += 32 * kThreads) {
                float f[W];
                Vec<T>::get(xv[v], f);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const uint32_t key = key_of(f[j]);
                    if (key >= least) {
                        const int at = atomicAdd(&count, 1);
                        if (at < kFound) found[at] = entry(key, v0 + head + v * W + j);
                    }
                }
            }
        }
        if (extra >= 0) {
            const uint32_t key = key_of(to_f32(x[extra]));
            if (key >= least) {
                const int at = atomicAdd(&count, 1);
                if (at < kFound) found[at] = entry(key, v0 + extra);
            }
        }
        __syncthreads();
        return count;
    };
    const int few = 2 * k + 16;
    uint64_t kept = 0;
    int have = kFound + 1;
    int reach;
    if (k == 1) {
        __shared__ uint32_t largest[kThreads / 32];
        bound = __reduce_max_sync(0xffffffffu, mine);
        if (lane == 0) largest[warp] = bound;
        __syncthreads();
        bound = __reduce_max_sync(0xffffffffu, largest[lane % (kThreads / 32)]);
        reach = __syncthreads_count(mine >= bound);
    } else reach = search(31, 16, kThreads);
    if (reach <= few) have = gather(bound);
    if (have > kFound) {
        // too many near the bound: the exact one
        __syncthreads();
        if (tid == 0) count = 0;
        reach = search(15, 0, reach);                                                    // its barriers stand between the zero and the entries
        have = kFound + 1;
        if (reach <= few) have = gather(bound);
        if (have > kFound) {
            // of the logits at the bound the first few, in their order, behind those above it
            __syncthreads();
            if (tid == 0) count = 0;
            __syncthreads();
            have = bound == ~0u ? 0 : gather(bound + 1);
            if (have > kFound) {
                // too many above it with fewer than k threads: one after another, each the largest below the one before
                uint64_t below = ~0ull;
                for (have = 0; have < k; ++have) {
                    uint64_t best = 0;
                    for (int i = tid; i < n; i += kThreads) {
                        const uint64_t e = entry(key_of(to_f32(x[i])), v0 + i);
                        if (e < below && e > best) best = e;
                    }
                    __syncthreads();
                    found[tid] = best;
                    __syncthreads();
                    for (int o = kThreads / 2; o > 0; o >>= 1) {
                        if (tid < o) found[tid] = max(found[tid], found[tid + o]);
                        __syncthreads();
                    }
                    below = found[0];
                    if (tid == have) kept = below;
                    if (below == 0) break;
                }
                __syncthreads();
                if (tid < have) found[tid] = kept;
                __syncthreads();
            }
            int need = k - have;
            for (int at = 0; at < n && need > 0; at += kThreads) {
                const bool is = at + tid < n && key_of(to_f32(x[at + tid])) == bound;
                const unsigned who = __ballot_sync(0xffffffffu, is);
                if (lane == 0) warp_counts[warp] = __popc(who);
                __syncthreads();
                int before = __popc(who & ((1u << lane) - 1)), all = 0;
                for (int w = 0; w < kThreads / 32; ++w) {
                    if (w < warp) before += warp_counts[w];
                    all += warp_counts[w];
                }
                if (is && before < need) found[have + before] = entry(bound, v0 + at + tid);
                have += min(all, need);
                need -= min(all, need);
                __syncthreads();
            }
        }
    }
    // the place of each among them
    for (int i = tid; i < have; i += kThreads) {
        const uint64_t e = found[i];
        int rank = 0;
        for (int j = 0; j < have; ++j) rank += found[j] > e;
        if (rank < k) {
            if (CLUSTER > 1) own_best[rank] = e;
            else if (splits == 1) {
                a.top_ids[row * k + rank] = 0xffffffffu - static_cast<uint32_t>(e);
                a.top_values[row * k + rank] = logprob_of(value_of(static_cast<uint32_t>(e >> 32)), t, a.scale);
            } else part_best(a.workspace, gridDim.x)[static_cast<size_t>(blockIdx.x) * k + rank] = e;
        }
    }
    // a part of fewer logits
    if (splits > 1 && tid >= have && tid < k) {
        if (CLUSTER > 1) own_best[tid] = 0;
        else part_best(a.workspace, gridDim.x)[static_cast<size_t>(blockIdx.x) * k + tid] = 0;
    }
    join();
}

// One block a row, where its parts went through the workspace.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) logprobs_join_kernel(const LogprobArgs a, int splits) {
    __shared__ uint64_t found[kMaxSplits * kMaxTop];
    __shared__ int count;
    const size_t row = blockIdx.x, parts = static_cast<size_t>(gridDim.x) * splits;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float4* sums = part_sums(a.workspace) + row * splits;
    const uint64_t* best = part_best(a.workspace, parts) + row * splits * a.top;
    join_row<T, kJoinThreads, kMaxSplits * kMaxTop>(a, row, splits, a.scale * kLog2e, found, &count, [&](int i) { return sums[i]; },
                                                    [&](int i) { return best[i]; });
}

// Parts of a row, each a block: up to two blocks an SM, of at least 2048 logits.  Up to eight are a cluster and joined there (one launch instead of two: one row of
// 49152 called from Python 22.7 -> 18.8 us); more, through the workspace, where eight would have long ways of their own on a GPU that is mostly idle.
struct Parts { int splits; bool cluster; };
constexpr int kMaxWideRows = 9;                   // rows that may go through the workspace
Parts parts_of(int m, int vocab) {
    int n = 8;
    while (n > 1 && (m > 2 * 152 / n || vocab / n < 2048)) n /= 2;
    if (n < 8 || vocab <= 8 * 32768 || m > kMaxWideRows) return {n, n > 1};
    return {std::min(kMaxSplits, std::min(3 * 152 / m, vocab / 16384)), false};
}

template <typename K, typename... A>
cudaError_t launch(K kernel, unsigned grid, int threads, int cluster, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
cudaError_t logprobs_type(const LogprobArgs& a, cudaStream_t s) {
    const Parts p = parts_of(a.m, a.vocab);
    const int part = (a.vocab + p.splits - 1) / p.splits;
    const unsigned blocks = static_cast<unsigned>(a.m) * p.splits;
    if (p.cluster) {
        if (p.splits == 8) return launch(logprobs_kernel<T, 512, 8>, blocks, 512, 8, s, a, 8, part);
        if (p.splits == 4) return launch(logprobs_kernel<T, 512, 4>, blocks, 512, 4, s, a, 4, part);
        return launch(logprobs_kernel<T, 512, 2>, blocks, 512, 2, s, a, 2, part);
    }
    // Many rows: four warps a block, as what a warp does once for a row then counts less (4096 bf16 rows of 49152: 95 -> 79 us; with a step's loads ahead and one check a step 74); few: the most
    // loads in flight for each.
    const cudaError_t e = blocks >= 152 * 8 ? launch(logprobs_kernel<T, 128, 1>, blocks, 128, 1, s, a, p.splits, part)
                                            : launch(logprobs_kernel<T, 512, 1>, blocks, 512, 1, s, a, p.splits, part);
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch(logprobs_join_kernel<T>, static_cast<unsigned>(a.m), kJoinThreads, 1, s, a, p.splits);
}

}  // namespace

// Of a call of up to m rows: few rows have more parts than many.
size_t logprobs_workspace_bytes(int m, int vocab, int top) {
    size_t parts = 0;
    for (int rows = 1; rows <= std::min(m, kMaxWideRows); ++rows) {
        const Parts p = parts_of(rows, vocab);
        if (p.splits > 1 && !p.cluster) parts = std::max(parts, static_cast<size_t>(rows) * p.splits);
    }
    return parts ? parts * (16 + 8 * static_cast<size_t>(top)) : 16;
}

cudaError_t launch_logprobs(const LogprobArgs& a, int type, cudaStream_t s) {
    if (type == GQ_F32) return logprobs_type<float>(a, s);
    if (type == GQ_F16) return logprobs_type<__half>(a, s);
    return logprobs_type<__nv_bfloat16>(a, s);
}

}  // namespace gq
