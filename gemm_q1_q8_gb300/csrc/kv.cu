// Rotary positions, the append to the paged Q8_0 cache, and reading it back.
//
// A head's row is hd values: a thread takes four consecutive dims (hd = 256: two such runs, 128 apart), so
// the eight threads of a 32-block find its scale by three shuffles, its codes make one 32-bit word a
// thread, and a row's words fill one contiguous run of the cache's chunk.  A pair's other half is read by
// its thread too (from L1), so no exchange between threads depends on the layout of the pairs.
// Each value is read once from HBM and written once: bound by HBM for many tokens, by latency for one.
#include "layer_ops.cuh"

namespace gq {
GQ_ERROR_ACCESSOR(kv)
namespace {

__global__ void rope_table_kernel(float2* __restrict__ table, int positions, int half, double base, int scaling,
                                  double factor, double original) {
    const long long n = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (n >= static_cast<long long>(positions) * half) return;
    const int i = static_cast<int>(n % half);
    const double rot = 2.0 * half;
    double b = base, size = 1.0;
    if (scaling == GQ_ROPE_NTK) b = base * pow(factor, rot / (rot - 2.0));
    double f = pow(b, -2.0 * i / rot);
    if (scaling == GQ_ROPE_LINEAR) f /= factor;
    if (scaling == GQ_ROPE_YARN) {
        const double two_pi = 6.283185307179586476925286766559;
        double low = floor(rot * log(original / (32.0 * two_pi)) / (2.0 * log(base)));
        double high = ceil(rot * log(original / two_pi) / (2.0 * log(base)));
        low = fmin(fmax(low, 0.0), rot - 1.0);
        high = fmin(fmax(high, 0.0), rot - 1.0);
        if (low == high) high += 0.001;
        const double r = 1.0 - fmin(fmax((i - low) / (high - low), 0.0), 1.0);
        f *= r + (1.0 - r) / factor;
        size = 1.0 + 0.1 * log(factor);
    }
    double s, c;
    sincos(static_cast<double>(n / half) * f, &s, &c);
    table[n] = make_float2(static_cast<float>(c * size), static_cast<float>(s * size));
}

// A token's angles for this thread's four dims: (cos, sin) of each of its pairs (half), or of its two (interleaved)
struct Turn {
    float4 z0, z1;
    int other;             // half: distance to the pairs' other dims (0: these dims are not turned)
    float sign;
    bool on;
};
// MODE 1: half, o the pairs' other dims; 2: interleaved
template <int MODE>
__device__ __forceinline__ float4 turned(const Turn& t, float4 v, float4 o) {
    if (MODE == 2)
        return make_float4(v.x * t.z0.x - v.y * t.z0.y, v.y * t.z0.x + v.x * t.z0.y, v.z * t.z0.z - v.w * t.z0.w, v.w * t.z0.z + v.z * t.z0.w);
    // first half: a cos - b sin; second: b cos + a sin, the sign in front of an exact product
    return make_float4(v.x * t.z0.x + t.sign * (o.x * t.z0.y), v.y * t.z0.z + t.sign * (o.y * t.z0.w), v.z * t.z1.x + t.sign * (o.z * t.z1.y),
                       v.w * t.z1.z + t.sign * (o.w * t.z1.w));
}

// A slot's page and its 16-token group there, in 32 bits where they allow
__device__ __forceinline__ void page_group(long long slot, int groups, long long& page, int& group) {
    const long long g = slot / kvGroup;
    if (g < 0x7fffffffll) {
        page = static_cast<int>(g) / groups;
        group = static_cast<int>(g) - static_cast<int>(page) * groups;
    } else {
        page = g / groups;
        group = static_cast<int>(g - page * groups);
    }
}

// The rows of a token are its q heads, k heads, v heads.  A warp takes rows part * per .. of one token (HD = 64: two at a time), so that
// a token's position, slot and angles are looked up once for all of them.
// Every load of a step is issued before any branch on what its rows are, the first step's before the token's position and slot are known.
// Bound by HBM for many tokens (8192 of 32 + 2 x 8 heads of 128 in f32, with the read of what was written: 80 us, 76% of the measured rate; with the
// loads in branches 110 us, behind the look-ups 93 us), by the chain of loads for few.
template <typename T, int HD, int MODE>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a, int parts, int per) {
    constexpr int kLanes = HD == 64 ? 16 : 32, kRuns = HD == 256 ? 2 : 1, kAt = 32 / kLanes, kU = 4 / kRuns;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int rows = a.q_heads + 2 * a.kv_heads;
    const int warp = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int n = warp / parts, from = (warp % parts) * per, to = min(from + per, rows);
    if (n >= a.tokens) return;
    const int l = threadIdx.x % kLanes, half_warp = (threadIdx.x & 31) / kLanes;
    long long slot = a.slots[n];
    const int pos = MODE ? a.positions[n] : 0;
    Turn turn[kRuns];
#pragma unroll
    for (int c = 0; c < kRuns; ++c) {
        const int d = c * 128 + 4 * l, half = a.rot / 2;
        turn[c].on = MODE && d < a.rot;
        turn[c].other = MODE == 1 && turn[c].on ? (d < half ? half : -half) : 0;
        turn[c].sign = d < half ? -1.0f : 1.0f;
    }
    float4 v[kU][kRuns], o[kU][kRuns];
    auto load = [&](int r0) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int r = min(r0 + u * kAt + half_warp, to - 1);          // past the end: the last row again, which nothing is done with
            const bool is_q = r < a.q_heads, is_k = r < a.q_heads + a.kv_heads;
            const T* p = static_cast<const T*>(is_q ? a.q : is_k ? a.k : a.v) + n * (is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride) +
                         (r - (is_q ? 0 : is_k ? a.q_heads : a.q_heads + a.kv_heads)) * HD;
#pragma unroll
            for (int c = 0; c < kRuns; ++c) {
                v[u][c] = load4(p + c * 128 + 4 * l);
                if (MODE == 1) o[u][c] = load4(p + c * 128 + 4 * l + turn[c].other);
            }
        }
    };
    load(from);                                           // before what the token's position and slot lead to
    if (MODE) {
        if (pos < 0 || pos >= a.rope_rows) {
            if (l == 0) report_error(kErrIndex);
            return;                                       // the token is left out
        }
        const float2* cs = reinterpret_cast<const float2*>(a.rope) + static_cast<size_t>(pos) * (a.rot / 2);
#pragma unroll
        for (int c = 0; c < kRuns; ++c) {
            const int d = c * 128 + 4 * l, half = a.rot / 2;
            if (!turn[c].on) continue;
            if (MODE == 2) {
                turn[c].z0 = *reinterpret_cast<const float4*>(cs + d / 2);
            } else {
                const float2* at = cs + (d < half ? d : d - half);
                turn[c].z0 = *reinterpret_cast<const float4*>(at);
                turn[c].z1 = *reinterpret_cast<const float4*>(at + 2);
            }
        }
    }
    if (slot >= static_cast<long long>(a.pages) * a.page_size) {
        if (l == 0) report_error(kErrIndex);
        slot = -1;
    }
    const int tok = static_cast<int>(slot & (kvGroup - 1)), groups = a.page_size / kvGroup;
    long long page;
    int group;
    page_group(slot < 0 ? 0 : slot, groups, page, group);
    uint8_t* chunk0 = a.cache + (page * a.kv_heads * groups + group) * kv_chunk_bytes(HD);

    for (int r0 = from; r0 < to; r0 += kAt * kU) {
        if (r0 > from) load(r0);
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int c = 0; c < kRuns; ++c)
                if (MODE) {
                    const float4 x = turned<MODE>(turn[c], v[u][c], o[u][c]);
                    const bool on = turn[c].on && r0 + u * kAt + half_warp < a.q_heads + a.kv_heads;
                    v[u][c] = make_float4(on ? x.x : v[u][c].x, on ? x.y : v[u][c].y, on ? x.z : v[u][c].z, on ? x.w : v[u][c].w);
                }
        __syncwarp();                                     // q_out may be q: every read of a row is before its writes
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int r = r0 + u * kAt + half_warp;
            if (r < min(to, a.q_heads)) {
                T* out = static_cast<T*>(a.q_out) + n * a.q_out_stride + r * HD;
#pragma unroll
                for (int c = 0; c < kRuns; ++c) store4(out + c * 128 + 4 * l, v[u][c]);
            }
            if (r0 + (u + 1) * kAt <= a.q_heads) continue;               // all of the warp's rows are queries
            const bool on = r >= a.q_heads && r < to && slot >= 0, is_k = r < a.q_heads + a.kv_heads;
            const int h = is_k ? r - a.q_heads : r - a.q_heads - a.kv_heads;
            uint8_t* chunk = chunk0 + static_cast<long long>(h) * groups * kv_chunk_bytes(HD);
#pragma unroll
            for (int c = 0; c < kRuns; ++c) {
                const int d = c * 128 + 4 * l;
                const float4 x = v[u][c];
                float amax = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                if (!on) continue;
                const float dd = q8_0_scale_fast(amax);
                int code[4];
                q8_0_quant4<false>(x, amax, dd, code);
                *reinterpret_cast<uint32_t*>(chunk + (is_k ? kv_k_word<HD>(tok, d) : kv_v_word<HD>(tok, d))) = cache_word(code);
                if ((l & 7) == 0)
                    *reinterpret_cast<uint16_t*>(chunk + (is_k ? kv_ks_offset(HD) : kv_vs_offset(HD)) + kv_scale<HD>(tok, d)) =
                        __half_as_ushort(__float2half_rn(dd));
            }
        }
    }
}

// A warp takes `per` heads of one slot (HD = 64: two at a time): a thread four dims of K and of V.
template <typename T, int HD>
__global__ void __launch_bounds__(256)
kv_read_kernel(const uint8_t* cache, long long slots_all, int page_size, int kv_heads, const int64_t* slots, int n, int parts, int per, T* k_out,
               T* v_out) {
    constexpr int kLanes = HD == 64 ? 16 : 32, kRuns = HD == 256 ? 2 : 1, kAt = 32 / kLanes, kU = 4 / kRuns;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int i = warp / parts, from = (warp % parts) * per, to = min(from + per, kv_heads);
    if (i >= n) return;
    const int l = threadIdx.x % kLanes, half_warp = (threadIdx.x & 31) / kLanes;
    long long slot = slots[i];
    if (slot >= slots_all) {
        if (l == 0) report_error(kErrIndex);
        slot = -1;
    }
    const int tok = static_cast<int>(slot & (kvGroup - 1)), groups = page_size / kvGroup;
    long long page;
    int group;
    page_group(slot < 0 ? 0 : slot, groups, page, group);
    const uint8_t* chunk0 = cache + (page * kv_heads * groups + group) * kv_chunk_bytes(HD);
    const size_t out0 = static_cast<size_t>(i) * kv_heads * HD;
    for (int h0 = from; h0 < to; h0 += kAt * kU) {
        uint32_t kw[kU][kRuns], vw[kU][kRuns], ks[kU][kRuns], vs[kU][kRuns];
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int c = 0; c < kRuns; ++c) {
                const int h = h0 + u * kAt + half_warp, d = c * 128 + 4 * l;
                kw[u][c] = vw[u][c] = ks[u][c] = vs[u][c] = 0;
                if (h >= to || slot < 0) continue;
                const uint8_t* chunk = chunk0 + static_cast<long long>(h) * groups * kv_chunk_bytes(HD);
                const int sc = kv_scale<HD>(tok, d);
                if (k_out) {
                    kw[u][c] = *reinterpret_cast<const uint32_t*>(chunk + kv_k_word<HD>(tok, d));
                    ks[u][c] = *reinterpret_cast<const uint16_t*>(chunk + kv_ks_offset(HD) + sc);
                }
                if (v_out) {
                    vw[u][c] = *reinterpret_cast<const uint32_t*>(chunk + kv_v_word<HD>(tok, d));
                    vs[u][c] = *reinterpret_cast<const uint16_t*>(chunk + kv_vs_offset(HD) + sc);
                }
            }
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int c = 0; c < kRuns; ++c) {
                const int h = h0 + u * kAt + half_warp, d = c * 128 + 4 * l;
                if (h >= to) continue;
                if (k_out) store4(k_out + out0 + h * HD + d, cache_values(kw[u][c], ks[u][c]));
                if (v_out) store4(v_out + out0 + h * HD + d, cache_values(vw[u][c], vs[u][c]));
            }
    }
}

// Rows of a token that a warp takes: all of them where the tokens fill the GPU (152 SMs, some 64 warps each), fewer for few tokens.  Below the
// `full` rows that it requests at once only while half as many warps are missing (2219 tokens of 25 heads of 64: 11.5 -> 10.6 us with the read)
int rows_per_warp(long long tokens, int rows, int step, int full) {
    int per = (rows + step - 1) / step * step;
    while (per > step && tokens * ((rows + per - 1) / per) < 152 * (per > full ? 64 : 32)) per = (per / 2 + step - 1) / step * step;
    return per;
}

template <typename K, typename... A>
cudaError_t launch_dependent(K kernel, long long blocks, int threads, cudaStream_t s, A... args) {
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int HD>
cudaError_t append_go(const AppendArgs& a, cudaStream_t s) {
    const int rows = a.q_heads + 2 * a.kv_heads, per = rows_per_warp(a.tokens, rows, HD == 64 ? 2 : 1, HD == 64 ? 8 : HD == 128 ? 4 : 2), parts = (rows + per - 1) / per;
    const long long blocks = (static_cast<long long>(a.tokens) * parts + 7) / 8;
    if (a.rot == 0) return launch_dependent(kv_append_kernel<T, HD, 0>, blocks, 256, s, a, parts, per);
    return a.interleaved ? launch_dependent(kv_append_kernel<T, HD, 2>, blocks, 256, s, a, parts, per)
                         : launch_dependent(kv_append_kernel<T, HD, 1>, blocks, 256, s, a, parts, per);
}
template <typename T, int HD>
cudaError_t read_go(const uint8_t* cache, int pages, int page_size, int kv_heads, const int64_t* slots, int n, void* k,
                    void* v, cudaStream_t s) {
    const int per = rows_per_warp(n, kv_heads, HD == 64 ? 2 : 1, HD == 64 ? 8 : HD == 128 ? 4 : 2), parts = (kv_heads + per - 1) / per;
    return launch_dependent(kv_read_kernel<T, HD>, (static_cast<long long>(n) * parts + 7) / 8, 256, s, cache,
                            static_cast<long long>(pages) * page_size, page_size, kv_heads, slots, n, parts, per, static_cast<T*>(k),
                            static_cast<T*>(v));
}

}  // namespace

cudaError_t launch_rope_table(float* table, int positions, int rot, double base, int scaling, double factor,
                              double original, cudaStream_t s) {
    const long long n = static_cast<long long>(positions) * (rot / 2);
    rope_table_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(reinterpret_cast<float2*>(table), positions,
                                                                             rot / 2, base, scaling, factor, original);
    return cudaGetLastError();
}

#define GQ_BY_TYPE_AND_WIDTH(F, ...)                                                                      \
    (type == GQ_F32    ? (head_dim == 64    ? F<float, 64>(__VA_ARGS__)                                   \
                          : head_dim == 128 ? F<float, 128>(__VA_ARGS__)                                  \
                                            : F<float, 256>(__VA_ARGS__))                                 \
     : type == GQ_F16  ? (head_dim == 64    ? F<__half, 64>(__VA_ARGS__)                                  \
                          : head_dim == 128 ? F<__half, 128>(__VA_ARGS__)                                 \
                                            : F<__half, 256>(__VA_ARGS__))                                \
                       : (head_dim == 64    ? F<__nv_bfloat16, 64>(__VA_ARGS__)                           \
                          : head_dim == 128 ? F<__nv_bfloat16, 128>(__VA_ARGS__)                          \
                                            : F<__nv_bfloat16, 256>(__VA_ARGS__)))

cudaError_t launch_kv_append(const AppendArgs& a, int type, int head_dim, cudaStream_t s) {
    return GQ_BY_TYPE_AND_WIDTH(append_go, a, s);
}

cudaError_t launch_kv_read(const uint8_t* cache, int pages, int page_size, int kv_heads, int head_dim,
                           const int64_t* slots, int n, int type, void* k_out, void* v_out, cudaStream_t s) {
    return GQ_BY_TYPE_AND_WIDTH(read_go, cache, pages, page_size, kv_heads, slots, n, k_out, v_out, s);
}

}  // namespace gq
