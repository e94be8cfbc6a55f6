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

__device__ __forceinline__ uint32_t sign_magnitude(int c) { return c < 0 ? static_cast<uint32_t>(128 - c) : static_cast<uint32_t>(c); }

// Four dims of a row, turned: v their values, row the head's row.
template <typename T>
__device__ __forceinline__ float4 turned(const AppendArgs& a, const T* row, int d, float4 v, const float2* cs) {
    if (d >= a.rot) return v;
    if (a.interleaved) {
        const float4 z = *reinterpret_cast<const float4*>(cs + d / 2);
        return make_float4(v.x * z.x - v.y * z.y, v.y * z.x + v.x * z.y, v.z * z.z - v.w * z.w, v.w * z.z + v.z * z.w);
    }
    const int half = a.rot / 2;
    const bool first = d < half;
    const float4 o = load4(row + (first ? d + half : d - half));
    const float2* at = cs + (first ? d : d - half);
    const float4 z0 = *reinterpret_cast<const float4*>(at), z1 = *reinterpret_cast<const float4*>(at + 2);
    if (first)
        return make_float4(v.x * z0.x - o.x * z0.y, v.y * z0.z - o.y * z0.w, v.z * z1.x - o.z * z1.y,
                           v.w * z1.z - o.w * z1.w);
    return make_float4(v.x * z0.x + o.x * z0.y, v.y * z0.z + o.y * z0.w, v.z * z1.x + o.z * z1.y, v.w * z1.z + o.w * z1.w);
}

// A warp takes 32 * 4 / HD rows (HD = 64: two; 128 and 256: one); the rows of a token are its q heads, k heads, v heads.
template <typename T, int HD>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a) {
    constexpr int kLanes = HD == 64 ? 16 : 32, kRuns = HD == 256 ? 2 : 1;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int rows = a.q_heads + 2 * a.kv_heads;
    const long long idx = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / kLanes;
    const int l = threadIdx.x % kLanes;
    const bool in = idx < static_cast<long long>(a.tokens) * rows;
    const int n = in ? static_cast<int>(idx / rows) : 0;
    int h = in ? static_cast<int>(idx % rows) : 0;
    const int kind = h < a.q_heads ? 0 : h < a.q_heads + a.kv_heads ? 1 : 2;
    if (kind == 1) h -= a.q_heads;
    if (kind == 2) h -= a.q_heads + a.kv_heads;
    const T* row = kind == 0   ? static_cast<const T*>(a.q) + n * a.q_stride
                   : kind == 1 ? static_cast<const T*>(a.k) + n * a.k_stride
                               : static_cast<const T*>(a.v) + n * a.v_stride;
    row += h * HD;
    bool ok = in;
    const float2* cs = nullptr;
    if (a.rot) {
        const int pos = a.positions[n];
        if (pos < 0 || pos >= a.rope_rows) {
            if (in && l == 0 && h == 0) report_error(kErrIndex);
            ok = false;
        } else {
            cs = reinterpret_cast<const float2*>(a.rope) + static_cast<size_t>(pos) * (a.rot / 2);
        }
    }
    float4 v[kRuns];
#pragma unroll
    for (int c = 0; c < kRuns; ++c) {
        const int d = c * 128 + 4 * l;
        v[c] = load4(row + d);
        if (kind != 2 && cs) v[c] = turned(a, row, d, v[c], cs);
    }
    __syncwarp();                                     // q_out may be q: every read of the row is before its writes
    if (kind == 0 && ok) {
        T* out = static_cast<T*>(a.q_out) + n * a.q_out_stride + h * HD;
#pragma unroll
        for (int c = 0; c < kRuns; ++c) store4(out + c * 128 + 4 * l, v[c]);
    }
    long long slot = -1;
    if (kind != 0 && ok) {
        slot = a.slots[n];
        if (slot >= static_cast<long long>(a.pages) * a.page_size) {
            if (l == 0) report_error(kErrIndex);
            slot = -1;
        }
    }
    const int tok = static_cast<int>(slot & (kvGroup - 1));
    const long long page = slot / a.page_size;
    const int place = static_cast<int>(slot - page * a.page_size);
    uint8_t* chunk = a.cache + ((page * a.kv_heads + h) * (a.page_size / kvGroup) + place / kvGroup) * kv_chunk_bytes(HD);
#pragma unroll
    for (int c = 0; c < kRuns; ++c) {
        const int d = c * 128 + 4 * l;
        float amax = fmaxf(fmaxf(fabsf(v[c].x), fabsf(v[c].y)), fmaxf(fabsf(v[c].z), fabsf(v[c].w)));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (slot < 0) continue;                       // after the shuffles: the warp's rows may differ
        const float dd = q8_0_scale(amax);
        const uint32_t word = sign_magnitude(q8_0_quant(v[c].x, amax, dd)) | sign_magnitude(q8_0_quant(v[c].y, amax, dd)) << 8 |
                              sign_magnitude(q8_0_quant(v[c].z, amax, dd)) << 16 | sign_magnitude(q8_0_quant(v[c].w, amax, dd)) << 24;
        *reinterpret_cast<uint32_t*>(chunk + (kind == 1 ? kv_k_word<HD>(tok, d) : kv_v_word<HD>(tok, d))) = word;
        if ((l & 7) == 0)
            *reinterpret_cast<uint16_t*>(chunk + (kind == 1 ? kv_ks_offset(HD) : kv_vs_offset(HD)) + kv_scale<HD>(tok, d)) =
                __half_as_ushort(__float2half_rn(dd));
    }
}

__device__ __forceinline__ float4 code_values(uint32_t w, float d) {
    auto one = [&](int e) {
        const uint32_t b = (w >> (8 * e)) & 0xffu;
        const float m = static_cast<float>(b & 127u) * d;
        return b & 128u ? -m : m;
    };
    return make_float4(one(0), one(1), one(2), one(3));
}

// As the append: four dims a thread, rows of slots and kv heads; K and V of a row by the same thread.
template <typename T, int HD>
__global__ void __launch_bounds__(256)
kv_read_kernel(const uint8_t* __restrict__ cache, long long slots_all, int page_size, int kv_heads,
               const int64_t* __restrict__ slots, int n, T* __restrict__ k_out, T* __restrict__ v_out) {
    constexpr int kWords = HD / 4;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const long long row = i / kWords;
    if (row >= static_cast<long long>(n) * kv_heads) return;
    const int d = 4 * static_cast<int>(i % kWords);
    const int h = static_cast<int>(row % kv_heads);
    const long long slot = slots[row / kv_heads];
    float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
    if (slot >= slots_all) {
        if (d == 0 && h == 0) report_error(kErrIndex);
    } else if (slot >= 0) {
        const int tok = static_cast<int>(slot & (kvGroup - 1));
        const long long page = slot / page_size;
        const int place = static_cast<int>(slot - page * page_size);
        const uint8_t* chunk = cache + ((page * kv_heads + h) * (page_size / kvGroup) + place / kvGroup) * kv_chunk_bytes(HD);
        const int sc = kv_scale<HD>(tok, d);
        if (k_out)
            kv = code_values(*reinterpret_cast<const uint32_t*>(chunk + kv_k_word<HD>(tok, d)),
                             f16_to_f32(*reinterpret_cast<const uint16_t*>(chunk + kv_ks_offset(HD) + sc)));
        if (v_out)
            vv = code_values(*reinterpret_cast<const uint32_t*>(chunk + kv_v_word<HD>(tok, d)),
                             f16_to_f32(*reinterpret_cast<const uint16_t*>(chunk + kv_vs_offset(HD) + sc)));
    }
    if (k_out) store4(k_out + row * HD + d, kv);
    if (v_out) store4(v_out + row * HD + d, vv);
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
    const long long rows = static_cast<long long>(a.tokens) * (a.q_heads + 2 * a.kv_heads);
    const int per = 256 / (HD == 64 ? 16 : 32);
    return launch_dependent(kv_append_kernel<T, HD>, (rows + per - 1) / per, 256, s, a);
}
template <typename T, int HD>
cudaError_t read_go(const uint8_t* cache, int pages, int page_size, int kv_heads, const int64_t* slots, int n, void* k,
                    void* v, cudaStream_t s) {
    const long long threads = static_cast<long long>(n) * kv_heads * (HD / 4);
    return launch_dependent(kv_read_kernel<T, HD>, (threads + 255) / 256, 256, s, cache,
                            static_cast<long long>(pages) * page_size, page_size, kv_heads, slots, n, static_cast<T*>(k),
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
