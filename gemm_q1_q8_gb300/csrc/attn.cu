// Attention over the paged Q8_0 cache: one warp a query row and head, one pass over the keys with the running
// maximum and sum of the softmax.
#include "layer_ops.cuh"

namespace gq {
GQ_ERROR_ACCESSOR(attn)
namespace {

__device__ __forceinline__ float4 code_values(uint32_t w, float d) {
    auto one = [&](int e) {
        const uint32_t b = (w >> (8 * e)) & 0xffu;
        const float m = static_cast<float>(b & 127u) * d;
        return b & 128u ? -m : m;
    };
    return make_float4(one(0), one(1), one(2), one(3));
}

template <typename T, int HD>
__global__ void __launch_bounds__(128) attn_kernel(const AttnArgs a) {
    constexpr int kRuns = HD == 256 ? 2 : 1;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const int t = warp / a.q_heads, h = warp % a.q_heads;
    const int q0 = a.q_start[b], L = a.kv_len[b];
    const int T_ = a.q_start[b + 1] - q0;
    if (warp == 0 && lane == 0 && (T_ > a.max_q || L > a.max_kv)) report_error(kErrIndex);
    if (t >= T_ || t >= a.max_q) return;
    const int kvh = h / (a.q_heads / a.kv_heads);
    const T* q = static_cast<const T*>(a.q) + (q0 + t) * a.q_stride + h * HD;
    const bool mine = HD != 64 || lane < 16;
    float4 qv[kRuns], o[kRuns];
#pragma unroll
    for (int c = 0; c < kRuns; ++c) {
        qv[c] = mine ? load4(q + c * 128 + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
        o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const unsigned long long mask = a.tree ? a.tree[q0 + t] : 0ull;
    const int Lc = min(L, a.max_kv);
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < Lc; ++j) {
        const int rel = j - (L - T_);
        if (rel >= 0 && (a.tree ? rel >= 64 || !((mask >> rel) & 1) : rel > t)) continue;
        const int page = a.table[static_cast<size_t>(b) * a.table_stride + j / a.page_size];
        if (page < 0 || page >= a.pages) {
            if (lane == 0) report_error(kErrIndex);
            continue;
        }
        const int place = j % a.page_size, tok = j % kvGroup;
        const uint8_t* chunk = a.cache + ((static_cast<size_t>(page) * a.kv_heads + kvh) * (a.page_size / kvGroup) + place / kvGroup) * kv_chunk_bytes(HD);
        float s = 0.f;
        float4 v[kRuns];
#pragma unroll
        for (int c = 0; c < kRuns; ++c) {
            const int d = (mine ? c * 128 + 4 * lane : 0);
            const int sc = kv_scale<HD>(tok, d);
            const float4 k = code_values(*reinterpret_cast<const uint32_t*>(chunk + kv_k_word<HD>(tok, d)),
                                         f16_to_f32(*reinterpret_cast<const uint16_t*>(chunk + kv_ks_offset(HD) + sc)));
            v[c] = code_values(*reinterpret_cast<const uint32_t*>(chunk + kv_v_word<HD>(tok, d)),
                               f16_to_f32(*reinterpret_cast<const uint16_t*>(chunk + kv_vs_offset(HD) + sc)));
            if (mine) s = fmaf(qv[c].x, k.x, fmaf(qv[c].y, k.y, fmaf(qv[c].z, k.z, fmaf(qv[c].w, k.w, s))));
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.scale;
        if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
        const float mn = fmaxf(m, s);
        const float old = m == -INFINITY ? 0.f : expf(m - mn), p = mn == -INFINITY ? 0.f : expf(s - mn);
        l = l * old + p;
        m = mn;
#pragma unroll
        for (int c = 0; c < kRuns; ++c)
            o[c] = make_float4(fmaf(p, v[c].x, o[c].x * old), fmaf(p, v[c].y, o[c].y * old), fmaf(p, v[c].z, o[c].z * old),
                               fmaf(p, v[c].w, o[c].w * old));
    }
    const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
    T* out = static_cast<T*>(a.out) + (q0 + t) * a.out_stride + h * HD;
#pragma unroll
    for (int c = 0; c < kRuns; ++c)
        if (mine) store4(out + c * 128 + 4 * lane, make_float4(o[c].x * inv, o[c].y * inv, o[c].z * inv, o[c].w * inv));
}

template <typename T, int HD>
cudaError_t attn_go(const AttnArgs& a, cudaStream_t s) {
    const long long warps = static_cast<long long>(a.max_q) * a.q_heads;
    attn_kernel<T, HD><<<dim3(static_cast<unsigned>((warps + 3) / 4), a.seqs), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t attn_workspace_bytes(int, int, int, int, int, int) { return 16; }

cudaError_t launch_attn(const AttnArgs& a, int type, int head_dim, cudaStream_t s) {
    if (type == GQ_F32)
        return head_dim == 64 ? attn_go<float, 64>(a, s) : head_dim == 128 ? attn_go<float, 128>(a, s) : attn_go<float, 256>(a, s);
    if (type == GQ_F16)
        return head_dim == 64 ? attn_go<__half, 64>(a, s) : head_dim == 128 ? attn_go<__half, 128>(a, s) : attn_go<__half, 256>(a, s);
    return head_dim == 64    ? attn_go<__nv_bfloat16, 64>(a, s)
           : head_dim == 128 ? attn_go<__nv_bfloat16, 128>(a, s)
                             : attn_go<__nv_bfloat16, 256>(a, s);
}

}  // namespace gq
