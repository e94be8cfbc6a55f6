// What the kernels between a layer's products share: values of three types, the cache's layout, and the
// launch bodies (norm.cu, kv.cu, attn.cu; arguments already validated).
#pragma once

#include <cuda_bf16.h>

#include "gq_internal.cuh"

namespace gq {

// Four consecutive values of a type as f32, and back with one rounding to nearest even.
template <typename T> struct Vec4;
template <> struct Vec4<float> {
    using Raw = float4;
    static __device__ __forceinline__ float4 widen(Raw r) { return r; }
    static __device__ __forceinline__ Raw narrow(float4 v) { return v; }
};
template <> struct Vec4<__half> {
    using Raw = uint2;
    static __device__ __forceinline__ float4 widen(Raw r) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    static __device__ __forceinline__ Raw narrow(float4 v) {
        Raw r;
        *reinterpret_cast<__half2*>(&r.x) = __floats2half2_rn(v.x, v.y);
        *reinterpret_cast<__half2*>(&r.y) = __floats2half2_rn(v.z, v.w);
        return r;
    }
};
template <> struct Vec4<__nv_bfloat16> {
    using Raw = uint2;
    static __device__ __forceinline__ float4 widen(Raw r) {
        return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                           __uint_as_float(r.y & 0xffff0000u));
    }
    static __device__ __forceinline__ Raw narrow(float4 v) {
        Raw r;
        *reinterpret_cast<__nv_bfloat162*>(&r.x) = __floats2bfloat162_rn(v.x, v.y);
        *reinterpret_cast<__nv_bfloat162*>(&r.y) = __floats2bfloat162_rn(v.z, v.w);
        return r;
    }
};
template <typename T> __device__ __forceinline__ float4 load4(const T* p) {
    return Vec4<T>::widen(*reinterpret_cast<const typename Vec4<T>::Raw*>(p));
}
template <typename T> __device__ __forceinline__ void store4(T* p, float4 v) {
    *reinterpret_cast<typename Vec4<T>::Raw*>(p) = Vec4<T>::narrow(v);
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_f32(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// amax / 127 rounded to nearest, as q8_0_scale has it: the product with the rounded reciprocal, corrected by its exact remainder (division by a
// divisor known in advance: Brisebarre, Muller and Raina, IEEE Trans. Computers 53, 2004; equal to the division for each of the 2^23
// mantissas); where a step could leave f32's normal range, the division itself.  It is 3 instructions of every thread: 8192 rows of 4096
// normed 96 -> 93 us, 8192 tokens appended 97 -> 93 us.
__device__ __forceinline__ float q8_0_scale_fast(float amax) {
    if (!(amax >= 0x1p-90f && amax <= 0x1p126f)) return q8_0_scale(amax);
    const float r = 1.0f / 127.0f, q = __fmul_rn(amax, r);
    return __fmaf_rn(__fmaf_rn(-127.0f, q, amax), r, q);
}
// Four values of a block quantized by the rule of q8_0_quant (round half up of the rounded quotient x / d), without its
// divisions: the approximate reciprocal is off by at most 2^-23 of itself, so x times it is within 127 * 2^-23 < 2^-16 of the quotient, whose rounding
// moves it by at most 2^-18: where it is further than 2^-14 from a tie its nearest integer is the code; the few others (and NaN) are divided (of 128
// values that a warp quantizes at once one in 64 times; with 2^-11 one in 8).  16 instructions instead of some 80.
// BYTES: only the codes' low bytes are meant.  q8_0_codes: false where they have to be divided; zero: the block is.
template <bool BYTES>
__device__ __forceinline__ bool q8_0_codes(float4 v, float dd, bool zero, int (&c)[4]) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(dd));
    if (!(dd >= 0x1p-120f)) r = 0.0f;
    const float2 magic = make_float2(12582912.0f, 12582912.0f);         // 1.5 * 2^23: the sum's low bits are the integer
    const float2 rr = make_float2(r, r), minus = make_float2(-1.0f, -1.0f);
    bool far = dd >= 0x1p-120f || zero;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float2 x = i ? make_float2(v.z, v.w) : make_float2(v.x, v.y), t = ffma2(x, rr, magic);
        const float2 rest = ffma2(x, rr, ffma2(t, minus, magic));
        c[i] = __float_as_int(t.x) - (BYTES ? 0 : __float_as_int(magic.x));
        c[i + 1] = __float_as_int(t.y) - (BYTES ? 0 : __float_as_int(magic.x));
        far = far && fabsf(rest.x) <= 0.5f - 0x1p-14f && fabsf(rest.y) <= 0.5f - 0x1p-14f;
    }
    return far;
}
template <bool BYTES>
__device__ __forceinline__ void q8_0_quant4(float4 v, float amax, float dd, int (&c)[4]) {
    if (q8_0_codes<BYTES>(v, dd, amax == 0.0f, c)) return;
    c[0] = q8_0_quant(v.x, amax, dd);
    c[1] = q8_0_quant(v.y, amax, dd);
    c[2] = q8_0_quant(v.z, amax, dd);
    c[3] = q8_0_quant(v.w, amax, dd);
}

// Four blocks' codes (low bytes), eight lanes a block, each lane with four values y[c] of block c and their largest magnitude m[c]: the maxima (by `most`) meet in
// halves, quarters and eighths of the lanes, so that two lanes have each scale, which the others get from them: 4 + 4 shuffles and one scale
// instead of 12 and four, and four chains beside one another.  Returns the scale of block (lane % 8) / 2.
template <typename F>
__device__ __forceinline__ float q8_0_four(const float4 (&y)[4], const float (&m)[4], F most, int (&cd)[4][4]) {
    const int lane = threadIdx.x & 31;
    const bool upper = lane & 4, odd = lane & 2;
    const float m0 = most(upper ? m[2] : m[0], __shfl_xor_sync(0xffffffffu, upper ? m[0] : m[2], 4));
    const float m1 = most(upper ? m[3] : m[1], __shfl_xor_sync(0xffffffffu, upper ? m[1] : m[3], 4));
    float amax = most(odd ? m1 : m0, __shfl_xor_sync(0xffffffffu, odd ? m0 : m1, 2));
    amax = most(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const float dd = q8_0_scale_fast(amax), sent = amax == 0.0f ? -0.0f : dd;       // blocks of zeros apart from those whose scale is below f32's range
    float d[4];
    bool far[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) d[c] = __shfl_sync(0xffffffffu, sent, (lane & 24) | 2 * c);
#pragma unroll
    for (int c = 0; c < 4; ++c) far[c] = q8_0_codes<true>(y[c], d[c], __float_as_uint(d[c]) == 0x80000000u, cd[c]);
    if (!(far[0] && far[1] && far[2] && far[3]))
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (!far[c]) {
                cd[c][0] = q8_0_quant(y[c].x, 1.0f, d[c]);
                cd[c][1] = q8_0_quant(y[c].y, 1.0f, d[c]);
                cd[c][2] = q8_0_quant(y[c].z, 1.0f, d[c]);
                cd[c][3] = q8_0_quant(y[c].w, 1.0f, d[c]);
            }
    return dd;
}

// Codes in the cache: sign bit and magnitude; four of them as a word, and a word's values times d
__device__ __forceinline__ uint32_t cache_word(const int (&c)[4]) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= static_cast<uint32_t>(c[i] < 0 ? 128 - c[i] : c[i]) << (8 * i);
    return w;
}
__device__ __forceinline__ float4 cache_values(uint32_t w, uint32_t d16) {
    const float d = f16_to_f32(d16) * 16777216.0f;                      // a code's bits as f16 are code * 2^-24
    const uint32_t lo = __byte_perm(w, 0, 0x1100) & 0x807f807fu, hi = __byte_perm(w, 0, 0x3322) & 0x807f807fu;
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo)), b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return make_float4(a.x * d, a.y * d, b.x * d, b.y * d);
}

// ---------------------------------------------------------------- the cache (layout: include/gq.h)
constexpr int kvGroup = 16;                                             // tokens of a chunk
__host__ __device__ constexpr int kv_chunk_bytes(int hd) { return 34 * hd; }
__host__ __device__ constexpr int kv_v_offset(int hd) { return 16 * hd; }
__host__ __device__ constexpr int kv_ks_offset(int hd) { return 32 * hd; }
__host__ __device__ constexpr int kv_vs_offset(int hd) { return 33 * hd; }

// Byte offsets in a chunk of the four codes d .. d + 3 (d a multiple of 4) of token `tok`, and of its scale.
template <int HD> __device__ __forceinline__ int kv_k_word(int tok, int d) {
    int u = 4 * (d >> 6) + ((d >> 2) & 3);
    if (HD > 64) u ^= 4 * (tok & 1);
    return tok * HD + u * 16 + ((d >> 4) & 3) * 4;
}
template <int HD> __device__ __forceinline__ int kv_v_word(int tok, int d) {
    const int t = (tok & 7) >> 1, p = (tok & 1) + 2 * (tok >> 3), g = (d >> 2) & 7;
    if (HD == 64) return kv_v_offset(HD) + (4 * p + t) * 64 + 8 * (g ^ (4 * (t >> 1))) + 4 * (d >> 5);
    return kv_v_offset(HD) + (4 * p + t) * HD + 128 * (d >> 7) + 16 * (g ^ (2 * t)) + 4 * ((d >> 5) & 3);
}
template <int HD> __device__ __forceinline__ int kv_scale(int tok, int d) {
    const int t = (tok & 7) >> 1, p = (tok & 1) + 2 * (tok >> 3);
    return 2 * ((4 * t + p) * (HD / 32) + (d >> 5));
}

cudaError_t launch_rmsnorm(const void* x, long long xs, const void* r, long long rs, const float* w, float eps, int type,
                           int m, int k, void* h, void* y, void* act, uint16_t* d, int8_t* q, uint16_t* op,
                           cudaStream_t s);
cudaError_t launch_block_norm(const void* block, long long bs, const void* x, long long xs, const float* post, const void* gate, long long gs,
                              float block_scale, float residual_scale, const float* w, float eps, int type, int m, int k, void* h,
                              void* y, void* act, uint16_t* d, int8_t* q, uint16_t* op, cudaStream_t s);
struct LogprobArgs {
    const void* x;
    long long stride;
    int m, vocab, top;
    float scale;
    const int64_t* tokens;
    float* logprob; float* entropy; float* top_values;
    int64_t* top_ids;
    void* workspace;
};
size_t logprobs_workspace_bytes(int m, int vocab, int top);
cudaError_t launch_logprobs(const LogprobArgs& a, int type, cudaStream_t s);
cudaError_t launch_dequantize_q8_0(const void* act, long long blocks, int type, void* out, cudaStream_t s);
cudaError_t launch_rope_table(float* table, int positions, int rot, double base, int scaling, double factor,
                              double original, cudaStream_t s);

struct AppendArgs {
    const void* q; void* q_out; const void* k; const void* v;
    long long q_stride, q_out_stride, k_stride, v_stride;
    const float* rope;
    int rope_rows, rot, interleaved;
    const int32_t* positions;
    const int64_t* slots;
    int tokens, q_heads, kv_heads;
    uint8_t* cache;
    int pages, page_size;
};
cudaError_t launch_kv_append(const AppendArgs& a, int type, int head_dim, cudaStream_t s);
cudaError_t launch_kv_read(const uint8_t* cache, int pages, int page_size, int kv_heads, int head_dim,
                           const int64_t* slots, int n, int type, void* k_out, void* v_out, cudaStream_t s);

struct AttnArgs {
    const void* q; void* out;
    long long q_stride, out_stride;
    const uint8_t* cache;
    int pages, page_size;
    const int32_t* table;
    int table_stride;
    const int32_t* kv_len;
    const int32_t* q_start;
    const uint64_t* tree;
    int rows;              // of q and out; negative: q_start[seqs]
    int seqs, max_q, max_kv, q_heads, kv_heads;
    float scale, softcap;
    void* workspace;
};
size_t attn_workspace_bytes(int seqs, int max_q, int q_heads, int kv_heads, int head_dim, int type);
cudaError_t launch_attn(const AttnArgs& a, int type, int head_dim, cudaStream_t s);
size_t attn_tiles_workspace_bytes(int head_dim, int type);
cudaError_t launch_attn_tiles(const AttnArgs& a, int type, int head_dim, cudaStream_t s);   // head_dim 64 or 128

}  // namespace gq
