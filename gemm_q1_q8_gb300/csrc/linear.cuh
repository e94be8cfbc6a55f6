// Q1_0 products with an epilogue: what the kernel for few tokens (linear.cu) and the one for many (linear_tiles.cu) share.
//
//   z[c, r] = sum_b d0[r, b] * sum_k d1[c, 4b + k] * sum_t (+-1) q   (+ bias[r])
//   linear:  y = act(z) (+ residual[c, r]);      pair: y = act(z_gate) * z_up
//
// Both kernels take +-d0 as f16 matrix operands, made from the sign bits by two logic operations a pair.  The one for few tokens takes the codes
// as they are and multiplies the sums of 32 by d1.  The one for many takes pv = d1 * q * 2^-e, e one power of two a token: pv has at
// most 18 significant bits, so two f16 parts hold it exactly while it is not below 2^-20 of 128 times the token's largest scale (then it is off
// by at most 2^-39 of that).  f32, f16 and Q8_0 results take both parts; a bf16 result (8 bits) takes one, off by 2^-12 of each value.
// Products are exact in f32, sums are f32; the tensor cores truncate the sum that they add to, so it goes to registers every 128 of n.
#pragma once

#include <algorithm>

#include "layer_ops.cuh"

namespace gq {

struct LinearArgs {
    const uint8_t* w[2];               // packed Q1_0; the pair: gate, up
    const uint8_t* act;                // Q8_0 blocks
    const float* bias[2];
    int rows, n, cols;
    int function;                      // gq_function
    int type;
    const void* residual;
    long long residual_stride;
    void* y;
    long long y_stride;
    uint8_t* blocks;                   // Q8_0 output
    void* workspace;
    bool vec;                          // y and residual allow four values at once
};

cudaError_t launch_linear(const LinearArgs& a, bool pair, cudaStream_t s);
size_t linear_workspace_bytes(int rows, int n, int cols);
int linear_plan(int rows, int n, int cols, int parts, bool pair);
int linear_tiles_plan(int rows, int n, int cols, int parts, bool pair);
cudaError_t launch_linear_tiles(const LinearArgs& a, bool pair, cudaStream_t s);
size_t linear_tiles_workspace_bytes(int rows, int n, int cols, bool pair);
float linear_tiles_us(int rows, int n, int cols, int parts, bool pair);

namespace {

// f16 parts that an activation takes
__host__ __device__ __forceinline__ int linear_parts(const LinearArgs& a) { return a.type == GQ_BF16 && !a.blocks ? 1 : 2; }

// 1 / (1 + e^-v); the exponential of 2^-v log2(e) and the reciprocal are off by two units each, and give 0 below 2^-126.  The exponent's product is rounded once and its
// factor by a quarter of a unit, so e^-v is off by |v| 2^-23 of itself too: at -20, where the result is 2e-9, by 2e-6 of it (outputs of
// 16 or 8 bits keep none of that, and a second term of the product would cost every value three instructions).
__device__ __forceinline__ float sigmoid_of(float v) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
__device__ __forceinline__ float bend(float z, int function) {
    switch (function) {
        case GQ_FN_RELU: return z < 0.f ? 0.f : z;                               // NaN stays
        case GQ_FN_RELU2: z = z < 0.f ? 0.f : z; return z * z;
        case GQ_FN_SILU: return z * sigmoid_of(z);
        case GQ_FN_GELU: return 0.5f * z * erfcf(z * -0.70710678f);              // no cancellation below zero
        case GQ_FN_GELU_TANH: return z * sigmoid_of(1.5957691f * fmaf(0.044715f * z * z, z, z));
        default: return z;
    }
}

// The same of several values: one branch, and their chains beside one another
template <int N>
__device__ __forceinline__ void bend_all(float (&z)[N], int function) {
    switch (function) {
#define GQ_BEND(f) case f: _Pragma("unroll") for (int i = 0; i < N; ++i) z[i] = bend(z[i], f); break
        GQ_BEND(GQ_FN_RELU);
        GQ_BEND(GQ_FN_RELU2);
        GQ_BEND(GQ_FN_SILU);
        GQ_BEND(GQ_FN_GELU);
        GQ_BEND(GQ_FN_GELU_TANH);
#undef GQ_BEND
        default: break;
    }
}

__device__ __forceinline__ float load_typed(const void* p, size_t i, int type) {
    if (type == GQ_F32) return static_cast<const float*>(p)[i];
    if (type == GQ_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_typed(void* p, size_t i, int type, float v) {
    if (type == GQ_F32) static_cast<float*>(p)[i] = v;
    else if (type == GQ_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// The epilogue of four neighbouring rows (`row` the first) of a token: eight neighbouring lanes hold a 32-row block, and all of a warp take
// part.  `other`: the pair's second factor, or what is added.
__device__ __forceinline__ void load_four(const LinearArgs& a, float* r, int row, size_t tok, bool on) {
    if (!on || !a.residual) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = 0.f;
    } else if (a.vec && row < a.rows) {
        const size_t at = tok * a.residual_stride + row;
        const float4 v = a.type == GQ_F32   ? load4(static_cast<const float*>(a.residual) + at)
                         : a.type == GQ_F16 ? load4(static_cast<const __half*>(a.residual) + at)
                                            : load4(static_cast<const __nv_bfloat16*>(a.residual) + at);
        r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = row + i < a.rows ? load_typed(a.residual, tok * a.residual_stride + row + i, a.type) : 0.f;
    }
}
// G tokens a lane, tok, tok + 4, ..., of which those below `end` exist: their chains run beside one another.
template <bool PAIR, int G>
__device__ __forceinline__ void finish_fours(const LinearArgs& a, float (&y)[4 * G], const float (&other)[4 * G], int row, int tok, int end, int lane) {
    bend_all(y, a.function);
#pragma unroll
    for (int i = 0; i < 4 * G; ++i) y[i] = PAIR ? y[i] * other[i] : a.residual ? y[i] + other[i] : y[i];
    if (a.y) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (tok + 4 * g >= end) continue;
            const size_t at = static_cast<size_t>(tok + 4 * g) * a.y_stride + row;
            if (a.vec && row < a.rows) {
                const float4 v = make_float4(y[4 * g], y[4 * g + 1], y[4 * g + 2], y[4 * g + 3]);
                if (a.type == GQ_F32) store4(static_cast<float*>(a.y) + at, v);
                else if (a.type == GQ_F16) store4(static_cast<__half*>(a.y) + at, v);
                else store4(static_cast<__nv_bfloat16*>(a.y) + at, v);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) if (row + i < a.rows) store_typed(a.y, at + i, a.type, y[4 * g + i]);
            }
        }
    }
    if (a.blocks) {
        uint32_t top[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float* v = y + 4 * g;
            top[g] = __float_as_uint(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
            const float sum = (v[0] + v[1]) + (v[2] + v[3]);
            if (sum != sum) top[g] = 0x7fffffffu;                                 // a NaN, or infinities that make one
        }
        const int sub = lane & 7;
        auto block = [&](int t) { return reinterpret_cast<uint16_t*>(a.blocks + (static_cast<size_t>(t) * (a.rows / 32) + row / 32) * 34); };
        if constexpr (G == 4) {
            float4 v[4];
            float m[4];
            int c[4][4];
#pragma unroll
            for (int g = 0; g < 4; ++g) v[g] = make_float4(y[4 * g], y[4 * g + 1], y[4 * g + 2], y[4 * g + 3]), m[g] = __uint_as_float(top[g]);
            const float dd = q8_0_four(v, m, [](float p, float q) { return __uint_as_float(max(__float_as_uint(p), __float_as_uint(q))); }, c);
            if (row < a.rows) {
                if (!(sub & 1) && tok + 2 * sub < end) block(tok + 2 * sub)[0] = __half_as_ushort(__float2half_rn(dd));
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (tok + 4 * g >= end) break;
                    uint16_t* p = block(tok + 4 * g) + 1 + 2 * sub;
                    p[0] = static_cast<uint16_t>(__byte_perm(c[g][0], c[g][1], 0x0040));
                    p[1] = static_cast<uint16_t>(__byte_perm(c[g][2], c[g][3], 0x0040));
                }
            }
        } else {
#pragma unroll
            for (int o = 4; o > 0; o >>= 1)
#pragma unroll
                for (int g = 0; g < G; ++g) top[g] = max(top[g], __shfl_xor_sync(0xffffffffu, top[g], o));   // as bits: NaN above all
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float amax = __uint_as_float(top[g]), dd = q8_0_scale_fast(amax);
                int c[4];
                q8_0_quant4<true>(make_float4(y[4 * g], y[4 * g + 1], y[4 * g + 2], y[4 * g + 3]), amax, dd, c);
                if (tok + 4 * g < end && row < a.rows) {
                    uint16_t* p = block(tok + 4 * g);
                    if (sub == 0) p[0] = __half_as_ushort(__float2half_rn(dd));
                    p[1 + 2 * sub] = static_cast<uint16_t>(__byte_perm(c[0], c[1], 0x0040));
                    p[2 + 2 * sub] = static_cast<uint16_t>(__byte_perm(c[2], c[3], 0x0040));
                }
            }
        }
    }
}

// The power of two that a token's values are multiplied by, 2^(7 - E) for scales below 2^(E + 1) (f16 bits without sign):
// codes times scales are then below 2^15, and it is undone after the sums.
__device__ __forceinline__ int token_shift(uint32_t largest) {
    const int e = static_cast<int>(largest >> 10);                               // 31: not finite, whatever comes
    if (e) return 7 - (e - 15);
    return 7 - (largest ? -24 + (31 - __clz(largest)) : -24);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Two f16 parts of a value
__device__ __forceinline__ void two_parts(float v, uint16_t& hi, uint16_t& lo) {
    const __half h = __float2half_rn(v);
    hi = __half_as_ushort(h);
    lo = __half_as_ushort(__float2half_rn(v - __half2float(h)));
}

}  // namespace
}  // namespace gq
