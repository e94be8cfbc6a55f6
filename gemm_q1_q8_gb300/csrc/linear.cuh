// Q1_0 products with an epilogue: what the kernel for few tokens (linear.cu) and the one for many (linear_tiles.cu) share.
//
//   z[c, r] = sum_b d0[r, b] * sum_k d1[c, 4b + k] * sum_t (+-1) q   (+ bias[r])
//   linear:  y = act(z) (+ residual[c, r]);      pair: y = act(z_gate) * z_up
//
// Both kernels take +-d0 as f16 matrix operands, made from the sign bits by two logic operations a pair, and the activations as
// pv = d1 * q * 2^-e, e one power of two a token: pv has at most 18 significant bits, so two f16 parts hold it exactly while it is
// not below 2^-20 of the token's largest (then it is off by at most 2^-39 of that).  f32, f16 and Q8_0 results take both
// parts; a bf16 result (8 bits) takes one, off by 2^-12 of each value.  Products are exact in f32, sums are f32; the tensor
// cores truncate the sum that they add to, so it goes to registers every few blocks of 128 (a chain of n steps costs n / 3 * 2^-23).
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
};

cudaError_t launch_linear(const LinearArgs& a, bool pair, cudaStream_t s);
size_t linear_workspace_bytes(int rows, int n, int cols, int type);
cudaError_t launch_linear_tiles(const LinearArgs& a, bool pair, cudaStream_t s);
size_t linear_tiles_workspace_bytes(int rows, int n, int cols, int parts);

namespace {

// f16 parts that an activation takes
__host__ __device__ __forceinline__ int linear_parts(const LinearArgs& a) { return a.type == GQ_BF16 && !a.blocks ? 1 : 2; }

// 1 / (1 + e^-v); the exponential of 2^-v log2(e) and the reciprocal are off by two units each, and give 0 below 2^-126
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

// Q8_0 blocks of a warp's values, one a lane (32 neighbouring rows of a token), of up to N neighbouring tokens `step` bytes apart, by the
// library's rule.  A NaN gives a NaN scale.  The tokens' chains run beside one another.
template <int N>
__device__ __forceinline__ void store_blocks(uint8_t* block, size_t step, const float (&v)[N], int count, int lane) {
    float amax[N], dd[N];
    int code[N];
    bool far = true;
#pragma unroll
    for (int i = 0; i < N; ++i) amax[i] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(v[i]))));
#pragma unroll
    for (int i = 0; i < N; ++i) {
        dd[i] = q8_0_scale_fast(amax[i]);
        bool sure;
        code[i] = q8_0_code_near(v[i], amax[i], dd[i], sure);
        far = far && sure;
    }
    if (!far)
#pragma unroll
        for (int i = 0; i < N; ++i) code[i] = q8_0_quant(v[i], amax[i], dd[i]);
    float mine = dd[0];                                                          // lane i stores the i-th scale
#pragma unroll
    for (int i = 1; i < N; ++i) mine = lane == i ? dd[i] : mine;
    if (lane < (N < count ? N : count)) *reinterpret_cast<uint16_t*>(block + lane * step) = __half_as_ushort(__float2half_rn(mine));
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < count) block[i * step + 2 + lane] = static_cast<uint8_t>(code[i]);
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
