// RMS norm with the residual's addition and a Q8_0 output, and Q8_0 blocks read back.
//
// h = x + r; y = h * rstd * w, rstd = 1 / sqrt(sum h^2 / k + eps); y quantized per 32 values as the library's
// quantizer does.  One pass over x and r: a thread block per row keeps h in registers between the sum and
// the outputs, so a value is read once and written once (5 to 13 bytes moved a value, 7 flops and a quantization).  Bound by HBM
// for many rows (8192 f32 rows of 4096 with residual and sum, and the read back of their blocks: 93 us, 86% of the measured rate), by
// two dependent round trips and two barriers for one (2560 values, with the read back: 3.2 us).
#include "layer_ops.cuh"

namespace gq {
namespace {

struct NormArgs {
    const void* x; const void* r; const float* w;
    long long xs, rs;
    float eps;
    int k;
    void* h; void* y;
    uint8_t* act;
    uint16_t* d; int8_t* q; uint16_t* op;
    size_t plane;                                     // m * k: the operand's plane stride
};

template <typename T, bool VEC>
__device__ __forceinline__ float4 load_row4(const T* row, int i, int k) {
    if (VEC) return i < k ? load4(row + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 v;
    v.x = i < k ? to_f32(row[i]) : 0.f;
    v.y = i + 1 < k ? to_f32(row[i + 1]) : 0.f;
    v.z = i + 2 < k ? to_f32(row[i + 2]) : 0.f;
    v.w = i + 3 < k ? to_f32(row[i + 3]) : 0.f;
    return v;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_row4(T* row, int i, int k, float4 v) {
    if (VEC) {
        if (i < k) store4(row + i, v);
        return;
    }
    if (i < k) from_f32(row + i, v.x);
    if (i + 1 < k) from_f32(row + i + 1, v.y);
    if (i + 2 < k) from_f32(row + i + 2, v.z);
    if (i + 3 < k) from_f32(row + i + 3, v.w);
}
template <typename T, bool VEC>
__device__ __forceinline__ float4 load_h(const NormArgs& a, const T* xr, const T* rr, int i) {
    float4 v = load_row4<T, VEC>(xr, i, a.k);
    if (rr) {
        const float4 u = load_row4<T, VEC>(rr, i, a.k);
        v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
    }
    return v;
}

// y of four values quantized and written: eight neighbouring threads hold one 32-block.  `on` is the
// same for the eight; every lane of the warp takes part in the shuffles.
__device__ __forceinline__ void quantize4(const NormArgs& a, size_t row, int i, bool on, float4 y) {
    const int lane = threadIdx.x & 31, sub = lane & 7;
    float amax = fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w)));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float dd = q8_0_scale_fast(amax);
    const uint16_t dbits = __half_as_ushort(__float2half_rn(dd));
    int cd[4];
    q8_0_quant4(y, amax, dd, cd);
    const uint32_t word = __byte_perm(__byte_perm(cd[0], cd[1], 0x0040), __byte_perm(cd[2], cd[3], 0x0040), 0x5410);
    const size_t block = row * (a.k / 32) + (i >> 5);
    if (a.act && on) {
        uint16_t* p = reinterpret_cast<uint16_t*>(a.act + block * 34);
        if (sub == 0) p[0] = dbits;
        p[1 + 2 * sub] = static_cast<uint16_t>(word);
        p[2 + 2 * sub] = static_cast<uint16_t>(word >> 16);
    }
    if (a.q && on) {
        *reinterpret_cast<uint32_t*>(a.q + block * 32 + 4 * sub) = word;
        if (sub == 0) a.d[block] = dbits;
    }
    if (a.op) {
        // three bf16 parts of f16(d) * q, element u and u + 16 of the block side by side: the lane of the
        // lower half takes its partner's four
        const float ds = f16_to_f32(dbits);
        float pv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pv[e] = __fmul_rn(ds, static_cast<float>(cd[e]));
        uint32_t w[3][4];
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat16 b = __float2bfloat16_rn(pv[e]);
                pv[e] = __fsub_rn(pv[e], __bfloat162float(b));
                const uint32_t mine = __bfloat16_as_ushort(b);
                w[p][e] = mine | __shfl_xor_sync(0xffffffffu, mine, 4) << 16;
            }
        if (on && sub < 4)
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *reinterpret_cast<uint4*>(a.op + p * a.plane + block * 32 + 8 * sub) =
                    make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
    }
}

// NV: four-value chunks a thread keeps in registers; a longer row's remaining chunks are read again
// (through L2) for the outputs.  VEC: rows and outputs allow four-value accesses.
template <typename T, int NV, bool VEC, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 3 : 1) rmsnorm_kernel(const NormArgs a) {
    __shared__ float part[32];
    const int tid = threadIdx.x, nt = blockDim.x;
    const size_t row = blockIdx.x;
    const T* xr = static_cast<const T*>(a.x) + row * a.xs;
    const T* rr = a.r ? static_cast<const T*>(a.r) + row * a.rs : nullptr;
    const int chunks = ((a.k + 3) / 4 + nt - 1) / nt;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // few rows: the weight's load goes out with the row's, behind the barrier it would cost a second round trip (2560 values: 3.6 -> 3.2 us
    // with the read back); many rows: its registers would cost resident blocks (8192 rows of 4096: 97 -> 108 us)
    float4 h[NV], w;
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < NV; ++c) h[c] = load_h<T, VEC>(a, xr, rr, 4 * (c * nt + tid));
    if (NV == 1) w = load_row4<float, VEC>(a.w, 4 * tid, a.k);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        s = fmaf(h[c].x, h[c].x, s);
        s = fmaf(h[c].y, h[c].y, s);
        s = fmaf(h[c].z, h[c].z, s);
        s = fmaf(h[c].w, h[c].w, s);
    }
    for (int c = NV; c < chunks; ++c) {
        const float4 v = load_h<T, VEC>(a, xr, rr, 4 * (c * nt + tid));
        s = fmaf(v.x, v.x, fmaf(v.y, v.y, fmaf(v.z, v.z, fmaf(v.w, v.w, s))));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((tid & 31) == 0) part[tid >> 5] = s;
    __syncthreads();
    s = (tid & 31) < nt / 32 ? part[tid & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(s, static_cast<float>(a.k)) + a.eps));

    auto emit = [&](int i, float4 v, float4 w) {
        if (a.h) store_row4<T, VEC>(static_cast<T*>(a.h) + row * a.k, i, a.k, v);
        const float4 y = make_float4(v.x * rstd * w.x, v.y * rstd * w.y, v.z * rstd * w.z, v.w * rstd * w.w);
        if (a.y) store_row4<T, VEC>(static_cast<T*>(a.y) + row * a.k, i, a.k, y);
        if (a.act || a.q) quantize4(a, row, i, i < a.k, y);
    };
#pragma unroll
    for (int c = 0; c < NV; ++c)
        if (c < chunks) emit(4 * (c * nt + tid), h[c], NV == 1 ? w : load_row4<float, VEC>(a.w, 4 * (c * nt + tid), a.k));
    for (int c = NV; c < chunks; ++c) {
        const int i = 4 * (c * nt + tid);
        emit(i, load_h<T, VEC>(a, xr, rr, i), load_row4<float, VEC>(a.w, i, a.k));
    }
}

template <typename T, int NV>
cudaError_t norm_go(const NormArgs& a, int m, int nt, bool vec, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(m);
    cfg.blockDim = dim3(nt);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // 40 registers let three blocks of 512 threads share an SM (bf16, 8192 rows of 4096: 60.6 -> 54.4 us, 777 of 6912 with the read back
    // 16.6 -> 15.6); where two a SM hold all rows they only cost loads in flight (300 of 8192: 5.7 -> 7.5), and f32 rows would spill
    // (8192 of 4096: 93 -> 102)
    if constexpr (NV == 4 && sizeof(T) == 2)
        if (vec && nt <= 512 && m > 2 * 152) return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<T, NV, true, 512>, a);
    return vec ? cudaLaunchKernelEx(&cfg, rmsnorm_kernel<T, NV, true, 1024>, a) : cudaLaunchKernelEx(&cfg, rmsnorm_kernel<T, NV, false, 1024>, a);
}

template <typename T>
cudaError_t norm_type(const NormArgs& a, int m, cudaStream_t s) {
    auto al = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    const size_t n = 4 * sizeof(T);
    const bool vec = a.k % 4 == 0 && a.xs % 4 == 0 && (!a.r || a.rs % 4 == 0) && al(a.x, n) && al(a.r, n) && al(a.h, n) &&
                     al(a.y, n) && al(a.w, 16);
    const int k4 = (a.k + 3) / 4;
    auto threads = [&](int nv) { return ((k4 + nv - 1) / nv + 31) / 32 * 32; };
    // few rows: one chunk a thread, the most loads in flight; many rows: fewer threads a row
    if (m <= 152 && threads(1) <= 1024) return norm_go<T, 1>(a, m, threads(1), vec, s);
    if (threads(4) <= 1024) return norm_go<T, 4>(a, m, threads(4), vec, s);
    return norm_go<T, 8>(a, m, threads(8) < 1024 ? threads(8) : 1024, vec, s);
}

// Eight threads a block, four values each.
template <typename T>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t* act, long long blocks, T* out) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < blocks * 8; i += step) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(act + (i >> 3) * 34);
        const int sub = static_cast<int>(i & 7);
        const float d = f16_to_f32(p[0]);
        const uint32_t lo = p[1 + 2 * sub], hi = p[2 + 2 * sub];
        store4(out + i * 4, make_float4(d * static_cast<float>(static_cast<int8_t>(lo & 0xff)),
                                        d * static_cast<float>(static_cast<int8_t>(lo >> 8)),
                                        d * static_cast<float>(static_cast<int8_t>(hi & 0xff)),
                                        d * static_cast<float>(static_cast<int8_t>(hi >> 8))));
    }
}

template <typename T>
cudaError_t dequantize_type(const void* act, long long blocks, void* out, cudaStream_t s) {
    const long long want = (blocks * 8 + 255) / 256;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < 152 * 16 ? want : 152 * 16));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dequantize_kernel<T>, static_cast<const uint8_t*>(act), blocks, static_cast<T*>(out));
}

}  // namespace

cudaError_t launch_rmsnorm(const void* x, long long xs, const void* r, long long rs, const float* w, float eps, int type,
                           int m, int k, void* h, void* y, void* act, uint16_t* d, int8_t* q, uint16_t* op,
                           cudaStream_t s) {
    const NormArgs a = {x, r, w, xs, rs, eps, k, h, y, static_cast<uint8_t*>(act), d, q, op, static_cast<size_t>(m) * k};
    if (type == GQ_F32) return norm_type<float>(a, m, s);
    if (type == GQ_F16) return norm_type<__half>(a, m, s);
    return norm_type<__nv_bfloat16>(a, m, s);
}

cudaError_t launch_dequantize_q8_0(const void* act, long long blocks, int type, void* out, cudaStream_t s) {
    if (type == GQ_F32) return dequantize_type<float>(act, blocks, out, s);
    if (type == GQ_F16) return dequantize_type<__half>(act, blocks, out, s);
    return dequantize_type<__nv_bfloat16>(act, blocks, out, s);
}

}  // namespace gq
