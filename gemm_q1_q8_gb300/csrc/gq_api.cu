// The C ABI of libgq: argument validation on the host, then one launch on the caller's stream.
// Nothing here allocates device memory or synchronizes, except gq_device_error().
#include <algorithm>
#include <cstdint>

#include "gq_internal.cuh"
#include "layer_ops.cuh"
#include "wq_mma.cuh"
#include "w1a32_mma.cuh"

namespace {

thread_local int t_last_cuda_error = 0;

constexpr int kMaxK = 65536;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return GQ_OK;
    t_last_cuda_error = static_cast<int>(e);
    return GQ_ECUDA;
}

int check_q1(const void* packed, const void* act, const float* y, int rows, int n) {
    if (rows < 1 || n < 128 || n % 128 != 0 || n > gq::kMaxN) return GQ_EINVAL_SHAPE;
    if (!packed || !act || !y) return GQ_EINVAL_PTR;
    if (!aligned(packed, 16) || !aligned(act, 2) || !aligned(y, 4)) return GQ_EINVAL_PTR;
    return GQ_OK;
}

}  // namespace

namespace gq {
void record_cuda_error(int err) { t_last_cuda_error = err; }
}  // namespace gq

extern "C" {

const char* gq_version(void) { return "gq 0.1.0 (sm_103a)"; }

const char* gq_status_string(int status) {
    switch (status) {
        case GQ_OK: return "ok";
        case GQ_EINVAL_SHAPE: return "invalid shape";
        case GQ_EINVAL_PTR: return "invalid pointer (null or misaligned)";
        case GQ_EUNSUPPORTED: return "unsupported path";
        case GQ_ECUDA: return "CUDA launch error";
        default: return "unknown status";
    }
}

int gq_last_cuda_error(void) { return t_last_cuda_error; }

int gq_device_error(void) {
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_status(e) == GQ_OK ? 0 : -1;
    const unsigned v = gq::error_read_clear_q1() | gq::error_read_clear_q1_gemv() | gq::error_read_clear_ternary() | gq::error_read_clear_prefill_mma() |
                       gq::error_read_clear_wq_mma() | gq::error_read_clear_w1a32() | gq::error_read_clear_probes() |
                       gq::error_read_clear_block_q8() | gq::error_read_clear_kv() | gq::error_read_clear_attn() |
                       gq::error_read_clear_attn_tiles();
    return v == ~0u ? -1 : static_cast<int>(v);
}

size_t gq_q1_0_packed_bytes(int rows, int n) {
    if (rows < 1 || n < 128 || n % 128 != 0 || n > gq::kMaxN) return 0;
    const size_t tiles = (static_cast<size_t>(rows) + gq::kTileRows - 1) / gq::kTileRows;
    return tiles * static_cast<size_t>(n / 128) * gq::kChunkBytes;
}

int gq_q1_0_pack(const void* raw, int rows, int n, void* packed, gq_stream_t stream) {
    if (rows < 1 || n < 128 || n % 128 != 0 || n > gq::kMaxN) return GQ_EINVAL_SHAPE;
    if (!raw || !packed || !aligned(packed, 16)) return GQ_EINVAL_PTR;
    return cuda_status(gq::launch_q1_pack(raw, rows, n, packed, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gq_q1_q8_workspace_bytes(int n) {
    if (n < 128 || n % 128 != 0 || n > gq::kMaxN) return 0;
    return gq::gemv_workspace_bytes(n);
}

int q1_q8_gemv(const void* packed_w, const void* act, float* y, int rows, int n, void* workspace,
               gq_stream_t stream) {
    const int st = check_q1(packed_w, act, y, rows, n);
    if (st != GQ_OK) return st;
    if (!workspace || !aligned(workspace, 16)) return GQ_EINVAL_PTR;
    return cuda_status(gq::launch_q1_gemv(packed_w, act, y, rows, n, workspace, GQ_ACT_Q8_0,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

int q1_q8_gemv_raw(const void* w_q1_0, const void* act, float* y, int rows, int n, gq_stream_t stream) {
    if (rows < 1 || n < 128 || n % 128 != 0 || n > gq::kMaxN) return GQ_EINVAL_SHAPE;
    if (!w_q1_0 || !act || !y || !aligned(w_q1_0, 2) || !aligned(act, 2) || !aligned(y, 4)) return GQ_EINVAL_PTR;
    return cuda_status(gq::launch_q1_gemv_raw(w_q1_0, act, y, rows, n, reinterpret_cast<cudaStream_t>(stream)));
}

int gq_pack_q8_0(const void* raw_q8_0, int cols, int n, float* d, uint32_t* q, gq_stream_t stream) {
    if (cols < 1 || n < 32 || n % 32 != 0 || n > gq::kMaxN) return GQ_EINVAL_SHAPE;
    if (!raw_q8_0 || !d || !q || !aligned(raw_q8_0, 2) || !aligned(d, 4) || !aligned(q, 4)) return GQ_EINVAL_PTR;
    return cuda_status(gq::launch_pack_q8_0(raw_q8_0, cols, n, d, q, reinterpret_cast<cudaStream_t>(stream)));
}

int q1_q8_gemv_f32(const void* packed_w, const float* x, float* y, int rows, int n, void* workspace,
                   gq_stream_t stream) {
    const int st = check_q1(packed_w, x, y, rows, n);
    if (st != GQ_OK) return st;
    if (!aligned(x, 16) || !workspace || !aligned(workspace, 16)) return GQ_EINVAL_PTR;
    return cuda_status(gq::launch_q1_gemv(packed_w, x, y, rows, n, workspace, GQ_ACT_F32,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

int gq_gemv_group_plan(gq_gemv_desc* descs, int count, int* total_tiles) {
    if (!descs || !total_tiles) return GQ_EINVAL_PTR;
    if (count < 1 || count > 65535) return GQ_EINVAL_SHAPE;
    for (int i = 0; i < count; ++i) {
        const int st = check_q1(descs[i].packed_w, descs[i].act, descs[i].y, descs[i].rows, descs[i].n);
        if (st != GQ_OK) return st;
        if (descs[i].act_format != GQ_ACT_Q8_0 && descs[i].act_format != GQ_ACT_F32) return GQ_EINVAL_SHAPE;
        if (descs[i].act_format == GQ_ACT_F32 && !aligned(descs[i].act, 16)) return GQ_EINVAL_PTR;
        if (!descs[i].workspace || !aligned(descs[i].workspace, 16)) return GQ_EINVAL_PTR;
    }
    // Largest n first (stable): the kernel hands tiles to warps in snake order over this list.
    std::stable_sort(descs, descs + count,
                     [](const gq_gemv_desc& a, const gq_gemv_desc& b) { return a.n > b.n; });
    long long tiles = 0;
    for (int i = 0; i < count; ++i) {
        descs[i].tile_begin = static_cast<int>(tiles);
        tiles += gq::gemv_tiles_for(descs[i].rows);
        if (tiles > 0x7fffffffLL) return GQ_EINVAL_SHAPE;
    }
    *total_tiles = static_cast<int>(tiles);
    return GQ_OK;
}

int q1_q8_gemv_grouped(const gq_gemv_desc* descs, int count, int total_tiles, int* counter, gq_stream_t stream) {
    if (!descs || !aligned(descs, 8) || !counter || !aligned(counter, 4)) return GQ_EINVAL_PTR;
    if (count < 1 || count > 65535 || total_tiles < 1) return GQ_EINVAL_SHAPE;
    return cuda_status(
        gq::launch_q1_gemv_grouped(descs, count, total_tiles, counter, reinterpret_cast<cudaStream_t>(stream)));
}

int q1_q8_gemm(const void* packed_w, const void* act, float* y, int rows, int n, int cols, int path,
               gq_stream_t stream) {
    const int st = check_q1(packed_w, act, y, rows, n);
    if (st != GQ_OK) return st;
    if (cols < 1 || cols > 65535 * 4) return GQ_EINVAL_SHAPE;
    if (path == GQ_PATH_AUTO) path = GQ_PATH_DP4A;
    if (path != GQ_PATH_DP4A && path != GQ_PATH_LUT4) return GQ_EUNSUPPORTED;
    return cuda_status(gq::launch_q1_gemm(packed_w, act, y, rows, n, cols, path, reinterpret_cast<cudaStream_t>(stream)));
}

int block_q8_matmul_nt(const float* x, const uint32_t* quants, const float* scales, float* y, int m, int k, int n,
                       gq_stream_t stream) {
    if (m < 1 || k < 32 || n < 1 || k % 32 != 0 || k > kMaxK || m > 65535 * 16) return GQ_EINVAL_SHAPE;
    if (!x || !quants || !scales || !y) return GQ_EINVAL_PTR;
    if (!aligned(x, 4) || !aligned(quants, 16) || !aligned(scales, 4) || !aligned(y, 4)) return GQ_EINVAL_PTR;
    return cuda_status(gq::launch_block_q8(x, quants, scales, y, m, k, n, reinterpret_cast<cudaStream_t>(stream)));
}

int q1s32_f32_gemm(const uint32_t* signs, const float* wscale, const float* x, float* y, int M, int N, int K, int path,
                   gq_stream_t stream) {
    if (N < 1 || M < 1 || M > 65535 || K < 32 || K % 32 != 0 || K > kMaxK) return GQ_EINVAL_SHAPE;
    if (path == GQ_PATH_AUTO) path = GQ_PATH_LUT4;
    if (path != GQ_PATH_LUT4 && path != GQ_PATH_FMA) return GQ_EUNSUPPORTED;
    if (!signs || !wscale || !x || !y) return GQ_EINVAL_PTR;
    if (!aligned(signs, 4) || !aligned(wscale, 4) || !aligned(x, 16) || !aligned(y, 4)) return GQ_EINVAL_PTR;
    return cuda_status(
        gq::launch_q1s32_f32(signs, wscale, x, y, M, N, K, path, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gq_q1s32_mma_workspace_bytes(int M, int K) {
    if (M < 1 || M > 65535 * 128 || K < 64 || K % 64 != 0 || K > kMaxK) return 0;
    return gq::w1a32_mma_workspace_bytes(M, K);
}

int q1s32_f32_gemm_mma(const uint32_t* signs, const float* wscale, const float* x, float* y, int M, int N, int K,
                       void* workspace, gq_stream_t stream) {
    if (N < 1 || M < 1 || M > 65535 * 128 || K < 64 || K % 64 != 0 || K > kMaxK) return GQ_EINVAL_SHAPE;
    if (!signs || !wscale || !x || !y || !workspace) return GQ_EINVAL_PTR;
    if (!aligned(signs, 16) || !aligned(wscale, 8) || !aligned(x, 4) || !aligned(y, 4) || !aligned(workspace, 16))
        return GQ_EINVAL_PTR;
    return cuda_status(
        gq::launch_w1a32_mma(signs, wscale, x, y, M, N, K, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

static int wq_call(int bits, const uint32_t* w, const float* scale, const float* x, float* y, int T, int N, int K,
                   gq_stream_t stream) {
    if (N < 1 || T < 1 || T > 65535 * 128 || K < 32 || K % 32 != 0 || K > kMaxK) return GQ_EINVAL_SHAPE;
    if (!w || !scale || !x || !y) return GQ_EINVAL_PTR;
    if (!aligned(w, 16) || !aligned(scale, 4) || !aligned(x, 16) || !aligned(y, 4)) return GQ_EINVAL_PTR;
    return cuda_status(gq::launch_wq(bits, w, scale, x, y, T, N, K, reinterpret_cast<cudaStream_t>(stream)));
}

int matvec_q8(const uint32_t* w, const float* scale, const float* x, float* y, int N, int K, gq_stream_t stream) {
    return wq_call(8, w, scale, x, y, 1, N, K, stream);
}
int matmul_q8(const uint32_t* w, const float* scale, const float* x, float* y, int T, int N, int K,
              gq_stream_t stream) {
    return wq_call(8, w, scale, x, y, T, N, K, stream);
}
size_t gq_wq_mma_workspace_bytes(int T, int K) {
    if (T < 1 || T > 65535 * 128 || K < 64 || K % 32 != 0 || K > kMaxK) return 0;
    return gq::wq_mma_workspace_bytes(T, K);
}

static int wq_mma_call(int bits, const uint32_t* w, const float* scale, const float* x, float* y, int T, int N, int K,
                       void* workspace, gq_stream_t stream) {
    if (N < 1 || T < 1 || T > 65535 * 128 || K < 64 || K % 32 != 0 || K > kMaxK) return GQ_EINVAL_SHAPE;
    if (!w || !scale || !x || !y || !workspace) return GQ_EINVAL_PTR;
    if (!aligned(w, 16) || !aligned(scale, 4) || !aligned(x, 16) || !aligned(y, 4) || !aligned(workspace, 16))
        return GQ_EINVAL_PTR;
    return cuda_status(
        gq::launch_wq_mma(bits, w, scale, x, y, T, N, K, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

int matmul_q8_mma(const uint32_t* w, const float* scale, const float* x, float* y, int T, int N, int K,
                  void* workspace, gq_stream_t stream) {
    return wq_mma_call(8, w, scale, x, y, T, N, K, workspace, stream);
}
int matmul_q4g128_mma(const uint32_t* w, const float* scale, const float* x, float* y, int T, int N, int K,
                      void* workspace, gq_stream_t stream) {
    return wq_mma_call(4, w, scale, x, y, T, N, K, workspace, stream);
}

int matvec_q4g128(const uint32_t* w, const float* scale, const float* x, float* y, int N, int K, gq_stream_t stream) {
    return wq_call(4, w, scale, x, y, 1, N, K, stream);
}
int matmul_q4g128(const uint32_t* w, const float* scale, const float* x, float* y, int T, int N, int K,
                  gq_stream_t stream) {
    return wq_call(4, w, scale, x, y, T, N, K, stream);
}

int ternary_bitplane_gemv(const uint32_t* P, const uint32_t* N, const uint32_t* X, int32_t* y, int rows, int k,
                          int batch, gq_stream_t stream) {
    if (rows < 1 || k < 1024 || batch < 1 || k % 1024 != 0 || k > kMaxK || batch > 64) return GQ_EINVAL_SHAPE;
    if (!P || !N || !X || !y) return GQ_EINVAL_PTR;
    if (!aligned(P, 16) || !aligned(N, 16) || !aligned(X, 16) || !aligned(y, 4)) return GQ_EINVAL_PTR;
    return cuda_status(gq::launch_ternary(P, N, X, y, rows, k, batch, reinterpret_cast<cudaStream_t>(stream)));
}

int gq_quantize_q8_0(const float* x, int m, int k, uint16_t* d, int8_t* q, uint16_t* op, gq_stream_t stream) {
    if (m < 1 || k < 32 || k % 32 != 0 || k > kMaxK) return GQ_EINVAL_SHAPE;
    if (!x || !d || !q) return GQ_EINVAL_PTR;
    if (!aligned(x, 4) || !aligned(d, 2) || !aligned(q, 16) || (op && !aligned(op, 16))) return GQ_EINVAL_PTR;
    return cuda_status(gq::launch_quantize(x, m, k, d, q, op, reinterpret_cast<cudaStream_t>(stream)));
}

int q1s32_q8_gemm(const uint32_t* signs, const float* wscale, const uint16_t* xd, const int8_t* xq,
                  const uint16_t* xq_mma, float* y, int M, int N, int K, int path, gq_stream_t stream) {
    if (M < 1 || N < 1 || K < 64 || K % 64 != 0 || K > kMaxK || M > 65535 * 32) return GQ_EINVAL_SHAPE;
    if (path == GQ_PATH_AUTO) path = (xq_mma && M >= 64) ? GQ_PATH_MMA : GQ_PATH_LUT4;
    if (path != GQ_PATH_LUT4 && path != GQ_PATH_MMA) return GQ_EUNSUPPORTED;
    if (!signs || !wscale || !xd || !xq || !y) return GQ_EINVAL_PTR;
    if (!aligned(signs, 16) || !aligned(wscale, 4) || !aligned(xd, 4) || !aligned(xq, 16) || !aligned(y, 4))
        return GQ_EINVAL_PTR;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (path == GQ_PATH_MMA) {
        if (!xq_mma || !aligned(xq_mma, 16) || !aligned(wscale, 8)) return GQ_EINVAL_PTR;   // row scales as pairs
        const cudaError_t e = gq::launch_prefill_mma(signs, wscale, xd, xq_mma, y, M, N, K, s);
        if (e == cudaErrorNotSupported) return GQ_EUNSUPPORTED;
        return cuda_status(e);
    }
    return cuda_status(gq::launch_prefill_lut4(signs, wscale, xd, xq, y, M, N, K, s));
}

// ---------------------------------------------------------------- between a layer's products

static size_t type_bytes(int type) { return type == GQ_F32 ? 4 : type == GQ_F16 || type == GQ_BF16 ? 2 : 0; }

static bool cache_shape(int pages, int page_size, int kv_heads, int head_dim) {
    return pages >= 1 && page_size >= 16 && page_size <= 65536 && page_size % 16 == 0 && kv_heads >= 1 && kv_heads <= 1024 &&
           (head_dim == 64 || head_dim == 128 || head_dim == 256) && static_cast<long long>(pages) * page_size < (1ll << 40);
}

int gq_rmsnorm(const void* x, long long x_stride, const void* residual, long long residual_stride, const float* weight,
               float eps, int type, int m, int k, void* sum, void* y, void* act, uint16_t* d, int8_t* q, uint16_t* op,
               gq_stream_t stream) {
    if (m < 1 || k < 1 || k > kMaxK || x_stride < k || (residual && residual_stride < k) || !(eps >= 0.0f))
        return GQ_EINVAL_SHAPE;
    if ((act || d || q || op) && k % 32 != 0) return GQ_EINVAL_SHAPE;
    const size_t b = type_bytes(type);
    if (!b) return GQ_EUNSUPPORTED;
    if (!x || !weight || (!sum && !y && !act && !d && !q && !op) || !d != !q || (op && !q)) return GQ_EINVAL_PTR;
    if (!aligned(x, b) || !aligned(residual, b) || !aligned(weight, 4) || !aligned(sum, b) || !aligned(y, b) ||
        !aligned(act, 2) || !aligned(d, 2) || !aligned(q, 16) || !aligned(op, 16))
        return GQ_EINVAL_PTR;
    if ((sum == x && sum && x_stride != k) || (sum && sum == residual && residual_stride != k)) return GQ_EINVAL_PTR;
    return cuda_status(gq::launch_rmsnorm(x, x_stride, residual, residual_stride, weight, eps, type, m, k, sum, y, act, d, q,
                                          op, reinterpret_cast<cudaStream_t>(stream)));
}

int gq_dequantize_q8_0(const void* act, long long blocks, int type, void* out, gq_stream_t stream) {
    if (blocks < 1 || blocks > (1ll << 40)) return GQ_EINVAL_SHAPE;
    if (!type_bytes(type)) return GQ_EUNSUPPORTED;
    if (!act || !out || !aligned(act, 2) || !aligned(out, 16)) return GQ_EINVAL_PTR;
    return cuda_status(gq::launch_dequantize_q8_0(act, blocks, type, out, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gq_kv_cache_bytes(int pages, int page_size, int kv_heads, int head_dim) {
    if (!cache_shape(pages, page_size, kv_heads, head_dim)) return 0;
    return static_cast<size_t>(pages) * (page_size / 16) * kv_heads * gq::kv_chunk_bytes(head_dim);
}

int gq_rope_table(float* table, int positions, int rot, double base, int scaling, double factor, double original,
                  gq_stream_t stream) {
    if (positions < 1 || rot < 8 || rot > 256 || rot % 8 != 0 || !(base > 1.0) || !(factor >= 1.0)) return GQ_EINVAL_SHAPE;
    if (scaling < GQ_ROPE_PLAIN || scaling > GQ_ROPE_YARN) return GQ_EUNSUPPORTED;
    if (scaling == GQ_ROPE_YARN && !(original >= 1.0)) return GQ_EINVAL_SHAPE;
    if (!table || !aligned(table, 8)) return GQ_EINVAL_PTR;
    return cuda_status(gq::launch_rope_table(table, positions, rot, base, scaling, factor, original,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

int gq_rope_kv_append(const void* q, long long q_stride, void* q_out, long long q_out_stride, const void* k,
                      long long k_stride, const void* v, long long v_stride, int type, const float* rope, int rope_rows,
                      int rot, int layout, const int32_t* positions, const int64_t* slots, int tokens, int q_heads,
                      int kv_heads, int head_dim, void* cache, int pages, int page_size, gq_stream_t stream) {
    if (tokens < 1 || q_heads < 0 || q_heads > 1024 || !cache_shape(pages, page_size, kv_heads, head_dim)) return GQ_EINVAL_SHAPE;
    if (!rope) rot = 0;
    if (rot < 0 || rot > head_dim || rot % 8 != 0 || (rot && rope_rows < 1)) return GQ_EINVAL_SHAPE;
    const long long qw = static_cast<long long>(q_heads) * head_dim, kw = static_cast<long long>(kv_heads) * head_dim;
    if ((q_heads && (q_stride < qw || q_out_stride < qw)) || k_stride < kw || v_stride < kw) return GQ_EINVAL_SHAPE;
    const size_t b = type_bytes(type);
    if (!b || (layout != GQ_ROPE_HALF && layout != GQ_ROPE_INTERLEAVED)) return GQ_EUNSUPPORTED;
    if ((q_heads && (!q || !q_out)) || !k || !v || !slots || !cache || (rot && !positions)) return GQ_EINVAL_PTR;
    if (!aligned(k, 4 * b) || !aligned(v, 4 * b) || k_stride % 4 || v_stride % 4 || !aligned(cache, 16) ||
        !aligned(slots, 8) || (rot && (!aligned(rope, 16) || !aligned(positions, 4))))
        return GQ_EINVAL_PTR;
    if (q_heads && (!aligned(q, 4 * b) || !aligned(q_out, 4 * b) || q_stride % 4 || q_out_stride % 4 ||
                    (q == q_out && q_stride != q_out_stride)))
        return GQ_EINVAL_PTR;
    const gq::AppendArgs a = {q, q_out, k, v, q_stride, q_out_stride, k_stride, v_stride, rope, rope_rows, rot,
                              layout == GQ_ROPE_INTERLEAVED, positions, slots, tokens, q_heads, kv_heads,
                              static_cast<uint8_t*>(cache), pages, page_size};
    return cuda_status(gq::launch_kv_append(a, type, head_dim, reinterpret_cast<cudaStream_t>(stream)));
}

int gq_kv_read(const void* cache, int pages, int page_size, int kv_heads, int head_dim, const int64_t* slots, int n,
               int type, void* k_out, void* v_out, gq_stream_t stream) {
    if (n < 1 || !cache_shape(pages, page_size, kv_heads, head_dim)) return GQ_EINVAL_SHAPE;
    if (!type_bytes(type)) return GQ_EUNSUPPORTED;
    if (!cache || !slots || (!k_out && !v_out) || !aligned(cache, 16) || !aligned(slots, 8) || !aligned(k_out, 16) ||
        !aligned(v_out, 16))
        return GQ_EINVAL_PTR;
    return cuda_status(gq::launch_kv_read(static_cast<const uint8_t*>(cache), pages, page_size, kv_heads, head_dim, slots, n,
                                          type, k_out, v_out, reinterpret_cast<cudaStream_t>(stream)));
}

static bool attn_shape(int seqs, int max_q, int q_heads, int kv_heads, int head_dim) {
    return seqs >= 1 && seqs <= 65535 && max_q >= 1 && q_heads >= 1 && kv_heads >= 1 && kv_heads <= 1024 &&
           q_heads % kv_heads == 0 && q_heads / kv_heads <= 64 && (head_dim == 64 || head_dim == 128 || head_dim == 256);
}

size_t gq_attn_workspace_bytes(int seqs, int max_q, int q_heads, int kv_heads, int head_dim, int type) {
    if (!attn_shape(seqs, max_q, q_heads, kv_heads, head_dim) || !type_bytes(type)) return 0;
    return gq::attn_workspace_bytes(seqs, max_q, q_heads, kv_heads, head_dim, type);
}

static int attn_call(const void* q, long long q_stride, void* out, long long out_stride, int type, const void* cache, int pages,
                     int page_size, const int32_t* table, int table_stride, const int32_t* kv_len, const int32_t* q_start,
                     const uint64_t* tree, int rows, int seqs, int max_q, int max_kv, int q_heads, int kv_heads, int head_dim,
                     float scale, float softcap, void* workspace, gq_stream_t stream) {
    if (!attn_shape(seqs, max_q, q_heads, kv_heads, head_dim) || !cache_shape(pages, page_size, kv_heads, head_dim) ||
        max_kv < 1 || (tree && max_q > 64))
        return GQ_EINVAL_SHAPE;
    const long long w = static_cast<long long>(q_heads) * head_dim;
    if (q_stride < w || out_stride < w || table_stride < (max_kv - 1) / page_size + 1) return GQ_EINVAL_SHAPE;
    if (!(scale - scale == 0.0f) || !(softcap >= 0.0f) || !(softcap - softcap == 0.0f)) return GQ_EINVAL_SHAPE;
    const size_t b = type_bytes(type);
    if (!b) return GQ_EUNSUPPORTED;
    if (!q || !out || !cache || !table || !kv_len || !q_start || !workspace) return GQ_EINVAL_PTR;
    if (!aligned(q, 4 * b) || !aligned(out, 4 * b) || q_stride % 4 || out_stride % 4 || !aligned(cache, 16) ||
        !aligned(workspace, 16) || !aligned(table, 4) || !aligned(kv_len, 4) || !aligned(q_start, 4) || !aligned(tree, 8))
        return GQ_EINVAL_PTR;
    // a cap that no score comes near is none, and below the other bound all weights are equal in f32: products of either with the scale could
    // leave f32's range
    if (softcap > 1e20f) softcap = 0.0f;
    if (softcap > 0.0f && softcap < 1e-30f) softcap = 1e-30f;
    const gq::AttnArgs a = {q, out, q_stride, out_stride, static_cast<const uint8_t*>(cache), pages, page_size, table,
                            table_stride, kv_len, q_start, tree, rows, seqs, max_q, max_kv, q_heads, kv_heads, scale, softcap,
                            workspace};
    return cuda_status(gq::launch_attn(a, type, head_dim, reinterpret_cast<cudaStream_t>(stream)));
}

int gq_attn_q8_0(const void* q, long long q_stride, void* out, long long out_stride, int type, const void* cache, int pages,
                 int page_size, const int32_t* table, int table_stride, const int32_t* kv_len, const int32_t* q_start,
                 const uint64_t* tree, int seqs, int max_q, int max_kv, int q_heads, int kv_heads, int head_dim, float scale,
                 float softcap, void* workspace, gq_stream_t stream) {
    return attn_call(q, q_stride, out, out_stride, type, cache, pages, page_size, table, table_stride, kv_len, q_start, tree, -1, seqs,
                     max_q, max_kv, q_heads, kv_heads, head_dim, scale, softcap, workspace, stream);
}

int gq_attn_q8_0_bounded(const void* q, long long q_stride, void* out, long long out_stride, int type, const void* cache,
                         int pages, int page_size, const int32_t* table, int table_stride, const int32_t* kv_len,
                         const int32_t* q_start, const uint64_t* tree, int rows, int seqs, int max_q, int max_kv, int q_heads,
                         int kv_heads, int head_dim, float scale, float softcap, void* workspace, gq_stream_t stream) {
    if (rows < 0) return GQ_EINVAL_SHAPE;
    return attn_call(q, q_stride, out, out_stride, type, cache, pages, page_size, table, table_stride, kv_len, q_start, tree, rows,
                     seqs, max_q, max_kv, q_heads, kv_heads, head_dim, scale, softcap, workspace, stream);
}

}  // extern "C"
