/*
 * gq.h -- C ABI of libgq: low-bit block-quantized weight x activation matvec / matmul on GB300
 * (sm_103a).
 *
 * Conventions for every entry point:
 *  - Pointers named *device* point to device memory owned by the caller; the library never
 *    allocates or frees device memory on a call, never synchronizes the stream, and keeps no
 *    per-call state.  Host pointers are named as such.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default stream) and
 *    completes asynchronously.
 *  - Every call validates its arguments on the host before launching anything and returns an
 *    int status: GQ_OK or one of the GQ_E* codes below.  A rejected call launches nothing.
 *    Nothing is truncated silently: a reduction length that is not a whole number of blocks is
 *    an error, not a dropped tail.
 *  - After GQ_ECUDA, gq_last_cuda_error() returns the cudaError_t of the failed launch (per
 *    calling thread).
 *  - Decode kernels are launched as programmatic dependents of the work before them on the stream:
 *    they may start, and read their weights, before that work has finished, and they wait for it
 *    before they read an activation or write an output.  Weights must therefore not be written by
 *    the immediately preceding launch on the stream if that launch signals programmatic completion
 *    early (no launch of this library writes weights; an ordinary kernel or copy is waited for).
 *  - Kernels wait on nothing but their own asynchronous copies, and every such wait is bounded
 *    (about one second).  A wait that runs out sets a device-side error word and the kernel
 *    returns; gq_device_error() reads and clears it.
 *
 * Sources (page title, section) for the operations:
 *  [P1] browseml-gpu.js (browseML / bankML): header comment on the arithmetic; Q1_DOT_WGSL,
 *       Q1_MM_WGSL, Q1_MM4_WGSL; packQ1 / packQ8; gpuMatMul.
 *  [P2] kopitiam-gpu src/shaders/block_q8_matmul_nt.wgsl: header (bindings, PACKING,
 *       ACCUMULATION ORDER), fn quant_at, fn main.
 *  [P3] BonsaiのWebGPUカーネルを読み解く: the ternary P/N bitplane popcount identity; the
 *       decode / prefill kernel figure (q1_bits + q1_scales, binary-lut4-matmul LUT4 prefill,
 *       subgroup-matrix third path).
 */
#ifndef GQ_H
#define GQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* gq_stream_t;   /* the same type as cudaStream_t */

enum gq_status {
    GQ_OK = 0,
    GQ_EINVAL_SHAPE = 1,   /* a size is <= 0, too large, or not a whole number of blocks  */
    GQ_EINVAL_PTR = 2,     /* a required pointer is NULL or not aligned as documented     */
    GQ_EUNSUPPORTED = 3,   /* the requested path does not exist for this operation/shape  */
    GQ_ECUDA = 4           /* a CUDA launch failed; see gq_last_cuda_error()               */
};

enum gq_path {
    GQ_PATH_AUTO = 0,      /* the library picks by shape                                    */
    GQ_PATH_DP4A = 1,      /* integer dot products (dp4a) on the CUDA cores                 */
    GQ_PATH_LUT4 = 2,      /* 16-entry subset-sum tables per 4 activations, nibble lookups  */
    GQ_PATH_MMA = 3,       /* tcgen05 tensor-core MMA (kind::f16) with a fixed-order epilogue */
    GQ_PATH_FMA = 4        /* weights expanded to +-1.0 and multiply-added on the CUDA cores  */
};

/* Library version string (static storage). */
const char* gq_version(void);
/* Human-readable name of a status code (static storage). */
const char* gq_status_string(int status);
/* cudaError_t of the last failed launch on this host thread (0 if none). */
int gq_last_cuda_error(void);
/* Reads and clears the device-side error word of the current device: 0 if no kernel has
 * reported a timed-out wait since the last call, else a nonzero code.  Synchronizes the device. */
int gq_device_error(void);

/* ============================================================================================
 * Q1_0 weights x Q8_0 activations  [P1]
 *
 * Q1_0 block (18 bytes, the pages' storage): f16 d0 (little-endian) then 128 sign bits; weight
 * j = 32k + e of the block is bit e%8 of byte 2 + 4k + e/8 (bit 1 -> +q, bit 0 -> -q).
 * Q8_0 block (34 bytes): f16 d1 (little-endian) then 32 int8 quants.
 * A row of n weights is n/128 Q1_0 blocks; an activation vector of n values is n/32 Q8_0 blocks;
 * Q1_0 block i pairs with Q8_0 blocks 4i..4i+3.
 *
 * Result per (row, activation) -- the pages' exact operation order, reproduced bit for bit:
 *   per block i, sub-block k = 0..3, lane l = 0..7 (weights 4l..4l+3 of the sub-block):
 *     s = sum (bit ? q : -q), the negate wrapping as int8 (-(-128) = -128)
 *     p = d1 * s (exact), ab[l] = p (k = 0) or ab[l] + p (k > 0)   (round to nearest even)
 *     acc[l] = fma(d0, ab[l], acc[l])                                 (correctly rounded)
 *   y = ((acc0+acc4)+(acc2+acc6)) + ((acc1+acc5)+(acc3+acc7)), acc from +0.
 * ========================================================================================== */

/* Bytes of the packed (resident) form of a rows x n Q1_0 matrix; 0 if the shape is invalid. */
size_t gq_q1_0_packed_bytes(int rows, int n);

/* One-time repack of Q1_0 weights into the kernels' resident layout ([P1] packQ1: "repacked
 * once"; the engine keeps weights resident).
 *   raw_device    rows * (n/128) * 18 bytes, the pages' AoS blocks, row-major; any alignment.
 *   packed_device gq_q1_0_packed_bytes(rows, n) bytes, 16-byte aligned; fully written
 *                 (rows are padded to a multiple of 128 with zero blocks).
 * Layout (private to the library; treat as opaque): 128-row tiles; per (tile, block) a 2304-byte
 * chunk of 128 x 16 bytes of sign bits (bit-permuted within each 32-bit word) then 128 f16 d0.
 * Errors: GQ_EINVAL_SHAPE if rows < 1, n < 128, n % 128 != 0 or n > 2^20;
 *         GQ_EINVAL_PTR if a pointer is NULL or packed_device is not 16-byte aligned. */
int gq_q1_0_pack(const void* raw_device, int rows, int n, void* packed_device, gq_stream_t stream);

/* Bytes of workspace one decode GEMV needs for an activation of n values: the activation's
 * per-32-value constants (96 bytes per 32 values), built by the call itself, and a 16-byte tile
 * counter. */
size_t gq_q1_q8_workspace_bytes(int n);

/* Decode GEMV ([P1] Q1_DOT_WGSL semantics): y[r] for r < rows.
 *   packed_w_device from gq_q1_0_pack(rows, n); act_device: n/32 Q8_0 blocks (34 bytes each,
 *   2-byte aligned); y_device: rows f32; workspace_device: gq_q1_q8_workspace_bytes(n) bytes,
 *   16-byte aligned, which the call may overwrite.  A matrix with fewer 128-row tiles than the
 *   GPU has SMs takes one launch that builds the activation's constants itself and leaves the
 *   workspace untouched; a larger one takes two launches on `stream` (the constants into the
 *   workspace, then the GEMV, which hands 128-row tiles to its warps through a counter at the
 *   end of the workspace).  Calls that share a workspace must not overlap on the GPU.
 * Errors: as gq_q1_0_pack, plus GQ_EINVAL_PTR if act_device is odd, y_device not 4-aligned or
 * the workspace NULL or not 16-aligned. */
int q1_q8_gemv(const void* packed_w_device, const void* act_device, float* y_device,
               int rows, int n, void* workspace_device, gq_stream_t stream);

/* Activation formats of the decode GEMV (gq_gemv_desc.act_format). */
enum gq_act_format {
    GQ_ACT_Q8_0 = 0,       /* n/32 Q8_0 blocks of 34 bytes (f16 d, 32 int8), 2-byte aligned       */
    GQ_ACT_F32 = 1         /* n f32 values, 16-byte aligned, quantized to Q8_0 inside the call     */
};

/* The decode GEMV over f32 activations, with the Q8_0 quantization of the activations fused into
 * the GEMV's activation-constant step (no separate quantize launch, no Q8_0 round trip through
 * memory).  The result is bit-identical to gq_quantize_q8_0 on x followed by q1_q8_gemv: each
 * 32-block is quantized as that call states (d = f16(amax / 127), q = round half up of x / d
 * with the f32 d, clamped to [-127, 127]; an all-zero block gives d = 0, q = 0).  The pages do
 * not describe a decode-side quantizer; this is the reading of the prefill one.
 *   x_device: n f32, 16-byte aligned; other arguments and launches as q1_q8_gemv.
 * Errors: as q1_q8_gemv, with GQ_EINVAL_PTR if x_device is NULL or not 16-aligned. */
int q1_q8_gemv_f32(const void* packed_w_device, const float* x_device, float* y_device, int rows, int n,
                   void* workspace_device, gq_stream_t stream);

/* Decode GEMV on the pages' own bytes, with no repack of the weights ([P1] Q1_DOT_WGSL reads the
 * 18-byte Q1_0 blocks as stored): the same result as gq_q1_0_pack followed by q1_q8_gemv, bit for
 * bit, for callers that keep their weights in the pages' layout.  Slower than the resident layout
 * (its sign bits are looked up by nibble in tables of the block's exact products d1 * s, built per
 * thread block and 32 rows).
 *   w_q1_0_device: rows * (n/128) * 18 bytes, the pages' AoS blocks, row-major, 2-byte aligned;
 *   act_device: n/32 Q8_0 blocks (34 bytes), 2-byte aligned; y_device: rows f32, 4-byte aligned.
 *   One launch on `stream`; no workspace.
 * Errors: GQ_EINVAL_SHAPE if rows < 1, n < 128, n % 128 != 0 or n > 2^20; GQ_EINVAL_PTR for a
 * NULL or misaligned pointer; GQ_ECUDA. */
int q1_q8_gemv_raw(const void* w_q1_0_device, const void* act_device, float* y_device, int rows, int n,
                   gq_stream_t stream);

/* [P1] packQ8: `cols` activation vectors of n values, each n/32 Q8_0 blocks of 34 bytes (vector
 * after vector, 2-byte aligned), repacked into d_device[c * n/32 + b] = the block's f16 scale as f32
 * (exact) and q_device[(c * n/32 + b) * 8 + v] = its quant bytes 4v..4v+3 as one little-endian word
 * (both 4-byte aligned).  The library's GEMV and GEMM read the 34-byte blocks directly; this is the
 * pages' layout for callers that keep activations in it.
 * Errors: GQ_EINVAL_SHAPE if cols < 1, n < 32, n % 32 != 0 or n > 2^20; GQ_EINVAL_PTR; GQ_ECUDA. */
int gq_pack_q8_0(const void* raw_q8_0_device, int cols, int n, float* d_device, uint32_t* q_device,
                 gq_stream_t stream);

/* Largest n that q1_q8_gemv_noalloc accepts. */
#define GQ_NOALLOC_MAX_N 16384

/* The decode GEMV for callers that cannot allocate device memory (code running inside another
 * allocator's arena, plugins handed raw pointers, paths where an allocation could block or fail):
 * the same result as q1_q8_gemv, bit for bit, with the workspace taken from a fixed block of
 * device memory built into the library (about 48 KB, held by every GPU that loads the library
 * until the process exits).  The pages describe no such variant.
 *   Arguments as q1_q8_gemv without the workspace; n <= GQ_NOALLOC_MAX_N.
 *   The first call on each device looks up that block's address (cudaGetSymbolAddress, with the
 *   device current) and keeps it: make that first call before any stream capture on the device,
 *   and do not reset the device (cudaDeviceReset) between calls.
 *   Every call shares the block, so calls whose work overlaps on the GPU (other streams, other
 *   host threads) race: issue them one after another.  The call itself clears what must start
 *   at zero.  It calls no allocator (no cudaMalloc / cudaFree, no library that allocates).
 * Errors: GQ_EINVAL_SHAPE for rows < 1, n < 128, n % 128 != 0 or n > GQ_NOALLOC_MAX_N;
 *         GQ_EINVAL_PTR as q1_q8_gemv; GQ_ECUDA if the address lookup or a launch fails. */
int q1_q8_gemv_noalloc(const void* packed_w_device, const void* act_device, float* y_device, int rows,
                       int n, gq_stream_t stream);

/* One matrix of a grouped GEMV sweep (all fields filled by the caller except tile_begin). */
typedef struct gq_gemv_desc {
    const void* packed_w;    /* device, from gq_q1_0_pack(rows, n)                      */
    const void* act;         /* device, n/32 Q8_0 blocks, or n f32 (act_format)         */
    float* y;                /* device, rows f32                                        */
    void* workspace;         /* device, gq_q1_q8_workspace_bytes(n), 16-aligned, its own */
    int rows;
    int n;
    int tile_begin;          /* filled by gq_gemv_group_plan                            */
    int act_format;          /* GQ_ACT_Q8_0 (0) or GQ_ACT_F32 (quantized in the call)   */
} gq_gemv_desc;

/* Host-side planning for q1_q8_gemv_grouped: validates every descriptor (host array), sorts the
 * array by n, largest first (stable; each entry keeps its own pointers, so results are
 * unaffected), and fills tile_begin (a prefix sum of 128-row tiles).  *total_tiles receives the
 * number of tiles of the whole group.
 * Errors: GQ_EINVAL_SHAPE / GQ_EINVAL_PTR as q1_q8_gemv for the first bad descriptor (the array
 * is then left unsorted), or GQ_EINVAL_SHAPE if count < 1, count > 65535 or the group exceeds
 * 2^31-1 tiles. */
int gq_gemv_group_plan(gq_gemv_desc* descs_host, int count, int* total_tiles);

/* Grouped decode GEMV: every matrix of a layer stack (e.g. one decode token's sweep) in two
 * launches (all activations' constants, then one persistent GEMV over every tile of the group,
 * which hands 128-row tiles to warps through *counter_device, largest matrix first).
 * descs_device is a device copy of the planned array (count entries, 8-byte aligned);
 * total_tiles is the value gq_gemv_group_plan returned; counter_device is one int of device
 * memory (4-aligned) that the call resets and uses -- calls sharing it, or sharing a
 * descriptor's workspace, must not overlap on the GPU.  Results are bit-identical to calling
 * q1_q8_gemv on each entry.  The host cannot re-validate device descriptors: pass only arrays
 * that gq_gemv_group_plan accepted, unchanged. */
int q1_q8_gemv_grouped(const gq_gemv_desc* descs_device, int count, int total_tiles, int* counter_device,
                       gq_stream_t stream);

/* Bonsai 1-bit weights times f32 activations ([P3] decode/prefill figure: the decode kernel
 * llama-decode-q1-proj.wgsl and the prefill kernel binary-lut4-matmul.wgsl):
 *   y[m * N + n] = sum_b wscale[n * K/32 + b] * sum_t s(n, 32 b + t) * x[m * K + 32 b + t]
 * with s = +1.0 where bit t of signs[n * K/32 + b] is set, -1.0 where it is clear (the same
 * weight arrays as q1s32_q8_gemm).  The page does not fix the order of the float operations, so
 * neither path is defined bit for bit; each result lies within c * 2^-24 * sum_b |wscale| *
 * sum_t |x| of the exact value, c = 32 + ceil(nb/8) for LUT4 at M <= 4 with K % 128 == 0,
 * c = 12 + nb for the other LUT4 cases and c = 40 + ceil(nb/32) for FMA (nb = K/32).  Results are
 * deterministic: the same inputs and path give the same bits on every call.
 *   path GQ_PATH_FMA: the decode formulation -- signs expanded to +-1, each block summed in
 *        order, acc = fma(scale, block_sum, acc), lanes added by a butterfly.
 *   path GQ_PATH_LUT4: per token and 4 activations a table of the 16 signed sums, indexed by the
 *        weight nibble; block sum = the 8 lookups in order; acc = fma(scale, block_sum, acc).
 *   path GQ_PATH_AUTO: LUT4.
 *   signs_device: N * K/32 u32; wscale_device: N * K/32 f32 (both 4-byte aligned; rows that
 *   start on 16 bytes are read with 16-byte loads); x_device: M * K f32, 16-byte aligned;
 *   y_device: M * N f32, 4-byte aligned.  One launch on `stream`; no workspace.
 * Errors: GQ_EINVAL_SHAPE unless N >= 1, 1 <= M <= 65535, 32 <= K <= 65536 and K % 32 == 0;
 *         GQ_EUNSUPPORTED for another path; GQ_EINVAL_PTR for a NULL or misaligned pointer;
 *         GQ_ECUDA. */
int q1s32_f32_gemm(const uint32_t* signs_device, const float* wscale_device, const float* x_device,
                   float* y_device, int M, int N, int K, int path, gq_stream_t stream);

/* q1s32_f32_gemm on the tensor cores (the prefill path; same operation and weight arrays).  The
 * activations are split exactly into three bf16 parts (hi = bf16(x), mid = bf16(x - hi),
 * lo = bf16(x - hi - mid), each rounded to nearest; hi + mid + lo = x for normal x) in the
 * workspace; the tensor cores form each 32-block's p = sum_t s * x (the +-1 weights are exact in
 * bf16), and acc = fma(wscale, p, acc) runs in block order.  The result lies within
 * c * 2^-24 * sum_b |wscale| * sum_t |x| of the exact value with c = nb + 16 (nb = K/32: one fma
 * per block, two units for each of the six tensor-core steps of a block, whose f32 accumulation
 * rounding is not published), and the same inputs give the same bits on every call.
 *   workspace_device: gq_q1s32_mma_workspace_bytes(M, K) bytes (3 * M * K bf16), 16-byte aligned,
 *   overwritten; signs_device 16-byte and wscale_device 8-byte aligned; x_device 4-byte aligned.
 *   Two launches on `stream` (the split, then the prefill MMA kernel).
 * Errors: GQ_EINVAL_SHAPE unless N >= 1, 1 <= M <= 65535 * 128, 64 <= K <= 65536 and K % 64 == 0;
 *         GQ_EINVAL_PTR for a NULL or misaligned pointer; GQ_ECUDA. */
size_t gq_q1s32_mma_workspace_bytes(int M, int K);     /* 0 for an invalid shape */
int q1s32_f32_gemm_mma(const uint32_t* signs_device, const float* wscale_device, const float* x_device,
                       float* y_device, int M, int N, int K, void* workspace_device, gq_stream_t stream);

/* Block-quantized weights times f32 activations (web-xpu-ops README: the op table rows
 * matvecQ8 / matmulQ8 and matvecQ4G128 / matmulQ4G128, and "The q4 format"):
 *   matvec_q8 / matmul_q8 (W8A32, per-row scale):
 *     code k of row n = byte (k % 4) of w[n * K/4 + k/4], least-significant byte first, signed;
 *     y[t * N + n] = scale[n] * sum_k code(n, k) * x[t * K + k].
 *   matvec_q4g128 / matmul_q4g128 (W4A32, one scale per 128 columns):
 *     code k of row n = nibble (k % 8) of w[n * K/8 + k/8], least-significant nibble first,
 *     4-bit two's complement (the page's quantizer emits [-7, 7]; a raw 0x8 reads as -8);
 *     y[t * N + n] = sum_g scale[n * ceil(K/128) + g] * sum_{k in g} code(n, k) * x[t * K + k].
 * The matvec is the matmul with T = 1.  The page fixes no float order, so the results are not
 * defined bit for bit; each lies within c * 2^-24 * sum |scale * code * x| of the exact value
 * (T <= 4: c = 16 * ceil(K/4096) + 10 for 8 bits, c = 28 + ceil(K/512) for 4 bits; T > 4:
 * c = K + 2), and the same inputs give the same bits on every call.
 *   w_device: N * K/4 (8 bits) or N * K/8 (4 bits) u32, 16-byte aligned; scale_device: N (8 bits)
 *   or N * ceil(K/128) (4 bits) f32; x_device: T * K f32, 16-byte aligned; y_device: T * N f32.
 *   One launch on `stream`; no workspace.
 * Errors: GQ_EINVAL_SHAPE unless N >= 1, 1 <= T <= 65535 * 128, 32 <= K <= 65536 and
 *         K % 32 == 0; GQ_EINVAL_PTR for a NULL or misaligned pointer; GQ_ECUDA. */
int matvec_q8(const uint32_t* w_device, const float* scale_device, const float* x_device, float* y_device,
              int N, int K, gq_stream_t stream);
int matmul_q8(const uint32_t* w_device, const float* scale_device, const float* x_device, float* y_device,
              int T, int N, int K, gq_stream_t stream);
int matvec_q4g128(const uint32_t* w_device, const float* scale_device, const float* x_device, float* y_device,
                  int N, int K, gq_stream_t stream);
int matmul_q4g128(const uint32_t* w_device, const float* scale_device, const float* x_device, float* y_device,
                  int T, int N, int K, gq_stream_t stream);

/* matmul_q8 / matmul_q4g128 on the tensor cores (same operations and code layouts as above).  Each
 * activation x is split exactly into three bf16 parts (hi = bf16(x), mid = bf16(x - hi),
 * lo = bf16(x - hi - mid), each rounded to nearest; hi + mid + lo == x for normal x), the int8
 * codes are exact in bf16, and the tensor cores accumulate the code * part products of one
 * 128-column round (three parts x 128 columns) into an f32 partial; 8 bits: the partials are added
 * in f32 with round to nearest, round after round, and y = scale[n] * sum; 4 bits: acc =
 * fma(scale[n, g], partial, acc) round after round (round g is group g), y = acc.  The result lies
 * within c * 2^-24 * sum |scale * code * x| of the exact value with c = ceil(K/128) + 56 (two units
 * per tensor-core step, whose f32 accumulation rounding is not published), and the same inputs
 * give the same bits on every call.  Activations below 2^-126 * 2^16 in magnitude may lose their lowest bits
 * (the residual planes are bf16, whose exponent range is f32's).
 *   workspace_device: gq_wq_mma_workspace_bytes(T, K) bytes (3 * T * K bf16), 16-byte aligned,
 *   overwritten; the other arguments as matmul_q8 / matmul_q4g128.  Two launches on `stream` (the split, then the
 *   tensor-core kernel).
 * Errors: GQ_EINVAL_SHAPE unless N >= 1, 1 <= T <= 65535 * 128, 64 <= K <= 65536 and K % 32 == 0;
 *         GQ_EINVAL_PTR for a NULL or misaligned pointer; GQ_ECUDA. */
size_t gq_wq_mma_workspace_bytes(int T, int K);     /* 0 for an invalid shape */
int matmul_q8_mma(const uint32_t* w_device, const float* scale_device, const float* x_device, float* y_device,
                  int T, int N, int K, void* workspace_device, gq_stream_t stream);
int matmul_q4g128_mma(const uint32_t* w_device, const float* scale_device, const float* x_device, float* y_device,
                      int T, int N, int K, void* workspace_device, gq_stream_t stream);

/* Prefill GEMM over `cols` Q8_0 activation vectors ([P1] Q1_MM_WGSL / Q1_MM4_WGSL): every
 * (row, column) is the GEMV chain above, stored at y[c * rows + r].
 *   act_device: cols * (n/32) Q8_0 blocks, column after column (2-byte aligned).
 *   path: GQ_PATH_DP4A, GQ_PATH_LUT4 or GQ_PATH_AUTO (DP4A); GQ_PATH_MMA -> GQ_EUNSUPPORTED
 *         (the per-4-weight lane sums of this format leave a tensor core nothing dense to do).
 * Errors: as q1_q8_gemv, plus GQ_EINVAL_SHAPE if cols < 1. */
int q1_q8_gemm(const void* packed_w_device, const void* act_device, float* y_device,
               int rows, int n, int cols, int path, gq_stream_t stream);

/* ============================================================================================
 * block_q8_matmul_nt  [P2]:  y = x . w^T with w block-scaled int8.
 *   x_device      [m, k] f32 row-major (4-byte aligned)
 *   quants_device k*n int8 packed four per u32, little-endian: element t of weight row `col` is
 *                 byte (t%4) of word (col*k + t)/4, sign-extended (16-byte aligned)
 *   scales_device [n, k/32] f32
 *   y_device      [m, n] f32 row-major
 * Order (bit for bit): per (row, col), for block b ascending: block_sum = 0; for t < 32:
 * block_sum = block_sum + x*q (a rounded multiply, then a rounded add); acc = acc +
 * scale*block_sum (the same); acc from +0.
 * Errors: GQ_EINVAL_SHAPE if m, k or n < 1, k % 32 != 0, k > 65536 or m > 65535;
 *         GQ_EINVAL_PTR for NULL or misaligned pointers. */
int block_q8_matmul_nt(const float* x_device, const uint32_t* quants_device,
                       const float* scales_device, float* y_device, int m, int k, int n,
                       gq_stream_t stream);

/* ============================================================================================
 * Ternary bitplane GEMV  [P3]:  weights w in {-1, 0, +1} as bitplanes P (w = +1) and N (w = -1),
 * activations binarized to a bitplane X (bit 1 -> +1, bit 0 -> -1); bit j of word v is element
 * 32v + j.  Per (batch b, row r), exactly:
 *   y = 2 * (sum popc(P & X) - sum popc(N & X)) - sum popc(P) + sum popc(N).
 * A position with both P and N set counts as weight 0.
 *   P_device, N_device [rows, k/32] u32 (16-byte aligned); X_device [batch, k/32] u32
 *   (16-byte aligned); y_device [batch, rows] int32.
 * Errors: GQ_EINVAL_SHAPE if rows or batch < 1, k < 1024, k % 1024 != 0 (tiles of 32 words),
 *         k > 65536 or batch > 64;
 *         GQ_EINVAL_PTR for NULL or misaligned pointers. */
int ternary_bitplane_gemv(const uint32_t* P_device, const uint32_t* N_device,
                          const uint32_t* X_device, int32_t* y_device, int rows, int k,
                          int batch, gq_stream_t stream);

/* ============================================================================================
 * Batched prefill with Bonsai-format 1-bit weights  [P3] and Q8_0 activations.
 *
 * Activation quantizer (the pages give none for Q8_0 blocks; the reading is stated here):
 * per 32-block of a row of x, amax = max |x|; d = amax / 127 (round to nearest); the stored
 * scale is f16(d) rounded to nearest even; q = clamp(floor(v) + (v - floor(v) >= 0.5), -127,
 * 127) with v = x / d (round to nearest, the f32 d); amax == 0 gives d = 0 and q = 0.
 *   x_device [m, k] f32; d_device [m, k/32] f16 bits; q_device [m, k] int8 (16-byte aligned);
 *   mma_operand_device: NULL, or [3, m, k] bf16 (16-byte aligned) receiving the operand
 *   q1s32_q8_gemm's MMA path reads: pv = f16(d) * q (exact) split into three bf16 parts,
 *   hi = bf16(pv), mid = bf16(pv - hi), lo = bf16(pv - hi - mid) (each rounded to nearest, so
 *   hi + mid + lo = pv), plane p at offset p * m * k, with the elements of each 32-block
 *   interleaved (position 2u <- element u, 2u+1 <- element u+16).
 * Errors: GQ_EINVAL_SHAPE if m or k < 1, k % 32 != 0 or k > 65536; GQ_EINVAL_PTR. */
int gq_quantize_q8_0(const float* x_device, int m, int k, uint16_t* d_device, int8_t* q_device,
                     uint16_t* mma_operand_device, gq_stream_t stream);

/* Prefill GEMM: y[m, n] = sum over 32-blocks b ascending of
 *     S = sum_t (sign bit ? q : -q) (int8-wrapping negate), p = f16(xd[m,b]) * S (exact),
 *     acc = fma(w_scale[n, b], p, acc) (correctly rounded), acc from +0.
 *   signs_device   [N, K/32] u32, bit t of word b = weight 32b+t, 1 -> +1 (16-byte aligned)
 *   wscale_device  [N, K/32] f32 (4-byte aligned; 8-byte aligned for GQ_PATH_MMA)
 *   xd_device      [M, K/32] f16 bits (4-byte aligned), xq_device [M, K] int8 (16-byte aligned)
 *   xq_mma_device  the three-plane bf16 operand from gq_quantize_q8_0 (required for
 *                  GQ_PATH_MMA, else may be NULL), made from the same d and q as xd_device and
 *                  xq_device, all q in [-127, 127] (as the quantizer produces).  The tensor
 *                  cores form p = f16(d) * S itself: every term and partial sum is a multiple of
 *                  the ulp of f16(d) below 2^12 f16(d), so its f32 accumulation is exact.
 *   y_device       [M, N] f32 row-major
 *   path: GQ_PATH_LUT4, GQ_PATH_MMA, or GQ_PATH_AUTO (MMA when M >= 64 and the operand is
 *   given, else LUT4).  Both paths are bit-identical to the order above.
 * Errors: GQ_EINVAL_SHAPE if M, N or K < 1, K % 64 != 0 or K > 65536; GQ_EUNSUPPORTED for an
 * unknown path or GQ_PATH_DP4A; GQ_EINVAL_PTR for NULL/misaligned pointers (xq_mma_device NULL
 * with GQ_PATH_MMA included). */
int q1s32_q8_gemm(const uint32_t* signs_device, const float* wscale_device,
                  const uint16_t* xd_device, const int8_t* xq_device,
                  const uint16_t* xq_mma_device, float* y_device, int M, int N, int K, int path,
                  gq_stream_t stream);

/* ============================================================================================
 * Between a layer's products: RMS norm into Q8_0, rotary positions, a paged Q8_0 key/value cache, and
 * attention over it.  Inputs and outputs are f32, f16 or bf16 (one type per call); every sum, norm,
 * softmax statistic and rotation is formed in f32 whatever the type, and rounded once on the store.
 * Kernels whose indices come from device memory check them: an index out of its range is skipped as
 * stated at the call and sets GQ_DEVERR_INDEX in the device error word (gq_device_error).
 * ========================================================================================== */

enum gq_dtype { GQ_F32 = 0, GQ_F16 = 1, GQ_BF16 = 2 };

#define GQ_DEVERR_INDEX 8   /* bit of gq_device_error(): an index read from device memory was out of range */

/* RMS norm with the residual's addition, and an output in Q8_0:
 *   h = x + r (r = 0 if residual_device is NULL), y_i = (h_i * (1 / sqrt(sum h^2 / k + eps))) * w_i, each step
 *   rounded to f32 (the sum's order is not stated).
 *   x_device [m, k] of `type`, rows x_stride elements apart (x_stride >= k); residual_device NULL or
 *   [m, k], rows residual_stride apart; weight_device k f32.  Any output may be NULL, not all of them:
 *     sum_device  [m, k] of `type`, contiguous: h; it may be x_device or residual_device itself if
 *                 those rows are contiguous (each row is read before it is written);
 *     y_device    [m, k] of `type`, contiguous;
 *     act_device  m * k/32 Q8_0 blocks of 34 bytes (2-byte aligned), as the Q1_0 GEMV and GEMM take them;
 *     d_device, q_device, mma_operand_device: the split form, as gq_quantize_q8_0 writes it (both of
 *                 d and q or neither; q and the operand 16-byte aligned; the operand only beside them).
 *   y is quantized in f32, before any rounding to `type`, by the rule stated at gq_quantize_q8_0.  Two
 *   calls on the same inputs give the same bits.
 * Errors: GQ_EINVAL_SHAPE if m < 1, k < 1, k > 65536, a stride < k, or a Q8_0 output with k % 32 != 0;
 *         GQ_EUNSUPPORTED for another type; GQ_EINVAL_PTR (elements aligned to their size, weight to 4
 *         bytes, or no output at all); GQ_ECUDA.  eps must be >= 0 (else GQ_EINVAL_SHAPE). */
int gq_rmsnorm(const void* x_device, long long x_stride, const void* residual_device, long long residual_stride,
               const float* weight_device, float eps, int type, int m, int k, void* sum_device, void* y_device,
               void* act_device, uint16_t* d_device, int8_t* q_device, uint16_t* mma_operand_device,
               gq_stream_t stream);

/* The values code * d of Q8_0 blocks (34 bytes, 2-byte aligned), `blocks` of them one after another,
 * as 32 values of `type` each (16-byte aligned).
 * Errors: GQ_EINVAL_SHAPE unless 1 <= blocks <= 2^40, GQ_EUNSUPPORTED for another type, GQ_EINVAL_PTR, GQ_ECUDA. */
int gq_dequantize_q8_0(const void* act_device, long long blocks, int type, void* out_device, gq_stream_t stream);

/* The key/value cache: `pages` pages of page_size token slots for kv_heads heads of head_dim; slot s is
 * place s % page_size of page s / page_size.  Keys and values are Q8_0: per slot, head and 32 dims an
 * f16 scale d and 32 codes q in [-127, 127] (rule: gq_quantize_q8_0; value = q * d).  A code is stored
 * as sign bit and 7-bit magnitude.  [page][head][16 slots] is one chunk of 34 * head_dim bytes:
 *   K codes 16 * hd | V codes 16 * hd | K scales 16 * hd/32 f16 | V scales 16 * hd/32 f16.
 * With tok the place in the 16, d the dim, t = (tok & 7) >> 1, p = (tok & 1) + 2 * (tok >> 3), byte offsets:
 *   K code  tok * hd + 16 * u + 4 * ((d >> 4) & 3) + (d & 3), u = 4 * (d >> 6) + ((d >> 2) & 3),
 *           with bit 2 of u flipped where hd > 64 and tok is odd;
 *   V code  hd = 64:  (4 p + t) * 64 + 8 * (g ^ (4 * (t >> 1))) + 4 * (d >> 5) + (d & 3),   g = (d >> 2) & 7;
 *           hd > 64:  (4 p + t) * hd + 128 * (d >> 7) + 16 * (g ^ (2 t)) + 4 * ((d >> 5) & 3) + (d & 3);
 *   scales  2 * ((4 t + p) * hd/32 + (d >> 5)).
 * (A warp's 16-byte shared-memory reads of this order give its matrix fragments directly, without bank
 * conflicts, and a token's codes stay together.)  A slot never written need not be initialised: nothing of it reaches
 * a result.  kv_heads 1 to 1024, head_dim 64, 128 or 256, page_size a multiple of 16 up to 65536,
 * pages * page_size < 2^40.  0 for an invalid shape. */
size_t gq_kv_cache_bytes(int pages, int page_size, int kv_heads, int head_dim);

/* Rotary frequencies scaled for long contexts (gq_rope_table). */
enum gq_rope_scaling {
    GQ_ROPE_PLAIN = 0,     /* f_i = base^(-2i/rot)                                                       */
    GQ_ROPE_LINEAR = 1,    /* f_i / factor                                                               */
    GQ_ROPE_NTK = 2,       /* base * factor^(rot / (rot - 2)) in the place of base                       */
    GQ_ROPE_YARN = 3       /* f_i * (r_i + (1 - r_i) / factor) with r_i = 1 - clamp((i - low) / (high - low), 0, 1);
                              low = floor(c(32)), high = ceil(c(1)), both clamped to [0, rot - 1],
                              high = low + 0.001 where they are equal,
                              c(n) = rot * ln(original / (2 pi n)) / (2 ln base); cos and sin are multiplied
                              by 1 + 0.1 ln(factor)                                                       */
};

/* cos and sin of every position's rotary angles, formed in 64 bits and rounded to f32 once:
 *   table_device [positions, rot/2, 2] f32 (8-byte aligned): cos, sin of position * f_i.
 * Errors: GQ_EINVAL_SHAPE unless positions >= 1, rot is a multiple of 8 in [8, 256], base > 1, factor >= 1 and
 *         (yarn) original >= 1; GQ_EUNSUPPORTED for another scaling; GQ_EINVAL_PTR; GQ_ECUDA. */
int gq_rope_table(float* table_device, int positions, int rot, double base, int scaling, double factor,
                  double original, gq_stream_t stream);

/* Pairs that a rotation turns: element i with i + rot/2 (half), or 2i with 2i + 1 (interleaved). */
enum gq_rope_layout { GQ_ROPE_HALF = 0, GQ_ROPE_INTERLEAVED = 1 };

/* Rotary positions on the first `rot` dims of every q and k head, and the append of k and v to the cache:
 *   (a, b) -> (a * cos - b * sin, b * cos + a * sin) for pair i of token n, cos and sin from row
 *   positions_device[n] of rope_device ([rope_rows, rot/2, 2] f32; NULL or rot = 0: no rotation).
 *   q_device [tokens, q_heads, head_dim] -> q_out_device of the same shape and `type` (it may be q_device
 *   itself, with the same stride); both NULL where q_heads = 0.  k_device, v_device [tokens, kv_heads, head_dim];
 *   heads are contiguous, tokens the given strides (in elements) apart, so that one fused q | k | v row serves.
 *   slots_device[n] (int64): where token n goes; a negative one is not written.  Two tokens with one slot in
 *   a call leave that slot unspecified: words of both may be mixed there, a code of one beside a scale of the other, and not
 *   the same ones every time.  Other slots are as they should be.
 *   A position outside [0, rope_rows) leaves that token's q_out and slot unwritten, a slot >= pages * page_size
 *   is not written; both set GQ_DEVERR_INDEX.
 *   k is quantized after the rotation, in f32.
 * Errors: GQ_EINVAL_SHAPE unless tokens >= 1, q_heads in [0, 1024], a valid cache shape, rot a multiple of 8 in [0, head_dim],
 *         strides >= the heads' width and rope_rows >= 1 with rot > 0; GQ_EUNSUPPORTED for another type
 *         or layout; GQ_EINVAL_PTR for NULL pointers, elements or strides not aligned to 4 elements, cache or rope not
 *         aligned to 16 bytes; GQ_ECUDA. */
int gq_rope_kv_append(const void* q_device, long long q_stride, void* q_out_device, long long q_out_stride,
                      const void* k_device, long long k_stride, const void* v_device, long long v_stride, int type,
                      const float* rope_device, int rope_rows, int rot, int layout, const int32_t* positions_device,
                      const int64_t* slots_device, int tokens, int q_heads, int kv_heads, int head_dim,
                      void* cache_device, int pages, int page_size, gq_stream_t stream);

/* Reads slots back: k_out_device, v_out_device [n, kv_heads, head_dim] of `type` (16-byte aligned; either may be
 * NULL) = code * d.  A negative slot gives zeros; one >= pages * page_size too, and sets GQ_DEVERR_INDEX.
 * Errors: GQ_EINVAL_SHAPE unless n >= 1 and the cache shape is valid; GQ_EUNSUPPORTED; GQ_EINVAL_PTR; GQ_ECUDA. */
int gq_kv_read(const void* cache_device, int pages, int page_size, int kv_heads, int head_dim,
               const int64_t* slots_device, int n, int type, void* k_out_device, void* v_out_device,
               gq_stream_t stream);

/* Attention of each sequence's newest tokens over its cached ones (themselves included: append first):
 *   s = scale * (q . k), capped to softcap * tanh(s / softcap) where softcap > 0; o = softmax(s) . v over the
 *   visible keys, 0 where none is visible.  Query head h reads kv head h / (q_heads / kv_heads).
 *   Sequence b has kv_len_device[b] cached tokens, token j in place j % page_size of page
 *   block_table_device[b * table_stride + j / page_size], and T = q_start_device[b + 1] - q_start_device[b] query tokens,
 *   rows q_start_device[b].. of q_device and out_device ([q_start_device[seqs], q_heads, head_dim] of `type`, tokens
 *   q_stride / out_stride elements apart).  Query i of them stands at token L - T + i.
 *   Keys before L - T are visible to every query; of the newest T, key j is visible to query i if
 *     tree_mask_device is NULL: j <= i (causal);
 *     else: bit j of tree_mask_device[row of query i] is set (its drafted ancestors and itself; T <= 64).
 *   T > L is allowed (the first queries then see nothing, and give 0), T = 0 and L = 0 too.
 *   T * (q_heads / kv_heads) * L of a sequence stays below 2^44.
 *   max_q and max_kv bound T and L of every sequence; a longer T or L, or a page index outside
 *   [0, pages), sets GQ_DEVERR_INDEX: what is past the bound is not computed or not seen.
 *   Row numbers are checked against [0, rows): gq_attn_q8_0_bounded is told how many rows q_device, out_device and
 *   tree_mask_device have, gq_attn_q8_0 takes q_start_device[seqs] for it (which must then be right).  A sequence that begins
 *   outside, or ends before it begins, is left out, of one that ends past it the rows inside are computed (each at its place
 *   L - T + i); both set GQ_DEVERR_INDEX.
 *   workspace_device: gq_attn_workspace_bytes(...) bytes, 16-byte aligned, overwritten; calls that
 *   share it must not overlap on the GPU.  Nothing of it is kept between calls.  Results do not depend on
 *   timing: the same inputs give the same bits.
 * Precision: sums and statistics are in f32, codes are exact.  f32 queries take two f16 parts after a row's scaling by a
 * power of two, and the softmax's numerators three bf16 parts; f16 and bf16 queries take one f16 part of both, the numerators
 * times the values' scales (off by up to 2^-40 of a row's largest such product besides their 11 bits).  From 256 (f32) or 128
 * (f16, bf16) rows a kv head on (max_q * q_heads / kv_heads; head_dim 64 and 128) keys, values and numerators take two f16 parts
 * (one): a numerator is off by up to 2^-36 of its row's largest besides its 22 (11) bits, a key or value by 2^-22 of its token's
 * largest, and a row that sees a value whose scale is not finite is NaN.  Where the scales of 64 neighbouring tokens differ by
 * more than 2^12, 2^-36 is of the row's largest product of a numerator and its token's largest scale.  What a token that a row does
 * not see holds does not matter to any of this.
 * Errors: GQ_EINVAL_SHAPE unless 1 <= seqs <= 65535, max_q >= 1, max_kv >= 1, q_heads a multiple of kv_heads with
 *         q_heads / kv_heads <= 64, a valid cache shape, strides >= q_heads * head_dim, table_stride >=
 *         ceil(max_kv / page_size), scale finite, softcap >= 0 and finite, and max_q <= 64 with tree_mask_device;
 *         GQ_EUNSUPPORTED for another type; GQ_EINVAL_PTR for NULL pointers, or elements and strides of q and out not
 *         aligned to 4 elements, cache or workspace not to 16 bytes; GQ_ECUDA. */
size_t gq_attn_workspace_bytes(int seqs, int max_q, int q_heads, int kv_heads, int head_dim, int type);  /* 0: invalid */
int gq_attn_q8_0(const void* q_device, long long q_stride, void* out_device, long long out_stride, int type,
                 const void* cache_device, int pages, int page_size, const int32_t* block_table_device,
                 int table_stride, const int32_t* kv_len_device, const int32_t* q_start_device,
                 const uint64_t* tree_mask_device, int seqs, int max_q, int max_kv, int q_heads, int kv_heads,
                 int head_dim, float scale, float softcap, void* workspace_device, gq_stream_t stream);
/* gq_attn_q8_0 with the number of rows given.  Errors: also GQ_EINVAL_SHAPE if rows < 0. */
int gq_attn_q8_0_bounded(const void* q_device, long long q_stride, void* out_device, long long out_stride, int type,
                         const void* cache_device, int pages, int page_size, const int32_t* block_table_device,
                         int table_stride, const int32_t* kv_len_device, const int32_t* q_start_device,
                         const uint64_t* tree_mask_device, int rows, int seqs, int max_q, int max_kv, int q_heads,
                         int kv_heads, int head_dim, float scale, float softcap, void* workspace_device,
                         gq_stream_t stream);

/* ============================================================================================
 * Roofline probes (measurement only; no hot-path entry point uses them).  The machine's own
 * ceilings, measured in the same session as the kernels whose fractions are quoted against them:
 * roofline.html's read-only bandwidth method (FILL a buffer with a non-zero pattern, then read it
 * with every load live, best of five after a warm-up) and the web-xpu-ops README's "Performance,
 * measured against the machine's own ceiling".
 * ========================================================================================== */

/* Number of SMs of the current device, or -1. */
int gq_probe_sm_count(void);

/* Writes a non-zero pattern derived from `seed` over `bytes` (a multiple of 16) of buf_device
 * (16-byte aligned).  One launch on `stream`.
 * Errors: GQ_EINVAL_SHAPE, GQ_EINVAL_PTR, GQ_ECUDA. */
int gq_probe_fill(void* buf_device, size_t bytes, uint32_t seed, gq_stream_t stream);

/* One read-only pass over `bytes` of buf_device with 16-byte loads that bypass L1 (eight in
 * flight per thread, grid-stride over blocks_per_sm x SMs blocks of `threads` threads), XOR of
 * everything read folded into *sink_device (one u32, 4-byte aligned, which the caller zeroes).
 * The caller times the launch; bytes / time is the read bandwidth.  Use a buffer several times
 * the L2 size.  Errors: GQ_EINVAL_SHAPE unless bytes is a positive multiple of 16,
 * 1 <= blocks_per_sm <= 32 and threads is a multiple of 32 in [32, 1024]; GQ_EINVAL_PTR. */
int gq_probe_read(const void* buf_device, size_t bytes, uint32_t* sink_device, int blocks_per_sm, int threads,
                  gq_stream_t stream);

/* Instruction kinds of gq_probe_issue: one kind alone, or two interleaved one to one. */
enum gq_probe_kind {
    GQ_PROBE_FFMA = 0,          /* fma.rn.f32                              */
    GQ_PROBE_FFMA2 = 1,         /* fma.rn.f32x2                            */
    GQ_PROBE_FADD2 = 2,         /* add.rn.f32x2                            */
    GQ_PROBE_FADD = 3,          /* add.rn.f32                              */
    GQ_PROBE_DP4A = 4,          /* dp4a.u32.s32                            */
    GQ_PROBE_LOP3 = 5,          /* lop3.b32                                */
    GQ_PROBE_POPC = 6,          /* popc.b32                                */
    GQ_PROBE_PRMT = 7,          /* prmt.b32                                */
    GQ_PROBE_SHF = 8,           /* shf.l.wrap.b32                          */
    GQ_PROBE_IMAD = 9,          /* mad.lo.u32                              */
    GQ_PROBE_SHFL = 10,         /* shfl.sync.idx.b32                       */
    GQ_PROBE_LDS = 11,          /* ld.shared.u32, conflict-free (+ one lop3 each) */
    GQ_PROBE_DP4A_FFMA2 = 12,   /* dp4a and fma.rn.f32x2 interleaved       */
    GQ_PROBE_LDS_SHFL = 13,     /* ld.shared.u32 and shfl.sync interleaved */
    GQ_PROBE_FFMA_FFMA2 = 14,   /* fma.rn.f32 and fma.rn.f32x2 interleaved */
    GQ_PROBE_LOP3_DP4A = 15,    /* lop3 and dp4a interleaved               */
    GQ_PROBE_FADD_FFMA2 = 16,   /* add.rn.f32 and fma.rn.f32x2 interleaved */
    GQ_PROBE_LOP3_FFMA2 = 17,   /* lop3 and fma.rn.f32x2 interleaved       */
    GQ_PROBE_HMMA_F16 = 18,     /* mma.sync m16n8k16 f16 x f16 + f32 (4096 flop each)  */
    GQ_PROBE_HMMA_BF16 = 19,    /* mma.sync m16n8k16 bf16 x bf16 + f32 (4096 flop)     */
    GQ_PROBE_QMMA_E4M3 = 20,    /* mma.sync m16n8k32 e4m3 x e4m3 + f32 (8192 flop),
                                   operand conversion included                          */
    GQ_PROBE_IMMA_S8 = 21,      /* mma.sync m16n8k32 s8 x s8 + s32 (8192 op)           */
    GQ_PROBE_HMMA_MIX = 22,     /* f16 mma.sync : lop3 : lop3 : fma.rn.f32, 1:2:1      */
    GQ_PROBE_QMMA_MIX = 23,     /* e4m3 mma.sync : lop3 : lop3 : fma.rn.f32, 1:2:1     */
    GQ_PROBE_LOP3_POPC = 24,    /* lop3 and popc interleaved               */
    GQ_PROBE_ISSUE_KINDS = 25
};

/* Instruction issue rate: one block of 32 warps per SM runs `iters` loop iterations of 32
 * instructions of `kind` per thread on eight independent chains; cycles_device[sm] receives the
 * block's elapsed SM clock cycles (one u64 per SM, 8-byte aligned); sink_device is one u32 that
 * keeps the chains live.  Warp instructions per SM per cycle = gq_probe_issue_insts(kind, iters)
 * / cycles.  Errors: GQ_EINVAL_SHAPE for an unknown kind or iters outside [1, 2^24];
 * GQ_EINVAL_PTR; GQ_ECUDA. */
int gq_probe_issue(int kind, int iters, unsigned long long* cycles_device, uint32_t* sink_device,
                   gq_stream_t stream);
/* Warp instructions of the measured kind(s) that one block of gq_probe_issue executes. */
double gq_probe_issue_insts(int kind, int iters);

/* tcgen05 MMA kinds of gq_probe_mma.  There is no int8 kind: ptxas rejects tcgen05.mma
 * kind::i8 for sm_103a. */
enum gq_probe_mma_kind {
    GQ_PROBE_MMA_F16 = 0,       /* kind::f16, bf16 operands, f32 accumulator, K = 16 per MMA  */
    GQ_PROBE_MMA_F8 = 1,        /* kind::f8f6f4, e4m3 operands, f32 accumulator, K = 32       */
    GQ_PROBE_MMA_F16_TMEM_A = 2 /* kind::f16 as kind 0, with the A operand in tensor memory   */
};

/* tcgen05 MMA rate: on every SM one thread issues `iters` MMAs of M = 128, N = n, with both
 * operands in shared memory, into one TMEM accumulator, then waits (bounded) for them to
 * complete; cycles_device[sm] receives the SM clock cycles from the first issue to completion.
 * (Kind GQ_PROBE_MMA_F16_TMEM_A takes A from tensor memory, as the library's prefill does.)
 * Flops per MMA = 2 * 128 * n * K.  Errors: GQ_EUNSUPPORTED for another kind; GQ_EINVAL_SHAPE
 * unless n is a multiple of 16 in [16, 256] and 1 <= iters <= 100000; GQ_EINVAL_PTR; GQ_ECUDA. */
int gq_probe_mma(int kind, int n, int iters, unsigned long long* cycles_device, gq_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* GQ_H */
