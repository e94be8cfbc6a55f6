// Q1_0 products with an epilogue, few tokens (one decoded token to a small batch): mma.sync, weights straight from memory.
//
// A thread block holds 32 rows (of both matrices of a pair) and up to 4 * NT (two parts) or 8 * NT tokens.  Its 16 warps are two groups
// of 16 rows by eight shares of the 128-blocks.  In a block, lane (g, t) takes word t of rows g and g + 8 and that is its share of eight
// m16n8k16 products: the bits p and p + 16 of a word, p = 0..15, are one register of +-d0, by a shift and one logic
// operation, so weights need no shuffles and no shared memory.  The columns of the other operand are tokens, or each token's
// two parts side by side, which puts both parts' sums into one thread.  It is written to shared memory once for a segment of the
// blocks, in the order of the lanes' 16-byte reads.
// Bound by latency for one token: weights requested before the wait for the preceding kernel, activations (two dependent
// loads), products, one sum over the shares through shared memory.
#include "linear.cuh"

namespace gq {
namespace {

constexpr int kWarps = 16, kShares = 8, kThreads = kWarps * 32, kBlockRows = 32;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What a lane loads of a 128-block: words of rows g and g + 8, and their scales
struct Piece { uint32_t w0, w1; uint16_t d0, d1; };

__host__ __device__ constexpr int segment_blocks(int nt) { return nt <= 2 ? 32 : 64 / nt; }         // 64 KB (one n-tile) or 128 KB of operand

template <int NT, int PARTS, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) linear_rows_kernel(const LinearArgs a) {
    constexpr int MT = PAIR ? 2 : 1, TOK = 8 * NT / PARTS, SEG = segment_blocks(NT), U = SEG / kShares;
    extern __shared__ __align__(16) uint8_t smem[];
    uint4* sb = reinterpret_cast<uint4*>(smem);                                 // [SEG][NT][4][32 lanes]
    float* red = reinterpret_cast<float*>(smem);                                // afterwards: [MT][kShares][TOK][32 rows]
    __shared__ uint32_t largest[TOK];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int group = warp & 1, share = warp >> 1;
    const int row0 = blockIdx.x * kBlockRows, tok0 = blockIdx.y * TOK, toks = min(TOK, a.cols - tok0);
    const int nb = a.n / 128;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // rows are padded to whole tiles of 128, so every row of the block is there
    const size_t tile = static_cast<size_t>(row0 / kTileRows) * nb * kChunkBytes;
    const int r = row0 % kTileRows + 16 * group + g;
    auto load = [&](int m, int b) {
        const uint8_t* ch = a.w[m] + tile + static_cast<size_t>(b) * kChunkBytes;
        Piece p;
        p.w0 = *reinterpret_cast<const uint32_t*>(ch + r * 16 + t * 4);
        p.w1 = *reinterpret_cast<const uint32_t*>(ch + (r + 8) * 16 + t * 4);
        p.d0 = *reinterpret_cast<const uint16_t*>(ch + kTileRows * 16 + r * 2);
        p.d1 = *reinterpret_cast<const uint16_t*>(ch + kTileRows * 16 + (r + 8) * 2);
        return p;
    };
    Piece next[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int m = 0; m < MT; ++m) next[u][m] = share + u * kShares < nb ? load(m, share + u * kShares) : Piece{0u, 0u, 0, 0};
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // the tokens' largest scales
    const size_t row_bytes = static_cast<size_t>(nb) * 4 * 34;
    if (tid < TOK) largest[tid] = 0;
    __syncthreads();
    for (int tk = warp; tk < toks; tk += kWarps) {
        const uint8_t* p = a.act + static_cast<size_t>(tok0 + tk) * row_bytes;
        uint32_t top = 0;
        for (int b = lane; b < 4 * nb; b += 32) top = max(top, *reinterpret_cast<const uint16_t*>(p + static_cast<size_t>(b) * 34) & 0x7fffu);
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) largest[tk] = top;
    }
    __syncthreads();

    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.f;

    for (int s0 = 0; s0 < nb; s0 += SEG) {
        const int blocks = min(SEG, nb - s0);
        if (s0) __syncthreads();
        // an item: four values of a token, e = 4 l .. 4 l + 3 of 32-block k of a 128-block: the pairs p = l (e, e + 2) and l + 8
        for (int i = tid; i < blocks * 32 * TOK; i += kThreads) {
            const int l = i & 7, k = (i >> 3) & 3, tk = (i >> 5) % TOK, b = (i >> 5) / TOK;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (tk < toks) {
                const uint16_t* p = reinterpret_cast<const uint16_t*>(a.act + static_cast<size_t>(tok0 + tk) * row_bytes +
                                                                      static_cast<size_t>(4 * (s0 + b) + k) * 34);
                const float d = f16_to_f32(p[0]) * pow2(token_shift(largest[tk]));
                const uint32_t lo = p[1 + 2 * l], hi = p[2 + 2 * l];
                v[0] = d * static_cast<float>(static_cast<int8_t>(lo & 0xff));
                v[1] = d * static_cast<float>(static_cast<int8_t>(lo >> 8));
                v[2] = d * static_cast<float>(static_cast<int8_t>(hi & 0xff));
                v[3] = d * static_cast<float>(static_cast<int8_t>(hi >> 8));
            }
            uint16_t h[4], low[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) two_parts(v[e], h[e], low[e]);
            const int col = PARTS * tk, nt = col >> 3, c = col & 7;
            // register p of lane (c, k) stands in chunk p / 4
            uint32_t* base = reinterpret_cast<uint32_t*>(sb) + static_cast<size_t>(b * NT + nt) * 512;
            const int at = ((l >> 2) * 32 + c * 4 + k) * 4 + (l & 3);
            base[at] = h[0] | static_cast<uint32_t>(h[2]) << 16;
            base[at + 2 * 32 * 4] = h[1] | static_cast<uint32_t>(h[3]) << 16;
            if (PARTS == 2) {
                base[at + 16] = low[0] | static_cast<uint32_t>(low[2]) << 16;
                base[at + 16 + 2 * 32 * 4] = low[1] | static_cast<uint32_t>(low[3]) << 16;
            }
        }
        __syncthreads();
        for (int b0 = share; b0 < blocks; b0 += U * kShares) {
            Piece now[U][MT];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    now[u][m] = next[u][m];
                    const int b = s0 + b0 + (U + u) * kShares;                  // SEG is a multiple of kShares: the share goes on
                    if (b < nb) next[u][m] = load(m, b);                        // of the next segment, at this one's end
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int b = b0 + u * kShares;
                if (b >= blocks) break;
                // a chain of eight products, then registers
                float c[MT][NT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) c[m][j][i] = 0.f;
                uint32_t da[MT], db[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) {                                  // -d0 for a clear bit
                    da[m] = (now[u][m].d0 * 0x00010001u) ^ 0x80008000u;
                    db[m] = (now[u][m].d1 * 0x00010001u) ^ 0x80008000u;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {                                   // registers 4 q .. 4 q + 3: two products
                    uint32_t av[2][MT][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const int p = 4 * q + 2 * h;
                            av[h][m][0] = ((now[u][m].w0 << (15 - p)) & 0x80008000u) ^ da[m];
                            av[h][m][1] = ((now[u][m].w1 << (15 - p)) & 0x80008000u) ^ db[m];
                            av[h][m][2] = ((now[u][m].w0 << (14 - p)) & 0x80008000u) ^ da[m];
                            av[h][m][3] = ((now[u][m].w1 << (14 - p)) & 0x80008000u) ^ db[m];
                        }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const uint4 bv = sb[static_cast<size_t>((b * NT + j) * 4 + q) * 32 + lane];
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            mma16816(c[m][j], av[0][m], bv.x, bv.y);
                            mma16816(c[m][j], av[1][m], bv.z, bv.w);
                        }
                    }
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[m][j][i] += c[m][j][i];
            }
        }
    }
    __syncthreads();
    // the shares' sums: a thread has rows g and g + 8 of its group, columns 2 t and 2 t + 1 of each eight
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float* at = red + (m * kShares + share) * TOK * 32 + 16 * group + 8 * h + g;
                if (PARTS == 2) at[(4 * j + t) * 32] = acc[m][j][2 * h] + acc[m][j][2 * h + 1];
                else {
                    at[(8 * j + 2 * t) * 32] = acc[m][j][2 * h];
                    at[(8 * j + 2 * t + 1) * 32] = acc[m][j][2 * h + 1];
                }
            }
    __syncthreads();
    // four tokens a warp, four rows a lane
    const int row = row0 + 4 * (lane & 7);
    float bias[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) bias[m][i] = a.bias[m] && row + i < a.rows ? a.bias[m][row + i] : 0.f;
    for (int t0 = 4 * warp; t0 < toks; t0 += 4 * kWarps) {
        const int tk = t0 + (lane >> 3);
        const bool on = tk < toks;
        const size_t tok = tok0 + tk;
        float other[4], z[MT][4];
        if (!PAIR) load_four(a, other, row, tok, on);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on)
#pragma unroll
                for (int q = 0; q < kShares; ++q) {
                    const float4 p = *reinterpret_cast<const float4*>(red + ((m * kShares + q) * TOK + tk) * 32 + 4 * (lane & 7));
                    v = make_float4(v.x + p.x, v.y + p.y, v.z + p.z, v.w + p.w);
                }
            const float s = on ? pow2(-token_shift(largest[tk])) : 0.f;          // the product is exact
            z[m][0] = fmaf(v.x, s, bias[m][0]);
            z[m][1] = fmaf(v.y, s, bias[m][1]);
            z[m][2] = fmaf(v.z, s, bias[m][2]);
            z[m][3] = fmaf(v.w, s, bias[m][3]);
        }
        finish_fours<PAIR, 1>(a, z[0], PAIR ? z[MT - 1] : other, row, static_cast<int>(tok), a.cols, lane);
    }
}

template <int NT, int PARTS, bool PAIR>
cudaError_t rows_go(const LinearArgs& a, cudaStream_t s) {
    constexpr int MT = PAIR ? 2 : 1, TOK = 8 * NT / PARTS;
    constexpr size_t sum = static_cast<size_t>(MT) * kShares * TOK * 32 * 4, operand = static_cast<size_t>(segment_blocks(NT)) * NT * 2048;
    constexpr size_t smem = sum > operand ? sum : operand;
    static std::atomic<uint64_t> raised{0};
    const cudaError_t e = allow_smem(linear_rows_kernel<NT, PARTS, PAIR>, smem, raised);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.rows + kBlockRows - 1) / kBlockRows, (a.cols + TOK - 1) / TOK);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_rows_kernel<NT, PARTS, PAIR>, a);
}

template <int PARTS, bool PAIR>
cudaError_t rows_tokens(const LinearArgs& a, cudaStream_t s) {
    const int columns = a.cols * PARTS;
    if (columns <= 8) return rows_go<1, PARTS, PAIR>(a, s);
    if (columns <= 16) return rows_go<2, PARTS, PAIR>(a, s);
    return rows_go<4, PARTS, PAIR>(a, s);
}

}  // namespace

// From this many columns on (tokens times parts) the tiles take over
constexpr int kRowColumns = 32;

cudaError_t launch_linear(const LinearArgs& a, bool pair, cudaStream_t s) {
    const int parts = linear_parts(a);
    if (a.cols * parts > kRowColumns) return launch_linear_tiles(a, pair, s);
    if (parts == 1) return pair ? rows_tokens<1, true>(a, s) : rows_tokens<1, false>(a, s);
    return pair ? rows_tokens<2, true>(a, s) : rows_tokens<2, false>(a, s);
}

size_t linear_workspace_bytes(int rows, int n, int cols, int type) {
    // bf16 may take one part or, with Q8_0 outputs, two
    size_t need = 16;
    for (int parts = type == GQ_BF16 ? 1 : 2; parts <= 2; ++parts)
        if (static_cast<long long>(cols) * parts > kRowColumns) need = std::max(need, linear_tiles_workspace_bytes(rows, n, cols, parts));
    return need;
}

}  // namespace gq
