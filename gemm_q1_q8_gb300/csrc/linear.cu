// Q1_0 products with an epilogue, few tokens (one decoded token to a batch): mma.sync, weights straight from memory.
//
// A thread block holds 32 rows (of both matrices of a pair) and 8 * NT tokens.  Its 16 (8) warps are two groups of 16 rows by eight (four) shares
// of the 128-blocks; the smaller block, of which an SM holds two, where the larger would come in two waves.  Signs become +-d0 as f16 by a shift and a logic operation a pair, codes are f16 as they are, so two
// m16n8k16 products give the 32-block sums d0 * sum(+-q) exactly; they are multiplied by the token's scale and added in f32 registers.  In a word,
// lane t of a row's four takes the bit pairs 4 t .. 4 t + 3 (bits p and p + 16 are one register): weights need no shuffles and no
// shared memory.  Codes are written to shared memory once for a segment of the blocks, in the order of the lanes' 16-byte reads.
// Bound by latency for one token (weights are requested before the wait for the preceding kernel; codes, products, one sum over the shares), by the
// rate of mma.sync for many.
#include "linear.cuh"

namespace gq {
namespace {

constexpr int kBlockRows = 32;
constexpr int kRowsAlways = 4;                    // tokens for which this kernel is taken: the faster one at every size that was measured

// d = a . b (from zero), then d += a . b
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What a lane loads of a 128-block: the words of rows g and g + 8, and their scales
struct Piece { uint4 w[2]; uint32_t d[2]; };

__device__ __forceinline__ void cp_async8(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Of a 128-block and 8 tokens: codes in [sub-block][lane][register], 2 KB; scales, [sub-block][token]; the tokens' bytes
__host__ __device__ constexpr int block_bytes(int nt) { return nt * (2048 + 4 * 8 * 4 + 8 * 136); }
// Blocks of a segment: up to 209 KB, a multiple of the shares
__host__ __device__ constexpr int most_blocks(int nt) { return 64 / nt; }

template <int NT, bool PAIR, int kShares>
__global__ void __launch_bounds__(64 * kShares, 8 / kShares) linear_rows_kernel(const LinearArgs a, int segment) {
    constexpr int kWarps = 2 * kShares, kThreads = 32 * kWarps;
    constexpr int MT = PAIR ? 2 : 1, TOK = 8 * NT, U = NT * MT <= 2 ? 3 : NT * MT <= 4 ? 2 : 1;
    extern __shared__ __align__(16) uint8_t smem[];
    uint32_t* codes = reinterpret_cast<uint32_t*>(smem);                        // [segment][NT][4][32 lanes][4]
    float* scales = reinterpret_cast<float*>(smem + static_cast<size_t>(segment) * NT * 2048);      // [segment][4][TOK]
    uint8_t* raw = smem + static_cast<size_t>(segment) * NT * (2048 + 128);     // [TOK][segment][136 bytes]
    float* red = reinterpret_cast<float*>(smem);                                // afterwards: [MT][kShares][TOK][32 rows]
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
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            p.w[h] = *reinterpret_cast<const uint4*>(ch + (r + 8 * h) * 16);
            p.d[h] = *reinterpret_cast<const uint16_t*>(ch + kTileRows * 16 + (r + 8 * h) * 2);
        }
        return p;
    };
    Piece next[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int m = 0; m < MT; ++m) next[u][m] = share + u * kShares < nb ? load(m, share + u * kShares) : Piece{};
    asm volatile("griddepcontrol.wait;" ::: "memory");

    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.f;

    const size_t row_bytes = static_cast<size_t>(nb) * 4 * 34;
    for (int s0 = 0; s0 < nb; s0 += segment) {
        const int blocks = min(segment, nb - s0);
        if (s0) __syncthreads();
        // The tokens' bytes of the segment to shared memory, all on their way at once: a 128-block has 17 words of 8 bytes.  (Each 4 codes loaded where
        // they are converted, by 2-byte loads: 8 tokens over 6912, 12.0 us.)
        const bool staged = (reinterpret_cast<uintptr_t>(a.act) & 7) == 0;
        const uint32_t words = blocks * 17, word_magic = 0xffffffffu / words + 1;
        if (staged) {
            for (uint32_t i = tid; i < toks * words; i += kThreads) {
                const uint32_t tk = toks == 1 ? 0 : __umulhi(i, word_magic), e = i - tk * words;
                cp_async8(raw + (tk * segment * 17 + e) * 8, a.act + (tok0 + tk) * row_bytes + static_cast<size_t>(s0) * 136 + e * 8);
            }
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
            __syncthreads();
        }
        // an item: four codes 4 l .. 4 l + 3 of a token's 32-block: the pairs (4 l, 4 l + 2) and (4 l + 1, 4 l + 3).  Columns of tokens that
        // do not exist stay as they are: a column's sums are its own.
        const uint32_t per = blocks * 32, magic = 0xffffffffu / per + 1;      // quotients are exact below 2^20
#pragma unroll 2
        for (uint32_t i = tid; i < toks * per; i += kThreads) {
            const uint32_t tk = toks == 1 ? 0 : __umulhi(i, magic), e = i - tk * per, l = e & 7, s = e >> 3, b = s >> 2, k = s & 3;
            const uint16_t* p = reinterpret_cast<const uint16_t*>(staged ? raw + tk * segment * 136 + s * 34
                                                                         : a.act + (tok0 + tk) * row_bytes + static_cast<size_t>(4 * s0 + s) * 34);
            const uint32_t lo = p[1 + 2 * l], hi = p[2 + 2 * l], w = (lo | hi << 16) ^ 0x80808080u;       // code + 128
            const uint32_t even = __byte_perm(w, 0x64646464u, 0x4240), odd = __byte_perm(w, 0x64646464u, 0x4341);   // 1024 + that, as f16
            const __half2 bias = __half2half2(__ushort_as_half(0x6480));                                  // 1152
            const __half2 v0 = __hsub2(*reinterpret_cast<const __half2*>(&even), bias), v1 = __hsub2(*reinterpret_cast<const __half2*>(&odd), bias);
            uint32_t* to = codes + ((b * NT + (tk >> 3)) * 4 + k) * 128 + ((tk & 7) * 4 + (l >> 2)) * 4 + (l & 3);
            to[0] = *reinterpret_cast<const uint32_t*>(&v0);
            to[2 * 4] = *reinterpret_cast<const uint32_t*>(&v1);
            if (l == 0) scales[s * TOK + tk] = f16_to_f32(p[0]);
        }
        __syncthreads();
#pragma unroll 1
        for (int b = share; b < blocks; b += kShares) {
            Piece now[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                now[m] = next[0][m];
#pragma unroll
                for (int u = 0; u + 1 < U; ++u) next[u][m] = next[u + 1][m];
                if (s0 + b + U * kShares < nb) next[U - 1][m] = load(m, s0 + b + U * kShares);   // segments are multiples of the shares: theirs go on
            }
            uint32_t neg[MT][2];                                                // -d0 for a clear bit
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) neg[m][h] = (now[m].d[h] * 0x00010001u) ^ 0x80008000u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t av[2][MT][4];                                          // two products: pairs 4 t + 2 i and 4 t + 2 i + 1
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t w = k == 0 ? now[m].w[h].x : k == 1 ? now[m].w[h].y : k == 2 ? now[m].w[h].z : now[m].w[h].w;
#pragma unroll
                        for (int p = 0; p < 4; ++p) av[p >> 1][m][2 * (p & 1) + h] = ((w << (15 - p - 4 * t)) & 0x80008000u) ^ neg[m][h];
                    }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint4 bv = *reinterpret_cast<const uint4*>(codes + (static_cast<size_t>((b * NT + j) * 4 + k) * 32 + lane) * 4);
                    const float2 d = *reinterpret_cast<const float2*>(scales + (4 * b + k) * TOK + 8 * j + 2 * t);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        float c[4] = {0.f, 0.f, 0.f, 0.f};
                        mma16816(c, av[0][m], bv.x, bv.y);
                        mma16816(c, av[1][m], bv.z, bv.w);
                        acc[m][j][0] = fmaf(d.x, c[0], acc[m][j][0]);
                        acc[m][j][1] = fmaf(d.y, c[1], acc[m][j][1]);
                        acc[m][j][2] = fmaf(d.x, c[2], acc[m][j][2]);
                        acc[m][j][3] = fmaf(d.y, c[3], acc[m][j][3]);
                    }
                }
            }
        }
    }
    __syncthreads();
    // the shares' sums: a thread has rows g and g + 8 of its group, tokens 2 t and 2 t + 1 of each eight
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[((m * kShares + share) * TOK + 8 * j + 2 * t + (i & 1)) * 32 + 16 * group + 8 * (i >> 1) + g] = acc[m][j][i];
    __syncthreads();
    // four tokens a warp, four rows a lane
    const int row = row0 + 4 * (lane & 7);
    float bias[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) bias[m][i] = a.bias[m] && row + i < a.rows ? a.bias[m][row + i] : 0.f;
    for (int t0 = 4 * warp; t0 < toks; t0 += 4 * kWarps) {
        const int tk = t0 + (lane >> 3), tok = tok0 + tk;
        const bool on = tk < toks;
        float other[4], z[MT][4];
        if (!PAIR) load_four(a, other, row, tok, on);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float4 v = make_float4(bias[m][0], bias[m][1], bias[m][2], bias[m][3]), s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on)
#pragma unroll
                for (int q = 0; q < kShares; ++q) {
                    const float4 p = *reinterpret_cast<const float4*>(red + ((m * kShares + q) * TOK + tk) * 32 + 4 * (lane & 7));
                    s = make_float4(s.x + p.x, s.y + p.y, s.z + p.z, s.w + p.w);
                }
            z[m][0] = s.x + v.x, z[m][1] = s.y + v.y, z[m][2] = s.z + v.z, z[m][3] = s.w + v.w;
        }
        finish_fours<PAIR, 1>(a, z[0], PAIR ? z[MT - 1] : other, row, tok, a.cols, lane);
    }
}

template <int NT, bool PAIR, int kShares>
cudaError_t rows_go(const LinearArgs& a, cudaStream_t s) {
    constexpr int MT = PAIR ? 2 : 1, TOK = 8 * NT, most_segment = most_blocks(NT) * kShares / 8 / kShares * kShares;
    const int nb = (a.n / 128 + kShares - 1) / kShares * kShares, segment = nb < most_segment ? nb : most_segment;
    const size_t sum = static_cast<size_t>(MT) * kShares * TOK * 32 * 4, operand = static_cast<size_t>(segment) * block_bytes(NT);
    const size_t smem = sum > operand ? sum : operand, most = std::max(sum, static_cast<size_t>(most_segment) * block_bytes(NT));
    static std::atomic<uint64_t> raised{0};
    const cudaError_t e = allow_smem(linear_rows_kernel<NT, PAIR, kShares>, most, raised);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.rows + kBlockRows - 1) / kBlockRows, (a.cols + TOK - 1) / TOK);
    cfg.blockDim = dim3(64 * kShares);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_rows_kernel<NT, PAIR, kShares>, a, segment);
}

template <bool PAIR>
cudaError_t launch_linear_rows(const LinearArgs& a, cudaStream_t s) {
    const bool small = (a.rows + kBlockRows - 1) / kBlockRows > 152;
    if (a.cols <= 8) return small ? rows_go<1, PAIR, 4>(a, s) : rows_go<1, PAIR, 8>(a, s);
    if (a.cols <= 16) return small ? rows_go<2, PAIR, 4>(a, s) : rows_go<2, PAIR, 8>(a, s);
    return rows_go<4, PAIR, 8>(a, s);
}

}  // namespace

// Up to 32 tokens the rows' kernel may be taken, where it is the faster one by its cost (linear_tiles.cu has the tiles'): fitted to 1 to 32 tokens of
// 400 x 1024, 2560 x 2560, 2560 x 6912 and 14336 x 8192 and the pairs of 6912 x 2560 and 14336 x 4096, in microseconds.
bool linear_by_rows(int rows, int n, int cols, bool pair, int parts) {
    if (cols > 32) return false;
    if (cols <= kRowsAlways) return true;
    const int nt = cols <= 8 ? 1 : cols <= 16 ? 2 : 4;
    const float waves = static_cast<float>(((rows + kBlockRows - 1) / kBlockRows + 151) / 152);
    const float us = 1.7f + waves * (0.5f + n * 1e-3f * (0.25f + 0.08f * cols + (pair ? 0.7f : 0.25f) * nt));
    return us < linear_tiles_us(rows, n, cols, parts, pair);
}

cudaError_t launch_linear(const LinearArgs& a, bool pair, cudaStream_t s) {
    if (!linear_by_rows(a.rows, a.n, a.cols, pair, linear_parts(a))) return launch_linear_tiles(a, pair, s);
    return pair ? launch_linear_rows<true>(a, s) : launch_linear_rows<false>(a, s);
}

int linear_plan(int rows, int n, int cols, int parts, bool pair) {
    return linear_by_rows(rows, n, cols, pair, parts) ? 0 : linear_tiles_plan(rows, n, cols, parts, pair);
}

size_t linear_workspace_bytes(int rows, int n, int cols) {
    // for either call, any outputs and any count of tokens up to this one
    if (cols <= kRowsAlways) return 16;
    return std::max(linear_tiles_workspace_bytes(rows, n, cols, false), linear_tiles_workspace_bytes(rows, n, cols, true));
}

}  // namespace gq
