// Attention over the paged Q8_0 cache for few rows (decode, drafted trees).
//
// Mathematics: s = scale * q.k; o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m), one pass over the keys with the
// running maximum m (base 2).  Rows are a kv head's query heads times its query tokens (row = token * group + head).
// The floor is the cache's bytes (17/16 a value) at the HBM rate; a row costs 4 flops a value, so up to some 16 rows
// a read the matrix work hides behind the copy.
//
// Work: the unit is one 16-token chunk of one (sequence, kv head, row tile); the units of the whole call, in that
// order, are cut into equal runs of consecutive units, one a thread block (one block an SM), whatever the sequences'
// lengths.  A run's warps take its units in turn, each from its own ring of bulk copies (a chunk is one contiguous
// copy), so nothing but the end of a row tile meets at a barrier.  A row tile that several blocks share leaves
// partial sums in the workspace, and a second kernel joins them in block order: the result does not depend on timing.
//
// Tensor cores: mma.sync m16n8k16 (f32 sums) with the queries as A and 8 keys as B.  Each code is its own exact 16-bit float: sign and
// 7-bit magnitude are the bits of the f16 subnormal magnitude * 2^-24, and of the bf16 one magnitude * 2^-133, so two codes become a
// register with one byte permute and one mask, and no conversion.  S: each 32-dim block has its own accumulator, multiplied by the
// key's scale in f32.  O: the weight times the value's scale is A, and the codes are B.
// 16-bit queries: one f16 part of each, 16 rows a tile, powers of two keeping A near the top of f16's range (a row's largest query value,
// and the largest value scale seen so far, go to 2^14..2^15): a rounding costs 2^-12 of the value, or 2^-40 of the largest.
// f32 queries: 8 rows a tile; A has the high f16 part of the queries in its rows 0-7 and the rest in rows 8-15 (22 bits together); both halves
// of a row end in one thread, which adds them.  The weights take three bf16 parts (24 bits, the third in a product of its own) for f32's
// range: a weight of 2^-90 counts where the larger ones meet zero codes.
// Why not tcgen05 here: its tiles are 128 rows, and B comes from shared memory only, so the codes would be
// converted through shared memory for rows that are mostly absent.
#include "layer_ops.cuh"

namespace gq {
GQ_ERROR_ACCESSOR(attn)
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kBlocks = 152;                       // one thread block an SM
constexpr float kNone = -1e30f;                    // running maximum of a row that has seen no key
constexpr float kLog2e = 1.4426950408889634f;

template <int HD> __host__ __device__ constexpr int stages() { return HD == 64 ? 6 : HD == 128 ? 4 : 2; }
// Rows of a tile, and the columns of it that meet in shared memory at a time (64 KB at most)
template <int PARTS, int MT> __host__ __device__ constexpr int tile_rows() { return MT * 16 / PARTS; }
template <int HD, int PARTS, int MT> __host__ __device__ constexpr int merge_cols() {
    return tile_rows<PARTS, MT>() * HD <= 2048 ? HD : 2048 / tile_rows<PARTS, MT>();
}
template <int HD, int PARTS, int MT> constexpr int smem_bytes() {
    return 1024 + kWarps * stages<HD>() * kv_chunk_bytes(HD) + kWarps * tile_rows<PARTS, MT>() * (merge_cols<HD, PARTS, MT>() + 4) * 4;
}

// One sequence's share of the work.
struct Seq {
    int L, T, q0;          // cached tokens, query tokens, first query row
    int groups;            // 16-token chunks
    int tiles;             // row tiles a kv head
    __device__ __forceinline__ long long units(int kv_heads) const { return static_cast<long long>(groups) * tiles * kv_heads; }
};
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b, int rows) {
    Seq s;
    s.q0 = a.q_start[b];
    s.T = a.q_start[b + 1] - s.q0;
    s.L = a.kv_len[b];
    if (s.T > a.max_q || s.L > a.max_kv) report_error(kErrIndex);
    s.groups = (min(max(s.L, 0), a.max_kv) + kvGroup - 1) / kvGroup;
    s.tiles = (min(max(s.T, 0), a.max_q) * (a.q_heads / a.kv_heads) + rows - 1) / rows;
    return s;
}

// The units of all sequences, by one warp.
__device__ __forceinline__ long long total_units(const AttnArgs& a, int rows, int lane) {
    long long sum = 0;
    for (int b = lane; b < a.seqs; b += 32) sum += load_seq(a, b, rows).units(a.kv_heads);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}
// The sequence that holds unit w, and its first unit.
__device__ __forceinline__ int locate(const AttnArgs& a, int rows, int lane, long long w, long long& first) {
    long long before = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += 32) {
        const int b = b0 + lane;
        const long long mine = b < a.seqs ? load_seq(a, b, rows).units(a.kv_heads) : 0;
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + upto > w);
        if (hit) {
            const int at = __ffs(hit) - 1;
            first = before + __shfl_sync(0xffffffffu, upto - mine, at);
            return b0 + at;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    first = before;
    return a.seqs;
}
// Units a block takes: whole rounds of its warps.
__device__ __forceinline__ long long run_length(long long total, int blocks) {
    const long long each = (total + blocks - 1) / blocks;
    return (each + kWarps - 1) / kWarps * kWarps;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }    // -126 <= e <= 127

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two codes as two f16 subnormals (magnitude * 2^-24), or bf16 ones (magnitude * 2^-133)
__device__ __forceinline__ uint32_t codes2(uint32_t lo, uint32_t hi, uint32_t sel) { return __byte_perm(lo, hi, sel) & 0x807f807fu; }
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2_bf16(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }

// A row of this thread's tile: where its query is, what it sees.
struct RowInfo {
    float rs;              // score multiplier: scale * log2(e) (or scale / softcap) and the powers of two taken out
    int last;              // causal: the last visible token; -1 for a row past the end
    uint32_t bits0, bits1; // tree: visible among the newest
};

template <typename T, int HD, int PARTS, int MT>
struct Tile {
    static constexpr int kKs = HD / 16, kNb = HD / 32, kRowsT = tile_rows<PARTS, MT>(), kSets = PARTS == 2 ? 1 : 2;
    uint32_t qa[MT][kKs][4];
    float o[MT][kNb][4][4];
    float m[MT][kSets], l[MT][kSets];
    RowInfo row[MT][kSets];
    int vexp;              // value scales are multiplied by 2^(15 - vexp)

    // Queries of rows tile0 .. as fragments, rows' multipliers and masks, empty sums
    __device__ __forceinline__ void start(const AttnArgs& a, const Seq& s, int hk, int tile0, int lane) {
        const int g = lane >> 2, t = lane & 3, group = a.q_heads / a.kv_heads;
        const int rows = min(max(s.T, 0), a.max_q) * group;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int set = 0; set < kSets; ++set) {
                const int r = tile0 + mt * (16 / PARTS) + set * 8 + g;
                const bool in = r < rows;
                const int tok = in ? r / group : 0, h = in ? r % group : 0;
                const T* q = static_cast<const T*>(a.q) + (s.q0 + tok) * a.q_stride + (hk * group + h) * HD;
                float4 v[kKs];
                float amax = 0.f;
#pragma unroll
                for (int ks = 0; ks < kKs; ++ks) {
                    v[ks] = in ? load4(q + 16 * ks + 4 * t) : make_float4(0.f, 0.f, 0.f, 0.f);
                    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(v[ks].x), fabsf(v[ks].y)), fmaxf(fabsf(v[ks].z), fabsf(v[ks].w))));
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // the largest value goes to [2^14, 2^15); not finite or zero: as it is
                const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
                const int up = amax > 0.f && e < 128 ? min(14 - e, 126) : 0;
                const float f = pow2i(up);
#pragma unroll
                for (int ks = 0; ks < kKs; ++ks) {
                    const float4 w = make_float4(v[ks].x * f, v[ks].y * f, v[ks].z * f, v[ks].w * f);
                    const uint32_t h0 = pack2(w.x, w.y), h1 = pack2(w.z, w.w);
                    qa[mt][ks][set] = h0;
                    qa[mt][ks][2 + set] = h1;
                    if (PARTS == 2) {
                        const float2 x = unpack2(h0), y = unpack2(h1);
                        qa[mt][ks][1] = pack2(w.x - x.x, w.y - x.y);
                        qa[mt][ks][3] = pack2(w.z - y.x, w.w - y.y);
                    }
                }
                RowInfo& ri = row[mt][set];
                // 2^24 for the codes, 2^-up for the query; in two steps, each within f32's range
                ri.rs = (a.softcap > 0.f ? a.scale / a.softcap : a.scale * kLog2e) * 16777216.f * pow2i(-up);
                ri.last = in ? s.L - s.T + tok : -1;
                const unsigned long long bits = a.tree && in ? a.tree[s.q0 + tok] : 0ull;
                ri.bits0 = static_cast<uint32_t>(bits);
                ri.bits1 = static_cast<uint32_t>(bits >> 32);
                m[mt][set] = kNone;
                l[mt][set] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < kNb; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[mt][c][e][i] = 0.f;
        }
        vexp = -24;
    }

    // One chunk of 16 tokens from j0 on.  MASKED: some of its tokens are new or past the end.
    template <bool MASKED>
    __device__ __forceinline__ void chunk(const AttnArgs& a, const Seq& s, const uint8_t* __restrict__ buf, int j0, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const int len = min(s.L, a.max_kv);
        // scales of this thread's four tokens (2t, 2t + 1, 2t + 8, 2t + 9), [token][block]
        uint32_t ksw[kNb * 2], vsw[kNb * 2];
#pragma unroll
        for (int i = 0; i < kNb / 2; ++i) {
            *reinterpret_cast<uint4*>(ksw + 4 * i) = *reinterpret_cast<const uint4*>(buf + kv_ks_offset(HD) + t * 8 * kNb + 16 * i);
            *reinterpret_cast<uint4*>(vsw + 4 * i) = *reinterpret_cast<const uint4*>(buf + kv_vs_offset(HD) + t * 8 * kNb + 16 * i);
        }
        if (MASKED) {
#pragma unroll
            for (int p = 0; p < 4; ++p)
                if (j0 + 2 * t + (p & 1) + 8 * (p >> 1) >= len)
#pragma unroll
                    for (int i = 0; i < kNb / 2; ++i) ksw[p * kNb / 2 + i] = vsw[p * kNb / 2 + i] = 0u;
        }
        float S[MT][2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t w[kKs];
#pragma unroll
            for (int c = 0; c < kKs / 4; ++c) {
                int u = 4 * c + t;
                if (HD > 64) u ^= 4 * (g & 1);
                *reinterpret_cast<uint4*>(w + 4 * c) = *reinterpret_cast<const uint4*>(buf + (8 * j + g) * HD + u * 16);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[mt][j][i] = 0.f;
#pragma unroll
            for (int b = 0; b < kNb; ++b) {
                const uint32_t b00 = codes2(w[2 * b], 0, 0x1100), b01 = codes2(w[2 * b], 0, 0x3322);
                const uint32_t b10 = codes2(w[2 * b + 1], 0, 0x1100), b11 = codes2(w[2 * b + 1], 0, 0x3322);
                float k0, k1;                                    // scales of tokens 2j and 2j + 1 of the thread's four
                {
                    const int i0 = 2 * j * kNb + b, i1 = i0 + kNb;
                    k0 = f16_to_f32(i0 & 1 ? ksw[i0 / 2] >> 16 : ksw[i0 / 2] & 0xffffu);
                    k1 = f16_to_f32(i1 & 1 ? ksw[i1 / 2] >> 16 : ksw[i1 / 2] & 0xffffu);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    float p[4] = {0.f, 0.f, 0.f, 0.f};
                    mma16816(p, qa[mt][2 * b], b00, b01);
                    mma16816(p, qa[mt][2 * b + 1], b10, b11);
                    S[mt][j][0] = fmaf(k0, p[0], S[mt][j][0]);
                    S[mt][j][1] = fmaf(k1, p[1], S[mt][j][1]);
                    S[mt][j][2] = fmaf(k0, p[2], S[mt][j][2]);
                    S[mt][j][3] = fmaf(k1, p[3], S[mt][j][3]);
                }
            }
        }
        // f16 weights: the largest value scale so far sets the power of two
        if (PARTS == 1) {
            __half2 mx = *reinterpret_cast<const __half2*>(vsw);
#pragma unroll
            for (int i = 1; i < kNb * 2; ++i) mx = __hmax2(mx, *reinterpret_cast<const __half2*>(vsw + i));
            uint32_t u = *reinterpret_cast<const uint32_t*>(&mx);
            int e = static_cast<int>(max((u >> 10) & 31u, (u >> 26) & 31u)) - 14;     // scale < 2^e
            if (__any_sync(0xffffffffu, e > vexp)) {
                e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
                e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
                const float down = pow2i(vexp - e);
                vexp = e;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int c = 0; c < kNb; ++c)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[mt][c][x][i] *= down;
            }
        }
        // scores to weights
        float P[MT][kSets][4];                                   // [row][token of the thread's four]
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            bool higher = false;
#pragma unroll
            for (int set = 0; set < kSets; ++set) {
                const RowInfo& ri = row[mt][set];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    float x = S[mt][p >> 1][2 * set + (p & 1)];
                    if (PARTS == 2) x += S[mt][p >> 1][2 + (p & 1)];
                    x *= ri.rs;
                    if (a.softcap > 0.f) {
                        // tanh in f32 for f32 queries; 1 - 2 / (e^2x + 1), off by some 2^-23 absolutely, for 16-bit ones
                        const float th = PARTS == 2 ? tanhf(x) : 1.f - __fdividef(2.f, ex2(2.f * kLog2e * x) + 1.f);
                        x = a.softcap * kLog2e * th;
                    }
                    if (MASKED) {
                        const int j = j0 + 2 * t + (p & 1) + 8 * (p >> 1);
                        const int rel = j - (s.L - s.T);
                        bool seen = ri.last >= 0 && j < len;
                        if (a.tree) {
                            const uint32_t word = rel < 32 ? ri.bits0 : ri.bits1;
                            seen = seen && (rel < 0 || (rel < 64 && ((word >> (rel & 31)) & 1u)));
                        } else {
                            seen = seen && j <= ri.last;
                        }
                        if (!seen) x = -INFINITY;
                    }
                    P[mt][set][p] = x;
                }
                const float top = fmaxf(fmaxf(P[mt][set][0], P[mt][set][1]), fmaxf(P[mt][set][2], P[mt][set][3]));
                higher |= top > m[mt][set];
            }
            if (__any_sync(0xffffffffu, higher)) {
#pragma unroll
                for (int set = 0; set < kSets; ++set) {
                    float top = fmaxf(fmaxf(P[mt][set][0], P[mt][set][1]), fmaxf(P[mt][set][2], P[mt][set][3]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    top = fmaxf(top, m[mt][set]);
                    const float down = ex2(m[mt][set] - top);
                    m[mt][set] = top;
                    l[mt][set] *= down;
#pragma unroll
                    for (int c = 0; c < kNb; ++c)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            o[mt][c][x][2 * set] *= down;
                            o[mt][c][x][2 * set + 1] *= down;
                            if (PARTS == 2) {
                                o[mt][c][x][2] *= down;
                                o[mt][c][x][3] *= down;
                            }
                        }
                }
            }
#pragma unroll
            for (int set = 0; set < kSets; ++set)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    P[mt][set][p] -= m[mt][set];
                    P[mt][set][p] = ex2(P[mt][set][p]);
                    l[mt][set] += P[mt][set][p];
                }
        }
        // values: words [token][block], four dims each
        uint32_t w[4][kNb];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint8_t* r = buf + kv_v_offset(HD) + (4 * p + t) * HD;
            if (HD == 64) {
                *reinterpret_cast<uint2*>(w[p]) = *reinterpret_cast<const uint2*>(r + 8 * (g ^ (4 * (t >> 1))));
            } else {
#pragma unroll
                for (int h = 0; h < HD / 128; ++h)
                    *reinterpret_cast<uint4*>(w[p] + 4 * h) = *reinterpret_cast<const uint4*>(r + 128 * h + 16 * (g ^ (2 * t)));
            }
        }
        const float vf = PARTS == 2 ? 0x1p110f : pow2i(15 - vexp);
#pragma unroll
        for (int c = 0; c < kNb; ++c) {
            float vs[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int i = p * kNb + c;
                vs[p] = f16_to_f32(i & 1 ? vsw[i / 2] >> 16 : vsw[i / 2] & 0xffffu) * vf;
            }
            uint32_t pa[MT][4], low[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int set = 0; set < kSets; ++set) {
                    float z[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        z[p] = P[mt][set][p] * vs[p];
                        if (MASKED && P[mt][set][p] == 0.f) z[p] = 0.f;          // whatever the masked value's scale is
                    }
                    if (PARTS == 1) {
                        pa[mt][set] = pack2(z[0], z[1]);
                        pa[mt][2 + set] = pack2(z[2], z[3]);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float x = z[2 * h], y = z[2 * h + 1];
                            pa[mt][2 * h] = pack2_bf16(x, y);
                            x -= __uint_as_float(pa[mt][2 * h] << 16);
                            y -= __uint_as_float(pa[mt][2 * h] & 0xffff0000u);
                            pa[mt][2 * h + 1] = pack2_bf16(x, y);
                            x -= __uint_as_float(pa[mt][2 * h + 1] << 16);
                            y -= __uint_as_float(pa[mt][2 * h + 1] & 0xffff0000u);
                            low[mt][h] = pack2_bf16(x, y);
                        }
                    }
                }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t sel = 0x4400u + 0x1111u * e;
                const uint32_t b0 = codes2(w[0][c], w[1][c], sel), b1 = codes2(w[2][c], w[3][c], sel);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if (PARTS == 1) {
                        mma16816(o[mt][c][e], pa[mt], b0, b1);
                    } else {
                        mma16816_bf16(o[mt][c][e], pa[mt][0], pa[mt][1], pa[mt][2], pa[mt][3], b0, b1);
                        mma16816_bf16(o[mt][c][e], low[mt][0], 0u, low[mt][1], 0u, b0, b1);
                    }
                }
            }
        }
    }
};

template <typename T, int HD, int PARTS, int MT>
__global__ void __launch_bounds__(kThreads, 1) attn_rows_kernel(const AttnArgs a, float* __restrict__ part_o, float2* __restrict__ part_ml,
                                                               int page_shift) {
    using TileT = Tile<T, HD, PARTS, MT>;
    constexpr int kRows = TileT::kRowsT, kNst = stages<HD>(), kChunk = kv_chunk_bytes(HD);
    constexpr int kCols = merge_cols<HD, PARTS, MT>(), kPitch = kCols + 4;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem);                              // [kWarps][kNst]
    uint8_t* ring_all = smem + 1024;
    float* merge = reinterpret_cast<float*>(ring_all + kWarps * kNst * kChunk);      // [kWarps][kRows][kPitch]
    __shared__ float sm[kWarps][kRows], sl[kWarps][kRows];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t* bar = bars + warp * kNst;
    uint8_t* ring = ring_all + warp * kNst * kChunk;
    if (lane == 0)
        for (int i = 0; i < kNst; ++i) mbar_init(&bar[i], 1);
    fence_barrier_init();
    __syncwarp();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const long long total = total_units(a, kRows, lane);
    const long long per = run_length(total, gridDim.x);
    const long long w0 = per * blockIdx.x;
    const long long count = min(total - w0, per);
    if (count <= 0) return;
    long long first;
    const int b_start = locate(a, kRows, lane, w0, first);
    Seq s = load_seq(a, b_start, kRows);
    const int at = static_cast<int>((w0 - first) / s.groups);            // (kv head, row tile) of the first unit
    const int g_start = static_cast<int>((w0 - first) % s.groups);

    // ---- the fetching side: this warp's units warp, warp + 8, ... of the run
    int f_b = b_start, f_at = at, f_g = g_start + warp;
    Seq f_s = s;
    const int gpp = a.page_size / kvGroup;
    int f_page = -1, f_off = 0;
    unsigned good = 0;                                                   // ring slots that hold a chunk
    auto settle = [&]() {                                                // carries f_g into its tile and sequence, and looks its page up
        while (f_g >= f_s.groups) {
            f_g -= f_s.groups;
            if (++f_at >= f_s.tiles * a.kv_heads) {
                f_at = 0;
                do f_s = load_seq(a, ++f_b, kRows); while (f_s.groups == 0 || f_s.tiles == 0);
            }
        }
        const int pi = page_shift >= 0 ? f_g >> page_shift : f_g / gpp;
        f_off = f_g - pi * gpp;
        f_page = __ldg(a.table + static_cast<size_t>(f_b) * a.table_stride + pi);
    };
    long long f_u = warp;
    if (f_u < count) settle();
    auto fetch = [&](int slot) {                                         // requests the warp's next unit into a ring slot
        if (f_u >= count) return;
        const bool ok = f_page >= 0 && f_page < a.pages;
        good = ok ? good | 1u << slot : good & ~(1u << slot);
        if (lane == 0) {
            if (ok) {
                mbar_arrive_expect_tx(&bar[slot], kChunk);
                const uint8_t* src = a.cache + ((static_cast<size_t>(f_page) * a.kv_heads + f_at / f_s.tiles) * gpp + f_off) * kChunk;
                bulk_g2s(ring + slot * kChunk, src, kChunk, &bar[slot]);
            } else {
                mbar_arrive(&bar[slot]);
                report_error(kErrIndex);
            }
        }
        f_u += kWarps;
        f_g += kWarps;
        if (f_u < count) settle();
    };
    for (int i = 0; i < kNst; ++i) fetch(i);

    // ---- the computing side: tile by tile, all warps together
    TileT tile;
    int slot = 0;
    uint32_t phase = 0;
    bool dead = false;
    int dead_slot = 0;
    uint32_t dead_phase = 0;
    int b = b_start, c_at = at, ga = g_start;
    for (long long done = 0; done < count;) {
        if (c_at >= s.tiles * a.kv_heads) {
            do s = load_seq(a, ++b, kRows); while (s.groups == 0 || s.tiles == 0);
            c_at = 0;
        }
        const int n = static_cast<int>(min(static_cast<long long>(s.groups - ga), count - done));
        const int turn = static_cast<int>(done) & (kWarps - 1);          // the warp that has the first of these
        const int hk = c_at / s.tiles, tile0 = (c_at % s.tiles) * kRows;
        const int mine = (warp - turn) & (kWarps - 1);
        if (mine < n) {
            tile.start(a, s, hk, tile0, lane);
            for (int i = mine; i < n; i += kWarps) {
                if (!dead && __any_sync(0xffffffffu, !mbar_wait(&bar[slot], phase))) {
                    dead = true;
                    dead_slot = slot;
                    dead_phase = phase;
                    if (lane == 0) report_error(kErrWaitTimeout);
                }
                if (!dead) {
                    if (good >> slot & 1u) {
                        const int j0 = (ga + i) * kvGroup;
                        if (j0 + kvGroup > min(s.L - s.T, a.max_kv))
                            tile.template chunk<true>(a, s, ring + slot * kChunk, j0, lane);
                        else
                            tile.template chunk<false>(a, s, ring + slot * kChunk, j0, lane);
                    }
                    __syncwarp();
                    fetch(slot);
                }
                if (++slot == kNst) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            // a row's sums in this warp: over the four threads that share it
            const int g = lane >> 2, t = lane & 3;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int set = 0; set < TileT::kSets; ++set) {
                    float l = tile.l[mt][set];
                    l += __shfl_xor_sync(0xffffffffu, l, 1);
                    l += __shfl_xor_sync(0xffffffffu, l, 2);
                    if (t == 0) {
                        sm[warp][mt * (16 / PARTS) + set * 8 + g] = tile.m[mt][set];
                        sl[warp][mt * (16 / PARTS) + set * 8 + g] = l;
                    }
                }
        }
        // ---- the warps' sums meet
        const bool whole = ga == 0 && n == s.groups;                     // this block has all of the tile
        const int live = min(n, kWarps);
        const int group = a.q_heads / a.kv_heads;
        const int rows = min(min(s.T, a.max_q) * group - tile0, kRows);
        const size_t out_slot = 2 * blockIdx.x + (done == 0 && ga > 0 ? 0 : 1);
#pragma unroll
        for (int c0 = 0; c0 < HD; c0 += kCols) {
            if (mine < n) {
                // 2^133 (2^24) for the codes, and the power of two of the value scales
                const float back = PARTS == 2 ? 0x1p23f : pow2i(9 + tile.vexp);
                const int g = lane >> 2, t = lane & 3;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int set = 0; set < TileT::kSets; ++set) {
                        float* dst = merge + (warp * kRows + mt * (16 / PARTS) + set * 8 + g) * kPitch;
#pragma unroll
                        for (int c = 0; c < kCols / 32; ++c) {
                            float v[8];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    float x = tile.o[mt][c0 / 32 + c][e][2 * set + i];
                                    if (PARTS == 2) x += tile.o[mt][c0 / 32 + c][e][2 + i];
                                    v[4 * i + e] = x * back;
                                }
                            *reinterpret_cast<float4*>(dst + 32 * c + 8 * t) = make_float4(v[0], v[1], v[2], v[3]);
                            *reinterpret_cast<float4*>(dst + 32 * c + 8 * t + 4) = make_float4(v[4], v[5], v[6], v[7]);
                        }
                    }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < kRows * (kCols / 4); i += kThreads) {
                const int r = i / (kCols / 4), c = 4 * (i % (kCols / 4));
                if (r >= rows) continue;
                float top = kNone;
                for (int k = 0; k < live; ++k) top = fmaxf(top, sm[(turn + k) & (kWarps - 1)][r]);
                float l = 0.f;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < live; ++k) {
                    const int wk = (turn + k) & (kWarps - 1);
                    const float f = ex2(sm[wk][r] - top);
                    const float4 x = *reinterpret_cast<const float4*>(merge + (wk * kRows + r) * kPitch + c);
                    l = fmaf(f, sl[wk][r], l);
                    v = make_float4(fmaf(f, x.x, v.x), fmaf(f, x.y, v.y), fmaf(f, x.z, v.z), fmaf(f, x.w, v.w));
                }
                if (whole) {
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    const int tok = (tile0 + r) / group, h = (tile0 + r) % group;
                    store4(static_cast<T*>(a.out) + (s.q0 + tok) * a.out_stride + (hk * group + h) * HD + c0 + c,
                           make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                } else {
                    *reinterpret_cast<float4*>(part_o + (out_slot * kRows + r) * HD + c0 + c) = v;
                    if (c0 + c == 0) part_ml[out_slot * kRows + r] = make_float2(top, l);
                }
            }
            __syncthreads();
        }
        done += n;
        ga = 0;
        ++c_at;
    }
    if (dead) {                                                          // copies in flight land before shared memory goes away
        for (int i = 0; i < kNst; ++i)
            if (lane == 0 && !mbar_wait(&bar[i], dead_phase ^ (i < dead_slot ? 1u : 0u))) report_error(kErrDrainTimeout);
    }
}

// Joins the partial sums of the tiles that more than one block shares, in block order.  Block (x, r): row r of the
// tile that the boundary between runs x and x + 1 cuts, if it is that tile's first boundary.  Rows of sequences
// without keys are written here too.
template <typename T, int HD, int PARTS, int MT>
__global__ void __launch_bounds__(HD) attn_join_kernel(const AttnArgs a, const float* __restrict__ part_o, const float2* __restrict__ part_ml,
                                                      int blocks) {
    constexpr int kRows = tile_rows<PARTS, MT>();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, group = a.q_heads / a.kv_heads;
    const int r = blockIdx.y;
    if (static_cast<int>(blockIdx.x) >= blocks - 1) {                    // the last column of blocks: outputs without keys
        for (int b = r; b < a.seqs; b += gridDim.y) {
            const int q0 = a.q_start[b], n = min(a.q_start[b + 1] - q0, a.max_q);
            if (a.kv_len[b] > 0) continue;
            for (int tok = 0; tok < n; ++tok)
                for (int h = 0; h < a.q_heads; ++h)
                    from_f32(static_cast<T*>(a.out) + (q0 + tok) * a.out_stride + h * HD + threadIdx.x, 0.f);
        }
        return;
    }
    const long long total = total_units(a, kRows, lane);
    const long long per = run_length(total, blocks);
    const int i = blockIdx.x + 1;
    const long long w = per * i;
    if (w >= total) return;
    long long first;
    const int b = locate(a, kRows, lane, w, first);
    const Seq s = load_seq(a, b, kRows);
    const int at = static_cast<int>((w - first) / s.groups);
    const long long begin = first + static_cast<long long>(at) * s.groups, end = begin + s.groups;
    if (begin >= w || begin < w - per) return;                           // not cut here, or cut earlier too
    const int tile0 = (at % s.tiles) * kRows;
    if (tile0 + r >= min(s.T, a.max_q) * group) return;
    const int last = static_cast<int>((end - 1) / per);
    float top = kNone, l = 0.f, v = 0.f;
    for (int k = i - 1; k <= last; ++k) {
        const size_t slot = 2 * k + (k == i - 1 ? 1 : 0);
        const float2 ml = part_ml[slot * kRows + r];
        const float x = part_o[(slot * kRows + r) * HD + threadIdx.x];
        const float up = fmaxf(top, ml.x), f = ex2(top - up), h = ex2(ml.x - up);
        l = fmaf(l, f, ml.y * h);
        v = fmaf(v, f, x * h);
        top = up;
    }
    const int tok = (tile0 + r) / group, h = (tile0 + r) % group, hk = at / s.tiles;
    from_f32(static_cast<T*>(a.out) + (s.q0 + tok) * a.out_stride + (hk * group + h) * HD + threadIdx.x, l == 0.f ? 0.f : v / l);
}

template <typename K, typename... A>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, int smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int HD, int PARTS, int MT>
cudaError_t rows_go(const AttnArgs& a, cudaStream_t s) {
    constexpr int kRows = tile_rows<PARTS, MT>(), smem = smem_bytes<HD, PARTS, MT>();
    static_assert(smem <= 227 * 1024, "shared memory");
    static bool configured = false;
    if (!configured) {
        const cudaError_t e = cudaFuncSetAttribute(attn_rows_kernel<T, HD, PARTS, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        configured = true;
    }
    const int gpp = a.page_size / kvGroup;
    int shift = -1;
    for (int i = 0; i < 16; ++i)
        if (gpp == 1 << i) shift = i;
    float* part_o = static_cast<float*>(a.workspace);
    float2* part_ml = reinterpret_cast<float2*>(part_o + static_cast<size_t>(2) * kBlocks * kRows * HD);
    const cudaError_t e = launch_dependent(attn_rows_kernel<T, HD, PARTS, MT>, dim3(kBlocks), kThreads, smem, s, a, part_o, part_ml, shift);
    if (e != cudaSuccess) return e;
    return launch_dependent(attn_join_kernel<T, HD, PARTS, MT>, dim3(kBlocks, kRows), HD, 0, s, a, part_o, part_ml, kBlocks);
}

// One 16-row (8-row for f32) tile where a kv head's rows fit it, else two of them at a time (head_dim 256: the
// accumulators leave no registers for the second).
template <typename T, int HD>
cudaError_t rows_type(const AttnArgs& a, cudaStream_t s) {
    constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
    const long long rows = static_cast<long long>(a.max_q) * (a.q_heads / a.kv_heads);
    if constexpr (HD < 256)
        if (rows > 16 / PARTS) return rows_go<T, HD, PARTS, 2>(a, s);
    return rows_go<T, HD, PARTS, 1>(a, s);
}

}  // namespace

size_t attn_workspace_bytes(int, int, int, int, int head_dim, int) {
    return static_cast<size_t>(2) * kBlocks * 32 * (head_dim + 2) * sizeof(float);      // 32: the largest tile's rows
}

cudaError_t launch_attn(const AttnArgs& a, int type, int head_dim, cudaStream_t s) {
    if (type == GQ_F32)
        return head_dim == 64 ? rows_type<float, 64>(a, s) : head_dim == 128 ? rows_type<float, 128>(a, s) : rows_type<float, 256>(a, s);
    if (type == GQ_F16)
        return head_dim == 64 ? rows_type<__half, 64>(a, s) : head_dim == 128 ? rows_type<__half, 128>(a, s) : rows_type<__half, 256>(a, s);
    return head_dim == 64    ? rows_type<__nv_bfloat16, 64>(a, s)
           : head_dim == 128 ? rows_type<__nv_bfloat16, 128>(a, s)
                             : rows_type<__nv_bfloat16, 256>(a, s);
}

}  // namespace gq
