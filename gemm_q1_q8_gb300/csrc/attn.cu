// Attention over the paged Q8_0 cache for few rows (decode, drafted trees).
//
// Mathematics: s = scale * q.k; o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m), one pass over the keys with the
// running maximum m (base 2).  Rows are a kv head's query heads times its query tokens (row = token * group + head).
// The floor is the cache's bytes (17/16 a value) at the HBM rate; a row costs 4 flops a value, so up to some 16 rows
// a read the matrix work hides behind the copy.
//
// Measured: one f32 token of 20 heads over 4096 tokens 11.8 us (latency: a chain of waits, ring, join); 32 f32 tokens over ragged 501 to 32768 tokens, 559 MB
// of cache, 108 us (5.2 TB/s, 76% of the measured copy; a scheduler issues in 55% of its cycles, 490 instructions a chunk); 8 bf16 trees of 9 to 33 tokens
// over 1111 to 9000 tokens 35 us (issue and latency: 490 instructions a chunk and 32 rows at 11 warps an SM, the cap's exponentials among them).
//
// Work: the unit is one 16-token chunk of one (sequence, kv head, row tile); the units of the whole call, in that order, are cut
// into equal runs of consecutive units, one a warp of every SM, whatever the sequences' lengths.  A warp goes through its run alone: it
// lays out a tile's queries in shared memory, takes the chunks from its own ring of bulk copies (a chunk is one contiguous copy),
// which one more warp of the block fills (its lane w for warp w), and writes the tiles that lie in its run.  A tile that runs share leaves
// partial sums: at the end of its run a warp's open tile meets those of the block's other warps, once; a second kernel joins what is left in
// the order of the runs, so the result does not depend on timing.
//
// Tensor cores: mma.sync m16n8k16 (f32 sums) with the queries as A and 8 keys as B.  Each code is its own exact 16-bit float: sign and
// 7-bit magnitude are the bits of the f16 subnormal magnitude * 2^-24, and of the bf16 one magnitude * 2^-133, so two codes become a
// register with one byte permute and one mask, and no conversion.  S: each 32-dim block has its own accumulator, multiplied by the
// key's scale in f32.  O: the weight times the value's scale is A, and the codes are B.
// 16-bit queries: one f16 part of each, 16 rows a tile, powers of two keeping A near the top of f16's range: a row's largest query value goes
// to 2^14..2^15, and so does its largest product of a weight and the exponent e of that token's largest value scale (below 2^e), because the
// running maximum is that of s + e.  A rounding costs 2^-12 of the product, or 2^-40 of the largest that the row has seen; hidden tokens
// and those of no weight do not count, whatever their scales are.
// f32 queries: 8 rows a tile; A has the high f16 part of the queries in its rows 0-7 and the rest in rows 8-15 (22 bits together); both halves
// of a row end in one thread, which adds them.  The weights take three bf16 parts (24 bits, the third in a product of its own) for f32's
// range: a weight of 2^-90 counts where the larger ones meet zero codes.
// Why not tcgen05 here: its tiles are 128 rows, and B comes from shared memory only, so the codes would be
// converted through shared memory for rows that are mostly absent.
#include "attn_join.cuh"

namespace gq {
GQ_ERROR_ACCESSOR(attn)
namespace {

// Rows a kv head (max_q tokens times its query heads) from which attn_tiles.cu takes the call.  32 query and 8 kv heads of 128, 8 sequences of
// 8192 tokens, this kernel against that one: f32 64 rows 214 / 136 us, 256 rows 805 / 249; bf16 64 rows 105 / 83, 128 rows 191 / 90, 16 rows
// 39 / 79.  16 bits: from one full 128-row tile, since max_q only bounds the rows (8 ragged trees of 27 to 99 rows: 35 / 45 us).  f32: from
// two tiles only, because up to there a weight below 2^-36 of the largest still counts here.
constexpr int many_rows(int type) { return type == GQ_F32 ? 256 : 128; }
constexpr int kBlocks = 152;                       // one thread block an SM

constexpr float kLift = 0x1p108f;                  // f32 weights are multiplied by it: times a scale below 2^16 and 2^kSlack they stay in f32's range
constexpr float kSlack = 2.f;                      // a score may pass the running maximum by this much before it moves: 1.02 (16 bits: 0)
// f32: chunks after which a tile's sums leave the registers, for the workspace.  An MMA truncates the sum that it adds to, always towards zero: 1024
// queries of 256 over 8192 tokens lost 6.7e-6 of the result, in plain f32 its error is 1.2e-6.  Every 16 / 32 / 64 chunks 2.7 / 2.1 / 2.0e-7 are lost at any
// length, for 110.9 / 109.1 / 108.2 us of 32 ragged sequences instead of 106.3 (each chunk's sums added outside the MMA: 110.8, and 8 sequences of 64
// rows 248 instead of 214 us).
constexpr int kDrain = 64;
// Rows of a tile by the parts of its operands: 16-bit queries 1; f32 2, or 3 for up to four rows
template <int PARTS, int MT> __host__ __device__ constexpr int tile_rows() { return PARTS == 1 ? 16 * MT : PARTS == 2 ? 8 * MT : 4; }
// Computing warps, by the registers that a warp's sums take, and the chunks of a warp's ring
template <int HD, int MT> __host__ __device__ constexpr int warps() { return HD * MT <= 64 ? 15 : HD * MT <= 128 ? 11 : 7; }
template <int HD, int MT> __host__ __device__ constexpr int stages() { return HD == 64 ? 4 : HD == 128 ? (MT == 1 ? 3 : 4) : 2; }
template <int HD, int MT> __host__ __device__ constexpr int ring_bytes() { return warps<HD, MT>() * stages<HD, MT>() * kv_chunk_bytes(HD); }
template <int HD, int MT> constexpr int smem_bytes() { return 1024 + ring_bytes<HD, MT>() + warps<HD, MT>() * MT * (HD / 16) * 512; }

// One sequence's share of the work.
struct Seq {
    int L, T, q0;          // cached tokens, query tokens, first query row
    int rows;              // that are computed, of a kv head
    int units;             // of one tile
    int tiles;             // row tiles a kv head
    __device__ __forceinline__ long long span(int kv_heads) const { return static_cast<long long>(units) * tiles * kv_heads; }
};
// ROWS a tile
template <int ROWS>
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b) {
    Seq s;
    const QueryRows q = query_rows(a, b);
    s.q0 = q.q0;
    s.T = q.T;
    s.L = a.kv_len[b];
    if (s.L > a.max_kv) report_error(kErrIndex);
    s.rows = q.tokens * (a.q_heads / a.kv_heads);
    s.units = (min(max(s.L, 0), a.max_kv) + kvGroup - 1) / kvGroup;
    s.tiles = (s.rows + ROWS - 1) / ROWS;
    return s;
}

// The units of all sequences, by one warp, and up to 32 sequences' own (this lane's) for locate().
template <int ROWS>
__device__ __forceinline__ long long total_units(const AttnArgs& a, int lane, long long& mine) {
    long long sum = 0;
    for (int b = lane; b < a.seqs; b += 32) sum += load_seq<ROWS>(a, b).span(a.kv_heads);
    mine = sum;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}
// The sequence that holds unit w, and its first unit.
template <int ROWS>
__device__ __forceinline__ int locate(const AttnArgs& a, int lane, long long w, long long mine, long long& first) {
    long long before = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += 32) {
        const int b = b0 + lane;
        if (a.seqs > 32) mine = b < a.seqs ? load_seq<ROWS>(a, b).span(a.kv_heads) : 0;
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
// c = a * b
__device__ __forceinline__ void mma16816_set(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// c += a * b
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
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

// A row of a tile, in shared memory
struct RowInfo {
    float rs;              // score multiplier: scale * log2(e) (or scale / softcap) and the powers of two taken out
    int last;              // causal: the last visible token; -1 for a row past the end
    uint32_t bits0, bits1; // tree: visible among the newest
};
// Bounded wait (~1 s) that also gives up when another warp has
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 16; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > 1000000000ull) {
            report_error(kErrWaitTimeout);
            *abort = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

// Requests the queries of m-tile mt of the tile from row tile0, and lays them out: fragments [k-step][lane], rows' multipliers and masks
template <typename T, int HD, int PARTS, int MT>
struct Queries {
    static constexpr int kKs = HD / 16, kSets = PARTS == 1 ? 2 : 1;
    using Raw = typename Vec4<T>::Raw;
    Raw raw[kSets][kKs];

    // The tile's row of this thread's set `set` of m-tile mt.  With three parts rows 0-3 stand twice.
    static __device__ __forceinline__ int row_of(int mt, int set, int g) {
        return PARTS == 1 ? 16 * mt + 8 * set + g : PARTS == 2 ? 8 * mt + g : g & 3;
    }
    __device__ __forceinline__ void request(const AttnArgs& a, const Seq& s, int hk, int tile0, int mt, int lane) {
        const int g = lane >> 2, t = lane & 3, group = a.q_heads / a.kv_heads;
#pragma unroll
        for (int set = 0; set < kSets; ++set) {
            const int r = tile0 + row_of(mt, set, g);
            const bool in = r < s.rows;
            const int tok = in ? r / group : 0, h = in ? r % group : 0;
            const T* q = static_cast<const T*>(a.q) + (s.q0 + tok) * a.q_stride + (hk * group + h) * HD;
#pragma unroll
            for (int ks = 0; ks < kKs; ++ks) raw[set][ks] = in ? *reinterpret_cast<const Raw*>(q + 16 * ks + 4 * t) : Raw{};
        }
    }
    __device__ __forceinline__ void lay(const AttnArgs& a, const Seq& s, int tile0, int mt, int lane, uint4* frag, RowInfo* info) const {
        const int g = lane >> 2, t = lane & 3, group = a.q_heads / a.kv_heads;
        float f[kSets];
#pragma unroll
        for (int set = 0; set < kSets; ++set) {
            float amax = 0.f;
#pragma unroll
            for (int ks = 0; ks < kKs; ++ks) {
                const float4 v = Vec4<T>::widen(raw[set][ks]);
                amax = fmaxf(amax, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // the largest value goes to [2^14, 2^15); not finite or zero: as it is
            const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
            const int up = amax > 0.f && e < 128 ? min(14 - e, 126) : 0;
            f[set] = pow2i(up);
            if (t == 0 && (PARTS != 3 || g < 4)) {
                const int r = tile0 + row_of(mt, set, g);
                const bool in = r < s.rows;
                const int tok = in ? r / group : 0;
                RowInfo ri;
                // 2^24 for the codes, 2^-up for the query; finite for queries near f32's largest value too, whose scores stay in their order
                const float rs = (a.softcap <= 0.f ? a.scale * kLog2e : a.scale / a.softcap * (PARTS > 1 ? 1.f : 2.f * kLog2e)) * 16777216.f * pow2i(-up);
                ri.rs = fminf(fmaxf(rs, -0x1p127f), 0x1p127f);
                ri.last = in ? s.L - s.T + tok : -1;
                const unsigned long long bits = a.tree && in ? a.tree[s.q0 + tok] : 0ull;
                ri.bits0 = static_cast<uint32_t>(bits);
                ri.bits1 = static_cast<uint32_t>(bits >> 32);
                info[row_of(mt, set, g)] = ri;
            }
        }
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks) {
            uint32_t q[4];
#pragma unroll
            for (int set = 0; set < kSets; ++set) {
                const float4 v = Vec4<T>::widen(raw[set][ks]);
                const float4 w = make_float4(v.x * f[set], v.y * f[set], v.z * f[set], v.w * f[set]);
                q[set] = pack2(w.x, w.y);
                q[2 + set] = pack2(w.z, w.w);
                if (PARTS > 1) {
                    const float2 x = unpack2(q[0]), y = unpack2(q[2]);
                    q[1] = pack2(w.x - x.x, w.y - x.y);
                    q[3] = pack2(w.z - y.x, w.w - y.y);
                }
            }
            frag[(mt * kKs + ks) * 32 + lane] = make_uint4(q[0], q[1], q[2], q[3]);
        }
    }
};

// A warp's sums over its units of a tile
template <typename T, int HD, int PARTS, int MT>
struct Tile {
    using Q = Queries<T, HD, PARTS, MT>;
    static constexpr int kKs = HD / 16, kNb = HD / 32, kSets = Q::kSets, kKeepers = PARTS == 3 ? 16 : 32;
    static constexpr float kEmpty = INFINITY;
    float o[MT][kNb][4][4];
    float m[MT][kSets], l[MT][kSets];
    RowInfo row[MT][kSets];
    // f32: what left the registers, relative to 2^m_kept, this thread's part of the run's place in the workspace
    float4* kept;
    float m_kept[MT];

    __device__ __forceinline__ void start(const RowInfo* info, int lane) {
        if (PARTS > 1) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) m_kept[mt] = kEmpty;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int set = 0; set < kSets; ++set) {
                row[mt][set] = info[Q::row_of(mt, set, lane >> 2)];
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
    }

    // Scales of this thread's four tokens (2t, 2t + 1, 2t + 8, 2t + 9), [token][block] in halves; tokens from `end` on have none
    static __device__ __forceinline__ void load_scales(const uint8_t* p, int t, int end, uint32_t (&w)[kNb * 2]) {
#pragma unroll
        for (int i = 0; i < kNb / 2; ++i) *reinterpret_cast<uint4*>(w + 4 * i) = *reinterpret_cast<const uint4*>(p + t * 8 * kNb + 16 * i);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (2 * t + (k & 1) + 8 * (k >> 1) >= end)
#pragma unroll
                for (int i = 0; i < kNb / 2; ++i) w[k * kNb / 2 + i] = 0u;
    }
    static __device__ __forceinline__ float scale_of(const uint32_t (&w)[kNb * 2], int k, int b) {
        const float2 v = unpack2(w[(k * kNb + b) / 2]);
        return b & 1 ? v.y : v.x;
    }

    // One chunk, its first token j0.  MASKED: some of its tokens are new or past the end.
    template <bool MASKED>
    __device__ __forceinline__ void unit(const AttnArgs& a, const Seq& s, const uint8_t* __restrict__ ch, const uint4* __restrict__ frag, int j0,
                                         bool have, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const int len = have ? min(s.L, a.max_kv) : 0, end = MASKED ? len - j0 : 16;
        float S[MT][2][4];
        {
            uint32_t ksw[kNb * 2];
            load_scales(ch + kv_ks_offset(HD), t, end, ksw);
#pragma unroll
            for (int c = 0; c < kKs / 4; ++c) {
                uint32_t w[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    int at = 4 * c + t;
                    if (HD > 64) at ^= 4 * (g & 1);
                    *reinterpret_cast<uint4*>(w[j]) = *reinterpret_cast<const uint4*>(ch + (8 * j + g) * HD + at * 16);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int b = 2 * c + h;
                    uint32_t k[2][4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        k[j][0] = codes2(w[j][2 * h], 0, 0x1100);
                        k[j][1] = codes2(w[j][2 * h], 0, 0x3322);
                        k[j][2] = codes2(w[j][2 * h + 1], 0, 0x1100);
                        k[j][3] = codes2(w[j][2 * h + 1], 0, 0x3322);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const uint4 q0 = frag[(mt * kKs + 2 * b) * 32 + lane], q1 = frag[(mt * kKs + 2 * b + 1) * 32 + lane];
                        const uint32_t a0[4] = {q0.x, q0.y, q0.z, q0.w}, a1[4] = {q1.x, q1.y, q1.z, q1.w};
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float p[4];
                            mma16816_set(p, a0, k[j][0], k[j][1]);
                            mma16816(p, a1, k[j][2], k[j][3]);
                            const float k0 = scale_of(ksw, 2 * j, b), k1 = scale_of(ksw, 2 * j + 1, b);
                            float (&x)[4] = S[mt][j];
                            x[0] = b ? fmaf(k0, p[0], x[0]) : k0 * p[0];
                            x[1] = b ? fmaf(k1, p[1], x[1]) : k1 * p[1];
                            x[2] = b ? fmaf(k0, p[2], x[2]) : k0 * p[2];
                            x[3] = b ? fmaf(k1, p[3], x[3]) : k1 * p[3];
                        }
                    }
                }
            }
        }
        uint32_t vsw[kNb * 2];
        load_scales(ch + kv_vs_offset(HD), t, end, vsw);
        // 16 bits: the exponent of each token's largest value scale
        float vexp[4];
        if (PARTS == 1) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t v = vsw[k * kNb / 2] & 0x7fff7fffu;
#pragma unroll
                for (int i = 1; i < kNb / 2; ++i) v = __vmaxu2(v, vsw[k * kNb / 2 + i] & 0x7fff7fffu);
                vexp[k] = static_cast<float>(static_cast<int>(max(v & 0xffffu, v >> 16) >> 10) - 14);
            }
        }
        // scores to weights, which carry a power of two: 16 bits 2^15 in the exponent's argument, f32 as a factor (an argument near 108 would have
        // steps of 2^-17)
        float P[MT][kSets][4];                                   // [row][token of the thread's four]
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int set = 0; set < kSets; ++set)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    float x = S[mt][p >> 1][2 * set + (p & 1)];
                    if (PARTS > 1) x += S[mt][p >> 1][2 + (p & 1)];
                    P[mt][set][p] = x * row[mt][set].rs;
                }
            if (a.softcap > 0.f) {
                const float cap = a.softcap * kLog2e;
                if (PARTS == 1 && a.softcap > kCapNear) {
#pragma unroll
                    for (int set = 0; set < kSets; ++set)
#pragma unroll
                        for (int p = 0; p < 4; ++p) P[mt][set][p] = capped16<true>(P[mt][set][p], cap);
                } else {
#pragma unroll
                    for (int set = 0; set < kSets; ++set)
#pragma unroll
                        for (int p = 0; p < 4; ++p) P[mt][set][p] = PARTS > 1 ? cap * tanhf(P[mt][set][p]) : capped16<false>(P[mt][set][p], cap);
                }
            }
            if (MASKED) {
#pragma unroll
                for (int set = 0; set < kSets; ++set)
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const RowInfo& ri = row[mt][set];
                        const int j = j0 + 2 * t + (p & 1) + 8 * (p >> 1);
                        const int rel = j - (s.L - s.T);
                        bool seen = ri.last >= 0 && j < len;
                        if (a.tree) {
                            const uint32_t word = rel < 32 ? ri.bits0 : ri.bits1;
                            seen = seen && (rel < 0 || (rel < 64 && ((word >> (rel & 31)) & 1u)));
                        } else {
                            seen = seen && j <= ri.last;
                        }
                        if (!seen) P[mt][set][p] = -INFINITY;
                    }
            }
            float top[kSets];
            bool higher = false;
#pragma unroll
            for (int set = 0; set < kSets; ++set) {
                if (PARTS == 1)
                    top[set] = fmaxf(fmaxf(P[mt][set][0] + vexp[0], P[mt][set][1] + vexp[1]), fmaxf(P[mt][set][2] + vexp[2], P[mt][set][3] + vexp[3]));
                else
                    top[set] = fmaxf(fmaxf(P[mt][set][0], P[mt][set][1]), fmaxf(P[mt][set][2], P[mt][set][3]));
                higher |= top[set] > m[mt][set] + (PARTS == 1 ? 0.f : kSlack);
            }
            if (__any_sync(0xffffffffu, higher)) {
#pragma unroll
                for (int set = 0; set < kSets; ++set) {
                    float up = fmaxf(top[set], __shfl_xor_sync(0xffffffffu, top[set], 1));
                    up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 2));
                    up = fmaxf(up, m[mt][set]);
                    const float down = ex2(m[mt][set] - up);
                    m[mt][set] = up;
                    l[mt][set] *= down;
                    // rows g and g + 8 of the accumulators; of more parts both belong to row g, or with three parts its copy
#pragma unroll
                    for (int c = 0; c < kNb; ++c)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
#pragma unroll
                            for (int i = 0; i < (PARTS == 1 ? 2 : 4); ++i) o[mt][c][x][2 * set + i] *= down;
                }
            }
#pragma unroll
            for (int set = 0; set < kSets; ++set) {
                const float from = PARTS == 1 ? m[mt][set] - 15.f : m[mt][set];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const float x = ex2(P[mt][set][p] - from);
                    P[mt][set][p] = PARTS == 1 ? x : x * kLift;
                    l[mt][set] = PARTS == 1 ? fmaf(x, 0x1p-15f, l[mt][set]) : l[mt][set] + x;
                }
            }
        }
        // values: words [token][block], four dims each
        uint32_t w[4][kNb];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint8_t* r = ch + kv_v_offset(HD) + (4 * p + t) * HD;
            if (HD == 64) {
                *reinterpret_cast<uint2*>(w[p]) = *reinterpret_cast<const uint2*>(r + 8 * (g ^ (4 * (t >> 1))));
            } else {
#pragma unroll
                for (int h = 0; h < HD / 128; ++h)
                    *reinterpret_cast<uint4*>(w[p] + 4 * h) = *reinterpret_cast<const uint4*>(r + 128 * h + 16 * (g ^ (2 * t)));
            }
        }
#pragma unroll
        for (int c = 0; c < kNb; ++c) {
            uint32_t pa[MT][4], low[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int set = 0; set < kSets; ++set) {
                    float z[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        z[p] = P[mt][set][p] * scale_of(vsw, p, c);
                        if (MASKED && P[mt][set][p] == 0.f) z[p] = 0.f;      // whatever the masked value's scale is
                    }
                    if (PARTS == 1) {
                        pa[mt][set] = pack2(z[0], z[1]);
                        pa[mt][2 + set] = pack2(z[2], z[3]);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float x = z[2 * h], y = z[2 * h + 1];
                            const uint32_t hi = pack2_bf16(x, y);
                            x -= __uint_as_float(hi << 16);
                            y -= __uint_as_float(hi & 0xffff0000u);
                            const uint32_t mid = pack2_bf16(x, y);
                            x -= __uint_as_float(mid << 16);
                            y -= __uint_as_float(mid & 0xffff0000u);
                            const uint32_t lo = pack2_bf16(x, y);
                            if (PARTS == 2) {
                                pa[mt][2 * h] = hi;
                                pa[mt][2 * h + 1] = mid;
                                low[mt][h] = lo;
                            } else {                          // rows 0-3 the high parts, 4-7 the middle ones, 8-11 the low ones
                                pa[mt][2 * h] = g < 4 ? hi : mid;
                                pa[mt][2 * h + 1] = lo;       // again in rows 12-15, which nothing reads
                            }
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
                        if (PARTS == 2) mma16816_bf16(o[mt][c][e], low[mt][0], 0u, low[mt][1], 0u, b0, b1);
                    }
                }
            }
        }
    }

    // The two float4 of block c: columns 8t .. and 8t + 4 .. of the row, its parts added
    __device__ __forceinline__ void sums(int mt, int c, int set, int g, float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = o[mt][c][e][2 * set + i];
                if (PARTS == 2 || (PARTS == 3 && g < 4)) x += o[mt][c][e][2 + i];
                if (PARTS == 3) x += __shfl_xor_sync(0xffffffffu, x, 16);
                v[4 * i + e] = x;
            }
    }
    __device__ __forceinline__ void add_kept(int mt, int c, float f, float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 k = kept[((mt * kNb + c) * 2 + i) * kKeepers];
            v[4 * i] = fmaf(k.x, f, v[4 * i]);
            v[4 * i + 1] = fmaf(k.y, f, v[4 * i + 1]);
            v[4 * i + 2] = fmaf(k.z, f, v[4 * i + 2]);
            v[4 * i + 3] = fmaf(k.w, f, v[4 * i + 3]);
        }
    }
    // f32: the sums go to the workspace
    __device__ __forceinline__ void drain(int lane) {
        const int g = lane >> 2;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const bool before = m_kept[mt] != kEmpty;
            const float f = ex2(m_kept[mt] - m[mt][0]);
#pragma unroll
            for (int c = 0; c < kNb; ++c) {
                float v[8];
                sums(mt, c, 0, g, v);
                if (lane < kKeepers) {
                    if (before) add_kept(mt, c, f, v);
                    kept[(mt * kNb + c) * 2 * kKeepers] = make_float4(v[0], v[1], v[2], v[3]);
                    kept[((mt * kNb + c) * 2 + 1) * kKeepers] = make_float4(v[4], v[5], v[6], v[7]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[mt][c][e][i] = 0.f;
            }
            m_kept[mt] = m[mt][0];
        }
    }

    // This warp's sums of a row to dst(row), four columns at a time; `norm`: divided by the row's sum
    template <typename F>
    __device__ __forceinline__ void put(int lane, bool norm, F&& store) const {
        const int g = lane >> 2, t = lane & 3;
        // 2^133 (2^24) for the codes, and the power of two of the weights
        constexpr float back = PARTS == 1 ? 0x1p9f : 0x1p25f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int set = 0; set < kSets; ++set) {
                float sum = l[mt][set];                                  // over the four threads that share the row
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                const float f = !norm ? back : sum == 0.f ? 0.f : back / sum;
#pragma unroll
                for (int c = 0; c < kNb; ++c) {
                    float v[8];
                    sums(mt, c, set, g, v);
                    if (PARTS > 1)
                        if (m_kept[mt] != kEmpty && lane < kKeepers) add_kept(mt, c, ex2(m_kept[mt] - m[mt][set]), v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] *= f;
                    if (PARTS != 3 || g < 4) {
                        store(Q::row_of(mt, set, g), 32 * c + 8 * t, make_float4(v[0], v[1], v[2], v[3]), m[mt][set], sum);
                        store(Q::row_of(mt, set, g), 32 * c + 8 * t + 4, make_float4(v[4], v[5], v[6], v[7]), m[mt][set], sum);
                    }
                }
            }
    }
};

// A place in the order of the units: unit g of tile `at` ((kv head, row tile)) of sequence b
template <int ROWS>
struct Place {
    Seq s;
    int b, at, g;
    // On from a tile's end to the next tile
    __device__ __forceinline__ void next_tile(const AttnArgs& a) {
        g = 0;
        if (++at >= s.tiles * a.kv_heads) {
            at = 0;
            do s = load_seq<ROWS>(a, ++b); while (s.units == 0 || s.tiles == 0);
        }
    }
};

template <typename T, int HD, int PARTS, int MT>
__global__ void __launch_bounds__((warps<HD, MT>() + 1) * 32, 1) attn_rows_kernel(const AttnArgs a, const Parts parts, int page_shift) {
    using TileT = Tile<T, HD, PARTS, MT>;
    using QT = typename TileT::Q;
    constexpr int kWarps = warps<HD, MT>(), kRows = tile_rows<PARTS, MT>(), kNst = stages<HD, MT>(), kChunk = kv_chunk_bytes(HD);
    constexpr int kFrags = MT * (HD / 16) * 32, kPitch = HD + 4;
    static_assert(2 * kWarps * kNst * 8 <= 1024 && kWarps * kRows * kPitch * 4 <= ring_bytes<HD, MT>(), "shared memory");
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem);                              // [kWarps][kNst] full, [kWarps][kNst] empty
    uint8_t* ring = smem + 1024;                                                     // [kWarps][kNst][kChunk]
    uint4* frag_all = reinterpret_cast<uint4*>(ring + kWarps * kNst * kChunk);       // [kWarps][MT][HD / 16][32]
    float* merge = reinterpret_cast<float*>(ring);                                   // at the end: [kWarps][kRows][kPitch]
    __shared__ RowInfo info_all[kWarps][kRows];
    __shared__ float sm[kWarps][kRows], sl[kWarps][kRows];
    __shared__ uint8_t have[kWarps][kNst];                                           // whether a ring slot's page exists
    __shared__ long long open[kWarps];                                               // the first unit of the tile that a warp's run ends in, or -1
    __shared__ volatile int abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < 2 * kWarps * kNst) mbar_init(&bars[threadIdx.x], 1);
    if (threadIdx.x == 0) abort = 0;
    fence_barrier_init();
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    long long own;
    const long long total = total_units<kRows>(a, lane, own);
    constexpr int kRunsAll = kBlocks * kWarps;
    const long long per = max((total + kRunsAll - 1) / kRunsAll, 1ll);
    const int gpp = a.page_size / kvGroup;

    if (warp == kWarps) {
        // ---- the fetching warp: lane w requests the units of warp w's run into its ring
        const long long w0 = per * (static_cast<long long>(blockIdx.x) * kWarps + lane);
        const int count = lane < kWarps && w0 < total ? static_cast<int>(min(total - w0, per)) : 0;
        Place<kRows> p;
        {
            // the block's first unit is found by the warp together; each lane goes on from there
            const long long first_unit = per * blockIdx.x * kWarps;
            if (first_unit >= total) return;
            long long first;
            p.b = locate<kRows>(a, lane, first_unit, own, first);
            p.s = load_seq<kRows>(a, p.b);
            if (count) {
                long long rest = w0 - first;
                while (rest >= p.s.span(a.kv_heads)) {
                    rest -= p.s.span(a.kv_heads);
                    p.s = load_seq<kRows>(a, ++p.b);
                }
                div_mod(rest, p.s.units, p.at, p.g);
            }
        }
        int fetched = 0, slot = 0, page = -1, off = 0;
        uint32_t parity = 1;                                             // of a ring's first round: nothing to wait for
        auto look_up = [&]() {                                           // used at the next fetch, not waited for here
            const int pi = page_shift >= 0 ? p.g >> page_shift : p.g / gpp;
            off = p.g - pi * gpp;
            page = a.table[static_cast<size_t>(p.b) * a.table_stride + pi];
        };
        if (count) look_up();
        uint64_t since = globaltimer_ns();
        while (__any_sync(0xffffffffu, fetched < count)) {
            bool did = false;
            if (fetched < count) {
                uint64_t* full = &bars[lane * kNst + slot];
                if (mbar_test(full + kWarps * kNst, parity)) {
                    const bool there = page >= 0 && page < a.pages;
                    have[lane][slot] = there;
                    if (there) {
                        mbar_arrive_expect_tx(full, kChunk);
                        bulk_g2s(ring + (lane * kNst + slot) * kChunk,
                                 a.cache + ((static_cast<size_t>(page) * a.kv_heads + p.at / p.s.tiles) * gpp + off) * kChunk, kChunk, full);
                    } else {
                        report_error(kErrIndex);
                        mbar_arrive(full);
                    }
                    if (++slot == kNst) {
                        slot = 0;
                        parity ^= 1;
                    }
                    if (++fetched < count) {
                        if (++p.g == p.s.units) p.next_tile(a);
                        look_up();
                    }
                    did = true;
                }
            }
            if (__any_sync(0xffffffffu, did)) {
                since = globaltimer_ns();
            } else {
                __nanosleep(32);
                if (__any_sync(0xffffffffu, abort || globaltimer_ns() - since > 2000000000ull)) break;    // a computing warp reports its own wait
            }
        }
        if (abort)                                                       // copies in flight land before shared memory goes away
            for (int i = 0; i < kNst; ++i) {
                const int times = (fetched + kNst - 1 - i) / kNst;
                if (times && !mbar_wait(&bars[lane * kNst + i], (times - 1) & 1)) report_error(kErrDrainTimeout);
            }
        return;
    }

    // ---- the computing warps: each its own run
    const int run = blockIdx.x * kWarps + warp, group = a.q_heads / a.kv_heads;
    const long long w0 = per * run;
    const int count = w0 < total ? static_cast<int>(min(total - w0, per)) : 0;
    uint4* frag = frag_all + warp * kFrags;
    RowInfo* info = info_all[warp];
    Head head = {-1, 0, 0, 0, 0};
    long long open_at = -1;
    if (count) {
        TileT tile;
        // until the block's warps meet, the place of the run's tail is free for its own sums
        if (PARTS > 1) tile.kept = reinterpret_cast<float4*>(parts.o + (static_cast<size_t>(kRunsAll) + run) * kRows * HD) + lane;
        uint64_t* full = &bars[warp * kNst];
        const uint8_t* ring_w = ring + warp * kNst * kChunk;
        int slot = 0;
        uint32_t phase = 0;
        Place<kRows> p;
        long long first;                                                 // the first unit of the tile
        p.b = locate<kRows>(a, lane, w0, own, first);
        p.s = load_seq<kRows>(a, p.b);
        div_mod(w0 - first, p.s.units, p.at, p.g);
        first = w0 - p.g;
        bool ok = true;
        for (int done = 0; ok;) {
            const int tile0 = (p.at % p.s.tiles) * kRows, hk = p.at / p.s.tiles;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                QT q;
                q.request(a, p.s, hk, tile0, mt, lane);
                q.lay(a, p.s, tile0, mt, lane, frag, info);
            }
            __syncwarp();
            tile.start(info, lane);
            const int end = min(p.s.units, p.g + count - done);
            const bool begun_here = p.g == 0;
            // units from here on hold new tokens, or the end
            const int old = min(p.s.L - p.s.T, a.max_kv), masked = old > 0 ? old / kvGroup : 0;
            done += end - p.g;
            for (int i = p.g, until;;) {
                for (until = PARTS > 1 ? min(end, i + kDrain) : end; i < until; ++i) {
                    if (!wait_for(&full[slot], phase, &abort)) {
                        ok = false;
                        break;
                    }
                    __syncwarp();
                    const uint8_t* ch = ring_w + slot * kChunk;
                    if (i >= masked)
                        tile.template unit<true>(a, p.s, ch, frag, i * kvGroup, have[warp][slot], lane);
                    else if (have[warp][slot])
                        tile.template unit<false>(a, p.s, ch, frag, 0, true, lane);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[kWarps * kNst + slot]);
                    if (++slot == kNst) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (PARTS == 1 || !ok || i >= end) break;
                tile.drain(lane);
            }
            if (!ok) break;
            if (end == p.s.units && begun_here) {                        // all of the tile
                const int rows = p.s.rows - tile0;
                T* out = static_cast<T*>(a.out) + p.s.q0 * a.out_stride + hk * group * HD;
                tile.put(lane, true, [&](int r, int c, float4 v, float, float) {
                    if (r < rows) store4(out + ((tile0 + r) / group) * a.out_stride + ((tile0 + r) % group) * HD + c, v);
                });
            } else if (end == p.s.units) {                               // its end: for the second kernel
                int begun, unused;
                div_mod(first, static_cast<int>(per), begun, unused);
                head = {begun, p.s.q0, tile0, min(p.s.rows - tile0, kRows), hk};
                tile.put(lane, false, [&](int r, int c, float4 v, float m, float l) {
                    const size_t at = static_cast<size_t>(run) * kRows + r;
                    *reinterpret_cast<float4*>(parts.o + at * HD + c) = v;
                    if (c == 0) parts.ml[at] = make_float2(m, l);
                });
            } else {
                open_at = first;
            }
            if (done == count) break;
            first += p.s.units;
            p.next_tile(a);
        }
        if (!ok) open_at = -1;
        if (lane == 0) open[warp] = open_at;
        // every warp's ring has been read: the open tiles meet there
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        if (open_at >= 0)
            tile.put(lane, false, [&](int r, int c, float4 v, float m, float l) {
                *reinterpret_cast<float4*>(merge + (warp * kRows + r) * kPitch + c) = v;
                if (c == 0) {
                    sm[warp][r] = m;
                    sl[warp][r] = l;
                }
            });
    } else {
        if (lane == 0) open[warp] = -1;
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
    }
    if (lane == 0) parts.head[run] = head;
    asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
    // neighbours in the same tile are joined; the sum is the tail of the first of them
    for (int w = 0; w < kWarps;) {
        const long long which = open[w];
        int n = 1;
        while (w + n < kWarps && which >= 0 && open[w + n] == which) ++n;
        if (which >= 0)
            for (int i = threadIdx.x; i < kRows * (HD / 4); i += kWarps * 32) {
                const int r = i / (HD / 4), c = 4 * (i % (HD / 4));
                float top = kNone;
                for (int k = 0; k < n; ++k) top = fmaxf(top, sm[w + k][r]);
                float l = 0.f;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < n; ++k) {
                    const float f = ex2(sm[w + k][r] - top);
                    const float4 x = *reinterpret_cast<const float4*>(merge + ((w + k) * kRows + r) * kPitch + c);
                    l = fmaf(f, sl[w + k][r], l);
                    v = make_float4(fmaf(f, x.x, v.x), fmaf(f, x.y, v.y), fmaf(f, x.z, v.z), fmaf(f, x.w, v.w));
                }
                const size_t at = (static_cast<size_t>(kRunsAll) + blockIdx.x * kWarps + w) * kRows + r;
                *reinterpret_cast<float4*>(parts.o + at * HD + c) = v;
                if (c == 0) parts.ml[at] = make_float2(top, l);
            }
        w += n;
    }
}

template <typename T, int HD, int PARTS, int MT>
cudaError_t rows_go(const AttnArgs& a, cudaStream_t s) {
    constexpr int kRows = tile_rows<PARTS, MT>(), kWarps = warps<HD, MT>(), smem = smem_bytes<HD, MT>();
    static_assert(smem <= 220 * 1024, "shared memory");
    static std::atomic<uint64_t> raised{0};
    cudaError_t e = allow_smem(attn_rows_kernel<T, HD, PARTS, MT>, smem, raised);
    if (e != cudaSuccess) return e;
    const int gpp = a.page_size / kvGroup;
    int shift = -1;
    for (int i = 0; i < 16; ++i)
        if (gpp == 1 << i) shift = i;
    const Parts parts = parts_at(a.workspace, kBlocks * kWarps, kRows, HD);
    e = launch_dependent(attn_rows_kernel<T, HD, PARTS, MT>, dim3(kBlocks), (kWarps + 1) * 32, smem, s, a, parts, shift);
    if (e != cudaSuccess) return e;
    return launch_join<T, HD, kRows, kWarps>(a, parts, kBlocks * kWarps, s);
}
template <int HD, int PARTS, int MT>
size_t rows_bytes() {
    return parts_bytes(kBlocks * warps<HD, MT>(), tile_rows<PARTS, MT>(), HD);
}

// One 16-row (8-row for f32) tile where a kv head's rows fit it, else two of them at a time (head_dim 256: the
// accumulators leave no registers for the second).  Up to four f32 rows take all three parts of a weight in one product.
template <typename T, int HD>
cudaError_t rows_type(const AttnArgs& a, cudaStream_t s) {
    constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
    const long long rows = static_cast<long long>(a.max_q) * (a.q_heads / a.kv_heads);
    if constexpr (PARTS == 2)
        if (rows <= 4) return rows_go<T, HD, 3, 1>(a, s);
    if constexpr (HD < 256)
        if (rows > 16 / PARTS) return rows_go<T, HD, PARTS, 2>(a, s);
    return rows_go<T, HD, PARTS, 1>(a, s);
}
template <typename T, int HD>
size_t rows_type_bytes(long long rows) {
    constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
    if constexpr (PARTS == 2)
        if (rows <= 4) return rows_bytes<HD, 3, 1>();
    if constexpr (HD < 256)
        if (rows > 16 / PARTS) return rows_bytes<HD, PARTS, 2>();
    return rows_bytes<HD, PARTS, 1>();
}

}  // namespace

size_t attn_workspace_bytes(int, int max_q, int q_heads, int kv_heads, int head_dim, int type) {
    const long long rows = static_cast<long long>(max_q) * (q_heads / kv_heads);
    if (head_dim <= 128 && rows >= many_rows(type)) return attn_tiles_workspace_bytes(head_dim, type);
    if (type == GQ_F32)
        return head_dim == 64 ? rows_type_bytes<float, 64>(rows) : head_dim == 128 ? rows_type_bytes<float, 128>(rows) : rows_type_bytes<float, 256>(rows);
    return head_dim == 64 ? rows_type_bytes<__half, 64>(rows) : head_dim == 128 ? rows_type_bytes<__half, 128>(rows) : rows_type_bytes<__half, 256>(rows);
}

cudaError_t launch_attn(const AttnArgs& a, int type, int head_dim, cudaStream_t s) {
    if (head_dim <= 128 && static_cast<long long>(a.max_q) * (a.q_heads / a.kv_heads) >= many_rows(type)) return launch_attn_tiles(a, type, head_dim, s);
    if (type == GQ_F32)
        return head_dim == 64 ? rows_type<float, 64>(a, s) : head_dim == 128 ? rows_type<float, 128>(a, s) : rows_type<float, 256>(a, s);
    if (type == GQ_F16)
        return head_dim == 64 ? rows_type<__half, 64>(a, s) : head_dim == 128 ? rows_type<__half, 128>(a, s) : rows_type<__half, 256>(a, s);
    return head_dim == 64    ? rows_type<__nv_bfloat16, 64>(a, s)
           : head_dim == 128 ? rows_type<__nv_bfloat16, 128>(a, s)
                             : rows_type<__nv_bfloat16, 256>(a, s);
}

}  // namespace gq
