// Attention over the paged Q8_0 cache for many rows (prefill chunks): 128 rows a thread block on the 5th-generation tensor cores.
//
// Mathematics as attn.cu: s = scale * q.k, o = sum 2^(s - m) v / sum 2^(s - m), rows (token * group + head) of one kv head, one pass over the
// keys in tiles of 64.  Bound: the tensor cores, 4 * hd flops a visible pair (three times that for f32), and the softmax's exponentials.
// Measured (2048 queries of 32 heads of 128 over 6144 tokens with them, 8 kv heads): f32 603 us (285 TFLOP/s of the formula, 855 of MMAs; 274 us at the
// measured rate), bf16 343 us.  A 64-token score MMA holds the tensor core for 48 cycles, a 128-token one for 64, so a tile's MMAs take 1920 cycles
// in f32 (128-token tiles would need 1536, and tensor memory that the queries and sums fill); a tile takes 4100, of which a scheduler
// issues in 1710: the rest is the chain scores - softmax - sums, the pieces' ends, and the drains below.
//
// Operands (kind::f16, f32 sums): the queries (A) and the weights (A) lie in tensor memory, written there by the softmax's threads, a row a
// thread; keys and values (B) in shared memory (128-byte swizzle), converted from the cache's codes by eight warps.  With A in tensor
// memory a 128 x 64 x 16 MMA reads 2 KB of shared memory instead of 6, which would bound it.
// A code is the f16 subnormal magnitude * 2^-24 (attn.cu); times 2^15 it is normal, times the scale it is the value, rounded once to f16; and
// fma(code, scale, -value) is the exact rest: two f16 parts hold all 18 bits.  f32 queries take two parts of everything and three
// products (high x high, low x high, high x low): 2^-22 of a term.  16-bit queries take one part: 2^-11.
//
// Powers of two keep the parts in f16's range.  A row's largest query goes to 2^14, its largest weight to 2^11 (2^15 before its maximum moves; a weight
// is off by up to 2^-36 of it besides its bits, the row kernel keeps the faint ones).  A tile's keys are divided by 2^e, e the exponent of its
// largest scale, its values by 2^ref, ref at most kAbove more than theirs; the sums are relative to ref and move with it, up or down, so what one tile
// holds takes nothing of another's range.  Within a tile the tokens' exponents may differ by kNear: a key or value is then off by up to 2^-22 of its
// token's largest besides its bits.  Where they differ by more, each token is divided by its own 2^e, which comes back on its column of scores and
// in its weights, and each row's sums are relative to the largest product of a weight and 2^e that it sees (wide_tile): a token that a row does
// not see, or that has no weight there, takes nothing of the others' range either, whatever its scale is.  The common way pays for that with 581 -> 603 us
// (f32 below), 333 -> 343 (bf16); with every other tile wide the chunk takes 706 (414).
//
// Keys' and values' orders are free where they are contracted: dims stand in the order in which a 16-byte unit of the cache holds them
// (the queries' too), tokens in the order of the cache's value rows (the score columns too), so both conversions go from words to 16-byte
// chunks without moving single bytes.
//
// Work: the key tiles of every (sequence, kv head, row tile) are cut into one equal run a thread block (attn_join.cuh), so 512 row tiles
// leave no SM idle, and few rows over a long context use them all.
//
//   warps 0-7   softmax, two groups that take every other tile, each with a running maximum and sums (in tensor memory) of its own, joined at
//               the end: scores from tensor memory, a row a thread (so no shuffles), the weights into the scores' place; the maximum moves
//               (and the sums are multiplied) only where a row's scores pass it by 2^kSlack
//   warps 8-15  keys and values of a tile, two stages
//   warp 16     MMA issue of the scores: those of tile i + 2 into the place of the weights of tile i, once its sums are done
//   warp 17     MMA issue of the sums
//   warp 18     bulk copies of the chunks, two stages
//   warp 19     the run's pieces (in a ring that the other roles read), and the exponents of a tile's scales
#include "attn_join.cuh"
#include "tc_common.cuh"

namespace gq {
GQ_ERROR_ACCESSOR(attn_tiles)
namespace {

constexpr int kRows = 128, kTok = 64, kGroups = kTok / kvGroup;
constexpr int kWarpKV = 8, kNumKV = 8, kWarpMma = 16, kThreads = 20 * 32;
// Registers a thread of each warpgroup, out of the 5 x 96 that a launch of 640 threads has: two softmax groups, two of keys and values, one
constexpr int kRegsSoftmax = 136, kRegsKV = 72, kRegsRest = 64;
static_assert(2 * kRegsSoftmax + 2 * kRegsKV + kRegsRest == 5 * 96, "registers");
constexpr int kBlocks = 152;                               // one thread block an SM
constexpr float kLift = 11.f, kSlack = 4.f;
constexpr int kNear = 12, kAbove = 3;              // how far the exponents of a tile's tokens may differ, and ref be above the values'
constexpr int kOwn = 100;                          // in the place of a tile's exponent: each token has its own
constexpr int kColS = 0, kColQ = 128, kColO = 256, kTmemCols = 512;        // scores (weights) 2 x 64, queries 128, sums 2 x 128
// f32: a group's sums leave tensor memory every kDrain of its tiles, for f32 sums in the workspace.  An MMA truncates the sum that it adds to,
// always towards zero, 12 times a tile: over 6144 tokens (48 tiles a group) the result lost 9.8e-6 of itself, against 1.7e-6 in plain f32.  Every
// 4 / 8 / 16 tiles, with the small products of the scores first: 1.5e-6 / 2.3e-6 / 3.8e-6, at any length, for 619 / 581 / 563 us instead of 543 (every 8 tiles 603 us since, see above).
// 16 bits (4 MMAs a tile) lose half of f16's last place at some 400,000 tokens: not drained (the code alone would cost 4-6%, by its registers).
constexpr int kDrain = 8;

__device__ __forceinline__ uint32_t u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 h2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ uint32_t codes2(uint32_t lo, uint32_t hi, uint32_t sel) { return __byte_perm(lo, hi, sel) & 0x807f807fu; }

// Bounded wait (~1 s) that also gives up when another role has.  Small, because it stands in many places and the roles' code together
// should stay in the instruction caches.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity)) return true;
        if (*abort) return false;
        if (__builtin_expect(globaltimer_ns() - t0 > 1000000000ull, 0)) {
            report_error(kErrMmaTimeout);
            *abort = 1;
            return false;
        }
    }
}

template <int N>
__device__ __forceinline__ constexpr uint32_t idesc() {                   // D f32, A and B f16, both K-major, M = 128
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
}
// One MMA, its B descriptor in halves (the low one moves by constants from MMA to MMA: little is left to issue per MMA)
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t desc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b_lo), "r"(b_hi), "r"(desc), "r"(accumulate)
        : "memory");
}
// 32 columns of this thread's TMEM lane
__device__ __forceinline__ void tc_ld32(uint32_t taddr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
          "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// 16 columns of it
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
          "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 16 columns
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Column n of a tile's scores holds this token of the tile
__device__ __forceinline__ constexpr int token_of(int n) { return (n & ~15) + 2 * (n & 3) + ((n >> 2) & 1) + 8 * ((n >> 3) & 1); }

// Columns of a 16-token chunk that hold tokens 0 .. k
__constant__ uint16_t kUpTo[16] = {0x0001, 0x0011, 0x0013, 0x0033, 0x0037, 0x0077, 0x007f, 0x00ff,
                                   0x01ff, 0x11ff, 0x13ff, 0x33ff, 0x37ff, 0x77ff, 0x7fff, 0xffff};

// The exponents e of the scales of this lane's two tokens, columns lane and 32 + lane: the finite ones are below 2^e (-14 where all are subnormal or
// 0).  -> that of the tile, also of tokens that are not `there`.  strange: the columns with a scale that is not finite.
template <int HD>
__device__ __forceinline__ int scale_exponents(const uint8_t* raw, int lane, const bool (&there)[2], int (&e)[2], uint32_t (&strange)[2]) {
    constexpr int kNb = HD / 32;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int n = 32 * half + lane;
        const uint32_t* at = reinterpret_cast<const uint32_t*>(raw + (n >> 4) * kv_chunk_bytes(HD) + 2 * (4 * (n & 3) + ((n >> 2) & 3)) * kNb);
        uint32_t largest = 0;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < kNb / 2; ++i) {
            const uint32_t w = there[half] ? at[i] & 0x7fff7fffu : 0u, lo = w & 0xffffu, hi = w >> 16;
            odd |= lo >= 0x7c00u || hi >= 0x7c00u;
            largest = max(largest, max(lo < 0x7c00u ? lo : 0u, hi < 0x7c00u ? hi : 0u));
        }
        e[half] = static_cast<int>(largest >> 10) - 14;
        strange[half] = __ballot_sync(0xffffffffu, odd);
    }
    const int top = __reduce_max_sync(0xffffffffu, max(e[0], e[1]));
#pragma unroll
    for (int half = 0; half < 2; ++half)
        if (!there[half]) e[half] = top;
    return top;
}
// 2^(15 - e) as the product of two f16 powers of two (a scale below 2^e goes below 2^15, and with code * 2^-9 a value below 2^13)
__device__ __forceinline__ void scale_factors(int e, uint32_t& f1, uint32_t& f2) {
    const int x = 15 - e, y = x >> 1;                                     // -4 <= x <= 29
    f1 = (15 + y) << 10;
    f2 = (15 + x - y) << 10;
}

// Eight values (four pairs) as one or two parts: 16 bytes each
template <int PARTS>
__device__ __forceinline__ void put8(uint8_t* dst, int part_bytes, const uint32_t (&code)[4], const __half2 (&s)[4]) {
    const __half2 up = __float2half2_rn(32768.0f);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 x = __hmul2(h2(code[i]), up);
        const __half2 v = __hmul2(x, s[i]);
        hi[i] = u32(v);
        if (PARTS == 2) lo[i] = u32(__hfma2(x, s[i], __hneg2(v)));
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if (PARTS == 2) *reinterpret_cast<uint4*>(dst + part_bytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// A sequence, and the key tiles of its row tiles
struct Seq {
    int L, T, q0, rows;    // cached tokens, query tokens, first query row, rows of a kv head
    int len;               // visible at most
    __device__ __forceinline__ int row_tiles() const { return (rows + kRows - 1) / kRows; }
};
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b) {
    Seq s;
    const QueryRows q = query_rows(a, b);
    s.q0 = q.q0;
    s.T = q.T;
    s.L = a.kv_len[b];
    if (s.L > a.max_kv) report_error(kErrIndex);
    s.rows = q.tokens * (a.q_heads / a.kv_heads);
    s.len = min(max(s.L, 0), a.max_kv);
    return s;
}
// Key tiles that row tile rt sees; one at least, which writes zeros where there is none
__device__ __forceinline__ int key_tiles(const AttnArgs& a, const Seq& s, int rt) {
    const int group = a.q_heads / a.kv_heads, end = min((rt + 1) * kRows, s.rows);
    const int seen = a.tree ? s.len : min(s.len, max(s.L - s.T + (end + group - 1) / group, 0));
    return max((seen + kTok - 1) / kTok, 1);
}
// The key tiles of one kv head of a sequence, by a warp
__device__ __forceinline__ long long head_units(const AttnArgs& a, const Seq& s, int lane) {
    int sum = 0;
    for (int rt = lane; rt < s.row_tiles(); rt += 32) sum += key_tiles(a, s, rt);
    return __reduce_add_sync(0xffffffffu, sum);
}

// A block's run, piece by piece: key tiles k0 .. k1 of row tile rt of kv head hk of sequence b
struct Piece {
    Seq s;
    int b, hk, rt, k0, k1, all, left;                      // left: units of the run from k0 on
    int begun;             // the run that began the tile, of the run's first piece
    // The first piece of a run (a whole warp together) -> whether there is one
    __device__ __forceinline__ bool first(const AttnArgs& a, int lane) {
        long long total = 0;
        for (int i = 0; i < a.seqs; ++i) total += head_units(a, load_seq(a, i), lane) * a.kv_heads;
        const long long per = max((total + kBlocks - 1) / kBlocks, 1ll), pos = per * blockIdx.x;
        if (pos >= total) return false;
        left = static_cast<int>(min(per, total - pos));
        long long before = 0, units = 0;
        for (b = 0;; ++b) {
            s = load_seq(a, b);
            units = head_units(a, s, lane);
            if (before + units * a.kv_heads > pos) break;
            before += units * a.kv_heads;
        }
        int rest;
        div_mod(pos - before, static_cast<int>(units), hk, rest);
        for (rt = 0;; rt += 32) {
            const int mine = rt + lane < s.row_tiles() ? key_tiles(a, s, rt + lane) : 0;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, upto > rest);
            if (hit) {
                const int at = __ffs(hit) - 1;
                rt += at;
                k0 = rest - __shfl_sync(0xffffffffu, upto - mine, at);
                break;
            }
            rest -= __shfl_sync(0xffffffffu, upto, 31);
        }
        cut(a);
        div_mod(pos - k0, static_cast<int>(per), begun, rest);
        return true;
    }
    __device__ __forceinline__ void cut(const AttnArgs& a) {
        all = key_tiles(a, s, rt);
        k1 = min(all, k0 + left);
    }
    __device__ __forceinline__ bool next(const AttnArgs& a) {
        left -= k1 - k0;
        if (left == 0) return false;
        k0 = 0;
        if (++rt >= s.row_tiles()) {
            rt = 0;
            if (++hk >= a.kv_heads) {
                hk = 0;
                do s = load_seq(a, ++b); while (s.rows == 0);
            }
        }
        cut(a);
        return true;
    }
};

struct Info {
    uint2 kf[kTok];        // two factors (f16, twice) of a key's scales, by column (token)
    uint16_t vf[2][kTok];  // two of a value's
    // e of the keys, ref of the values, a bit for each chunk whose page exists, and whether each token was divided by its own 2^e instead (then
    // kOwn for that of the keys):
    alignas(16) int4 tile;
    signed char ke[kTok], ve[kTok];                        // those
    int odd;               // whether some value scale is not finite:
    uint32_t bad[2];       // those tokens' columns
};
struct Bars {
    uint64_t rawfull[2], rawfree[2], expfull[2], kfull[2], vfull[2], qk[2], pv[2], pfull[2], qfull, final_, piecefull[4], piecefree[4], meet;
    uint32_t tmem;
    int abort;
    int have[2];
    alignas(16) Info info[4];
    float amax[2][kRows];                                  // of the groups' halves of the queries
    float m[2][kRows], l[2][kRows];                        // the groups' maxima and sums, at the end
    float kept[2][kRows];                                  // and the factor of the sums that left tensor memory
    int ref[2][kRows];
    Piece piece[4];                                        // a ring, filled by one warp; k1 = 0 ends it
};

// A capped score; CAP 2: 16-bit queries, any cap
template <int PARTS, int CAP>
__device__ __forceinline__ float capped(float x, float cap) {
    return PARTS == 2 ? cap * tanhf(x) : capped16<CAP == 2>(x, cap);
}

// A row's softmax state: running maximum, sum relative to it, and the exponent that its sums of values are relative to
struct RowState {
    float m, l;
    int ref;
};
// Which tokens of a tile from key j0 on a row sees
struct Sees {
    int j0, last, len, base;                               // last: the row's own place (negative: it sees nothing)
    const uint64_t* mask;                                  // tree: the row's mask (NULL: causal)
};
// A tile whose tokens have exponents of their own, from its scores to its weights, as the common way does it below, with the e of each column.  Also one
// whose scores may pass 2^23: the common way subtracts the maximum from products that are not rounded, as the maximum was, and up to there the
// difference is 1/2 at most.  Sixteen columns at a time, and not inlined: the common way keeps its registers and its code small.
template <int HD, int PARTS, int CAP>
__device__ __noinline__ RowState wide_tile(uint32_t cs, uint32_t co, const Info* info, float rs, float softcap, Sees sees, RowState row, bool sums) {
    float top = -INFINITY, top_e = -INFINITY;
    uint32_t y[16];
    const int4 tile = info->tile;
    const unsigned long long bad = info->bad[0] | static_cast<unsigned long long>(info->bad[1]) << 32;
    unsigned long long vis = 0;                            // the columns that the row sees
    if (!sees.mask) {
        const int upto = min(sees.last, sees.len - 1) - sees.j0;
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            if (upto >= 16 * g && (tile.z >> g & 1)) vis |= static_cast<unsigned long long>(kUpTo[min(upto - 16 * g, 15)]) << (16 * g);
    } else {
        const unsigned long long bits = *sees.mask;
#pragma unroll 1
        for (int n = 0; n < kTok; ++n) {
            const int key = sees.j0 + token_of(n), rel = key - sees.base;
            const bool v = key < sees.len && (tile.z >> (n >> 4) & 1) && (rel < 0 || (rel < 64 && (bits >> (rel & 63) & 1)));
            vis |= static_cast<unsigned long long>(v) << n;
        }
    }
    if (vis & bad) row.l = __int_as_float(0x7fc00000);
#pragma unroll 1
    for (int c = 0; c < kTok; c += 16) {
        tc_ld16(cs + c, y);
        tc_wait_ld();
        const uint32_t now = static_cast<uint32_t>(vis >> c);
#pragma unroll
        for (int n = 0; n < 16; ++n) {
            float v = __uint_as_float(y[n]) * (rs * pow2i(info->ke[c + n]));
            if (CAP) v = capped<PARTS, CAP>(v, softcap * kLog2e);
            if (!(now >> n & 1)) v = -INFINITY;
            top = fmaxf(top, v);
            top_e = fmaxf(top_e, v + static_cast<float>(info->ve[c + n]));
            y[n] = __float_as_uint(v);
        }
        tc_st16(cs + c, y);
    }
    tc_wait_st();
    const float m = top > row.m + kSlack ? top : row.m;
    const int ref = static_cast<int>(fminf(fmaxf(ceilf(top_e - m), -16.f), 32.f));       // (no token at all, or scores that are not finite)
    const float down = ex2(row.m - m), downo = down * pow2i(row.ref - ref);
    if (sums)
#pragma unroll 1
        for (int c = 0; c < HD; c += 16) {
            tc_ld16(co + c, y);
            tc_wait_ld();
#pragma unroll
            for (int n = 0; n < 16; ++n) y[n] = __float_as_uint(__uint_as_float(y[n]) * downo);
            tc_st16(co + c, y);
        }
    // the weights' first half takes the first quarter of the scores' place, and of the third (their low parts): the second half is read before
    uint32_t z[32];
    tc_ld16(cs + 32, z);
    tc_ld16(cs + 48, z + 16);
    float sum = 0.f;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        uint32_t w[32];
        if (half == 0) {
            tc_ld16(cs, w);
            tc_ld16(cs + 16, w + 16);
        } else {
#pragma unroll
            for (int n = 0; n < 32; ++n) w[n] = z[n];
        }
        tc_wait_ld();
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int n = 0; n < 16; ++n) {
            const float x0 = __uint_as_float(w[2 * n]) - m, x1 = __uint_as_float(w[2 * n + 1]) - m;
            sum += ex2(x0) + ex2(x1);
            const float p0 = ex2(x0 + (kLift + static_cast<float>(info->ve[32 * half + 2 * n] - ref)));
            const float p1 = ex2(x1 + (kLift + static_cast<float>(info->ve[32 * half + 2 * n + 1] - ref)));
            const __half2 v = __floats2half2_rn(p0, p1);
            hi[n] = u32(v);
            if (PARTS == 2) {
                const float2 f = __half22float2(v);
                lo[n] = u32(__floats2half2_rn(p0 - f.x, p1 - f.y));
            }
        }
        tc_st16(cs + 16 * half, hi);
        if (PARTS == 2) tc_st16(cs + 32 + 16 * half, lo);
    }
    return {m, fmaf(row.l, down, sum), ref};
}

template <int HD, int PARTS> struct Smem {
    static constexpr int kRaw = kGroups * kv_chunk_bytes(HD);             // a tile's chunks
    static constexpr int kK = kTok * HD * 2, kV = HD * kTok * 2;          // one part of a tile's keys, values
    static constexpr int kKat = 0, kVat = 2 * PARTS * kK, kRawAt = kVat + 2 * PARTS * kV, kBars = kRawAt + 2 * kRaw;
    static constexpr int kAll = 1024 + kBars + sizeof(Bars);
};

template <typename T, int HD, int PARTS, int CAP>
__global__ void __launch_bounds__(kThreads, 1) attn_tiles_kernel(const AttnArgs a, const Parts parts, float4* kept) {
    using M = Smem<HD, PARTS>;
    constexpr int kChunk = kv_chunk_bytes(HD), kNb = HD / 32;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_align1024(smem_raw);
    uint8_t* sk = base + M::kKat;                          // [2][PARTS][HD / 64][64 rows x 128 bytes]
    uint8_t* sv = base + M::kVat;                          // [2][PARTS][HD rows x 128 bytes]
    uint8_t* sraw = base + M::kRawAt;                      // [2][kGroups][chunk]
    Bars* bars = reinterpret_cast<Bars*>(base + M::kBars);
    volatile int* abort = &bars->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int group = a.q_heads / a.kv_heads;
    if (threadIdx.x == 0) parts.head[blockIdx.x].first = -1;               // the piece that ends a shared tile says so later
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars->rawfull[s], 1);
            mbar_init(&bars->rawfree[s], kNumKV);
            mbar_init(&bars->expfull[s], 1);
            mbar_init(&bars->kfull[s], kNumKV);
            mbar_init(&bars->vfull[s], kNumKV);
            mbar_init(&bars->qk[s], 1);
            mbar_init(&bars->pv[s], 1);
            mbar_init(&bars->pfull[s], 4);
        }
        mbar_init(&bars->qfull, 8);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars->piecefull[i], 1);
            mbar_init(&bars->piecefree[i], 8 + kNumKV + 3);
        }
        mbar_init(&bars->meet, 8);
        mbar_init(&bars->final_, 2);
        bars->abort = 0;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    // the run's pieces, as every role takes them: piece n is there (false: no more, or given up); this warp is done with it
    auto take = [&](int n) { return wait_for(&bars->piecefull[n & 3], (n >> 2) & 1, abort) && bars->piece[n & 3].k1 > 0; };
    auto done = [&](int n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->piecefree[n & 3]);
    };

    if (warp < kWarpKV) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---------------- softmax: row tile0 + 32 * (warp % 4) + lane, tiles wg, wg + 2, ...
        const int wg = warp >> 2, lr = (warp & 3) * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16), cs = tl + kColS + wg * kTok, co = tl + kColO + wg * HD;
        int it = 0;                                                       // tiles so far
        bool ok = true, more = take(0);
        // this thread's half of its row's queries, requested before the piece before it is written out: positions 4 i .. of atom c = wg
        // (HD = 64: of half of the atom)
        constexpr int kQ = HD / 8;                                        // runs of four dims
        typename Vec4<T>::Raw q[kQ];
        auto request = [&](const Piece& p) {
            const int r = p.rt * kRows + lr, tok = r < p.s.rows ? r / group : 0, h = r < p.s.rows ? r % group : 0;
            const T* at = static_cast<const T*>(a.q) + (p.s.q0 + tok) * a.q_stride + (p.hk * group + h) * HD;
#pragma unroll
            for (int i = 0; i < kQ; ++i) {
                const int k = HD == 64 ? i + 8 * wg : i, t = k >> 2, hh = (k >> 1) & 1, bb = k & 1;
                q[i] = *reinterpret_cast<const typename Vec4<T>::Raw*>(at + (HD == 64 ? 0 : 64 * wg) + 32 * hh + 16 * bb + 4 * t);
            }
        };
        uint32_t met = 0;
        auto meet = [&]() {                                               // all softmax warps
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->meet);
            ok = wait_for(&bars->meet, met++ & 1, abort) && ok;
            __syncwarp();
        };
        if (more) request(bars->piece[0]);
        for (int pi = 0; ok && more; ++pi) {
        const Piece& p = bars->piece[pi & 3];
        const int q0 = p.s.q0, hk = p.hk, tile0 = p.rt * kRows, group0 = tile0 / group;
        // tokens that every row of the tile sees
        const int all_see = min(p.s.L - p.s.T + (a.tree ? 0 : group0 + 1), a.max_kv);
        const int r = tile0 + lr;
        const bool in = r < p.s.rows;
        const int tok = in ? r / group : 0, h = in ? r % group : 0;
        float rs;
        int far = kOwn - 1;
        {
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < kQ; ++i) {
                const float4 v = Vec4<T>::widen(q[i]);
                amax = fmaxf(amax, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
            }
            bars->amax[wg][lr] = amax;
            meet();
            amax = fmaxf(bars->amax[0][lr], bars->amax[1][lr]);
            const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
            const int up = amax > 0.f && e < 128 ? min(14 - e, 126) : 0;
            // the scale's sign goes into the queries, and a scale of 0 (equal weights) too: the scores' factor stays positive
            const float f = !in || a.scale == 0.f ? 0.f : copysignf(pow2i(up), a.scale), size = a.scale == 0.f ? 1.f : fabsf(a.scale);
            rs = (!CAP ? size * kLog2e : size / a.softcap * (PARTS == 2 ? 1.f : 2.f * kLog2e)) * 0x1p-6f * pow2i(-up);    // 2^6 of the keys
            rs = fminf(fmaxf(rs, 0x1p-100f), 0x1p107f);                   // times a scale's power of two neither 0 nor infinite, for queries of any size
            // the keys' exponent up to which no row's score here is beyond 2^23 (products of 2^15 and 2^13, 2^7 of them); the common way wants that
            // (rows of zeros, rows past the end among them, have no scores, and those that are not finite no order)
            if (!CAP) {
                const uint32_t most = __reduce_max_sync(0xffffffffu, amax > 0.f && e < 128 ? __float_as_uint(rs) : 0u);
                far = min(-13 - (static_cast<int>(most >> 23) - 127), kOwn - 1);
            }
#pragma unroll
            for (int part = 0; part < kQ / 8; ++part) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float4 v = Vec4<T>::widen(q[8 * part + i]);
                    v = f == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
                    const __half2 x = __floats2half2_rn(v.x, v.y), y = __floats2half2_rn(v.z, v.w);
                    hi[2 * i] = u32(x);
                    hi[2 * i + 1] = u32(y);
                    if (PARTS == 2) {
                        const float2 fx = __half22float2(x), fy = __half22float2(y);
                        lo[2 * i] = u32(__floats2half2_rn(v.x - fx.x, v.y - fx.y));
                        lo[2 * i + 1] = u32(__floats2half2_rn(v.z - fy.x, v.w - fy.y));
                    }
                }
                const uint32_t col = tl + kColQ + 16 * (wg * (kQ / 8) + part);
                tc_st16(col, hi);
                if (PARTS == 2) tc_st16(col + HD / 2, lo);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->qfull);
        }
        const int last = in ? p.s.L - p.s.T + tok : -1;
        float m = kNone, l = 0.f, m_kept = 0.f;                               // (m_kept, ref_kept: what the drained sums are relative to)
        int ref = 0, ref_kept = 0;
        const int tiles = p.k1 - p.k0;
        for (int j = (it ^ wg) & 1; ok && j < tiles; j += 2) {                  // tile it + j of all, which is in this group's place
            const int i = it + j;
            // (the scores' MMAs were issued after the keys' barrier, so what stands in `info` was written before; and after the sums of
            // tile i - 2, so those are complete)
            if (!wait_for(&bars->qk[wg], (i >> 1) & 1, abort)) {
                ok = false;
                break;
            }
            __syncwarp();
            tc_fence_after();
            const bool drain = PARTS == 2 && j >= 2 && (j >> 1) % kDrain == 0;
            if (drain) {
                const bool first = j < 4 * kDrain;
                const float f = ex2(m_kept - m) * pow2i(ref_kept - ref);
                float4* at = kept + (blockIdx.x * 2 + wg) * (HD / 4) * kRows + lr;
#pragma unroll 1
                for (int c = 0; c < HD; c += 16) {
                    uint32_t o[16];
                    float4 before[4];
                    tc_ld16(co + c, o);
                    if (!first)
#pragma unroll
                        for (int n = 0; n < 4; ++n) before[n] = at[(c / 4 + n) * kRows];
                    tc_wait_ld();
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        float4 v = make_float4(__uint_as_float(o[4 * n]), __uint_as_float(o[4 * n + 1]), __uint_as_float(o[4 * n + 2]), __uint_as_float(o[4 * n + 3]));
                        if (!first) v = make_float4(fmaf(before[n].x, f, v.x), fmaf(before[n].y, f, v.y), fmaf(before[n].z, f, v.z), fmaf(before[n].w, f, v.w));
                        at[(c / 4 + n) * kRows] = v;
                    }
                }
                m_kept = m;
                ref_kept = ref;
            }
            const Info& info = bars->info[i & 3];
            const int4 tile = info.tile;
            const int have = tile.z, j0 = (p.k0 + j) * kTok;
            float x[kTok];
            auto load = [&]() {
                tc_ld32(cs, x);
                tc_ld32(cs + 32, x + 32);
                tc_wait_ld();
            };
            constexpr bool kEarly = !CAP && !(PARTS == 2 && HD == 128);   // (these spill more with the scores in registers at the branch: 606 against 599 us)
            if (kEarly) load();
            if (__builtin_expect(tile.x > far, 0)) {
                const RowState row = wide_tile<HD, PARTS, CAP>(cs, co, &info, rs, a.softcap,
                                                               {j0, last, p.s.len, p.s.L - p.s.T, last >= 0 && a.tree ? a.tree + q0 + tok : nullptr},
                                                               {m, l, ref}, j >= 2 && !drain);
                m = row.m;
                l = row.l;
                ref = row.ref;
            } else {
                float x_of = rs * pow2i(tile.x);
                const int vn = tile.y;
                if (!kEarly) load();
                if (CAP) {
#pragma unroll
                    for (int n = 0; n < kTok; ++n) x[n] = capped<PARTS, CAP>(x[n] * x_of, a.softcap * kLog2e);
                    x_of = 1.f;
                }
                if (j0 + kTok > all_see || have != (1 << kGroups) - 1) {
                    const int len = p.s.len, base = p.s.L - p.s.T;
                    unsigned long long vis = 0;
                    if (!a.tree) {
                        const int upto = min(last, len - 1) - j0;             // the last visible token of the tile
#pragma unroll
                        for (int g = 0; g < kGroups; ++g)
                            if (upto >= 16 * g && (have >> g & 1)) vis |= static_cast<unsigned long long>(kUpTo[min(upto - 16 * g, 15)]) << (16 * g);
                    } else {
                        const unsigned long long bits = last >= 0 ? a.tree[q0 + tok] : 0ull;
#pragma unroll 1
                        for (int n = 0; n < kTok; ++n) {
                            const int key = j0 + token_of(n), rel = key - base;
                            const bool v = in && key < len && (have >> (n >> 4) & 1) && (rel < 0 || (rel < 64 && ((bits >> (rel & 63)) & 1)));
                            vis |= static_cast<unsigned long long>(v) << n;
                        }
                    }
                    const uint32_t vis0 = static_cast<uint32_t>(vis), vis1 = static_cast<uint32_t>(vis >> 32);
#pragma unroll
                    for (int n = 0; n < kTok; ++n)
                        if (!((n < 32 ? vis0 : vis1) >> (n & 31) & 1u)) x[n] = -INFINITY;
                }
                float top = x[0];
#pragma unroll
                for (int n = 1; n < kTok; ++n) top = fmaxf(top, x[n]);
                top *= x_of;
                if (__any_sync(0xffffffffu, top > m + kSlack || vn != ref)) {
                    const float mn = top > m + kSlack ? top : m, down = ex2(m - mn), downo = down * pow2i(ref - vn);
                    l *= down;
                    m = mn;
                    ref = vn;
                    if (j >= 2 && !drain) {
#pragma unroll 1
                        for (int c = 0; c < HD; c += 16) {
                            uint32_t o[16];
                            tc_ld16(co + c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int n = 0; n < 16; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * downo);
                            tc_st16(co + c, o);
                        }
                    }
                }
                const float from = m - kLift;
                if (info.odd) {                                               // a value that is not finite, seen by this row
                    const unsigned long long bad = info.bad[0] | static_cast<unsigned long long>(info.bad[1]) << 32;
#pragma unroll
                    for (int n = 0; n < kTok; ++n)
                        if ((bad >> n & 1) && x[n] > -INFINITY) l = __int_as_float(0x7fc00000);
                }
                float sum0 = 0.f, sum1 = 0.f;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {                        // (half the code)
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int n = 0; n < 16; ++n) {
                        const float p0 = ex2(fmaf(x[2 * n], x_of, -from)), p1 = ex2(fmaf(x[2 * n + 1], x_of, -from));
                        sum0 += p0;
                        sum1 += p1;
                        const __half2 v = __floats2half2_rn(p0, p1);
                        hi[n] = u32(v);
                        if (PARTS == 2) {
                            const float2 g = __half22float2(v);
                            lo[n] = u32(__floats2half2_rn(p0 - g.x, p1 - g.y));
                        }
                    }
                    tc_st16(cs + 16 * half, hi);
                    if (PARTS == 2) tc_st16(cs + 32 + 16 * half, lo);
#pragma unroll
                    for (int n = 0; n < 32; ++n) x[n] = x[32 + n];
                }
                l = fmaf(sum0 + sum1, 0x1p-11f, l);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->pfull[wg]);
        }
        // ---- the groups' sums meet: each group takes half of the dims
        it += tiles;
        const int e0 = (it - 1 - ((it - 1 ^ wg) & 1));                    // this group's last tile, if it had one of the piece
        if (ok && e0 >= it - tiles && !wait_for(&bars->pv[wg], (e0 >> 1) & 1, abort)) ok = false;
        const bool has = e0 >= it - tiles;
        more = take(pi + 1);
        if (more) request(bars->piece[(pi + 1) & 3]);
        bars->m[wg][lr] = !ok ? __int_as_float(0x7fc00000) : has ? m : kNone;
        bars->l[wg][lr] = has ? l : 0.f;
        bars->ref[wg][lr] = ref;
        if (PARTS == 2) bars->kept[wg][lr] = ex2(m_kept - m) * pow2i(ref_kept - ref);
        meet();
        {
            tc_fence_after();
            const float m0 = bars->m[0][lr], m1 = bars->m[1][lr], top = fmaxf(m0, m1), f0 = ex2(m0 - top), f1 = ex2(m1 - top);
            const float sum = fmaf(bars->l[0][lr], f0, bars->l[1][lr] * f1);
            const bool has0 = tiles > 1 || !((it - 1) & 1), has1 = tiles > 1 || ((it - 1) & 1);      // a group without tiles has no sums
            const bool whole = p.k0 == 0 && p.k1 == p.all, head = p.k1 == p.all;
            const float inv = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
            const float a0 = f0 * pow2i(bars->ref[0][lr] - 17) * inv, a1 = f1 * pow2i(bars->ref[1][lr] - 17) * inv;    // 2^11 of the weights, 2^6 of the values
            T* out = static_cast<T*>(a.out) + (q0 + tok) * a.out_stride + (hk * group + h) * HD + wg * (HD / 2);
            // whether a group's sums have been drained: it had more than kDrain tiles, every other one from its first on
            const int begin0 = (it - tiles) & 1;
            const bool kept0 = PARTS == 2 && (tiles - begin0 + 1) / 2 > kDrain, kept1 = PARTS == 2 && (tiles - (begin0 ^ 1) + 1) / 2 > kDrain;
            const size_t slot = (static_cast<size_t>(head ? 0 : kBlocks) + blockIdx.x) * kRows + lr;
#pragma unroll 1
            for (int c = 0; c < HD / 2; c += 16) {
                uint32_t o0[16], o1[16];
                tc_ld16(tl + kColO + wg * (HD / 2) + c, o0);
                tc_ld16(tl + kColO + HD + wg * (HD / 2) + c, o1);
                tc_wait_ld();
                auto add_kept = [&](uint32_t* o, int g) {
                    const float f = bars->kept[g][lr];
                    const float4* at = kept + (blockIdx.x * 2 + g) * (HD / 4) * kRows + lr;
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float4 k = at[((wg * (HD / 2) + c) / 4 + n) * kRows];
                        o[4 * n] = __float_as_uint(fmaf(k.x, f, __uint_as_float(o[4 * n])));
                        o[4 * n + 1] = __float_as_uint(fmaf(k.y, f, __uint_as_float(o[4 * n + 1])));
                        o[4 * n + 2] = __float_as_uint(fmaf(k.z, f, __uint_as_float(o[4 * n + 2])));
                        o[4 * n + 3] = __float_as_uint(fmaf(k.w, f, __uint_as_float(o[4 * n + 3])));
                    }
                };
                if (kept0) add_kept(o0, 0);
                if (kept1) add_kept(o1, 1);
                float v[16];
#pragma unroll
                for (int n = 0; n < 16; ++n) {
                    v[n] = has0 && sum != 0.f ? __uint_as_float(o0[n]) * a0 : 0.f;
                    if (has1 && sum != 0.f) v[n] = fmaf(__uint_as_float(o1[n]), a1, v[n]);
                }
                if (in)
#pragma unroll
                    for (int n = 0; n < 16; n += 4) {
                        const float4 x = make_float4(v[n], v[n + 1], v[n + 2], v[n + 3]);
                        if (whole) store4(out + c + n, x);
                        else *reinterpret_cast<float4*>(parts.o + slot * HD + wg * (HD / 2) + c + n) = x;
                    }
            }
            if (!whole && wg == 0) parts.ml[slot] = make_float2(top, sum);
            if (head && !whole && threadIdx.x == 0) {                     // (only the run's first piece can be one)
                parts.head[blockIdx.x] = {p.begun, q0, tile0, min(p.s.rows - tile0, kRows), hk};
            }
        }
        tc_fence_before();
        meet();                                                           // the sums have been read: the next piece's may begin
        tc_fence_after();
        done(pi);
        }
    } else if (warp < kWarpMma) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsKV));
        // ---------------- keys and values
        const int w8 = warp - kWarpKV, dt = threadIdx.x - kWarpKV * 32;
        // this thread's part of the keys: unit k_up of token k_tok (of the first kStep), as chunk 2 t (+ 1) of its row
        constexpr int kUnits = HD / 16, kStep = kNumKV * 32 / kUnits, kUnitsPer = kTok / kStep;
        static_assert(kStep % 16 == 0, "a unit's token has the same place in every chunk");
        const int k_tok = dt / kUnits, k_up = dt % kUnits, k_in = k_tok & 15;
        const int k_u = HD > 64 ? k_up ^ (4 * (k_in & 1)) : k_up, k_tt = (k_in & 7) >> 1, k_p = (k_in & 1) + 2 * (k_in >> 3);
        const int k_src = (k_tok >> 4) * kChunk + k_in * HD + k_up * 16;
        const int k_scale = (k_tok >> 4) * kChunk + kv_ks_offset(HD) + 2 * ((4 * k_tt + k_p) * kNb + 2 * (k_u >> 2));
        const bool k_swap = HD > 64 ? (k_u >> 2) & 1 : k_in & 1;          // the two chunks of a unit in this order: a store's chunks differ in their banks
        const int k_col = (k_tok & ~15) + 4 * k_p + k_tt;
        const int k_dst = (k_u >> 2) * (kTok * 128) + static_cast<int>(swz128(k_col, 2 * (k_u & 3) + (k_swap ? 1 : 0)));
        // and of the values: four dims 32 v_c + 4 v_g .. of eight tokens
        const int v_g = HD == 64 ? (lane >> 1) & 7 : lane >> 2, v_c = HD == 64 ? lane & 1 : lane & 3;
        const int v_src = kv_v_offset(HD) + (w8 & 1) * 8 * HD + 4 * v_c, v_scale = kv_vs_offset(HD) + 2 * (2 * (w8 & 1) * kNb + v_c);
        int i = 0;                                                        // tiles so far
        bool ok = true;
        for (int pi = 0; ok && take(pi); done(pi), ++pi)
        for (int kt = bars->piece[pi & 3].k0; kt < bars->piece[pi & 3].k1; ++kt, ++i) {
            const int s = i & 1;
            const uint32_t par = (i >> 1) & 1;
            ok = wait_for(&bars->expfull[s], par, abort) && wait_for(&bars->rawfull[s], par, abort);
            if (!ok) break;
            __syncwarp();
            const uint8_t* raw = sraw + s * M::kRaw;
            const Info& info = bars->info[i & 3];
            const int have = info.tile.z, j0 = kt * kTok, len = bars->piece[pi & 3].s.len;
            const bool odd = info.odd;
            const bool edge = j0 + kTok > len || have != (1 << kGroups) - 1;      // some of the tile's tokens do not exist
            // keys, once the scores of the tile before the last are done
            if (i >= 2 && !(ok = wait_for(&bars->qk[s], par ^ 1, abort))) break;
            __syncwarp();
            {
                // a thread has one 16-byte unit of one token in every 128 / units tokens
                uint4 w[kUnitsPer];
                uint32_t sc[kUnitsPer];
#pragma unroll
                for (int k = 0; k < kUnitsPer; ++k) {
                    const uint8_t* ch = raw + (kStep * k >> 4) * kChunk;
                    w[k] = *reinterpret_cast<const uint4*>(ch + k_src);
                    sc[k] = *reinterpret_cast<const uint32_t*>(ch + k_scale);
                    if (edge && (j0 + k_tok + kStep * k >= len || !(have >> ((k_tok + kStep * k) >> 4) & 1))) sc[k] = 0;
                }
#pragma unroll
                for (int k = 0; k < kUnitsPer; ++k) {
                    const uint2 f = info.kf[k_col + kStep * k];
                    sc[k] = u32(__hmul2(__hmul2(h2(sc[k]), h2(f.x)), h2(f.y)));
                }
                uint8_t* dst = sk + s * PARTS * M::kK;
#pragma unroll
                for (int k = 0; k < kUnitsPer; ++k) {
                    const __half2 s0 = h2(__byte_perm(sc[k], 0, k_swap ? 0x3232 : 0x1010)), s1 = h2(__byte_perm(sc[k], 0, k_swap ? 0x1010 : 0x3232));
                    const uint32_t wa = k_swap ? w[k].z : w[k].x, wb = k_swap ? w[k].w : w[k].y, wc = k_swap ? w[k].x : w[k].z,
                                   wd = k_swap ? w[k].y : w[k].w;
                    const uint32_t ca[4] = {codes2(wa, 0, 0x1100), codes2(wa, 0, 0x3322), codes2(wb, 0, 0x1100), codes2(wb, 0, 0x3322)};
                    const uint32_t cb[4] = {codes2(wc, 0, 0x1100), codes2(wc, 0, 0x3322), codes2(wd, 0, 0x1100), codes2(wd, 0, 0x3322)};
                    const __half2 sa[4] = {s0, s0, s0, s0}, sb[4] = {s1, s1, s1, s1};
                    put8<PARTS>(dst + k_dst + kStep * 128 * k, M::kK, ca, sa);
                    put8<PARTS>(dst + (k_dst ^ 16) + kStep * 128 * k, M::kK, cb, sb);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->kfull[s]);
            // values, once the sums of the tile before the last are done: this warp eight tokens (value rows 8 o ..)
            if (i >= 2 && !(ok = wait_for(&bars->pv[s], par ^ 1, abort))) break;
            __syncwarp();
            {
                uint8_t* dst = sv + s * PARTS * M::kV;
#pragma unroll
                for (int j = 0; j < kTok / 8 / kNumKV; ++j) {             // octets w8, w8 + kNumKV ..
                    const uint8_t* ch = raw + ((w8 >> 1) + kNumKV / 2 * j) * kChunk;
                    const int t0 = j0 + 16 * ((w8 >> 1) + kNumKV / 2 * j) + 8 * (w8 & 1);
                    uint32_t w[8], sc[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {                         // value rows 8 o + k: p = 2 o + (k >> 2), t = k & 3
                        const int t = k & 3;
                        w[k] = *reinterpret_cast<const uint32_t*>(ch + v_src + (k >> 2) * 4 * HD + t * HD + (HD == 64 ? 8 * (v_g ^ (4 * (t >> 1))) : 16 * (v_g ^ (2 * t))));
                        sc[k] = *reinterpret_cast<const uint16_t*>(ch + v_scale + 2 * (4 * t + (k >> 2)) * kNb);
                    }
                    if (edge) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)                       // tokens 2 t + (p & 1) + 8 (p >> 1)
                            if (t0 + 2 * (k & 3) + (k >> 2) >= len || !(have >> ((w8 >> 1) + kNumKV / 2 * j) & 1)) sc[k] = 0;
                    }
                    if (odd) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if ((sc[k] & 0x7c00u) == 0x7c00u) sc[k] = 0;
                    }
                    __half2 sh[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) sh[k] = h2(sc[2 * k] | sc[2 * k + 1] << 16);
                    const uint4 f1 = *reinterpret_cast<const uint4*>(info.vf[0] + 8 * (w8 + kNumKV * j)), f2 = *reinterpret_cast<const uint4*>(info.vf[1] + 8 * (w8 + kNumKV * j));
                    sh[0] = __hmul2(__hmul2(sh[0], h2(f1.x)), h2(f2.x));
                    sh[1] = __hmul2(__hmul2(sh[1], h2(f1.y)), h2(f2.y));
                    sh[2] = __hmul2(__hmul2(sh[2], h2(f1.z)), h2(f2.z));
                    sh[3] = __hmul2(__hmul2(sh[3], h2(f1.w)), h2(f2.w));
#pragma unroll
                    for (int x = 0; x < (HD == 64 ? 2 : 4); ++x) {
                        const int e = HD == 64 ? 2 * (lane >> 4) + ((x + v_c) & 1) : (x + v_c) & 3;      // a store's chunks differ in their banks
                        const uint32_t sel = 0x4400u + 0x1111u * e;
                        const uint32_t code[4] = {codes2(w[0], w[1], sel), codes2(w[2], w[3], sel), codes2(w[4], w[5], sel), codes2(w[6], w[7], sel)};
                        put8<PARTS>(dst + swz128(32 * v_c + 4 * v_g + e, w8 + kNumKV * j), M::kV, code, sh);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars->vfull[s]);
                mbar_arrive(&bars->rawfree[s]);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    }
    if (warp == kWarpMma) {
        // ---------------- scores, by one thread: of tile i into the place of the weights of tile i - 2
        if (lane == 0) {
            bool ok = true;
            const uint64_t desc = smem_desc(sk);
            const uint32_t hi = static_cast<uint32_t>(desc >> 32);
            int i = 0;                                                    // tiles so far
            for (int pi = 0; ok && take(pi); mbar_arrive(&bars->piecefree[pi & 3]), ++pi)
            for (int k0 = bars->piece[pi & 3].k0, k1 = bars->piece[pi & 3].k1, kt = k0; kt < k1; ++kt, ++i) {
                const int s = i & 1;
                const uint32_t par = (i >> 1) & 1;
                ok = (kt > k0 || wait_for(&bars->qfull, pi & 1, abort)) && wait_for(&bars->kfull[s], par, abort) &&
                     (i < 2 || wait_for(&bars->pv[s], par ^ 1, abort));
                if (!ok) break;
                tc_fence_after();
                const uint32_t lo = static_cast<uint32_t>(desc) + s * (PARTS * M::kK >> 4), d = tmem + kColS + s * kTok;
#pragma unroll 1
                for (int t = 0; t < (PARTS == 2 ? 3 : 1); ++t) {          // low x high, high x low, high x high: small sums lose less (kDrain)
                    const uint32_t q = tmem + kColQ + (PARTS == 2 && t == 0 ? HD / 2 : 0), k0 = lo + (t == 1 ? M::kK >> 4 : 0);
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k)
                        mma_ts(d, q + 8 * k, k0 + (((k >> 2) * (kTok * 128) + 32 * (k & 3)) >> 4), hi, idesc<kTok>(), k ? 1u : t);
                }
                tc_commit(&bars->qk[s]);
            }
            tc_commit(&bars->final_);                                     // all MMAs issued so far complete before TMEM is freed
        }
    } else if (warp == kWarpMma + 1) {
        // ---------------- sums, by one thread: o += weights * values of tile i
        if (lane == 0) {
            const uint64_t desc = smem_desc(sv);
            const uint32_t hi = static_cast<uint32_t>(desc >> 32);
            int i = 0;                                                    // tiles so far
            bool ok = true;
            for (int pi = 0; ok && take(pi); mbar_arrive(&bars->piecefree[pi & 3]), ++pi)
            for (int k0 = bars->piece[pi & 3].k0, k1 = bars->piece[pi & 3].k1, kt = k0; kt < k1; ++kt, ++i) {
                const int s = i & 1;
                const uint32_t par = (i >> 1) & 1;
                ok = wait_for(&bars->vfull[s], par, abort) && wait_for(&bars->pfull[s], par, abort);
                if (!ok) break;
                tc_fence_after();
                const uint32_t lo = static_cast<uint32_t>(desc) + s * (PARTS * M::kV >> 4), d = tmem + kColO + s * HD, w = tmem + kColS + s * kTok;
                // a group's first tile of a piece begins its sums, and the first after they were drained
                const uint32_t acc = PARTS == 2 ? ((kt - k0) >> 1) % kDrain != 0 : kt > k0 + 1;
#pragma unroll 1
                for (int t = 0; t < (PARTS == 2 ? 3 : 1); ++t) {
                    const uint32_t w0 = w + (t == 1 ? 32 : 0), v0 = lo + (t == 2 ? M::kV >> 4 : 0);
#pragma unroll
                    for (int k = 0; k < kTok / 16; ++k) mma_ts(d, w0 + 8 * k, v0 + (32 * k >> 4), hi, idesc<HD>(), k || t ? 1u : acc);
                }
                tc_commit(&bars->pv[s]);
            }
            tc_commit(&bars->final_);
        }
    } else if (warp == kWarpMma + 2) {
        // ---------------- chunks of a tile: lane g one of its groups
        const int gpp = a.page_size / kvGroup;
        int i = 0;                                                        // tiles so far
        bool ok = true;
        for (int pi = 0; ok && take(pi); done(pi), ++pi)
        for (int kt = bars->piece[pi & 3].k0; kt < bars->piece[pi & 3].k1; ++kt, ++i) {
            const Piece& p = bars->piece[pi & 3];
            const int s = i & 1;
            int page = -1, off = 0;
            const int g = kt * kGroups + lane;
            const bool wanted = lane < kGroups && g * kvGroup < p.s.len;
            if (wanted) {
                const int pi = g / gpp;
                off = g - pi * gpp;
                page = a.table[static_cast<size_t>(p.b) * a.table_stride + pi];
                if (page < 0 || page >= a.pages) {
                    page = -1;
                    report_error(kErrIndex);
                }
            }
            const unsigned there = __ballot_sync(0xffffffffu, page >= 0), missing = __ballot_sync(0xffffffffu, wanted && page < 0);
            if (i >= 2 && !(ok = wait_for(&bars->rawfree[s], ((i >> 1) & 1) ^ 1, abort))) break;
            __syncwarp();
            if (lane == 0) {
                bars->have[s] = ((1 << kGroups) - 1) & ~missing;          // chunks past the end count as there: their tokens are past the end
                if (there) mbar_arrive_expect_tx(&bars->rawfull[s], __popc(there) * kChunk);
                else mbar_arrive(&bars->rawfull[s]);
            }
            __syncwarp();
            if (page >= 0)
                bulk_g2s(sraw + s * M::kRaw + lane * kChunk, a.cache + ((static_cast<size_t>(page) * a.kv_heads + p.hk) * gpp + off) * kChunk, kChunk,
                         &bars->rawfull[s]);
        }
        __syncwarp();
        if (*abort)                                                       // copies in flight land before shared memory goes away
            for (int k = max(i - 2, 0); k < i; ++k)
                if (lane == 0 && !mbar_wait(&bars->rawfull[k & 1], (k >> 1) & 1)) report_error(kErrDrainTimeout);
    } else if (warp == kWarpMma + 3) {
        // ---------------- the run's pieces, a piece ahead, and the exponents of a tile's scales
        Piece now, then;
        int i = 0, pi = 0, ref = -14;                                     // tiles so far, pieces, what values are divided by
        bool more = then.first(a, lane), ok = true;
        auto publish = [&](int n) {                                       // `then`, or the end
            if (n >= 4 && !wait_for(&bars->piecefree[n & 3], ((n >> 2) & 1) ^ 1, abort)) ok = false;
            __syncwarp();
            if (lane == 0) {
                if (!more) then.k1 = 0;
                bars->piece[n & 3] = then;
                mbar_arrive(&bars->piecefull[n & 3]);
            }
        };
        publish(0);
        while (ok && more) {
        now = then;
        more = then.next(a);
        publish(++pi);
        for (int kt = now.k0; ok && kt < now.k1; ++kt, ++i) {
            const int s = i & 1;
            if (!(ok = wait_for(&bars->rawfull[s], (i >> 1) & 1, abort))) break;
            __syncwarp();
            const uint8_t* raw = sraw + s * M::kRaw;
            const int have = bars->have[s], left = now.s.len - kt * kTok;
            Info& info = bars->info[i & 3];
            uint32_t bad[2];
            int ke[2], ve[2];
            bool there[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int n = 32 * half + lane;
                there[half] = token_of(n) < left && (have >> (n >> 4) & 1);
            }
            const int kexp = scale_exponents<HD>(raw + kv_ks_offset(HD), lane, there, ke, bad);
            const int vexp = scale_exponents<HD>(raw + kv_vs_offset(HD), lane, there, ve, bad);
            const bool wide = __any_sync(0xffffffffu, kexp - min(ke[0], ke[1]) > kNear || vexp - min(ve[0], ve[1]) > kNear);
            if (vexp > ref || vexp < ref - kAbove) ref = vexp;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int n = 32 * half + lane;
                const int kn = wide ? ke[half] : kexp, vn = wide ? ve[half] : ref;
                uint32_t f1, f2;
                scale_factors(kn, f1, f2);
                info.kf[n] = make_uint2(f1 * 0x10001u, f2 * 0x10001u);
                scale_factors(vn, f1, f2);
                info.vf[0][n] = static_cast<uint16_t>(f1);
                info.vf[1][n] = static_cast<uint16_t>(f2);
                info.ke[n] = static_cast<signed char>(kn);
                info.ve[n] = static_cast<signed char>(vn);
            }
            __syncwarp();
            if (lane == 0) {
                info.tile = make_int4(wide ? kOwn : kexp, ref, have, wide);
                info.odd = bad[0] | bad[1];
                info.bad[0] = bad[0];
                info.bad[1] = bad[1];
                mbar_arrive(&bars->expfull[s]);
            }
        }
        }
    }

    // ---------------- teardown
    __syncwarp();
    if (warp == kWarpMma) {
        if (lane == 0 && !mbar_wait(&bars->final_, 0)) report_error(kErrMmaTimeout);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// The workspace: the joining kernel's, then f32's drained sums [block][group][HD / 4][row] of four columns
size_t kept_at(int hd) { return (parts_bytes(kBlocks, kRows, hd) + 255) / 256 * 256; }

template <typename T, int HD, int CAP>
cudaError_t tiles_go(const AttnArgs& a, cudaStream_t s) {
    constexpr int PARTS = sizeof(T) == 4 ? 2 : 1, smem = Smem<HD, PARTS>::kAll;
    static_assert(smem <= 227 * 1024, "shared memory");
    static std::atomic<uint64_t> raised{0};
    cudaError_t e = allow_smem(attn_tiles_kernel<T, HD, PARTS, CAP>, smem, raised);
    if (e != cudaSuccess) return e;
    const Parts parts = parts_at(a.workspace, kBlocks, kRows, HD);
    float4* kept = reinterpret_cast<float4*>(static_cast<uint8_t*>(a.workspace) + kept_at(HD));
    e = launch_dependent(attn_tiles_kernel<T, HD, PARTS, CAP>, dim3(kBlocks), kThreads, smem, s, a, parts, kept);
    if (e != cudaSuccess) return e;
    return launch_join<T, HD, kRows, 1>(a, parts, kBlocks, s);
}

template <typename T>
cudaError_t tiles_type(const AttnArgs& a, int head_dim, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (a.softcap > kCapNear) return head_dim == 64 ? tiles_go<T, 64, 2>(a, s) : tiles_go<T, 128, 2>(a, s);
    if (a.softcap > 0.f) return head_dim == 64 ? tiles_go<T, 64, 1>(a, s) : tiles_go<T, 128, 1>(a, s);
    return head_dim == 64 ? tiles_go<T, 64, 0>(a, s) : tiles_go<T, 128, 0>(a, s);
}

}  // namespace

size_t attn_tiles_workspace_bytes(int head_dim, int type) {
    return type == GQ_F32 ? kept_at(head_dim) + static_cast<size_t>(kBlocks) * 2 * kRows * head_dim * 4 : parts_bytes(kBlocks, kRows, head_dim);
}

cudaError_t launch_attn_tiles(const AttnArgs& a, int type, int head_dim, cudaStream_t s) {
    if (type == GQ_F32) return tiles_type<float>(a, head_dim, s);
    if (type == GQ_F16) return tiles_type<__half>(a, head_dim, s);
    return tiles_type<__nv_bfloat16>(a, head_dim, s);
}

}  // namespace gq
