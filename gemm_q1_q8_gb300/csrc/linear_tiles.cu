// Q1_0 products with an epilogue, many tokens: tcgen05 (kind::f16), weights as +-d0 in tensor memory.
//
// A first kernel writes the activations' f16 parts (linear.cuh) once, in the order in which a sign word's bits become pairs.  A tile of the second
// is two 128-row matrices (gate and up of a pair, or two neighbouring row tiles) by 64 to 128 tokens, so that a copied activation meets 256 rows.
// Roles of a thread block (one an SM, tiles in turn):
//   warps 0, 1: MMAs, a warp for each matrix.  A stage is 64 of n: four steps of 16 for each part.
//   warp 2: TMA copies of the stage's parts (128-byte swizzle)
//   warps 4-11: weights.  A thread has a row of one matrix; two words of signs become 32 registers of +-d0 pairs by a shift and a logic
//              operation each, and go to the stage's slot of tensor memory (the operand A), so shared memory is read for B alone
//   warps 12-19: sums.  A round is 128 of n (65536 where one part is taken: bf16 results): the tensor cores truncate the sum that they add to, so
//              it leaves tensor memory after each round and is added in registers; the rounds of the two matrices are staggered, so one
//              is drained while the other's MMAs run.  The small parts of a round come first, while its sum is small: 1.0e-7 of the
//              result over 6912 (large and small by stages: 1.9e-7, in rounds of 256 3.1e-7; f32 products by cuBLAS 6.8e-7).  Behind the last
//              round the function, the residual, the conversion and the stores, while the next tile's MMAs start.
// Tensor memory: 2 x 128 columns of sums, 4 stages x 64 columns of weights.  Where the tiles are fewer than the SMs, n is cut into equal
// shares, whose sums a third kernel adds in order before the epilogue.
#include "linear.cuh"
#include "tc_common.cuh"

namespace gq {
GQ_ERROR_ACCESSOR(linear_tiles)

namespace {

constexpr int BM = 128, BK = 64, kStages = 4, kTmemCols = 512;
constexpr int kDCols = 128, kA0 = 2 * kDCols, kACols = BK / 2;            // a stage's slot: kACols for each matrix
constexpr int kTileB = 128 * BK * 2;                                       // a part of up to 128 tokens; a stage has two
constexpr int kStaged = 2 * 32 * 32 * 4;                                   // of a sums warp: half its columns of both matrices
constexpr int kWarpA0 = 4, kWarpE0 = 12, kEWarps = 8, kThreads = 640;
constexpr int kRegs = 96, kRegsSums = 176, kRegsRest = 40;                 // a thread's at launch, of 8 warps, of the other 12
static_assert(kA0 + kStages * 2 * kACols <= kTmemCols, "TMEM columns");
static_assert(kRegsSums * 256 + kRegsRest * 384 <= kRegs * kThreads && kRegs * kThreads <= 65536, "registers");

struct Bars {
    uint64_t full[kStages];            // eight weight warps, the copy's expect_tx and its bytes
    uint64_t done[kStages];            // both matrices' MMAs of the stage are complete: its slots are free
    uint64_t accfull[2], accempty[2];  // a matrix's round is complete; drained
    uint64_t final_;
    int last_copy[kStages];            // the last copy into each slot, -1: none
    uint32_t tmem_base;
    int abort;
};

struct Plan {
    int row_tiles, tok_tiles, splits, units, round, parts, pad_rows;
    const float* scale;                // a token's power of two, undone after the sums
    float* partial;                    // [split][matrix][token][pad_rows], splits > 1
};

// Issued by the one lane whose `leader` is set, with the whole warp on the way: descriptors then stay in uniform registers (from a branch of one
// lane an issue took 130 cycles: 4096 tokens, 14336 x 4096, bf16: 937 us)
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t leader, void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)), "r"(leader)
        : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t* r) {     // 32 lanes x 16 columns
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void ld8(uint32_t taddr, uint32_t* r) {            // 32 lanes x 8 columns
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// A unit's tile and its stages [k0, k1)
struct Unit { int row_tile, tok0, split, k0, k1; };
template <int BN>
__device__ __forceinline__ Unit unit_of(const Plan& p, int u, int nb) {
    const int split = u % p.splits, tile = u / p.splits;
    Unit r;
    r.row_tile = tile % p.row_tiles;
    r.tok0 = tile / p.row_tiles * BN;
    r.split = split;
    r.k0 = 2 * static_cast<int>(static_cast<long long>(nb) * split / p.splits);
    r.k1 = 2 * static_cast<int>(static_cast<long long>(nb) * (split + 1) / p.splits);
    return r;
}

template <int BN, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) linear_tiles_kernel(const __grid_constant__ CUtensorMap tmB, const LinearArgs a, const Plan plan) {
    constexpr uint32_t kIdesc = (1u << 4) | (static_cast<uint32_t>(BN >> 3) << 17) | (static_cast<uint32_t>(BM >> 4) << 24);   // f32 += f16 x f16
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sB = smem_align1024(smem_raw);                                // [stage][part][BN rows of 128 bytes]
    uint8_t* staged = sB + kStages * 2 * kTileB;                               // [sums warp][matrix][column][32 rows] f32
    Bars* bars = reinterpret_cast<Bars*>(staged + kEWarps * kStaged);
    volatile int* abort = &bars->abort;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int nb = a.n / 128, parts = plan.parts, half_round = plan.round / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars->full[s], 9);
            mbar_init(&bars->done[s], 2);
            bars->last_copy[s] = -1;
        }
        for (int m = 0; m < 2; ++m) {
            mbar_init(&bars->accfull[m], 1);
            mbar_init(&bars->accempty[m], kEWarps);
        }
        mbar_init(&bars->final_, 2);
        bars->abort = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp >= kWarpE0) {
        // ---------------- sums
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSums));
        asm volatile("griddepcontrol.wait;" ::: "memory");
        constexpr int NC = BN / 2;                                         // columns of this warp, of each matrix
        const int q = warp & 3, h = (warp - kWarpE0) >> 2;
        const uint32_t at = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h * NC);
        uint32_t turn[2] = {0, 0};                                         // rounds of each matrix so far
        bool ok = true;
        for (int u = blockIdx.x; u < plan.units && ok; u += gridDim.x) {
            const Unit w = unit_of<BN>(plan, u, nb);
            const int row0 = (PAIR ? w.row_tile : 2 * w.row_tile) * BM + q * 32, row1 = PAIR ? row0 : row0 + BM;
            const int tok0 = w.tok0 + h * NC;
            // what the epilogue needs is loaded before the sums come: a column's power of two is with lane column % 32
            const int sub = lane & 7, r0 = row0 + 4 * sub, r1 = row1 + 4 * sub;
            float b0[4], b1[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                b0[i] = a.bias[0] && r0 + i < a.rows ? a.bias[0][r0 + i] : 0.f;
                b1[i] = a.bias[1] && r1 + i < a.rows ? a.bias[1][r1 + i] : 0.f;
            }
            const int second = NC / 2 + ((lane - NC / 2) & 31);            // the second half's columns
            const float scales = tok0 + lane < a.cols ? plan.scale[tok0 + lane] : 0.f;
            const float scales2 = second < NC && tok0 + second < a.cols ? plan.scale[tok0 + second] : 0.f;
            if (!PAIR && a.residual && plan.splits == 1)
                for (int i = lane; i < 2 * NC; i += 32) {                  // a line of 32 rows of each token, into L2
                    const int tok = tok0 + i % NC, row = i < NC ? row0 : row1;
                    if (tok < a.cols && row < a.rows) {
                        const size_t at = (tok * static_cast<size_t>(a.residual_stride) + row) * (a.type == GQ_F32 ? 4 : 2);
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(a.residual) + at));
                    }
                }
            float acc[2][NC];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < NC; ++i) acc[m][i] = 0.f;
            auto drain = [&](int m, float (&sum)[NC]) {
                ok = __all_sync(0xffffffffu, ok && wait_or_abort_sleep(&bars->accfull[m], turn[m] & 1u, abort));
                if (!ok) return;
                ++turn[m];
                tc_fence_after();
                constexpr int AT_ONCE = NC <= 48 ? NC : 16;                // columns whose loads are in flight together
#pragma unroll
                for (int c = 0; c < NC; c += AT_ONCE) {
                    uint32_t v[AT_ONCE];
#pragma unroll
                    for (int o = 0; o < AT_ONCE && c + o < NC; o += 16) {
                        if (o + 16 <= AT_ONCE && c + o + 16 <= NC) ld16(at + static_cast<uint32_t>(m * kDCols + c + o), v + o);
                        else ld8(at + static_cast<uint32_t>(m * kDCols + c + o), v + o);
                    }
                    wait_ld();
                    if (c + AT_ONCE >= NC) {                               // read: the next round may begin
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars->accempty[m]);
                    }
#pragma unroll
                    for (int i = 0; i < AT_ONCE; ++i)
                        if (c + i < NC) sum[c + i] += __uint_as_float(v[i]);
                }
            };
            // the second matrix's rounds end in the middle of the first one's
            for (int k = half_round; k < w.k1 - w.k0; k += 2 * half_round) {
                drain(1, acc[1]);
                if (k + half_round < w.k1 - w.k0) drain(0, acc[0]);
            }
            drain(0, acc[0]);
            drain(1, acc[1]);
            if (!ok) break;
            if (plan.splits > 1) {
                float* to = plan.partial + (static_cast<size_t>(w.split) * (PAIR ? 2 : 1) * a.cols + tok0) * plan.pad_rows;
                const size_t second = PAIR ? static_cast<size_t>(a.cols) * plan.pad_rows : 0;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    if (tok0 + i >= a.cols) break;
                    to[static_cast<size_t>(i) * plan.pad_rows + row0 + lane] = acc[0][i];
                    if (PAIR || row1 < plan.pad_rows) to[second + static_cast<size_t>(i) * plan.pad_rows + row1 + lane] = acc[1][i];
                }
                continue;
            }
            // Through shared memory, in two halves, to four rows a lane and four tokens a step: a loop that fits the instruction cache, with a third of
            // the instructions that a row a lane takes.  (Unrolled over registers: 517 tokens of the 6912 x 2560 pair in f32 to Q8_0, 22,000
            // of a tile's 62,000 cycles went into this.)
            constexpr int HC = NC / 2;
            float* own = reinterpret_cast<float*>(staged + (warp - kWarpE0) * kStaged);
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < HC; ++i) {
                    own[i * 32 + lane] = acc[0][i];
                    own[(HC + i) * 32 + lane] = acc[1][i];
                    acc[0][i] = acc[0][HC + i];
                    acc[1][i] = acc[1][HC + i];
                }
                __syncwarp();
                constexpr int G = HC % 16 == 0 || HC % 16 == 12 ? 4 : 2;   // steps of 16 or 8 tokens, the last one's up to four too many without effect
                const int end = min(a.cols, tok0 + (half + 1) * HC);
#pragma unroll 1
                for (int c = lane >> 3; c < HC; c += 4 * G) {
                    const int tok = tok0 + half * HC + c;
                    float other[4 * G], z0[4 * G], z1[4 * G], more[4 * G];
                    if (!PAIR)
#pragma unroll
                        for (int g = 0; g < G; ++g) {
                            load_four(a, other + 4 * g, r0, tok + 4 * g, tok + 4 * g < end);
                            load_four(a, more + 4 * g, r1, tok + 4 * g, tok + 4 * g < end);
                        }
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const float s = __shfl_sync(0xffffffffu, half ? scales2 : scales, (half * HC + c + 4 * g) & 31);
                        const float4 u = *reinterpret_cast<const float4*>(own + (c + 4 * g) * 32 + 4 * sub);
                        const float4 v = *reinterpret_cast<const float4*>(own + (HC + c + 4 * g) * 32 + 4 * sub);
                        const float u4[4] = {u.x, u.y, u.z, u.w}, v4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            z0[4 * g + i] = fmaf(u4[i], s, b0[i]);         // the products are exact
                            z1[4 * g + i] = fmaf(v4[i], s, b1[i]);
                        }
                    }
                    if constexpr (PAIR) {
                        finish_fours<true, G>(a, z0, z1, r0, tok, end, lane);
                    } else {
                        finish_fours<false, G>(a, z0, other, r0, tok, end, lane);
                        finish_fours<false, G>(a, z1, more, r1, tok, end, lane);
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
        if (warp < 2) {
            // ---------------- MMAs: an issuer for each matrix
            asm volatile("griddepcontrol.wait;" ::: "memory");         // the limit of a wait counts from here, not while earlier work runs
            const int m = warp;
            const uint32_t leader = elect_one();
            const uint32_t d = tmem + static_cast<uint32_t>(m * kDCols);
            uint32_t g = 0, turn = 0;
            bool live = true;
            for (int u = blockIdx.x; u < plan.units && live; u += gridDim.x) {
                const Unit w = unit_of<BN>(plan, u, nb);
                int r = m * half_round;                                    // stages of the round
                bool first = true;
                for (int k = w.k0; k < w.k1;) {
                    // up to two stages of a round, the small parts of both first
                    const int here = parts == 2 && r < 2 * half_round - 1 && k < w.k1 - 1 ? 2 : 1;
                    const int s[2] = {static_cast<int>(g % kStages), static_cast<int>((g + 1) % kStages)};
                    bool ready = wait_or_abort_sleep(&bars->full[s[0]], (g / kStages) & 1u, abort);
                    if (here == 2) ready = ready && wait_or_abort_sleep(&bars->full[s[1]], ((g + 1) / kStages) & 1u, abort);
                    ready = ready && (!first || turn == 0 || wait_or_abort_sleep(&bars->accempty[m], (turn - 1) & 1u, abort));
                    if (!__all_sync(0xffffffffu, ready)) {
                        live = false;
                        break;
                    }
                    tc_fence_after();
                    const bool last = r + here == 2 * half_round || k + here == w.k1;
                    bool fresh = first;
#pragma unroll
                    for (int p = 1; p >= 0; --p) {
                        if (p == 1 && parts == 1) continue;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (i == here) break;
                            const uint64_t bdesc = smem_desc(sB + s[i] * 2 * kTileB);
                            const uint32_t av = tmem + static_cast<uint32_t>(kA0 + (2 * s[i] + m) * kACols);
#pragma unroll
                            for (int j = 0; j < BK / 16; ++j) {
                                mma_ts(leader, d, av + static_cast<uint32_t>(j * 8), bdesc + static_cast<uint64_t>((p * kTileB + j * 32) >> 4), kIdesc, fresh ? 0u : 1u);
                                fresh = false;
                            }
                            if (p == 0 && leader) tc_commit(&bars->done[s[i]]);
                        }
                    }
                    if (last && leader) tc_commit(&bars->accfull[m]);
                    __syncwarp();
                    first = last;
                    r = last ? 0 : r + here;
                    turn += last;
                    k += here;
                    g += here;
                }
            }
            if (leader) tc_commit(&bars->final_);
            __syncwarp();
        } else if (warp == 2) {
            // ---------------- copies of the activations
            const uint32_t leader = elect_one();
            if (leader) prefetch_tmap(&tmB);
            asm volatile("griddepcontrol.wait;" ::: "memory");
            uint32_t g = 0;
            bool live = true;
            for (int u = blockIdx.x; u < plan.units && live; u += gridDim.x) {
                const Unit w = unit_of<BN>(plan, u, nb);
                for (int k = w.k0; k < w.k1; ++k, ++g) {
                    const int s = g % kStages;
                    if (g >= kStages && !__all_sync(0xffffffffu, wait_or_abort_sleep(&bars->done[s], (g / kStages - 1) & 1u, abort))) {
                        live = false;
                        break;
                    }
                    if (leader) {
                        mbar_arrive_expect_tx(&bars->full[s], static_cast<uint32_t>(parts * BN * 128));
                        bars->last_copy[s] = static_cast<int>(g);
                    }
                    __syncwarp();
                    for (int p = 0; p < parts; ++p)
                        tma_load(leader, sB + (s * 2 + p) * kTileB, &tmB, k * BK, p * a.cols + w.tok0, &bars->full[s]);
                }
            }
        } else if (warp >= kWarpA0) {
            // ---------------- weights: four warps for each matrix
            const int r = (warp & 3) * 32 + lane, m = (warp - kWarpA0) >> 2;
            const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + static_cast<uint32_t>(kA0 + m * kACols);
            const int tiles = (a.rows + BM - 1) / BM;
            uint32_t g = 0;
            bool live = true;
            for (int u = blockIdx.x; u < plan.units && live; u += gridDim.x) {
                const Unit w = unit_of<BN>(plan, u, nb);
                const uint8_t* src = (m ? a.w[1] : a.w[0]) + static_cast<size_t>(PAIR ? w.row_tile : min(2 * w.row_tile + m, tiles - 1)) * nb * kChunkBytes +
                                     static_cast<size_t>(w.k0 / 2) * kChunkBytes;
                uint4 bits;
                uint32_t d0;
                auto load = [&] {
                    bits = *reinterpret_cast<const uint4*>(src + r * 16);
                    d0 = *reinterpret_cast<const uint16_t*>(src + BM * 16 + r * 2);
                    src += kChunkBytes;
                };
                load();
                for (int k = w.k0; k < w.k1 && live; k += 2) {
                    const uint32_t words[4] = {bits.x, bits.y, bits.z, bits.w}, neg = (d0 * 0x00010001u) ^ 0x80008000u;   // a clear bit gives -d0
                    if (k + 2 < w.k1) load();
#pragma unroll
                    for (int half = 0; half < 2; ++half, ++g) {
                        const int s = g % kStages;
                        uint32_t av[16];
                        auto expand = [&](uint32_t word) {
#pragma unroll
                            for (int p = 0; p < 16; ++p) av[p] = ((word << (15 - p)) & 0x80008000u) ^ neg;
                        };
                        expand(words[2 * half]);
                        // the first stages' weights go ahead of earlier work, as the packed weights are no part of it
                        if (g == kStages) asm volatile("griddepcontrol.wait;" ::: "memory");
                        if (g >= kStages && !__all_sync(0xffffffffu, wait_or_abort_sleep(&bars->done[s], (g / kStages - 1) & 1u, abort))) {
                            live = false;
                            break;
                        }
                        tc_fence_after();
                        st16(at + static_cast<uint32_t>(2 * s * kACols), av);
                        expand(words[2 * half + 1]);
                        st16(at + static_cast<uint32_t>(2 * s * kACols + 16), av);
                        // at once: arriving behind the next stage's expansion, or for two stages together, costs more than it hides
                        // (4096 tokens, 14336 x 4096, bf16: 531 us; 546, 571)
                        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars->full[s]);
                    }
                }
            }
        }
    }

    // ---------------- teardown
    __syncwarp();
    if (warp == 0) {
        if (lane == 0 && !mbar_wait(&bars->final_, 0)) report_error(kErrMmaTimeout);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 64 && *abort) {
        // an aborted block may hold copies that no MMA waited for
        for (int s = 0; s < kStages; ++s) {
            const int g = bars->last_copy[s];
            if (g >= 0 && !mbar_wait(&bars->full[s], static_cast<uint32_t>(g / kStages) & 1u)) report_error(kErrDrainTimeout);
        }
    }
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    __syncthreads();
}

// The f16 parts [part][token][n] of the activations, and each token's power of two.  One block a token.  In a 32-block, place 2 p + i holds
// element 4 (p % 8) + p / 8 + 2 i, as bits p and p + 16 of a packed sign word.
constexpr int kSplitThreads = 256;
__global__ void __launch_bounds__(kSplitThreads) linear_split_kernel(const uint8_t* act, int nb32, int cols, int parts, uint32_t* out, float* scale) {
    __shared__ uint32_t largest[kSplitThreads / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const size_t tok = blockIdx.x;
    const uint8_t* p = act + tok * nb32 * 34;
    uint32_t top = 0;
    for (int b = threadIdx.x; b < nb32; b += kSplitThreads) top = max(top, *reinterpret_cast<const uint16_t*>(p + static_cast<size_t>(b) * 34) & 0x7fffu);
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) largest[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSplitThreads / 32; ++i) top = max(top, largest[i]);
    const int shift = token_shift(top);
    if (threadIdx.x == 0) scale[tok] = pow2(-shift);
    uint32_t* row = out + tok * nb32 * 16;
    const size_t second = static_cast<size_t>(cols) * nb32 * 16;
    for (int i = threadIdx.x; i < nb32 * 8; i += kSplitThreads) {
        const uint16_t* blk = reinterpret_cast<const uint16_t*>(p + static_cast<size_t>(i >> 3) * 34);
        const int l = i & 7;
        const float d = f16_to_f32(blk[0]) * pow2(shift);
        const uint32_t lo = blk[1 + 2 * l], hi = blk[2 + 2 * l];
        const float v[4] = {d * static_cast<float>(static_cast<int8_t>(lo & 0xff)), d * static_cast<float>(static_cast<int8_t>(lo >> 8)),
                            d * static_cast<float>(static_cast<int8_t>(hi & 0xff)), d * static_cast<float>(static_cast<int8_t>(hi >> 8))};
        uint16_t h[4], low[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) two_parts(v[e], h[e], low[e]);
        uint32_t* to = row + static_cast<size_t>(i >> 3) * 16 + l;
        to[0] = h[0] | static_cast<uint32_t>(h[2]) << 16;
        to[8] = h[1] | static_cast<uint32_t>(h[3]) << 16;
        if (parts == 2) {
            to[second] = low[0] | static_cast<uint32_t>(low[2]) << 16;
            to[second + 8] = low[1] | static_cast<uint32_t>(low[3]) << 16;
        }
    }
}

// The shares' sums in order, and the epilogue.  A warp has 32 rows of four tokens.
template <bool PAIR>
__global__ void __launch_bounds__(256) linear_join_kernel(const LinearArgs a, const Plan plan) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, groups = (a.rows + 31) / 32, quads = (a.cols + 3) / 4;
    const long long id = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) >> 5;
    if (id >= static_cast<long long>(groups) * quads) return;
    const int tok = static_cast<int>(id / groups) * 4 + (lane >> 3), row = static_cast<int>(id % groups) * 32 + 4 * (lane & 7);
    const bool on = tok < a.cols;
    const size_t matrix = static_cast<size_t>(a.cols) * plan.pad_rows;
    const float* from = plan.partial + static_cast<size_t>(on ? tok : 0) * plan.pad_rows + row;
    float other[4], y[4];
    if (!PAIR) load_four(a, other, row, tok, on);
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
#pragma unroll 4
    for (int s = 0; s < plan.splits; ++s) {
        const float4 p = *reinterpret_cast<const float4*>(from + (PAIR ? 2 : 1) * s * matrix);
        u = make_float4(u.x + p.x, u.y + p.y, u.z + p.z, u.w + p.w);
        if (PAIR) {
            const float4 o = *reinterpret_cast<const float4*>(from + (2 * s + 1) * matrix);
            v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
        }
    }
    const float sc = on ? plan.scale[tok] : 0.f;
    const float z0[4] = {u.x, u.y, u.z, u.w}, z1[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool there = row + i < a.rows;
        y[i] = fmaf(z0[i], sc, a.bias[0] && there ? a.bias[0][row + i] : 0.f);
        if (PAIR) other[i] = fmaf(z1[i], sc, a.bias[1] && there ? a.bias[1][row + i] : 0.f);
    }
    finish_fours<PAIR, 1>(a, y, other, row, tok, a.cols, lane);
}

template <typename K, typename... A>
cudaError_t launch(K kernel, unsigned grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
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

constexpr int kSMs = 152, kMaxTokens = 128;

struct Shape { int bn; Plan p; float us; };
int most_splits(int nb) { return std::min(16, std::max(1, nb / 2)); }
struct Tile { int tokens; float once[2], stage[2]; };                      // once: linear, pair; a stage: of one part, of two
// Tokens a tile and shares of n, by their cost in microseconds, fitted to calls of 16 to 517 tokens (2560 x 2560, 2560 x 6912, pairs of 6912 x 2560 and
// 14336 x 4096): what a tile takes once (start, epilogue), its stages (two parts: the MMAs; one: the weights' way into tensor memory), more
// tiles an SM, and the shares' sums written and read again.  For long prompts they only rank the tiles, and are no times: 4096 tokens of 2560 x 6912 f32 149 us by them,
// 207 measured with the parts' write; of the 14336 x 4096 bf16 pair 481 and 537.
Shape shape_of(int rows, int n, int cols, int parts, bool pair) {
    const int tiles = (rows + BM - 1) / BM, nb = n / 128;
    Shape best = {};
    static constexpr Tile kTiles[] = {{128, {13.6f, 8.9f}, {0.278f, 0.541f}}, {112, {10.7f, 9.0f}, {0.255f, 0.476f}}, {96, {10.1f, 7.9f}, {0.272f, 0.412f}},
                                      {80, {9.0f, 8.4f}, {0.256f, 0.354f}}, {64, {7.7f, 6.5f}, {0.278f, 0.346f}}};
    for (const Tile& tile : kTiles) {
        const int bn = tile.tokens;
        const float once = tile.once[pair], stage = tile.stage[parts - 1];
        const int row_tiles = pair ? tiles : (tiles + 1) / 2, tok_tiles = (cols + bn - 1) / bn;
        const long long all = static_cast<long long>(row_tiles) * tok_tiles;
        for (int splits = 1; splits <= most_splits(nb); ++splits) {
            const long long units = all * splits, waves = (units + kSMs - 1) / kSMs;
            if (splits > 1 && units > kSMs) break;                         // shares are for SMs that would be idle
            const float sums = splits == 1 ? 0.f : 0.2f + static_cast<float>(splits) * cols * rows * (pair ? 2 : 1) * 4 * (1 / 2.4e6f);
            const float us = once + waves * 2 * ((nb + splits - 1) / splits) * stage + (waves - 1) * (once - 5) * 0.5f + sums;
            if (best.bn == 0 || us < best.us) {
                Plan p = {};
                p.row_tiles = row_tiles;
                p.tok_tiles = tok_tiles;
                p.splits = splits;
                p.units = static_cast<int>(std::min<long long>(units, 0x7fffffff));
                p.parts = parts;
                // two parts: 128 of n, 16 steps; one (bf16): 65536
                p.round = parts == 2 ? 2 : 1024;
                p.pad_rows = tiles * BM;
                best = {bn, p, us};
            }
        }
    }
    return best;
}

size_t up(size_t v) { return (v + 255) / 256 * 256; }
size_t parts_bytes(int n, int cols) { return up(static_cast<size_t>(2) * cols * n * 2); }

template <int BN, bool PAIR>
cudaError_t tiles_go(const LinearArgs& a, const Plan& p, const void* parts, cudaStream_t s) {
    CUtensorMap tmB;
    if (!make_tmap_2d(&tmB, parts, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, static_cast<uint64_t>(a.n), static_cast<uint64_t>(p.parts) * a.cols,
                      static_cast<uint64_t>(a.n) * 2, BK, BN, true))
        return cudaErrorInvalidValue;
    constexpr size_t smem = 1024 + static_cast<size_t>(kStages) * 2 * kTileB + kEWarps * kStaged + sizeof(Bars);
    static std::atomic<uint64_t> raised{0};
    cudaError_t e = allow_smem(linear_tiles_kernel<BN, PAIR>, smem, raised);
    if (e != cudaSuccess) return e;
    e = launch(linear_tiles_kernel<BN, PAIR>, static_cast<unsigned>(std::min(p.units, kSMs)), kThreads, smem, s, tmB, a, p);
    if (e != cudaSuccess || p.splits == 1) return e;
    const long long warps = static_cast<long long>((a.rows + 31) / 32) * ((a.cols + 3) / 4);
    return launch(linear_join_kernel<PAIR>, static_cast<unsigned>((warps + 7) / 8), 256, 0, s, a, p);
}

template <bool PAIR>
cudaError_t tiles_by(const Shape& t, const LinearArgs& a, const void* parts, cudaStream_t s) {
    switch (t.bn) {
        case 128: return tiles_go<128, PAIR>(a, t.p, parts, s);
        case 112: return tiles_go<112, PAIR>(a, t.p, parts, s);
        case 96: return tiles_go<96, PAIR>(a, t.p, parts, s);
        case 80: return tiles_go<80, PAIR>(a, t.p, parts, s);
        default: return tiles_go<64, PAIR>(a, t.p, parts, s);
    }
}

}  // namespace

// Of a call of up to `cols` tokens: shares are taken for few tokens only, so that fewer tokens may need more than many do.  A call of s > 1 shares has at most
// kSMs units, so tokens of at most kSMs / (s row_tiles) tiles of up to kMaxTokens.
size_t linear_tiles_workspace_bytes(int rows, int n, int cols, bool pair) {
    const long long tiles = (rows + BM - 1) / BM, row_tiles = pair ? tiles : (tiles + 1) / 2;
    const size_t row_bytes = static_cast<size_t>(tiles) * BM * 4 * (pair ? 2 : 1);         // a token's sums of one share
    size_t partial = 0;
    for (int s = 2; s <= most_splits(n / 128) && s * row_tiles <= kSMs; ++s) {
        const size_t tokens = std::min<long long>(cols, kSMs / (s * row_tiles) * kMaxTokens);
        partial = std::max(partial, s * tokens * row_bytes);
    }
    return parts_bytes(n, cols) + up(static_cast<size_t>(cols) * 4) + partial;
}

int linear_tiles_plan(int rows, int n, int cols, int parts, bool pair) {
    const Shape t = shape_of(rows, n, cols, parts, pair);
    return t.bn + 256 * t.p.splits;
}

float linear_tiles_us(int rows, int n, int cols, int parts, bool pair) { return shape_of(rows, n, cols, parts, pair).us; }

cudaError_t launch_linear_tiles(const LinearArgs& a, bool pair, cudaStream_t s) {
    Shape t = shape_of(a.rows, a.n, a.cols, linear_parts(a), pair);
    uint8_t* work = static_cast<uint8_t*>(a.workspace);
    float* scale = reinterpret_cast<float*>(work + parts_bytes(a.n, a.cols));
    t.p.scale = scale;
    t.p.partial = reinterpret_cast<float*>(work + parts_bytes(a.n, a.cols) + up(static_cast<size_t>(a.cols) * 4));
    const cudaError_t e = launch(linear_split_kernel, static_cast<unsigned>(a.cols), kSplitThreads, 0, s, a.act, a.n / 32, a.cols, t.p.parts,
                                 reinterpret_cast<uint32_t*>(work), scale);
    if (e != cudaSuccess) return e;
    return pair ? tiles_by<true>(t, a, work, s) : tiles_by<false>(t, a, work, s);
}

}  // namespace gq
