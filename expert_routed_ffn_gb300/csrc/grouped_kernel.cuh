// The persistent kernel of the products over expert-grouped rows (grouped.cu says how it works)
// and what fills its arguments: the forward product and its two gradients, and the three products
// of the gated block (gated.cu), which differ in where an operand's tile comes from and in what
// the epilogue makes of the sums.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "gated.cuh"
#include "grouped.cuh"
#include "kernels.h"
#include "op_host.h"

namespace moe {

// kGated: Wg and Wu as one operand, act(gate, up) stored; kGatedBack: a dgrad whose sums are dH, dG
// and dU stored; kDgradTwo: the sum of two dgrads, as one reduction over both
enum : int { kForward = 0, kDgrad = 1, kWgrad = 2, kGated = 3, kGatedBack = 4, kDgradTwo = 5 };
template <int OP>
constexpr bool kColumnsKMajor = OP == kForward || OP == kGated;  // the A operand's tile
constexpr int kGranule = 16;           // kGated: columns of one projection side by side in a tile

constexpr int kBK = 64;                // reduction steps per stage: 128 bytes of bf16
constexpr int kMaxStages = 12;
// Epilogue warps per TMEM lane quadrant.  One against two: a small product 11.7 / 11.0 us, a
// small bf16 weight gradient 26.6 / 24.6 us, prefill the same.
// Twice as many where the epilogue computes the activation or its gradients (gated.cuh).
template <int OP>
constexpr int kParts = OP == kGated || OP == kGatedBack ? 4 : 2;
template <int OP>
constexpr int kEpiWarps = kQuads * kParts<OP>;
template <int OP>
constexpr int kThreads = 64 + 32 * kEpiWarps<OP> + (OP == kWgrad ? 32 : 0);  // the wgrad's last warp zeroes tails
static_assert(kThreads<kForward> >= kMaxExperts, "load_table: a thread per expert");
constexpr int kAccCols = 256;          // TMEM columns of one accumulator
constexpr uint32_t kTmemCols = 2 * kAccCols;
constexpr int kRow = kBK * 2;          // bytes of a K-major row, or of 64 columns in MN-major
constexpr int kChunk = 64 * kRow;      // an MN-major tile of 64 columns x 64 reduction rows
constexpr int kBoxes = 8;              // B boxes of 16, 32, .. 128 rows (K-major)
constexpr int kStageSpace = 229376;    // 224 KB of stages

// Shared memory: the header, then the stages.
struct Header {
    uint64_t bars[4 * kMaxStages + 5];
    TileTable table;
    GatedOut gated;
    uint32_t tmem;
    volatile int abort;
};
constexpr int kHeaderBytes = 3 << 10;
constexpr int kSmemBytes = kHeaderBytes + kStageSpace;
static_assert(sizeof(Header) <= kHeaderBytes && kSmemBytes <= 232448, "shared memory of one CTA");

struct GroupedArgs {
    CUtensorMap map_a, map_b[kBoxes];
    GroupedOut o;
    int a_block, b_block;  // bytes of 64 reduction steps per CTA
    int stages;
};
struct GatedArgs : GroupedArgs {
    CUtensorMap map_a2;  // Wu
    GatedOut gated;
};
struct DgradTwoArgs : GroupedArgs {
    CUtensorMap map_a2, map_b2[kBoxes];
    int split;  // reduction steps of the first product, a multiple of 64
};
template <int OP>
struct ArgsOf {
    using type = GroupedArgs;
};
template <>
struct ArgsOf<kGated> {
    using type = GatedArgs;
};
template <>
struct ArgsOf<kGatedBack> {
    using type = GatedArgs;
};
template <>
struct ArgsOf<kDgradTwo> {
    using type = DgradTwoArgs;
};

// Tensor-core descriptor of an MN-major tile: 64 contiguous elements (128 bytes) per
// reduction row, 128-byte swizzle; 8 reduction rows are 1024 bytes apart (stride byte
// offset) and the next 64 elements one kChunk (leading byte offset).
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(kChunk >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
}
// BLOCKS: most blocks of 64 reduction steps of a stage; ADD: to what the output holds (wgrad);
// SEGMENTS: a sum may come in several (grouped.cuh)
template <int OP, int BLOCKS, bool ADD, bool SEGMENTS>
__global__ void __launch_bounds__(kThreads<OP>, 1) grouped_kernel(const __grid_constant__ typename ArgsOf<OP>::type p) {
    constexpr bool kDense = OP == kWgrad;
    constexpr bool kRegisters = SEGMENTS && OP == kDgradTwo;  // a tile's segments: RegisterSums
    constexpr bool kWalkSegments = SEGMENTS && !kRegisters;
    extern __shared__ __align__(1024) uint8_t smem[];
    Header &h = *reinterpret_cast<Header *>(smem);
    const TileTable &tab = h.table;
    const uint32_t base = smem_u32(smem) + kHeaderBytes;
    const int a_block = p.a_block, b_block = p.b_block, stages = p.stages;
    // all A blocks first: the MMA reads 128 columns of A where the box brought 64; the rest is
    // whatever follows, and its results are not stored
    const uint32_t sA = base, sB = base + (uint32_t)(stages * BLOCKS * a_block);
    const uint32_t bar0 = smem_u32(h.bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    auto tail_bar = [&](int s) { return bar0 + 8u * (2 * kMaxStages + s); };
    auto zeroed_bar = [&](int s) { return bar0 + 8u * (3 * kMaxStages + s); };
    auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (4 * kMaxStages + a); };
    auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (4 * kMaxStages + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (4 * kMaxStages + 4);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = rank == 0;
    volatile int *abort_flag = &h.abort;
    auto raise = [&]() {  // stops both CTAs' roles
        atomicOr(p.o.err, ERR_TIMEOUT);
        *abort_flag = 1;
        st_cluster_s32(mapa_shared(smem_u32(const_cast<int *>(&h.abort)), (uint32_t)rank ^ 1u), 1);
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
            mbar_init(tail_bar(s), 1);
            mbar_init(zeroed_bar(s), 2);  // both CTAs'
        }
        for (uint32_t a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 2 * kEpiWarps<OP>);  // both CTAs'
        }
        mbar_init(drain_bar, 1);
        fence_mbar_init();
        h.abort = 0;
        tma_prefetch_desc(&p.map_a);
        tma_prefetch_desc(&p.map_b[0]);
    }
    if (threadIdx.x == 64) {
        start_table<kDense>(p.o, h.table);
        if constexpr (OP == kGated || OP == kGatedBack) h.gated = p.gated;
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&h.tmem), kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any copy or arrival crosses over
    tc_fence_after();
    const uint32_t tmem_base = h.tmem;
    pdl_wait();  // the offsets and operands of earlier kernels on the stream
    pdl_trigger();
    if (!load_table<kDense>(h.table) && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.o.err, ERR_BOUNDS);
    const int first = (int)blockIdx.x / 2, stride = (int)gridDim.x / 2;
    const int half_cols = tab.o.cols / 2;
    // blocks of the stage at reduction step r: those left, of the wgrad two only if both are whole
    auto blocks_at = [&](const Tile &t, int r) {
        if (BLOCKS == 1) return 1;
        return kDense ? (t.r1 - r >= BLOCKS * kBK ? BLOCKS : 1) : min(BLOCKS, (t.r1 - r + kBK - 1) / kBK);
    };
    // wgrad: the stage at reduction row r ends inside a 16-row step
    auto is_tail = [&](const Tile &t, int r) { return kDense && t.r1 - r < kBK && (t.r1 - r) % 16 != 0; };

    if (warp == 0) {
        uint32_t ph = 1;
        int s = 0;
        bool ok = true;
        for (TileWalk<kDense, kWalkSegments> walk(tab, first, stride); ok && walk.more(); walk.next()) {
            const Tile t = walk.get();
            const int col = t.col0 + rank * half_cols, row = t.row0 + rank * (t.n / 2);
            const bool two_b = t.n / 2 > 64;  // MN-major B: two chunks of 64 columns
            const CUtensorMap *map_b = kDense ? &p.map_b[0] : &p.map_b[t.n / 32 - 1];  // K-major B: n / 2 rows
            const uint32_t bytes = a_block + (kDense ? (two_b ? 2 : 1) * kChunk : (t.n / 2) * kRow);
            for (int r = t.r0, here; r < t.r1; r += here * kBK) {
                here = blocks_at(t, r);
                if (!__all_sync(0xffffffffu, wait_bar(empty_bar(s), ph, p.o.wait + walk.slack, abort_flag))) {
                    ok = false;
                    break;
                }
                uint32_t da = sA + s * BLOCKS * a_block, db = sB + s * BLOCKS * b_block;
                const uint32_t bar = mapa_shared(full_bar(s), 0);
                if (is_tail(t, r)) {  // complete on this CTA's own barrier, for warp 10 to zero the rest
                    if (elect_one()) {
                        if (leader) mbar_arrive(full_bar(s));
                        mbar_arrive_expect_tx(tail_bar(s), bytes);
                        tma_load_2d(da, &p.map_a, tail_bar(s), col, r);
                        if (half_cols > 64) tma_load_2d(da + kChunk, &p.map_a, tail_bar(s), col + 64, r);
                        tma_load_2d(db, map_b, tail_bar(s), row, r);
                        if (two_b) tma_load_2d(db + kChunk, map_b, tail_bar(s), row + 64, r);
                    }
                } else if (elect_one()) {
                    if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * bytes * here);
#pragma unroll
                    for (int b = 0; b < BLOCKS; ++b, da += a_block, db += b_block) {
                        if (b >= here) break;
                        const int rb = r + b * kBK;
                        if constexpr (OP == kDgradTwo) {
                            const bool second = rb >= p.split;
                            const CUtensorMap *map_a = second ? &p.map_a2 : &p.map_a;
                            const int rs = rb - (second ? p.split : 0);
                            tma_load_3d_pair(da, map_a, bar, col, rs, t.e);
                            if (half_cols > 64) tma_load_3d_pair(da + kChunk, map_a, bar, col + 64, rs, t.e);
                            tma_load_2d_pair(db, second ? &p.map_b2[t.n / 32 - 1] : map_b, bar, rs, row);
                            continue;
                        } else if constexpr (OP == kGated) {
                            for (int c = 0; c < half_cols; c += 2 * kGranule) {
                                tma_load_3d_pair(da + c * kRow, &p.map_a, bar, rb, (col + c) / 2, t.e);
                                tma_load_3d_pair(da + (c + kGranule) * kRow, &p.map_a2, bar, rb, (col + c) / 2, t.e);
                            }
                        } else if (OP == kForward) {
                            tma_load_3d_pair(da, &p.map_a, bar, rb, col, t.e);
                        } else if (OP == kDgrad || OP == kGatedBack) {
                            tma_load_3d_pair(da, &p.map_a, bar, col, rb, t.e);
                            if (half_cols > 64) tma_load_3d_pair(da + kChunk, &p.map_a, bar, col + 64, rb, t.e);
                        } else {
                            tma_load_2d_pair(da, &p.map_a, bar, col, rb);
                            if (half_cols > 64) tma_load_2d_pair(da + kChunk, &p.map_a, bar, col + 64, rb);
                        }
                        if (OP != kWgrad) {
                            tma_load_2d_pair(db, map_b, bar, rb, row);
                        } else {
                            tma_load_2d_pair(db, map_b, bar, row, rb);
                            if (two_b) tma_load_2d_pair(db + kChunk, map_b, bar, row + 64, rb);
                        }
                    }
                }
                __syncwarp();
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) raise();
    } else if (warp == 1) {
        if (leader) {
            constexpr uint32_t kStepA = kColumnsKMajor<OP> ? 2 : (16 * kRow) >> 4;  // 16 reduction steps on,
            constexpr uint32_t kStepB = OP == kWgrad ? (16 * kRow) >> 4 : 2;    // in units of 16 bytes
            const uint64_t desc_a = kColumnsKMajor<OP> ? smem_desc_k128(sA) : smem_desc_mn128(sA);
            const uint64_t desc_b = kDense ? smem_desc_mn128(sB) : smem_desc_k128(sB);
            Accumulators accs;
            uint32_t ph = 0, zeroed_ph = 0;
            int s = 0;
            bool ok = p.o.wait != 0, issued = false;  // a bound of 0: give up at once
            TileWalk<kDense, kWalkSegments> walk(tab, first, stride);
            Tile next;
            [[maybe_unused]] int at = 0;  // kRegisters: the first of the segment's reduction steps
            auto advance = [&]() {
                walk.next();
                if (walk.more()) next = walk.get();
            };
            if (walk.more()) next = walk.get();
            while (ok && walk.more()) {
                Tile t = next;
                if (kRegisters) {
                    t.r0 = at;
                    t.r1 = min(t.r1, at + tab.o.segment);
                    at = t.r1 == tab.o.red ? 0 : t.r1;
                }
                if (t.r0 >= t.r1) {  // an expert without rows: the epilogue writes its zeros
                    advance();
                    continue;
                }
                const uint32_t idesc = idesc_bf16_f32(256, t.n) | (!kColumnsKMajor<OP> ? 1u << 15 : 0u) | (kDense ? 1u << 16 : 0u);
                const uint32_t a = accs.next, d = tmem_base + a * kAccCols;
                if (!__all_sync(0xffffffffu, wait_bar<true>(tempty_bar(a), accs.take(), p.o.wait + walk.slack, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int r = t.r0, here; r < t.r1; r += here * kBK) {
                    here = blocks_at(t, r);
                    bool got = wait_bar(full_bar(s), ph, p.o.wait, abort_flag);
                    if (is_tail(t, r)) {
                        got = got && wait_bar<true>(zeroed_bar(s), zeroed_ph >> s & 1u, p.o.wait, abort_flag);
                        zeroed_ph ^= 1u << s;
                    }
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    uint64_t ad = desc_a + (uint32_t)(s * BLOCKS * a_block >> 4), bd = desc_b + (uint32_t)(s * BLOCKS * b_block >> 4);
                    const int left = t.r1 - r;
                    if (elect_one()) {
#pragma unroll
                        for (int b = 0; b < BLOCKS; ++b) {
                            if (b >= here) break;
#pragma unroll
                            for (int k = 0; k < kBK / 16; ++k)
                                if (!kDense || b * kBK + 16 * k < left)
                                    tc_mma_bf16_pair(d, ad + k * kStepA, bd + k * kStepB, idesc, (r != t.r0) | (b + k != 0));
                            ad += (uint32_t)a_block >> 4;
                            bd += (uint32_t)b_block >> 4;
                        }
                        tc_commit_pair(empty_bar(s), 3);  // frees the stage in both CTAs
                        if (left <= here * kBK) tc_commit_pair(tfull_bar(a), 3);
                    }
                    __syncwarp();
                    issued = true;
                    // the next tile's place, while this one's products run
                    if (r == t.r0 && (!kRegisters || at == 0)) advance();
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                accs.done(t);
            }
            if (!ok && lane == 0) {
                raise();
                if (issued) {
                    tc_commit_pair(drain_bar, 1);
                    wait_bar(drain_bar, 0, kDrainCycles, nullptr);
                }
            }
        }
    } else if (kDense && warp == 2 + kEpiWarps<OP>) {
        // wgrad: zero the rows past each tail's end, then hand the stage to the MMA
        uint32_t tail_ph = 0;
        int s = 0;
        // This warp does not wait in tiles without a tail, so that its next wait may last as long as
        // all their stages do: the bound grows with them, by as much a stage as in wait_cycles.
        long long passed = 0;
        const int chunks_a = half_cols / 64;
        for (TileWalk<kDense, kWalkSegments> walk(tab, first, stride); walk.more(); walk.next()) {
            const Tile t = walk.get();
            const int whole = (t.r1 - t.r0) / (BLOCKS * kBK), rest = t.r1 - t.r0 - whole * (BLOCKS * kBK);
            const int tile_stages = whole + (rest + kBK - 1) / kBK;
            const int last = t.r1 - ((t.r1 - t.r0 - 1) % kBK + 1);  // first row of the last block
            if (tile_stages > 0 && is_tail(t, last)) {
                const int st = (s + tile_stages - 1) % stages;
                if (!__all_sync(0xffffffffu, wait_bar(tail_bar(st), tail_ph >> st & 1u, p.o.wait + walk.slack + passed, abort_flag))) {
                    if (lane == 0) raise();
                    break;
                }
                tail_ph ^= 1u << st;
                const uint32_t da = sA + st * BLOCKS * a_block, db = sB + st * BLOCKS * b_block;
                const int valid = t.r1 - last, words = ((valid + 15) / 16 * 16 - valid) * (kRow / 16);
                const int chunks = chunks_a + (t.n / 2 > 64 ? 2 : 1);
                for (int c = 0; c < chunks; ++c) {
                    const uint32_t at = (c < chunks_a ? da + c * kChunk : db + (c - chunks_a) * kChunk) + valid * kRow;
                    for (int w = lane; w < words; w += 32) st_shared_zero16(at + 16 * w);
                }
                fence_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(mapa_shared(zeroed_bar(st), 0));
            }
            passed += kStageCycles * tile_stages;
            s = (s + tile_stages) % stages;
        }
    } else {
        const int q = warp & 3;  // the TMEM lane quadrant this warp may read
        const int in_half = 32 * q + lane;  // column within this CTA's half
        const int part = (warp - 2) >> 2;
        const bool mine = 32 * q < half_cols;
        Accumulators accs;
        [[maybe_unused]] GatedBack back;
        auto release = [&](uint32_t a) {  // the MMA may write accumulator a
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(mapa_shared(tempty_bar(a), 0));
        };
        for (TileWalk<kDense, kWalkSegments> walk(tab, first, stride); walk.more(); walk.next()) {
            const Tile t = walk.get();
            const bool empty = t.r0 >= t.r1;
            uint32_t a = accs.next;
            const uint32_t tmem_q = tmem_base + ((uint32_t)(q * 32) << 16);
            const int col = t.col0 + rank * half_cols + in_half;
            if constexpr (OP == kGatedBack) {
                if (t.last && mine && kGatedRows * part < t.rows) back.fetch(h.gated, t, col, kGatedRows * part, lane);
            }
            if (!empty) {
                if (!__all_sync(0xffffffffu, wait_bar<true>(tfull_bar(a), accs.ready(), p.o.wait + walk.slack, abort_flag))) {
                    if (lane == 0) raise();
                    break;
                }
                tc_fence_after();
            }
            uint32_t from = a;
            if constexpr (kRegisters) {
                RegisterSums<kParts<OP>> sums = {};
                bool ok = true;
                for (int at = tab.o.segment; at < tab.o.red; at += tab.o.segment) {
                    if (mine) sums.add(t, tmem_q + a * kAccCols, part, false);
                    release(a);
                    accs.done(t);
                    a = accs.next;
                    ok = __all_sync(0xffffffffu, wait_bar<true>(tfull_bar(a), accs.ready(), p.o.wait, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                }
                if (!ok) {
                    if (lane == 0) raise();
                    break;
                }
                if (mine) sums.add(t, tmem_q + a * kAccCols, part, true);
                from = a;
            } else if (SEGMENTS && !(t.first && t.last)) {
                from = a ^ 1u;
                if constexpr (OP == kGated || OP == kGatedBack) {
                    if (mine) add_gated_segment<kParts<OP>>(t, tmem_q + a * kAccCols, tmem_q + from * kAccCols, part);
                } else {
                    if (mine) add_segment<kDense, kParts<OP>>(tab.o, t, tmem_q + a * kAccCols, tmem_q + from * kAccCols, part);
                }
                release(a);
            }
            if (!SEGMENTS || t.last) {
                if constexpr (OP == kGated) {
                    const int out_col = (t.col0 + rank * half_cols + 32 * q) / 2 + (lane & (kGranule - 1));
                    if (mine) store_gated<kParts<OP>>(h.gated, tab.o.out, t, tmem_q + from * kAccCols, out_col, part, lane);
                } else if constexpr (OP == kGatedBack) {
                    if (mine) back.template store<kParts<OP>>(h.gated, t, tmem_q + from * kAccCols, col, part, lane);
                } else {
                    if (mine) store_tile<kDense, ADD, kParts<OP>>(tab.o, t, tmem_q + from * kAccCols, empty, col, part, lane);
                }
                if (!empty) release(from);
            }
            if (!empty) accs.done(t);
        }
    }

    leave_pair(abort_flag);
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

// Tile sizes.  Rows: up to 256, fewer where the experts average fewer.  Columns: 256, or 128 (64
// per CTA) where there are no more (with 256, 0.1 us slower).  128 where 256 leave CTA pairs
// without a tile are slower: a tile's MMAs take the same time (one token's six experts, N 2048, K
// 1408: 11.6 against 8.7 us; one expert, 256 rows, N 6144, K 2048: 16.0 against 11.7; the other
// way round 16 experts of 48 rows, dgrad to 200 columns, 7.0 against 7.4).  Where there are not
// half as many tiles as pairs and the experts' rows fill 64, tiles of fewer rows, down to 64
// (dgrad of one expert, 256 rows, N 6144, K 2048: 33 -> 20 us; of four experts of 108 rows, N
// 2040, K 224: 12.5 -> 10.6; wgrad of 4096 rows, N 256, K 1024: 23 -> 17; 16 experts of 48 rows
// would lose 0.9 of 6.9 us).  Stages of two blocks where a tile has so few rows that its waits and
// commits take longer than its MMAs (one expert, 2048 rows, N 256, K 2048: 9.4 -> 8.4 us; dgrad of
// 256 rows, N 6144, K 2048: 18.2 -> 15.8; wgrad of 8192 rows, N = K = 128: 28.8 -> 19.7; up to 128
// rows the dgrad gains, 61.5 -> 59.6 for 48 rows each of 64 experts, and the forward loses, 62.7 -> 63.7).
inline int choose_tiles(GroupedArgs &g, int op, bool one_block, int sms) {
    GroupedOut &o = g.o;
    const long long pairs = sms / 2, active = std::max<long long>(1, std::min(o.E, o.rows));
    const long long most = op == kWgrad ? o.m_dense : std::min<long long>(256, 2 * (o.rows / active) + 1);
    o.tile_rows = 256;
    while (o.tile_rows > 32 && o.tile_rows / 2 >= most) o.tile_rows /= 2;
    auto row_tiles = [&] {
        return op == kWgrad ? (long long)o.E * ((o.m_dense + o.tile_rows - 1) / o.tile_rows)
                            : std::max<long long>(active, o.rows / o.tile_rows);
    };
    o.cols = o.n_out > 128 ? 256 : 128;
    o.col_tiles = (o.n_out + o.cols - 1) / o.cols;
    const long long fill = op == kWgrad ? o.m_dense : o.rows / active;  // rows that an expert's tiles share
    while (o.tile_rows > 64 && fill >= 64 && 2 * row_tiles() * o.col_tiles <= pairs) o.tile_rows /= 2;
    o.row_tiles = (o.m_dense + o.tile_rows - 1) / o.tile_rows;
    const bool two = o.tile_rows <= (op == kForward || op == kWgrad || op == kGated ? 64 : 128);
    const int blocks = two && !one_block ? 2 : 1;
    g.a_block = o.cols / 2 * kRow;
    g.b_block = op == kWgrad ? (o.tile_rows / 2 + 63) / 64 * kChunk : o.tile_rows / 2 * kRow;
    g.stages = std::min(kMaxStages, kStageSpace / (blocks * (g.a_block + g.b_block)));
    return blocks;
}

}  // namespace moe
