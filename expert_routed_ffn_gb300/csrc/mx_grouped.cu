// Grouped product with both operands in MXFP4: rows grouped by expert (grouped.cuh),
//   Y[r, n] = sum_b 2^(xs[b, r] + ws[e, b, n] - 254) sum_{i in block b} x[r, i] w[e, n, i]
// x, w: E2M1 values, blocks b of 32 along K, one scale byte each.  The block-scaled tensor
// instruction (tcgen05.mma kind::mxf4, K = 64) multiplies the packed codes and applies both
// scales as it accumulates in fp32: nothing is decoded, so a k-step of 256 values is 128
// bytes of codes per row, a quarter of bf16's.
//
// Persistent kernel on CTA pairs with the tiles of the bf16 products (grouped.cu): 256
// weight rows as the MMA's M, up to 192 token rows as its N.  Warps of a CTA:
//   warp 0       TMA producer: codes of this CTA's weight rows and half of the token rows,
//                256 values (128 bytes, 128-byte swizzle) per stage
//   warp 1       allocates tensor memory; in the even CTA copies a stage's scales from shared
//                to tensor memory of both CTAs (tcgen05.cp, in order with the MMAs that
//                follow) and issues the MMAs
//   warps 2-5    epilogue (grouped.cuh), overlapping the next tile's main loop
//   fetch        scales, four stages' at a time: those of this CTA's weight rows and of all the
//                tile's tokens, as they lie (a block's scales for consecutive rows).  Where rows
//                and N are multiples of 16, which TMA wants of a tensor's strides: one warp, two
//                copies, the token run starting at the 16 bytes that hold the tile's first row.
//                Else four warps with 4-byte asynchronous copies, for an expert's first row has
//                any alignment (24576 rows 47 against 51 us; one stage at a time, the waits
//                between the copies bounded the kernel: 61 us)
//   8 warps      two sets of four, on alternate stages: the tensor core wants four consecutive
//                blocks' scales of a row in one word, so they transpose from the fetched runs
//                into the words that tcgen05.cp reads
// Tensor memory (512 columns): two accumulators of up to 192 columns, then per stage the
// scales of the weights (8 columns) and of the tokens (8 per 128 of them).
//
// Measured on GB300, one call in a row of them on the same tensors (part of the weights stays in
// L2) / alone with cold caches (64 experts, N 1408, K 2048): 24576 rows 41 / 50 us, 3.4 PFLOP/s,
// 4.7 TB/s; 384 rows 19 / 32 us; one expert, 8192 rows, N and K 2048: 19 / 25 us, 3.7 PFLOP/s.
// Neither memory nor the tensor pipe is at its limit (24576 rows): HBM is 44% busy, the tensor pipe
// 42% of its active cycles (58% with the copies of scales), and L2 delivers 9.5 TB/s, less than it
// gives the bf16 products.  Without products it took 4 of 46 us less, without scales 1.  Part of
// it are tiles that are not full: experts of 385 rows take three where 384 take two, and
// of 1408 columns the sixth tile is half empty.  Tiles of 224 rows, for which tensor memory has
// room for two stages' scales beside the accumulators, took the same time.
#include <algorithm>

#include "common.cuh"
#include "grouped.cuh"
#include "kernels.h"
#include "moe.h"
#include "op_host.h"

namespace moe {
namespace {

constexpr int kBK = 256;           // values per stage
constexpr int kRow = kBK / 2;      // their bytes: one row of codes
constexpr int kBlocks = kBK / 32;  // scale blocks per stage
constexpr int kMaxStages = 16;
constexpr int kEpiWarps = kQuads;
constexpr int kSets = 2;           // sets of transposing warps
constexpr int kFetch = 2 + kEpiWarps;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxRows = 192;      // token rows of a tile
constexpr int kBoxes = kMaxRows / 32;
// fetched scales of four stages: per block of tokens (192 and an alignment of up to 3) and weights
constexpr int kFetchStages = 4, kFetchBlocks = kFetchStages * kBlocks;
constexpr int kRaw = 3;
constexpr int kRawToken = 208, kRawWeight = 128;
constexpr int kRawBytes = kFetchBlocks * (kRawToken + kRawWeight);
constexpr int kStageSpace = 195584;

struct Header {
    uint64_t bars[2 * kMaxStages + 2 * kRaw + 5];
    TileTable table;
    uint32_t tmem;
    volatile int abort;
};
constexpr int kHeaderBytes = 4096;
static_assert(segment_of(true, 64) % (kFetchStages * kBK) == 0 && segment_of(false, 64) % (kFetchStages * kBK) == 0,
              "a segment's scales are whole fetches");
constexpr int kSmemBytes = kHeaderBytes + kStageSpace + kRaw * kRawBytes + 16;  // (a word behind the last run is read)
static_assert(sizeof(Header) <= kHeaderBytes && kSmemBytes <= 232448, "shared memory of one CTA");

struct MxGroupedArgs {
    CUtensorMap map_xs, map_ws;        // scales: four stages' blocks of a tile
    CUtensorMap map_a, map_b[kBoxes];  // weight codes; token codes in boxes of 16, 32, .. rows
    GroupedOut o;
    const uint8_t *xs, *ws;            // [K / 32, rows], [E, K / 32, N]
    int a_stage, b_stage;              // bytes of codes per stage and CTA
    uint32_t x_run;                    // bytes fetched of a block's token scales
    int atoms;                         // 128-row groups of token scales
    int stages;
};

// Instruction descriptor of kind::mxf4: E2M1 operands (bits 7-9 and 10-11 = 1), N >> 3 at bits
// 17-22, scales UE8M0 (bit 23), M >> 4 at bits 24-28; which half of a scale word a K step of 64
// uses: bits 29-30 (A) and 4-5 (B).
__device__ __forceinline__ uint32_t idesc_mxf4(int M, int N) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_mxf4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                                 uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// 512 bytes of scales in shared memory: no swizzle; 8-lane groups of 16-byte rows 128 bytes apart
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}
// 512 bytes of shared memory (32 lanes x 16 bytes) to four columns of tensor memory, the same
// in each of its four lane quadrants; in both CTAs, each from its own shared memory
__device__ __forceinline__ void tc_copy_scales_pair(uint32_t taddr, uint64_t d) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// 4 bytes to shared memory; only `bytes` of them are read, the rest is zero
__device__ __forceinline__ void copy_word(uint32_t dst, const uint8_t *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// arrive on `bar` when this thread's copies so far have landed
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// Scales of four rows of four blocks, whose runs (of bytes, one per row) lie `run` bytes apart
// at `from`, the first row `shift` bytes further, in each next block `move` more (modulo 4): to
// one word per row, 16 bytes apart at `to`, byte j for block j.
__device__ __forceinline__ void transpose(uint32_t from, uint32_t run, uint32_t shift, uint32_t move, uint32_t to) {
    uint32_t w[4];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
        const uint32_t bytes = move ? (shift + j * move) & 3u : shift;
        const uint32_t at = from + j * run + (bytes & ~3u);
        w[j] = __funnelshift_r(ld_shared_u32(at), ld_shared_u32(at + 4), 8 * (bytes & 3u));
    }
    const uint32_t p01 = __byte_perm(w[0], w[1], 0x5140), p23 = __byte_perm(w[2], w[3], 0x5140);
    const uint32_t q01 = __byte_perm(w[0], w[1], 0x7362), q23 = __byte_perm(w[2], w[3], 0x7362);
    st_shared_u32(to, __byte_perm(p01, p23, 0x5410));
    st_shared_u32(to + 16, __byte_perm(p01, p23, 0x7632));
    st_shared_u32(to + 32, __byte_perm(q01, q23, 0x5410));
    st_shared_u32(to + 48, __byte_perm(q01, q23, 0x7632));
}

// First warp of the transposing role
__host__ __device__ constexpr int transpose_warp(bool tma) { return kFetch + (tma ? 1 : 4); }
__host__ __device__ constexpr int num_threads(bool tma) { return 32 * (transpose_warp(tma) + 4 * kSets); }
static_assert(num_threads(true) >= kMaxExperts, "load_table: a thread per expert");

// TMA: scales are fetched by TMA; SEGMENTS: a sum comes in several (grouped.cuh)
template <bool TMA, bool SEGMENTS>
__global__ void __launch_bounds__(num_threads(TMA), 1) mx_grouped_kernel(const __grid_constant__ MxGroupedArgs p) {
    constexpr int kTranspose = transpose_warp(TMA);
    extern __shared__ __align__(1024) uint8_t smem[];
    Header &h = *reinterpret_cast<Header *>(smem);
    const TileTable &tab = h.table;
    const uint32_t base = smem_u32(smem) + kHeaderBytes;
    const int a_stage = p.a_stage, b_stage = p.b_stage, stages = p.stages;
    const int scale_stage = 1024 + 1024 * p.atoms;
    // A first: the MMA reads 128 rows of A where the box brought 64; the rest is whatever
    // follows, and its results are not stored
    const uint32_t sA = base, sB = sA + (uint32_t)(stages * a_stage), sS = sB + (uint32_t)(stages * b_stage);
    const uint32_t sR = base + kStageSpace;  // the fetched scales
    const uint32_t bar0 = smem_u32(h.bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * kMaxStages + a); };
    auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * kMaxStages + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * kMaxStages + 4);
    auto raw_full_bar = [&](int i) { return bar0 + 8u * (2 * kMaxStages + 5 + i); };
    auto raw_empty_bar = [&](int i) { return bar0 + 8u * (2 * kMaxStages + 5 + kRaw + i); };
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
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full_bar(s), 9);  // the copies of codes, four scale warps of each CTA
            mbar_init(empty_bar(s), 1);
        }
        for (uint32_t a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 2 * kEpiWarps);
        }
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(raw_full_bar(i), TMA ? 1 : 128);
            mbar_init(raw_empty_bar(i), 4 * kSets);
        }
        mbar_init(drain_bar, 1);
        fence_mbar_init();
        h.abort = 0;
        tma_prefetch_desc(&p.map_a);
        tma_prefetch_desc(&p.map_b[0]);
        if (TMA) {
            tma_prefetch_desc(&p.map_ws);
            tma_prefetch_desc(&p.map_xs);
        }
    }
    if (threadIdx.x == 64) start_table<false>(p.o, h.table);
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&h.tmem), kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any copy or arrival crosses over
    tc_fence_after();
    const uint32_t tmem_base = h.tmem;
    pdl_wait();
    pdl_trigger();
    if (!load_table<false>(h.table) && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.o.err, ERR_BOUNDS);
    const int first = (int)blockIdx.x / 2, stride = (int)gridDim.x / 2;
    const int half_cols = tab.o.cols / 2, atoms = p.atoms;
    const uint32_t w_run = half_cols, x_run = p.x_run;  // fetched bytes of a block's scales
    const int K = tab.o.red;
    // stages of a sum, or of a segment of it, which begins and ends between two fetches of scales
    auto first_stage = [](const Tile &t) { return t.r0 / kBK; };
    auto end_stage = [](const Tile &t) { return (t.r1 + kBK - 1) / kBK; };

    if (warp == 0) {
        uint32_t ph = 1;
        int s = 0;
        bool ok = true;
        for (TileWalk<false, SEGMENTS> walk(tab, first, stride); ok && walk.more(); walk.next()) {
            const Tile t = walk.get();
            const int col = t.col0 + rank * half_cols, row = t.row0 + rank * (t.n / 2);
            const CUtensorMap *map_b = &p.map_b[t.n / 32 - 1];
            const uint32_t bytes = a_stage + (t.n / 2) * kRow;
            for (int k = first_stage(t); k < end_stage(t); ++k) {
                if (!__all_sync(0xffffffffu, wait_bar(empty_bar(s), ph, p.o.wait, abort_flag))) {
                    ok = false;
                    break;
                }
                const uint32_t bar = mapa_shared(full_bar(s), 0);
                if (elect_one()) {
                    if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * bytes);
                    tma_load_3d_pair(sA + s * a_stage, &p.map_a, bar, k * kRow, col, t.e);
                    tma_load_2d_pair(sB + s * b_stage, map_b, bar, k * kRow, row);
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
            const uint32_t acc_cols = tab.o.tile_rows;
            const uint32_t cols_s = 8 + 8 * atoms;  // scale columns of a stage
            const uint32_t scale0 = tmem_base + 2 * acc_cols;
            const uint64_t desc_a = smem_desc_k128(sA), desc_b = smem_desc_k128(sB), desc_s = scale_desc(sS);
            Accumulators accs;
            uint32_t ph = 0;
            int s = 0;
            bool ok = p.o.wait != 0, issued = false;  // a bound of 0: give up at once
            TileWalk<false, SEGMENTS> walk(tab, first, stride);
            Tile next;
            if (walk.more()) next = walk.get();
            while (ok && walk.more()) {
                const Tile t = next;
                const uint32_t idesc = idesc_mxf4(256, t.n);
                const uint32_t a = accs.next, d = tmem_base + a * acc_cols;
                if (!__all_sync(0xffffffffu, wait_bar<true>(tempty_bar(a), accs.take(), p.o.wait, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int k0 = first_stage(t), k1 = end_stage(t);
                for (int k = k0; k < k1; ++k) {
                    if (!__all_sync(0xffffffffu, wait_bar<true>(full_bar(s), ph, p.o.wait, abort_flag))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t ta = scale0 + s * cols_s, tb = ta + 8;
                    const uint64_t ad = desc_a + (uint32_t)(s * a_stage >> 4), bd = desc_b + (uint32_t)(s * b_stage >> 4);
                    const uint64_t sd = desc_s + (uint32_t)(s * scale_stage >> 4);
                    const int left = K - k * kBK;  // values
                    if (elect_one()) {
#pragma unroll
                        for (int g = 0; g < 2; ++g) {  // four blocks (128 values) each
                            if (128 * g >= left) break;
                            tc_copy_scales_pair(ta + 4 * g, sd + 32 * g);
                            tc_copy_scales_pair(tb + 4 * g * atoms, sd + 64 + 32 * (g * atoms));
                            if (atoms > 1) tc_copy_scales_pair(tb + 4 * (g * atoms + 1), sd + 64 + 32 * (g * atoms + 1));
                        }
#pragma unroll
                        for (int i = 0; i < kBK / 64; ++i) {
                            if (64 * i >= left) break;
                            const uint32_t half = (uint32_t)(i & 1) * 2u;  // the step's two blocks within the word
                            tc_mma_mxf4_pair(d, ad + 2 * i, bd + 2 * i, idesc | half << 29 | half << 4, ta + 4 * (i >> 1),
                                             tb + 4 * atoms * (i >> 1), (k != k0) | (i != 0));
                        }
                        tc_commit_pair(empty_bar(s), 3);
                        if (k + 1 == k1) tc_commit_pair(tfull_bar(a), 3);
                    }
                    __syncwarp();
                    issued = true;
                    if (k == k0) {  // the next tile's place, while this one's products run
                        walk.next();
                        if (walk.more()) next = walk.get();
                    }
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
    } else if (warp < 2 + kEpiWarps) {
        const int q = warp & 3;  // the TMEM lane quadrant this warp may read
        const uint32_t tmem_q = tmem_base + ((uint32_t)(q * 32) << 16), acc_cols = tab.o.tile_rows;
        const bool mine = 32 * q < half_cols;
        Accumulators accs;
        auto release = [&](uint32_t a) {  // the MMA may write accumulator a
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(mapa_shared(tempty_bar(a), 0));
        };
        for (TileWalk<false, SEGMENTS> walk(tab, first, stride); walk.more(); walk.next()) {
            const Tile t = walk.get();
            const uint32_t a = accs.next;
            if (!__all_sync(0xffffffffu, wait_bar<true>(tfull_bar(a), accs.ready(), p.o.wait, abort_flag))) {
                if (lane == 0) raise();
                break;
            }
            tc_fence_after();
            uint32_t from = a;
            if (SEGMENTS && !(t.first && t.last)) {
                from = a ^ 1u;
                if (mine) add_segment<false, 1>(tab.o, t, tmem_q + a * acc_cols, tmem_q + from * acc_cols, 0);
                release(a);
            }
            if (!SEGMENTS || t.last) {
                if (mine)
                    store_tile<false, false, 1>(tab.o, t, tmem_q + from * acc_cols, false,
                                                t.col0 + rank * half_cols + 32 * q + lane, 0, lane);
                release(from);
            }
            accs.done(t);
        }
    } else if (TMA && warp == kFetch) {
        int raw = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (TileWalk<false, SEGMENTS> walk(tab, first, stride); ok && walk.more(); walk.next()) {
            const Tile t = walk.get();
            for (int b0 = t.r0 / 32; b0 < t.r1 / 32; b0 += kFetchBlocks) {
                if (!__all_sync(0xffffffffu, wait_bar(raw_empty_bar(raw), ph, p.o.wait, abort_flag))) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    const uint32_t to = sR + raw * kRawBytes, bar = raw_full_bar(raw);
                    mbar_arrive_expect_tx(bar, kFetchBlocks * (w_run + x_run));
                    tma_load_3d(to + kFetchBlocks * kRawToken, &p.map_ws, bar, t.col0 + rank * half_cols, b0, t.e);
                    tma_load_2d(to, &p.map_xs, bar, t.row0 & ~15, b0);
                }
                __syncwarp();
                if (++raw == kRaw) {
                    raw = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) raise();
    } else if (!TMA && warp < kTranspose) {
        // 16 threads per block: of its weights 4-byte words 16 m + i % 16 (m < 2), of its tokens
        // those with m < 4; a thread's blocks are 8 apart, which moves a token run by a multiple
        // of 8 bytes, so its alignment holds for the tile.
        const int i = (int)threadIdx.x - 32 * kFetch, b = i >> 4, w0 = 4 * (i & 15);
        const int n_blocks = K / 32, rows = tab.o.rows, n_out = tab.o.n_out;
        const uint8_t *const xs_end = p.xs + (size_t)n_blocks * rows;
        const size_t x_step = (size_t)kBlocks * rows, w_step = (size_t)kBlocks * n_out;
        const uint32_t rt0 = sR + b * x_run + w0, rw0 = sR + kFetchBlocks * kRawToken + b * w_run + w0;
        int raw = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (TileWalk<false, SEGMENTS> walk(tab, first, stride); ok && walk.more(); walk.next()) {
            const Tile t = walk.get();
            const int col = t.col0 + rank * half_cols + w0;
            const uint8_t *ws = p.ws + ((size_t)t.e * n_blocks + t.r0 / 32 + b) * n_out + col;
            // n_out and half_cols are multiples of 8 and 64: a word is inside or outside
            const bool w_in[2] = {w0 < half_cols && col < n_out, w0 + 64 < half_cols && col + 64 < n_out};
            const size_t at = (size_t)(t.r0 / 32 + b) * rows + t.row0;
            const uint8_t *xs = p.xs + (at & ~(size_t)3) + w0;
            const int x_bytes = (int)(at & 3) + t.rows - w0;  // of the run from this thread's first word on
            for (int b0 = t.r0 / 32; b0 < t.r1 / 32; b0 += kFetchBlocks) {
                if (!__all_sync(0xffffffffu, wait_bar(raw_empty_bar(raw), ph, p.o.wait, abort_flag))) {
                    ok = false;
                    break;
                }
                const uint32_t off = (uint32_t)(raw * kRawBytes);
#pragma unroll
                for (int f = 0; f < kFetchStages; ++f) {
                    const int stage_b = b0 + f * kBlocks;
                    if (stage_b >= n_blocks) break;
                    const bool in = stage_b + b < n_blocks;  // else a block past K: zeros
                    const uint32_t rw = rw0 + off + f * kBlocks * w_run, rt = rt0 + off + f * kBlocks * x_run;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        if (!in || w_in[m]) copy_word(rw + 64 * m, in ? ws + 64 * m : p.ws, in ? 4 : 0);
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        if (x_bytes > 64 * m) {  // at the tensor's end a word may hold fewer bytes
                            const uint8_t *src = in ? xs + 64 * m : p.xs;
                            copy_word(rt + 64 * m, src, in ? (int)min((ptrdiff_t)4, xs_end - src) : 0);
                        }
                    ws += w_step;
                    xs += x_step;
                }
                copies_arrive(raw_full_bar(raw));
                if (++raw == kRaw) {
                    raw = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) raise();
        asm volatile("cp.async.wait_all;" ::: "memory");  // none outlives the CTA
    } else {
        const int set = (warp - kTranspose) >> 2;
        const int i = (int)threadIdx.x - 32 * kTranspose - 128 * set;  // 0..127 within the set
        // a block's run begins with the 16 (or 4) aligned bytes that hold its first scale
        const uint32_t x_move = TMA ? 0 : (uint32_t)tab.o.rows & 3u;
        int s = 0, raw = 0;
        uint32_t ph = 1, raw_ph = 0;
        bool ok = true;
        for (TileWalk<false, SEGMENTS> walk(tab, first, stride); ok && walk.more(); walk.next()) {
            const Tile t = walk.get();
            const uint32_t x_at = (uint32_t)t.row0 & (TMA ? 15u : 3u);
            const int k1 = end_stage(t);
            for (int k = first_stage(t); k < k1; ++k) {
                const int f = k % kFetchStages;
                if (f == 0 && !__all_sync(0xffffffffu, wait_bar(raw_full_bar(raw), raw_ph, p.o.wait, abort_flag))) {
                    ok = false;
                    break;
                }
                if (k % kSets == set) {
                    if (!__all_sync(0xffffffffu, wait_bar(empty_bar(s), ph, p.o.wait, abort_flag))) {
                        ok = false;
                        break;
                    }
                    const uint32_t rt = sR + raw * kRawBytes + f * kBlocks * x_run;
                    const uint32_t rw = sR + raw * kRawBytes + kFetchBlocks * kRawToken + f * kBlocks * w_run;
                    const uint32_t sc = sS + s * scale_stage;
                    // a task: four blocks' scales of four rows, first the weights', then the tokens'
                    for (int task = i; task < 64 + t.n / 2; task += 128) {
                        if (task < 64) {
                            const uint32_t m = (uint32_t)task & 31u, g = (uint32_t)task >> 5;
                            transpose(rw + g * (4 * w_run) + 4 * m, w_run, 0, 0, sc + 512 * g + (m & 7) * 64 + (m >> 3) * 4);
                        } else {
                            const uint32_t at = (uint32_t)task - 64, g = at >= (uint32_t)t.n / 4 ? 1 : 0;
                            const uint32_t m = at - g * (uint32_t)t.n / 4, r = 4 * m;
                            transpose(rt + g * (4 * x_run) + r, x_run, x_at + 4 * g * x_move, x_move,
                                      sc + 1024 + 512 * (g * atoms + (r >> 7)) + (r & 31) * 16 + ((r & 127) >> 5) * 4);
                        }
                    }
                    fence_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(mapa_shared(full_bar(s), 0));
                }
                if (f + 1 == kFetchStages || k + 1 == k1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(raw_empty_bar(raw));
                    if (++raw == kRaw) {
                        raw = 0;
                        raw_ph ^= 1u;
                    }
                }
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) raise();
    }

    leave_pair(abort_flag);
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

OpDone g_attr[4];

// Tile sizes, by the bf16 products' rule: rows up to 192, fewer where the experts average fewer;
// 256 columns, or 128 where there are no more (128 where 256 leave CTA pairs without a tile: 11.4
// against 9.3 us for one expert, 256 rows, N 6144, K 2048); where there are not half as many tiles
// as pairs and the experts' rows fill 64, tiles of fewer rows, down to 64.
void choose_tiles(MxGroupedArgs &g, int sms) {
    GroupedOut &o = g.o;
    const long long pairs = sms / 2, active = std::max<long long>(1, std::min(o.E, o.rows)), fill = o.rows / active;
    const long long most = 2 * fill + 1;
    o.tile_rows = most <= 32 ? 32 : most <= 64 ? 64 : most <= 128 ? 128 : kMaxRows;
    auto row_tiles = [&] { return std::max<long long>(active, o.rows / o.tile_rows); };
    o.cols = o.n_out > 128 ? 256 : 128;
    o.col_tiles = (o.n_out + o.cols - 1) / o.cols;
    while (o.tile_rows > 64 && fill >= 64 && 2 * row_tiles() * o.col_tiles <= pairs)
        o.tile_rows = (o.tile_rows / 2 + 31) / 32 * 32;
    g.a_stage = o.cols / 2 * kRow;
    g.b_stage = o.tile_rows / 2 * kRow;
    g.x_run = o.tile_rows + 16;
    g.atoms = (o.tile_rows + 127) / 128;
    g.stages = std::min({kMaxStages, kStageSpace / (g.a_stage + g.b_stage + 1024 + 1024 * g.atoms),
                         ((int)kTmemCols - 2 * o.tile_rows) / (8 + 8 * g.atoms)});
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_mx_grouped_forward(const void *Xc, const uint8_t *Xs, const void *Wc, const uint8_t *Ws,
                                             const int32_t *offs, int rows, int E, int N, int K, int out_dtype, void *Y,
                                             moe_stream_t stream) {
    using namespace moe;
    const char *op = "moe_mx_grouped_forward";
    if (rows < 0 || E < 1 || N < 1 || K < 1)
        return op_fail(MOE_ERR_INVALID_ARG, "%s: need rows >= 0, E >= 1, N >= 1, K >= 1", op);
    if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_F32)
        return op_fail(MOE_ERR_INVALID_ARG, "%s: unknown out_dtype %d", op, out_dtype);
    if (E > kMaxExperts || N % 8 || K % 32 || N > (1 << 20) || K > (1 << 20) || rows > (1 << 30))
        return op_fail(MOE_ERR_UNSUPPORTED,
                       "%s: E up to 256, N a multiple of 8 and K of 32, up to 2^20, rows up to 2^30 (E %d, N %d, K %d, rows %d)",
                       op, E, N, K, rows);
    if (rows > 0 && (!Xc || !Xs || !Wc || !Ws || !offs || !Y)) return op_fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer", op);
    if (!op_aligned16(Xc) || !op_aligned16(Xs) || !op_aligned16(Wc) || !op_aligned16(Ws) || !op_aligned16(Y) ||
        (reinterpret_cast<uintptr_t>(offs) & 3u))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned, the offsets 4-byte aligned", op);
    if (rows == 0) return MOE_OK;
    const uint64_t n = N, c = K / 2, b = K / 32, r = rows, e = E, y_bytes = (out_dtype == MOE_DTYPE_F32 ? 4 : 2) * r * n;
    if (op_overlap(Y, y_bytes, Xc, r * c) || op_overlap(Y, y_bytes, Xs, r * b) || op_overlap(Y, y_bytes, Wc, e * n * c) ||
        op_overlap(Y, y_bytes, Ws, e * n * b) || op_overlap(Y, y_bytes, offs, 4 * (e + 1)))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: the output overlaps an input", op);
    const int sms = op_num_sms();
    int *err = op_error_word();
    if (sms < 2 || err == nullptr) return op_fail(MOE_ERR_CUDA, "%s: no usable current device", op);
    MxGroupedArgs g = {};
    GroupedOut &o = g.o;
    o.offs = offs;
    o.out = Y;
    o.err = err;
    o.E = E;
    o.rows = rows;
    o.n_out = N;
    o.red = K;
    o.f32 = out_dtype == MOE_DTYPE_F32;
    o.segment = segment_of(o.f32, 64);
    o.wait = wait_cycles(K / kBK + 1);
    g.xs = Xs;
    g.ws = Ws;
    choose_tiles(g, sms);
    const bool tma = rows % 16 == 0 && N % 16 == 0;
    const long long tiles = ((long long)rows / o.tile_rows + std::min(E, rows)) * o.col_tiles;
    if (tiles > (1ll << 30)) return op_fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^30 output tiles", op);
    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
    CUresult cr = op_encode(&g.map_a, {u8, 3, Wc, {c, n, e}, {c, n * c}, {kRow, (uint32_t)o.cols / 2, 1}, sw});
    for (int i = 0; i < o.tile_rows / 32 && cr == CUDA_SUCCESS; ++i)
        cr = op_encode(&g.map_b[i], {u8, 2, Xc, {c, r}, {c}, {kRow, 16u * (i + 1)}, sw});
    const auto flat = CU_TENSOR_MAP_SWIZZLE_NONE;
    if (tma && cr == CUDA_SUCCESS)
        cr = op_encode(&g.map_ws, {u8, 3, Ws, {n, b, e}, {n, n * b}, {(uint32_t)o.cols / 2, kFetchBlocks, 1}, flat});
    if (tma && cr == CUDA_SUCCESS) cr = op_encode(&g.map_xs, {u8, 2, Xs, {r, b}, {r}, {g.x_run, kFetchBlocks}, flat});
    if (cr != CUDA_SUCCESS) return op_fail(MOE_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", op, (int)cr);
    const bool segments = K > o.segment;
    auto kernel = segments ? (tma ? mx_grouped_kernel<true, true> : mx_grouped_kernel<false, true>)
                           : (tma ? mx_grouped_kernel<true, false> : mx_grouped_kernel<false, false>);
    cudaError_t ce = op_allow_smem(reinterpret_cast<const void *>(kernel), kSmemBytes, &g_attr[2 * segments + tma]);
    if (ce == cudaSuccess)
        ce = launch_pdl_cluster(kernel, dim3(2u * (unsigned)std::min<long long>(sms / 2, tiles)), dim3(num_threads(tma)),
                                (size_t)kSmemBytes, reinterpret_cast<cudaStream_t>(stream), dim3(2, 1, 1), g);
    return op_cuda(ce, op);
}
