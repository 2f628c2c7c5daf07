// What the products over expert-grouped rows share: the tile list derived from the row
// offsets, and the epilogue that moves a tile from tensor memory to its output rows.
//
// A tile is computed with the output's columns as the MMA's M and the output's rows (the
// tokens) as its N.  N goes in steps of 32, so an expert with 300 rows costs two tiles of
// 160 rather than three of 128, and one token costs 32; and since a TMEM lane is an output
// column, a warp's store of one row is 32 consecutive columns: results go from registers
// straight to memory, whatever the number of valid rows.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "op_host.h"

namespace moe {

constexpr int kMaxExperts = 256;
constexpr int kQuads = 4;              // TMEM lane quadrants, of 32 lanes
constexpr long long kDrainCycles = 2000000000ll;  // after an abort: bound of the wait for the MMAs issued
constexpr unsigned long long kGraceNs = 1000000ull;  // and the time given to the copies in flight

// The output and its tiles.  Row-grouped (forward, dgrad): out [rows, n_out], the rows of
// expert e are [offs[e], offs[e + 1]).  Dense (wgrad): out [E, m_dense, n_out], and the
// offsets bound the reduction.
struct GroupedOut {
    const int32_t *offs;
    void *out;
    int *err;
    int E, rows;
    int n_out;       // columns of the output
    int m_dense;     // dense: rows of one expert's output
    int red;         // row-grouped: length of the reduction
    int cols;        // a tile's output columns, half of them in each CTA of a pair
    int tile_rows;   // most output rows of a tile, a multiple of 32
    int col_tiles;   // tiles along the output columns
    int row_tiles;   // dense: tiles along m_dense
    int f32;         // output type: fp32, else bf16
    int segment;     // reduction steps that one accumulator sums, see segment_of
    long long wait;  // bound of every wait in SM cycles, see wait_cycles
};

struct Tile {
    int e, row0, rows, n, col0;  // expert, first output row, valid rows, MMA N, first output column
    int r0, r1;                  // reduction range: the sum's, or one segment's
    bool first, last;            // of its sum's segments
};

__device__ __forceinline__ void fence_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 2D load into this CTA's shared memory, completing on a barrier of either CTA of the pair
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

// What a stage, and the epilogue of a tile, may take at most.
constexpr long long kStageCycles = 4096, kTileCycles = 65536;

// About 2 s, and what the longest sum may take: the epilogue waits for all of a tile's stages.
// moe_operators_wait_limit replaces it.
inline long long wait_cycles(long long stages_per_tile) {
    const long long limit = op_wait_limit();
    if (limit >= 0) return std::min(limit, 1ll << 62);  // roles add to it
    return 4000000000ll + kStageCycles * stages_per_tile;
}

// Wait until the phase of parity `parity` of a barrier has completed; CLUSTER: a barrier that
// threads of the other CTA arrive on.  Bounded by the SM's clock (the global timer is slow to
// read beside waits this short).  False after the bound, or once *abort is set.  (A try may
// suspend the thread for a while, so a bound of 0 is not seen here: the MMA's role gives up at
// its first wait then.  Checked in every wait it cost up to 70 cycles a stage.)
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, long long limit, volatile int *abort) {
    auto done = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    if (done()) return true;
    const long long t0 = clock64();
    for (;;) {
        if (done()) return true;
        if (abort != nullptr && *abort) return false;
        if (clock64() - t0 > limit) return false;
    }
}

// Arrive on a barrier of either CTA (address from mapa_shared), with the default semantics, a
// release at CTA scope: what it hands over stays within the arriving CTA (an accumulator whose
// reads tcgen05.wait::ld has completed; shared memory that this CTA's own tensor core reads next,
// and that fence.proxy.async has made visible to it before the arrival), so nothing has to become
// visible to threads of the other one, which only issue the instruction.  The form that releases
// at cluster scope waits for the warp's outstanding stores and loads: for the scales alone the
// MXFP4 product takes 73 for 40 us (24576 rows; 34 for 18 with 384), for the zeroed tails alone
// weight gradients 10 to 18% more (bf16, 24576 rows in ragged experts: 128 for 108 us).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// The end of both kernels, by all threads: no arrival, MMA or copy of the pair outlives either
// CTA.  After an abort a stage's copies may never complete their barrier together, so those in
// flight are given a fixed time.
__device__ __forceinline__ void leave_pair(volatile int *abort) {
    tc_fence_before();
    __syncthreads();
    if (*abort) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < kGraceNs) __nanosleep(1000);
    }
    __syncthreads();
    cluster_sync();
}

// One lane of a converged warp.  The roles that issue copies and MMAs run their loops on the
// whole warp and only the instructions themselves on one lane: the addresses and descriptors
// stay warp-uniform, which is what those instructions take (with the loop itself on one lane,
// issuing a stage's four MMAs measured 350 cycles of the 416 that they run).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// What every role reads per tile, in shared memory.
struct TileTable {
    GroupedOut o;                      // a parameter read that misses the constant cache costs more
    int offs[kMaxExperts + 1];         // first row of each expert
    int tiles[kMaxExperts];            // row-grouped: its first row tile; INT_MAX behind the last
    uint8_t share[kMaxExperts];        // row-grouped: rows of its tiles but the last, in units of 32
    int total;                         // tiles, 0 where the offsets decrease or leave [0, rows]
    int sums[kMaxExperts / 32];        // row-grouped: row tiles of 32 experts
    int c, r, e, dc, dr, de;           // this pair's first tile and the stride, see TileWalk
};

// What of the table depends on the launch alone, by one thread, before earlier kernels have ended.
template <bool DENSE>
__device__ __forceinline__ void start_table(const GroupedOut &p, TileTable &tab) {
    const int first = (int)blockIdx.x / 2, step = (int)gridDim.x / 2;
    int r = first / p.col_tiles, dr = step / p.col_tiles;
    tab.o = p;
    tab.c = first - r * p.col_tiles;
    tab.dc = step - dr * p.col_tiles;
    tab.e = DENSE ? r / p.row_tiles : 0;
    tab.de = DENSE ? dr / p.row_tiles : 0;
    tab.r = r - tab.e * p.row_tiles;
    tab.dr = dr - tab.de * p.row_tiles;
}

// The rest, from the offsets, by all threads of the CTA (at least 256, one per expert, so that the
// divisions take their time once: with 32 threads for them and more barriers this took 3800 cycles
// of every call, one token's six experts 8.7 instead of 7.5 us); false, in every CTA alike, for
// bad offsets.
template <bool DENSE>
__device__ __forceinline__ bool load_table(TileTable &tab) {
    const GroupedOut &p = tab.o;
    const int i = threadIdx.x, E = p.E, lane = i & 31, warp = i >> 5;
    int bad = 0, cnt = 0;
    if (i < E) {
        const int a = p.offs[i], b = p.offs[i + 1];
        tab.offs[i] = a;
        if (i == E - 1) tab.offs[E] = b;
        bad = a < 0 || a > b || b > p.rows;
        if (!DENSE && !bad && a < b) {
            cnt = (b - a + p.tile_rows - 1) / p.tile_rows;
            tab.share[i] = (uint8_t)(((cnt == 1 ? b - a : (b - a + cnt - 1) / cnt) + 31) / 32);
        }
    }
    int incl = cnt;
    if (!DENSE) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 31 && warp < kMaxExperts / 32) tab.sums[warp] = incl;
    }
    const bool ok = !__syncthreads_or(bad);
    if (i < kMaxExperts) {
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; !DENSE && w < kMaxExperts / 32; ++w) {
            if (w < warp) before += tab.sums[w];
            all += tab.sums[w];
        }
        if (!DENSE) tab.tiles[i] = i < E ? before + incl - cnt : 0x7fffffff;
        if (i == 0) tab.total = !ok ? 0 : DENSE ? E * p.row_tiles * p.col_tiles : all * p.col_tiles;
    }
    __syncthreads();
    return ok;
}

// The tensor core's additions truncate, so a sum's error grows with the number of instructions that
// add to one accumulator: 256 of them are up to 1.4e-5 off (products of one sign; 4.4e-6 of mixed
// ones), 4096 3.6e-4, 65536 6e-3, more than bf16's own rounding.  Longer sums are taken in segments,
// added to nearest in tensor memory, and the error stays that of one: of 256 instructions for fp32
// results, and for bf16 ones of 1024, at most 2^-14, a 64th of half a bf16 step.  `step`: products
// that an instruction adds.
__host__ __device__ constexpr int segment_of(bool f32, int step) { return (f32 ? 256 : 1024) * step; }

// What a role knows of the two accumulators: which one the next tile takes, and the parity of
// each one's next phase as full and as empty.  A sum of several segments takes one for all its
// segments and the other for their running sum, which frees that other when it has been stored;
// the next tile takes the first again, since that is free sooner.
struct Accumulators {
    uint32_t next = 0, full = 0, empty = 0;
    // MMA: the parity to wait for before a segment's products
    __device__ __forceinline__ uint32_t take() {
        const uint32_t parity = (empty >> next & 1u) ^ 1u;
        empty ^= 1u << next;
        return parity;
    }
    // epilogue: the parity to wait for before a segment's sums are read
    __device__ __forceinline__ uint32_t ready() {
        const uint32_t parity = full >> next & 1u;
        full ^= 1u << next;
        return parity;
    }
    // after a segment: the MMA counts the running sum's release, which it waits for in take()
    __device__ __forceinline__ void done(const Tile &t) {
        if (t.first && t.last)
            next ^= 1u;
        else if (t.last)
            empty ^= 1u << (next ^ 1u);
    }
};

// Walks a CTA pair's tiles first, first + stride, .. (a converged warp), numbered with the column
// tile innermost: the position is kept in digits, so that a step takes no division (one took a
// thousand cycles of the thread that feeds the tensor core).  An expert's rows are dealt evenly
// to its row tiles, in multiples of 32 (no tile is left empty: with `parts` tiles of at most T
// rows either parts <= T / 32, and rounding shares up takes fewer than `parts` * 32 of the more
// than T * (parts - 1) rows, or the shares are T).
template <bool DENSE, bool SEGMENTS = true>
struct TileWalk {
    const TileTable &tab;
    int tile, stride;
    int c, r, e;                 // column tile; row tile (dense: within the expert); dense: expert
    int dc, dr, de;              // the stride in the same digits
    int at = 0;                  // the first of the current segment's reduction steps
    // Dense: what the epilogue may take for the tiles passed.  Those of experts without rows are
    // nothing to the other roles, whose next wait then lasts as long as the zeros are stored.
    long long slack = 0;

    __device__ __forceinline__ TileWalk(const TileTable &table, int first, int step)
        : tab(table), tile(first), stride(step), c(table.c), r(table.r), e(table.e), dc(table.dc), dr(table.dr), de(table.de) {}
    __device__ __forceinline__ bool more() const { return tile < tab.total; }
    __device__ __forceinline__ void next() {
        if (SEGMENTS && at + tab.o.segment < (DENSE ? tab.offs[e + 1] - tab.offs[e] : tab.o.red)) {
            at += tab.o.segment;
            return;
        }
        at = 0;
        if (DENSE) slack += kTileCycles;
        tile += stride;
        c += dc;
        r += dr;
        e += de;
        if (c >= tab.o.col_tiles) {
            c -= tab.o.col_tiles;
            ++r;
        }
        if (DENSE && r >= tab.o.row_tiles) {
            r -= tab.o.row_tiles;
            ++e;
        }
    }
    // the current tile (more() holds)
    __device__ __forceinline__ Tile get() const {
        const GroupedOut &p = tab.o;
        Tile t;
        t.col0 = c * p.cols;
        if (DENSE) {
            t.e = e;
            t.row0 = r * p.tile_rows;
            t.rows = min(p.tile_rows, p.m_dense - t.row0);
            t.r0 = tab.offs[e] + at;
            t.r1 = SEGMENTS ? t.r0 + min(tab.offs[e + 1] - t.r0, p.segment) : tab.offs[e + 1];
            t.last = !SEGMENTS || t.r1 == tab.offs[e + 1];
        } else {
            // the last expert whose first row tile is <= r (one with rows: the next ones start later)
            constexpr int kPer = kMaxExperts / 32;
            const int lane = threadIdx.x & 31;
            const int group = __popc(__ballot_sync(0xffffffffu, tab.tiles[lane * kPer] <= r)) - 1;
            const int in = __popc(__ballot_sync(0xffffffffu, lane < kPer && tab.tiles[group * kPer + lane] <= r));
            t.e = group * kPer + in - 1;
            const int share = 32 * tab.share[t.e];
            t.row0 = tab.offs[t.e] + (r - tab.tiles[t.e]) * share;
            t.rows = min(share, tab.offs[t.e + 1] - t.row0);
            t.r0 = at;
            t.r1 = SEGMENTS ? at + min(p.red - at, p.segment) : p.red;
            t.last = !SEGMENTS || t.r1 == p.red;
        }
        t.n = (t.rows + 31) & ~31;
        t.first = !SEGMENTS || at == 0;
        return t;
    }
};

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// fp32 weight gradients are bound by their own stores: with both warps storing, their bursts
// delay the operand loads (160 against 166 us; bf16 ones 26.6 against 24.6 us the other way)
template <bool DENSE, int PARTS>
__device__ __forceinline__ int storing_parts(const GroupedOut &p) {
    return DENSE && p.f32 ? 1 : PARTS;
}

// Add a segment's accumulator to the running sum of its tile (fp32, to nearest): by the warp, and
// in the chunks, that store_tile then stores.
template <bool DENSE, int PARTS>
__device__ __forceinline__ void add_segment(const GroupedOut &p, const Tile &t, uint32_t acc, uint32_t run, int part) {
    const int parts = storing_parts<DENSE, PARTS>(p);
    if (part >= parts) return;
    for (int c = 32 * part; c < t.rows; c += 32 * parts) {
        uint32_t v[32], sum[32];
        tmem_ld32(acc + c, v);
        if (!t.first) tmem_ld32(run + c, sum);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));  // not read before the wait
        if (!t.first) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                asm volatile("" : "+r"(sum[i]));
                v[i] = __float_as_uint(__uint_as_float(sum[i]) + __uint_as_float(v[i]));
            }
        }
        tmem_st32(run + c, v);
    }
    tmem_st_wait();
}

// A tile's epilogue by one warp: TMEM lane = output column `col` (its own lane's), column = row.
// `tcol`: the accumulator, at the warp's lane quadrant; `empty`: there is no sum, zeros are
// stored; PARTS warps share a quadrant, this one takes the 32-row chunks `part`, part + PARTS, ..
// ADD: to what the output holds, in fp32.
template <bool DENSE, bool ADD, int PARTS>
__device__ __forceinline__ void store_tile(const GroupedOut &p, const Tile &t, uint32_t tcol, bool empty, int col,
                                           int part, int lane) {
    const int parts = storing_parts<DENSE, PARTS>(p);
    if ((ADD && empty) || part >= parts) return;
    const bool ok = col < p.n_out;
    const size_t row0 = (DENSE ? (size_t)t.e * p.m_dense : 0) + t.row0;
    const size_t ld = p.n_out;
    for (int c = 32 * part; c < t.rows; c += 32 * parts) {
        uint32_t v[32];
        if (DENSE && empty) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
        } else {
            tmem_ld32(tcol + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));  // not read before the wait
        }
        const int rows = ok ? min(32, t.rows - c) : 0;
        if (p.f32) {
            float *o = static_cast<float *>(p.out) + (row0 + c) * ld + col;
            if (ADD) {
#pragma unroll
                for (int g = 0; g < 32; g += 8) {  // eight loads in flight
                    float old[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) old[j] = g + j < rows ? o[(g + j) * ld] : 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (g + j < rows) o[(g + j) * ld] = old[j] + __uint_as_float(v[g + j]);
                }
            } else if (rows == 32) {
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j * ld] = __uint_as_float(v[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j < rows) o[j * ld] = __uint_as_float(v[j]);
            }
        } else {
            // n_out is even, so lanes 2i and 2i + 1 are in or out together: the even lane takes
            // both columns of row j, the odd one of row j + 1, in one 4-byte access
            const int odd = lane & 1;
            uint32_t *o = reinterpret_cast<uint32_t *>(static_cast<bf16 *>(p.out) + (row0 + c + odd) * ld + (col & ~1));
            const int left = rows - odd;
            uint32_t w[16], old[16];
            if (ADD) {
#pragma unroll
                for (int j = 0; j < 16; ++j) old[j] = 2 * j < left ? o[j * ld] : 0u;  // two rows on: n_out words
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (ADD) {
                    const uint32_t mine = odd ? v[2 * j + 1] : v[2 * j], give = odd ? v[2 * j] : v[2 * j + 1];
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
                    w[j] = pack_bf16x2(__uint_as_float(odd ? got : mine) + bf16_lo(old[j]),
                                       __uint_as_float(odd ? mine : got) + bf16_hi(old[j]));
                } else {
                    const uint32_t mine = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, mine, 1);
                    w[j] = __byte_perm(mine, got, odd ? 0x3276 : 0x5410);
                }
            }
            if (rows == 32) {
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j * ld] = w[j];
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (2 * j < left) o[j * ld] = w[j];
            }
        }
    }
}

}  // namespace moe
