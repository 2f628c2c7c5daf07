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
constexpr int kEpiWarps = 4;          // epilogue warps, one per TMEM lane quadrant
constexpr long long kWaitCycles = 4000000000ll;         // bound of every wait (about 2 s)
constexpr unsigned long long kPairDrainNs = 1000000ull; // grace for the copies in flight after an abort

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
    int accumulate;  // dense: add to the output
};

struct Tile {
    int e, row0, rows, n, col0;  // expert, first output row, valid rows, MMA N, first output column
    int r0, r1;                  // reduction range
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

// Wait until the phase of parity `parity` of a barrier has completed; CLUSTER: a barrier that
// threads of the other CTA arrive on.  Bounded by the SM's clock (the global timer is slow to
// read beside waits this short).  False after the bound, or once *abort is set.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort) {
    auto done = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    if (done()) return true;
    const long long t0 = clock64();
    for (;;) {
        if (done()) return true;
        if (abort != nullptr && *abort) return false;
        if (clock64() - t0 > kWaitCycles) return false;
    }
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
    uint16_t share[kMaxExperts];       // row-grouped: rows of its tiles but the last, a multiple of 32
    int total;                         // tiles, 0 where the offsets decrease or leave [0, rows]
};

// Fill the table (all threads of the CTA); false, in every CTA alike, for bad offsets.
template <bool DENSE>
__device__ __forceinline__ bool load_table(const GroupedOut &p, TileTable &tab) {
    const int E = p.E;
    if (threadIdx.x == 0) tab.o = p;
    for (int i = threadIdx.x; i <= E; i += blockDim.x) tab.offs[i] = p.offs[i];
    __syncthreads();
    int bad = 0;
    for (int i = threadIdx.x; i < E; i += blockDim.x) bad |= tab.offs[i] > tab.offs[i + 1];
    bad |= tab.offs[0] < 0 || tab.offs[E] > p.rows;
    const bool ok = !__syncthreads_or(bad);
    if (threadIdx.x < 32) {
        constexpr int kPer = kMaxExperts / 32;
        const int lane = threadIdx.x;
        int cnt[kPer], sum = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int e = lane * kPer + j, rows = !DENSE && ok && e < E ? tab.offs[e + 1] - tab.offs[e] : 0;
            cnt[j] = (rows + p.tile_rows - 1) / p.tile_rows;
            if (!DENSE && cnt[j] > 0) tab.share[e] = (uint16_t)(((rows + cnt[j] - 1) / cnt[j] + 31) & ~31);
            sum += cnt[j];
        }
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        int run = incl - sum;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int e = lane * kPer + j;
            tab.tiles[e] = e < E ? run : 0x7fffffff;
            run += cnt[j];
        }
        if (lane == 31) tab.total = !ok ? 0 : DENSE ? E * p.row_tiles * p.col_tiles : run * p.col_tiles;
    }
    __syncthreads();
    return ok;
}

// Tile number -> tile, by a converged warp.  Inside an expert the row tiles of one column tile
// are adjacent, so that concurrent CTAs share its weights in L2; its rows are dealt evenly to
// its row tiles, in multiples of 32 (no tile is left empty: with `parts` tiles of at most T
// rows either parts <= T / 32, and rounding shares up takes fewer than `parts` * 32 of the more
// than T * (parts - 1) rows, or the shares are T).
template <bool DENSE>
__device__ __forceinline__ Tile decode(const TileTable &tab, int tile) {
    const GroupedOut &p = tab.o;
    Tile t;
    if (DENSE) {
        const int parts = p.row_tiles, strip = tile / parts;  // (expert, column tile)
        t.e = strip / p.col_tiles;
        t.col0 = (strip - t.e * p.col_tiles) * p.cols;
        t.row0 = (tile - strip * parts) * p.tile_rows;
        t.rows = min(p.tile_rows, p.m_dense - t.row0);
        t.r0 = tab.offs[t.e];
        t.r1 = tab.offs[t.e + 1];
    } else {
        // the last expert whose first tile is <= tile (one with rows: the next ones start later)
        const int lane = threadIdx.x & 31;
        const int row_tile = tile / p.col_tiles;  // experts are whole multiples of col_tiles
        const int group = __popc(__ballot_sync(0xffffffffu, tab.tiles[lane * (kMaxExperts / 32)] <= row_tile)) - 1;
        const int in = __popc(__ballot_sync(0xffffffffu, lane < kMaxExperts / 32 &&
                                                              tab.tiles[group * (kMaxExperts / 32) + lane] <= row_tile));
        t.e = group * (kMaxExperts / 32) + in - 1;
        const int first = tab.offs[t.e], end = tab.offs[t.e + 1];
        const int share = tab.share[t.e], parts = (end - first + p.tile_rows - 1) / p.tile_rows;
        const int local = tile - tab.tiles[t.e] * p.col_tiles, strip = local / parts;
        t.col0 = strip * p.cols;
        t.row0 = first + (local - strip * parts) * share;
        t.rows = min(share, end - t.row0);
        t.r0 = 0;
        t.r1 = p.red;
    }
    t.n = (t.rows + 31) & ~31;
    return t;
}

// A tile's epilogue by one warp: TMEM lane = output column `col` (its own lane's; `col_ok`:
// inside the output), column = row.  `tcol`: the accumulator, at the warp's lane quadrant;
// `empty`: there is no sum, zeros are stored.  ADD: to what the output holds, in fp32.
template <bool DENSE, bool ADD>
__device__ __forceinline__ void store_rows(const GroupedOut &p, const Tile &t, uint32_t tcol, bool empty, int col,
                                           int lane) {
    const bool ok = col < p.n_out;
    const size_t row0 = (DENSE ? (size_t)t.e * p.m_dense : 0) + t.row0;
    const size_t ld = p.n_out;
    for (int c = 0; c < t.rows; c += 32) {
        uint32_t v[32];
        if (DENSE && empty) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
        } else {
            tmem_ld32(tcol + c, v);
            tmem_ld_wait();
        }
        const int rows = ok ? min(32, t.rows - c) : 0;
        if (p.f32) {
            float *o = static_cast<float *>(p.out) + (row0 + c) * ld + col;
            if (ADD) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j < rows) v[j] = __float_as_uint(__uint_as_float(v[j]) + o[j * ld]);
            }
            if (rows == 32) {
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
                const uint32_t mine = odd ? v[2 * j + 1] : v[2 * j], give = odd ? v[2 * j] : v[2 * j + 1];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
                float lo = __uint_as_float(odd ? got : mine), hi = __uint_as_float(odd ? mine : got);
                if (ADD) {
                    lo += bf16_lo(old[j]);
                    hi += bf16_hi(old[j]);
                }
                w[j] = pack_bf16x2(lo, hi);
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
template <bool DENSE>
__device__ __forceinline__ void store_tile(const GroupedOut &p, const Tile &t, uint32_t tcol, bool empty, int col,
                                           int lane) {
    if (DENSE && p.accumulate) {
        if (!empty) store_rows<DENSE, true>(p, t, tcol, false, col, lane);
    } else {
        store_rows<DENSE, false>(p, t, tcol, empty, col, lane);
    }
}

}  // namespace moe
