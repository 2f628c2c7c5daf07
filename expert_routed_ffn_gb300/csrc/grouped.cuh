// What the products over expert-grouped rows share: the tile list derived from the row
// offsets, and the epilogue that moves a tile from tensor memory to its output rows.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "op_host.h"

namespace moe {

constexpr int kMaxExperts = 256;
constexpr int kEpiWarps = 4;          // epilogue warps, one per TMEM lane quadrant
constexpr int kEpiBytes = kEpiWarps * 4096;
constexpr unsigned long long kWaitNs = 2000000000ull;   // bound of every wait
constexpr unsigned long long kDrainNs = 1000000000ull;  // bound of the drain after an abort

// The output and its tiles.  Row-grouped (forward, dgrad): out [rows, n_out], the rows of
// expert e are [offs[e], offs[e + 1]).  Dense (wgrad): out [E, m_dense, n_out], and the
// offsets bound the reduction.
struct GroupedOut {
    CUtensorMap map;  // boxes of [32 rows][128 bytes], 128-byte swizzle
    const int32_t *offs;
    void *out;
    int *err;
    int E, rows;
    int n_out;       // columns of the output
    int m_dense;     // dense: rows of one expert's output
    int red;         // row-grouped: length of the reduction
    int bm, bn;      // tile: rows (32 or 128) and columns
    int n_tiles;     // tiles along the output columns
    int m_tiles;     // dense: tiles along m_dense
    int f32;         // output type: fp32, else bf16
    int accumulate;  // dense: add to the output
};

struct Tile {
    int e, row0, m_valid, col0;  // expert, first output row, valid rows, first output column
    int r0, r1;                  // reduction range
};

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void fence_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// Expert offsets into s_offs, their tile prefix into s_tiles; false (in every CTA alike)
// if they decrease or leave [0, rows].
template <bool DENSE>
__device__ __forceinline__ bool load_offsets(const GroupedOut &p, int *s_offs, int *s_tiles) {
    const int E = p.E;
    for (int i = threadIdx.x; i <= E; i += blockDim.x) s_offs[i] = p.offs[i];
    __syncthreads();
    int bad = 0;
    for (int i = threadIdx.x; i < E; i += blockDim.x) bad |= s_offs[i] > s_offs[i + 1];
    bad |= s_offs[0] < 0 || s_offs[E] > p.rows;
    if (__syncthreads_or(bad)) return false;
    if (!DENSE && threadIdx.x < 32) {
        constexpr int kPer = kMaxExperts / 32;
        const int lane = threadIdx.x;
        int cnt[kPer], sum = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int e = lane * kPer + j;
            cnt[j] = e < E ? (s_offs[e + 1] - s_offs[e] + p.bm - 1) / p.bm : 0;
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
            if (e <= E) s_tiles[e] = run;
            run += cnt[j];
        }
        if (lane == 31 && E == kMaxExperts) s_tiles[E] = run;
    }
    __syncthreads();
    return true;
}

// Tile number -> tile.  Inside an expert the row tiles of one column tile are adjacent, so
// that concurrent CTAs share its weights in L2.
template <bool DENSE>
__device__ __forceinline__ Tile decode(const GroupedOut &p, int tile, const int *s_offs, const int *s_tiles) {
    Tile t;
    if (DENSE) {
        const int per = p.m_tiles * p.n_tiles;
        t.e = tile / per;
        const int local = tile - t.e * per;
        t.col0 = (local / p.m_tiles) * p.bn;
        t.row0 = (local % p.m_tiles) * 128;
        t.m_valid = min(128, p.m_dense - t.row0);
        t.r0 = s_offs[t.e];
        t.r1 = s_offs[t.e + 1];
    } else {
        int lo = 0, hi = p.E - 1;  // the last expert whose first tile is <= tile
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_tiles[mid] * p.n_tiles <= tile)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int mt = s_tiles[lo + 1] - s_tiles[lo];
        const int local = tile - s_tiles[lo] * p.n_tiles;
        t.e = lo;
        t.col0 = (local / mt) * p.bn;
        t.row0 = s_offs[lo] + (local % mt) * p.bm;
        t.m_valid = min(p.bm, s_offs[lo + 1] - t.row0);
        t.r0 = 0;
        t.r1 = p.red;
    }
    return t;
}

// One warp's slice of the output, [32 rows][128 bytes of fp32 or bf16 columns] in its
// swizzled staging buffer `sb` (lane i wrote row i; 16-byte unit j at j ^ (i % 8)).
template <bool DENSE>
__device__ __forceinline__ void flush(const GroupedOut &p, const Tile &t, uint32_t sb, int row, int rows, int col,
                                      int lane) {
    const int u = lane & 7;
    if (DENSE && p.accumulate) {  // staged as 32 fp32 columns: dW + the product, in fp32
        __syncwarp();
        const int c = col + 4 * u;
        for (int i = lane >> 3; i < rows; i += 4) {
            const uint4 v = ld_shared_v4(sb + (uint32_t)i * 128u + ((uint32_t)(u ^ (i & 7)) << 4));
            if (c >= p.n_out) continue;
            const size_t at = ((size_t)t.e * p.m_dense + row + i) * p.n_out + c;
            if (p.f32) {
                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at);
                float4 old = *o;
                old.x += __uint_as_float(v.x);
                old.y += __uint_as_float(v.y);
                old.z += __uint_as_float(v.z);
                old.w += __uint_as_float(v.w);
                *o = old;
            } else {
                uint2 *o = reinterpret_cast<uint2 *>(static_cast<bf16 *>(p.out) + at);
                const uint2 old = *o;
                *o = make_uint2(pack_bf16x2(bf16_lo(old.x) + __uint_as_float(v.x), bf16_hi(old.x) + __uint_as_float(v.y)),
                                pack_bf16x2(bf16_lo(old.y) + __uint_as_float(v.z), bf16_hi(old.y) + __uint_as_float(v.w)));
            }
        }
        __syncwarp();
    } else if (DENSE || rows == 32) {  // past N or n_out the copy engine writes nothing
        fence_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(&p.map, sb, col, row, DENSE ? t.e : 0);
            bulk_commit();
        }
    } else {
        __syncwarp();
        const int es = p.f32 ? 4 : 2, c = col + (16 / es) * u;
        for (int i = lane >> 3; i < rows; i += 4) {
            const uint4 v = ld_shared_v4(sb + (uint32_t)i * 128u + ((uint32_t)(u ^ (i & 7)) << 4));
            if (c < p.n_out)
                *reinterpret_cast<uint4 *>(static_cast<char *>(p.out) + ((size_t)(row + i) * p.n_out + c) * es) = v;
        }
        __syncwarp();
    }
}

// The epilogue of one tile by one warp (TMEM lane quadrant q): its accumulator's columns at
// `tcol`, `empty` where there is no sum and zeros are stored.  `sb`: the warp's 4 KB staging
// buffer in shared memory.
template <bool DENSE>
__device__ __forceinline__ void store_tile(const GroupedOut &p, const Tile &t, uint32_t tcol, bool empty, uint32_t sb,
                                           int q, int lane) {
    const int rows = min(32, t.m_valid - 32 * q);
    if (rows <= 0 || (DENSE && empty && p.accumulate)) return;  // warp-uniform
    const bool wide = p.f32 || (DENSE && p.accumulate);         // staged as fp32
    const uint32_t tb = tcol + ((uint32_t)(q * 32) << 16), srow = sb + (uint32_t)lane * 128u;
    const int sw = lane & 7, end = min(p.bn, p.n_out - t.col0), step = wide ? 32 : 64;
#pragma unroll 1
    for (int c0 = 0; c0 < end; c0 += step) {
        if (lane == 0) bulk_wait_read_all();  // the previous slice's store has read the buffer
        __syncwarp();
#pragma unroll 1
        for (int h = 0; h < step; h += 32) {
            uint32_t v[32];
            if (DENSE && empty) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0u;
            } else {
                tmem_ld32(tb + c0 + h, v);
                tmem_ld_wait();
            }
            if (wide) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    st_shared_v4(srow + ((uint32_t)(j ^ sw) << 4), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            } else {
                uint32_t o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    st_shared_v4(srow + ((uint32_t)((h / 8 + j) ^ sw) << 4), o[4 * j], o[4 * j + 1], o[4 * j + 2],
                                 o[4 * j + 3]);
            }
        }
        flush<DENSE>(p, t, sb, t.row0 + 32 * q, rows, t.col0 + c0, lane);
    }
}

}  // namespace moe
