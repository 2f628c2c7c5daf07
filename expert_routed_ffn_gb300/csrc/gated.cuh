// The epilogues of the gated block's products: from a tile's sums in tensor memory to the
// activation (forward) or to its two gradients (backward).
//
//   silu      H = g s(g) u
//   clamped   H = g' s(alpha g') (u' + beta),  g' = min(g, limit), u' = clamp(u, -limit, limit)
// with s(x) = 1 / (1 + exp(-x)).  For the gradients let p = s(alpha g'), v = u' + beta (silu: alpha
// 1, v = u, nothing clamped):
//   dG = dH v p (1 + alpha g' (1 - p))   and 0 where g > limit
//   dU = dH g' p                         and 0 where |u| > limit
#pragma once

#include "grouped.cuh"

namespace moe {

struct GatedOut {
    bf16 *g, *u;         // forward: where both projections go, or NULL; backward: dG, dU
    const bf16 *gi, *ui; // backward: both projections
    int I;               // their columns
    int act;
    float alpha, limit, beta;
};

// Approximate exponential and reciprocal, each good to a few units in the last place, far below bf16's
// rounding: s(x) = 1 / (1 + 2^(-x log2 e)), 0 where the power overflows.  NaN passes through the clamps (fmin
// would drop it).
__device__ __forceinline__ float gated_sigmoid(float x) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return s;
}
template <bool CLAMPED>
__device__ __forceinline__ float gated_act(float g, float u, const GatedOut &p) {
    if (CLAMPED) {
        g = g > p.limit ? p.limit : g;
        u = u > p.limit ? p.limit : u < -p.limit ? -p.limit : u;
        return g * gated_sigmoid(p.alpha * g) * (u + p.beta);
    }
    return g * gated_sigmoid(g) * u;
}
template <bool CLAMPED>
__device__ __forceinline__ void gated_grad(float dh, float g, float u, const GatedOut &p, float &dg, float &du) {
    if (CLAMPED) {
        const bool pass_g = !(g > p.limit), pass_u = !(u > p.limit || u < -p.limit);
        g = pass_g ? g : p.limit;
        u = pass_u ? u : u > 0.0f ? p.limit : -p.limit;
        const float s = gated_sigmoid(p.alpha * g), a = g * s;
        dg = pass_g ? dh * (u + p.beta) * fmaf(p.alpha * a, 1.0f - s, s) : 0.0f;
        du = pass_u ? dh * a : 0.0f;
    } else {
        const float s = gated_sigmoid(g), a = g * s;
        dg = dh * u * fmaf(a, 1.0f - s, s);
        du = dh * a;
    }
}

// 16 consecutive fp32 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Rows of a chunk: 16, so that the state of a chunk and of the next one's loads fits the registers of
// four epilogue warps per TMEM lane quadrant.
constexpr int kGatedRows = 16;

// Lanes 2i and 2i + 1 hold two columns' values of rows 2j and 2j + 1: the even lane gets both
// columns of row 2j, the odd one of row 2j + 1, as one word.
__device__ __forceinline__ uint32_t pack_pair(float row0, float row1, int odd) {
    const uint32_t mine = pack_bf16x2(row0, row1), got = __shfl_xor_sync(0xffffffffu, mine, 1);
    return __byte_perm(mine, got, odd ? 0x3276 : 0x5410);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// add_segment (grouped.cuh) in this file's chunks: a warp adds up what it will store itself.
template <int PARTS>
__device__ __forceinline__ void add_gated_segment(const Tile &t, uint32_t acc, uint32_t run, int part) {
    for (int c = kGatedRows * part; c < t.rows; c += kGatedRows * PARTS) {
        uint32_t v[kGatedRows], sum[kGatedRows];
        tmem_ld16(acc + c, v);
        if (!t.first) tmem_ld16(run + c, sum);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < kGatedRows; ++i) asm volatile("" : "+r"(v[i]));  // not read before the wait
        if (!t.first) {
#pragma unroll
            for (int i = 0; i < kGatedRows; ++i) {
                asm volatile("" : "+r"(sum[i]));
                v[i] = __float_as_uint(__uint_as_float(sum[i]) + __uint_as_float(v[i]));
            }
        }
        tmem_st16(run + c, v);
    }
    tmem_st_wait();
}

// The running sums of a tile's segments, to nearest, in the registers of the warps that store them: a warp
// has its 32-row chunks of store_tile.  Segments so take the two accumulators in turn, and the MMA goes
// on with one while the other is added here; with the sums in tensor memory (add_segment) it waits for
// each segment's addition (32 instructions a segment, 24576 rows of 64 experts: 237 for 209 us).  All
// roles walk tiles and count the segments inside (walking segments, as the other long sums do, 218).
// The last segment's sums end in its accumulator, where store_tile reads them.
template <int PARTS>
struct RegisterSums {
    static constexpr int kPieces = 2 * (256 / 32 / PARTS);  // of 16 rows
    float sum[kPieces][16];
    __device__ __forceinline__ void add(const Tile &t, uint32_t acc, int part, bool last) {
#pragma unroll
        for (int g = 0; g < kPieces; ++g) {
            const int c = 32 * (part + PARTS * (g / 2)) + 16 * (g % 2);
            if (c < t.rows) {
                uint32_t v[16];
                tmem_ld16(acc + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    asm volatile("" : "+r"(v[i]));  // not read before the wait
                    sum[g][i] += __uint_as_float(v[i]);
                    v[i] = __float_as_uint(sum[g][i]);
                }
                if (last) tmem_st16(acc + c, v);
            }
        }
        if (last) tmem_st_wait();
    }
};

// Forward.  The MMA's columns alternate 16 of the gate's and the same 16 of the up projection's, so
// that lanes l and l + 16 of a warp hold both values of a column: lane l takes the first half of a
// chunk's rows, lane l + 16 the second, exchanged by shuffles.  (With 64 columns of each in the
// lane halves the exchange would go through shared memory and barriers of two warps.)
// col: the lane's output column.
template <bool CLAMPED, int PARTS>
__device__ __forceinline__ void store_gated_as(const GatedOut &p, void *out, const Tile &t, uint32_t tcol, int col, int part,
                                               int lane) {
    constexpr int kHalf = kGatedRows / 2;
    const int up = lane >> 4, odd = lane & 1;
    const size_t ld = p.I / 2;  // in words
    for (int c = kGatedRows * part; c < t.rows; c += kGatedRows * PARTS) {
        uint32_t v[kGatedRows];
        tmem_ld16(tcol + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < kGatedRows; ++i) asm volatile("" : "+r"(v[i]));  // not read before the wait
        const int row = c + kHalf * up + odd;  // of the tile; this lane stores rows row, row + 2, ..
        const int left = col < p.I ? t.rows - row : 0;  // I is even: both lanes of a pair or none
        const size_t at = (size_t)(t.row0 + row) * ld + col / 2;
        uint32_t *h = static_cast<uint32_t *>(out) + at;
        uint32_t *gs = reinterpret_cast<uint32_t *>(p.g) + at, *us = reinterpret_cast<uint32_t *>(p.u) + at;
#pragma unroll
        for (int j = 0; j < kHalf; j += 2) {
            float g[2], u[2], r[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v[j + i] : v[kHalf + j + i], 16);
                g[i] = __uint_as_float(up ? got : v[j + i]);
                u[i] = __uint_as_float(up ? v[kHalf + j + i] : got);
                r[i] = gated_act<CLAMPED>(g[i], u[i], p);
            }
            const uint32_t w = pack_pair(r[0], r[1], odd);
            if (j < left) h[j * ld] = w;
            if (p.g != nullptr) {
                const uint32_t wg = pack_pair(g[0], g[1], odd), wu = pack_pair(u[0], u[1], odd);
                if (j < left) {
                    gs[j * ld] = wg;
                    us[j * ld] = wu;
                }
            }
        }
    }
}
template <int PARTS>
__device__ __forceinline__ void store_gated(const GatedOut &p, void *out, const Tile &t, uint32_t tcol, int col, int part, int lane) {
    if (p.act == MOE_ACT_SWIGLU_OAI)
        store_gated_as<true, PARTS>(p, out, t, tcol, col, part, lane);
    else
        store_gated_as<false, PARTS>(p, out, t, tcol, col, part, lane);
}

// Backward: the sums are dH, a lane's column is its output column.  A lane pair exchanges sums so that
// each lane has both columns of every other row: one word of G, U, dG and dU.  A chunk's G and U are
// asked for a chunk ahead (fetch), the first before the sums are there.
struct GatedBack {
    uint32_t g[kGatedRows / 2], u[kGatedRows / 2];  // of the next chunk
    __device__ __forceinline__ void fetch(const GatedOut &p, const Tile &t, int col, int c, int lane) {
        const int row = c + (lane & 1), left = col < p.I ? t.rows - row : 0;
        const size_t ld = p.I / 2, at = (size_t)(t.row0 + row) * ld + col / 2;  // in words
        const uint32_t *gi = reinterpret_cast<const uint32_t *>(p.gi) + at, *ui = reinterpret_cast<const uint32_t *>(p.ui) + at;
#pragma unroll
        for (int j = 0; j < kGatedRows / 2; ++j) {
            g[j] = 2 * j < left ? gi[2 * j * ld] : 0u;
            u[j] = 2 * j < left ? ui[2 * j * ld] : 0u;
        }
    }
    template <bool CLAMPED, int PARTS>
    __device__ __forceinline__ void store_as(const GatedOut &p, const Tile &t, uint32_t tcol, int col, int part, int lane) {
        const int odd = lane & 1;
        const size_t ld = p.I / 2;
        for (int c = kGatedRows * part; c < t.rows; c += kGatedRows * PARTS) {
            const int row = c + odd, left = col < p.I ? t.rows - row : 0;
            const size_t at = (size_t)(t.row0 + row) * ld + col / 2;
            uint32_t *dg = reinterpret_cast<uint32_t *>(p.g) + at, *du = reinterpret_cast<uint32_t *>(p.u) + at;
            uint32_t wg[kGatedRows / 2], wu[kGatedRows / 2];
#pragma unroll
            for (int j = 0; j < kGatedRows / 2; ++j) wg[j] = g[j], wu[j] = u[j];
            if (c + kGatedRows * PARTS < t.rows) fetch(p, t, col, c + kGatedRows * PARTS, lane);
            uint32_t v[kGatedRows];
            tmem_ld16(tcol + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < kGatedRows; ++i) asm volatile("" : "+r"(v[i]));  // not read before the wait
#pragma unroll
            for (int j = 0; j < kGatedRows / 2; ++j) {
                const uint32_t mine = odd ? v[2 * j + 1] : v[2 * j], give = odd ? v[2 * j] : v[2 * j + 1];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
                const float lo = __uint_as_float(odd ? got : mine), hi = __uint_as_float(odd ? mine : got);
                float a[2], b[2];
                gated_grad<CLAMPED>(lo, bf16_lo(wg[j]), bf16_lo(wu[j]), p, a[0], b[0]);
                gated_grad<CLAMPED>(hi, bf16_hi(wg[j]), bf16_hi(wu[j]), p, a[1], b[1]);
                if (2 * j < left) {
                    dg[2 * j * ld] = pack_bf16x2(a[0], a[1]);
                    du[2 * j * ld] = pack_bf16x2(b[0], b[1]);
                }
            }
        }
    }
    template <int PARTS>
    __device__ __forceinline__ void store(const GatedOut &p, const Tile &t, uint32_t tcol, int col, int part, int lane) {
        if (p.act == MOE_ACT_SWIGLU_OAI)
            store_as<true, PARTS>(p, t, tcol, col, part, lane);
        else
            store_as<false, PARTS>(p, t, tcol, col, part, lane);
    }
};

}  // namespace moe
