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

// Fast exponential and quotient: relative errors near 1e-6, far below bf16's rounding.  NaN passes
// through the clamps (fmin would drop it).
__device__ __forceinline__ float gated_sigmoid(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }
__device__ __forceinline__ float gated_act(float g, float u, const GatedOut &p) {
    if (p.act == MOE_ACT_SWIGLU_OAI) {
        g = g > p.limit ? p.limit : g;
        u = u > p.limit ? p.limit : u < -p.limit ? -p.limit : u;
        return g * gated_sigmoid(p.alpha * g) * (u + p.beta);
    }
    return g * gated_sigmoid(g) * u;
}
__device__ __forceinline__ void gated_grad(float dh, float g, float u, const GatedOut &p, float &dg, float &du) {
    if (p.act == MOE_ACT_SWIGLU_OAI) {
        const bool pass_g = !(g > p.limit), pass_u = !(u > p.limit || u < -p.limit);
        g = pass_g ? g : p.limit;
        u = pass_u ? u : u > 0.0f ? p.limit : -p.limit;
        const float s = gated_sigmoid(p.alpha * g);
        dg = pass_g ? dh * (u + p.beta) * (s * (1.0f + p.alpha * g * (1.0f - s))) : 0.0f;
        du = pass_u ? dh * (g * s) : 0.0f;
    } else {
        const float s = gated_sigmoid(g);
        dg = dh * u * (s * (1.0f + g * (1.0f - s)));
        du = dh * (g * s);
    }
}

// Lanes 2i and 2i + 1 hold two columns' values of rows 2j and 2j + 1: the even lane gets both
// columns of row 2j, the odd one of row 2j + 1, as one word.
__device__ __forceinline__ uint32_t pack_pair(float row0, float row1, int odd) {
    const uint32_t mine = pack_bf16x2(row0, row1), got = __shfl_xor_sync(0xffffffffu, mine, 1);
    return __byte_perm(mine, got, odd ? 0x3276 : 0x5410);
}

// Forward.  The MMA's columns alternate 16 of the gate's and the same 16 of the up projection's, so
// that lanes l and l + 16 of a warp hold both values of a column: lane l takes rows 0-15 of a
// chunk of 32, lane l + 16 rows 16-31, exchanged by shuffles.  (With 64 columns of each in the
// lane halves the exchange would go through shared memory and barriers of two warps.)
// col: the lane's output column.
template <int PARTS>
__device__ __forceinline__ void store_gated(const GroupedOut &o, const GatedOut &p, const Tile &t, uint32_t tcol, int col,
                                            int part, int lane) {
    const int up = lane >> 4, odd = lane & 1;
    const bool ok = col < p.I;  // I is even: both lanes of a pair or none
    const size_t ld = p.I;
    for (int c = 32 * part; c < t.rows; c += 32 * PARTS) {
        uint32_t v[32];
        tmem_ld32(tcol + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));  // not read before the wait
        const int row = c + 16 * up + odd;  // of the tile; this lane stores rows row, row + 2, ..
        const int left = ok ? t.rows - row : 0;
        const size_t at = ((size_t)(t.row0 + row) * ld + (col & ~1)) / 2;
        uint32_t *h = static_cast<uint32_t *>(o.out) + at;
        uint32_t *gs = reinterpret_cast<uint32_t *>(p.g) + at, *us = reinterpret_cast<uint32_t *>(p.u) + at;
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            float g[2], u[2], r[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v[j + i] : v[16 + j + i], 16);
                g[i] = __uint_as_float(up ? got : v[j + i]);
                u[i] = __uint_as_float(up ? v[16 + j + i] : got);
                r[i] = gated_act(g[i], u[i], p);
            }
            const uint32_t w = pack_pair(r[0], r[1], odd);
            if (j < left) h[j * (ld / 2)] = w;
            if (p.g != nullptr) {
                const uint32_t wg = pack_pair(g[0], g[1], odd), wu = pack_pair(u[0], u[1], odd);
                if (j < left) {
                    gs[j * (ld / 2)] = wg;
                    us[j * (ld / 2)] = wu;
                }
            }
        }
    }
}

// Backward: the sums are dH, a lane's column is its output column.  A lane pair exchanges sums so that
// each lane has both columns of every other row: one word of G, U, dG and dU.  A chunk's G and U are
// asked for a chunk ahead (fetch), the first before the sums are there: with the loads after it each
// chunk waited for them (24576 rows, 64 experts of 1408 x 2048: 179 us).
struct GatedBack {
    uint32_t g[16], u[16];  // of the next chunk
    __device__ __forceinline__ void fetch(const GatedOut &p, const Tile &t, int col, int c, int lane) {
        const int row = c + (lane & 1), left = col < p.I ? t.rows - row : 0;
        const size_t ld = p.I / 2, at = (size_t)(t.row0 + row) * ld + col / 2;  // in words
        const uint32_t *gi = reinterpret_cast<const uint32_t *>(p.gi) + at, *ui = reinterpret_cast<const uint32_t *>(p.ui) + at;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            g[j] = 2 * j < left ? gi[2 * j * ld] : 0u;
            u[j] = 2 * j < left ? ui[2 * j * ld] : 0u;
        }
    }
    template <int PARTS>
    __device__ __forceinline__ void store(const GatedOut &p, const Tile &t, uint32_t tcol, int col, int part, int lane) {
        const int odd = lane & 1;
        const size_t ld = p.I / 2;
        for (int c = 32 * part; c < t.rows; c += 32 * PARTS) {
            const int row = c + odd, left = col < p.I ? t.rows - row : 0;
            const size_t at = (size_t)(t.row0 + row) * ld + col / 2;
            uint32_t *dg = reinterpret_cast<uint32_t *>(p.g) + at, *du = reinterpret_cast<uint32_t *>(p.u) + at;
            uint32_t wg[16], wu[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) wg[j] = g[j], wu[j] = u[j];
            if (c + 32 * PARTS < t.rows) fetch(p, t, col, c + 32 * PARTS, lane);
            uint32_t v[32];
            tmem_ld32(tcol + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));  // not read before the wait
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const uint32_t mine = odd ? v[2 * j + 1] : v[2 * j], give = odd ? v[2 * j] : v[2 * j + 1];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
                const float lo = __uint_as_float(odd ? got : mine), hi = __uint_as_float(odd ? mine : got);
                float a[2], b[2];
                gated_grad(lo, bf16_lo(wg[j]), bf16_lo(wu[j]), p, a[0], b[0]);
                gated_grad(hi, bf16_hi(wg[j]), bf16_hi(wu[j]), p, a[1], b[1]);
                if (2 * j < left) {
                    dg[2 * j * ld] = pack_bf16x2(a[0], a[1]);
                    du[2 * j * ld] = pack_bf16x2(b[0], b[1]);
                }
            }
        }
    }
};

}  // namespace moe
