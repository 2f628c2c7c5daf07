// Newton-Schulz products that move the singular values of stacked matrices G [E, N, K] towards one
// (the update of the Muon optimiser).  With m the smaller side, X0 = G / (|G|_F + eps) and for
// each step's (a, b, c)
//   A = X X^T,   B = a + b A + c A^2,   X <- B X          (N <= K; else A = X^T X, X <- X B)
//
// Three products a step, m^2 n + m^3 + 2 m^2 n FLOP (A and B are symmetric: tiles above their
// diagonal are not computed but mirrored), all batched over the matrices.  Bound by the tensor
// cores.  No operand is transposed in memory: whichever side is smaller, a tile is read with its
// reduction index innermost or outermost, as in grouped.cu, whose tiles, pipeline of CTA pairs,
// descriptors and bounded waits this kernel has.
//
// Precision.  Every value between the products is fp16: X, A and B are bounded (|X| <= 1.3 for the
// usual coefficients; the host bounds the singular values step by step and picks power-of-two
// scales that keep them inside fp16), so fp16's 11 bits cost nothing over bf16's 8 and are eight
// times as accurate.  What rounding X still does: noise of 2^-12 of its largest directions enters
// the small ones, which the polynomial multiplies by up to a = 3.4 a step.  Of a small direction's
// change nearly all is a X, and b A + c A^2 nearly nothing; so the steps that matter (all but the last two)
// keep the rounding of X, hi + lo, and take lo through a X alone: X <- B hi + a lo, an
// epilogue's work; the tensor cores see hi only.  Where 16 directions are 300 times as large as
// the rest, the result's error (2-norm, relative) is 2.2e-3, of which its rounding to bf16 is 1.7e-3;
// with hi alone it would be 2.0e-2, with bf16 throughout 0.16.  Gaussian matrices and singular values
// falling as 1 / j: 2.1e-3 and 1.8e-3 (five steps; six of a Gaussian 224 x 96 in fp32: 2.4e-3).
// X0 is G times a power of two (exact for bf16 G: no lo), the rest of 1 / (|G| + eps) is a factor
// s in (1/2, 1] of the first A and B.  Sums are fp32 in tensor memory, over at most 16384
// products: the tensor core's truncation stays below 2^-13 (1.2e-4) of a sum of one sign.  Further steps of these
// coefficients, which move singular values about in [0.7, 1.2] for good, raise the error (3.4e-3 for 8, 7e-3 for 20,
// up to 3e-2 for 64); coefficients that converge keep it below 2e-3.
//
// Measured on GB300, 32 x 1408 x 2048 in fp32, five steps: 1.93 ms after a pause, 1.24 PFLOP/s of the products
// counted above, and 2.26 ms when called for seconds (power: 1.37 GHz); |G| 57 us and X0 with its lo 113 us (6.6 and 6.1 TB/s), then per
// step A 104, B 76 to 80 and X 187 us (with lo) or 160.  The tensor pipe is busy 70 to 78% of the cycles
// and the clock falls to 1.5 to 1.7 GHz of 2.07 (power): 5.5 tiles of 256 to a side make 18 tiles' work of the 15.1 below
// the diagonal, a tile's epilogue shares shared memory's bandwidth with the MMAs' operands, and a
// launch's first and last tiles leave SMs idle.  256 x 1024: 74 us in 17 launches, each
// bound by its latency (64 x 64: 49 us); 8 x 512 x 512 116, 1024 x 1024 101.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda_fp16.h>

#include "common.cuh"
#include "grouped.cuh"
#include "kernels.h"
#include "moe.h"
#include "op_host.h"

namespace moe {
namespace {

constexpr int kMaxSide = 16384;
constexpr int kBK = 64;                // reduction steps per stage: 128 bytes
constexpr int kMaxStages = 12;
// SMALL: half of an SM's shared memory, tensor memory and registers, so that while one product ends
// the next one's CTAs are there, with their barriers and tensor memory, and wait for it.  For
// products whose tiles are one wave of up to 128 rows (1024 x 1024 101 us for 109, 256 x 1024 74 for 76).
template <bool SMALL>
constexpr int kParts = SMALL ? 2 : 4;  // epilogue warps per TMEM lane quadrant
template <bool SMALL>
constexpr int kEpiWarps = kQuads * kParts<SMALL>;
template <bool SMALL>
constexpr int kThreads = 64 + 32 * kEpiWarps<SMALL>;
template <bool SMALL>
constexpr int kAccCols = SMALL ? 128 : 256;
constexpr int kRow = kBK * 2;          // bytes of a K-major row, or of 64 columns in MN-major
constexpr int kChunk = 64 * kRow;
template <bool SMALL>
constexpr int kStageSpace = SMALL ? 110592 : 229376;

struct Header {
    uint64_t bars[2 * kMaxStages + 5];
    uint32_t tmem;
    volatile int abort;
};
constexpr int kHeaderBytes = 1 << 10;
template <bool SMALL>
constexpr int kSmemBytes = kHeaderBytes + kStageSpace<SMALL>;
static_assert(sizeof(Header) <= kHeaderBytes && kSmemBytes<false> <= 232448, "shared memory of one CTA");
static_assert(2 * (kSmemBytes<true> + 1024) <= 233472, "shared memory of two on an SM");

// One batched product: out[e] [R, C], summed over `red`; columns are the MMA's M.
struct ProductArgs {
    CUtensorMap map_a, map_b;
    int E, R, C, red;
    int cols, tile_rows, row_tiles, col_tiles, tiles;
    int a_block, b_block, stages;
    long long wait;
    int *err;
    int col_shift;        // log2(cols)
    int ld;               // symmetric results: elements between rows, a multiple of 16
    // epilogue, see Symmetric and Update
    const float *table;   // first step: s of each matrix, else NULL
    const half *other;    // B: A; X: lo, or NULL
    half *out, *out_lo;   // out_lo: X, or NULL
    bf16 *final;          // X: the result, `scale` times, in place of out
    float scale;
    float k_acc, k_other, k_diag;
};

struct Place {
    int e, row0, rows, n, col0;  // matrix, first row, rows, the MMA's N, first column
};

// Walks tiles first, first + step, .. of all matrices, the column tile innermost.  SYM: of a row
// tile only the column tiles that begin at its last row or before.  (The lower triangle: the last
// row tile may be short, and then takes fewer of the MMA's N, where a short column tile takes
// all of its M, so few tiles should be of the last columns.)  The order is the matrices', for L2:
// with all short row tiles last, which deals them evenly, five steps of 32 x 1408 x 2048 took
// 2077 us for 1998.
template <bool SYM>
struct Walk {
    const ProductArgs &p;
    int tile, step, e = 0, r = 0, c;
    __device__ __forceinline__ Walk(const ProductArgs &args, int first, int by) : p(args), tile(first), step(by), c(first) { settle(); }
    __device__ __forceinline__ int reach() const {
        return SYM ? ((min(p.R, (r + 1) * p.tile_rows) - 1) >> p.col_shift) + 1 : p.col_tiles;
    }
    __device__ __forceinline__ void settle() {
        if (!SYM) {
            const int per = p.row_tiles * p.col_tiles;
            if (c >= per) {  // a matrix or more on
                const int n = c / per;
                e += n;
                c -= n * per;
            }
        }
        for (int here = reach(); c >= here; here = reach()) {
            c -= here;
            if (++r == p.row_tiles) {
                r = 0;
                ++e;
            }
        }
    }
    __device__ __forceinline__ bool more() const { return tile < p.tiles; }
    __device__ __forceinline__ void next() {
        tile += step;
        c += step;
        if (more()) settle();
    }
    __device__ __forceinline__ Place get() const {
        const int row0 = r * p.tile_rows, rows = min(p.tile_rows, p.R - row0);
        return {e, row0, rows, (rows + 31) & ~31, c * p.cols};
    }
};

// 16 fp16 values at a 32-byte boundary
struct Half16 {
    uint32_t w[8];
};
__device__ __forceinline__ Half16 load_half16(const half *p) {
    Half16 v;
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ void store_half16(half *p, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                 "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
                 : "memory");
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t v) { return __half22float2(*reinterpret_cast<const half2 *>(&v)); }

// The epilogues, by one warp for its chunks of 32 columns (lanes) x 32 rows (TMEM columns).  What
// a chunk reads from memory is asked for a chunk ahead (fetch), the first before the sums are there; with
// four warps per lane quadrant (two: five steps of 32 x 1408 x 2048 took 2277 us for 2178).

// A symmetric result (A, or B from A): v = f (k_acc sum + k_other other + k_diag on the diagonal),
// f: s^2 for A, s for B.  Element (r, c) with c <= r is stored there and at (c, r), 32 bytes of a lane's
// column at a time; `other` is read in its mirror image too.  A chunk on the diagonal holds its own
// mirror image (the same products summed in the same order) and is stored once.
struct Symmetric {
    const ProductArgs &p;
    int lane;
    Half16 ahead[2];
    __device__ __forceinline__ void fetch(const Place &t, int col, int c) {
        const int rows = col < p.C && p.other != nullptr && col - lane <= t.row0 + c ? t.rows - c : 0;
        const half *o = p.other + ((size_t)t.e * p.R + col) * p.ld + t.row0 + c;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (16 * i < rows) {
                ahead[i] = load_half16(o + 16 * i);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) ahead[i].w[j] = 0u;
            }
        }
    }
    __device__ __forceinline__ void finish(const Place &t, uint32_t tcol, int col, int c, int next) {
        const size_t ld = p.ld, base = (size_t)t.e * p.R * ld;
        const bool ok = col < p.C;
        const int col_first = col - lane, r0 = t.row0 + c, rows = min(32, t.rows - c);  // a multiple of 8, as all sizes are
        Half16 a[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) a[i] = ahead[i];
        if (next < t.rows) fetch(t, col, next);
        if (col_first > r0) return;  // above the diagonal (both are multiples of 32)
        float f = 1.0f;
        if (p.table != nullptr) {
            const float s = p.table[t.e];
            f = p.other != nullptr ? s : s * s;
        }
        uint32_t v[32];
        tmem_ld32(tcol + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));  // not read before the wait
        const int diagonal = col_first == r0 ? lane : -1;  // its row
        uint32_t h[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 o = unpack_half2(a[i / 8].w[i % 8]);
            float x = fmaf(p.k_other, o.x, p.k_acc * __uint_as_float(v[2 * i]));
            float y = fmaf(p.k_other, o.y, p.k_acc * __uint_as_float(v[2 * i + 1]));
            if (2 * i == diagonal) x += p.k_diag;
            if (2 * i + 1 == diagonal) y += p.k_diag;
            h[i] = pack_half2(f * x, f * y);
        }
        if (ok && col_first < r0) {  // (the last 16 values may reach into the rows' padding)
            half *across = p.out + base + (size_t)col * ld + r0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (16 * i < rows) store_half16(across + 16 * i, h + 8 * i);
        }
        // both columns of a lane pair in one word, rows 2i (even lane) and 2i + 1
        const int odd = lane & 1;
        uint32_t *o = reinterpret_cast<uint32_t *>(p.out + base + (size_t)(r0 + odd) * ld + (col & ~1));
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, h[i], 1);
            if (ok && 2 * i < rows) o[i * ld] = __byte_perm(h[i], got, odd ? 0x3276 : 0x5410);
        }
    }
};

// X: v = k_acc sum + f k_other lo, f: s in the first step; stored as hi (and lo, in place of the old one), or as bf16 at the
// end.  Lane pairs exchange values so that each lane has both columns of every other row, one word.
struct Update {
    const ProductArgs &p;
    int lane;
    uint32_t ahead[16];
    __device__ __forceinline__ size_t at(const Place &t, int col, int c) const {
        return ((size_t)t.e * p.R + t.row0 + c + (lane & 1)) * p.C + (col & ~1);
    }
    __device__ __forceinline__ void fetch(const Place &t, int col, int c) {
        const int left = col < p.C && p.other != nullptr ? t.rows - c - (lane & 1) : 0;
        const uint32_t *o = reinterpret_cast<const uint32_t *>(p.other + at(t, col, c));
#pragma unroll
        for (int i = 0; i < 16; ++i) ahead[i] = 2 * i < left ? o[(size_t)i * p.C] : 0u;
    }
    __device__ __forceinline__ void finish(const Place &t, uint32_t tcol, int col, int c, int next) {
        const int odd = lane & 1, left = col < p.C ? t.rows - c - odd : 0;
        const size_t ld = p.C, from = at(t, col, c);
        const float scale = p.table != nullptr ? p.k_other * p.table[t.e] : p.k_other;
        uint32_t lo[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) lo[i] = ahead[i];
        if (next < t.rows) fetch(t, col, next);
        uint32_t v[32];
        tmem_ld32(tcol + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));  // not read before the wait
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t mine = odd ? v[2 * i + 1] : v[2 * i], give = odd ? v[2 * i] : v[2 * i + 1];
            const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
            const float2 old = unpack_half2(lo[i]);
            const float x = fmaf(scale, old.x, p.k_acc * __uint_as_float(odd ? got : mine));
            const float y = fmaf(scale, old.y, p.k_acc * __uint_as_float(odd ? mine : got));
            if (2 * i >= left) continue;
            if (p.final != nullptr) {
                *reinterpret_cast<uint32_t *>(p.final + from + 2 * i * ld) = pack_bf16x2(p.scale * x, p.scale * y);
            } else {
                const uint32_t h = pack_half2(x, y);
                *reinterpret_cast<uint32_t *>(p.out + from + 2 * i * ld) = h;
                if (p.out_lo != nullptr) {
                    const float2 b = unpack_half2(h);
                    *reinterpret_cast<uint32_t *>(p.out_lo + from + 2 * i * ld) = pack_half2(x - b.x, y - b.y);
                }
            }
        }
    }
};

__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr) {  // as grouped_kernel.cuh
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(kChunk >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// A_MN, B_MN: the operand of the columns, of the rows, has its reduction index outermost.
template <bool A_MN, bool B_MN, bool SYM, bool SMALL>
__global__ void __launch_bounds__(kThreads<SMALL>, SMALL ? 2 : 1) product_kernel(const __grid_constant__ ProductArgs p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Header &h = *reinterpret_cast<Header *>(smem);
    const uint32_t base = smem_u32(smem) + kHeaderBytes;
    const int a_block = p.a_block, b_block = p.b_block, stages = p.stages;
    // all A blocks first: the MMA reads 128 columns of A where the box brought 64; the rest is
    // whatever follows, and its results are not stored
    const uint32_t sA = base, sB = base + (uint32_t)(stages * a_block);
    const uint32_t bar0 = smem_u32(h.bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * kMaxStages + a); };
    auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * kMaxStages + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * kMaxStages + 4);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = rank == 0;
    volatile int *abort_flag = &h.abort;
    auto raise = [&]() {  // stops both CTAs' roles
        atomicOr(p.err, ERR_TIMEOUT);
        *abort_flag = 1;
        st_cluster_s32(mapa_shared(smem_u32(const_cast<int *>(&h.abort)), (uint32_t)rank ^ 1u), 1);
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (uint32_t a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 2 * kEpiWarps<SMALL>);  // both CTAs'
        }
        mbar_init(drain_bar, 1);
        fence_mbar_init();
        h.abort = 0;
        tma_prefetch_desc(&p.map_a);
        tma_prefetch_desc(&p.map_b);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&h.tmem), 2 * kAccCols<SMALL>);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any copy or arrival crosses over
    tc_fence_after();
    const uint32_t tmem_base = h.tmem;
    pdl_wait();  // the operands, by earlier kernels on the stream
    pdl_trigger();
    const int first = (int)blockIdx.x / 2, stride = (int)gridDim.x / 2;
    const int half_cols = p.cols / 2;

    if (warp == 0) {
        // a short tile is loaded as a whole one: what comes beyond its rows is not multiplied
        const bool two_b = p.tile_rows / 2 > 64;
        const uint32_t bytes = a_block + (B_MN ? (two_b ? 2 : 1) * kChunk : (p.tile_rows / 2) * kRow);
        uint32_t ph = 1;
        int s = 0;
        bool ok = true;
        for (Walk<SYM> walk(p, first, stride); ok && walk.more(); walk.next()) {
            const Place t = walk.get();
            const int col = t.col0 + rank * half_cols, row = t.row0 + rank * (t.n / 2);
            for (int r = 0; r < p.red; r += kBK) {
                if (!__all_sync(0xffffffffu, wait_bar(empty_bar(s), ph, p.wait, abort_flag))) {
                    ok = false;
                    break;
                }
                const uint32_t da = sA + s * a_block, db = sB + s * b_block, bar = mapa_shared(full_bar(s), 0);
                if (elect_one()) {
                    if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * bytes);
                    if (A_MN) {
                        tma_load_3d_pair(da, &p.map_a, bar, col, r, t.e);
                        if (half_cols > 64) tma_load_3d_pair(da + kChunk, &p.map_a, bar, col + 64, r, t.e);
                    } else {
                        tma_load_3d_pair(da, &p.map_a, bar, r, col, t.e);
                    }
                    if (B_MN) {
                        tma_load_3d_pair(db, &p.map_b, bar, row, r, t.e);
                        if (two_b) tma_load_3d_pair(db + kChunk, &p.map_b, bar, row + 64, r, t.e);
                    } else {
                        tma_load_3d_pair(db, &p.map_b, bar, r, row, t.e);
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
            constexpr uint32_t kStepA = A_MN ? (16 * kRow) >> 4 : 2;  // 16 reduction steps on,
            constexpr uint32_t kStepB = B_MN ? (16 * kRow) >> 4 : 2;  // in units of 16 bytes
            const uint64_t desc_a = A_MN ? smem_desc_mn(sA) : smem_desc_k128(sA);
            const uint64_t desc_b = B_MN ? smem_desc_mn(sB) : smem_desc_k128(sB);
            // fp16 operands (their format fields are 0), fp32 sums
            constexpr uint32_t kDesc = (1u << 4) | (256u >> 4) << 24 | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
            uint32_t ph = 0, acc = 0, free_ph = 1;
            int s = 0;
            bool ok = p.wait != 0, issued = false;  // a bound of 0: give up at once
            for (Walk<SYM> walk(p, first, stride); ok && walk.more(); walk.next()) {
                const uint32_t idesc = kDesc | (uint32_t)(walk.get().n >> 3) << 17;
                const uint32_t d = tmem_base + acc * kAccCols<SMALL>;
                if (!__all_sync(0xffffffffu, wait_bar<true>(tempty_bar(acc), free_ph, p.wait, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int r = 0; r < p.red; r += kBK) {
                    if (!__all_sync(0xffffffffu, wait_bar(full_bar(s), ph, p.wait, abort_flag))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = desc_a + (uint32_t)(s * a_block >> 4), bd = desc_b + (uint32_t)(s * b_block >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k)
                            tc_mma_bf16_pair(d, ad + k * kStepA, bd + k * kStepB, idesc, (r + k) != 0);
                        tc_commit_pair(empty_bar(s), 3);  // frees the stage in both CTAs
                        if (r + kBK >= p.red) tc_commit_pair(tfull_bar(acc), 3);
                    }
                    __syncwarp();
                    issued = true;
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                acc ^= 1u;
                if (acc == 0) free_ph ^= 1u;
            }
            if (!ok && lane == 0) {
                raise();
                if (issued) {
                    tc_commit_pair(drain_bar, 1);
                    wait_bar(drain_bar, 0, kDrainCycles, nullptr);
                }
            }
        }
    } else {
        const int q = warp & 3;  // the TMEM lane quadrant this warp may read
        const int part = (warp - 2) >> 2;
        const bool mine = 32 * q < half_cols;
        uint32_t acc = 0, ph = 0;
        typename std::conditional<SYM, Symmetric, Update>::type epilogue{p, lane};
        for (Walk<SYM> walk(p, first, stride); walk.more(); walk.next()) {
            const Place t = walk.get();
            const uint32_t tcol = tmem_base + ((uint32_t)(q * 32) << 16) + acc * kAccCols<SMALL>;
            const int col = t.col0 + rank * half_cols + 32 * q + lane;
            if (mine && 32 * part < t.rows) epilogue.fetch(t, col, 32 * part);
            if (!__all_sync(0xffffffffu, wait_bar<true>(tfull_bar(acc), ph, p.wait, abort_flag))) {
                if (lane == 0) raise();
                break;
            }
            tc_fence_after();
            if (mine)
                for (int c = 32 * part; c < t.rows; c += 32 * kParts<SMALL>) epilogue.finish(t, tcol, col, c, c + 32 * kParts<SMALL>);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(mapa_shared(tempty_bar(acc), 0));
            acc ^= 1u;
            if (acc == 0) ph ^= 1u;
        }
    }

    leave_pair(abort_flag);
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 2 * kAccCols<SMALL>);
    }
}

// ------------------------------------------------------------------ |G|, X0

constexpr int kNormThreads = 256;
constexpr int kPerThread = 32;                       // values of a thread
constexpr int kBlock = kNormThreads * kPerThread;    // values of a CTA: one matrix's, in turn

// 8 values from p, as loaded
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&o)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float *p, float (&o)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<bf16>(const bf16 *p, float (&o)[8]) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    o[0] = bf16_lo(v.x), o[1] = bf16_hi(v.x), o[2] = bf16_lo(v.y), o[3] = bf16_hi(v.y);
    o[4] = bf16_lo(v.z), o[5] = bf16_hi(v.z), o[6] = bf16_lo(v.w), o[7] = bf16_hi(v.w);
}

// Sum over the CTA, in thread 0 alone.
__device__ __forceinline__ double cta_sum(double v, double *shared) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < kNormThreads / 32; ++w) v += shared[w];
    return v;
}

// Squares of a part of one matrix: a thread's 32 in fp32, the rest in fp64 (squares outside
// [1e-30, 1e30] in sum are taken again in fp64).
template <typename T>
__global__ void __launch_bounds__(kNormThreads) square_kernel(const T *g, long long size, int parts, double *partial) {
    __shared__ double shared[kNormThreads / 32];
    const int e = blockIdx.x / parts, part = blockIdx.x - e * parts;
    pdl_wait();
    pdl_trigger();
    const T *at = g + (size_t)e * size;
    double sum = 0.0;
    for (long long i = (long long)part * kBlock + 8 * threadIdx.x; i < size; i += (long long)parts * kBlock) {
        float s = 0.0f, most = 0.0f, v[8];
#pragma unroll
        for (int j = 0; j < kPerThread / 8; ++j) {
            const long long k = i + (long long)j * 8 * kNormThreads;
            if (k >= size) break;
            load8(at + k, v);
#pragma unroll
            for (int x = 0; x < 8; ++x) s = fmaf(v[x], v[x], s), most = fmaxf(most, fabsf(v[x]));
        }
        if ((s > 1e-30f && s < 1e30f) || most == 0.0f) {  // (a NaN beside zeros is in s)
            sum += s;
        } else {
            for (int j = 0; j < kPerThread / 8; ++j) {
                const long long k = i + (long long)j * 8 * kNormThreads;
                if (k >= size) break;
                load8(at + k, v);
                for (int x = 0; x < 8; ++x) sum += (double)v[x] * v[x];
            }
        }
    }
    sum = cta_sum(sum, shared);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// table[e] = s = 2^k / (|G| + eps) with 2^k <= |G| + eps < 2^(k + 1); X0 = up 2^-k G, as hi and, where lo
// is not NULL, lo.  Each CTA adds up its matrix's sums.  The matrices come in reverse order, so
// that what was read last is still in L2.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) scale_kernel(const T *g, long long size, int parts, const double *partial,
                                                             float eps, float up, float *table, half *x, half *lo) {
    __shared__ double shared[kNormThreads / 32];
    __shared__ float shrink_of;
    const int block = gridDim.x - 1 - blockIdx.x, e = block / parts, part = block - e * parts;
    pdl_wait();
    pdl_trigger();
    double v = 0.0;
    for (int i = threadIdx.x; i < parts; i += kNormThreads) v += partial[e * parts + i];
    v = cta_sum(v, shared);
    if (threadIdx.x == 0) {
        const double norm = sqrt(v) + (double)eps;
        float s = nanf(""), shrink = 1.0f;  // an infinity or a NaN: all of the result is NaN
        if (norm < INFINITY) {
            int k;
            s = (float)(1.0 / (2.0 * frexp(norm, &k)));
            shrink = (float)ldexp(1.0, 1 - k);
        }
        shrink_of = shrink;
        if (part == 0) table[e] = s;
    }
    __syncthreads();
    const float shrink = shrink_of;
    const T *at = g + (size_t)e * size;
    half *to = x + (size_t)e * size;
    for (long long i = (long long)part * kBlock + 8 * threadIdx.x; i < size; i += (long long)parts * kBlock) {
#pragma unroll
        for (int j = 0; j < kPerThread / 8; ++j) {
            const long long k = i + (long long)j * 8 * kNormThreads;
            if (k >= size) break;
            float o[8];
            load8(at + k, o);
#pragma unroll
            for (int x8 = 0; x8 < 8; ++x8) o[x8] = o[x8] * shrink * up;
            const uint4 hi = make_uint4(pack_half2(o[0], o[1]), pack_half2(o[2], o[3]), pack_half2(o[4], o[5]), pack_half2(o[6], o[7]));
            *reinterpret_cast<uint4 *>(to + k) = hi;
            if (lo == nullptr) continue;
            uint32_t l[4];
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
                const float2 h = unpack_half2((&hi.x)[i4]);
                l[i4] = pack_half2(o[2 * i4] - h.x, o[2 * i4 + 1] - h.y);
            }
            *reinterpret_cast<uint4 *>(lo + (size_t)e * size + k) = make_uint4(l[0], l[1], l[2], l[3]);
        }
    }
}

// ---------------------------------------------------------------------- host

OpDone g_attr[8];

constexpr int kMaxSteps = 64;
// CTAs of a matrix in the two kernels above: about 2048 in all, each with a block of values at least
// (with at most 64 a matrix, 2048 x 2048 in fp32 took 18 and 23 us)
int parts_of(int E, long long size) { return (int)std::min<long long>(std::max(1, 2048 / std::max(1, E)), (size + kBlock - 1) / kBlock); }

// Offsets from the workspace rounded up to kRoom bytes: the rows of A and B are read and written 32
// bytes at a time, and callers' workspaces are only sure to begin at 16.
constexpr size_t kRoom = 1024;
struct Workspace {
    size_t table, partial, x[2], lo, a, b, bytes;
};
int padded(int m) { return (m + 15) / 16 * 16; }  // rows of A and B begin at 32-byte boundaries
Workspace lay_out(int E, int N, int K) {
    const size_t n = (size_t)N * K, m = std::min(N, K), e = E;
    auto room = [](size_t bytes) { return (bytes + kRoom - 1) / kRoom * kRoom; };
    Workspace w;
    w.table = 0;
    w.partial = w.table + room(e * sizeof(float));
    w.x[0] = w.partial + room(e * parts_of(E, (long long)n) * sizeof(double));
    w.x[1] = w.x[0] + room(2 * e * n);
    w.lo = w.x[1] + room(2 * e * n);
    w.a = w.lo + room(2 * e * n);
    w.b = w.a + room(2 * e * m * padded((int)m));
    w.bytes = w.b + room(2 * e * m * padded((int)m)) + kRoom - 16;  // and what rounding up may take
    return w;
}

// Scales of one step's A and B, and of X: powers of two that keep what is stored below 60000.
struct Scales {
    float a, b;
};
// Samples of a polynomial of degree 5: between two of them it rises by at most 100 / kSamples^2 of
// its largest value (its second derivative is at most 800 / limit^2 of that, by Markov's inequality)
constexpr int kSamples = 128;
double largest(double limit, double (*of)(double, const float *), const float *c) {
    double most = 0.0;
    for (int i = 0; i <= kSamples; ++i) most = std::max(most, std::fabs(of(limit * i / kSamples, c)));
    return 1.01 * most;
}
float power_below(double bound, int most) {
    return (float)std::ldexp(1.0, std::min(most, std::ilogb(60000.0 / std::max(bound, 1e-6))));
}
// Steps whose X keeps its rounding.
bool keeps_lo(int step, int steps) { return step < steps - 2; }

// Largest singular values and polynomials that fp16 holds beside others: X's scale is one for all steps.
constexpr double kMostValue = 1024.0, kLeastValue = 1.0 / 1024.0;
// false: the polynomials let the singular values grow beyond that, or all of them shrink
bool choose_scales(const float *coef, int steps, Scales *scales, float *up) {
    double x = 1.0, most = 1.0;
    for (int i = 0; i < steps; ++i) {
        const float *c = coef + 3 * i;
        auto whole = [](double l, const float *k) { return k[0] + l * (k[1] + l * k[2]); };
        auto step = [](double v, const float *k) { return v * (k[0] + v * v * (k[1] + v * v * k[2])); };
        scales[i].a = power_below(1.01 * x * x, 14);
        const double b = largest(x * x, whole, c);
        scales[i].b = power_below(b, 14);
        x = largest(x, step, c);
        if (!(x < kMostValue && b > kLeastValue)) return false;
        if (i + 1 == steps) break;
        if (!(x > kLeastValue)) return false;
        most = std::max(most, x);
    }
    *up = power_below(1.01 * most, 12);
    return true;
}

// Tile sizes: 256 columns (128 where there are no more) and 32 to 256 rows, dealt evenly to a
// matrix's tiles in multiples of 32 (the pair's MMA takes N in steps of 32); what takes the least
// time by: waves of tiles times a tile's stages, each 150 + 0.6 ns for each row (the copies of 128
// columns and half of the rows to an SM at 110 bytes a ns, or as long for the MMAs), 600 ns to fill
// the pipeline, and at the end an epilogue.  (256 rows, halved while the pairs outnumber the tiles: 4096
// x 4096 1012 us for 874, 2 x 1408 x 2048 270 for 241, 4 x 1024 x 1024 188 for 175.)
long long count_tiles(const ProductArgs &g, bool sym) {
    if (!sym) return (long long)g.E * g.row_tiles * g.col_tiles;
    long long n = 0;
    for (int r = 0; r < g.row_tiles; ++r) n += (std::min(g.R, (r + 1) * g.tile_rows) - 1) / g.cols + 1;
    return n * g.E;
}
long long choose_tiles(ProductArgs &g, bool b_mn, bool sym, int sms) {
    g.cols = g.C > 128 ? 256 : 128;
    g.col_shift = g.cols == 256 ? 8 : 7;
    g.col_tiles = (g.C + g.cols - 1) / g.cols;
    const long long pairs = sms / 2;
    long long tiles = 0;
    double least = 0.0;
    int best = 0;
    for (int rows = 256; rows >= 32; rows -= 32) {
        const int parts = (g.R + rows - 1) / rows;
        const int share = ((g.R + parts - 1) / parts + 31) / 32 * 32;
        if (share != rows && rows < 256) continue;  // the same as a size before
        g.tile_rows = share;
        g.row_tiles = (g.R + share - 1) / share;
        const long long waves = (count_tiles(g, sym) + pairs - 1) / pairs;
        const double cost = waves * ((g.red + kBK - 1) / kBK * (150 + 0.6 * share) + 600) + 8.0 * share;
        if (best == 0 || cost < least) best = share, least = cost;
    }
    g.tile_rows = best;
    g.row_tiles = (g.R + best - 1) / best;
    tiles = count_tiles(g, sym);
    g.a_block = g.cols / 2 * kRow;
    g.b_block = b_mn ? (g.tile_rows / 2 + 63) / 64 * kChunk : g.tile_rows / 2 * kRow;
    return tiles;
}

// An operand [E, outer, inner] of fp16, ld elements from row to row; `mn`: its reduction index is the outer one.
struct Operand {
    const half *p;
    int outer, inner, ld;
};
CUresult operand_map(CUtensorMap *m, const Operand &o, int E, bool mn, int box) {
    return op_encode(m, {CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, o.p, {(uint64_t)o.inner, (uint64_t)o.outer, (uint64_t)E},
                         {(uint64_t)o.ld * 2, (uint64_t)o.ld * o.outer * 2}, {64, mn ? (uint32_t)kBK : (uint32_t)box, 1},
                         CU_TENSOR_MAP_SWIZZLE_128B});
}

// A product's kernel and arguments but what changes from step to step.
struct Product {
    ProductArgs g;
    void (*kernel)(const ProductArgs);
    int grid, threads, smem;
};
template <bool A_MN, bool B_MN, bool SYM>
moe_status plan(const char *name, Product &p, const Operand &a, const Operand &b, int which, int sms) {
    ProductArgs &g = p.g;
    const long long tiles = choose_tiles(g, B_MN, SYM, sms);
    g.tiles = (int)tiles;  // at most 65535 * 64^2
    g.wait = wait_cycles(g.red / kBK + 1);
    p.grid = 2 * (int)std::min<long long>(sms / 2, tiles);
    const bool small = tiles <= sms / 2 && g.tile_rows <= 128;
    p.kernel = small ? product_kernel<A_MN, B_MN, SYM, true> : product_kernel<A_MN, B_MN, SYM, false>;
    p.threads = small ? kThreads<true> : kThreads<false>;
    p.smem = small ? kSmemBytes<true> : kSmemBytes<false>;
    g.stages = std::min(kMaxStages, (p.smem - kHeaderBytes) / (g.a_block + g.b_block));
    CUresult cr = operand_map(&g.map_a, a, g.E, A_MN, g.cols / 2);
    if (cr == CUDA_SUCCESS) cr = operand_map(&g.map_b, b, g.E, B_MN, g.tile_rows / 2);
    if (cr != CUDA_SUCCESS) return op_fail(MOE_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", name, (int)cr);
    return op_cuda(op_allow_smem(reinterpret_cast<const void *>(p.kernel), p.smem, &g_attr[2 * which + small]), name);
}
cudaError_t launch(const Product &p, cudaStream_t s) {
    return launch_pdl_cluster(p.kernel, dim3(p.grid), dim3(p.threads), (size_t)p.smem, s, dim3(2, 1, 1), p.g);
}

moe_status check_sizes(const char *name, int E, int N, int K) {
    if (E < 0 || N < 1 || K < 1) return op_fail(MOE_ERR_INVALID_ARG, "%s: need E >= 0, N >= 1, K >= 1", name);
    if (E > 65535 || N % 8 || K % 8 || N > kMaxSide || K > kMaxSide)
        return op_fail(MOE_ERR_UNSUPPORTED, "%s: E up to 65535, N and K multiples of 8 up to %d (E %d, N %d, K %d)", name,
                       kMaxSide, E, N, K);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_orthogonalize_workspace(int E, int N, int K, size_t *bytes) {
    using namespace moe;
    const char *name = "moe_orthogonalize_workspace";
    const moe_status st = check_sizes(name, E, N, K);
    if (st != MOE_OK) return st;
    if (bytes == nullptr) return op_fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer", name);
    *bytes = lay_out(E, N, K).bytes;
    return MOE_OK;
}

extern "C" moe_status moe_orthogonalize(const void *G, int dtype, int E, int N, int K, const float *coefficients, int steps,
                                        float eps, float scale, void *out, void *workspace, size_t workspace_bytes,
                                        moe_stream_t stream) {
    using namespace moe;
    const char *name = "moe_orthogonalize";
    moe_status st = check_sizes(name, E, N, K);
    if (st != MOE_OK) return st;
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32) return op_fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype %d", name, dtype);
    if (steps < 1 || steps > kMaxSteps || coefficients == nullptr)
        return op_fail(MOE_ERR_INVALID_ARG, "%s: need 1 to %d steps and their coefficients", name, kMaxSteps);
    for (int i = 0; i < 3 * steps; ++i)
        if (!(coefficients[i] - coefficients[i] == 0.0f)) return op_fail(MOE_ERR_INVALID_ARG, "%s: coefficients must be finite", name);
    if (!(eps >= 1e-30f && eps < INFINITY) || !(scale - scale == 0.0f))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: need eps >= 1e-30 and a finite scale", name);
    Scales scales[kMaxSteps];
    float up;
    if (!choose_scales(coefficients, steps, scales, &up))
        return op_fail(MOE_ERR_UNSUPPORTED, "%s: these coefficients let singular values grow beyond 1024, or all of them shrink below 1 / 1024", name);
    if (E == 0) return MOE_OK;
    const Workspace w = lay_out(E, N, K);
    if (!G || !out || !workspace || workspace_bytes < w.bytes)
        return op_fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer, or less than %zu bytes of workspace", name, w.bytes);
    if (!op_aligned16(G) || !op_aligned16(out) || !op_aligned16(workspace))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", name);
    const uint64_t n = (uint64_t)E * N * K, gb = n * (dtype == MOE_DTYPE_F32 ? 4 : 2);
    const bool in_place = out == G && dtype == MOE_DTYPE_BF16;
    if ((op_overlap(out, 2 * n, G, gb) && !in_place) || op_overlap(workspace, w.bytes, G, gb) || op_overlap(workspace, w.bytes, out, 2 * n))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: the output or the workspace overlaps another tensor", name);
    const int sms = op_num_sms();
    int *err = op_error_word();
    if (sms < 2 || err == nullptr) return op_fail(MOE_ERR_CUDA, "%s: no usable current device", name);

    uint8_t *ws = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(workspace) + kRoom - 1) / kRoom * kRoom);
    float *table = reinterpret_cast<float *>(ws + w.table);
    double *partial = reinterpret_cast<double *>(ws + w.partial);
    half *x[2] = {reinterpret_cast<half *>(ws + w.x[0]), reinterpret_cast<half *>(ws + w.x[1])};
    half *lo = reinterpret_cast<half *>(ws + w.lo), *A = reinterpret_cast<half *>(ws + w.a), *B = reinterpret_cast<half *>(ws + w.b);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // the products, by the buffer that X is in, before anything is launched
    const bool wide = N <= K;
    const int m = std::min(N, K), ld = padded(m);
    Product gram[2] = {}, poly = {}, update[2] = {};
    const Operand sym_a{A, m, m, ld}, sym_b{B, m, m, ld};
    poly.g.E = E, poly.g.R = poly.g.C = poly.g.red = m, poly.g.ld = ld, poly.g.err = err;
    poly.g.other = A, poly.g.out = B;
    st = plan<false, false, true>(name, poly, sym_a, sym_a, 0, sms);
    for (int i = 0; i < 2 && st == MOE_OK; ++i) {
        const Operand X{x[i], N, K, K};
        ProductArgs &a = gram[i].g, &u = update[i].g;
        a.E = E, a.R = a.C = m, a.ld = ld, a.red = wide ? K : N, a.err = err, a.out = A;
        u.E = E, u.R = N, u.C = K, u.red = m, u.err = err, u.out = x[i ^ 1];
        st = wide ? plan<false, false, true>(name, gram[i], X, X, 0, sms) : plan<true, true, true>(name, gram[i], X, X, 1, sms);
        if (st != MOE_OK) break;
        st = wide ? plan<true, false, false>(name, update[i], X, sym_b, 2, sms) : plan<false, false, false>(name, update[i], sym_b, X, 3, sms);
    }
    if (st != MOE_OK) return st;

    const long long size = (long long)N * K;
    const int parts = parts_of(E, size);
    const dim3 grid((unsigned)(E * parts));
    // X0 of bf16 values is exact
    half *lo0 = dtype == MOE_DTYPE_F32 && keeps_lo(0, steps) ? lo : nullptr;
    cudaError_t ce;
    if (dtype == MOE_DTYPE_F32) {
        const float *g = static_cast<const float *>(G);
        ce = launch_pdl(square_kernel<float>, grid, dim3(kNormThreads), 0, s, g, size, parts, partial);
        if (ce == cudaSuccess)
            ce = launch_pdl(scale_kernel<float>, grid, dim3(kNormThreads), 0, s, g, size, parts, static_cast<const double *>(partial), eps, up, table, x[0], lo0);
    } else {
        const bf16 *g = static_cast<const bf16 *>(G);
        ce = launch_pdl(square_kernel<bf16>, grid, dim3(kNormThreads), 0, s, g, size, parts, partial);
        if (ce == cudaSuccess)
            ce = launch_pdl(scale_kernel<bf16>, grid, dim3(kNormThreads), 0, s, g, size, parts, static_cast<const double *>(partial), eps, up, table, x[0], lo0);
    }
    if (ce != cudaSuccess) return op_cuda(ce, name);

    for (int i = 0; i < steps; ++i) {
        const float *c = coefficients + 3 * i, sa = scales[i].a, sb = scales[i].b;
        ProductArgs &a = gram[i & 1].g, &b = poly.g, &u = update[i & 1].g;
        a.table = b.table = u.table = i == 0 ? table : nullptr;
        a.k_acc = sa / (up * up);
        b.k_acc = c[2] / sa / sa * sb;
        b.k_other = c[1] / sa * sb;
        b.k_diag = c[0] * sb;
        const bool last = i + 1 == steps;
        u.k_acc = 1.0f / sb / (last ? up : 1.0f);  // a power of two; `scale`, of any size, comes after it
        u.scale = scale;
        u.other = i == 0 ? lo0 : keeps_lo(i, steps) ? lo : nullptr;
        u.k_other = c[0];  // (the last step has no lo)
        u.out_lo = !last && keeps_lo(i + 1, steps) ? lo : nullptr;
        u.final = last ? static_cast<bf16 *>(out) : nullptr;
        ce = launch(gram[i & 1], s);
        if (ce == cudaSuccess) ce = launch(poly, s);
        if (ce == cudaSuccess) ce = launch(update[i & 1], s);
        if (ce != cudaSuccess) return op_cuda(ce, name);
    }
    return MOE_OK;
}
