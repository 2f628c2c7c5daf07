// Grouped product with both operands in MXFP4: rows grouped by expert (grouped.cuh),
//   Y[r, n] = sum_b 2^(xs[b, r] + ws[e, b, n] - 254) sum_{i in block b} x[r, i] w[e, n, i]
// x, w: E2M1 values, blocks b of 32 along K, one scale byte each.  The block-scaled tensor
// instruction (tcgen05.mma kind::mxf4, K = 64) multiplies the packed codes and applies both
// scales as it accumulates in fp32: nothing is decoded, so a k-step of 256 values is 128
// bytes of codes per row, a quarter of bf16's.
//
// Persistent kernel, 14 warps:
//   warp 0      TMA producer: codes of bm token rows and bn weight rows, 256 values
//               (128 bytes, 128-byte swizzle) per stage
//   warp 1      allocates tensor memory; copies a stage's scales from shared to tensor
//               memory (tcgen05.cp, in order with the MMAs that follow) and issues the MMAs
//   warps 2-5   epilogue (grouped.cuh), overlapping the next tile's main loop
//   warps 6-13  scales, two sets of four warps taking alternate stages.  The tensor core
//               wants four consecutive blocks' scales of a row in one word, the tensors hold a
//               block's scales for consecutive rows: the warps read runs along the rows,
//               transpose in registers and write the words where tcgen05.cp reads them.  A
//               set's loads for its next stage are in flight while it waits to store this one.
// Tensor memory (512 columns): two accumulators of bn columns, then per stage the scales of
// the tokens (8 columns) and of the weights (8 per 128 of them).
#include <algorithm>

#include "common.cuh"
#include "grouped.cuh"
#include "kernels.h"
#include "moe.h"
#include "op_host.h"

namespace moe {
namespace {

constexpr int kBK = 256;           // values per stage: 128 bytes of codes
constexpr int kBlocks = kBK / 32;  // scale blocks per stage
constexpr int kMaxStages = 12;
constexpr int kScaleSets = 2;
constexpr int kThreads = 64 + 32 * kEpiWarps + 128 * kScaleSets;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxBn = 192;
constexpr int kScaleStage = 1024 + 2048;  // tokens' and weights' scale words of a stage
constexpr int kStageSpace = 196608;
constexpr int kSmemBytes = kStageSpace + kEpiBytes + 1024 /* alignment */;

struct MxGroupedArgs {
    CUtensorMap map_a, map_b;
    GroupedOut o;
    const uint8_t *xs, *ws;  // [K / 32, rows], [E, K / 32, N]
    int stages;
};

// Instruction descriptor of kind::mxf4: E2M1 operands (bits 7-9 and 10-11 = 1), N >> 3 at bits
// 17-22, scales UE8M0 (bit 23), M >> 4 at bits 24-28; which half of a scale word a K step of 64
// uses: bits 29-30 (A) and 4-5 (B).
__device__ __forceinline__ uint32_t idesc_mxf4(int M, int N) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// 512 bytes of shared memory (32 lanes x 16 bytes) to four columns of tensor memory, the same
// in each of its four lane quadrants
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint32_t saddr) {
    // no swizzle; 8-lane groups of 16-byte rows 128 bytes apart
    const uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// One scale thread's share of a stage, between its loads and its stores.
struct Scales {
    uint32_t a[2];  // its token row's words (blocks 0-3, 4-7)
    uint32_t b[4];  // four weight rows' bytes of four blocks
};

__global__ void __launch_bounds__(kThreads, 1) mx_grouped_kernel(const __grid_constant__ MxGroupedArgs p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t s_bars[3 * kMaxStages + 5];
    __shared__ int s_offs[kMaxExperts + 1], s_tiles[kMaxExperts + 1];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int bn = p.o.bn, atoms = (bn + 127) / 128;  // 128-row groups of weight scales
    const int a_stage = p.o.bm * 128, b_stage = bn * 128;
    const uint32_t sA = base, sB = base + (uint32_t)(p.stages * a_stage), sS = sB + (uint32_t)(p.stages * b_stage),
                   sE = base + kStageSpace;
    const uint32_t bar0 = smem_u32(s_bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto scale_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    auto empty_bar = [&](int s) { return bar0 + 8u * (2 * kMaxStages + s); };
    auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (3 * kMaxStages + a); };
    auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (3 * kMaxStages + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (3 * kMaxStages + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort_flag = &s_abort;
    auto raise = [&]() {
        atomicOr(p.o.err, ERR_TIMEOUT);
        *abort_flag = 1;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(scale_bar(s), 4);
            mbar_init(empty_bar(s), 1);
        }
        for (uint32_t a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), kEpiWarps);
        }
        mbar_init(drain_bar, 1);
        fence_mbar_init();
        s_abort = 0;
        tma_prefetch_desc(&p.map_a);
        tma_prefetch_desc(&p.map_b);
        tma_prefetch_desc(&p.o.map);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&s_tmem), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = s_tmem;
    pdl_wait();
    pdl_trigger();
    const bool good = load_offsets<false>(p.o, s_offs, s_tiles);
    if (!good && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.o.err, ERR_BOUNDS);
    const int total = good ? s_tiles[p.o.E] * p.o.n_tiles : 0;
    const int stride = (int)gridDim.x;
    const int K = p.o.red, k_stages = (K + kBK - 1) / kBK;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t L = 0, ph = 1;
            int s = 0;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < total; tile += stride) {
                const Tile t = decode<false>(p.o, tile, s_offs, s_tiles);
                for (int k = 0; k < k_stages; ++k) {
                    if (!mbar_wait(empty_bar(s), ph, kWaitNs, abort_flag)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(full_bar(s), a_stage + b_stage);
                    tma_load_2d(sA + s * a_stage, &p.map_a, full_bar(s), k * 128, t.row0);
                    tma_load_3d(sB + s * b_stage, &p.map_b, full_bar(s), k * 128, t.col0, t.e);
                    ++L;
                    if (++s == p.stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) {
                raise();
                for (uint32_t i = 0; i < (uint32_t)p.stages && i < L; ++i) {  // the copies still in flight
                    const uint32_t l = L - 1 - i;
                    mbar_wait(full_bar(l % p.stages), (l / p.stages) & 1u, kDrainNs, nullptr);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_mxf4(128, bn);
            const uint32_t cols_a = 8, cols_s = cols_a + 8 * atoms;  // scale columns of a stage
            const uint32_t scale0 = tmem_base + 2 * bn;
            uint32_t n_acc = 0, ph = 0;
            int s = 0;
            bool ok = true, issued = false;
            for (int tile = blockIdx.x; ok && tile < total; tile += stride) {
                const uint32_t a = n_acc & 1u;
                if (!mbar_wait(tempty_bar(a), ((n_acc >> 1) & 1u) ^ 1u, kWaitNs, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + a * bn;
                for (int k = 0; k < k_stages; ++k) {
                    if (!mbar_wait(full_bar(s), ph, kWaitNs, abort_flag) ||
                        !mbar_wait(scale_bar(s), ph, kWaitNs, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t ta = scale0 + s * cols_s, tb = ta + cols_a;
                    const uint32_t sc = sS + s * kScaleStage;
                    for (int g = 0; g < 2; ++g) {  // four blocks (128 values) each
                        tc_copy_scales(ta + 4 * g, sc + 512 * g);
                        for (int j = 0; j < atoms; ++j)
                            tc_copy_scales(tb + 4 * (g * atoms + j), sc + 1024 + 512 * (g * atoms + j));
                    }
                    const uint64_t ad = smem_desc_k128(sA + s * a_stage), bd = smem_desc_k128(sB + s * b_stage);
                    const int steps = (min(K - k * kBK, kBK) + 63) / 64;
                    for (int i = 0; i < steps; ++i) {
                        const uint32_t half = (uint32_t)(i & 1) * 2u;  // the step's two blocks within the word
                        tc_mma_mxf4(d, ad + 2 * i, bd + 2 * i, idesc | half << 29 | half << 4, ta + 4 * (i >> 1),
                                    tb + 4 * atoms * (i >> 1), (k | i) != 0);
                    }
                    tc_commit(empty_bar(s));
                    issued = true;
                    if (++s == p.stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                tc_commit(tfull_bar(a));
                ++n_acc;
            }
            if (!ok) {
                raise();
                if (issued) {
                    tc_commit(drain_bar);
                    mbar_wait(drain_bar, 0, kDrainNs, nullptr);
                }
            }
        }
    } else if (warp < 2 + kEpiWarps) {
        const int q = warp & 3;  // the TMEM lane quadrant this warp may read
        const uint32_t sb = sE + (uint32_t)q * 4096u;
        uint32_t n_acc = 0;
        for (int tile = blockIdx.x; tile < total; tile += stride, ++n_acc) {
            const Tile t = decode<false>(p.o, tile, s_offs, s_tiles);
            const uint32_t a = n_acc & 1u;
            if (!__all_sync(0xffffffffu, mbar_wait(tfull_bar(a), (n_acc >> 1) & 1u, kWaitNs, abort_flag))) {
                if (lane == 0) raise();
                break;
            }
            tc_fence_after();
            store_tile<false>(p.o, t, tmem_base + a * bn, false, sb, q, lane);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(a));
        }
        if (lane == 0) bulk_wait_all();  // the stores are performed before the CTA ends
    } else {
        const int set = (warp - 2 - kEpiWarps) >> 2;
        const int i = (int)threadIdx.x - 64 - 32 * kEpiWarps - 128 * set;  // 0..127 within the set
        const int quads = bn / 4;                                          // groups of four weight rows
        const int bg = i / quads, bj = i % quads;                          // this thread's four blocks and four rows
        const int n_blocks = K / 32;
        const size_t ws_e = (size_t)n_blocks * p.o.n_out;
        auto load = [&](const Tile &t, int k) {
            Scales v;
            v.a[0] = v.a[1] = 0;
            v.b[0] = v.b[1] = v.b[2] = v.b[3] = 0;
            const int b0 = k * kBlocks;
            if (i < t.m_valid) {
                const uint8_t *src = p.xs + (size_t)b0 * p.o.rows + t.row0 + i;
#pragma unroll
                for (int j = 0; j < kBlocks; ++j)
                    if (b0 + j < n_blocks) v.a[j >> 2] |= (uint32_t)__ldg(src + (size_t)j * p.o.rows) << (8 * (j & 3));
            }
            const int n = t.col0 + 4 * bj;
            if (bg < 2 && n < p.o.n_out) {  // n_out is a multiple of 8
                const uint8_t *src = p.ws + t.e * ws_e + (size_t)(b0 + 4 * bg) * p.o.n_out + n;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (b0 + 4 * bg + j < n_blocks)
                        v.b[j] = __ldg(reinterpret_cast<const uint32_t *>(src + (size_t)j * p.o.n_out));
            }
            return v;
        };
        auto store = [&](const Scales &v, int s) {
            const uint32_t sc = sS + s * kScaleStage;
            const uint32_t at = sc + (uint32_t)(i & 31) * 16u + (uint32_t)(i >> 5) * 4u;
            st_shared_u32(at, v.a[0]);
            st_shared_u32(at + 512, v.a[1]);
            if (bg < 2) {
                const uint32_t p01 = __byte_perm(v.b[0], v.b[1], 0x5140), p23 = __byte_perm(v.b[2], v.b[3], 0x5140);
                const uint32_t q01 = __byte_perm(v.b[0], v.b[1], 0x7362), q23 = __byte_perm(v.b[2], v.b[3], 0x7362);
                const uint32_t w[4] = {__byte_perm(p01, p23, 0x5410), __byte_perm(p01, p23, 0x7632),
                                       __byte_perm(q01, q23, 0x5410), __byte_perm(q01, q23, 0x7632)};
                const int r0 = 4 * bj, rr = r0 & 127;
                const uint32_t bt = sc + 1024u + 512u * (uint32_t)(bg * atoms + (r0 >> 7)) + (uint32_t)(rr >> 5) * 4u +
                                    (uint32_t)(rr & 31) * 16u;
#pragma unroll
                for (int j = 0; j < 4; ++j) st_shared_u32(bt + 16 * j, w[j]);
            }
        };
        // this set's stages: number n = set, set + kScaleSets, .. of the CTA's sequence
        int tile = blockIdx.x, k = set;
        auto settle = [&]() {
            while (tile < total && k >= k_stages) {
                k -= k_stages;
                tile += stride;
            }
        };
        settle();
        Scales next;
        Tile t;
        int t_of = -1;
        auto fetch = [&]() {
            if (tile >= total) return;
            if (t_of != tile) {
                t = decode<false>(p.o, tile, s_offs, s_tiles);
                t_of = tile;
            }
            next = load(t, k);
        };
        fetch();
        for (uint32_t n = set; tile < total; n += kScaleSets) {
            const Scales now = next;
            k += kScaleSets;
            settle();
            fetch();
            const int s = n % p.stages;
            if (!__all_sync(0xffffffffu, mbar_wait(empty_bar(s), ((n / p.stages) & 1u) ^ 1u, kWaitNs, abort_flag))) {
                if (lane == 0) raise();
                break;
            }
            store(now, s);
            fence_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(scale_bar(s));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

unsigned long long g_attr;

// Tile sizes.  Rows: 32-row boxes while the experts average at most 16 rows.  Columns: the
// widest tile that still gives every SM one.
void choose_tiles(MxGroupedArgs &g, int sms) {
    GroupedOut &a = g.o;
    const long long active = std::min<long long>(a.E, a.rows);
    a.bm = a.rows <= 16ll * a.E ? 32 : 128;
    a.bn = kMaxBn;
    while (a.bn > 64) {
        const long long n = (a.n_out + a.bn - 1) / a.bn;
        if (n * std::max<long long>(active, a.rows / a.bm) >= sms && a.bn - 64 < a.n_out) break;
        a.bn -= 64;
    }
    a.n_tiles = (a.n_out + a.bn - 1) / a.bn;
    const int atoms = (a.bn + 127) / 128;
    g.stages = std::min({kMaxStages, kStageSpace / ((a.bm + a.bn) * 128 + kScaleStage),
                         ((int)kTmemCols - 2 * a.bn) / (8 + 8 * atoms)});
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
    const int sms = op_num_sms();
    int *err = op_error_word();
    if (sms < 1 || err == nullptr) return op_fail(MOE_ERR_CUDA, "%s: no usable current device", op);
    MxGroupedArgs g = {};
    g.o.offs = offs;
    g.o.out = Y;
    g.o.err = err;
    g.o.E = E;
    g.o.rows = rows;
    g.o.n_out = N;
    g.o.red = K;
    g.o.f32 = out_dtype == MOE_DTYPE_F32;
    g.xs = Xs;
    g.ws = Ws;
    choose_tiles(g, sms);
    const long long tiles = ((long long)rows / g.o.bm + std::min(E, rows)) * g.o.n_tiles;
    if (tiles > (1ll << 30)) return op_fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^30 output tiles", op);
    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const uint64_t n = N, c = K / 2, r = rows, e = E, es = g.o.f32 ? 4 : 2;
    const OpMap ma = {u8, 2, Xc, {c, r}, {c}, {128, (uint32_t)g.o.bm}, sw};
    const OpMap mb = {u8, 3, Wc, {c, n, e}, {c, n * c}, {128, (uint32_t)g.o.bn, 1}, sw};
    const OpMap mo = {g.o.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      3, Y, {n, r, 1}, {n * es, n * es * r}, {(uint32_t)(128 / es), 32, 1}, sw};
    if (op_encode(&g.map_a, ma) != CUDA_SUCCESS || op_encode(&g.map_b, mb) != CUDA_SUCCESS ||
        op_encode(&g.o.map, mo) != CUDA_SUCCESS)
        return op_fail(MOE_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", op);
    cudaError_t ce = op_allow_smem(reinterpret_cast<const void *>(mx_grouped_kernel), kSmemBytes, &g_attr);
    if (ce == cudaSuccess)
        ce = launch_pdl(mx_grouped_kernel, dim3((unsigned)std::min<long long>(sms, tiles)), dim3(kThreads),
                        (size_t)kSmemBytes, reinterpret_cast<cudaStream_t>(stream), g);
    return op_cuda(ce, op);
}
