// Matrix products grouped by expert with ragged sizes, and their gradients: the rows
// offs[e] <= r < offs[e + 1] belong to expert e (the expert-sorted order of the
// dispatch), W is the stacked [E, N, K] tensor.
//
//   forward  Y[r, n]    = sum_k X[r, k] W[e][n, k]
//   dgrad    dX[r, k]   = sum_n dY[r, n] W[e][n, k]
//   wgrad    dW[e][n, k] (+)= sum_r dY[r, n] X[r, k]
//
// bf16 operands, products and sums in fp32 on the tensor cores (tcgen05, accumulators in
// tensor memory), one rounding to the output type.  No operand is transposed in memory:
// the tensor core reads a shared-memory tile with its reduction index innermost
// ("K-major": X, dY and W of the forward) or outermost ("MN-major": W of the dgrad, both
// operands of the wgrad), so all three read the tensors as they are stored.
//
// Persistent kernel, 6 warps:
//   warp 0     TMA producer: per stage one k-block of 64 reduction steps, A tile
//              [bm rows] and B tile [bn columns], 128-byte swizzle
//   warp 1     allocates tensor memory; issues tcgen05.mma (M 128, N bn, K 16) into one of
//              two accumulators, so a tile's epilogue overlaps the next tile's main loop
//   warps 2-5  epilogue: tcgen05.ld, conversion, a swizzled 4 KB slice per warp in shared
//              memory, one TMA store (or coalesced stores of the valid rows where the next
//              expert's rows follow; or load-add-store when accumulating)
// Every CTA reads the offsets, checks them and derives the tile list itself, so there is
// no workspace, no launch before the product and no atomic; a tile's sum has a fixed order
// and results are the same from call to call.
//
// The wgrad reduces over an expert's rows, whose number is arbitrary: the last k-block
// also brings rows of the next expert (or past the buffer).  Whole 16-row steps past the
// end are not issued, and the MMA warp zeroes the rest of the last step in both operand
// tiles (a zero in one would not do: the other may hold an infinity or a NaN).
//
// Decreasing or out-of-range offsets: every CTA sees the same, records ERR_BOUNDS and
// writes nothing.  Every wait is bounded; on a timeout the kernel records ERR_TIMEOUT,
// drains its copies and MMAs, frees tensor memory and returns.
#include <algorithm>

#include "common.cuh"
#include "grouped.cuh"
#include "kernels.h"
#include "moe.h"
#include "op_host.h"

namespace moe {
namespace {

enum : int { kForward = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kBK = 64;           // reduction steps per stage: 128 bytes of bf16
constexpr int kMaxStages = 12;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kAccCols = 256;     // columns of one accumulator
constexpr uint32_t kTmemCols = 2 * kAccCols;
constexpr int kChunk = 64 * kBK * 2;  // an MN-major tile of 64 columns x 64 reduction rows
constexpr int kStageSpace = 196608;  // 192 KB of stages
constexpr int kSmemBytes = kStageSpace + kEpiBytes + 1024 /* alignment */;

struct GroupedArgs {
    CUtensorMap map_a, map_b;
    GroupedOut o;
    int stages;
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

template <int OP>
__global__ void __launch_bounds__(kThreads, 1) grouped_kernel(const __grid_constant__ GroupedArgs p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t s_bars[2 * kMaxStages + 5];
    __shared__ int s_offs[kMaxExperts + 1], s_tiles[kMaxExperts + 1];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int a_stage = (OP == kWgrad ? 128 : p.o.bm) * kBK * 2, b_stage = p.o.bn * kBK * 2;
    // all A stages first: the MMA reads 128 rows of A where the box brought 32 or 64; the
    // rest is whatever follows, and its results are not stored
    const uint32_t sA = base, sB = base + (uint32_t)(p.stages * a_stage), sE = base + kStageSpace;
    const uint32_t bar0 = smem_u32(s_bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * kMaxStages + a); };
    auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * kMaxStages + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * kMaxStages + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort_flag = &s_abort;
    auto raise = [&]() {
        atomicOr(p.o.err, ERR_TIMEOUT);
        *abort_flag = 1;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(full_bar(s), 1);
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
    pdl_wait();  // the offsets and operands of earlier kernels on the stream
    pdl_trigger();
    const bool good = load_offsets<OP == kWgrad>(p.o, s_offs, s_tiles);
    if (!good && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.o.err, ERR_BOUNDS);
    const int total = !good ? 0 : OP == kWgrad ? p.o.E * p.o.m_tiles * p.o.n_tiles : s_tiles[p.o.E] * p.o.n_tiles;
    const int stride = (int)gridDim.x;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t L = 0;
            int s = 0;
            uint32_t ph = 1;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < total; tile += stride) {
                const Tile t = decode<OP == kWgrad>(p.o, tile, s_offs, s_tiles);
                for (int r = t.r0; r < t.r1; r += kBK) {
                    if (!mbar_wait(empty_bar(s), ph, kWaitNs, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = full_bar(s), da = sA + s * a_stage, db = sB + s * b_stage;
                    mbar_arrive_expect_tx(bar, a_stage + b_stage);
                    if (OP == kWgrad) {
                        tma_load_2d(da, &p.map_a, bar, t.row0, r);
                        tma_load_2d(da + kChunk, &p.map_a, bar, t.row0 + 64, r);
                        for (int c = 0; c < p.o.bn; c += 64) tma_load_2d(db + c * (kBK * 2), &p.map_b, bar, t.col0 + c, r);
                    } else {
                        tma_load_2d(da, &p.map_a, bar, r, t.row0);
                        if (OP == kForward)
                            tma_load_3d(db, &p.map_b, bar, r, t.col0, t.e);
                        else
                            for (int c = 0; c < p.o.bn; c += 64)
                                tma_load_3d(db + c * (kBK * 2), &p.map_b, bar, t.col0 + c, r, t.e);
                    }
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
        // The wgrad's last k-block is zeroed by the whole warp, so there all lanes follow the
        // loop; otherwise lane 0 alone.
        if (OP == kWgrad || lane == 0) {
            const uint32_t idesc = idesc_bf16_f32(128, p.o.bn) | (OP == kWgrad ? 1u << 15 : 0u) | (OP != kForward ? 1u << 16 : 0u);
            constexpr uint32_t kStepA = OP == kWgrad ? (16 * 128) >> 4 : 2;   // 16 reduction steps on,
            constexpr uint32_t kStepB = OP == kForward ? 2 : (16 * 128) >> 4;  // in units of 16 bytes
            uint32_t n_acc = 0, ph = 0;
            int s = 0;
            bool ok = true, issued = false;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                const bool got = mbar_wait(bar, parity, kWaitNs, abort_flag);
                return OP == kWgrad ? __all_sync(0xffffffffu, got) != 0 : got;
            };
            for (int tile = blockIdx.x; ok && tile < total; tile += stride) {
                const Tile t = decode<OP == kWgrad>(p.o, tile, s_offs, s_tiles);
                if (t.r0 >= t.r1) continue;  // an expert without rows: the epilogue writes its zeros
                const uint32_t a = n_acc & 1u;
                if (!wait(tempty_bar(a), ((n_acc >> 1) & 1u) ^ 1u)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + a * kAccCols;
                for (int r = t.r0; r < t.r1; r += kBK) {
                    if (!wait(full_bar(s), ph)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t da = sA + s * a_stage, db = sB + s * b_stage;
                    int steps = kBK / 16;
                    if (OP == kWgrad && t.r1 - r < kBK) {
                        const int valid = t.r1 - r;
                        steps = (valid + 15) / 16;
                        const int words = (steps * 16 - valid) * 8;  // 16-byte units per 64-column chunk
                        for (int c = 0; c < 2 + p.o.bn / 64; ++c) {
                            const uint32_t chunk = (c < 2 ? da + c * kChunk : db + (c - 2) * kChunk) + valid * 128;
                            for (int w = lane; w < words; w += 32) st_shared_v4(chunk + 16 * w, 0, 0, 0, 0);
                        }
                        fence_smem();
                        __syncwarp();
                    }
                    if (lane == 0) {
                        const uint64_t ad = OP == kWgrad ? smem_desc_mn128(da) : smem_desc_k128(da);
                        const uint64_t bd = OP == kForward ? smem_desc_k128(db) : smem_desc_mn128(db);
                        for (int k = 0; k < steps; ++k)
                            tc_mma_bf16(d, ad + k * kStepA, bd + k * kStepB, idesc, (r != t.r0) | (k != 0));
                        tc_commit(empty_bar(s));
                        issued = true;
                    }
                    if (++s == p.stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                if (lane == 0) tc_commit(tfull_bar(a));
                ++n_acc;
            }
            if (!ok && lane == 0) {
                raise();
                if (issued) {
                    tc_commit(drain_bar);
                    mbar_wait(drain_bar, 0, kDrainNs, nullptr);
                }
            }
        }
    } else {
        const int q = warp & 3;  // the TMEM lane quadrant this warp may read
        const uint32_t sb = sE + (uint32_t)q * 4096u;
        uint32_t n_acc = 0;
        for (int tile = blockIdx.x; tile < total; tile += stride) {
            const Tile t = decode<OP == kWgrad>(p.o, tile, s_offs, s_tiles);
            const bool empty = t.r0 >= t.r1;
            const uint32_t a = n_acc & 1u;
            if (!empty) {
                if (!__all_sync(0xffffffffu, mbar_wait(tfull_bar(a), (n_acc >> 1) & 1u, kWaitNs, abort_flag))) {
                    if (lane == 0) raise();
                    break;
                }
                tc_fence_after();
            }
            store_tile<OP == kWgrad>(p.o, t, tmem_base + a * kAccCols, empty, sb, q, lane);
            if (!empty) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(tempty_bar(a));
                ++n_acc;
            }
        }
        if (lane == 0) bulk_wait_all();  // the stores are performed before the CTA ends
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

unsigned long long g_attr[3];

// Tile sizes.  Rows: 32-row boxes while the experts average at most 16 rows, as the fused
// block's decode tiles.  Columns: the widest tile that still gives every SM one.
void choose_tiles(GroupedArgs &g, int op, int sms) {
    GroupedOut &a = g.o;
    const long long active = std::min<long long>(a.E, a.rows);
    if (op == kWgrad) {
        a.bm = 128;
        a.m_tiles = (a.m_dense + 127) / 128;
    } else {
        a.bm = a.rows <= 16ll * a.E ? 32 : 128;
    }
    a.bn = 256;
    while (a.bn > 64) {
        const long long n = (a.n_out + a.bn - 1) / a.bn;
        const long long tiles = op == kWgrad ? n * a.m_tiles * a.E : n * std::max<long long>(active, a.rows / a.bm);
        if (tiles >= sms && a.bn - 64 < a.n_out) break;
        a.bn /= 2;
    }
    a.n_tiles = (a.n_out + a.bn - 1) / a.bn;
    g.stages = std::min(kMaxStages, kStageSpace / ((a.bm + a.bn) * kBK * 2));
}

moe_status check(const char *op, const void *a, const void *b, const int32_t *offs, const void *out, int rows, int E,
                 int N, int K, int dtype, bool need_rows) {
    if (rows < 0 || E < 1 || N < 1 || K < 1)
        return op_fail(MOE_ERR_INVALID_ARG, "%s: need rows >= 0, E >= 1, N >= 1, K >= 1", op);
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32)
        return op_fail(MOE_ERR_INVALID_ARG, "%s: unknown out_dtype %d", op, dtype);
    if (E > kMaxExperts || N % 8 || K % 8 || N > (1 << 20) || K > (1 << 20) || rows > (1 << 30))
        return op_fail(MOE_ERR_UNSUPPORTED,
                       "%s: E up to 256, N and K multiples of 8 up to 2^20, rows up to 2^30 (E %d, N %d, K %d, rows %d)", op,
                       E, N, K, rows);
    if (need_rows && (!a || !b || !offs || !out)) return op_fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer", op);
    if (!op_aligned16(a) || !op_aligned16(b) || !op_aligned16(out) || (reinterpret_cast<uintptr_t>(offs) & 3u))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned, the offsets 4-byte aligned", op);
    return MOE_OK;
}

// a: X or dY [rows, ..]; b: W [E, N, K], or X for the wgrad
moe_status launch(const char *name, int op, const void *a, const void *b, const int32_t *offs, void *out, int rows, int E,
                  int N, int K, int dtype, int accumulate, moe_stream_t stream) {
    const int sms = op_num_sms();
    int *err = op_error_word();
    if (sms < 1 || err == nullptr) return op_fail(MOE_ERR_CUDA, "%s: no usable current device", name);
    GroupedArgs g = {};
    g.o.offs = offs;
    g.o.out = out;
    g.o.err = err;
    g.o.E = E;
    g.o.rows = rows;
    g.o.n_out = op == kForward ? N : K;
    g.o.m_dense = N;
    g.o.red = op == kForward ? K : N;
    g.o.f32 = dtype == MOE_DTYPE_F32;
    g.o.accumulate = accumulate;
    choose_tiles(g, op, sms);
    const long long tiles = op == kWgrad ? (long long)E * g.o.m_tiles * g.o.n_tiles
                                         : ((long long)rows / g.o.bm + std::min(E, rows)) * g.o.n_tiles;
    if (tiles > (1ll << 30)) return op_fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^30 output tiles", name);

    const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const uint64_t n = N, k = K, r = rows, e = E;
    OpMap ma, mb;
    if (op == kWgrad) {
        ma = {bf, 2, a, {n, r}, {n * 2}, {64, kBK}, sw};
        mb = {bf, 2, b, {k, r}, {k * 2}, {64, kBK}, sw};
    } else {
        const uint64_t c = g.o.red;
        ma = {bf, 2, a, {c, r}, {c * 2}, {kBK, (uint32_t)g.o.bm}, sw};
        mb = {bf, 3, b, {k, n, e}, {k * 2, n * k * 2}, {64, op == kForward ? (uint32_t)g.o.bn : (uint32_t)kBK, 1}, sw};
    }
    const uint64_t es = g.o.f32 ? 4 : 2, cols = g.o.n_out;
    const OpMap mo = {g.o.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : bf,
                      3,
                      out,
                      {cols, op == kWgrad ? n : r, op == kWgrad ? e : 1},
                      {cols * es, cols * es * (op == kWgrad ? n : r)},
                      {(uint32_t)(128 / es), 32, 1},
                      sw};
    if (op_encode(&g.map_a, ma) != CUDA_SUCCESS || op_encode(&g.map_b, mb) != CUDA_SUCCESS ||
        op_encode(&g.o.map, mo) != CUDA_SUCCESS)
        return op_fail(MOE_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", name);
    const dim3 grid((unsigned)std::min<long long>(sms, tiles));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto kernel) -> cudaError_t {
        const cudaError_t err2 = op_allow_smem(reinterpret_cast<const void *>(kernel), kSmemBytes, &g_attr[op]);
        return err2 != cudaSuccess ? err2 : launch_pdl(kernel, grid, dim3(kThreads), (size_t)kSmemBytes, s, g);
    };
    return op_cuda(op == kForward ? go(grouped_kernel<kForward>)
                                  : op == kDgrad ? go(grouped_kernel<kDgrad>) : go(grouped_kernel<kWgrad>),
                   name);
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_grouped_forward(const void *X, const void *W, const int32_t *offs, int rows, int E, int N, int K,
                                          int out_dtype, void *Y, moe_stream_t stream) {
    using namespace moe;
    const moe_status st = check("moe_grouped_forward", X, W, offs, Y, rows, E, N, K, out_dtype, rows > 0);
    if (st != MOE_OK || rows == 0) return st;
    return launch("moe_grouped_forward", kForward, X, W, offs, Y, rows, E, N, K, out_dtype, 0, stream);
}

extern "C" moe_status moe_grouped_dgrad(const void *dY, const void *W, const int32_t *offs, int rows, int E, int N, int K,
                                        int out_dtype, void *dX, moe_stream_t stream) {
    using namespace moe;
    const moe_status st = check("moe_grouped_dgrad", dY, W, offs, dX, rows, E, N, K, out_dtype, rows > 0);
    if (st != MOE_OK || rows == 0) return st;
    return launch("moe_grouped_dgrad", kDgrad, dY, W, offs, dX, rows, E, N, K, out_dtype, 0, stream);
}

extern "C" moe_status moe_grouped_wgrad(const void *dY, const void *X, const int32_t *offs, int rows, int E, int N, int K,
                                        int out_dtype, int accumulate, void *dW, moe_stream_t stream) {
    using namespace moe;
    const char *name = "moe_grouped_wgrad";
    const moe_status st = check(name, dY, X, offs, dW, rows, E, N, K, out_dtype, rows > 0);
    if (st != MOE_OK) return st;
    if (accumulate != 0 && accumulate != 1) return op_fail(MOE_ERR_INVALID_ARG, "%s: accumulate must be 0 or 1", name);
    if (dW == nullptr) return op_fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer", name);
    if (rows == 0) {
        if (accumulate) return MOE_OK;
        const size_t bytes = (size_t)E * N * K * (out_dtype == MOE_DTYPE_F32 ? 4 : 2);
        return op_cuda(cudaMemsetAsync(dW, 0, bytes, reinterpret_cast<cudaStream_t>(stream)), name);
    }
    return launch(name, kWgrad, dY, X, offs, dW, rows, E, N, K, out_dtype, accumulate, stream);
}
