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
// ("K-major": both operands of the forward, dY of the dgrad) or outermost ("MN-major": W of
// the dgrad, both operands of the wgrad), so all three read the tensors as they are stored.
//
// Persistent kernel on CTA pairs (tcgen05 cta_group::2): a tile is up to 256 output columns
// (M; 128 in each CTA) x up to 256 output rows (N; each CTA stages half of them), so a CTA
// brings 32 KB per 64 reduction steps instead of the 48 KB of a 128 x 256 tile of its own,
// and L2 keeps up with the tensor cores.  Warps of a CTA:
//   warp 0     TMA producer: per stage one or two blocks of 64 reduction steps of this CTA's A
//              (columns) and B (rows) operand, 128-byte swizzle; both CTAs' copies complete on the barrier
//              of the even CTA
//   warp 1     allocates tensor memory; in the even CTA issues tcgen05.mma (K 16) into one
//              of two accumulators, so a tile's epilogue overlaps the next one's main loop
//   warps 2-9  epilogue (grouped.cuh)
//   warp 10    (wgrad) zeroes the rest of tails, see below
// Every CTA reads the offsets, checks them and derives the tile list itself, so there is
// no workspace, no launch before the product and no atomic; a tile's sum has a fixed order
// and results are the same from call to call.
//
// The wgrad reduces over an expert's rows, whose number is arbitrary: the last stage also
// brings rows of the next expert (or past the buffer).  Whole 16-row steps past the end are
// not issued, and the rest of the last step is zeroed in both operand tiles by warp 10 of
// each CTA (a zero in one would not do: the other may hold an infinity or a NaN).  Such a
// stage's copies complete on a barrier of their own CTA, and the stage is handed to the MMA
// when both CTAs have zeroed.
//
// Measured on GB300, one call in a row of them on the same tensors, / alone with cold caches (bf16;
// 64 experts, N 1408, K 2048):
//   forward, 24576 rows    105 / 113 us, 1.35 PFLOP/s, 5.1 TB/s.  The tensor pipe is 77% busy and
//                          HBM 65%: of 1408 columns the sixth tile is half empty (8% of the
//                          products), and eight of 76 pairs take an eleventh tile
//   dgrad, 24576 rows      98 / 105 us to 2048 columns
//   wgrad, 24576 rows      fp32 146 / 148 us, 6.2 TB/s: the 738 MB it writes; bf16 105 / 105
//   the same, accumulating fp32 888 / 895 us, bf16 219 / 222: store_tile has eight loads of the old
//                          values in flight per lane, and waits for them between its stores
//   forward, 384 rows      58 / 76 us, 6.5 TB/s: the weights, streamed once
//   forward, one expert, 16384 rows, K 1408, N 2048   54 / 58 us, 1.76 PFLOP/s
//   forward, one token's six experts   7.4 / 17 us: start and end of the launch around 35 MB
// One CTA per 128 x 256 tile with the rows as M took 128 (forward), 145 and 181 us.
//
// Decreasing or out-of-range offsets: every CTA sees the same, records ERR_BOUNDS and
// writes nothing.  Every wait is bounded; on a timeout the kernel records ERR_TIMEOUT in
// both CTAs, lets its copies and MMAs end, frees tensor memory and returns.
#include <algorithm>

#include "grouped_kernel.cuh"
#include "moe.h"

namespace moe {
namespace {

OpDone g_attr[12];

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

// x: X or dY [rows, ..]; w: W [E, N, K], or X for the wgrad
moe_status launch(const char *name, int op, const void *x, const void *w, const int32_t *offs, void *out, int rows, int E,
                  int N, int K, int dtype, int accumulate, moe_stream_t stream) {
    GroupedArgs g = {};
    GroupedOut &o = g.o;
    o.offs = offs;
    o.out = out;
    o.E = E;
    o.rows = rows;
    o.n_out = op == kForward ? N : K;
    o.m_dense = N;
    o.red = op == kForward ? K : N;
    o.f32 = dtype == MOE_DTYPE_F32;
    o.segment = segment_of(o.f32, 16);
    o.wait = wait_cycles((op == kWgrad ? rows : o.red) / kBK + 1);
    const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const uint64_t n = N, k = K, r = rows, e = E;
    const uint64_t x_bytes = 2 * r * (op == kForward ? k : n), w_bytes = 2 * (op == kWgrad ? r * k : e * n * k);
    const uint64_t out_bytes = (o.f32 ? 4 : 2) * (op == kWgrad ? e * n * k : r * (uint64_t)o.n_out);
    if (op_overlap(out, out_bytes, x, x_bytes) || op_overlap(out, out_bytes, w, w_bytes) ||
        op_overlap(out, out_bytes, offs, 4 * (e + 1)))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: the output overlaps an input", name);
    const int sms = op_num_sms();
    o.err = op_error_word();
    if (sms < 2 || o.err == nullptr) return op_fail(MOE_ERR_CUDA, "%s: no usable current device", name);
    const bool segments = (op == kWgrad ? rows : o.red) > o.segment;
    const int blocks = choose_tiles(g, op, op == kWgrad ? accumulate != 0 : segments, sms);
    const long long tiles = op == kWgrad ? (long long)E * o.row_tiles * o.col_tiles
                                         : ((long long)rows / o.tile_rows + std::min(E, rows)) * o.col_tiles;
    if (tiles > (1ll << 30)) return op_fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^30 output tiles", name);

    CUresult cr;
    if (op == kWgrad) {
        cr = op_encode(&g.map_a, {bf, 2, w, {k, r}, {k * 2}, {64, kBK}, sw});
        if (cr == CUDA_SUCCESS) cr = op_encode(&g.map_b[0], {bf, 2, x, {n, r}, {n * 2}, {64, kBK}, sw});
    } else {
        cr = op_encode(&g.map_a, {bf, 3, w, {k, n, e}, {k * 2, n * k * 2},
                                  {64, op == kForward ? (uint32_t)o.cols / 2 : (uint32_t)kBK, 1}, sw});
        const uint64_t c = o.red;
        for (int i = 0; i < o.tile_rows / 32 && cr == CUDA_SUCCESS; ++i)
            cr = op_encode(&g.map_b[i], {bf, 2, x, {c, r}, {c * 2}, {kBK, 16u * (i + 1)}, sw});
    }
    if (cr != CUDA_SUCCESS) return op_fail(MOE_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", name, (int)cr);
    const dim3 grid(2u * (unsigned)std::min<long long>(sms / 2, tiles));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto kernel, int threads, int which) -> cudaError_t {
        const cudaError_t ce = op_allow_smem(reinterpret_cast<const void *>(kernel), kSmemBytes, &g_attr[which]);
        return ce != cudaSuccess
                   ? ce
                   : launch_pdl_cluster(kernel, grid, dim3((unsigned)threads), (size_t)kSmemBytes, s,
                                        dim3(2, 1, 1), g);
    };
    // sums of one segment have kernels without the walk over segments (128 experts of 16 rows, wgrad:
    // 16.4 against 16.9 us; 16 of 48, dgrad: 7.4 against 7.8)
    cudaError_t ce;
    if (op == kForward)
        ce = segments      ? go(grouped_kernel<kForward, 1, false, true>, kThreads<kForward>, 0)
             : blocks == 1 ? go(grouped_kernel<kForward, 1, false, false>, kThreads<kForward>, 1)
                           : go(grouped_kernel<kForward, 2, false, false>, kThreads<kForward>, 2);
    else if (op == kDgrad)
        ce = segments      ? go(grouped_kernel<kDgrad, 1, false, true>, kThreads<kDgrad>, 3)
             : blocks == 1 ? go(grouped_kernel<kDgrad, 1, false, false>, kThreads<kDgrad>, 4)
                           : go(grouped_kernel<kDgrad, 2, false, false>, kThreads<kDgrad>, 5);
    else if (accumulate)
        ce = segments ? go(grouped_kernel<kWgrad, 1, true, true>, kThreads<kWgrad>, 6)
                      : go(grouped_kernel<kWgrad, 1, true, false>, kThreads<kWgrad>, 11);
    else if (segments)
        ce = blocks == 1 ? go(grouped_kernel<kWgrad, 1, false, true>, kThreads<kWgrad>, 7)
                         : go(grouped_kernel<kWgrad, 2, false, true>, kThreads<kWgrad>, 8);
    else
        ce = blocks == 1 ? go(grouped_kernel<kWgrad, 1, false, false>, kThreads<kWgrad>, 9)
                         : go(grouped_kernel<kWgrad, 2, false, false>, kThreads<kWgrad>, 10);
    return op_cuda(ce, name);
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
