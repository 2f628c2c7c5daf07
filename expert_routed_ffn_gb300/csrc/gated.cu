// The gated feed-forward block over expert-grouped rows, for training and serving:
//
//   forward   G = X Wg^T, U = X Wu^T, H = act(G, U)      (gated.cuh: the activation)
//   backward  dH = dY Wd; dG = dH dact/dG, dU = dH dact/dU
//   dgrad     dX = dG Wg + dU Wu
//
// Each is one launch of the grouped products' kernel (grouped_kernel.cuh), whose tiles, offsets,
// pipeline and bounded waits it shares.
//   forward: the MMA's 256 columns are 128 of the gate's and the same 128 of the up projection's,
//     in turns of 16, so that the epilogue has both values of a column in one warp.  G and U leave
//     as bf16 only where the caller keeps them for the backward pass; H comes from the fp32 sums.
//   backward: a dgrad through Wd whose epilogue reads G and U and stores both gradients: dH never
//     is in memory, and is not rounded.
//   dgrad: one sum over both projections' columns, so dX is written once and rounded once.  Each
//     half of the sum is padded to whole steps of 64, whose copies bring zeros in both operands.
// The weights' gradients are moe_grouped_wgrad's of dG, dU with X and of dY with H.
//
// Measured on GB300, 30 calls in a row after a pause, at 1.7 GHz (in brackets: called for seconds, when power
// brings the clock to 1.33 to 1.4 GHz; the same or other tensors from call to call make no difference); 64
// experts, I 1408, K 2048:
//   forward, 24576 rows, G and U kept   201 us (243), without them 186 (227): 1.41 PFLOP/s, 5.1 TB/s, the
//              tensor pipe busy 72% of the cycles and HBM 65%; with all rows in one expert, whose weights
//              stay in L2, 153 (185) and 145 us, 1.95 PFLOP/s
//   backward, 24576 rows   130 us (148), 5.6 TB/s, tensor pipe 62%: 553 MB of dY, G, U, dG and dU beside 369 MB of
//              weights.  With two epilogue warps per lane quadrant it waited for the gradients' arithmetic
//              (180 us), with loads of G and U after the sums for those
//   dgrad, 24576 rows, fp32   209 us (239), 5.2 TB/s, tensor pipe 71%
// What bounds forward and dgrad: experts of 384 rows (tiles of 192) take as many cycles as experts of 448
// (322 and 321 us x GHz; of 512 341, 89% of the MMAs' rate), so a stage of few rows takes as long as its
// operands need into shared memory, 16 KB of weights and 12 KB of rows, and not as long as its MMAs.
//
//   forward, one token's six experts   12.8 us (14.9 with changing inputs), 69 MB of weights
//   dgrad, 2000 rows, 128 experts, 256 x 1024   25.5 us with changing inputs, 5.5 TB/s
#include <algorithm>

#include "grouped_kernel.cuh"
#include "moe.h"

namespace moe {
namespace {

OpDone g_attr[12];

// Products that one accumulator sums for fp32 results: 32 instructions, 4.6e-7 off (2-norm) over 2 x 1408
// columns where a sum in fp32 is 3e-7 off, and at 24576 rows of 64 experts 209 us.  With 256, as the
// single products' have, 3.0e-6 and 206; 64 9.3e-7 and 207; 16 2.4e-7 and 217.  A multiple of a stage's 128.
constexpr int kExactSegment = 32 * 16;

struct Sizes {
    int rows, E, I, K;
};

moe_status check_sizes(const char *op, const Sizes &z) {
    if (z.rows < 0 || z.E < 1 || z.I < 1 || z.K < 1)
        return op_fail(MOE_ERR_INVALID_ARG, "%s: need rows >= 0, E >= 1, I >= 1, K >= 1", op);
    if (z.E > kMaxExperts || z.I % 8 || z.K % 8 || z.I > (1 << 20) || z.K > (1 << 20) || z.rows > (1 << 30))
        return op_fail(MOE_ERR_UNSUPPORTED,
                       "%s: E up to 256, I and K multiples of 8 up to 2^20, rows up to 2^30 (E %d, I %d, K %d, rows %d)", op,
                       z.E, z.I, z.K, z.rows);
    return MOE_OK;
}

moe_status check_act(const char *op, int act, float alpha, float limit, float beta) {
    if (act != MOE_ACT_SILU && act != MOE_ACT_SWIGLU_OAI) return op_fail(MOE_ERR_INVALID_ARG, "%s: unknown activation %d", op, act);
    // NaN fails every comparison
    if (act == MOE_ACT_SWIGLU_OAI && !(limit > 0.0f && alpha - alpha == 0.0f && beta - beta == 0.0f))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: need limit > 0, finite alpha and beta", op);
    return MOE_OK;
}

struct Buffer {
    const void *p;
    uint64_t bytes;
};

// All there and aligned, the outputs (the first n_out) apart from each other and from the rest.
moe_status check_buffers(const char *op, const Buffer *b, int n_out, int n, const int32_t *offs, int E) {
    for (int i = 0; i < n; ++i) {
        if (b[i].p == nullptr) return op_fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer", op);
        if (!op_aligned16(b[i].p)) return op_fail(MOE_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", op);
    }
    if (offs == nullptr || (reinterpret_cast<uintptr_t>(offs) & 3u))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: the offsets are NULL or not 4-byte aligned", op);
    for (int i = 0; i < n_out; ++i) {
        for (int j = i + 1; j < n; ++j)
            if (op_overlap(b[i].p, b[i].bytes, b[j].p, b[j].bytes))
                return op_fail(MOE_ERR_INVALID_ARG, "%s: an output overlaps another tensor", op);
        if (op_overlap(b[i].p, b[i].bytes, offs, 4 * ((uint64_t)E + 1)))
            return op_fail(MOE_ERR_INVALID_ARG, "%s: an output overlaps the offsets", op);
    }
    return MOE_OK;
}

// What all three set; n_out: columns of the MMA's output, red: the reduction.
moe_status start(const char *name, GroupedArgs &g, int op, const Sizes &z, const int32_t *offs, int n_out, int red, bool f32,
                 int &blocks, bool &segments, long long &tiles) {
    GroupedOut &o = g.o;
    o.offs = offs;
    o.E = z.E;
    o.rows = z.rows;
    o.n_out = n_out;
    o.m_dense = 1;
    o.red = red;
    o.f32 = f32;
    o.segment = f32 ? kExactSegment : segment_of(false, 16);
    o.wait = wait_cycles(red / kBK + 1);
    const int sms = op_num_sms();
    o.err = op_error_word();
    if (sms < 2 || o.err == nullptr) return op_fail(MOE_ERR_CUDA, "%s: no usable current device", name);
    segments = red > o.segment;
    blocks = choose_tiles(g, op, segments && op != kDgradTwo, sms);
    tiles = ((long long)z.rows / o.tile_rows + std::min(z.E, z.rows)) * o.col_tiles;
    if (tiles > (1ll << 30)) return op_fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^30 output tiles", name);
    return MOE_OK;
}

// [E, n, k] in boxes of 64 x `high`, and [rows, c] in boxes of 64 steps x 16, 32, .. rows
CUresult weights_map(CUtensorMap *m, const void *w, uint64_t k, uint64_t n, uint64_t e, uint32_t high) {
    return op_encode(m, {CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, w, {k, n, e}, {k * 2, n * k * 2}, {64, high, 1},
                         CU_TENSOR_MAP_SWIZZLE_128B});
}
CUresult rows_maps(CUtensorMap *m, const void *x, uint64_t c, uint64_t rows, int tile_rows) {
    CUresult cr = CUDA_SUCCESS;
    for (int i = 0; i < tile_rows / 32 && cr == CUDA_SUCCESS; ++i)
        cr = op_encode(&m[i], {CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, {c, rows}, {c * 2}, {kBK, 16u * (i + 1)},
                               CU_TENSOR_MAP_SWIZZLE_128B});
    return cr;
}

template <int OP>
moe_status go(const char *name, const typename ArgsOf<OP>::type &g, CUresult cr, int blocks, bool segments, long long tiles,
              moe_stream_t stream) {
    if (cr != CUDA_SUCCESS) return op_fail(MOE_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", name, (int)cr);
    const dim3 grid(2u * (unsigned)std::min<long long>(op_num_sms() / 2, tiles));
    auto launch = [&](auto kernel, int which) -> cudaError_t {
        const cudaError_t ce = op_allow_smem(reinterpret_cast<const void *>(kernel), kSmemBytes, &g_attr[4 * (OP - kGated) + which]);
        return ce != cudaSuccess ? ce
                                 : launch_pdl_cluster(kernel, grid, dim3((unsigned)kThreads<OP>), (size_t)kSmemBytes,
                                                      reinterpret_cast<cudaStream_t>(stream), dim3(2, 1, 1), g);
    };
    if constexpr (OP == kDgradTwo) {
        if (segments && blocks == 2) return op_cuda(launch(grouped_kernel<OP, 2, false, true>, 3), name);
    }
    return op_cuda(segments      ? launch(grouped_kernel<OP, 1, false, true>, 0)
                   : blocks == 1 ? launch(grouped_kernel<OP, 1, false, false>, 1)
                                 : launch(grouped_kernel<OP, 2, false, false>, 2),
                   name);
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_grouped_gated_forward(const void *X, const void *Wg, const void *Wu, const int32_t *offs, int rows,
                                                int E, int I, int K, int act, float alpha, float limit, float beta, void *H,
                                                void *G, void *U, moe_stream_t stream) {
    using namespace moe;
    const char *name = "moe_grouped_gated_forward";
    const Sizes z{rows, E, I, K};
    moe_status st = check_sizes(name, z);
    if (st == MOE_OK) st = check_act(name, act, alpha, limit, beta);
    if (st != MOE_OK) return st;
    if ((G == nullptr) != (U == nullptr)) return op_fail(MOE_ERR_INVALID_ARG, "%s: G and U go together", name);
    if (rows == 0) return MOE_OK;
    const uint64_t out = 2ull * rows * I, w = 2ull * E * I * K;
    const Buffer all[] = {{H, out}, {G, out}, {U, out}, {X, 2ull * rows * K}, {Wg, w}, {Wu, w}};
    const Buffer some[] = {all[0], all[3], all[4], all[5]};
    st = G ? check_buffers(name, all, 3, 6, offs, E) : check_buffers(name, some, 1, 4, offs, E);
    if (st != MOE_OK) return st;
    GatedArgs g = {};
    g.gated = {static_cast<bf16 *>(G), static_cast<bf16 *>(U), nullptr, nullptr, I, act, alpha, limit, beta};
    g.o.out = H;
    int blocks;
    bool segments;
    long long tiles;
    st = start(name, g, kGated, z, offs, 2 * ((I + kGranule - 1) / kGranule * kGranule), K, false, blocks, segments, tiles);
    if (st != MOE_OK) return st;
    CUresult cr = weights_map(&g.map_a, Wg, K, I, E, kGranule);
    if (cr == CUDA_SUCCESS) cr = weights_map(&g.map_a2, Wu, K, I, E, kGranule);
    if (cr == CUDA_SUCCESS) cr = rows_maps(g.map_b, X, K, rows, g.o.tile_rows);
    return go<kGated>(name, g, cr, blocks, segments, tiles, stream);
}

extern "C" moe_status moe_grouped_gated_backward(const void *dY, const void *Wd, const void *G, const void *U,
                                                 const int32_t *offs, int rows, int E, int I, int K, int act, float alpha,
                                                 float limit, float beta, void *dG, void *dU, moe_stream_t stream) {
    using namespace moe;
    const char *name = "moe_grouped_gated_backward";
    const Sizes z{rows, E, I, K};
    moe_status st = check_sizes(name, z);
    if (st == MOE_OK) st = check_act(name, act, alpha, limit, beta);
    if (st != MOE_OK || rows == 0) return st;
    const uint64_t of_i = 2ull * rows * I;
    const Buffer all[] = {{dG, of_i}, {dU, of_i}, {G, of_i}, {U, of_i}, {dY, 2ull * rows * K}, {Wd, 2ull * E * I * K}};
    st = check_buffers(name, all, 2, 6, offs, E);
    if (st != MOE_OK) return st;
    GatedArgs g = {};
    g.gated = {static_cast<bf16 *>(dG), static_cast<bf16 *>(dU), static_cast<const bf16 *>(G), static_cast<const bf16 *>(U),
               I, act, alpha, limit, beta};
    int blocks;
    bool segments;
    long long tiles;
    st = start(name, g, kGatedBack, z, offs, I, K, false, blocks, segments, tiles);
    if (st != MOE_OK) return st;
    CUresult cr = weights_map(&g.map_a, Wd, I, K, E, kBK);
    if (cr == CUDA_SUCCESS) cr = rows_maps(g.map_b, dY, K, rows, g.o.tile_rows);
    return go<kGatedBack>(name, g, cr, blocks, segments, tiles, stream);
}

extern "C" moe_status moe_grouped_gated_dgrad(const void *dG, const void *dU, const void *Wg, const void *Wu,
                                              const int32_t *offs, int rows, int E, int I, int K, int out_dtype, void *dX,
                                              moe_stream_t stream) {
    using namespace moe;
    const char *name = "moe_grouped_gated_dgrad";
    const Sizes z{rows, E, I, K};
    moe_status st = check_sizes(name, z);
    if (st != MOE_OK) return st;
    if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_F32)
        return op_fail(MOE_ERR_INVALID_ARG, "%s: unknown out_dtype %d", name, out_dtype);
    if (rows == 0) return MOE_OK;
    const bool f32 = out_dtype == MOE_DTYPE_F32;
    const uint64_t of_i = 2ull * rows * I, w = 2ull * E * I * K;
    const Buffer all[] = {{dX, (f32 ? 4ull : 2ull) * rows * K}, {dG, of_i}, {dU, of_i}, {Wg, w}, {Wu, w}};
    st = check_buffers(name, all, 1, 5, offs, E);
    if (st != MOE_OK) return st;
    DgradTwoArgs g = {};
    g.o.out = dX;
    g.split = (I + kBK - 1) / kBK * kBK;
    int blocks;
    bool segments;
    long long tiles;
    st = start(name, g, kDgradTwo, z, offs, K, 2 * g.split, f32, blocks, segments, tiles);
    if (st != MOE_OK) return st;
    CUresult cr = weights_map(&g.map_a, Wg, K, I, E, kBK);
    if (cr == CUDA_SUCCESS) cr = weights_map(&g.map_a2, Wu, K, I, E, kBK);
    if (cr == CUDA_SUCCESS) cr = rows_maps(g.map_b, dG, I, rows, g.o.tile_rows);
    if (cr == CUDA_SUCCESS) cr = rows_maps(g.map_b2, dU, I, rows, g.o.tile_rows);
    return go<kDgradTwo>(name, g, cr, blocks, segments, tiles, stream);
}
