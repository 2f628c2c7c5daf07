// Block-scaled (OCP microscaling) quantisation and its inverse.
//
// Per block of 32 consecutive values along a row, with a = max |x|:
//   scale byte  c = max(floor(log2 a) - emax + 127, 0)      (emax: 2 for E2M1, 8 for E4M3)
//   codes       rne_saturate(x * 2^(127 - c))               (multiplying by a power of two is exact)
// floor(log2 a) is the exponent field of a; a zero or subnormal a gives c = 0.  A block
// that holds an infinity or a NaN gets c = 255 (NaN) and zero codes: all of it decodes to
// NaN, as a sum over it would be.
//
// Bound by HBM: one read of the tensor, one write of codes and scales.  A CTA takes 32 rows
// x 256 columns; a lane loads 8 consecutive values (four lanes hold a block, so a warp's
// loads are contiguous) of four rows at once (64 rows per CTA: 28.2 against 26.7 us for 24576 x
// 2048 bf16; 16: slower everywhere; CTAs that walk the tiles with the next one in flight: 30.4).
// The instructions count as well, at a CTA per 700 cycles of an SM: without divisions, with one
// address for four rows, and bf16 values scaled in pairs, 64 x 1408 x 2048 values take 68.5
// instead of 79.9 us (of that 13 us because loads are not marked as streaming).  The scales lie
// block-major ([K / 32, rows]), across the rows' direction: they are collected in shared memory
// and leave as 32-byte runs.
// Measured on GB300, 64 x 1408 x 2048 values, one call in a row: bf16 to MXFP4 70.8 us, 6.6 TB/s,
// and back 67.3; to MXFP8 81.6 us, 6.9 TB/s, and back 79.6; fp32 to MXFP4 117 us, 7.1 TB/s (part
// of the tensor is still in L2), and back 136, 6.1 TB/s.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "moe.h"
#include "op_host.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 32;    // rows per CTA
constexpr int kCols = 256;   // columns per CTA: eight values per lane
constexpr int kPerWarp = kRows / (kThreads / 32);
static_assert(kRows == 32 && kCols == kThreads, "scales: a warp per block, a lane per row");

// Division of n < 2^31 by d <= 2^l, l >= 1 (and d > 2^(l - 1)): mul = floor(2^(31 + l) / d) + 1
// exceeds 2^(31 + l) / d by at most 1, that is n mul / 2^(31 + l) exceeds n / d by less than
// 2^-l <= 1 / d.  (A division by instructions costs each warp as much as a row's conversion.)
struct Divisor {
    uint32_t mul;
    int shift;  // l - 1; -1: d = 1
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return shift < 0 ? n : __umulhi(n, mul) >> shift; }
};
Divisor divisor(int d) {
    int l = 0;
    while ((1ll << l) < d) ++l;
    return {l == 0 ? 0u : (uint32_t)((1ull << (31 + l)) / (uint32_t)d + 1), l - 1};
}

struct MxArgs {
    const void *x;        // quantise: [slices, rows, K]; dequantise: unused
    void *out;            // dequantise: [slices, rows, K]
    uint8_t *codes, *scales;
    int rows, K;
    int row_tiles, col_tiles;
    Divisor by_rows, by_cols;  // by row_tiles, by col_tiles
};

struct Place {
    int slice, row0, col0;
};
__device__ __forceinline__ Place place(const MxArgs &p) {
    const uint32_t b = blockIdx.x, r = p.by_cols(b), slice = p.by_rows(r);
    return {(int)slice, (int)(r - slice * p.row_tiles) * kRows, (int)(b - r * p.col_tiles) * kCols};
}

// 8 values of a row
template <bool F32>
struct Eight {
    uint4 a, b;
    __device__ __forceinline__ void load(const void *x, size_t at) {
        if (F32) {
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const float *>(x) + at);
            a = __ldg(src);
            b = __ldg(src + 1);
        } else {
            a = __ldg(reinterpret_cast<const uint4 *>(static_cast<const bf16 *>(x) + at));
        }
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    // the exponent field of the largest magnitude among the 32 values of this lane and its three
    // neighbours, 255 if one is not finite (bf16: two magnitudes per word, maxima that keep a NaN)
    __device__ __forceinline__ int exponent() const {
        if (F32) {
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, w[j] & 0x7fffffffu);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            return (int)(m >> 23);
        }
        auto most = [](uint32_t x, uint32_t y) {
            uint32_t r;
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
            return r;
        };
        uint32_t m = most(most(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu), most(a.z & 0x7fff7fffu, a.w & 0x7fff7fffu));
        m = most(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = most(m, __shfl_xor_sync(0xffffffffu, m, 2));
        m = most(m, __byte_perm(m, m, 0x1032));
        return (int)(m >> 23);
    }
    // the values times 2^(127 - c), c <= 253.  Products of bf16 values stay bf16: exact but for
    // those below its normal range, which are zero as codes.
    __device__ __forceinline__ void scaled(int c, float (&v)[8]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, e = (uint32_t)(254 - c);
        if (F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]) * __uint_as_float(e << 23);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t x;
                asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w[i]), "r"((e << 7) * 0x10001u));
                v[2 * i] = bf16_lo(x);
                v[2 * i + 1] = bf16_hi(x);
            }
        }
    }
};

template <bool F32, bool FP4>
__global__ void __launch_bounds__(kThreads) mx_quantize_kernel(const MxArgs p) {
    __shared__ uint8_t s_scale[kCols / 32][kRows];
    pdl_trigger();
    const Place t = place(p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = t.col0 + 8 * lane;
    const bool in_cols = col < p.K;  // K is a multiple of 32: a block's four lanes agree
    const int first = t.row0 + warp * kPerWarp;  // the warp's rows
    const size_t at0 = ((size_t)t.slice * p.rows + first) * p.K + col;
    Eight<F32> in[kPerWarp];
#pragma unroll
    for (int i = 0; i < kPerWarp; ++i) {
        in[i].zero();
        if (in_cols && first + i < p.rows) in[i].load(p.x, at0 + (size_t)i * p.K);
    }
#pragma unroll
    for (int i = 0; i < kPerWarp; ++i) {
        const int ex = in[i].exponent();
        const bool finite = ex < 255;
        const int c = finite ? max(ex - (FP4 ? 2 : 8), 0) : 255;
        float v[8];
        in[i].scaled(min(c, 253), v);
        if ((lane & 3) == 0) s_scale[lane >> 2][warp * kPerWarp + i] = (uint8_t)c;
        if (in_cols && first + i < p.rows) {
            const size_t at = at0 + (size_t)i * p.K;
            if (FP4) {
                uint32_t o;
                asm("{\n\t.reg .b8 a, b, c, d;\n\t"
                    "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
                    "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
                    "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
                    "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
                    "mov.b32 %0, {a, b, c, d};\n\t}"
                    : "=r"(o)
                    : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
                *reinterpret_cast<uint32_t *>(p.codes + at / 2) = finite ? o : 0u;
            } else {
                uint16_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(o[j]) : "f"(v[2 * j]), "f"(v[2 * j + 1]));
                *reinterpret_cast<uint2 *>(p.codes + at) =
                    finite ? make_uint2(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16) : make_uint2(0u, 0u);
            }
        }
    }
    __syncthreads();
    // scales: a warp per block, two rows per lane (K / 32 blocks and the rows may end inside)
    const int kb = threadIdx.x >> 5, r = 2 * lane, row = t.row0 + r;
    if (r < kRows && t.col0 + 32 * kb < p.K && row < p.rows) {
        uint8_t *dst = p.scales + ((size_t)t.slice * (p.K / 32) + t.col0 / 32 + kb) * p.rows + row;
        const uint8_t c0 = s_scale[kb][r], c1 = s_scale[kb][r + 1];
        if ((reinterpret_cast<uintptr_t>(dst) & 1u) == 0 && row + 1 < p.rows) {
            *reinterpret_cast<uint16_t *>(dst) = (uint16_t)(c0 | (uint16_t)c1 << 8);
        } else {
            dst[0] = c0;
            if (row + 1 < p.rows) dst[1] = c1;
        }
    }
}

// A lane's values: 8 in a row (16 bytes of bf16), or of fp32 twice 4, 128 columns apart (16 bytes
// each, so that a warp stores 512 in a row: 141 against 155 us; with streaming stores 137).
template <bool F32, bool FP4>
__global__ void __launch_bounds__(kThreads) mx_dequantize_kernel(const MxArgs p) {
    __shared__ uint8_t s_scale[kCols / 32][kRows];
    pdl_wait();
    pdl_trigger();
    const Place t = place(p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = t.col0 + (F32 ? 4 : 8) * lane;
    const bool in_cols = col < p.K, in_next = F32 && col + 128 < p.K;
    const int first = t.row0 + warp * kPerWarp;  // the warp's rows
    const size_t at0 = ((size_t)t.slice * p.rows + first) * p.K + col;
    uint2 code[kPerWarp];
#pragma unroll
    for (int i = 0; i < kPerWarp; ++i) {
        code[i] = make_uint2(0, 0);
        if (!in_cols || first + i >= p.rows) continue;
        const size_t at = at0 + (size_t)i * p.K;
        if (F32 && FP4) {
            const uint16_t *src = reinterpret_cast<const uint16_t *>(p.codes + at / 2);
            code[i].x = __ldcs(src) | (in_next ? (uint32_t)__ldcs(src + 32) << 16 : 0u);
        } else if (F32) {
            const uint32_t *src = reinterpret_cast<const uint32_t *>(p.codes + at);
            code[i] = make_uint2(__ldcs(src), in_next ? __ldcs(src + 32) : 0u);
        } else if (FP4) {
            code[i].x = __ldcs(reinterpret_cast<const uint32_t *>(p.codes + at / 2));
        } else {
            code[i] = __ldcs(reinterpret_cast<const uint2 *>(p.codes + at));
        }
    }
    {
        const int kb = threadIdx.x >> 5;
        if (t.col0 + 32 * kb < p.K && t.row0 + lane < p.rows)
            s_scale[kb][lane] = p.scales[((size_t)t.slice * (p.K / 32) + t.col0 / 32 + kb) * p.rows + t.row0 + lane];
    }
    __syncthreads();
    // 2^(c - 127): c = 0 is the subnormal 2^-127, c = 255 NaN
    auto factor = [&](int block, int i) {
        const uint32_t c = s_scale[block][warp * kPerWarp + i];
        return __uint_as_float(c == 255u ? 0x7fc00000u : c == 0u ? 0x00400000u : c << 23);
    };
#pragma unroll
    for (int i = 0; i < kPerWarp; ++i) {
        if (!in_cols || first + i >= p.rows) continue;
        uint32_t h[4];  // pairs of f16, which holds every element value exactly
        if (FP4) {
            asm("{\n\t.reg .b8 a, b, c, d;\n\t"
                "mov.b32 {a, b, c, d}, %4;\n\t"
                "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
                "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
                "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
                "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
                : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
                : "r"(code[i].x));
        } else {
            const uint16_t w[4] = {(uint16_t)code[i].x, (uint16_t)(code[i].x >> 16), (uint16_t)code[i].y,
                                   (uint16_t)(code[i].y >> 16)};
#pragma unroll
            for (int j = 0; j < 4; ++j) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[j]) : "h"(w[j]));
        }
        const float mul[2] = {factor(F32 ? lane >> 3 : lane >> 2, i), F32 ? factor(4 + (lane >> 3), i) : 0.f};
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
            v[2 * j] = f.x * mul[F32 ? j / 2 : 0];
            v[2 * j + 1] = f.y * mul[F32 ? j / 2 : 0];
        }
        const size_t at = at0 + (size_t)i * p.K;
        if (F32) {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at);
            __stcs(o, make_float4(v[0], v[1], v[2], v[3]));
            if (in_next) __stcs(o + 32, make_float4(v[4], v[5], v[6], v[7]));
        } else {
            __stcs(reinterpret_cast<uint4 *>(static_cast<bf16 *>(p.out) + at),
                   make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                              pack_bf16x2(v[6], v[7])));
        }
    }
}

moe_status check(const char *op, const void *x, int dtype, int slices, int rows, int K, int format, const void *codes,
                 const void *scales, MxArgs *a, unsigned *grid) {
    if (slices < 0 || rows < 0 || K < 1) return op_fail(MOE_ERR_INVALID_ARG, "%s: need slices >= 0, rows >= 0, K >= 1", op);
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32)
        return op_fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype %d", op, dtype);
    if (format != MOE_WEIGHTS_MXFP8 && format != MOE_WEIGHTS_MXFP4)
        return op_fail(MOE_ERR_INVALID_ARG, "%s: format must be MXFP8 or MXFP4", op);
    if (K % 32) return op_fail(MOE_ERR_UNSUPPORTED, "%s: K must be a multiple of 32 (K %d)", op, K);
    a->rows = rows;
    a->K = K;
    a->row_tiles = (int)((rows + (kRows - 1ll)) / kRows);
    a->col_tiles = (int)((K + (kCols - 1ll)) / kCols);
    a->by_rows = divisor(std::max(1, a->row_tiles));
    a->by_cols = divisor(a->col_tiles);
    const long long tiles = (long long)slices * a->row_tiles;
    if (tiles > 0 && tiles > ((1ll << 31) - 1) / a->col_tiles)
        return op_fail(MOE_ERR_UNSUPPORTED, "%s: the tensor is too large for one call", op);
    *grid = (unsigned)(tiles * a->col_tiles);
    if (*grid == 0) return MOE_OK;
    if (!x || !codes || !scales) return op_fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer", op);
    if (!op_aligned16(x) || !op_aligned16(codes) || !op_aligned16(scales))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", op);
    const uint64_t n = (uint64_t)slices * rows * K, x_bytes = n * (dtype == MOE_DTYPE_F32 ? 4 : 2);
    const uint64_t c_bytes = format == MOE_WEIGHTS_MXFP8 ? n : n / 2;
    if (op_overlap(x, x_bytes, codes, c_bytes) || op_overlap(x, x_bytes, scales, n / 32) ||
        op_overlap(codes, c_bytes, scales, n / 32))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: tensors overlap", op);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_mx_quantize(const void *X, int dtype, int slices, int rows, int K, int format, void *codes,
                                      uint8_t *scales, moe_stream_t stream) {
    using namespace moe;
    MxArgs a = {};
    unsigned grid = 0;
    const moe_status st = check("moe_mx_quantize", X, dtype, slices, rows, K, format, codes, scales, &a, &grid);
    if (st != MOE_OK || grid == 0) return st;
    a.x = X;
    a.codes = static_cast<uint8_t *>(codes);
    a.scales = scales;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // Not started before the kernel ahead has ended: it may write the tensor, and the loads (__ldg)
    // take it for constant while the kernel runs.  Loads without that, and an early start: 25 for 20.5
    // us (24576 x 2048 bf16; 384 rows 1.65 for 1.96), 64.9 for 57.0 with the MXFP4 product behind and
    // the next call's quantisation behind that, which then disturbs the product's last wave.
    void *args[] = {&a};
    auto go = [&](auto kernel) {
        return cudaLaunchKernel(reinterpret_cast<const void *>(kernel), dim3(grid), dim3(kThreads), args, 0, s);
    };
    const bool f32 = dtype == MOE_DTYPE_F32, fp4 = format == MOE_WEIGHTS_MXFP4;
    return op_cuda(f32 ? (fp4 ? go(mx_quantize_kernel<true, true>) : go(mx_quantize_kernel<true, false>))
                       : (fp4 ? go(mx_quantize_kernel<false, true>) : go(mx_quantize_kernel<false, false>)),
                   "moe_mx_quantize");
}

extern "C" moe_status moe_mx_dequantize(const void *codes, const uint8_t *scales, int format, int slices, int rows, int K,
                                        int dtype, void *X, moe_stream_t stream) {
    using namespace moe;
    MxArgs a = {};
    unsigned grid = 0;
    const moe_status st = check("moe_mx_dequantize", X, dtype, slices, rows, K, format, codes, scales, &a, &grid);
    if (st != MOE_OK || grid == 0) return st;
    a.out = X;
    a.codes = static_cast<uint8_t *>(const_cast<void *>(codes));
    a.scales = const_cast<uint8_t *>(scales);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, s, a); };
    const bool f32 = dtype == MOE_DTYPE_F32, fp4 = format == MOE_WEIGHTS_MXFP4;
    return op_cuda(f32 ? (fp4 ? go(mx_dequantize_kernel<true, true>) : go(mx_dequantize_kernel<true, false>))
                       : (fp4 ? go(mx_dequantize_kernel<false, true>) : go(mx_dequantize_kernel<false, false>)),
                   "moe_mx_dequantize");
}
