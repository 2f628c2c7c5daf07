// The global norm of a list of gradients, and the gradients scaled by
//   c = min(1, max_norm / norm),   norm = sqrt(sum of all g^2)
// (c = 1 where the norm is not finite: the caller sees it and skips the step).
//
// Two kernels.  The first sums squares: 32 values per thread and chunk in fp32, those sums
// in fp64 (per thread, CTA, and over the CTAs in a fixed order, so the result is the same
// from call to call).  A thread whose fp32 sum overflowed, or is so small that squares may
// have been flushed, squares its values again in fp64.  In the second kernel every CTA adds
// up the first one's partial sums, then scales chunks; it goes through them from the last to
// the first, so that what the first kernel read last is still in L2.  Where the result goes
// to the gradients themselves and c is 1, nothing is written.
//
// Bound by HBM: one read to sum, one read (from L2 up to its size) and one write to scale.
//
// The tensors' addresses travel as kernel parameters (up to kMaxTensors per launch, more in
// further launches): no table is copied to the device and a captured call owns its list.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "moe.h"
#include "op_host.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 32;                       // values per thread and chunk
constexpr int kChunkElems = kThreads * kPerThread;   // 8192
constexpr int kCtasPerSm = 8;
constexpr int kMaxGrid = 2048;                       // partial sums per launch
constexpr int kMaxTensors = 960;

struct Entry {
    const void *grad;
    void *out;
    long long count;
};
template <int N>
struct ClipArgs {
    Entry t[N];
    int first[N];       // number of the tensor's first chunk
    uint32_t f32[(N + 31) / 32];  // bit set: fp32, else bf16
    int tensors, chunks;
    double *partial;    // norm kernel: this launch's sums; scale kernel: all of them
    int num_partial;
    float max_norm;
    float *norm;        // scale kernel: written by CTA 0 of the first launch (else NULL)
};
static_assert(sizeof(ClipArgs<kMaxTensors>) <= 32764, "kernel parameter space");

struct Chunk {
    const void *src;
    void *dst;
    int n;       // values in the chunk
    bool f32, vec;
};

template <int N>
__device__ __forceinline__ Chunk find(const ClipArgs<N> &p, int chunk) {
    int lo = 0, hi = p.tensors - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.first[mid] <= chunk)
            lo = mid;
        else
            hi = mid - 1;
    }
    const long long at = (long long)(chunk - p.first[lo]) * kChunkElems;
    Chunk c;
    c.f32 = p.f32[lo >> 5] >> (lo & 31) & 1u;
    const long long bytes = at * (c.f32 ? 4 : 2);
    c.src = static_cast<const char *>(p.t[lo].grad) + bytes;
    c.dst = static_cast<char *>(p.t[lo].out) + bytes;
    c.n = (int)min((long long)kChunkElems, p.t[lo].count - at);
    // full chunks of aligned tensors go in 16-byte accesses
    c.vec = c.n == kChunkElems && ((reinterpret_cast<uintptr_t>(c.src) | reinterpret_cast<uintptr_t>(c.dst)) & 15u) == 0;
    return c;
}

__device__ __forceinline__ float load1(const Chunk &c, int i) {
    return c.f32 ? static_cast<const float *>(c.src)[i]
                 : __bfloat162float(static_cast<const bf16 *>(c.src)[i]);
}

// Sum of squares of one thread's values, as a double.
template <int W>
__device__ __forceinline__ double squares(const uint32_t (&w)[W], bool f32) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if (f32) {
            const float v = __uint_as_float(w[i]);
            s[i & 3] = fmaf(v, v, s[i & 3]);
            any |= w[i] << 1;
        } else {
            const float a = bf16_lo(w[i]), b = bf16_hi(w[i]);
            s[i & 1] = fmaf(a, a, s[i & 1]);
            s[2 + (i & 1)] = fmaf(b, b, s[2 + (i & 1)]);
            any |= w[i] & 0x7fff7fffu;
        }
    }
    const float t = (s[0] + s[1]) + (s[2] + s[3]);
    // 2^-80: what a flushed or subnormal square (< 2^-126 each) could add is far below 2^-24 of it
    if ((t >= 8.271806e-25f && t <= 3.0e38f) || any == 0) return (double)t;
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if (f32) {
            const double v = __uint_as_float(w[i]);
            d += v * v;
        } else {
            const double a = bf16_lo(w[i]), b = bf16_hi(w[i]);
            d += a * a + b * b;
        }
    }
    return d;
}

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double s[kThreads / 32];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    double r = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) r += s[i];
    return r;
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ ClipArgs<N> p) {
    pdl_wait();
    pdl_trigger();
    double sum = 0.0;
    for (int chunk = blockIdx.x; chunk < p.chunks; chunk += gridDim.x) {
        const Chunk c = find(p, chunk);
        if (c.vec) {
            const uint4 *src = static_cast<const uint4 *>(c.src) + threadIdx.x;
            if (c.f32) {
                uint32_t w[32];
#pragma unroll
                for (int j = 0; j < 8; ++j) reinterpret_cast<uint4 *>(w)[j] = src[j * kThreads];
                sum += squares(w, true);
            } else {
                uint32_t w[16];
#pragma unroll
                for (int j = 0; j < 4; ++j) reinterpret_cast<uint4 *>(w)[j] = src[j * kThreads];
                sum += squares(w, false);
            }
        } else {
            uint32_t w[kPerThread];
#pragma unroll
            for (int j = 0; j < kPerThread; ++j) {
                const int i = threadIdx.x + j * kThreads;
                w[j] = i < c.n ? __float_as_uint(load1(c, i)) : 0u;
            }
            sum += squares(w, true);
        }
    }
    const double total = block_sum(sum);
    if (threadIdx.x == 0) p.partial[blockIdx.x] = total;
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ ClipArgs<N> p) {
    pdl_wait();
    pdl_trigger();
    double sum = 0.0;
    for (int i = threadIdx.x; i < p.num_partial; i += kThreads) sum += p.partial[i];
    const double norm = sqrt(block_sum(sum));
    if (p.norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = (float)norm;
    // a NaN or an infinity among the gradients: they pass through
    const bool clip = norm > (double)p.max_norm && norm <= 1.7e308;
    const float scale = clip ? (float)((double)p.max_norm / norm) : 1.0f;
    for (int chunk = p.chunks - 1 - (int)blockIdx.x; chunk >= 0; chunk -= gridDim.x) {
        const Chunk c = find(p, chunk);
        if (!clip && c.src == c.dst) continue;
        if (c.vec) {
            const uint4 *src = static_cast<const uint4 *>(c.src) + threadIdx.x;
            uint4 *dst = static_cast<uint4 *>(c.dst) + threadIdx.x;
            if (c.f32) {
                uint4 w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = src[j * kThreads];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float4 f = *reinterpret_cast<float4 *>(&w[j]);
                    f.x *= scale;
                    f.y *= scale;
                    f.z *= scale;
                    f.w *= scale;
                    __stcs(reinterpret_cast<float4 *>(dst + j * kThreads), f);
                }
            } else {
                uint4 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = src[j * kThreads];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t *x = reinterpret_cast<uint32_t *>(&w[j]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = pack_bf16x2(bf16_lo(x[k]) * scale, bf16_hi(x[k]) * scale);
                    __stcs(dst + j * kThreads, w[j]);
                }
            }
        } else {
            for (int i = threadIdx.x; i < c.n; i += kThreads) {
                const float v = load1(c, i) * scale;
                if (c.f32)
                    static_cast<float *>(c.dst)[i] = v;
                else
                    static_cast<bf16 *>(c.dst)[i] = __float2bfloat16_rn(v);
            }
        }
    }
}

// One launch's share of the list; -1: a count whose chunks do not fit an int.
template <int N>
int fill(ClipArgs<N> &a, const moe_grad *g, int n) {
    long long chunks = 0;
    a.tensors = 0;
    for (int i = 0; i < n; ++i) {
        if (g[i].count == 0) continue;
        const int k = a.tensors++;
        a.t[k] = {g[i].grad, g[i].out, g[i].count};
        a.first[k] = (int)chunks;
        if (g[i].dtype == MOE_DTYPE_F32) a.f32[k >> 5] |= 1u << (k & 31);
        chunks += (g[i].count + kChunkElems - 1) / kChunkElems;
        if (chunks > (1ll << 30)) return -1;
    }
    a.chunks = (int)chunks;
    return a.chunks;
}

int launches_of(int count) { return std::max(1, (count + kMaxTensors - 1) / kMaxTensors); }

template <int N>
moe_status run(const moe_grad *grads, int count, float max_norm, float *norm, double *partial, int sms, cudaStream_t s) {
    const char *op = "moe_clip_grad_norm";
    const int launches = launches_of(count), most = std::min(kMaxGrid, kCtasPerSm * sms);
    int used = 0;
    for (int pass = 0; pass < 2; ++pass)
        for (int l = 0; l < launches; ++l) {
            ClipArgs<N> a = {};
            const int at = l * kMaxTensors;
            if (fill(a, grads + at, std::min(kMaxTensors, count - at)) < 0)
                return op_fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^43 values in one launch", op);
            const int grid = std::max(1, std::min(a.chunks, most));
            a.max_norm = max_norm;
            cudaError_t e;
            if (pass == 0) {
                a.partial = partial + used;
                used += grid;
                e = launch_pdl(grad_norm_kernel<N>, dim3(grid), dim3(kThreads), 0, s, a);
            } else {
                a.partial = partial;
                a.num_partial = used;
                a.norm = l == 0 ? norm : nullptr;
                e = launch_pdl(grad_scale_kernel<N>, dim3(grid), dim3(kThreads), 0, s, a);
            }
            if (e != cudaSuccess) return op_cuda(e, op);
        }
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_clip_workspace(int count, size_t *bytes) {
    using namespace moe;
    if (count < 0 || bytes == nullptr) return op_fail(MOE_ERR_INVALID_ARG, "moe_clip_workspace: need count >= 0 and bytes");
    *bytes = sizeof(double) * kMaxGrid * (size_t)launches_of(count);
    return MOE_OK;
}

extern "C" moe_status moe_clip_grad_norm(const moe_grad *grads, int count, float max_norm, float *norm, void *workspace,
                                         size_t workspace_bytes, moe_stream_t stream) {
    using namespace moe;
    const char *op = "moe_clip_grad_norm";
    if (count < 0 || (count > 0 && grads == nullptr) || norm == nullptr || workspace == nullptr)
        return op_fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer or a negative count", op);
    if (!(max_norm > 0.0f)) return op_fail(MOE_ERR_INVALID_ARG, "%s: max_norm must be positive", op);
    size_t need = 0;
    moe_clip_workspace(count, &need);
    if (workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u) || (reinterpret_cast<uintptr_t>(norm) & 3u))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: needs a 16-byte aligned workspace of %zu bytes and an aligned norm", op, need);
    for (int i = 0; i < count; ++i) {
        const moe_grad &g = grads[i];
        if (g.dtype != MOE_DTYPE_BF16 && g.dtype != MOE_DTYPE_F32)
            return op_fail(MOE_ERR_INVALID_ARG, "%s: tensor %d: unknown dtype %d", op, i, g.dtype);
        const uintptr_t mask = g.dtype == MOE_DTYPE_F32 ? 3u : 1u;
        if (g.count < 0 || (g.count > 0 && (!g.grad || !g.out)) ||
            ((reinterpret_cast<uintptr_t>(g.grad) | reinterpret_cast<uintptr_t>(g.out)) & mask))
            return op_fail(MOE_ERR_INVALID_ARG, "%s: tensor %d: a NULL or misaligned pointer, or a negative count", op, i);
    }
    const int sms = op_num_sms();
    if (sms < 1) return op_fail(MOE_ERR_CUDA, "%s: no usable current device", op);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    double *partial = static_cast<double *>(workspace);
    // short lists: a small parameter block (launches copy it)
    return count <= 64 ? run<64>(grads, count, max_norm, norm, partial, sms, s)
                       : run<kMaxTensors>(grads, count, max_norm, norm, partial, sms, s);
}
