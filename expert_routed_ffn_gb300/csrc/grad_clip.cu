// The global norm of a list of gradients, and the gradients scaled by
//   c = min(1, max_norm / norm),   norm = sqrt(sum of all g^2)
// (c = 1 where a gradient is not finite: the caller sees it in the norm and skips the step; a norm
// that is finite but beyond fp32 is reported as an infinity, and c comes from its value).
//
// Two kernels, whose CTAs walk blocks of the list's values.  The first sums squares: per thread
// and step (up to 64 values) in fp32; over steps, threads and warps as unevaluated sums of two
// fp32 numbers; over CTAs in fp64, always in the same order.  (fp64 everywhere past the steps
// cost more than the memory: its units are few, 33 us for the second kernel of a list of 5
// million values.)  A step whose fp32 sum may have overflowed, or is so small that squares may
// have been flushed, is squared again in fp64.  In the second kernel every CTA adds up the
// first one's partial sums, then scales its blocks from the last to the first, so that what was
// read last is still in L2.  Where the result goes to the gradients themselves and c is 1,
// nothing is written.
//
// Bound by HBM: one read to sum, one read (from L2 up to its size) and one write to scale.
// Concurrent CTAs read neighbouring blocks; with one long run per CTA instead, 2.2 GB took 1022
// against 989 us.
//
// The tensors' addresses travel as kernel parameters (up to kMaxTensors per launch, more in
// further launches), with the tensor each CTA's first block is in: no table is copied to the
// device, a captured call owns its list, and a short list needs no search of the table, each
// step of which can be a miss of the constant cache.
#include <stdlib.h>

#include <algorithm>
#include <iterator>

#include "common.cuh"
#include "kernels.h"
#include "moe.h"
#include "op_host.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 2048;      // values: what blocks are made of
constexpr int kVecs = 8;          // 16-byte accesses per thread and step
constexpr int kCtasPerSm = 8;
constexpr int kMaxGrid = 1280;    // CTAs, and partial sums, per launch
constexpr int kMaxTensors = 960;

struct Entry {
    const void *grad;
    void *out;
    long long count;
};
template <int N>
struct ClipArgs {
    Entry t[N];
    int first[N + 1];             // number of the tensor's first chunk; the total
    uint32_t f32[(N + 31) / 32];  // bit set: fp32, else bf16
    uint16_t start[kMaxGrid];     // the tensor a CTA's first chunk is in
    int tensors, chunks, block;   // block: chunks of a block
    double *partial;    // norm kernel: this launch's sums; scale kernel: all of them
    int num_partial;
    float max_norm;
    float *norm;        // scale kernel: written by CTA 0 of the first launch (else NULL)
};
static_assert(sizeof(ClipArgs<kMaxTensors>) <= 32764, "kernel parameter space");

// The tensor that chunk `c`, the first of a CTA's block number `blk`, lies in
template <int N>
__device__ __forceinline__ int tensor_of(const ClipArgs<N> &p, int blk, int c) {
    if (blk < (int)gridDim.x) return p.start[blk];
    int lo = 0, hi = p.tensors - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.first[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// The part of the chunks [c0, c1) that lies in tensor k
struct Segment {
    const char *src;
    char *dst;
    int n;          // values
    bool f32, vec;  // vec: 16-byte accesses
};
template <int N>
__device__ __forceinline__ Segment segment(const ClipArgs<N> &p, int k, int c0, int c1) {
    const Entry &e = p.t[k];
    const int first = p.first[k], a = max(c0, first) - first, b = min(c1, p.first[k + 1]) - first;
    const long long at = (long long)a * kChunk;
    Segment s;
    s.f32 = p.f32[k >> 5] >> (k & 31) & 1u;
    s.n = (int)(min(e.count, (long long)b * kChunk) - at);
    s.src = static_cast<const char *>(e.grad) + at * (s.f32 ? 4 : 2);
    s.dst = static_cast<char *>(e.out) + at * (s.f32 ? 4 : 2);
    s.vec = ((reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst)) & 15u) == 0;
    return s;
}
__device__ __forceinline__ float load1(const Segment &s, int i) {
    return s.f32 ? reinterpret_cast<const float *>(s.src)[i] : __bfloat162float(reinterpret_cast<const bf16 *>(s.src)[i]);
}

// A running sum hi + lo, and what does not fit its range
struct Sum {
    float hi = 0.f, lo = 0.f;
    double far = 0.0;
    __device__ __forceinline__ void add(float t) {  // exact: hi + t = s + the rounding error
        const float s = hi + t, b = s - hi;
        lo += (hi - (s - b)) + (t - b);
        hi = s;
    }
};

// Add the squares of a step's values.
template <int W>
__device__ __forceinline__ void squares(const uint32_t (&w)[W], bool f32, Sum &sum) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t any = 0;
    if (f32) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float v = __uint_as_float(w[i]);
            s[i & 3] = fmaf(v, v, s[i & 3]);
            any |= w[i] << 1;
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float a = bf16_lo(w[i]), b = bf16_hi(w[i]);
            s[i & 1] = fmaf(a, a, s[i & 1]);
            s[2 + (i & 1)] = fmaf(b, b, s[2 + (i & 1)]);
            any |= w[i] & 0x7fff7fffu;
        }
    }
    const float t = (s[0] + s[1]) + (s[2] + s[3]);
    // from 2^-80 (what flushed or subnormal squares, < 2^-126 each, could add is far below 2^-24
    // of it) to 2^90 (2^37 of them do not overflow)
    if ((t >= 8.271806e-25f && t <= 1.2379400e27f) || any == 0) {
        sum.add(t);
        return;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const double a = f32 ? __uint_as_float(w[i]) : bf16_lo(w[i]), b = f32 ? 0.f : bf16_hi(w[i]);
        sum.far += a * a + b * b;
    }
}

// The CTA's sum, in thread 0
__device__ __forceinline__ double block_sum(Sum v) {
    __shared__ Sum s[kThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float hi = __shfl_xor_sync(0xffffffffu, v.hi, d), lo = __shfl_xor_sync(0xffffffffu, v.lo, d);
        v.add(hi);
        v.lo += lo;
    }
    if (__any_sync(0xffffffffu, !(v.far == 0.0))) {  // (a NaN too)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v.far += __shfl_xor_sync(0xffffffffu, v.far, d);
    }
    if (lane == 0) s[warp] = v;
    __syncthreads();
    if (threadIdx.x != 0) return 0.0;
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) {
        v.add(s[i].hi);
        v.lo += s[i].lo;
        if (!(s[i].far == 0.0)) v.far += s[i].far;
    }
    return (double)v.hi + (double)v.lo + v.far;
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ ClipArgs<N> p) {
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    Sum sum;
    for (int blk = blockIdx.x; (long long)blk * p.block < p.chunks; blk += gridDim.x) {
        const int c0 = blk * p.block, c1 = min(c0 + p.block, p.chunks);
        for (int k = tensor_of(p, blk, c0); k < p.tensors && p.first[k] < c1; ++k) {
            const Segment s = segment(p, k, c0, c1);
            int done = 0;  // values covered by whole vectors
            if (s.vec) {
                const uint4 *src = reinterpret_cast<const uint4 *>(s.src);
                const int per = s.f32 ? 4 : 8, nv = s.n / per;
                for (int base = 0; base < nv; base += kVecs * kThreads) {
                    uint32_t w[4 * kVecs];
#pragma unroll
                    for (int j = 0; j < kVecs; ++j) {
                        const int i = base + j * kThreads + tid;
                        reinterpret_cast<uint4 *>(w)[j] = i < nv ? src[i] : make_uint4(0, 0, 0, 0);
                    }
                    squares(w, s.f32, sum);
                }
                done = nv * per;
            }
            for (int base = done; base < s.n; base += 8 * kThreads) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = base + j * kThreads + tid;
                    w[j] = i < s.n ? __float_as_uint(load1(s, i)) : 0u;
                }
                squares(w, true, sum);
            }
        }
    }
    const double total = block_sum(sum);
    if (tid == 0) p.partial[blockIdx.x] = total;
}

// What the gradients are multiplied by: near, or where that is no normal fp32 number (norms of
// more than about 2^125 max_norm) far, which is 0 otherwise.
struct Factor {
    float near = 1.0f;
    double far = 0.0;
    bool clip = false;
};

// The norm and the factor from the sum of squares, with the exponent apart: the square of a
// value may be out of fp32's range, and fp64 square roots and quotients are slow here.
__device__ __forceinline__ Factor factor_of(double sum, float max_norm, float &norm) {
    const long long bits = __double_as_longlong(sum);
    const int ex = (int)(bits >> 52 & 0x7ff);
    Factor f;
    norm = 0.0f;
    if (sum == 0.0) return f;
    if (ex == 0x7ff) {  // a NaN or an infinity among the gradients: they pass through
        norm = (float)sum;
        return f;
    }
    const int e = ex - 1023, h = e >> 1;  // sum = m 2^(2 h), 1 <= m < 4
    const float root = sqrtf((float)__longlong_as_double((bits & 0xfffffffffffffll) | (long long)(1023 + e - 2 * h) << 52));
    norm = scalbnf(root, h);
    f.clip = norm > max_norm;
    if (!f.clip) return f;
    const int em = ilogbf(max_norm), t = em - h;            // max_norm may be subnormal
    const float q = scalbnf(max_norm, -em) / root;          // the factor is q 2^t, 1/2 < q < 2
    if (t >= -125)
        f.near = scalbnf(q, t);
    else  // t >= -149 - 147
        f.far = (double)q * __longlong_as_double((long long)(1023 + t) << 52);
    return f;
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ ClipArgs<N> p) {
    __shared__ Factor s_factor;
    const int tid = threadIdx.x;
    const int blocks = (p.chunks + p.block - 1) / p.block;
    pdl_wait();
    pdl_trigger();
    if (tid < 32) {
        double sum = 0.0;
        for (int i = tid; i < p.num_partial; i += 32) sum += p.partial[i];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        float norm;
        const Factor f = factor_of(sum, p.max_norm, norm);
        if (tid == 0) {
            s_factor = f;
            if (p.norm != nullptr && blockIdx.x == 0) *p.norm = norm;
        }
    }
    __syncthreads();
    const float scale = s_factor.near;
    const bool clip = s_factor.clip, is_far = s_factor.far != 0.0;
    if ((int)blockIdx.x >= blocks) return;
    for (int blk = ((blocks - 1 - (int)blockIdx.x) / (int)gridDim.x) * (int)gridDim.x + (int)blockIdx.x; blk >= 0; blk -= gridDim.x) {
        const int c0 = blk * p.block, c1 = min(c0 + p.block, p.chunks);
        for (int k = tensor_of(p, blk, c0); k < p.tensors && p.first[k] < c1; ++k) {
            const Segment s = segment(p, k, c0, c1);
            if (!clip && s.src == s.dst) continue;
            int done = 0;
            if (s.vec && !is_far) {
                const uint4 *src = reinterpret_cast<const uint4 *>(s.src);
                uint4 *dst = reinterpret_cast<uint4 *>(s.dst);
                const int per = s.f32 ? 4 : 8, nv = s.n / per;
                done = nv * per;
                for (int base = 0; base < nv; base += kVecs * kThreads) {
                    uint4 w[kVecs];
#pragma unroll
                    for (int j = 0; j < kVecs; ++j) {
                        const int i = base + j * kThreads + tid;
                        if (i < nv) w[j] = src[i];
                    }
#pragma unroll
                    for (int j = 0; j < kVecs; ++j) {
                        const int i = base + j * kThreads + tid;
                        uint32_t *x = reinterpret_cast<uint32_t *>(&w[j]);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            x[q] = s.f32 ? __float_as_uint(__uint_as_float(x[q]) * scale)
                                         : pack_bf16x2(bf16_lo(x[q]) * scale, bf16_hi(x[q]) * scale);
                        if (i < nv) __stcs(dst + i, w[j]);
                    }
                }
            }
            for (int i = done + tid; i < s.n; i += kThreads) {
                const float g = load1(s, i), v = is_far ? (float)((double)g * s_factor.far) : g * scale;
                if (s.f32)
                    reinterpret_cast<float *>(s.dst)[i] = v;
                else
                    reinterpret_cast<bf16 *>(s.dst)[i] = __float2bfloat16_rn(v);
            }
        }
    }
}

// A CTA's part of a tensor, and the chunks of a launch's tensors, are counted in an int
constexpr long long kMaxChunks = 1ll << 26;
long long chunks_of(const moe_grad &g) { return g.count == 0 ? 0 : (g.count - 1) / kChunk + 1; }

// One launch's share of the list (at most kMaxChunks); the grid.  Short lists: blocks of up
// to 8 chunks, as many CTAs as blocks; long ones: blocks of 4 (a thread's step of fp32 values),
// kCtasPerSm CTAs per SM.
template <int N>
int fill(ClipArgs<N> &a, const moe_grad *g, int n, int sms) {
    int chunks = 0;
    a.tensors = 0;
    for (int i = 0; i < n; ++i) {
        if (g[i].count == 0) continue;
        const int k = a.tensors++;
        a.t[k] = {g[i].grad, g[i].out, g[i].count};
        a.first[k] = chunks;
        if (g[i].dtype == MOE_DTYPE_F32) a.f32[k >> 5] |= 1u << (k & 31);
        chunks += (int)chunks_of(g[i]);
    }
    a.chunks = chunks;
    a.first[a.tensors] = a.chunks;
    const int most = std::min(kMaxGrid, kCtasPerSm * sms);
    a.block = a.chunks > 8 * most ? 4 : std::max(1, std::min(8, a.chunks / (2 * sms)));
    const int grid = std::max(1, std::min((a.chunks + a.block - 1) / a.block, most));
    for (int b = 0, k = 0; b < grid; ++b) {
        const int c = b * a.block;
        while (k + 1 < a.tensors && a.first[k + 1] <= c) ++k;
        a.start[b] = (uint16_t)k;
    }
    return grid;
}

int launches_of(int count) { return std::max(1, (count + kMaxTensors - 1) / kMaxTensors); }

template <int N>
moe_status run(const moe_grad *grads, int count, float max_norm, float *norm, double *partial, int sms, cudaStream_t s) {
    const int launches = launches_of(count);
    int used = 0;
    for (int pass = 0; pass < 2; ++pass)
        for (int l = 0; l < launches; ++l) {
            ClipArgs<N> a;
            std::fill(std::begin(a.f32), std::end(a.f32), 0u);
            const int at = l * kMaxTensors;
            const int grid = fill(a, grads + at, std::min(kMaxTensors, count - at), sms);
            a.max_norm = max_norm;
            a.partial = pass == 0 ? partial + used : partial;
            a.num_partial = used;
            a.norm = pass == 1 && l == 0 ? norm : nullptr;
            if (pass == 0) used += grid;
            const cudaError_t e = pass == 0 ? launch_pdl(grad_norm_kernel<N>, dim3(grid), dim3(kThreads), 0, s, a)
                                            : launch_pdl(grad_scale_kernel<N>, dim3(grid), dim3(kThreads), 0, s, a);
            if (e != cudaSuccess) return op_cuda(e, "moe_clip_grad_norm");
        }
    return MOE_OK;
}

// The bytes of a buffer
struct Range {
    uintptr_t begin, end;
};
bool operator<(const Range &a, const Range &b) { return a.begin < b.begin; }

// Whether a result shares bytes with another result, with a gradient that is not its own, or
// only in part with its own; or the norm or the workspace with any of them.  Blocks run in any
// order, so such a value might be scaled twice, or be summed after it was scaled.  `r`: room
// for `count` ranges.
bool lists_overlap(const moe_grad *grads, int count, Range norm, Range work, Range *r) {
    auto bytes = [](const void *p, const moe_grad &g) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        return Range{at, at + (uintptr_t)g.count * (g.dtype == MOE_DTYPE_F32 ? 4 : 2)};
    };
    auto meet = [](const Range &a, const Range &b) { return a.begin < b.end && b.begin < a.end; };
    int n = 0;
    for (int i = 0; i < count; ++i)
        if (grads[i].count > 0) r[n++] = bytes(grads[i].out, grads[i]);
    if (!std::is_sorted(r, r + n)) std::sort(r, r + n);
    for (int i = 1; i < n; ++i)
        if (r[i].begin < r[i - 1].end) return true;
    auto meets_result = [&](const Range &x) {  // the results are disjoint: only the last that begins before x ends
        const Range *after = std::lower_bound(r, r + n, Range{x.end, 0});
        return after != r && after[-1].end > x.begin;
    };
    if (meet(norm, work) || meets_result(norm) || meets_result(work)) return true;
    for (int i = 0; i < count; ++i) {
        if (grads[i].count == 0 || grads[i].grad == grads[i].out) continue;
        const Range x = bytes(grads[i].grad, grads[i]);
        if (meet(x, norm) || meet(x, work) || meets_result(x)) return true;
    }
    return false;
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
    for (int at = 0; at < count; at += kMaxTensors) {  // before anything is launched
        long long chunks = 0;
        for (int i = at; i < std::min(count, at + kMaxTensors); ++i)
            if (chunks_of(grads[i]) > kMaxChunks || (chunks += chunks_of(grads[i])) > kMaxChunks)
                return op_fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^37 values in %d tensors", op, kMaxTensors);
    }
    if (count > 0) {
        Range *room = static_cast<Range *>(malloc(sizeof(Range) * (size_t)count));
        if (room == nullptr) return op_fail(MOE_ERR_OOM, "%s: no host memory for a list of %d", op, count);
        const uintptr_t at = reinterpret_cast<uintptr_t>(norm), w = reinterpret_cast<uintptr_t>(workspace);
        const bool overlap = lists_overlap(grads, count, {at, at + sizeof(float)}, {w, w + need}, room);
        free(room);
        if (overlap)
            return op_fail(MOE_ERR_INVALID_ARG, "%s: tensors overlap (a result may only be its own gradient)", op);
    }
    const int sms = op_num_sms();
    if (sms < 1) return op_fail(MOE_ERR_CUDA, "%s: no usable current device", op);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    double *partial = static_cast<double *>(workspace);
    // short lists: a small parameter block (launches copy it)
    return count <= 64 ? run<64>(grads, count, max_norm, norm, partial, sms, s)
                       : run<kMaxTensors>(grads, count, max_norm, norm, partial, sms, s);
}
