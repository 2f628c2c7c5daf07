// The norms around a block, fused with its gate and the residual, and their gradients:
//
//   X' = a X + g * P,   P = F rf w_post   (F itself without a post-norm),   rf = (mean F^2 + eps)^-1/2
//   N  = X' rx w_pre,                                                       rx = (mean X'^2 + eps)^-1/2
// (w: the weight, or 1 + it).  From dX' and dN, with xh = X' rx and fh = F rf,
//   T  = dX' + rx (dN w_pre - xh mean(dN w_pre xh)),     dX = a T
//   dF = rf (T g w_post - fh mean(T g w_post fh))        (T g without a post-norm)
//   dw_pre = sum over rows of dN xh,  dw_post = of T g fh,  dg = T P summed over what shares a gate
//
// Bound by HBM: each tensor is read or written once.  A row belongs to a team of warps, 8 values of
// it to a thread (16 beyond 4096), so that its norms are sums over the team and its values stay in
// registers from the load to the store; the next row of a team is loaded while this one is
// computed.  The backward pass needs two sums over the team per row: X' and F's norms and
// mean(dN w_pre xh) come in the first one (the last up to a factor rx, known afterwards).  The
// weights' gradients are summed per thread over the rows of its team, then over the teams of a CTA
// in shared memory, then by a second kernel over the CTAs (one per SM, so that these partial sums
// are few): always in the same order, in fp32.
//
// A sum of squares beyond fp32 is taken again of values scaled by 2^-100.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "moe.h"
#include "op_host.h"

namespace moe {
namespace {

constexpr int kMaxH = 8192;
constexpr int kForwardThreads = 512;
// Threads of the backward kernel's CTAs (one per SM): as many as have registers for a thread's
// sums (24) and the row's values.
template <typename TX, typename TF>
constexpr int kBackwardThreads = sizeof(TX) + sizeof(TF) == 4 ? 1024 : sizeof(TX) + sizeof(TF) == 6 ? 768 : 512;
constexpr int kMaxTeams = 1024 / 32;
constexpr int kMaxCtas = 256;  // of the backward kernel: partial sums of the weights' gradients
constexpr float kDown = 0x1p-100f;

struct SandwichArgs {
    const void *x, *f;
    const void *dx, *dn;  // backward: X' and F in x and f
    const float *pre, *post, *gate;
    void *xo, *fo;        // forward: X', N; backward: dX, dF
    float *dgate;         // backward, a gate per token
    float *partial;       // backward: [grid][3][H]
    float alpha, eps, one;  // one: added to the weights
    int T, H, gate_kind, team;  // team: threads
};

// 8 consecutive values as loaded.
template <typename T>
struct Raw;
template <>
struct Raw<bf16> {
    uint4 v;
    __device__ __forceinline__ void load(const bf16 *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&o)[8]) const {
        o[0] = bf16_lo(v.x), o[1] = bf16_hi(v.x), o[2] = bf16_lo(v.y), o[3] = bf16_hi(v.y);
        o[4] = bf16_lo(v.z), o[5] = bf16_hi(v.z), o[6] = bf16_lo(v.w), o[7] = bf16_hi(v.w);
    }
    static __device__ __forceinline__ void store(bf16 *p, const float (&o)[8]) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
    }
};
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&o)[8]) const {
        o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&o)[8]) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(o[4], o[5], o[6], o[7]);
    }
};

// Sums over a team, in all its threads.  slots: [2][16][3] of the team; two sums in a row use
// different halves, so one barrier each is enough: who writes a half again has passed the barrier
// of the sum between, which everyone reaches after reading.
struct Team {
    int threads, id, warps, warp;
    float *slots;
    int half;
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N]) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (warps == 1) return;
        float *s = slots + half * 48;
        half ^= 1;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) s[warp * 3 + i] = v[i];
        asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.0f;
        for (int w = 0; w < warps; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += s[w * 3 + i];
    }
};

__device__ __forceinline__ Team make_team(float *slots, int threads) {
    Team t;
    t.threads = threads;
    t.id = threadIdx.x / threads;
    t.warps = threads / 32;
    t.warp = (threadIdx.x - t.id * threads) / 32;
    t.slots = slots + t.id * 96;
    t.half = 0;
    return t;
}

__device__ __forceinline__ float inverse_root(float sum, float inv_h, float eps) { return 1.0f / sqrtf(sum * inv_h + eps); }

// V: groups of 8 values per thread, `team` threads apart.
template <typename TX, typename TF, int V>
__global__ void __launch_bounds__(kForwardThreads, 1) norm_forward_kernel(const SandwichArgs p) {
    __shared__ float slots[kMaxTeams * 96];
    Team team = make_team(slots, p.team);
    const int me = threadIdx.x - team.id * p.team, H = p.H;
    const int stride = gridDim.x * (blockDim.x / p.team);
    const float inv_h = 1.0f / H;
    const bool has_f = p.f != nullptr, has_pre = p.pre != nullptr, has_post = p.post != nullptr;
    float pre[V][8], post[V][8];
    bool in[V];
    pdl_wait();
    pdl_trigger();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = 8 * (me + i * p.team);
        in[i] = at < H;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            pre[i][j] = has_pre && in[i] ? p.pre[at + j] + p.one : 0.0f;
            post[i][j] = !in[i] ? 0.0f : has_post ? p.post[at + j] + p.one : 1.0f;
            // the channels' gate is one more factor of the weight
            if (in[i] && p.gate_kind == MOE_GATE_CHANNEL) post[i][j] *= p.gate[at + j];
        }
    }
    Raw<TX> xr[V];
    Raw<TF> fr[V];
    float gate = 1.0f;
    auto fetch = [&](int row) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const size_t at = (size_t)row * H + 8 * (me + i * p.team);
            if (row < p.T && in[i]) {
                xr[i].load(static_cast<const TX *>(p.x) + at);
                if (has_f) fr[i].load(static_cast<const TF *>(p.f) + at);
            } else {
                xr[i].zero();
                fr[i].zero();
            }
        }
        if (p.gate_kind == MOE_GATE_TOKEN && row < p.T) gate = p.gate[row];
    };
    int row = blockIdx.x * (blockDim.x / p.team) + team.id;
    fetch(row);
    for (; row < p.T; row += stride) {
        float x[V][8], f[V][8];
        const float g = gate;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            xr[i].get(x[i]);
            if (has_f) fr[i].get(f[i]);
        }
        fetch(row + stride < p.T ? row + stride : p.T);
        if (has_f) {
            float rf = 1.0f;
            if (has_post) {
                float ss[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss[0] = fmaf(f[i][j], f[i][j], ss[0]);
                team.sum(ss);
                rf = inverse_root(ss[0], inv_h, p.eps);
                if (!(ss[0] < INFINITY)) {
                    ss[0] = 0.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j) ss[0] = fmaf(f[i][j] * kDown, f[i][j] * kDown, ss[0]);
                    team.sum(ss);
                    rf = inverse_root(ss[0], inv_h, p.eps * kDown * kDown) * kDown;
                }
            }
            rf *= g;
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = fmaf(p.alpha, x[i][j], f[i][j] * rf * post[i][j]);
                if (in[i]) Raw<TX>::store(static_cast<TX *>(p.xo) + (size_t)row * H + 8 * (me + i * p.team), x[i]);
            }
        }
        if (has_pre) {
            float ss[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) ss[0] = fmaf(x[i][j], x[i][j], ss[0]);
            team.sum(ss);
            float rx = inverse_root(ss[0], inv_h, p.eps);
            if (!(ss[0] < INFINITY)) {
                ss[0] = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss[0] = fmaf(x[i][j] * kDown, x[i][j] * kDown, ss[0]);
                team.sum(ss);
                rx = inverse_root(ss[0], inv_h, p.eps * kDown * kDown) * kDown;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = x[i][j] * rx * pre[i][j];
                if (in[i]) Raw<TF>::store(static_cast<TF *>(p.fo) + (size_t)row * H + 8 * (me + i * p.team), x[i]);
            }
        }
    }
}

template <typename TX, typename TF, int V>
__global__ void __launch_bounds__(kBackwardThreads<TX, TF>, 1) norm_backward_kernel(const SandwichArgs p) {
    // the effective weights and the channels' gate, later the teams' sums: three arrays of H values, the first
    // four values of each group of 8 in one half, the other four in the other, so that a warp's loads have no bank conflicts
    extern __shared__ float4 smem[];
    __shared__ float slots[kMaxTeams * 96];
    Team team = make_team(slots, p.team);
    const int me = threadIdx.x - team.id * p.team, H = p.H;
    const int stride = gridDim.x * (blockDim.x / p.team);
    const float inv_h = 1.0f / H;
    const bool has_f = p.f != nullptr, has_pre = p.pre != nullptr, has_post = p.post != nullptr;
    const bool channel = p.gate_kind == MOE_GATE_CHANNEL, token = p.gate_kind == MOE_GATE_TOKEN;
    pdl_wait();
    pdl_trigger();
    const int groups = H / 8;
    for (int i = threadIdx.x; i < 2 * groups; i += blockDim.x) {  // i: group of 4 values
        const int to = (i & 1) * groups + i / 2;
        auto four = [&](const float *w, float otherwise, float more) {
            if (w == nullptr) return make_float4(otherwise, otherwise, otherwise, otherwise);
            const float4 v = reinterpret_cast<const float4 *>(w)[i];
            return make_float4(v.x + more, v.y + more, v.z + more, v.w + more);
        };
        smem[to] = four(p.pre, 0.0f, p.one);
        smem[2 * groups + to] = four(p.post, 1.0f, p.one);
        smem[4 * groups + to] = four(channel ? p.gate : nullptr, 1.0f, 0.0f);
    }
    auto weights = [&](int which, int i, float (&w)[8]) {
        const int g = me + i * p.team;
        const float4 *at = smem + 2 * which * groups + (g < groups ? g : 0);  // (values beyond H are zeros)
        const float4 a = at[0], b = at[groups];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    };
    bool in[V];
    float d_pre[V][8], d_post[V][8], d_gate[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        in[i] = 8 * (me + i * p.team) < H;
#pragma unroll
        for (int j = 0; j < 8; ++j) d_pre[i][j] = d_post[i][j] = d_gate[i][j] = 0.0f;
    }
    __syncthreads();

    int row = blockIdx.x * (blockDim.x / p.team) + team.id;
    for (; row < p.T; row += stride) {
        Raw<TX> xr[V], dxr[V];
        Raw<TF> fr[V], dnr[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const size_t at = (size_t)row * H + 8 * (me + i * p.team);
            xr[i].zero(), dxr[i].zero(), fr[i].zero(), dnr[i].zero();
            if (in[i] && has_pre) xr[i].load(static_cast<const TX *>(p.x) + at), dnr[i].load(static_cast<const TF *>(p.dn) + at);
            if (in[i] && has_f) fr[i].load(static_cast<const TF *>(p.f) + at);
            if (in[i] && p.dx != nullptr) dxr[i].load(static_cast<const TX *>(p.dx) + at);
        }
        const float g = token ? p.gate[row] : 1.0f;
        float w[8], a[8], b[8];
        // the squares of X' and F, and dN w_pre X'
        float sx = 1.0f, sf = 1.0f, s[3];
        auto sums = [&]() {
            s[0] = s[1] = s[2] = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (has_pre) {
                    weights(0, i, w);
                    xr[i].get(a);
                    dnr[i].get(b);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float x = a[j] * sx;
                        s[0] = fmaf(x, x, s[0]);
                        s[2] = fmaf(b[j] * w[j], x, s[2]);
                    }
                }
                if (has_post) {
                    fr[i].get(a);
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[1] = fmaf(a[j] * sf, a[j] * sf, s[1]);
                }
            }
            team.sum(s);
        };
        sums();
        if (!(s[0] < INFINITY) || !(s[1] < INFINITY)) {
            if (!(s[0] < INFINITY)) sx = kDown;
            if (!(s[1] < INFINITY)) sf = kDown;
            sums();
        }
        const float rxs = inverse_root(s[0], inv_h, p.eps * sx * sx), rx = rxs * sx, mean = rxs * s[2] * inv_h;
        const float rf = has_post ? inverse_root(s[1], inv_h, p.eps * sf * sf) * sf : 1.0f;
        float t[V][8], m[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            dxr[i].get(t[i]);
            if (has_pre) {
                weights(0, i, w);
                xr[i].get(a);
                dnr[i].get(b);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float xh = a[j] * rx;
                    d_pre[i][j] = fmaf(b[j], xh, d_pre[i][j]);
                    t[i][j] = fmaf(rx, fmaf(-xh, mean, b[j] * w[j]), t[i][j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = has_f ? p.alpha * t[i][j] : t[i][j];
            if (in[i]) Raw<TX>::store(static_cast<TX *>(p.xo) + (size_t)row * H + 8 * (me + i * p.team), a);
            if (!has_f) continue;
            fr[i].get(a);
            weights(1, i, w);
            if (channel) {  // from here t is T times the gate
                weights(2, i, b);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    d_gate[i][j] = fmaf(t[i][j], a[j] * rf * w[j], d_gate[i][j]);
                    t[i][j] *= b[j];
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float fh = a[j] * rf;
                m[0] = fmaf(t[i][j] * w[j], fh, m[0]);
                t[i][j] *= g;
                d_post[i][j] = fmaf(t[i][j], fh, d_post[i][j]);
            }
        }
        if (!has_f) continue;
        float mean_f = 0.0f;
        if (has_post || token) {
            team.sum(m);
            if (token && me == 0 && p.dgate != nullptr) p.dgate[row] = m[0];
            mean_f = has_post ? g * m[0] * inv_h : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            fr[i].get(a);
            weights(1, i, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = rf * (has_post ? fmaf(-a[j] * rf, mean_f, t[i][j] * w[j]) : t[i][j]);
            if (in[i]) Raw<TF>::store(static_cast<TF *>(p.fo) + (size_t)row * H + 8 * (me + i * p.team), a);
        }
    }

    // the teams' sums one after the other, then this CTA's
    const int teams = blockDim.x / p.team;
    __syncthreads();
    for (int k = 0; k < teams; ++k) {
        if (team.id == k) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!in[i]) continue;
                auto add = [&](float4 *at, const float *d) {
                    const float4 v = k ? *at : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    *at = make_float4(v.x + d[0], v.y + d[1], v.z + d[2], v.w + d[3]);
                };
                float4 *at = smem + me + i * p.team;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    add(at + h * groups, d_pre[i] + 4 * h);
                    add(at + (2 + h) * groups, d_post[i] + 4 * h);
                    if (channel) add(at + (4 + h) * groups, d_gate[i] + 4 * h);
                }
            }
        }
        __syncthreads();
    }
    float4 *mine = reinterpret_cast<float4 *>(p.partial + (size_t)blockIdx.x * 3 * H);
    for (int i = threadIdx.x; i < 2 * groups; i += blockDim.x) {
        const int from = (i & 1) * groups + i / 2;
        mine[i] = smem[from];
        mine[2 * groups + i] = smem[2 * groups + from];
        if (channel) mine[4 * groups + i] = smem[4 * groups + from];
    }
}

// The CTAs' sums, one column of one result per lane of a warp row.
constexpr int kSumRows = 8;
__global__ void __launch_bounds__(32 * kSumRows) norm_sum_kernel(const float *partial, int parts, int H, float *d_pre,
                                                                 float *d_post, float *d_gate) {
    __shared__ float s[kSumRows][33];
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane, which = blockIdx.y;
    float *out = which == 0 ? d_pre : which == 1 ? d_post : d_gate;
    pdl_wait();
    pdl_trigger();
    if (out == nullptr) return;
    float v = 0.0f;
    if (col < H)
        for (int i = r; i < parts; i += kSumRows) v += partial[((size_t)i * 3 + which) * H + col];
    s[r][lane] = v;
    __syncthreads();
    if (r != 0 || col >= H) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumRows; ++i) v += s[i][lane];
    out[col] = v;
}

OpDone g_attr[8];

int groups_of(int H, int threads) { return H > 8 * threads ? 2 : 1; }
int backward_threads(int x_dtype, int f_dtype) {
    if (x_dtype == MOE_DTYPE_F32 && f_dtype == MOE_DTYPE_F32) return kBackwardThreads<float, float>;
    return x_dtype == f_dtype ? kBackwardThreads<bf16, bf16> : kBackwardThreads<float, bf16>;
}

// Teams of several warps have a named barrier each, of 15.
int most_teams(int team) { return team > 32 ? 15 : kMaxTeams; }

// Threads per team and teams per CTA: as many as fit, fewer where rows would leave SMs without one.
void shape(int T, int H, int sms, int threads, int &team, int &teams) {
    const int per = 8 * groups_of(H, threads);
    team = 32 * ((H + 32 * per - 1) / (32 * per));
    teams = std::max(1, std::min(std::min(threads / team, most_teams(team)), (T + sms - 1) / sms));
}

struct Buffer {
    const void *p;
    uint64_t bytes;
};

// No two of the buffers share bytes, unless neither is an output (the first n_out) or they are the
// same one read and written in place: same[i] is the input that output i may be.
bool apart(const Buffer *b, int n_out, int n, const int *same) {
    for (int i = 0; i < n_out; ++i)
        for (int j = i + 1; j < n; ++j)
            if (op_overlap(b[i].p, b[i].bytes, b[j].p, b[j].bytes) && !(same[i] == j && b[i].p == b[j].p)) return false;
    return true;
}

moe_status check(const char *op, int T, int H, int x_dtype, int f_dtype, int kind, int gate_kind, const float *gate,
                 float alpha, float eps, bool has_f, const float *post, const float *pre) {
    if (T < 0 || H < 1) return op_fail(MOE_ERR_INVALID_ARG, "%s: need T >= 0, H >= 1", op);
    for (int d : {x_dtype, f_dtype})
        if (d != MOE_DTYPE_BF16 && d != MOE_DTYPE_F32) return op_fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype %d", op, d);
    if (kind != MOE_NORM_RMS && kind != MOE_NORM_GEMMA) return op_fail(MOE_ERR_INVALID_ARG, "%s: unknown norm %d", op, kind);
    if (gate_kind != MOE_GATE_NONE && gate_kind != MOE_GATE_TOKEN && gate_kind != MOE_GATE_CHANNEL)
        return op_fail(MOE_ERR_INVALID_ARG, "%s: unknown gate %d", op, gate_kind);
    if (!(alpha - alpha == 0.0f) || !(eps >= 1e-30f && eps < INFINITY))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: need a finite residual_scale, eps >= 1e-30", op);
    if (T > 0 && (gate == nullptr) != (gate_kind == MOE_GATE_NONE))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: a gate needs its kind, and the other way round", op);
    // (the pointers of empty tensors may be NULL)
    if (T > 0 && !has_f && (post != nullptr || gate_kind != MOE_GATE_NONE))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: post_w and the gate belong to a block's result F", op);
    if (T > 0 && !has_f && pre == nullptr) return op_fail(MOE_ERR_INVALID_ARG, "%s: neither F nor pre_w: nothing to do", op);
    if (H % 8 || H > kMaxH) return op_fail(MOE_ERR_UNSUPPORTED, "%s: H %d: need a multiple of 8 up to %d", op, H, kMaxH);
    return MOE_OK;
}

bool aligned(std::initializer_list<const void *> all) {
    return std::all_of(all.begin(), all.end(), [](const void *p) { return op_aligned16(p); });
}

// fn(kernel) for the types and the groups per thread
template <template <typename, typename, int> class Kernel, typename Fn>
cudaError_t pick(int x_dtype, int f_dtype, int groups, Fn fn) {
    const int which = (x_dtype == MOE_DTYPE_F32) * 4 + (f_dtype == MOE_DTYPE_F32) * 2 + (groups - 1);
    switch (which) {
    case 0: return fn(Kernel<bf16, bf16, 1>::get(), which);
    case 1: return fn(Kernel<bf16, bf16, 2>::get(), which);
    case 2: return fn(Kernel<bf16, float, 1>::get(), which);
    case 3: return fn(Kernel<bf16, float, 2>::get(), which);
    case 4: return fn(Kernel<float, bf16, 1>::get(), which);
    case 5: return fn(Kernel<float, bf16, 2>::get(), which);
    case 6: return fn(Kernel<float, float, 1>::get(), which);
    default: return fn(Kernel<float, float, 2>::get(), which);
    }
}
using KernelFn = void (*)(const SandwichArgs);
template <typename TX, typename TF, int V>
struct Forward {
    static KernelFn get() { return norm_forward_kernel<TX, TF, V>; }
};
template <typename TX, typename TF, int V>
struct Backward {
    static KernelFn get() { return norm_backward_kernel<TX, TF, V>; }
};

size_t workspace_of(int T, int H) { return (size_t)std::max(1, std::min(T, kMaxCtas)) * 3 * H * sizeof(float); }

}  // namespace
}  // namespace moe

extern "C" moe_status moe_sandwich_norm(const void *X, const void *F, const float *pre_w, const float *post_w,
                                        const float *gate, int gate_kind, float residual_scale, float eps, int kind, int T,
                                        int H, int x_dtype, int f_dtype, void *X_out, void *N, moe_stream_t stream) {
    using namespace moe;
    const char *name = "moe_sandwich_norm";
    moe_status st = check(name, T, H, x_dtype, f_dtype, kind, gate_kind, gate, residual_scale, eps, F != nullptr, post_w, pre_w);
    if (st != MOE_OK || T == 0) return st;
    if (!X || (F == nullptr) != (X_out == nullptr) || (pre_w == nullptr) != (N == nullptr))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: need X, X_out where F is, N where pre_w is, and neither without", name);
    if (!aligned({X, F, pre_w, post_w, gate, X_out, N}))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", name);
    const uint64_t n = (uint64_t)T * H, xb = n * (x_dtype == MOE_DTYPE_F32 ? 4 : 2), fb = n * (f_dtype == MOE_DTYPE_F32 ? 4 : 2);
    const uint64_t wb = 4ull * H, gb = gate_kind == MOE_GATE_TOKEN ? 4ull * T : gate ? wb : 0;
    const Buffer all[] = {{X_out, X_out ? xb : 0}, {N, N ? fb : 0}, {X, xb}, {F, F ? fb : 0}, {pre_w, pre_w ? wb : 0},
                          {post_w, post_w ? wb : 0}, {gate, gb}};
    const int same[] = {2, 3};
    if (!apart(all, 2, 7, same)) return op_fail(MOE_ERR_INVALID_ARG, "%s: an output overlaps another tensor", name);
    const int sms = op_num_sms();
    if (sms < 1) return op_fail(MOE_ERR_CUDA, "%s: no usable current device", name);
    SandwichArgs a = {};
    a.x = X, a.f = F, a.pre = pre_w, a.post = post_w, a.gate = gate, a.xo = X_out, a.fo = N;
    a.alpha = residual_scale, a.eps = eps, a.one = kind == MOE_NORM_GEMMA ? 1.0f : 0.0f;
    a.T = T, a.H = H, a.gate_kind = gate_kind;
    int teams;
    shape(T, H, sms, kForwardThreads, a.team, teams);
    const unsigned grid = (unsigned)std::min<long long>(sms, ((long long)T + teams - 1) / teams);
    return op_cuda(pick<Forward>(x_dtype, f_dtype, groups_of(H, kForwardThreads), [&](KernelFn k, int) {
                       return launch_pdl(k, dim3(grid), dim3(a.team * teams), 0, reinterpret_cast<cudaStream_t>(stream), a);
                   }), name);
}

extern "C" moe_status moe_sandwich_norm_workspace(int T, int H, size_t *bytes) {
    using namespace moe;
    const char *name = "moe_sandwich_norm_workspace";
    if (T < 0 || H < 1 || bytes == nullptr) return op_fail(MOE_ERR_INVALID_ARG, "%s: need T >= 0, H >= 1, bytes", name);
    if (H % 8 || H > kMaxH) return op_fail(MOE_ERR_UNSUPPORTED, "%s: H %d: need a multiple of 8 up to %d", name, H, kMaxH);
    *bytes = workspace_of(T, H);
    return MOE_OK;
}

extern "C" moe_status moe_sandwich_norm_backward(const void *dX_out, const void *dN, const void *X_out, const void *F,
                                                 const float *pre_w, const float *post_w, const float *gate, int gate_kind,
                                                 float residual_scale, float eps, int kind, int T, int H, int x_dtype,
                                                 int f_dtype, void *dX, void *dF, float *dpre_w, float *dpost_w,
                                                 float *dgate, void *workspace, size_t workspace_bytes,
                                                 moe_stream_t stream) {
    using namespace moe;
    const char *name = "moe_sandwich_norm_backward";
    moe_status st = check(name, T, H, x_dtype, f_dtype, kind, gate_kind, gate, residual_scale, eps, F != nullptr, post_w, pre_w);
    if (st != MOE_OK) return st;
    if ((dpre_w && !pre_w) || (dpost_w && !post_w) || (dgate && gate_kind == MOE_GATE_NONE))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: a gradient of what was not given", name);
    if (T > 0 && (!dX || (F == nullptr) != (dF == nullptr) || (pre_w == nullptr) != (dN == nullptr) ||
                  (pre_w != nullptr && !X_out) || (!pre_w && !dX_out)))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: need dX, dF where F is, dN and X_out where pre_w is, dX_out without pre_w", name);
    if (!aligned({dX_out, dN, X_out, F, pre_w, post_w, gate, dX, dF, dpre_w, dpost_w, dgate, workspace}))
        return op_fail(MOE_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", name);
    const size_t need = workspace_of(T, H);
    if (!workspace || workspace_bytes < need) return op_fail(MOE_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed", name, need);
    const uint64_t n = (uint64_t)T * H, xb = n * (x_dtype == MOE_DTYPE_F32 ? 4 : 2), fb = n * (f_dtype == MOE_DTYPE_F32 ? 4 : 2);
    const uint64_t wb = 4ull * H, gb = gate_kind == MOE_GATE_TOKEN ? 4ull * T : wb;
    auto of = [](const void *p, uint64_t b) { return Buffer{p, p ? b : 0}; };
    const Buffer all[] = {of(dX, xb), of(dF, fb), of(dpre_w, wb), of(dpost_w, wb), of(dgate, gb), of(workspace, need),
                          of(dX_out, xb), of(dN, fb), of(X_out, xb), of(F, fb), of(pre_w, wb), of(post_w, wb), of(gate, gb)};
    const int same[] = {6, 7, -1, -1, -1, -1};
    if (!apart(all, 6, 13, same)) return op_fail(MOE_ERR_INVALID_ARG, "%s: an output overlaps another tensor", name);
    const int sms = op_num_sms();
    if (sms < 1) return op_fail(MOE_ERR_CUDA, "%s: no usable current device", name);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int grid = 0;
    if (T > 0) {
        SandwichArgs a = {};
        a.x = X_out, a.f = F, a.dx = dX_out, a.dn = dN, a.pre = pre_w, a.post = post_w, a.gate = gate;
        a.xo = dX, a.fo = dF, a.dgate = dgate, a.partial = static_cast<float *>(workspace);
        a.alpha = residual_scale, a.eps = eps, a.one = kind == MOE_NORM_GEMMA ? 1.0f : 0.0f;
        a.T = T, a.H = H, a.gate_kind = gate_kind;
        const int threads = backward_threads(x_dtype, f_dtype);
        int teams;
        shape(T, H, sms, threads, a.team, teams);
        grid = (int)std::min<long long>(std::min(sms, kMaxCtas), ((long long)T + teams - 1) / teams);
        const cudaError_t e = pick<Backward>(x_dtype, f_dtype, groups_of(H, threads), [&](KernelFn k, int which) {
            const cudaError_t ce = op_allow_smem(reinterpret_cast<const void *>(k), 3 * kMaxH * 4, &g_attr[which]);
            return ce != cudaSuccess ? ce : launch_pdl(k, dim3(grid), dim3(a.team * teams), 3ull * H * 4, s, a);
        });
        if (e != cudaSuccess) return op_cuda(e, name);
    }
    float *d_gate = gate_kind == MOE_GATE_CHANNEL ? dgate : nullptr;
    if (!dpre_w && !dpost_w && !d_gate) return MOE_OK;
    return op_cuda(launch_pdl(norm_sum_kernel, dim3((H + 31) / 32, 3), dim3(32 * kSumRows), 0, s,
                              static_cast<const float *>(workspace), grid, H, dpre_w, dpost_w, d_gate), name);
}
