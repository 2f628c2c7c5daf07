// The norms around a block, fused with its gate and the residual, and their gradients:
//
//   X' = a X + g * P,   P = F rf w_post   (F itself without a post-norm),   rf = (mean F^2 + eps)^-1/2
//   N  = X' rx w_pre,                                                       rx = (mean X'^2 + eps)^-1/2
// (w: the weight, or 1 + it).  From dX' and dN, with xh = X' rx and fh = F rf,
//   T  = dX' + rx (dN w_pre - xh mean(dN w_pre xh)),     dX = a T
//   dF = rf (T g w_post - fh mean(T g w_post fh))        (T g without a post-norm)
//   dw_pre = sum over rows of dN xh,  dw_post = of T g fh,  dg = T P summed over what shares a gate
//
// Bound by HBM: each tensor is read or written once.  A row belongs to a team of warps, 16 values of
// it to a thread (8 where it has no more for a warp), so that its norms are sums over the team and its
// values stay in registers from the load to the store; the next row of a team comes to shared
// memory by bulk copies meanwhile.  The backward pass needs two sums over the team per row: X' and
// F's norms and mean(dN w_pre xh) come in the first one (the last up to a factor rx, known
// afterwards).  The weights' gradients are summed per thread over the rows of its team, then over the
// teams of a CTA in shared memory, then by a second kernel over the CTAs: always in the same order, in fp32.
// There is one CTA per SM, so that these partial sums are few, and a multiple of that where a team would have
// more than 1024 rows; the second kernel keeps what its additions round off.  So the error is that of
// 1075 additions at most, 2^-13.9 of the sum of magnitudes, however many rows there are.
//
// A sum of squares beyond fp32 is taken again of values scaled by 2^-100.
//
// Measured on GB300 (captured into a graph, one call after the other on the same tensors):
//   forward, 8192 x 2048, fp32 stream, bf16 block   39 us, 5.1 TB/s; 65536 rows 247 us, 6.5 TB/s; bf16
//                              throughout 28.6 and 163 us.  A call has 8 us beside the copying: launch,
//                              weights, a team's first rows and last stores
//   backward, 16384 x 2048, bf16   85 us, 4.7 TB/s (a gate per channel: 106, registers spill): half of an SM's issue slots are taken, 46
//                              instructions per value of a warp's lane, and 16 warps wait for one
//                              another twice a row.  (With 8 values per thread and weights read across
//                              banks it took 203 us, without bank conflicts 109, with 768 threads of fewer
//                              registers 103.)  Rows beyond 4096 leave a CTA to one team, whose steps
//                              then wait for one another: 20000 x 6144 340 us, 4.3 TB/s, x 4104 330
//   without a block, 16384 x 2048, bf16   25 us (partly from L2), backward 66
//   one row of 2048            6.2 us
#include <algorithm>

#include "common.cuh"
#include "grouped.cuh"
#include "kernels.h"
#include "moe.h"
#include "op_host.h"

namespace moe {
namespace {

constexpr int kMaxH = 8192;
// Threads of a CTA, one per SM: as many as have the registers (backward with 640: 16384 x 2048 111 us
// for 86, spills; forward with 512: 8192 x 4104 96 us for 76, one team where there could be two).
constexpr int kForwardThreads = 768, kBackwardThreads = 512;
constexpr int kMaxTeams = kForwardThreads / 32;
constexpr int kSmem = 206 << 10;   // dynamic shared memory, most
constexpr int kMaxCtas = 256;      // at one per SM; backward: a partial sum of the weights' gradients each
constexpr int kMaxTeamRows = 1024; // backward: rows of a team, whose gradients are one fp32 sum
constexpr float kDown = 0x1p-100f;
constexpr int kMaxStages = 2;  // rows (8192 x 2048 with an fp32 stream: 39 us, with 3 41, with 4 43)

struct SandwichArgs {
    const void *x, *f;
    const void *dx, *dn;  // backward: X' and F in x and f
    const float *pre, *post, *gate;
    void *xo, *fo;        // forward: X', N; backward: dX, dF
    float *dgate;         // backward, a gate per token
    float *partial;       // backward: [grid][3][H]
    float alpha, eps, one;  // one: added to the weights
    int T, H, gate_kind, team;  // team: threads
    int *err;
    uint32_t wait_us;       // bound of the wait for a row
    int stages;             // rows in flight, the present one among them
    bool weights_in_smem;   // backward
};

// Two fp32 values in one 64-bit register, and arithmetic on both in one instruction (16384 x 2048
// backward: 86 us, with one value each 92).
typedef unsigned long long f2;
__device__ __forceinline__ f2 make2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ f2 both(float v) { return make2(v, v); }
__device__ __forceinline__ float2 split(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float sum_of(f2 v) {
    const float2 s = split(v);
    return s.x + s.y;
}

// 8 consecutive values to memory.
__device__ __forceinline__ void store8(bf16 *p, const f2 (&o)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 s = split(o[i]);
        w[i] = pack_bf16x2(s.x, s.y);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const f2 (&o)[4]) {
    const float2 w = split(o[0]), x = split(o[1]), y = split(o[2]), z = split(o[3]);
    reinterpret_cast<float4 *>(p)[0] = make_float4(w.x, w.y, x.x, x.y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(y.x, y.y, z.x, z.y);
}

// Sums over a team, in all its threads.  slots: [2][3][32], zeros where there is no warp; two sums
// in a row use different halves, so one barrier each is enough: who writes a half again has passed
// the barrier of the sum between, which everyone reaches after reading.
constexpr int kSlots = 2 * 3 * 32;
struct Team {
    int threads, id, warps, warp, lane;
    float *slots;
    int half;
    __device__ __forceinline__ Team(float *all, int team_threads) {
        threads = team_threads;
        id = threadIdx.x / threads;
        warps = threads / 32;
        warp = (threadIdx.x - id * threads) / 32;
        lane = threadIdx.x & 31;
        slots = all + id * kSlots;
        half = 0;
    }
    __device__ __forceinline__ void sync() const {
        if (warps == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
    }
    __device__ __forceinline__ float over_warps(const float *s) const {
        f2 a = 0, b = 0;
        for (int w = 0; w < warps; w += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(s + w);
            a = add2(a, make2(v.x, v.y));
            b = add2(b, make2(v.z, v.w));
        }
        return sum_of(add2(a, b));
    }
    __device__ __forceinline__ void sum(float &v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (warps == 1) {
            __syncwarp();  // as the barrier does, this orders what was read before
            return;
        }
        float *s = slots + half * 96;
        half ^= 1;
        if (lane == 0) s[warp] = v;
        sync();
        v = over_warps(s);
    }
    // Three at once: the first exchanges leave each quarter of the warp one of them to add up.
    __device__ __forceinline__ void sum(float &x, float &y, float &z) {
        const bool high = lane & 16, odd = lane & 8;
        float a = (high ? z : x) + __shfl_xor_sync(0xffffffffu, high ? x : z, 16);
        float b = (high ? 0.0f : y) + __shfl_xor_sync(0xffffffffu, high ? y : 0.0f, 16);
        float v = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (warps == 1) {
            x = __shfl_sync(0xffffffffu, v, 0);
            y = __shfl_sync(0xffffffffu, v, 8);
            z = __shfl_sync(0xffffffffu, v, 16);
            return;
        }
        float *s = slots + half * 96;
        half ^= 1;
        if ((lane & 7) == 0 && lane < 24) s[lane * 4 + warp] = v;
        sync();
        x = over_warps(s);
        y = over_warps(s + 32);
        z = over_warps(s + 64);
    }
};

// (good to 2.2 units of 2^-24, where the sum may be off by 24)
__device__ __forceinline__ float inverse_root(float sum, float inv_h, float eps) { return rsqrtf(fmaf(sum, inv_h, eps)); }

// Weights in shared memory: `count` arrays of H values, the first four values of each group of 8 in
// one half of an array, the other four in the other, so that a warp's loads have no bank conflicts.
struct Weights {
    float4 *smem;
    int groups;  // H / 8
    template <typename Fn>
    __device__ __forceinline__ void fill(int which, Fn four) const {  // four(i): values 4 i ..
        for (int i = threadIdx.x; i < 2 * groups; i += blockDim.x) smem[2 * which * groups + (i & 1) * groups + i / 2] = four(i);
    }
    __device__ __forceinline__ void get(int which, int group, f2 (&w)[4]) const {
        const float4 *at = smem + 2 * which * groups + group;
        const float4 a = at[0], b = at[groups];
        w[0] = make2(a.x, a.y), w[1] = make2(a.z, a.w), w[2] = make2(b.x, b.y), w[3] = make2(b.z, b.w);
    }
};
__device__ __forceinline__ float4 four_of(const float *w, int i, float otherwise, float more) {
    if (w == nullptr) return make_float4(otherwise, otherwise, otherwise, otherwise);
    const float4 v = reinterpret_cast<const float4 *>(w)[i];
    return make_float4(v.x + more, v.y + more, v.z + more, v.w + more);
}

// A team's next rows, in shared memory: a row's tensors one after the other, by one bulk copy each
// that a thread of the team starts, `stages` rows at most (the present one among them).  (Copies by
// every thread for itself, 16 bytes at a time, took half of each sector of fp32 rows twice: 8192 rows
// with an fp32 stream 48 us for 39; backward, 16384 x 8192 in fp32, 965 us for 745.)
struct Ring {
    uint32_t rows, bars;  // the team's: stage 0, and its barrier (8 bytes per stage)
    uint32_t bytes;       // of a stage
    int stages, stage;
    uint32_t parity;      // of the present stage's barrier
    __device__ __forceinline__ void init() const {
        for (int s = 0; s < stages; ++s) mbar_init(bars + 8 * s, 1);
    }
    __device__ __forceinline__ void next() {
        if (++stage == stages) {
            stage = 0;
            parity ^= 1u;
        }
    }
    // False: the row is not there within the bound (0: give up at once).  Lanes may differ (one answer for
    // a warp cost the gradients up to 5%).
    __device__ __forceinline__ bool wait(uint32_t limit_us) const {
        return limit_us != 0 && mbar_wait(bars + 8 * stage, parity, 1000ull * limit_us, nullptr);
    }
    __device__ __forceinline__ uint32_t present() const { return rows + stage * bytes; }
    // 8 values in shared memory
    template <typename T>
    static __device__ __forceinline__ void get(uint32_t at, f2 (&o)[4]) {
        auto load = [&](uint32_t from) {
            uint4 v;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(from) : "memory");
            return v;
        };
        if constexpr (sizeof(T) == 2) {
            const uint4 v = load(at);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = make2(bf16_lo((&v.x)[i]), bf16_hi((&v.x)[i]));
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint4 v = load(at + 16 * k);
                o[2 * k] = make2(__uint_as_float(v.x), __uint_as_float(v.y));
                o[2 * k + 1] = make2(__uint_as_float(v.z), __uint_as_float(v.w));
            }
        }
    }
};

// What both kernels keep in static shared memory.
struct Shared {
    float slots[kMaxTeams * kSlots];
    uint64_t bars[kMaxTeams * kMaxStages];
    uint4 zeros[2];  // what lanes beyond H read
    int abort;       // a wait of the CTA ran out
    // The row that a team did not get.  A thread whose wait ran out writes it here and goes on with whatever is
    // there up to the team's next sum, which it makes a NaN: where a sum is not finite all of the team's
    // threads look here and leave, so nobody asks for another row.  A row is given by its number, so that a
    // thread that is a row ahead is not taken for it.
    int lost[kMaxTeams];
};
__device__ __forceinline__ bool lost_row(const Shared &sh, const Team &team, int row) {
    __syncwarp();  // (a team of one warp has passed no other barrier)
    return *(const volatile int *)&sh.lost[team.id] == row;
}
// A team's end.  Where it did not get `row`: record it, and wait for the copies in flight, again with a bound.
__device__ __forceinline__ void end_team(Shared &sh, Ring &ring, int row, int stride, int T, int *err) {
    if (row >= T) return;
    *(volatile int *)&sh.abort = 1;
    atomicOr(err, ERR_TIMEOUT);
    for (int s = 0; s < ring.stages && row < T; ++s, row += stride, ring.next())
        wait_bar(ring.bars + 8 * ring.stage, ring.parity, kDrainCycles, nullptr);
}
__device__ __forceinline__ Ring make_ring(Shared &sh, const Team &team, uint32_t rings, uint32_t row_bytes, int stages) {
    Ring r;
    r.rows = rings + team.id * stages * row_bytes;
    r.bars = smem_u32(sh.bars + team.id * kMaxStages);
    r.bytes = row_bytes;
    r.stages = stages;
    r.stage = 0;
    r.parity = 0;
    for (int i = threadIdx.x; i < kMaxTeams * kSlots; i += blockDim.x) sh.slots[i] = 0.0f;
    if (threadIdx.x < kMaxTeams) sh.lost[threadIdx.x] = -1;
    if (threadIdx.x == 0) {
        sh.abort = 0;
        sh.zeros[0] = sh.zeros[1] = make_uint4(0, 0, 0, 0);
    }
    if ((int)threadIdx.x == team.id * team.threads) {
        r.init();
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    return r;
}

// V: groups of 8 values per thread, `team` threads apart.
template <typename TX, typename TF, int V>
__global__ void __launch_bounds__(kForwardThreads, 1) norm_forward_kernel(const SandwichArgs p) {
    extern __shared__ float4 smem[];  // the effective weights, the rings
    __shared__ __align__(16) Shared sh;
    Team team(sh.slots, p.team);
    const int me = threadIdx.x - team.id * p.team, H = p.H;
    const int stride = gridDim.x * (blockDim.x / p.team);
    const float inv_h = 1.0f / H;
    const bool has_f = p.f != nullptr, has_pre = p.pre != nullptr, has_post = p.post != nullptr;
    const bool channel = p.gate_kind == MOE_GATE_CHANNEL, token = p.gate_kind == MOE_GATE_TOKEN;
    const Weights weights{smem, H / 8};
    const uint32_t x_bytes = H * sizeof(TX), f_bytes = H * sizeof(TF), row_bytes = x_bytes + f_bytes;
    Ring ring = make_ring(sh, team, smem_u32(smem) + 2u * H * 4, row_bytes, p.stages);
    auto ask = [&](int row, int s) {  // by the team's first thread
        if (row >= p.T) return;
        const uint32_t to = ring.rows + s * row_bytes, bar = ring.bars + 8 * s;
        mbar_arrive_expect_tx(bar, has_f ? row_bytes : x_bytes);
        bulk_g2s(to, static_cast<const TX *>(p.x) + (size_t)row * H, x_bytes, bar);
        if (has_f) bulk_g2s(to + x_bytes, static_cast<const TF *>(p.f) + (size_t)row * H, f_bytes, bar);
    };
    const uint32_t zeros = smem_u32(sh.zeros);
    int group[V];
    bool in[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        in[i] = 8 * (me + i * p.team) < H;
        group[i] = in[i] ? me + i * p.team : 0;
    }
    pdl_wait();
    pdl_trigger();
    int row = blockIdx.x * (blockDim.x / p.team) + team.id;
    if (me == 0)
        for (int s = 0; s < p.stages; ++s) ask(row + s * stride, s);
    weights.fill(0, [&](int i) { return four_of(p.pre, i, 0.0f, p.one); });
    weights.fill(1, [&](int i) {  // the channels' gate is one more factor of the weight
        const float4 w = four_of(p.post, i, 1.0f, p.one), g = four_of(channel ? p.gate : nullptr, i, 1.0f, 0.0f);
        return make_float4(w.x * g.x, w.y * g.y, w.z * g.z, w.w * g.w);
    });
    float gate_next = token && row < p.T ? p.gate[row] : 1.0f;
    __syncthreads();
    for (; row < p.T; row += stride, ring.next()) {
        const float gate = gate_next;
        if (token && row + stride < p.T) gate_next = p.gate[row + stride];
        const bool got = ring.wait(p.wait_us);
        if (!got) *(volatile int *)&sh.lost[team.id] = row;
        const size_t base = (size_t)row * H;
        f2 x[V][4], f[V][4], w[4];
        auto squares = [&](const f2 (&v)[V][4], float scale) {  // (values beyond H are zeros)
            f2 s = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f2 a = scale != 1.0f ? mul2(v[i][j], both(scale)) : v[i][j];
                    s = fma2(a, a, s);
                }
            float total = got ? sum_of(s) : NAN;
            team.sum(total);
            return total;
        };
        bool lost = false;
        // the factor that norms v; of values whose squares are beyond fp32 it may be under fp32's normal
        // range, so those are normed here and the factor is 1
        auto norm = [&](f2 (&v)[V][4]) {
            float ss = squares(v, 1.0f);
            if (ss < INFINITY) return inverse_root(ss, inv_h, p.eps);
            lost = lost_row(sh, team, row);
            ss = squares(v, kDown);
            const float r = inverse_root(ss, inv_h, p.eps * kDown * kDown);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = mul2(mul2(v[i][j], both(r)), both(kDown));
            return 1.0f;
        };
#pragma unroll
        for (int i = 0; i < V; ++i) Ring::get<TX>(in[i] ? ring.present() + 8 * sizeof(TX) * group[i] : zeros, x[i]);
        if (has_f) {
#pragma unroll
            for (int i = 0; i < V; ++i) Ring::get<TF>(in[i] ? ring.present() + x_bytes + 8 * sizeof(TF) * group[i] : zeros, f[i]);
        }
        if (has_f) {
            float rf = gate;
            if (has_post) {
                rf *= norm(f);
                if (lost) break;
                if (me == 0) ask(row + p.stages * stride, ring.stage);  // the team has read the row
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                weights.get(1, group[i], w);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = fma2(both(p.alpha), x[i][j], mul2(mul2(f[i][j], both(rf)), w[j]));
                if (in[i]) store8(static_cast<TX *>(p.xo) + base + 8 * group[i], x[i]);
            }
        }
        if (!has_post && !has_pre) {
            team.sync();
            lost = lost_row(sh, team, row);
        }
        if (has_pre) {
            const float rx = norm(x);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                weights.get(0, group[i], w);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = mul2(mul2(x[i][j], both(rx)), w[j]);
                if (in[i]) store8(static_cast<TF *>(p.fo) + base + 8 * group[i], w);
            }
        }
        if (!has_post) {
            if (lost) break;
            if (me == 0) ask(row + p.stages * stride, ring.stage);
        }
    }
    end_team(sh, ring, row, stride, p.T, p.err);
}

// CHANNEL: the gate is one per channel.
template <typename TX, typename TF, int V, bool CHANNEL>
__global__ void __launch_bounds__(kBackwardThreads, 1) norm_backward_kernel(const SandwichArgs p) {
    // the effective weights and the channels' gate (where they fit), and the rings; later the teams' sums
    extern __shared__ float4 smem[];
    __shared__ __align__(16) Shared sh;
    Team team(sh.slots, p.team);
    const int me = threadIdx.x - team.id * p.team, H = p.H;
    const int stride = gridDim.x * (blockDim.x / p.team);
    const float inv_h = 1.0f / H;
    const bool has_f = p.f != nullptr, has_pre = p.pre != nullptr, has_post = p.post != nullptr;
    const bool token = p.gate_kind == MOE_GATE_TOKEN;
    const int groups = H / 8;
    const Weights weights{smem, groups};
    // X', dN, F, dX'
    const uint32_t x_bytes = H * sizeof(TX), f_bytes = H * sizeof(TF), row_bytes = 2 * (x_bytes + f_bytes);
    const uint32_t of_dn = x_bytes, of_f = x_bytes + f_bytes, of_dx = x_bytes + 2 * f_bytes;
    Ring ring = make_ring(sh, team, smem_u32(smem) + (p.weights_in_smem ? (CHANNEL ? 3u : 2u) * H * 4 : 0u), row_bytes, p.stages);
    auto ask = [&](int row, int s) {  // by the team's first thread
        if (row >= p.T) return;
        const uint32_t to = ring.rows + s * row_bytes, bar = ring.bars + 8 * s;
        const size_t at = (size_t)row * H;
        mbar_arrive_expect_tx(bar, (has_pre ? x_bytes + f_bytes : 0) + (has_f ? f_bytes : 0) + (p.dx != nullptr ? x_bytes : 0));
        if (has_pre) {
            bulk_g2s(to, static_cast<const TX *>(p.x) + at, x_bytes, bar);
            bulk_g2s(to + of_dn, static_cast<const TF *>(p.dn) + at, f_bytes, bar);
        }
        if (has_f) bulk_g2s(to + of_f, static_cast<const TF *>(p.f) + at, f_bytes, bar);
        if (p.dx != nullptr) bulk_g2s(to + of_dx, static_cast<const TX *>(p.dx) + at, x_bytes, bar);
    };
    const uint32_t zeros = smem_u32(sh.zeros);
    int group[V];
    bool in[V];
    f2 d_pre[V][4], d_post[V][4], d_gate[CHANNEL ? V : 1][4];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        in[i] = 8 * (me + i * p.team) < H;
        group[i] = in[i] ? me + i * p.team : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            d_pre[i][j] = d_post[i][j] = 0;
            if (CHANNEL) d_gate[i][j] = 0;
        }
    }
    auto weight = [&](int which, int i, f2 (&w)[4]) {
        if (p.weights_in_smem) {
            weights.get(which, group[i], w);
        } else {
            const float *from = which == 0 ? p.pre : which == 1 ? p.post : CHANNEL ? p.gate : nullptr;
            const float otherwise = which == 0 ? 0.0f : 1.0f, more = which == 2 ? 0.0f : p.one;
            const float4 a = four_of(from, 2 * group[i], otherwise, more), b = four_of(from, 2 * group[i] + 1, otherwise, more);
            w[0] = make2(a.x, a.y), w[1] = make2(a.z, a.w), w[2] = make2(b.x, b.y), w[3] = make2(b.z, b.w);
        }
    };
    pdl_wait();
    pdl_trigger();
    int row = blockIdx.x * (blockDim.x / p.team) + team.id;
    // tensors that the call does not have are zeros in every stage
    if (!has_pre || !has_f || p.dx == nullptr) {
        for (uint32_t s = 0; s < p.stages * row_bytes; s += row_bytes)
            for (uint32_t i = 16 * me; i < row_bytes; i += 16 * p.team) {
                const bool here = i < of_f ? has_pre : i < of_dx ? has_f : p.dx != nullptr;
                if (!here) asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(ring.rows + s + i), "r"(0u) : "memory");
            }
    }
    if (me == 0)
        for (int s = 0; s < p.stages; ++s) ask(row + s * stride, s);
    if (p.weights_in_smem) {
        weights.fill(0, [&](int i) { return four_of(p.pre, i, 0.0f, p.one); });
        weights.fill(1, [&](int i) { return four_of(p.post, i, 1.0f, p.one); });
        if (CHANNEL) weights.fill(2, [&](int i) { return four_of(p.gate, i, 1.0f, 0.0f); });
    }
    float gate_next = token && row < p.T ? p.gate[row] : 1.0f;
    __syncthreads();

    for (; row < p.T; row += stride, ring.next()) {
        // What is not there is zeros or ones, so that the values take no branches.
        const float g = gate_next, alpha = has_f ? p.alpha : 1.0f;
        if (token && row + stride < p.T) gate_next = p.gate[row + stride];
        const bool got = ring.wait(p.wait_us);
        if (!got) *(volatile int *)&sh.lost[team.id] = row;
        const size_t base = (size_t)row * H;
        f2 x[V][4], dn[V][4], f[V][4], w[4];
        uint32_t at_x[V], at_f[V];  // a thread's values of the first tensor of either type in this stage
#pragma unroll
        for (int i = 0; i < V; ++i) {
            at_x[i] = ring.present() + 8 * sizeof(TX) * group[i];
            at_f[i] = ring.present() + of_dn + 8 * sizeof(TF) * group[i];
            Ring::get<TX>(in[i] ? at_x[i] : zeros, x[i]);
            Ring::get<TF>(in[i] ? at_f[i] : zeros, dn[i]);
            Ring::get<TF>(in[i] ? at_f[i] + f_bytes : zeros, f[i]);
        }
        // the squares of X' and F, and dN w_pre X'; of values scaled down where that is not enough
        float sx = 1.0f, sf = 1.0f, s0, s1, s2;
        auto sums = [&](bool scaled) {
            f2 xx = 0, ff = 0, dx = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                weight(0, i, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f2 a = scaled ? mul2(x[i][j], both(sx)) : x[i][j], b = scaled ? mul2(f[i][j], both(sf)) : f[i][j];
                    xx = fma2(a, a, xx);
                    ff = fma2(b, b, ff);
                    dx = fma2(mul2(dn[i][j], w[j]), a, dx);
                }
            }
            s0 = got ? sum_of(xx) : NAN, s1 = sum_of(ff), s2 = sum_of(dx);
            team.sum(s0, s1, s2);
        };
        sums(false);
        if (!(s0 < INFINITY) || !(s1 < INFINITY)) {
            if (lost_row(sh, team, row)) break;
            if (!(s0 < INFINITY)) sx = kDown;
            if (!(s1 < INFINITY)) sf = kDown;
            sums(true);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) f[i][j] = mul2(f[i][j], both(sf));  // scaled from here, for the sum below
        }
        const float rxs = inverse_root(s0, inv_h, p.eps * sx * sx), rx = rxs * sx, mean = rxs * s2 * inv_h;
        const float rf = has_post ? inverse_root(s1, inv_h, p.eps * sf * sf) : 1.0f / sf;  // of f as it is now
        f2 t[V][4], m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            weight(0, i, w);
            Ring::get<TX>(in[i] ? at_x[i] + of_dx : zeros, t[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f2 xh = mul2(x[i][j], both(rx));
                d_pre[i][j] = fma2(dn[i][j], xh, d_pre[i][j]);
                t[i][j] = fma2(both(rx), fma2(xh, both(-mean), mul2(dn[i][j], w[j])), t[i][j]);
                w[j] = mul2(both(alpha), t[i][j]);
            }
            if (in[i]) store8(static_cast<TX *>(p.xo) + base + 8 * group[i], w);
            if (!has_f) continue;
            // t: from T to T (times the channel's gate) times w_post
            weight(1, i, w);
            f2 gates[4];
            if (CHANNEL) weight(2, i, gates);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f2 fh = mul2(f[i][j], both(rf * g));
                if (CHANNEL) {
                    d_gate[i][j] = fma2(mul2(t[i][j], w[j]), fh, d_gate[i][j]);
                    t[i][j] = mul2(t[i][j], gates[j]);
                }
                d_post[i][j] = fma2(t[i][j], fh, d_post[i][j]);
                t[i][j] = mul2(t[i][j], w[j]);
                m = fma2(t[i][j], f[i][j], m);
            }
        }
        float total = sum_of(m) * rf;
        if (has_f && (has_post || token))
            team.sum(total);
        else
            team.sync();
        if (me == 0) ask(row + p.stages * stride, ring.stage);  // the team has read the row
        if (!has_f) continue;
        if (token && me == 0 && p.dgate != nullptr) p.dgate[row] = total;
        // dF = g rf (T w_post - fh mean(T w_post fh)), or g T
        const float out = has_post ? g * rf : g, back = has_post ? -total * inv_h * rf : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = mul2(both(out), has_post ? fma2(f[i][j], both(back), t[i][j]) : t[i][j]);
            if (has_post && sf != 1.0f) {  // (g rf sf may be under fp32's normal range)
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = mul2(w[j], both(sf));
            }
            if (in[i]) store8(static_cast<TF *>(p.fo) + base + 8 * group[i], w);
        }
    }
    end_team(sh, ring, row, stride, p.T, p.err);

    // the teams' sums one after the other, then this CTA's
    const int teams = blockDim.x / p.team;
    __syncthreads();
    if (*(volatile int *)&sh.abort) return;  // (a copy that did not end may still write to shared memory)
    for (int k = 0; k < teams; ++k) {
        if (team.id == k) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!in[i]) continue;
                auto add = [&](float4 *at, f2 lo, f2 hi) {
                    const float2 a = split(lo), b = split(hi);
                    const float4 v = k ? *at : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    *at = make_float4(v.x + a.x, v.y + a.y, v.z + b.x, v.w + b.y);
                };
                float4 *at = smem + group[i];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    add(at + h * groups, d_pre[i][2 * h], d_pre[i][2 * h + 1]);
                    add(at + (2 + h) * groups, d_post[i][2 * h], d_post[i][2 * h + 1]);
                    if (CHANNEL) add(at + (4 + h) * groups, d_gate[i][2 * h], d_gate[i][2 * h + 1]);
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
        if (CHANNEL) mine[4 * groups + i] = smem[4 * groups + from];
    }
}

// The CTAs' sums, one column of one result per lane of a warp row.  A thread's additions, 5 with one CTA per
// SM and any number beyond, with their rounding errors (a + b = s + e exactly; in fp64 a call took 3 to 6 us
// longer).
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows) norm_sum_kernel(const float *partial, int parts, int H, float *d_pre,
                                                                 float *d_post, float *d_gate) {
    __shared__ float s[kSumRows][33];
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane, which = blockIdx.y;
    float *out = which == 0 ? d_pre : which == 1 ? d_post : d_gate;
    pdl_wait();
    pdl_trigger();
    if (out == nullptr) return;
    float v = 0.0f, lost = 0.0f;
    if (col < H)
        for (int i = r; i < parts; i += kSumRows) {
            const float b = partial[((size_t)i * 3 + which) * H + col], sum = __fadd_rn(v, b), of_b = __fsub_rn(sum, v);
            lost = __fadd_rn(lost, __fadd_rn(__fsub_rn(v, __fsub_rn(sum, of_b)), __fsub_rn(b, of_b)));
            v = sum;
        }
    s[r][lane] = fabsf(v) < INFINITY ? v + lost : v;  // (beside an infinity, `lost` is a NaN)
    __syncthreads();
    if (r != 0 || col >= H) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumRows; ++i) v += s[i][lane];
    out[col] = v;
}

OpDone g_attr[24];

// Teams of several warps have a named barrier each, of 15.
int most_teams(int team) { return team > 32 ? 15 : kMaxTeams; }

// 16 values per thread where a row has them for a warp: the sums over a team cost a warp as much as 4
// values per lane.
bool two_groups(int H) { return H > 256; }
// Threads per team and teams per CTA: as many as fit (shape: fewer where rows would leave SMs without one).
int team_threads(int H) {
    const int per = 32 * (two_groups(H) ? 16 : 8);
    return 32 * ((H + per - 1) / per);
}
int full_teams(int H, int threads) { return std::min(threads / team_threads(H), most_teams(team_threads(H))); }
void shape(int T, int H, int sms, int threads, int &team, int &teams) {
    team = team_threads(H);
    teams = std::max(1, std::min(full_teams(H, threads), (T + sms - 1) / sms));
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
    if (H % 8 || H > kMaxH || T > (1 << 30))
        return op_fail(MOE_ERR_UNSUPPORTED, "%s: T up to 2^30, H a multiple of 8 up to %d (T %d, H %d)", op, kMaxH, T, H);
    return MOE_OK;
}

bool aligned(std::initializer_list<const void *> all) {
    return std::all_of(all.begin(), all.end(), [](const void *p) { return op_aligned16(p); });
}

using KernelFn = void (*)(const SandwichArgs);
struct Choice {
    KernelFn kernel;
    int which;
};
template <typename TX, typename TF, int V>
Choice choose(bool backward, bool channel, int which) {
    if (!backward) return {norm_forward_kernel<TX, TF, V>, which};
    return channel ? Choice{norm_backward_kernel<TX, TF, V, true>, which + 1} : Choice{norm_backward_kernel<TX, TF, V, false>, which + 2};
}
template <int V>
Choice choose(int x_dtype, int f_dtype, bool backward, bool channel) {
    const int which = 12 * (V - 1);
    if (x_dtype == MOE_DTYPE_BF16)
        return f_dtype == MOE_DTYPE_BF16 ? choose<bf16, bf16, V>(backward, channel, which) : choose<bf16, float, V>(backward, channel, which + 3);
    return f_dtype == MOE_DTYPE_BF16 ? choose<float, bf16, V>(backward, channel, which + 6) : choose<float, float, V>(backward, channel, which + 9);
}

moe_status launch(const char *name, bool backward, SandwichArgs &a, int x_dtype, int f_dtype, int sms, int &grid, cudaStream_t s) {
    const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
    const Choice c = two_groups(a.H) ? choose<2>(x_dtype, f_dtype, backward, channel) : choose<1>(x_dtype, f_dtype, backward, channel);
    int teams;
    shape(a.T, a.H, sms, backward ? kBackwardThreads : kForwardThreads, a.team, teams);
    grid = (int)std::min<long long>(std::min(sms, kMaxCtas), ((long long)a.T + teams - 1) / teams);
    if (backward) {  // times the waves that bring a team's rows to kMaxTeamRows
        const long long wave = (long long)grid * teams * kMaxTeamRows;
        grid *= (int)((a.T + wave - 1) / wave);
    }
    // X and F, backward also their gradients, of a row of each team
    const int stage = teams * a.H * ((x_dtype == MOE_DTYPE_F32 ? 4 : 2) + (f_dtype == MOE_DTYPE_F32 ? 4 : 2)) * (backward ? 2 : 1);
    const int weights = (backward && channel ? 3 : 2) * a.H * 4;
    a.weights_in_smem = weights + stage <= kSmem;
    a.stages = std::min(kMaxStages, (kSmem - (a.weights_in_smem ? weights : 0)) / stage);
    a.err = op_error_word();
    a.wait_us = (uint32_t)std::min<uint64_t>(~0u, ((uint64_t)wait_cycles(0) + 1999) / 2000);  // of cycles at 2 GHz; 0 for 0 alone
    if (a.err == nullptr) return op_fail(MOE_ERR_CUDA, "%s: no usable current device", name);
    const int smem = std::max(weights, (a.weights_in_smem ? weights : 0) + a.stages * stage);
    const cudaError_t e = op_allow_smem(reinterpret_cast<const void *>(c.kernel), kSmem, &g_attr[c.which]);
    if (e != cudaSuccess) return op_cuda(e, name);
    return op_cuda(launch_pdl(c.kernel, dim3(grid), dim3(a.team * teams), (size_t)smem, s, a), name);
}

// A partial sum of each CTA, whatever the device: up to kMaxCtas, or what is needed for T rows rounded up to
// a multiple of as many.  (More than one wave is of full teams.)
size_t workspace_of(int T, int H) {
    const int ctas = std::min(T, kMaxCtas + T / (kMaxTeamRows * full_teams(H, kBackwardThreads)));
    return (size_t)std::max(1, ctas) * 3 * H * sizeof(float);
}

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
    int grid;
    return launch(name, false, a, x_dtype, f_dtype, sms, grid, reinterpret_cast<cudaStream_t>(stream));
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
        st = launch(name, true, a, x_dtype, f_dtype, sms, grid, s);
        if (st != MOE_OK) return st;
    }
    float *d_gate = gate_kind == MOE_GATE_CHANNEL ? dgate : nullptr;
    if (!dpre_w && !dpost_w && !d_gate) return MOE_OK;
    return op_cuda(launch_pdl(norm_sum_kernel, dim3((H + 31) / 32, 3), dim3(32 * kSumRows), 0, s,
                              static_cast<const float *>(workspace), grid, H, dpre_w, dpost_w, d_gate), name);
}
