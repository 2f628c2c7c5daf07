// Host helpers of the stateless operators, and their device error word: the
// bounded waits and offset checks of the grouped products record failures in one
// word per context, which moe_operators_status() reads and clears in one exchange: other threads
// and streams may record the next error at any time.
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "kernels.h"
#include "op_host.h"

namespace moe {
namespace {

__device__ int g_op_error;
__device__ int g_taken;  // what the last exchange took out of it

__global__ void take_error_kernel() { g_taken = atomicExch(&g_op_error, 0); }

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

std::mutex g_mutex;
std::mutex g_take_mutex;  // from an exchange until its result has been read
int g_sms[kOpMaxDevices];
int *g_error_word[kOpMaxDevices];  // where g_op_error lies on each,
OpDone g_error_word_of;            // and in which context
std::atomic<long long> g_wait_limit{-1};

}  // namespace

moe_status op_fail(moe_status st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    ::moe_set_last_error_internal(buf);
    return st;
}

moe_status op_cuda(cudaError_t e, const char *op) {
    return e == cudaSuccess ? MOE_OK : op_fail(MOE_ERR_CUDA, "%s: %s", op, cudaGetErrorString(e));
}

int op_num_sms() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kOpMaxDevices) return 0;
    std::lock_guard<std::mutex> lock(g_mutex);
    if (g_sms[dev] == 0 && cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        g_sms[dev] = 0;
    return g_sms[dev];
}

cudaError_t op_allow_smem(const void *kernel, int bytes, OpDone *done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kOpMaxDevices) return cudaErrorInvalidDevice;
    const unsigned long long ctx = current_context_id();
    std::lock_guard<std::mutex> lock(g_mutex);
    if (ctx != 0 && done->ctx[dev] == ctx) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done->ctx[dev] = ctx;
    return e;
}

CUresult op_encode(CUtensorMap *m, const OpMap &d) {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    if (fn == nullptr) return CUDA_ERROR_NOT_FOUND;
    cuuint64_t dims[4], strides[3];
    cuuint32_t box[4], estr[4];
    for (int i = 0; i < d.rank; ++i) {
        dims[i] = d.dims[i];
        box[i] = d.box[i];
        estr[i] = 1;
        if (i + 1 < d.rank) strides[i] = d.strides[i];
    }
    return fn(m, d.type, (cuuint32_t)d.rank, const_cast<void *>(d.base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, d.swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

long long op_wait_limit() { return g_wait_limit.load(std::memory_order_relaxed); }

int *op_error_word() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kOpMaxDevices) return nullptr;
    const unsigned long long ctx = current_context_id();
    std::lock_guard<std::mutex> lock(g_mutex);
    if (ctx != 0 && g_error_word_of.ctx[dev] == ctx) return g_error_word[dev];
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_op_error) != cudaSuccess) return nullptr;
    g_error_word[dev] = static_cast<int *>(p);
    g_error_word_of.ctx[dev] = ctx;
    return g_error_word[dev];
}

}  // namespace moe

extern "C" moe_status moe_operators_wait_limit(long long cycles) {
    if (cycles < -1) return moe::op_fail(MOE_ERR_INVALID_ARG, "moe_operators_wait_limit: need cycles >= -1");
    moe::g_wait_limit.store(cycles, std::memory_order_relaxed);
    return MOE_OK;
}

extern "C" moe_status moe_operators_status(void) {
    using namespace moe;
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return op_cuda(e, "moe_operators_status");
    int word = 0;
    {
        std::lock_guard<std::mutex> lock(g_take_mutex);
        e = cudaLaunchKernel(reinterpret_cast<const void *>(take_error_kernel), dim3(1), dim3(1), nullptr, 0, nullptr);
        if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&word, g_taken, sizeof word);  // waits for the kernel
    }
    if (e != cudaSuccess) return op_cuda(e, "moe_operators_status");
    if (word == 0) return MOE_OK;
    if (word & ERR_BOUNDS)
        return op_fail(MOE_ERR_DEVICE_CHECK, "an operator met row offsets that decrease or leave [0, rows]; it wrote nothing%s",
                       word & ERR_TIMEOUT ? "; and a device-side wait of an operator ran past its bound" : "");
    return op_fail(MOE_ERR_TIMEOUT, "a device-side wait of an operator ran past its bound");
}
