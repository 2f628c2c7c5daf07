// Host helpers shared by the stateless operators (grouped products, MX
// quantisation, gradient clipping): error reporting, argument checks, the
// driver's tensor-map encoder and per-device facts.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

void moe_set_last_error_internal(const char *msg);

namespace moe {

// Set the thread's error message (printf style) and return `st`.
moe_status op_fail(moe_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));

// MOE_OK, or the failure of a CUDA call made by operator `op`.
moe_status op_cuda(cudaError_t e, const char *op);

inline bool op_aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether two buffers share bytes.
inline bool op_overlap(const void *a, uint64_t na, const void *b, uint64_t nb) {
    const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

// SM count of the current device (looked up once per device), or 0 after an error.
int op_num_sms();

constexpr int kOpMaxDevices = 64;

// The context (its id) of each device in which something has been set.
struct OpDone {
    unsigned long long ctx[kOpMaxDevices];
};

// Allow `kernel` `bytes` of dynamic shared memory in the current context, once in each.
cudaError_t op_allow_smem(const void *kernel, int bytes, OpDone *done);

// A tiled tensor map of up to 4 dimensions (innermost first; strides in bytes, of
// dimensions 1 ..), zero fill out of bounds.
struct OpMap {
    CUtensorMapDataType type;
    int rank;
    const void *base;
    uint64_t dims[4];
    uint64_t strides[3];
    uint32_t box[4];
    CUtensorMapSwizzle swizzle;
};
CUresult op_encode(CUtensorMap *m, const OpMap &d);

// The bound set with moe_operators_wait_limit, -1: none.
long long op_wait_limit();

// Device address of the operators' error word (op_capi.cu) in the current context.
int *op_error_word();

}  // namespace moe
