// loss_common.cuh -- device and host code shared by the loss kernels
// (logits.cu, preference.cu) and the tensor-list kernels (tensors.cu).
// Included inside an anonymous namespace after step_common.cuh and
// step_end.cuh.
#pragma once

#include "packed.cuh"

// ---------------------------------------------------------------- scratch ---

// The caller's scratch buffer: an arrival counter, 0 between calls, and the
// blocks' partial sums.
struct Work {
    uint32_t arrivals;
    uint32_t pad[31];
    double part[(ZS_WORK_BYTES - 128) / 8];
};
static_assert(sizeof(Work) == ZS_WORK_BYTES, "the scratch buffer's documented size");
constexpr int kWorkParts = (ZS_WORK_BYTES - 128) / 8;

// Called by every thread of each of the `total` blocks of a launch after the
// block's thread 0 wrote its partial sums: true in the block that arrives
// last, for which every partial sum is then visible.  That block resets the
// counter.  Nothing waits.
__device__ __forceinline__ bool last_to_arrive(Work* w, uint32_t total) {
    __shared__ int s_last;
    if (threadIdx.x == 0) {
        __threadfence();
        s_last = atomicAdd(&w->arrivals, 1u) == total - 1 ? 1 : 0;
        if (s_last) {
            w->arrivals = 0u;
            __threadfence();
        }
    }
    __syncthreads();
    return s_last != 0;
}

// Sum over the warp, valid in every lane; the order is fixed.
__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The loss scale of a control block (1 without one).
__device__ __forceinline__ float loss_scale_of(const zs_ctrl* c) {
    return c == nullptr ? 1.0f : __double2float_rn(*(const volatile double*)&c->loss_scale);
}

inline bool finite_double(double x) { return x == x && x <= 1e300 && x >= -1e300; }
