// loss_common.cuh -- device and host code shared by the loss kernels
// (logits.cu, preference.cu) and the tensor-list kernels (tensors.cu).
// Included inside an anonymous namespace after step_common.cuh and
// step_end.cuh; cluster_counts.h before it, outside.
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

// A sum in two fp32 parts, hi + lo: what hi's rounding drops goes to lo exactly
// (the TwoSum of Knuth).  GB300's fp64 rate is a small part of its fp32 rate.
// Once hi is infinite or NaN it is the sum, and lo, a difference of infinities,
// is not read.
struct Sum2 {
    float hi, lo;
    __device__ __forceinline__ double value() const {
        return fabsf(hi) <= 3.402823466e38f ? (double)hi + (double)lo : (double)hi;
    }
    __device__ __forceinline__ void add(float p) {
        const float s = __fadd_rn(hi, p), bp = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, bp)), __fsub_rn(p, bp)));
        hi = s;
    }
};

// The loss scale of a control block (1 without one).
__device__ __forceinline__ float loss_scale_of(const zs_ctrl* c) {
    return c == nullptr ? 1.0f : __double2float_rn(*(const volatile double*)&c->loss_scale);
}

inline bool finite_double(double x) { return x == x && x <= 1e300 && x >= -1e300; }

// --------------------------------------------------------------- clusters ---

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

constexpr int kMaxCluster = 8;

// How many clusters of a kernel run at once on the current device; 0 and *err
// set if that could not be found.
int active_clusters(const void* kernel, int threads, int ctas, int smem, cudaError_t* err) {
    static zs::ClusterCounts counts;
    int device = 0;
    *err = cudaGetDevice(&device);
    if (*err != cudaSuccess) return 0;
    return counts.get(device, kernel, ctas, smem, [&] {
        int n = 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(ctas * zs::device_sm_count()));
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = (size_t)smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        *err = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (*err == cudaSuccess && n < 1) *err = cudaErrorInvalidConfiguration;
        if (*err == cudaSuccess) return n;
        cudaGetLastError();
        return 0;
    });
}

// Enqueues `clusters` clusters of `ctas` blocks with programmatic serialization.
template <typename Args>
int32_t launch_clusters(void (*kernel)(Args), int clusters, int ctas, int threads, int smem, cudaStream_t stream,
                        const Args& args, const char* name) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * ctas));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, args);
    if (err != cudaSuccess) return zs::cuda_fail(err, name);
    return zs::check_launch(name);
}
