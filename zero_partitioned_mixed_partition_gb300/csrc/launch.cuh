// launch.cuh -- launches of the head, norm and embedding kernels: with
// programmatic serialization, so that every kernel waits by griddep_wait() before it
// touches global memory.  Included inside an anonymous namespace after loss_common.cuh.
#pragma once

template <typename... P, typename... A>
int32_t launch_shared(void (*kernel)(P...), dim3 grid, int threads, size_t shared, cudaStream_t stream, const char* name,
                      A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
    if (err != cudaSuccess) return zs::cuda_fail(err, name);
    return zs::check_launch(name);
}

template <typename... P, typename... A>
int32_t launch(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream, const char* name, A... args) {
    return launch_shared(kernel, grid, threads, 0, stream, name, args...);
}

constexpr int kMaxShared = 200 * 1024;  // dynamic shared memory that these kernels ask for at most

// The blocks of a grid that fill the current device, no more than there is work for; 0 and
// the error recorded if that could not be found.
unsigned grid_of(const void* kernel, int threads, size_t shared, int64_t work) {
    static zs::ClusterCounts counts;
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    const int most = err != cudaSuccess ? 0 : counts.get(device, kernel, threads, (int)shared, [&] {
        int per_sm = 0;
        // (the limit is the kernel's, for calls of any size)
        if (shared > 32 * 1024)  // (48 KB with what the kernel has statically need no asking)
            err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
        if (err == cudaSuccess) err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, shared);
        if (err == cudaSuccess && per_sm < 1) err = cudaErrorInvalidConfiguration;
        if (err != cudaSuccess) cudaGetLastError();
        return err == cudaSuccess ? per_sm * zs::device_sm_count() : 0;
    });
    if (most < 1) {
        zs::cuda_fail(err != cudaSuccess ? err : cudaErrorInvalidConfiguration, "grid_of");
        return 0;
    }
    return (unsigned)(work < 1 ? 1 : work < most ? work : most);
}

// Clusters of `ctas` blocks of a kernel that run at once on the current device; 0 and the
// error recorded if that could not be found.
int clusters_of(const void* kernel, int threads, int ctas, size_t shared) {
    static zs::ClusterCounts counts;
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    const int most = err != cudaSuccess ? 0 : counts.get(device, kernel, ctas, (int)shared, [&] {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
        return err == cudaSuccess ? active_clusters(kernel, threads, ctas, (int)shared, &err) : 0;
    });
    if (most < 1) zs::cuda_fail(err != cudaSuccess ? err : cudaErrorInvalidConfiguration, "clusters_of");
    return most;
}

#define ZS_TRY(call)                          \
    do {                                      \
        const int32_t rc_ = (call);           \
        if (rc_ != ZS_OK) return rc_;         \
    } while (0)
