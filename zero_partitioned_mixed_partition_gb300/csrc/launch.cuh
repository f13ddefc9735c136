// launch.cuh -- launches of the head, norm and embedding kernels: with
// programmatic serialization, so that every kernel waits by griddep_wait() before it
// touches global memory.  Included inside an anonymous namespace.
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

#define ZS_TRY(call)                          \
    do {                                      \
        const int32_t rc_ = (call);           \
        if (rc_ != ZS_OK) return rc_;         \
    } while (0)
