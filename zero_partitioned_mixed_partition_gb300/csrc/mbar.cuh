// mbar.cuh -- barriers in shared memory and bounded waits for them, shared by the
// logits and head kernels.  Included inside an anonymous namespace after
// loss_common.cuh.
#pragma once

// Barriers in shared memory that count arrivals and copied bytes.
__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
    asm volatile("{\n\t.reg .b64 t;\n\tmbarrier.arrive.shared::cta.b64 t, [%0];\n\t}" ::"r"(smem_addr(b)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* b, uint32_t bytes) {
    asm volatile("{\n\t.reg .b64 t;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1;\n\t}" ::"r"(smem_addr(b)),
                 "r"(bytes) : "memory");
}
// Counts bytes of a copy that will not be made.
__device__ __forceinline__ void mbar_give(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(bytes) : "memory");
}
// Whether the phase of the given parity is over; waits up to 2 us for it.  CTA: what the
// arrivals order is this CTA's own, or no ordinary memory at all (copies, tensor memory);
// else the cluster's, for which the SM drops what its L1 holds.
template <bool CTA = false>
__device__ __forceinline__ bool mbar_try(uint64_t* b, uint32_t parity) {
    uint32_t done = 0;
    if (CTA)
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(done) : "r"(smem_addr(b)), "r"(parity), "r"(2000u) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(done) : "r"(smem_addr(b)), "r"(parity), "r"(2000u) : "memory");
    return done != 0;
}
// The tries of a wait: a second or two.
constexpr int kWaitLimit = 1 << 20;
#if ZS_CHECKED
__device__ int32_t g_wait_limit = kWaitLimit;  // zero_debug_wait_limit
__device__ __forceinline__ int wait_limit() { return *(volatile int32_t*)&g_wait_limit; }
#else
__device__ __forceinline__ int wait_limit() { return kWaitLimit; }
#endif
// Sets this translation unit's limit (1: set; 0: not this build; ZS_ERR_CUDA).
int32_t set_unit_wait_limit(int32_t tries) {
#if ZS_CHECKED
    const cudaError_t err = cudaMemcpyToSymbol(g_wait_limit, &tries, sizeof(tries));
    return err == cudaSuccess ? 1 : zs::cuda_fail(err, "zero_debug_wait_limit");
#else
    (void)tries;
    return 0;
#endif
}
template <bool RELAXED, bool CTA>
__device__ __forceinline__ bool mbar_wait_on(uint64_t* b, uint32_t parity, int32_t* failed) {
    const int limit = wait_limit();
#pragma unroll 1
    for (int i = 0; i < limit; ++i) {
        if (mbar_try<CTA>(b, parity)) return true;
        if (*(volatile int32_t*)failed) return false;
        if (RELAXED) __nanosleep(100);
    }
    *(volatile int32_t*)failed = 1;
    return false;
}
// Waits for the phase, within the limit.  A wait that runs out sets *failed and
// returns false; so do the block's other waits from then on, at once.  RELAXED: for
// the warps that mostly wait; they leave the issue slots to the others.  (Most waits
// are over at the first try; with that in the loop, 708 us for 684 in the largest
// case of the logits kernels.)
template <bool RELAXED = false, bool CTA = false>
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity, int32_t* failed) {
#if ZS_CHECKED
    if (wait_limit() == 0) return mbar_wait_on<RELAXED, CTA>(b, parity, failed);
#endif
    return mbar_try<CTA>(b, parity) || mbar_wait_on<RELAXED, CTA>(b, parity, failed);
}
// Whether every lane of the warp may go on.
__device__ __forceinline__ bool all_lanes(bool ok) { return __all_sync(0xffffffffu, ok); }
// Waits, within the ordinary limit, until the barrier counts no copy in flight.
__device__ __forceinline__ void drain(uint64_t* b, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < kWaitLimit; ++i)
        if (mbar_try(b, parity)) return;
}
