// tensor_core.cuh -- what the head's products need of the fifth-generation tensor
// cores and the tensor copies: CTAS = 2, a pair of CTAs (two SMs), or 1, works on one
// tile, operands lie in shared memory in the 128-byte swizzle, sums in tensor memory.  Included
// inside an anonymous namespace after mbar.cuh.
#pragma once

// ------------------------------------------------------------ tensor copies ---

// A box of a tensor map at (x, y), x the contiguous coordinate (a multiple of 16
// bytes), into this CTA's shared memory, counted by a barrier that may be the
// pair's other CTA's (a shared::cluster address).
template <int CTAS>
__device__ __forceinline__ void copy_box(void* dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t barrier) {
    if (CTAS == 2)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
            ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(barrier) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
            ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(barrier) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// The address of the same place in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
// Arrives at a barrier of the pair after loads from tensor memory, which the fences of
// tensor memory order.  (A release to the cluster would wait for the warp's stores to
// global memory besides.)
__device__ __forceinline__ void arrive_at(uint32_t barrier) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(barrier) : "memory");
}
__device__ __forceinline__ int32_t load_from_peer(const int32_t* p, uint32_t rank) {
    int32_t v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(peer_addr(p, rank)) : "memory");
    return v;
}

// ------------------------------------------------------------ tensor memory ---

constexpr uint32_t kTensorColumns = 512;  // of 128 lanes and 32 bits: all there are

// By one warp of each CTA; the address is written to *at.
template <int CTAS>
__device__ __forceinline__ void tensor_alloc(uint32_t* at) {
    if (CTAS == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(kTensorColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(kTensorColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <int CTAS>
__device__ __forceinline__ void tensor_free(uint32_t base) {
    if (CTAS == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(kTensorColumns));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(kTensorColumns));
}
__device__ __forceinline__ void tensor_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tensor_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of the warp's 32 lanes: lane l gets those of lane (address's lane) + l.
__device__ __forceinline__ void tensor_load(uint32_t at, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}
// Until the loads have come.  (What uses the values has to stay behind this: `loaded` on each
// 32 of them, which is no instruction, says so to the compiler.)
__device__ __forceinline__ void tensor_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void loaded(float* v) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]),
                          "+f"(v[i + 6]), "+f"(v[i + 7]) :: "memory");
}

// ------------------------------------------------------------------ products ---

// An operand in shared memory, in 128-byte rows with the 128-byte swizzle (groups of
// eight rows, 1024 bytes).  Along k: a row holds 64 k of one m (or n).  Across k: a row
// holds 64 m of one k, and the next 64 m lie `next` bytes on.
__device__ __forceinline__ uint64_t operand(const void* p, uint32_t next, bool along) {
    const uint64_t lead = along ? 1 : next >> 4, group = 1024 >> 4;
    return (uint64_t)((smem_addr(p) >> 4) & 0x3fff) | lead << 16 | group << 32 | 1ull << 46 | 2ull << 61;
}
// The step of 16 k of an operand's descriptor: 32 bytes along a row, or 16 rows.
__device__ __forceinline__ uint64_t operand_step(bool along) { return (along ? 32 : 2048) >> 4; }

// What an instruction multiplies: A of 128 rows to a CTA and B of n columns in all, an
// even share in each CTA, 16-bit types, fp32 sums.
template <typename T> constexpr uint32_t operand_type();
template <> constexpr uint32_t operand_type<__half>() { return 0; }
template <> constexpr uint32_t operand_type<__nv_bfloat16>() { return 1; }
template <int CTAS, typename T>
__device__ __forceinline__ uint32_t product_kind(uint32_t n, bool a_along, bool b_along) {
    return 1u << 4 | operand_type<T>() << 7 | operand_type<T>() << 10 | (a_along ? 0u : 1u) << 15 | (b_along ? 0u : 1u) << 16 |
           (n >> 3) << 17 | (128u * CTAS >> 4) << 24;
}
// sums [+]= A B over 16 k, by one thread of the (first) CTA.
template <int CTAS>
__device__ __forceinline__ void multiply(uint32_t sums, uint64_t a, uint64_t b, uint32_t kind, bool add) {
    if (CTAS == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(sums), "l"(a), "l"(b), "r"(kind),
            "r"(add ? 1u : 0u) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(sums), "l"(a), "l"(b), "r"(kind),
            "r"(add ? 1u : 0u) : "memory");
}
// Arrives at the barrier of this CTA once the thread's products so far are done.
template <int CTAS>
__device__ __forceinline__ void signal_after_products(uint64_t* barrier) {
    if (CTAS == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(barrier))
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(barrier))
                     : "memory");
}
// The same at the barrier at this place in every CTA of the tile.
template <int CTAS>
__device__ __forceinline__ void arrive_after_products(uint64_t* barrier) {
    if (CTAS == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_addr(barrier)), "h"((uint16_t)3) : "memory");
    else
        signal_after_products<1>(barrier);
}

// ----------------------------------------------------------------- registers ---

// The executing warpgroup (four warps, all of them) goes down to, or up to, N registers a
// thread.  Those taken have to be given up by others of the block.
template <int N> __device__ __forceinline__ void give_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void take_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
