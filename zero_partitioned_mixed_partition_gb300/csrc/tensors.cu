// tensors.cu -- the AdamW step over a list of tensors, in place, with fp32 or
// 8-bit states; the gradients' squared norm and non-finite test before it;
// and the values of 8-bit states.
//
// The list travels in the kernel parameters (nothing is kept on the device
// between calls): each launch takes as many tensors as fit there and walks
// their chunks of 2048 elements back to back with a persistent grid.  A chunk
// is found in the list by binary search on the tensors' first chunks.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <cmath>
#include <cstring>

#include "cluster_counts.h"
#include "zs_internal.h"

namespace {

#include "step_common.cuh"
#include "step_end.cuh"
#include "loss_common.cuh"
#include "adam8_math.cuh"
#include "tensors_math.cuh"

// index-check sites of this file
[[maybe_unused]] constexpr uint32_t kSiteTensor = 14, kSiteTensorScale = 15, kSiteTensorNorm = 16;

constexpr int kChunk = ZS_ADAM8_BLOCK;  // elements of a chunk: one block of 8-bit states
constexpr int kShares = kChunk / 8;     // a chunk is taken in shares of 8 elements

// ------------------------------------------------------------------ layout ---

// Which elements of a chunk a share is, by the tensor's `peel`:
//   peel in [0, 8)  every buffer of the tensor is on a 16-byte boundary (8 for
//                   codes) at element peel, and so at peel + 8 i: share v < 255
//                   is the eight from peel + 8 v, as vectors; share 255 is the
//                   chunk's edges, [0, peel) and [2040 + peel, 2048)
//   kScattered      no such element: share v is v + 256 j, one at a time
constexpr int kScattered = 8;

__device__ __forceinline__ int share_element(int peel, int v, int j) {
    if (peel == kScattered) return v + kShares * j;
    if (v < kShares - 1) return peel + 8 * v + j;
    return j < peel ? j : kChunk - 8 + j;
}
__device__ __forceinline__ bool share_is_vector(int peel, int v, int rem) {
    if (peel == kScattered) return false;
    if (v < kShares - 1) return peel + 8 * v + 8 <= rem;
    return peel == 0 && rem == kChunk;
}

// ------------------------------------------------------------- element access ---

__device__ __forceinline__ float load_one(const void* p, int type, int64_t e) {
    if (type == ZS_F32) return __ldcs((const float*)p + e);
    const unsigned short h = __ldcs((const unsigned short*)p + e);
    return type == ZS_F16 ? __half2float(__ushort_as_half(h)) : __bfloat162float(__ushort_as_bfloat16(h));
}
// Eight gradients as they lie in memory: 16-bit ones in w[0..3], else w[0..7].
__device__ __forceinline__ void load_raw8(const void* p, int type, int64_t e, uint32_t* w) {
    if (type == ZS_F32) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>((const float*)p + e));
        const uint4 b = __ldcs(reinterpret_cast<const uint4*>((const float*)p + e + 4));
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
        Mem<8>::load_h_words((const uint16_t*)p + e, w);
    }
}
// The same from eight fp32 values (every value of the types is one).
__device__ __forceinline__ void raw_of(const float* g, int type, uint32_t* w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(g[i]);
    if (type == ZS_F32) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(g[2 * i], g[2 * i + 1]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(g[2 * i], g[2 * i + 1]);
        w[i] = type == ZS_F16 ? *reinterpret_cast<const uint32_t*>(&h) : *reinterpret_cast<const uint32_t*>(&b);
    }
}
// As fp32 pairs.
__device__ __forceinline__ void widen_raw(const uint32_t* w, int type, uint64_t* x) {
    if (type == ZS_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else if (type == ZS_F16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[i] = pair(f.x, f.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)  // bf16 is the upper half of an fp32
            x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
}
__device__ __forceinline__ void store_one16(void* p, int type, int64_t e, float x) {
    __stcs((unsigned short*)p + e, type == ZS_F16 ? __half_as_ushort(__float2half_rn(x))
                                                  : __bfloat16_as_ushort(__float2bfloat16_rn(x)));
}
__device__ __forceinline__ void store_param8(void* p, int type, int64_t e, const float* x) {
    if (type == ZS_F16) {
        Mem<8>::store_h((uint16_t*)p + e, x);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        __stcs(reinterpret_cast<uint4*>((uint16_t*)p + e), make_uint4(w[0], w[1], w[2], w[3]));
    }
}

// ------------------------------------------------------------------- norm ---

struct NormEntry {
    const void* grad;
    int64_t n;
    int32_t type;
};
// Tensors of a launch: as many as the parameters hold, or a few, with parameters
// of a few KB (the launch of 30 small tensors takes 0.6 to 0.9 us less so).
constexpr int kNormGroup = 1024, kStepGroup32 = 448, kStepGroup8 = 240, kFewTensors = 48;
constexpr int kNormThreads = 256, kNormVectors = 8;                // 16-byte vectors of a thread in a chunk
constexpr int kNormChunk = kNormThreads * kNormVectors;            // vectors of a chunk

template <int G>
struct NormArgs {
    NormEntry t[G];
    uint32_t first[G + 1];  // first chunk of each tensor in the launch
    int32_t count;
    int32_t base;      // where this launch's partial sums start
    int32_t finish;    // the call's last launch adds up all of them
    zs_ctrl* ctrl;
    double* out;
    Work* work;
};
static_assert(sizeof(NormArgs<kNormGroup>) <= 32764, "kernel parameters");

// The elements of a gradient before its first 16-byte vector.
__host__ __device__ __forceinline__ int64_t norm_head(const void* grad, int size, int64_t n) {
    const int64_t head = (int64_t)(((16u - ((uintptr_t)grad & 15u)) & 15u) / (unsigned)size);
    return head < n ? head : n;
}

// The tensor of chunk q: the last one whose first chunk is not above q.  i: one
// that is not past it (a block's chunks only go up, most often within a tensor).
__device__ __forceinline__ int tensor_of(const uint32_t* first, int count, uint32_t q, int i) {
    if (q < first[i + 1]) return i;
    int lo = i + 1, hi = count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= q) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// 2 or 4 bytes read for an element and some 6 instructions: 204 us for 667 M fp16
// elements, 6.5 TB/s, which is the copy rate less 4 %.  A chunk is 2048
// vectors of one gradient, each thread's eight under way together; elements
// outside whole vectors are taken by the first chunk of a tensor.
template <int G>
__global__ void __launch_bounds__(kNormThreads) tensors_sqnorm_kernel(const __grid_constant__ NormArgs<G> p) {
    constexpr int kWarps = kNormThreads / 32;
    __shared__ double s_part[kWarps];
    griddep_wait();
    griddep_launch_dependents();
    const float inv = __double2float_rn(__ddiv_rn(1.0, p.ctrl->loss_scale));
    const uint64_t inv2 = pair(inv, inv);
    Sum2 sum{0.0f, 0.0f};
    bool bad = false;
    const uint32_t total = p.first[p.count];
    int i = 0;
    // eight squares, or four: a gradient too large, an infinity or a NaN shows
    auto add = [&](uint64_t part) {
        float a, b;
        split(part, a, b);
        a = __fadd_rn(a, b);
        bad |= !(a < 0x1p124f);
        sum.add(a);
    };
    for (uint32_t q = blockIdx.x; q < total; q += gridDim.x) {
        i = tensor_of(p.first, p.count, q, i);
        const NormEntry& t = p.t[i];
        const int type = t.type, size = type == ZS_F32 ? 4 : 2;
        const int64_t n = t.n, head = norm_head(t.grad, size, n), nvec = (n - head) * size / 16;
        const uint32_t c = q - p.first[i];
        const uint4* v = reinterpret_cast<const uint4*>((const char*)t.grad + head * size);
        uint4 r[kNormVectors];
        const int64_t v0 = (int64_t)c * kNormChunk + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kNormVectors; ++k) {
            const int64_t x = v0 + k * kNormThreads;
            const bool have = x < nvec && ZS_RANGE_OK(kSiteTensorNorm, head + x * (16 / size), 16 / size, n);
            r[k] = have ? __ldcs(v + x) : make_uint4(0u, 0u, 0u, 0u);
        }
        if (c == 0 && threadIdx.x < 16) {  // the head's elements, and the tail's
            const int64_t e = threadIdx.x < 8 ? (int64_t)threadIdx.x : head + nvec * (16 / size) + threadIdx.x - 8;
            if ((threadIdx.x < 8 ? e < head : e < n) && ZS_RANGE_OK(kSiteTensorNorm, e, 1, n)) {
                const float x = __fmul_rn(load_one(t.grad, type, e), inv);
                add(pair(__fmul_rn(x, x), 0.0f));
            }
        }
#pragma unroll
        for (int k = 0; k < kNormVectors; ++k) {
            const uint32_t w[8] = {r[k].x, r[k].y, r[k].z, r[k].w, 0u, 0u, 0u, 0u};
            uint64_t x[4], part = 0ull;
            widen_raw(w, type, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= 2 && type == ZS_F32) break;
                x[j] = mul2(x[j], inv2);
                part = fma2(x[j], x[j], part);
            }
            add(part);
        }
    }
    // (sixteen parts just below the test's bound already pass the largest fp32)
    bad |= !(fabsf(sum.hi) < INFINITY);
    if (__syncthreads_or(bad) && threadIdx.x == 0) atomicOr(&p.ctrl->overflow, 1);
    auto block_sum = [&](double x) {  // in the first thread; the order is fixed
        x = warp_sum(x);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = x;
        __syncthreads();
        x = 0.0;
        if (threadIdx.x == 0)
            for (int w = 0; w < kWarps; ++w) x += s_part[w];
        return x;
    };
    const double block = block_sum(sum.value());
    if (threadIdx.x == 0) p.work->part[p.base + blockIdx.x] = block;
    if (!p.finish || !last_to_arrive(p.work, gridDim.x)) return;
    double all = 0.0;
    const int parts = p.base + (int)gridDim.x;
    for (int k = threadIdx.x; k < parts; k += kNormThreads) all += *(volatile double*)&p.work->part[k];
    all = block_sum(all);
    if (threadIdx.x == 0) *p.out = all;
}

// ------------------------------------------------------------------ update ---

struct StepEntry {
    const void* grad;
    float* master;
    float *m, *v;
    void* param;
    int64_t n;
    float lr, wd;
    int16_t grad_type, param_type;  // param_type only where param is set
    int32_t peel;
};
struct StepEntry8 : StepEntry {
    float *m_scale, *v_scale;
    __device__ __forceinline__ uint8_t* m_codes() const { return (uint8_t*)m; }
    __device__ __forceinline__ uint8_t* v_codes() const { return (uint8_t*)v; }
};

struct StepShared {
    zs_adam hp;
    double max_norm;
    const double* sqnorm;
    zs_ctrl* ctrl;
    int32_t count;
    int32_t finish;  // the call's last launch ends the step in the control block
    float one;       // 1: see add2_apart
};
template <typename Entry, int G>
struct StepArgs : StepShared {
    Entry t[G];
    uint32_t first[G + 1];
};
// (of the code maps only the values and thresholds)
struct MapValues {
    float dec7[256], mag8[256], thr7[128], thr8[256];
};
template <int G>
struct StepArgs8 : StepArgs<StepEntry8, G> {
    MapValues maps;
};
template <int G>
using StepArgs32 = StepArgs<StepEntry, G>;
static_assert(sizeof(StepArgs32<kStepGroup32>) <= 32764 && sizeof(StepArgs8<kStepGroup8>) <= 32764, "kernel parameters");

// The step's coefficients, whether it is skipped, and the clip factor.
struct StepCoef {
    Coef c;
    float clip;
    int skip;
};
__device__ __forceinline__ void step_coef(const StepShared& p, StepCoef* s) {
    const zs_ctrl* ctrl = p.ctrl;
    s->c = coef_device(p.hp, __dmul_rn(ctrl->beta1_pow, p.hp.beta1), __dmul_rn(ctrl->beta2_pow, p.hp.beta2), 1,
                       ctrl->loss_scale);
    double c = 1.0;
    if (p.max_norm > 0.0) {
        c = __ddiv_rn(p.max_norm, __dadd_rn(__dsqrt_rn(*p.sqnorm), 1e-6));
        if (!(c < 1.0)) c = 1.0;
    }
    s->clip = __double2float_rn(c);
    s->skip = ctrl->overflow;
}

// The step's coefficients twice each, for pairs of elements.
struct Coef2 {
    uint64_t b1, c1, b2, c2, inv, clip, one;
    float bc1, bc2, rcp_bc1, rcp_bc2, eps;
    // where adam_eight's smallest and largest value start: a low below 2^-80 sends
    // every group to the scalar operations, a high above 0 groups of zeros
    float low, high;
};
__device__ __forceinline__ Coef2 coef2_of(const StepCoef& s, float one) {
    // (with these a root's argument is at most 2^80 and its sum with eps 2^41)
    const bool fast = s.c.eps <= 0x1p40f && s.c.bc1 >= 0x1p-40f && s.c.bc2 >= 0x1p-40f;
    return Coef2{pair(s.c.b1, s.c.b1), pair(s.c.c1, s.c.c1), pair(s.c.b2, s.c.b2), pair(s.c.c2, s.c.c2),
                 pair(s.c.inv, s.c.inv), pair(s.clip, s.clip), pair(one, one), s.c.bc1, s.c.bc2, __frcp_rn(s.c.bc1),
                 __frcp_rn(s.c.bc2), s.c.eps, fast ? 1.0f : 0.0f, fast && s.c.eps > 0.0f ? 0.0f : 0x1p-80f};
}

// a + b for products of pairs that have been rounded: as a 1 + b, with a 1 that
// the compiler does not see.  It makes one fused multiply-add of a packed
// product and a packed sum, rounding modifiers or not, and m and v came out a
// unit of the last place off.
__device__ __forceinline__ uint64_t add2_apart(uint64_t a, uint64_t b, uint64_t one) { return fma2(a, one, b); }

// The larger of two, NaN if one is (fmaxf passes over a NaN).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The Adam / AdamW update of eight coordinates from their gradients (raw, as
// pairs): the operations of adam_apply, two coordinates at a time.  Divisions and
// square roots are the correctly rounded ones above where all of a warp's values
// lie in [2^-80, 2^40] and eps and the bias corrections keep what follows in those
// operations' ranges, or all eight of a thread's are 0 (weights that no gradient
// has reached; with eps = 0 they have no quotient, and the scalar operations say
// so), and else the scalar ones.  The tests pass over a NaN, which comes out of
// either as a NaN.  m, v: in and out, as pairs.
__device__ __forceinline__ void adam_eight(const Coef2& c, float lr, float wd, const uint64_t* g, float* th, uint64_t* m,
                                           uint64_t* v) {
    float low = c.low, high = c.high;  // the smallest and largest |m'|, v'
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint64_t x = mul2(mul2(g[j], c.inv), c.clip);
        m[j] = add2_apart(mul2(c.b1, m[j]), mul2(c.c1, x), c.one);
        v[j] = add2_apart(mul2(c.b2, v[j]), mul2(c.c2, mul2(x, x)), c.one);
        float a, b, p, q;
        split(m[j], a, b);
        split(v[j], p, q);
        low = fminf(fminf(low, fminf(fabsf(a), fabsf(b))), fminf(p, q));
        high = fmaxf(fmaxf(high, fmaxf(fabsf(a), fabsf(b))), fmaxf(p, q));
    }
    if (__any_sync(0xffffffffu, !(low >= 0x1p-80f && high <= 0x1p40f) && high != 0.0f)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float a[2], p[2];
            split(m[j / 2], a[0], a[1]);
            split(v[j / 2], p[0], p[1]);
            const float u = __fdiv_rn(__fdiv_rn(a[j & 1], c.bc1), __fadd_rn(__fsqrt_rn(__fdiv_rn(p[j & 1], c.bc2)), c.eps));
            th[j] = __fsub_rn(th[j], __fmul_rn(lr, __fadd_rn(u, __fmul_rn(wd, th[j]))));
        }
        return;
    }
    const uint64_t eps = pair(c.eps, c.eps);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint64_t mh = div2_by_constant(m[j], c.bc1, c.rcp_bc1), vh = div2_by_constant(v[j], c.bc2, c.rcp_bc2);
        float u0, u1, p, q;
        split(vh, p, q);  // (a v' of 0 belongs to an m' of 0: any root will do)
        split(div2(mh, add2(sqrt2(pair(max_nan(p, 0x1p-80f), max_nan(q, 0x1p-80f))), eps)), u0, u1);
        th[2 * j] = __fsub_rn(th[2 * j], __fmul_rn(lr, __fadd_rn(u0, __fmul_rn(wd, th[2 * j]))));
        th[2 * j + 1] = __fsub_rn(th[2 * j + 1], __fmul_rn(lr, __fadd_rn(u1, __fmul_rn(wd, th[2 * j + 1]))));
    }
}

// Where a chunk is: its tensor, its first element there and its length.
struct Place {
    int i;
    int64_t at;
    int rem;
};
template <typename Args>
__device__ __forceinline__ Place place_of(const Args& p, uint32_t q, int from) {
    const int i = tensor_of(p.first, p.count, q, from);
    const int64_t at = (int64_t)(q - p.first[i]) * kChunk, left = p.t[i].n - at;
    return Place{i, at, (int)(left < kChunk ? left : kChunk)};
}

// Threads of the step's blocks and blocks of an SM.  fp32 states, 1200 tensors of
// 94 M elements in all, with the norm: 493 us so, 509 us with four blocks of 128
// threads (two vectors each), 532 us with four of 256 (64 registers).  8-bit
// states, 667 M elements, norm, step and values in an earlier form of them: 4.44 ms
// so, 4.54 with three blocks of 256, 4.66 and 5.36 with four and five blocks of 128
// threads (two shares each).
constexpr int kThreads32 = 256, kBlocks32 = 3, kThreads8 = 256, kBlocks8 = 4;

// fp32 states have no blocks, so their chunks start at the tensor's first vector
// boundary; the elements before it and after the last whole vector, at most
// seven each, are taken one to a thread by the first chunk.
__host__ __device__ __forceinline__ int64_t chunks_of(int64_t n, int peel) {
    const int64_t body = n - (peel == kScattered ? 0 : peel);
    return body > kChunk ? (body + kChunk - 1) / kChunk : 1;
}

// 28 bytes in and out for an element with a 16-bit gradient and copy, and some
// 50 instructions.  With the norm before it, 1200 tensors of 94 M elements end to
// end in the gradient buffer: 492 us, 5.7 TB/s of the two passes' 30 bytes.
template <int G>
__global__ void __launch_bounds__(kThreads32, kBlocks32) tensors_adamw_kernel(const __grid_constant__ StepArgs32<G> p) {
    constexpr int kPer = kChunk / 8 / kThreads32;  // vectors of a thread in a chunk
    __shared__ StepCoef s_coef;
    griddep_wait();
    griddep_launch_dependents();
    if (threadIdx.x == 0) step_coef(p, &s_coef);
    __syncthreads();
    const Coef2 c = coef2_of(s_coef, p.one);
    const uint32_t total = s_coef.skip ? 0u : p.first[p.count];
    int i = 0;
    for (uint32_t q = blockIdx.x; q < total; q += gridDim.x) {
        i = tensor_of(p.first, p.count, q, i);
        const StepEntry& t = p.t[i];
        const int64_t n = t.n;
        const int peel = t.peel, type = t.grad_type;
        const uint32_t chunk = q - p.first[i];
        const float lr = t.lr, wd = t.wd;
        auto one = [&](int64_t e) {
            if (e >= n || !ZS_RANGE_OK(kSiteTensor, e, 1, n)) return;
            float th = __ldcs(t.master + e), m = __ldcs(t.m + e), v = __ldcs(t.v + e);
            Coef k = s_coef.c;
            k.lr = lr;
            k.wd = wd;
            adam_apply<false>(k, __fmul_rn(__fmul_rn(load_one(t.grad, type, e), k.inv), s_coef.clip), th, m, v);
            __stcs(t.master + e, th);
            __stcs(t.m + e, m);
            __stcs(t.v + e, v);
            if (t.param != nullptr) store_one16(t.param, t.param_type, e, th);
        };
        if (peel == kScattered) {
            for (int j = threadIdx.x; j < kChunk; j += kThreads32) one((int64_t)chunk * kChunk + j);
            continue;
        }
        const int64_t e0 = peel + (int64_t)chunk * kChunk + 8 * threadIdx.x;
        uint32_t w[kPer][8];
        float th[kPer][8], m8[kPer][8], v8[kPer][8];
#pragma unroll
        for (int h = 0; h < kPer; ++h) {
            const int64_t e = e0 + 8 * h * kThreads32;
            if (e + 8 <= n && ZS_RANGE_OK(kSiteTensor, e, 8, n)) {
                load_raw8(t.grad, type, e, w[h]);
                Mem<8>::load_f(t.master + e, th[h]);
                Mem<8>::load_f(t.m + e, m8[h]);
                Mem<8>::load_f(t.v + e, v8[h]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {  // not there: anything harmless
                    w[h][j] = 0u;
                    th[h][j] = 0.0f;
                    m8[h][j] = v8[h][j] = 1.0f;
                }
            }
        }
        if (chunk == 0 && threadIdx.x < 16) {
            const int64_t tail = n > peel ? n - (n - peel) % 8 : n;
            const int64_t e = threadIdx.x < 8 ? (int64_t)threadIdx.x : tail + threadIdx.x - 8;
            if (threadIdx.x >= 8 || e < peel) one(e);
        }
#pragma unroll
        for (int h = 0; h < kPer; ++h) {
            uint64_t g[4], m[4], v[4];
            widen_raw(w[h], type, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                m[j] = pair(m8[h][2 * j], m8[h][2 * j + 1]);
                v[j] = pair(v8[h][2 * j], v8[h][2 * j + 1]);
            }
            adam_eight(c, lr, wd, g, th[h], m, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                split(m[j], m8[h][2 * j], m8[h][2 * j + 1]);
                split(v[j], v8[h][2 * j], v8[h][2 * j + 1]);
            }
            const int64_t e = e0 + 8 * h * kThreads32;
            if (e + 8 <= n && ZS_RANGE_OK(kSiteTensor, e, 8, n)) {
                Mem<8>::store_f(t.master + e, th[h]);
                Mem<8>::store_f(t.m + e, m8[h]);
                Mem<8>::store_f(t.v + e, v8[h]);
                if (t.param != nullptr) store_param8(t.param, t.param_type, e, th[h]);
            }
        }
    }
    if (p.finish && threadIdx.x == 0) arrive_and_finish(p.ctrl, gridDim.x, p.hp.beta1, p.hp.beta2);
}

// The nearest-code search of adam8_math.cuh with a bucket's threshold and code
// in one 8-byte entry, and without the octaves below each map's lowest
// threshold (5e-7 and 5e-8).
constexpr int kOctaves7 = 21, kOctaves8 = 25;
constexpr int kLut7 = kOctaves7 * (1 << kMantBits) + 1, kLut8 = kOctaves8 * (1 << kMantBits) + 1;
struct CodeTables {
    uint2 lut7[kLut7], lut8[kLut8];  // {threshold, number of thresholds below the bucket}
    float dec7[256], mag8[256], thr7[128], thr8[256];
};
template <int OCTAVES>
__device__ __forceinline__ uint32_t lut_code(float a, const uint2* lut) {
    constexpr uint32_t lowest = (uint32_t)(127 - OCTAVES) << 23;
    a = fmaxf(a, __uint_as_float(lowest));  // (a NaN becomes the lowest: code 0)
    const uint2 e = lut[(int)(__float_as_uint(a) >> kBucketShift) - (int)(lowest >> kBucketShift)];
    return e.y + (a > __uint_as_float(e.x) ? 1u : 0u);
}
// From the thresholds: thr[k] lies in bucket b_k, and the buckets above b_(k-1)
// up to b_k have k thresholds below them.  A warp fills one k's at a time (some
// have hundreds; one to a thread took 25 us); the buckets below the lowest
// threshold and above the highest are the first's and the last's.
template <int OCTAVES, int COUNT, int SIZE>
__device__ __forceinline__ void build_lut(const float (&thr)[COUNT], uint2 (&lut)[SIZE]) {
    constexpr uint32_t lowest = (uint32_t)(127 - OCTAVES) << 23;
    auto bucket = [&](int k) { return (int)((__float_as_uint(thr[k]) - lowest) >> kBucketShift); };
    for (int k = threadIdx.x / 32; k < COUNT; k += blockDim.x / 32) {
        const int from = k == 0 ? 0 : bucket(k - 1) + 1, to = k == COUNT - 1 ? SIZE - 1 : bucket(k);
        for (int b = from + (int)(threadIdx.x & 31); b <= to; b += 32) lut[b] = make_uint2(__float_as_uint(thr[k]), (uint32_t)k);
    }
}

// A thread's shares of a chunk with 8-bit states, as they lie in memory.
template <int kPerThread>
struct Shares8 {
    uint32_t g[kPerThread][8];
    float th[kPerThread][8];
    uint2 cm[kPerThread], cv[kPerThread];
    float ms, vs;
};
template <int kPerThread>
__device__ __forceinline__ void load_shares8(const StepEntry8& t, const Place& at, Shares8<kPerThread>& s) {
    constexpr int kStepThreads = kShares / kPerThread;
    const int64_t block = at.at / kChunk;
    const int peel = t.peel, type = t.grad_type;
    const void* grad = (const char*)t.grad + at.at * (type == ZS_F32 ? 4 : 2);
    const float* master = t.master + at.at;
    const uint8_t *mc = t.m_codes() + at.at, *vc = t.v_codes() + at.at;
    [[maybe_unused]] const int64_t left = t.n - at.at;
    const bool scale_ok = ZS_RANGE_OK(kSiteTensorScale, block, 1, (t.n + kChunk - 1) / kChunk);
    s.ms = scale_ok ? __ldcs(t.m_scale + block) : 0.0f;
    s.vs = scale_ok ? __ldcs(t.v_scale + block) : 0.0f;
#pragma unroll
    for (int h = 0; h < kPerThread; ++h) {
        const int v = threadIdx.x + h * kStepThreads, e = share_element(peel, v, 0);
        if (share_is_vector(peel, v, at.rem) && ZS_RANGE_OK(kSiteTensor, e, 8, left)) {
            load_raw8(grad, type, e, s.g[h]);
            Mem<8>::load_f(master + e, s.th[h]);
            s.cm[h] = __ldcs(reinterpret_cast<const uint2*>(mc + e));
            s.cv[h] = __ldcs(reinterpret_cast<const uint2*>(vc + e));
        } else {
            // (elements that are not there: code 0, gradient 0; their m' = v' = 0
            // changes no block maximum)
            float g[8];
            uint32_t cm[8], cv[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = share_element(peel, v, j);
                const bool have = k < at.rem && ZS_RANGE_OK(kSiteTensor, k, 1, left);
                g[j] = have ? load_one(grad, type, k) : 0.0f;
                s.th[h][j] = have ? __ldcs(master + k) : 0.0f;
                cm[j] = have ? mc[k] : 0u;
                cv[j] = have ? vc[k] : 0u;
            }
            raw_of(g, type, s.g[h]);
            s.cm[h] = make_uint2(cm[0] | cm[1] << 8 | cm[2] << 16 | cm[3] << 24, cm[4] | cm[5] << 8 | cm[6] << 16 | cm[7] << 24);
            s.cv[h] = make_uint2(cv[0] | cv[1] << 8 | cv[2] << 16 | cv[3] << 24, cv[4] | cv[5] << 8 | cv[6] << 16 | cv[7] << 24);
        }
    }
}

// 8-bit states: 16 bytes in and out for an element with a 16-bit gradient and
// copy, but 99 instructions for an element, pairs of elements sharing them where they
// can: 2.72 ms for 667 M elements, 3.9 TB/s, 58 % of the copy rate, with 2.5 of 4
// issue slots used.  A chunk is a block of states: its largest |m'| and v' take
// one barrier (the slots alternate).
template <int G>
__global__ void __launch_bounds__(kThreads8, kBlocks8) tensors_adamw8_kernel(const __grid_constant__ StepArgs8<G> p) {
    constexpr int kStepThreads = kThreads8, kPerThread = kShares / kStepThreads, kWarps = kStepThreads / 32;
    extern __shared__ __align__(16) unsigned char s_dynamic[];
    CodeTables& s_tab = *reinterpret_cast<CodeTables*>(s_dynamic);
    __shared__ StepCoef s_coef;
    __shared__ __align__(16) uint32_t s_max[2][2][kWarps];
    static_assert(kWarps % 4 == 0, "the warps' maxima are read four at a time");
    // the tables, from the kernel parameters; global memory only from here
    for (int i = threadIdx.x; i < 256; i += kStepThreads) {
        s_tab.dec7[i] = p.maps.dec7[i];
        s_tab.mag8[i] = p.maps.mag8[i];
        s_tab.thr8[i] = p.maps.thr8[i];
        if (i < 128) s_tab.thr7[i] = p.maps.thr7[i];
    }
    __syncthreads();
    build_lut<kOctaves7>(s_tab.thr7, s_tab.lut7);
    build_lut<kOctaves8>(s_tab.thr8, s_tab.lut8);
    griddep_wait();
    griddep_launch_dependents();
    if (threadIdx.x == 0) step_coef(p, &s_coef);
    __syncthreads();
    const Coef2 c = coef2_of(s_coef, p.one);
    const uint32_t total = s_coef.skip ? 0u : p.first[p.count];
    int par = 0;
    Place at{0, 0, 0};
    if (blockIdx.x < total) at = place_of(p, blockIdx.x, 0);
    for (uint32_t q = blockIdx.x; q < total; q += gridDim.x, par ^= 1) {
        const StepEntry8& t = p.t[at.i];
        const int64_t block = at.at / kChunk;
        const int peel = t.peel, type = t.grad_type, rem = at.rem, param_type = t.param_type;
        float* master = t.master + at.at;
        uint8_t *mc = t.m_codes() + at.at, *vc = t.v_codes() + at.at;
        uint16_t* param = t.param == nullptr ? nullptr : (uint16_t*)t.param + at.at;
        float *m_scale = t.m_scale + block, *v_scale = t.v_scale + block;
        const float lr = t.lr, wd = t.wd;
        [[maybe_unused]] const int64_t left = t.n - at.at;
        Shares8<kPerThread> s;
        load_shares8<kPerThread>(t, at, s);
        if (q + gridDim.x < total) at = place_of(p, q + gridDim.x, at.i);
        uint64_t g[kPerThread][4], m[kPerThread][4], v2[kPerThread][4];
        const uint64_t ms = pair(s.ms, s.ms), vs = pair(s.vs, s.vs);
#pragma unroll
        for (int h = 0; h < kPerThread; ++h) {
            widen_raw(s.g[h], type, g[h]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t wm = j < 2 ? s.cm[h].x : s.cm[h].y, wv = j < 2 ? s.cv[h].x : s.cv[h].y;
                const int b = 2 * (j & 1);
                m[h][j] = mul2(pair(s_tab.dec7[__byte_perm(wm, 0u, 0x4440u + b)], s_tab.dec7[__byte_perm(wm, 0u, 0x4441u + b)]), ms);
                v2[h][j] = mul2(pair(s_tab.mag8[__byte_perm(wv, 0u, 0x4440u + b)], s_tab.mag8[__byte_perm(wv, 0u, 0x4441u + b)]), vs);
            }
        }
        float am = 0.0f, av = 0.0f;
#pragma unroll
        for (int h = 0; h < kPerThread; ++h) {
            adam_eight(c, lr, wd, g[h], s.th[h], m[h], v2[h]);
            const int v = threadIdx.x + h * kStepThreads, e = share_element(peel, v, 0);
            if (share_is_vector(peel, v, rem) && ZS_RANGE_OK(kSiteTensor, e, 8, left)) {
                Mem<8>::store_f(master + e, s.th[h]);
                if (param != nullptr) store_param8(param, param_type, e, s.th[h]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int k = share_element(peel, v, j);
                    if (k >= rem || !ZS_RANGE_OK(kSiteTensor, k, 1, left)) continue;
                    __stcs(master + k, s.th[h][j]);
                    if (param != nullptr) store_one16(param, param_type, k, s.th[h][j]);
                }
            }
            // the block's largest |m'| and v', by their bit patterns
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a, b;
                split(m[h][j], a, b);
                am = fmaxf(am, fmaxf(fabsf(a), fabsf(b)));
                split(v2[h][j], a, b);
                av = fmaxf(av, fmaxf(a, b));
            }
        }
        const uint32_t wm = __reduce_max_sync(0xffffffffu, __float_as_uint(am));
        const uint32_t wv = __reduce_max_sync(0xffffffffu, __float_as_uint(av));
        if ((threadIdx.x & 31) == 0) {
            s_max[par][0][threadIdx.x >> 5] = wm;
            s_max[par][1][threadIdx.x >> 5] = wv;
        }
        __syncthreads();  // one barrier per block: a parity's slots are not rewritten before every warp read them
        uint32_t bm = 0u, bv = 0u;
#pragma unroll
        for (int w = 0; w < kWarps; w += 4) {
            const uint4 a = *reinterpret_cast<const uint4*>(&s_max[par][0][w]), b = *reinterpret_cast<const uint4*>(&s_max[par][1][w]);
            bm = max(bm, max(max(a.x, a.y), max(a.z, a.w)));
            bv = max(bv, max(max(b.x, b.y), max(b.z, b.w)));
        }
        am = __uint_as_float(bm);
        av = __uint_as_float(bv);
        // codes of m' / am and v' / av, each quotient rounded once
        const bool usual = scale_divisor_ok(am) && scale_divisor_ok(av);
        float rm = 0.0f, rv = 0.0f;
        if (usual) split(reciprocal2(pair(am, av)), rm, rv);
#pragma unroll
        for (int h = 0; h < kPerThread; ++h) {
            uint32_t cm[8], cv[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x[2], y[2];
                if (usual) {
                    split(div2_by_constant(m[h][j], am, rm), x[0], x[1]);
                    split(div2_by_constant(v2[h][j], av, rv), y[0], y[1]);
                } else {
                    split(m[h][j], x[0], x[1]);
                    split(v2[h][j], y[0], y[1]);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        x[b] = am > 0.0f ? __fdiv_rn(x[b], am) : 0.0f;
                        y[b] = av > 0.0f ? __fdiv_rn(y[b], av) : 0.0f;
                    }
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint32_t k = lut_code<kOctaves7>(fabsf(x[b]), s_tab.lut7);
                    cm[2 * j + b] = x[b] < 0.0f && k > 0u ? k | 0x80u : k;
                    cv[2 * j + b] = lut_code<kOctaves8>(y[b], s_tab.lut8);
                }
            }
            const int v = threadIdx.x + h * kStepThreads, e = share_element(peel, v, 0);
            if (share_is_vector(peel, v, rem) && ZS_RANGE_OK(kSiteTensor, e, 8, left)) {
                auto four = [](const uint32_t* x) {
                    return __byte_perm(__byte_perm(x[0], x[1], 0x0040u), __byte_perm(x[2], x[3], 0x0040u), 0x5410u);
                };
                __stcs(reinterpret_cast<uint2*>(mc + e), make_uint2(four(cm), four(cm + 4)));
                __stcs(reinterpret_cast<uint2*>(vc + e), make_uint2(four(cv), four(cv + 4)));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int k = share_element(peel, v, j);
                    if (k >= rem || !ZS_RANGE_OK(kSiteTensor, k, 1, left)) continue;
                    mc[k] = (uint8_t)cm[j];
                    vc[k] = (uint8_t)cv[j];
                }
            }
        }
        if (threadIdx.x == 0 && ZS_RANGE_OK(kSiteTensorScale, block, 1, (left + block * kChunk + kChunk - 1) / kChunk)) {
            *m_scale = am;
            *v_scale = av;
        }
    }
    if (p.finish && threadIdx.x == 0) arrive_and_finish(p.ctrl, gridDim.x, p.hp.beta1, p.hp.beta2);
}

// ------------------------------------------------------------- 8-bit values ---

constexpr int kValueThreads = 256;

struct ValueArgs {
    const uint8_t* codes;
    const float* scales;
    float* out;
    int64_t n;
    int32_t wide;        // codes on 4-byte, out on 16-byte boundaries
    float map[256];
};

// 5 bytes in and out for an element: 667 M elements in 543 us, 6.1 TB/s, 90 % of the
// copy rate.
__global__ void __launch_bounds__(kValueThreads) adam8_values_kernel(const __grid_constant__ ValueArgs p) {
    __shared__ float s_map[256];
    s_map[threadIdx.x] = p.map[threadIdx.x];
    griddep_wait();
    griddep_launch_dependents();
    __syncthreads();
    // a warp takes 512 codes: each lane 4, 128 apart, so that its stores are
    // whole lines
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kValueThreads / 32), warp = ((int64_t)blockIdx.x * kValueThreads + threadIdx.x) / 32;
    const int64_t whole = p.wide ? p.n / 512 : 0;
    for (int64_t i = warp; i < whole; i += warps) {
        const uint32_t* from = reinterpret_cast<const uint32_t*>(p.codes + 512 * i) + lane;
        const float s = __ldg(p.scales + 512 * i / ZS_ADAM8_BLOCK);
        uint32_t c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = __ldcs(from + 32 * k);
        float4* to = reinterpret_cast<float4*>(p.out + 512 * i) + lane;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            __stcs(to + 32 * k, make_float4(__fmul_rn(s_map[c[k] & 0xffu], s), __fmul_rn(s_map[c[k] >> 8 & 0xffu], s),
                                            __fmul_rn(s_map[c[k] >> 16 & 0xffu], s), __fmul_rn(s_map[c[k] >> 24], s)));
    }
    const int64_t stride = (int64_t)gridDim.x * kValueThreads;
    for (int64_t i = whole * 512 + (int64_t)blockIdx.x * kValueThreads + threadIdx.x; i < p.n; i += stride)
        p.out[i] = __fmul_rn(s_map[p.codes[i]], __ldg(p.scales + i / ZS_ADAM8_BLOCK));
}

// -------------------------------------------------------------------- host ---

struct HostMaps {
    float dec7[256];
    Maps maps;
    bool ok;
};

const HostMaps& host_maps() {
    static const HostMaps built = [] {
        HostMaps h;
        std::memset(&h, 0, sizeof(h));
        float mag7[128];
        for (int k = 0; k < 128; ++k) mag7[k] = map_value(k, 7);
        for (int c = 0; c < 256; ++c) h.maps.dec7[c] = (c & 0x80) ? -mag7[c & 0x7f] : mag7[c & 0x7f];
        for (int k = 0; k < 256; ++k) h.maps.mag8[k] = map_value(k, 8);
        h.ok = build_search(mag7, 128, h.maps.thr7, h.maps.bucket7) &&
               build_search(h.maps.mag8, 256, h.maps.thr8, h.maps.bucket8);
        return h;
    }();
    return built;
}

bool known_type(int32_t t) { return t == ZS_F32 || t == ZS_F16 || t == ZS_BF16; }

int32_t check_grads(const zs_tensor* t, int32_t n) {
    if (t == nullptr || n < 1 || n > ZS_MAX_TENSORS) return ZS_ERR_ARG;
    int64_t chunks = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (t[i].n < 0 || t[i].n > (1ll << 40) || !known_type(t[i].grad_type) || t[i].reserved != 0) return ZS_ERR_ARG;
        if (t[i].n > 0 && t[i].grad == nullptr) return ZS_ERR_ARG;
        if (!zs::aligned_to(t[i].grad, t[i].grad_type == ZS_F32 ? 4 : 2)) return ZS_ERR_ALIGN;
        chunks += t[i].n / kChunk + 1;
    }
    return chunks < (1ll << 31) ? ZS_OK : ZS_ERR_ARG;
}

int32_t check_states(const zs_tensor* t, int32_t n) {
    for (int32_t i = 0; i < n; ++i) {
        const zs_tensor& x = t[i];
        if (x.state != ZS_STATE_F32 && x.state != ZS_STATE_U8) return ZS_ERR_ARG;
        if (!finite_double(x.lr_mult) || !finite_double(x.decay_mult)) return ZS_ERR_ARG;
        if (x.param != nullptr && x.param_type != ZS_F16 && x.param_type != ZS_BF16) return ZS_ERR_ARG;
        const bool small = x.state == ZS_STATE_U8;
        if (x.n > 0 && (x.master == nullptr || x.m == nullptr || x.v == nullptr)) return ZS_ERR_ARG;
        if (x.n > 0 && small && (x.m_scale == nullptr || x.v_scale == nullptr)) return ZS_ERR_ARG;
        if (!zs::aligned_to(x.master, 4) || !zs::aligned_to(x.param, 2)) return ZS_ERR_ALIGN;
        if (small ? !zs::aligned_to(x.m_scale, 4) || !zs::aligned_to(x.v_scale, 4)
                  : !zs::aligned_to(x.m, 4) || !zs::aligned_to(x.v, 4))
            return ZS_ERR_ALIGN;
    }
    return ZS_OK;
}

// The first element in [0, 8) at which every given buffer is on a vector
// boundary; kScattered if there is none.
struct Buffer {
    const void* p;
    int size;  // bytes of an element; 0: not there
};
int common_peel(std::initializer_list<Buffer> bufs) {
    for (int peel = 0; peel < 8; ++peel) {
        bool ok = true;
        for (const Buffer& b : bufs)
            if (b.size != 0 && b.p != nullptr)
                ok = ok && ((uintptr_t)b.p + (uintptr_t)(peel * b.size)) % (b.size == 1 ? 8 : 16) == 0;
        if (ok) return peel;
    }
    return kScattered;
}
int type_size(int32_t t) { return t == ZS_F32 ? 4 : 2; }

// Launches the norm of the tensors, as many at a time as fit.  The partial sums
// of all launches share the scratch buffer.
template <int G>
int32_t launch_norms(const zs_tensor* t, int32_t n, zs_ctrl* ctrl, double* out, Work* work, cudaStream_t stream) {
    const void* kernel = (const void*)tensors_sqnorm_kernel<G>;
    NormArgs<G> a;
    a.ctrl = ctrl;
    a.out = out;
    a.work = work;
    a.base = 0;
    int launches = (n + G - 1) / G;
    for (int32_t i = 0; i < n; --launches) {
        a.first[0] = 0;
        for (a.count = 0; a.count < G && i < n; ++i) {
            const zs_tensor& x = t[i];
            if (x.n == 0) continue;
            a.t[a.count] = NormEntry{x.grad, x.n, x.grad_type};
            const int size = type_size(x.grad_type);
            const int64_t vectors = (x.n - norm_head(x.grad, size, x.n)) * size / 16;
            a.first[a.count + 1] = a.first[a.count] + (uint32_t)(vectors > kNormChunk ? (vectors + kNormChunk - 1) / kNormChunk : 1);
            ++a.count;
        }
        a.finish = i == n;
        const uint32_t chunks = a.first[a.count];
        int blocks = zs::persistent_blocks(kernel, kNormThreads, (int64_t)(chunks > 0 ? chunks : 1) * kNormThreads);
        const int fit = (kWorkParts - a.base) / launches;
        blocks = blocks < fit ? blocks : fit;
        const int32_t rc = launch_ex(tensors_sqnorm_kernel<G>, blocks, kNormThreads, 0, true, stream, a, "tensors_sqnorm_kernel");
        if (rc != ZS_OK) return rc;
        a.base += blocks;
    }
    return ZS_OK;
}

void fill_entry(StepEntry* e, const zs_tensor& x, const zs_adam& hp) {
    e->grad = x.grad;
    e->master = x.master;
    e->m = (float*)x.m;
    e->v = (float*)x.v;
    e->param = x.param;
    e->n = x.n;
    e->lr = (float)(hp.lr * x.lr_mult);
    e->wd = (float)(hp.weight_decay * x.decay_mult);
    e->grad_type = (int16_t)x.grad_type;
    e->param_type = (int16_t)x.param_type;
    const int state = x.state == ZS_STATE_U8 ? 1 : 4;
    e->peel = common_peel({{x.grad, type_size(x.grad_type)}, {x.master, 4}, {x.m, state}, {x.v, state}, {x.param, 2}});
}
void fill(StepEntry* e, const zs_tensor& x, const zs_adam& hp) { fill_entry(e, x, hp); }
void fill(StepEntry8* e, const zs_tensor& x, const zs_adam& hp) {
    fill_entry(e, x, hp);
    e->m_scale = x.m_scale;
    e->v_scale = x.v_scale;
}

// Launches the tensors of one kind of state, as many at a time as fit; the last
// launch ends the step if `finish`.
template <typename Args>
int32_t launch_steps(void (*kernel)(Args), Args& a, int threads, int per_sm, int smem, int32_t state, const zs_tensor* t,
                     int32_t n, const zs_adam& hp, bool finish, cudaStream_t stream, const char* name) {
    constexpr int G = (int)(sizeof(a.t) / sizeof(a.t[0]));
    if (smem > 48 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (err != cudaSuccess) return zs::cuda_fail(err, name);
    }
    int32_t left = 0;
    for (int32_t i = 0; i < n; ++i) left += t[i].state == state && t[i].n > 0;
    a.count = 0;
    a.first[0] = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (t[i].state != state || t[i].n == 0) continue;
        fill(&a.t[a.count], t[i], hp);
        a.first[a.count + 1] = a.first[a.count] + (uint32_t)(state == ZS_STATE_U8 ? (t[i].n + kChunk - 1) / kChunk : chunks_of(t[i].n, a.t[a.count].peel));
        ++a.count;
        --left;
        if (a.count < G && left > 0) continue;
        a.finish = finish && left == 0;
        const int64_t full = (int64_t)per_sm * zs::device_sm_count(), chunks = a.first[a.count];
        const int32_t rc = launch_ex(kernel, (int)(chunks < full ? chunks : full), threads, smem, true, stream, a, name);
        if (rc != ZS_OK) return rc;
        a.count = 0;
    }
    return ZS_OK;
}

template <int G>
int32_t launch_steps8(const StepShared& shared, const zs_tensor* t, int32_t n, bool finish, cudaStream_t stream) {
    if (!host_maps().ok) return zs::fail_with(ZS_ERR_CUDA, "zero_tensors_adamw_async: code tables");
    StepArgs8<G> a;
    static_cast<StepShared&>(a) = shared;
    const Maps& maps = host_maps().maps;
    std::memcpy(a.maps.dec7, maps.dec7, sizeof(a.maps.dec7));
    std::memcpy(a.maps.mag8, maps.mag8, sizeof(a.maps.mag8));
    std::memcpy(a.maps.thr7, maps.thr7, sizeof(a.maps.thr7));
    std::memcpy(a.maps.thr8, maps.thr8, sizeof(a.maps.thr8));
    return launch_steps(tensors_adamw8_kernel<G>, a, kThreads8, kBlocks8, (int)sizeof(CodeTables), ZS_STATE_U8, t, n,
                        shared.hp, finish, stream, "tensors_adamw8_kernel");
}
template <int G>
int32_t launch_steps32(const StepShared& shared, const zs_tensor* t, int32_t n, bool finish, cudaStream_t stream) {
    StepArgs32<G> a;
    static_cast<StepShared&>(a) = shared;
    return launch_steps(tensors_adamw_kernel<G>, a, kThreads32, kBlocks32, 0, ZS_STATE_F32, t, n, shared.hp, finish, stream,
                        "tensors_adamw_kernel");
}

}  // namespace

namespace zs {
uint64_t take_fault_tensors() { return take_fault(); }
}  // namespace zs

extern "C" {

ZS_API int32_t zero_tensors_sqnorm_async(const zs_tensor* tensors, int32_t n_tensors, zs_ctrl* ctrl_dev,
                                         double* sqnorm_dev, void* work_dev, void* stream) {
    zs::NvtxRange nvtx_range("zero_tensors_sqnorm_async");
    const int32_t rc = check_grads(tensors, n_tensors);
    if (rc != ZS_OK) return rc;
    if (ctrl_dev == nullptr || sqnorm_dev == nullptr || work_dev == nullptr) return ZS_ERR_ARG;
    if (!zs::aligned_to(ctrl_dev, 8) || !zs::aligned_to(sqnorm_dev, 8) || !zs::aligned_to(work_dev, 8))
        return ZS_ERR_ALIGN;
    const auto launch = n_tensors <= kFewTensors ? launch_norms<kFewTensors> : launch_norms<kNormGroup>;
    return launch(tensors, n_tensors, ctrl_dev, sqnorm_dev, (Work*)work_dev, (cudaStream_t)stream);
}

ZS_API int32_t zero_tensors_adamw_async(const zs_tensor* tensors, int32_t n_tensors, const zs_adam* hp,
                                        double max_norm, const double* sqnorm_dev, zs_ctrl* ctrl_dev,
                                        void* stream) {
    zs::NvtxRange nvtx_range("zero_tensors_adamw_async");
    int32_t rc = check_grads(tensors, n_tensors);
    if (rc == ZS_OK) rc = check_states(tensors, n_tensors);
    if (rc != ZS_OK) return rc;
    if (!zs::valid_hp(hp) || !finite_double(max_norm) || ctrl_dev == nullptr || (max_norm > 0.0 && sqnorm_dev == nullptr))
        return ZS_ERR_ARG;
    if (!zs::aligned_to(ctrl_dev, 8) || !zs::aligned_to(sqnorm_dev, 8)) return ZS_ERR_ALIGN;
    bool has[2] = {false, false};
    for (int32_t i = 0; i < n_tensors; ++i)
        if (tensors[i].n > 0) has[tensors[i].state] = true;
    const StepShared shared{*hp, max_norm, sqnorm_dev, ctrl_dev, 0, 0, 1.0f};
    cudaStream_t st = (cudaStream_t)stream;
    const bool few = n_tensors <= kFewTensors;
    if (has[ZS_STATE_U8]) {
        const auto launch = few ? launch_steps8<kFewTensors> : launch_steps8<kStepGroup8>;
        rc = launch(shared, tensors, n_tensors, !has[ZS_STATE_F32], st);
        if (rc != ZS_OK) return rc;
    }
    if (has[ZS_STATE_F32]) {
        const auto launch = few ? launch_steps32<kFewTensors> : launch_steps32<kStepGroup32>;
        return launch(shared, tensors, n_tensors, true, st);
    }
    if (has[ZS_STATE_U8]) return ZS_OK;
    // nothing to update: the step still ends in the control block
    zs_shard none;
    std::memset(&none, 0, sizeof(none));
    return zs::launch_commit(&none, 1, *hp, ctrl_dev, st);
}

ZS_API int32_t zero_adam8_dequantize(const uint8_t* codes_dev, const float* scales_dev, int64_t n,
                                     int32_t is_signed, float* out_dev, void* stream) {
    zs::NvtxRange nvtx_range("zero_adam8_dequantize");
    if (n < 0 || (is_signed != 0 && is_signed != 1)) return ZS_ERR_ARG;
    if (n == 0) return ZS_OK;
    if (codes_dev == nullptr || scales_dev == nullptr || out_dev == nullptr) return ZS_ERR_ARG;
    if (!zs::aligned_to(scales_dev, 4) || !zs::aligned_to(out_dev, 4)) return ZS_ERR_ALIGN;
    ValueArgs a;
    a.codes = codes_dev;
    a.scales = scales_dev;
    a.out = out_dev;
    a.n = n;
    a.wide = zs::aligned_to(codes_dev, 4) && zs::aligned_to(out_dev, 16);
    const Maps& maps = host_maps().maps;
    std::memcpy(a.map, is_signed ? maps.dec7 : maps.mag8, sizeof(a.map));
    const int blocks = zs::persistent_blocks((const void*)adam8_values_kernel, kValueThreads, a.wide ? n / 16 + 1 : n);
    return launch_ex(adam8_values_kernel, blocks, kValueThreads, 0, true, (cudaStream_t)stream, a, "adam8_values_kernel");
}

}  // extern "C"
