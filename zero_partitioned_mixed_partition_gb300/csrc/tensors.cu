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

#include "zs_internal.h"

namespace {

#include "step_common.cuh"
#include "step_end.cuh"
#include "loss_common.cuh"
#include "adam8_math.cuh"

// index-check sites of this file
[[maybe_unused]] constexpr uint32_t kSiteTensor = 14, kSiteTensorScale = 15, kSiteTensorNorm = 16;

constexpr int kChunk = ZS_ADAM8_BLOCK;  // elements of a chunk: one block of 8-bit states
constexpr int kThreads = 256;           // 8 elements each
static_assert(kChunk == kThreads * 8, "a thread takes 8 elements of a chunk");

// ------------------------------------------------------------------ layout ---

// Which elements of a chunk a thread takes, by the tensor's `peel`:
//   peel in [0, 8)  every buffer of the tensor is on a 16-byte boundary (8 for
//                   codes) at element peel, and so at peel + 8 i: thread t < 255
//                   takes the eight from peel + 8 t, as vectors; thread 255 takes
//                   the chunk's edges, [0, peel) and [2040 + peel, 2048)
//   kScattered      no such element: thread t takes t + 256 j, one at a time
constexpr int kScattered = 8;

__device__ __forceinline__ int chunk_element(int peel, int j) {
    const int t = threadIdx.x;
    if (peel == kScattered) return t + kThreads * j;
    if (t < kThreads - 1) return peel + 8 * t + j;
    return j < peel ? j : kChunk - 8 + j;
}
__device__ __forceinline__ bool chunk_vector(int peel, int rem) {
    if (peel == kScattered) return false;
    if (threadIdx.x < kThreads - 1) return peel + 8 * (int)threadIdx.x + 8 <= rem;
    return peel == 0 && rem == kChunk;
}

// ------------------------------------------------------------- element access ---

__device__ __forceinline__ float load_one(const void* p, int type, int64_t e) {
    if (type == ZS_F32) return __ldcs((const float*)p + e);
    const unsigned short h = __ldcs((const unsigned short*)p + e);
    return type == ZS_F16 ? __half2float(__ushort_as_half(h)) : __bfloat162float(__ushort_as_bfloat16(h));
}
__device__ __forceinline__ void load_grad8(const void* p, int type, int64_t e, float* g) {
    if (type == ZS_F32) {
        Mem<8>::load_f((const float*)p + e, g);
    } else if (type == ZS_F16) {
        Mem<8>::load_h((const uint16_t*)p + e, g);
    } else {
        uint32_t w[4];
        Mem<8>::load_h_words((const uint16_t*)p + e, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // bf16 is the upper half of an fp32
            g[2 * i] = __uint_as_float(w[i] << 16);
            g[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
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
    int32_t type, peel;
};
constexpr int kNormGroup = 1024;

struct NormArgs {
    NormEntry t[kNormGroup];
    uint32_t first[kNormGroup + 1];  // first chunk of each tensor in the launch
    int32_t count;
    int32_t base;      // where this launch's partial sums start
    int32_t finish;    // the call's last launch adds up all of them
    zs_ctrl* ctrl;
    double* out;
    Work* work;
};
static_assert(sizeof(NormArgs) <= 32764, "kernel parameters");

// The tensor of chunk q: the last one whose first chunk is not above q.
__device__ __forceinline__ int tensor_of(const uint32_t* first, int count, uint32_t q) {
    int lo = 0, hi = count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= q) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) tensors_sqnorm_kernel(const __grid_constant__ NormArgs p) {
    __shared__ double s_part[kThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    const float inv = __double2float_rn(__ddiv_rn(1.0, p.ctrl->loss_scale));
    double sum = 0.0;
    bool bad = false;
    const uint32_t total = p.first[p.count];
    for (uint32_t q = blockIdx.x; q < total; q += gridDim.x) {
        const NormEntry& t = p.t[tensor_of(p.first, p.count, q)];
        const int64_t at = (int64_t)(q - p.first[&t - p.t]) * kChunk;
        const int rem = (int)(t.n - at < kChunk ? t.n - at : kChunk);
        float g[8];
        if (chunk_vector(t.peel, rem) && ZS_RANGE_OK(kSiteTensorNorm, at + chunk_element(t.peel, 0), 8, t.n)) {
            load_grad8(t.grad, t.type, at + chunk_element(t.peel, 0), g);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = chunk_element(t.peel, j);
                g[j] = e < rem && ZS_RANGE_OK(kSiteTensorNorm, at + e, 1, t.n) ? load_one(t.grad, t.type, at + e) : 0.0f;
            }
        }
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = __fmul_rn(g[j], inv);
            bad |= !(fabsf(x) < 0x1p62f);  // also a NaN
            part = __fmaf_rn(x, x, part);
        }
        sum += (double)part;
    }
    if (__syncthreads_or(bad) && threadIdx.x == 0) atomicOr(&p.ctrl->overflow, 1);
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double b = 0.0;
        for (int w = 0; w < kThreads / 32; ++w) b += s_part[w];
        p.work->part[p.base + blockIdx.x] = b;
    }
    if (!p.finish || !last_to_arrive(p.work, gridDim.x)) return;
    sum = 0.0;
    const int parts = p.base + (int)gridDim.x;
    for (int i = threadIdx.x; i < parts; i += kThreads) sum += *(volatile double*)&p.work->part[i];
    sum = warp_sum(sum);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double b = 0.0;
        for (int w = 0; w < kThreads / 32; ++w) b += s_part[w];
        *p.out = b;
    }
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
};
template <typename Entry, int G>
struct StepArgs : StepShared {
    Entry t[G];
    uint32_t first[G + 1];
};
struct StepArgs8 : StepArgs<StepEntry8, 240> {
    Maps maps;
};
using StepArgs32 = StepArgs<StepEntry, 448>;
static_assert(sizeof(StepArgs32) <= 32764 && sizeof(StepArgs8) <= 32764, "kernel parameters");

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

__global__ void __launch_bounds__(kThreads) tensors_adamw_kernel(const __grid_constant__ StepArgs32 p) {
    __shared__ StepCoef s_coef;
    griddep_wait();
    griddep_launch_dependents();
    if (threadIdx.x == 0) step_coef(p, &s_coef);
    __syncthreads();
    Coef c = s_coef.c;
    const float clip = s_coef.clip;
    const uint32_t total = s_coef.skip ? 0u : p.first[p.count];
    for (uint32_t q = blockIdx.x; q < total; q += gridDim.x) {
        const int i = tensor_of(p.first, p.count, q);
        const StepEntry& t = p.t[i];
        const int64_t at = (int64_t)(q - p.first[i]) * kChunk;
        const int rem = (int)(t.n - at < kChunk ? t.n - at : kChunk);
        c.lr = t.lr;
        c.wd = t.wd;
        if (chunk_vector(t.peel, rem) && ZS_RANGE_OK(kSiteTensor, at + chunk_element(t.peel, 0), 8, t.n)) {
            const int64_t e = at + chunk_element(t.peel, 0);
            float g[8], th[8], m[8], v[8];
            load_grad8(t.grad, t.grad_type, e, g);
            Mem<8>::load_f(t.master + e, th);
            Mem<8>::load_f(t.m + e, m);
            Mem<8>::load_f(t.v + e, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) adam_apply<false>(c, __fmul_rn(__fmul_rn(g[j], c.inv), clip), th[j], m[j], v[j]);
            Mem<8>::store_f(t.master + e, th);
            Mem<8>::store_f(t.m + e, m);
            Mem<8>::store_f(t.v + e, v);
            if (t.param != nullptr) store_param8(t.param, t.param_type, e, th);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = chunk_element(t.peel, j);
                const int64_t e = at + k;
                if (k >= rem || !ZS_RANGE_OK(kSiteTensor, e, 1, t.n)) continue;
                float th = __ldcs(t.master + e), m = __ldcs(t.m + e), v = __ldcs(t.v + e);
                const float g = load_one(t.grad, t.grad_type, e);
                adam_apply<false>(c, __fmul_rn(__fmul_rn(g, c.inv), clip), th, m, v);
                __stcs(t.master + e, th);
                __stcs(t.m + e, m);
                __stcs(t.v + e, v);
                if (t.param != nullptr) store_one16(t.param, t.param_type, e, th);
            }
        }
    }
    if (p.finish && threadIdx.x == 0) arrive_and_finish(p.ctrl, gridDim.x, p.hp.beta1, p.hp.beta2);
}

// Sum-free block maximum of two non-negative floats by their bit patterns.
__device__ __forceinline__ void block_max2(float& a, float& b, uint32_t (&slots)[2][kThreads / 32]) {
    const uint32_t wa = __reduce_max_sync(0xffffffffu, __float_as_uint(a));
    const uint32_t wb = __reduce_max_sync(0xffffffffu, __float_as_uint(b));
    __syncthreads();  // the last chunk's maxima have been read
    if ((threadIdx.x & 31) == 0) {
        slots[0][threadIdx.x >> 5] = wa;
        slots[1][threadIdx.x >> 5] = wb;
    }
    __syncthreads();
    uint32_t ma = 0u, mb = 0u;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        ma = max(ma, slots[0][w]);
        mb = max(mb, slots[1][w]);
    }
    a = __uint_as_float(ma);
    b = __uint_as_float(mb);
}

__global__ void __launch_bounds__(kThreads) tensors_adamw8_kernel(const __grid_constant__ StepArgs8 p) {
    __shared__ StepCoef s_coef;
    __shared__ Maps s_maps;
    __shared__ uint32_t s_max[2][kThreads / 32];
    {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(&p.maps);
        uint32_t* dst = reinterpret_cast<uint32_t*>(&s_maps);
        for (int i = threadIdx.x; i < (int)(sizeof(Maps) / 4); i += kThreads) dst[i] = src[i];
    }
    griddep_wait();
    griddep_launch_dependents();
    if (threadIdx.x == 0) step_coef(p, &s_coef);
    __syncthreads();
    Coef c = s_coef.c;
    const float clip = s_coef.clip;
    const uint32_t total = s_coef.skip ? 0u : p.first[p.count];
    for (uint32_t q = blockIdx.x; q < total; q += gridDim.x) {
        const int i = tensor_of(p.first, p.count, q);
        const StepEntry8& t = p.t[i];
        const int64_t block = q - p.first[i], at = block * kChunk;
        const int rem = (int)(t.n - at < kChunk ? t.n - at : kChunk);
        c.lr = t.lr;
        c.wd = t.wd;
        const bool scale_ok = ZS_RANGE_OK(kSiteTensorScale, block, 1, (t.n + kChunk - 1) / kChunk);
        const float ms = scale_ok ? t.m_scale[block] : 0.0f, vs = scale_ok ? t.v_scale[block] : 0.0f;
        float m[8], v[8], am = 0.0f, av = 0.0f;
        const bool wide = chunk_vector(t.peel, rem) && ZS_RANGE_OK(kSiteTensor, at + chunk_element(t.peel, 0), 8, t.n);
        if (wide) {
            const int64_t e = at + chunk_element(t.peel, 0);
            float g[8], th[8];
            load_grad8(t.grad, t.grad_type, e, g);
            Mem<8>::load_f(t.master + e, th);
            const uint2 cm = __ldcs(reinterpret_cast<const uint2*>(t.m_codes() + e));
            const uint2 cv = __ldcs(reinterpret_cast<const uint2*>(t.v_codes() + e));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                m[j] = __fmul_rn(s_maps.dec7[__byte_perm(j < 4 ? cm.x : cm.y, 0u, 0x4440u + (j & 3))], ms);
                v[j] = __fmul_rn(s_maps.mag8[__byte_perm(j < 4 ? cv.x : cv.y, 0u, 0x4440u + (j & 3))], vs);
                adam_apply<false>(c, __fmul_rn(__fmul_rn(g[j], c.inv), clip), th[j], m[j], v[j]);
            }
            Mem<8>::store_f(t.master + e, th);
            if (t.param != nullptr) store_param8(t.param, t.param_type, e, th);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = chunk_element(t.peel, j);
                const int64_t e = at + k;
                m[j] = v[j] = 0.0f;  // changes no block maximum
                if (k >= rem || !ZS_RANGE_OK(kSiteTensor, e, 1, t.n)) continue;
                m[j] = __fmul_rn(s_maps.dec7[t.m_codes()[e]], ms);
                v[j] = __fmul_rn(s_maps.mag8[t.v_codes()[e]], vs);
                float th = __ldcs(t.master + e);
                const float g = load_one(t.grad, t.grad_type, e);
                adam_apply<false>(c, __fmul_rn(__fmul_rn(g, c.inv), clip), th, m[j], v[j]);
                __stcs(t.master + e, th);
                if (t.param != nullptr) store_one16(t.param, t.param_type, e, th);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            am = fmaxf(am, fabsf(m[j]));
            av = fmaxf(av, v[j]);
        }
        block_max2(am, av, s_max);
        uint32_t cm[8], cv[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float xm = am > 0.0f ? __fdiv_rn(m[j], am) : 0.0f, xv = av > 0.0f ? __fdiv_rn(v[j], av) : 0.0f;
            const uint32_t k = nearest_code(fabsf(xm), s_maps.thr7, s_maps.bucket7);
            cm[j] = xm < 0.0f && k > 0u ? k | 0x80u : k;
            cv[j] = nearest_code(xv, s_maps.thr8, s_maps.bucket8);
        }
        if (wide) {
            const int64_t e = at + chunk_element(t.peel, 0);
            auto four = [](const uint32_t* x) { return x[0] | x[1] << 8 | x[2] << 16 | x[3] << 24; };
            __stcs(reinterpret_cast<uint2*>(t.m_codes() + e), make_uint2(four(cm), four(cm + 4)));
            __stcs(reinterpret_cast<uint2*>(t.v_codes() + e), make_uint2(four(cv), four(cv + 4)));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = chunk_element(t.peel, j);
                if (k >= rem || !ZS_RANGE_OK(kSiteTensor, at + k, 1, t.n)) continue;
                t.m_codes()[at + k] = (uint8_t)cm[j];
                t.v_codes()[at + k] = (uint8_t)cv[j];
            }
        }
        if (threadIdx.x == 0 && scale_ok) {
            t.m_scale[block] = am;
            t.v_scale[block] = av;
        }
    }
    if (p.finish && threadIdx.x == 0) arrive_and_finish(p.ctrl, gridDim.x, p.hp.beta1, p.hp.beta2);
}

// ------------------------------------------------------------- 8-bit values ---

struct ValueArgs {
    const uint8_t* codes;
    const float* scales;
    float* out;
    int64_t n;
    int32_t wide;        // codes on 8-byte, out on 16-byte boundaries
    float map[256];
};

__global__ void __launch_bounds__(kThreads) adam8_values_kernel(const __grid_constant__ ValueArgs p) {
    __shared__ float s_map[256];
    s_map[threadIdx.x] = p.map[threadIdx.x];
    griddep_wait();
    griddep_launch_dependents();
    __syncthreads();
    const int64_t stride = (int64_t)gridDim.x * kThreads, first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t nvec = p.wide ? p.n / 8 : 0;
    for (int64_t i = first; i < nvec; i += stride) {
        const uint2 c = __ldcs(reinterpret_cast<const uint2*>(p.codes + 8 * i));
        const float s = __ldg(p.scales + 8 * i / ZS_ADAM8_BLOCK);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = __fmul_rn(s_map[__byte_perm(j < 4 ? c.x : c.y, 0u, 0x4440u + (j & 3))], s);
        Mem<8>::store_f(p.out + 8 * i, x);
    }
    for (int64_t i = nvec * 8 + first; i < p.n; i += stride)
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
        chunks += (t[i].n + kChunk - 1) / kChunk;
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

int launch_blocks(const void* kernel, uint32_t chunks) {
    return zs::persistent_blocks(kernel, kThreads, (int64_t)(chunks > 0 ? chunks : 1) * kThreads);
}

// The partial sums of one norm call share the scratch buffer: this many each.
int norm_blocks(uint32_t chunks, int launches_left, int base) {
    const int fit = (kWorkParts - base) / launches_left;
    const int blocks = launch_blocks((const void*)tensors_sqnorm_kernel, chunks);
    return blocks < fit ? blocks : fit;
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
int32_t launch_steps(void (*kernel)(Args), Args& a, int32_t state, const zs_tensor* t, int32_t n, const zs_adam& hp,
                     bool finish, cudaStream_t stream, const char* name) {
    constexpr int G = (int)(sizeof(a.t) / sizeof(a.t[0]));
    int32_t left = 0;
    for (int32_t i = 0; i < n; ++i) left += t[i].state == state && t[i].n > 0;
    a.count = 0;
    a.first[0] = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (t[i].state != state || t[i].n == 0) continue;
        fill(&a.t[a.count], t[i], hp);
        a.first[a.count + 1] = a.first[a.count] + (uint32_t)((t[i].n + kChunk - 1) / kChunk);
        ++a.count;
        --left;
        if (a.count < G && left > 0) continue;
        a.finish = finish && left == 0;
        const int32_t rc = launch_ex(kernel, launch_blocks((const void*)kernel, a.first[a.count]), kThreads, 0, true,
                                     stream, a, name);
        if (rc != ZS_OK) return rc;
        a.count = 0;
    }
    return ZS_OK;
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
    NormArgs a;
    a.ctrl = ctrl_dev;
    a.out = sqnorm_dev;
    a.work = (Work*)work_dev;
    a.base = 0;
    int launches = (n_tensors + kNormGroup - 1) / kNormGroup;
    for (int32_t i = 0; i < n_tensors; --launches) {
        a.first[0] = 0;
        for (a.count = 0; a.count < kNormGroup && i < n_tensors; ++i) {
            const zs_tensor& x = tensors[i];
            a.t[a.count] = NormEntry{x.grad, x.n, x.grad_type, common_peel({{x.grad, type_size(x.grad_type)}})};
            a.first[a.count + 1] = a.first[a.count] + (uint32_t)((x.n + kChunk - 1) / kChunk);
            ++a.count;
        }
        a.finish = i == n_tensors;
        const int blocks = norm_blocks(a.first[a.count], launches, a.base);
        const int32_t lrc = launch_ex(tensors_sqnorm_kernel, blocks, kThreads, 0, true, (cudaStream_t)stream, a,
                                      "tensors_sqnorm_kernel");
        if (lrc != ZS_OK) return lrc;
        a.base += blocks;
    }
    return ZS_OK;
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
    const StepShared shared{*hp, max_norm, sqnorm_dev, ctrl_dev, 0, 0};
    cudaStream_t st = (cudaStream_t)stream;
    if (has[ZS_STATE_U8]) {
        static_assert(sizeof(StepArgs8) < 64 * 1024, "on the stack");
        StepArgs8 a;
        static_cast<StepShared&>(a) = shared;
        a.maps = host_maps().maps;
        if (!host_maps().ok) return zs::fail_with(ZS_ERR_CUDA, "zero_tensors_adamw_async: code tables");
        rc = launch_steps(tensors_adamw8_kernel, a, ZS_STATE_U8, tensors, n_tensors, *hp, !has[ZS_STATE_F32], st,
                          "tensors_adamw8_kernel");
        if (rc != ZS_OK) return rc;
    }
    if (has[ZS_STATE_F32]) {
        StepArgs32 a;
        static_cast<StepShared&>(a) = shared;
        return launch_steps(tensors_adamw_kernel, a, ZS_STATE_F32, tensors, n_tensors, *hp, true, st,
                            "tensors_adamw_kernel");
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
    a.wide = zs::aligned_to(codes_dev, 8) && zs::aligned_to(out_dev, 16);
    const Maps& maps = host_maps().maps;
    std::memcpy(a.map, is_signed ? maps.dec7 : maps.mag8, sizeof(a.map));
    const int blocks = zs::persistent_blocks((const void*)adam8_values_kernel, kThreads, a.wide ? n / 8 + 1 : n);
    return launch_ex(adam8_values_kernel, blocks, kThreads, 0, true, (cudaStream_t)stream, a, "adam8_values_kernel");
}

}  // extern "C"
