// logits.cu -- token log-probabilities of a language model's logits, their
// gradient, and the clipped policy loss with its gradient.
//
// Per row of V logits, in fp32: top = max x, d_i = (x_i - top) it, S = sum
// exp(d_i), logp = d_y - ln S, H = ln S - sum exp(d_i) d_i / S, and for
// coefficients a (of logp) and b (of H)
//   dx_i = L it [ a (1[i=y] - p_i) - b p_i (ln p_i + H) ],  p_i = exp(d_i - ln S).
// Both losses of a row depend on the rest of the batch only through given
// weights, so the policy loss's gradient is formed while the row is at hand:
// the logits come from memory once and the gradient goes there once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <cfloat>

#include "zs_internal.h"

namespace {

#include "step_common.cuh"
#include "step_end.cuh"
#include "loss_common.cuh"

[[maybe_unused]] constexpr uint32_t kSiteLogits = 12, kSiteDlogits = 13;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// ------------------------------------------------------------ element types ---

template <typename T> __device__ __forceinline__ float to_float(T x);
template <> __device__ __forceinline__ float to_float<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Elements of one 16-byte vector.
template <typename T> constexpr int vec_of() { return 16 / (int)sizeof(T); }

template <typename T>
__device__ __forceinline__ void unpack(const uint4& r, float* x) {
    union { uint4 v; T e[vec_of<T>()]; } u;
    u.v = r;
#pragma unroll
    for (int j = 0; j < vec_of<T>(); ++j) x[j] = to_float<T>(u.e[j]);
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float* x) {
    union { uint4 v; T e[vec_of<T>()]; } u;
#pragma unroll
    for (int j = 0; j < vec_of<T>(); ++j) u.e[j] = from_float<T>(x[j]);
    return u.v;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------ row statistics ---

// Running statistics of a part of a row, in units of log2: top = the largest
// logit so far, s = sum 2^a, u = sum 2^a a with a = (x - top) k, k = it log2 e.
// top starts at the lowest finite float, so that a row of nothing but -inf
// keeps s = 0 and no difference of infinities is formed.
struct Stats {
    float top, s, u;
};

template <bool ENT>
__device__ __forceinline__ void shift_to(Stats& st, float top, float k) {
    // a <- a + (old top - new top) k; the bound keeps -inf * 0 out of u
    const float sh = fmaxf((st.top - top) * k, -1e30f);
    const float f = exp2_approx(sh);
    if (ENT) st.u = f * (st.u + sh * st.s);
    st.s *= f;
    st.top = top;
}

template <bool ENT, int N>
__device__ __forceinline__ void add_values(Stats& st, const float* x, float k) {
    float top = x[0];
#pragma unroll
    for (int j = 1; j < N; ++j) top = fmaxf(top, x[j]);
    if (top > st.top) shift_to<ENT>(st, top, k);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float a = (x[j] - st.top) * k;
        const float e = exp2_approx(a);
        st.s += e;
        // e = 0 where a is below -126: the bound keeps 0 * -inf out of u
        if (ENT) st.u = fmaf(e, fmaxf(a, -1e4f), st.u);
    }
}

template <bool ENT>
__device__ __forceinline__ void join(Stats& a, Stats b, float k) {
    const float top = fmaxf(a.top, b.top);
    shift_to<ENT>(a, top, k);
    shift_to<ENT>(b, top, k);
    a.s += b.s;
    if (ENT) a.u += b.u;
}

constexpr int kRowThreads = 512;

// Statistics of a whole row by one block, valid in every thread.
template <typename T, bool ENT>
__device__ __forceinline__ Stats row_stats(const T* row, int64_t vocab, float k) {
    constexpr int N = vec_of<T>();
    __shared__ Stats s_part[kRowThreads / 32];
    Stats st{-FLT_MAX, 0.0f, 0.0f};
    int64_t head = (int64_t)(((16u - ((uintptr_t)row & 15u)) & 15u) / sizeof(T));
    if (head > vocab) head = vocab;
    const int64_t nvec = (vocab - head) / N, tail = head + nvec * N;
    if (threadIdx.x < head) {
        const float x = to_float<T>(row[threadIdx.x]);
        add_values<ENT, 1>(st, &x, k);
    }
    if (tail + threadIdx.x < vocab) {
        const float x = to_float<T>(row[tail + threadIdx.x]);
        add_values<ENT, 1>(st, &x, k);
    }
    const uint4* vec = reinterpret_cast<const uint4*>(row + head);
    int64_t i = threadIdx.x;
    for (; i + 3 * kRowThreads < nvec; i += 4 * kRowThreads) {
        uint4 r[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) r[q] = vec[i + q * kRowThreads];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float x[N];
            unpack<T>(r[q], x);
            add_values<ENT, N>(st, x, k);
        }
    }
    for (; i < nvec; i += kRowThreads) {
        float x[N];
        unpack<T>(vec[i], x);
        add_values<ENT, N>(st, x, k);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Stats b;
        b.top = __shfl_xor_sync(0xffffffffu, st.top, o);
        b.s = __shfl_xor_sync(0xffffffffu, st.s, o);
        b.u = ENT ? __shfl_xor_sync(0xffffffffu, st.u, o) : 0.0f;
        join<ENT>(st, b, k);
    }
    __syncthreads();  // the last row's partial statistics have been read
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = st;
    __syncthreads();
    st = s_part[0];
#pragma unroll
    for (int w = 1; w < kRowThreads / 32; ++w) join<ENT>(st, s_part[w], k);
    return st;
}

// ---------------------------------------------------------------- gradient ---

// Coefficients of a row's gradient: dx_i = p_i (c0 + c1 q_i) + cy [i = y],
// q_i = log2 p_i = (x_i - top) k - l2.
struct GradCoef {
    float top, l2, c0, c1, cy;
};

template <typename T, bool ENT, int N>
__device__ __forceinline__ void grad_values(const GradCoef& c, float k, float* x) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float q = fmaf(x[j] - c.top, k, -c.l2);
        const float p = exp2_approx(q);
        // p = 0 where q is below -126: the bound keeps 0 * -inf out
        x[j] = ENT ? p * fmaf(c.c1, fmaxf(q, -1e4f), c.c0) : p * c.c0;
    }
}

template <typename T, bool ENT>
__device__ __forceinline__ void grad_row(const T* row, T* out, int64_t vocab, int64_t label, float k, const GradCoef& c) {
    constexpr int N = vec_of<T>();
    int64_t head = (int64_t)(((16u - ((uintptr_t)row & 15u)) & 15u) / sizeof(T));
    if (head > vocab) head = vocab;
    const int64_t nvec = (vocab - head) / N, tail = head + nvec * N;
    const bool wide = ((uintptr_t)(out + head) & 15u) == 0;
    auto one = [&](int64_t i) {
        float x = to_float<T>(row[i]);
        grad_values<T, ENT, 1>(c, k, &x);
        if (i == label) x += c.cy;
        out[i] = from_float<T>(x);
    };
    if (threadIdx.x < head) one(threadIdx.x);
    if (tail + threadIdx.x < vocab) one(tail + threadIdx.x);
    for (int64_t i = threadIdx.x; i < nvec; i += kRowThreads) {
        const int64_t e = head + i * N;
        float x[N];
        unpack<T>(*reinterpret_cast<const uint4*>(row + e), x);
        grad_values<T, ENT, N>(c, k, x);
        if (label >= e && label < e + N) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (label == e + j) x[j] += c.cy;
        }
        if (wide) {
            *reinterpret_cast<uint4*>(out + e) = pack<T>(x);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) out[e + j] = from_float<T>(x[j]);
        }
    }
}

template <typename T>
__device__ __forceinline__ void zero_row(T* out, int64_t vocab) {
    constexpr int N = vec_of<T>();
    int64_t head = (int64_t)(((16u - ((uintptr_t)out & 15u)) & 15u) / sizeof(T));
    if (head > vocab) head = vocab;
    const int64_t nvec = (vocab - head) / N, tail = head + nvec * N;
    if (threadIdx.x < head) out[threadIdx.x] = from_float<T>(0.0f);
    if (tail + threadIdx.x < vocab) out[tail + threadIdx.x] = from_float<T>(0.0f);
    for (int64_t i = threadIdx.x; i < nvec; i += kRowThreads)
        *reinterpret_cast<uint4*>(out + head + i * N) = make_uint4(0u, 0u, 0u, 0u);
}

// ----------------------------------------------------------------- kernels ---

struct LogpArgs {
    const void* data;
    int64_t rows, vocab, stride;
    float it;
    const int64_t* labels;
    float *logp, *entropy, *saved;
};

template <typename T, bool ENT>
__global__ void __launch_bounds__(kRowThreads) token_logp_kernel(const __grid_constant__ LogpArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    const float k = p.it * kLog2e;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const int64_t y = p.labels[r];
        const T* row = (const T*)p.data + r * p.stride;
        float logp = 0.0f, ent = 0.0f, top = 0.0f, lns = 0.0f;
        if (y >= 0 && y < p.vocab) {
            const Stats st = row_stats<T, ENT>(row, p.vocab, k);
            if (st.s == 0.0f) {
                logp = top = lns = -INFINITY;
            } else {
                top = st.top;
                lns = logf(st.s);
                logp = (to_float<T>(row[y]) - top) * p.it - lns;
                if (ENT) ent = lns - st.u / st.s * kLn2;
            }
        }
        if (threadIdx.x == 0) {
            p.logp[r] = logp;
            if (ENT && p.entropy != nullptr) p.entropy[r] = ent;
            if (p.saved != nullptr) {
                p.saved[2 * r] = top;
                p.saved[2 * r + 1] = lns;
            }
        }
    }
}

struct GradArgs {
    const void* data;
    void* out;
    int64_t rows, vocab, stride, out_stride;
    float it;
    const int64_t* labels;
    const float *saved, *dlogp, *entropy, *dentropy;
    const zs_ctrl* ctrl;
};

template <typename T, bool ENT>
__global__ void __launch_bounds__(kRowThreads) token_logp_grad_kernel(const __grid_constant__ GradArgs p) {
    griddep_wait();
    griddep_launch_dependents();
    const float k = p.it * kLog2e, scale = loss_scale_of(p.ctrl) * p.it;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const int64_t y = p.labels[r];
        const T* row = (const T*)p.data + r * p.stride;
        T* out = (T*)p.out + r * p.out_stride;
        const float top = p.saved[2 * r], lns = p.saved[2 * r + 1];
        if (y < 0 || y >= p.vocab || lns == -INFINITY) {
            zero_row<T>(out, p.vocab);
            continue;
        }
        const float a = scale * p.dlogp[r], b = ENT ? scale * p.dentropy[r] : 0.0f;
        const GradCoef c{top, lns * kLog2e, ENT ? -(a + b * p.entropy[r]) : -a, -b * kLn2, a};
        grad_row<T, ENT>(row, out, p.vocab, y, k, c);
    }
}

struct PolicyArgs {
    const void* data;
    void* out;
    int64_t rows, vocab, stride, out_stride;
    float it;
    const int64_t* labels;
    const float *old_logp, *adv, *ref_logp, *weights;
    float uniform_weight;       // the rows' weight without `weights`
    float lo, hi, dual, kl, ent_coef;
    const zs_ctrl* ctrl;
    float *logp, *entropy, *token_loss, *totals;
    Work* work;
};

template <typename T, bool ENT, bool GRAD>
__global__ void __launch_bounds__(kRowThreads) policy_loss_kernel(const __grid_constant__ PolicyArgs p) {
    __shared__ double s_sum[ZS_POLICY_TOTALS];
    griddep_wait();
    griddep_launch_dependents();
    const float k = p.it * kLog2e, scale = GRAD ? loss_scale_of(p.ctrl) * p.it : 0.0f;
    double sum[ZS_POLICY_TOTALS] = {};  // thread 0's
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const int64_t y = p.labels[r];
        const float w = p.weights != nullptr ? p.weights[r] : p.uniform_weight;
        const T* row = (const T*)p.data + r * p.stride;
        T* out = (T*)p.out + r * p.out_stride;
        float logp = 0.0f, ent = 0.0f, loss = 0.0f;
        bool live = y >= 0 && y < p.vocab && w != 0.0f;
        if (live) {
            const Stats st = row_stats<T, ENT>(row, p.vocab, k);
            if (st.s == 0.0f) {
                logp = -INFINITY;
                live = false;
            } else {
                const float lns = logf(st.s);
                logp = (to_float<T>(row[y]) - st.top) * p.it - lns;
                if (ENT) ent = lns - st.u / st.s * kLn2;
                const float adv = p.adv[r], ratio = expf(logp - p.old_logp[r]);
                const float held = fminf(fmaxf(ratio, p.lo), p.hi);
                const float free_pg = -adv * ratio, held_pg = -adv * held;
                bool cut = free_pg < held_pg;
                float pg = cut ? held_pg : free_pg;
                if (p.dual > 0.0f && adv < 0.0f && pg > -adv * p.dual) {
                    pg = -adv * p.dual;
                    cut = true;
                }
                if (ratio != ratio) pg = ratio;  // a NaN passes through
                float kl = 0.0f, dlogp = cut ? 0.0f : free_pg;
                if (p.ref_logp != nullptr) {
                    const float gap = p.ref_logp[r] - logp, rise = expm1f(gap);
                    kl = rise - gap;
                    dlogp -= p.kl * rise;
                }
                loss = pg + p.kl * kl;
                if (ENT) loss -= p.ent_coef * ent;
                if (threadIdx.x == 0) {
                    sum[0] += (double)w * loss;
                    sum[1] += (double)w * pg;
                    sum[2] += (double)w * kl;
                    sum[3] += (double)w * ent;
                    sum[4] += cut ? (double)w : 0.0;
                }
                if (GRAD) {
                    __syncthreads();  // out may be the logits: every thread has read its label's logit
                    const float a = scale * w * dlogp, b = ENT ? -scale * w * p.ent_coef : 0.0f;
                    const GradCoef c{st.top, lns * kLog2e, ENT ? -(a + b * ent) : -a, -b * kLn2, a};
                    grad_row<T, ENT>(row, out, p.vocab, y, k, c);
                }
            }
        }
        if (GRAD && !live) zero_row<T>(out, p.vocab);
        if (threadIdx.x == 0) {
            p.logp[r] = logp;
            if (ENT && p.entropy != nullptr) p.entropy[r] = ent;
            if (p.token_loss != nullptr) p.token_loss[r] = loss;
        }
    }
    // partial sums by block, then in block order by the last block to arrive
    if (threadIdx.x == 0)
        for (int i = 0; i < ZS_POLICY_TOTALS; ++i) p.work->part[blockIdx.x * ZS_POLICY_TOTALS + i] = sum[i];
    if (!last_to_arrive(p.work, gridDim.x)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < ZS_POLICY_TOTALS) {
        double t = 0.0;
        for (unsigned b = lane; b < gridDim.x; b += 32) t += *(volatile double*)&p.work->part[b * ZS_POLICY_TOTALS + warp];
        t = warp_sum(t);
        if (lane == 0) s_sum[warp] = t;
    }
    __syncthreads();
    if (threadIdx.x < ZS_POLICY_TOTALS) p.totals[threadIdx.x] = __double2float_rn(s_sum[threadIdx.x]);
}

// ------------------------------------------------------------------- checks ---

int32_t check_logits(const zs_logits* x) {
    if (x == nullptr || x->rows < 0 || x->vocab < 1 || x->vocab > (1ll << 30) || x->row_stride < x->vocab ||
        x->reserved != 0 || (x->type != ZS_F32 && x->type != ZS_F16 && x->type != ZS_BF16) ||
        !(x->inv_temperature > 0.0) || x->inv_temperature > 1e6 || x->inv_temperature < 1e-6)
        return ZS_ERR_ARG;
    if (x->rows > 0 && x->data == nullptr) return ZS_ERR_ARG;
    return zs::aligned_to(x->data, x->type == ZS_F32 ? 4 : 2) ? ZS_OK : ZS_ERR_ALIGN;
}

int32_t check_dlogits(const zs_logits* x, const void* dlogits, int64_t stride) {
    if (stride < x->vocab) return ZS_ERR_ARG;
    if (x->rows > 0 && dlogits == nullptr) return ZS_ERR_ARG;
    return zs::aligned_to(dlogits, x->type == ZS_F32 ? 4 : 2) ? ZS_OK : ZS_ERR_ALIGN;
}

bool all_aligned4(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!zs::aligned_to(p, 4)) return false;
    return true;
}

template <typename Args>
int32_t launch_rows(void (*kernel)(Args), int64_t rows, const Args& a, cudaStream_t stream, const char* name) {
    const int blocks = zs::persistent_blocks((const void*)kernel, kRowThreads, rows * kRowThreads);
    return launch_ex(kernel, blocks, kRowThreads, 0, true, stream, a, name);
}

// Calls go(T{}) with the element type of the logits.
template <typename F>
int32_t with_type(int32_t type, F go) {
    if (type == ZS_F32) return go(float{});
    if (type == ZS_F16) return go(__half{});
    return go(__nv_bfloat16{});
}

}  // namespace

namespace zs {
uint64_t take_fault_logits() { return take_fault(); }
}  // namespace zs

extern "C" {

ZS_API int32_t zero_token_logp_async(const zs_logits* x, const int64_t* labels, float* logp, float* entropy,
                                     float* saved, void* stream) {
    zs::NvtxRange nvtx_range("zero_token_logp_async");
    const int32_t rc = check_logits(x);
    if (rc != ZS_OK) return rc;
    if (x->rows == 0) return ZS_OK;
    if (labels == nullptr || logp == nullptr) return ZS_ERR_ARG;
    if (!zs::aligned_to(labels, 8) || !all_aligned4({logp, entropy, saved})) return ZS_ERR_ALIGN;
    const LogpArgs a{x->data, x->rows, x->vocab, x->row_stride, (float)x->inv_temperature, labels, logp, entropy, saved};
    return with_type(x->type, [&](auto t) {
        using T = decltype(t);
        return launch_rows(entropy != nullptr ? token_logp_kernel<T, true> : token_logp_kernel<T, false>, x->rows, a,
                           (cudaStream_t)stream, "token_logp_kernel");
    });
}

ZS_API int32_t zero_token_logp_grad_async(const zs_logits* x, const int64_t* labels, const float* saved,
                                          const float* dlogp, const float* entropy, const float* dentropy,
                                          const zs_ctrl* ctrl_dev, void* dlogits, int64_t dlogits_stride,
                                          void* stream) {
    zs::NvtxRange nvtx_range("zero_token_logp_grad_async");
    int32_t rc = check_logits(x);
    if (rc != ZS_OK) return rc;
    rc = check_dlogits(x, dlogits, dlogits_stride);
    if (rc != ZS_OK) return rc;
    if (x->rows == 0) return ZS_OK;
    if (labels == nullptr || saved == nullptr || dlogp == nullptr || (entropy == nullptr) != (dentropy == nullptr))
        return ZS_ERR_ARG;
    if (!zs::aligned_to(labels, 8) || !zs::aligned_to(ctrl_dev, 8) ||
        !all_aligned4({saved, dlogp, entropy, dentropy}))
        return ZS_ERR_ALIGN;
    const GradArgs a{x->data, dlogits, x->rows, x->vocab, x->row_stride, dlogits_stride, (float)x->inv_temperature,
                     labels, saved, dlogp, entropy, dentropy, ctrl_dev};
    return with_type(x->type, [&](auto t) {
        using T = decltype(t);
        return launch_rows(dentropy != nullptr ? token_logp_grad_kernel<T, true> : token_logp_grad_kernel<T, false>,
                           x->rows, a, (cudaStream_t)stream, "token_logp_grad_kernel");
    });
}

ZS_API int32_t zero_policy_loss_async(const zs_logits* x, const int64_t* labels, const float* old_logp,
                                      const float* advantages, const float* ref_logp, const float* weights,
                                      const zs_policy* hp, const zs_ctrl* ctrl_dev, float* logp, float* entropy,
                                      float* token_loss, void* dlogits, int64_t dlogits_stride, float* totals,
                                      void* work_dev, void* stream) {
    zs::NvtxRange nvtx_range("zero_policy_loss_async");
    int32_t rc = check_logits(x);
    if (rc != ZS_OK) return rc;
    if (hp == nullptr || !(hp->clip_low >= 0.0 && hp->clip_low <= 1.0) || !(hp->clip_high >= 0.0) ||
        !finite_double(hp->clip_high) || !finite_double(hp->kl_coef) || !finite_double(hp->entropy_coef) ||
        !(hp->dual_clip == 0.0 || (hp->dual_clip > 1.0 && finite_double(hp->dual_clip))))
        return ZS_ERR_ARG;
    if (totals == nullptr || work_dev == nullptr) return ZS_ERR_ARG;
    if (x->rows > 0 && (labels == nullptr || old_logp == nullptr || advantages == nullptr || logp == nullptr))
        return ZS_ERR_ARG;
    if (dlogits != nullptr) {
        rc = check_dlogits(x, dlogits, dlogits_stride);
        if (rc != ZS_OK) return rc;
    }
    if (!zs::aligned_to(labels, 8) || !zs::aligned_to(ctrl_dev, 8) || !zs::aligned_to(work_dev, 8) ||
        !all_aligned4({old_logp, advantages, ref_logp, weights, logp, entropy, token_loss, totals}))
        return ZS_ERR_ALIGN;
    PolicyArgs a;
    a.data = x->data;
    a.out = dlogits;
    a.rows = x->rows;
    a.vocab = x->vocab;
    a.stride = x->row_stride;
    a.out_stride = dlogits_stride;
    a.it = (float)x->inv_temperature;
    a.labels = labels;
    a.old_logp = old_logp;
    a.adv = advantages;
    a.ref_logp = ref_logp;
    a.weights = weights;
    a.uniform_weight = x->rows > 0 ? (float)(1.0 / (double)x->rows) : 0.0f;
    a.lo = (float)(1.0 - hp->clip_low);
    a.hi = (float)(1.0 + hp->clip_high);
    a.dual = (float)hp->dual_clip;
    a.kl = (float)hp->kl_coef;
    a.ent_coef = (float)hp->entropy_coef;
    a.ctrl = ctrl_dev;
    a.logp = logp;
    a.entropy = entropy;
    a.token_loss = token_loss;
    a.totals = totals;
    a.work = (Work*)work_dev;
    const bool ent = entropy != nullptr || hp->entropy_coef != 0.0, grad = dlogits != nullptr;
    return with_type(x->type, [&](auto t) {
        using T = decltype(t);
        auto kernel = ent ? (grad ? policy_loss_kernel<T, true, true> : policy_loss_kernel<T, true, false>)
                          : (grad ? policy_loss_kernel<T, false, true> : policy_loss_kernel<T, false, false>);
        return launch_rows(kernel, x->rows, a, (cudaStream_t)stream, "policy_loss_kernel");
    });
}

}  // extern "C"
