// preference.cu -- the paired preference loss over packed token
// log-probabilities, with its gradient.
//
// Per pair: the two sequences' sums (or means) of logp - ref over unmasked
// tokens, one scalar loss of their difference, and a gradient that is the same
// number for every unmasked token of a sequence.  So a pair is read once for
// its sums and its gradient is written without reading the values again.
#include <stdint.h>

#include <cuda_fp16.h>

#include "zs_internal.h"

namespace {

#include "step_common.cuh"
#include "step_end.cuh"
#include "loss_common.cuh"

constexpr int kPairThreads = 256;

struct PairArgs {
    const float *logp, *ref;
    const uint8_t* mask;
    int64_t n;
    const int64_t* cu;
    const float* weights;
    float uniform_weight;
    int32_t n_pairs, kind, average;
    float beta, smooth, margin, target;  // target = 1 / (2 beta)
    float *loss, *reward, *dlogp, *totals;
    Work* work;
};

// Sum over the block, valid in every thread; the order is fixed.
__device__ __forceinline__ double block_total(double x, double* slots) {
    x = warp_sum(x);
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = x;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kPairThreads / 32; ++w) t += slots[w];
    __syncthreads();
    return t;
}

__device__ __forceinline__ float softplus(float z) { return fmaxf(z, 0.0f) + log1pf(expf(-fabsf(z))); }

__global__ void __launch_bounds__(kPairThreads) preference_loss_kernel(const __grid_constant__ PairArgs p) {
    __shared__ double s_slots[kPairThreads / 32];
    __shared__ double s_sum[ZS_PREFERENCE_TOTALS];
    griddep_wait();
    griddep_launch_dependents();
    double sum[ZS_PREFERENCE_TOTALS] = {};  // thread 0's
    for (int32_t i = blockIdx.x; i < p.n_pairs; i += gridDim.x) {
        const float w = p.weights != nullptr ? p.weights[i] : p.uniform_weight;
        float score[2] = {0.0f, 0.0f}, share[2] = {1.0f, 1.0f};
        int64_t first[2], last[2];
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            int64_t a = p.cu[2 * (int64_t)i + side], b = p.cu[2 * (int64_t)i + side + 1];
            a = a < 0 ? 0 : a;
            b = b > p.n ? p.n : b;
            first[side] = a;
            last[side] = b;
            if (w == 0.0f) continue;
            double part = 0.0, count = 0.0;
            for (int64_t j = a + threadIdx.x; j < b; j += kPairThreads) {
                if (p.mask != nullptr && p.mask[j] == 0) continue;
                part += (double)(p.ref != nullptr ? p.logp[j] - p.ref[j] : p.logp[j]);
                count += 1.0;
            }
            part = block_total(part, s_slots);
            if (p.average) {
                count = block_total(count, s_slots);
                const double one = count > 0.0 ? 1.0 / count : 1.0;
                part *= one;
                share[side] = (float)one;
            }
            score[side] = (float)part;
        }
        float loss = 0.0f, dh = 0.0f, reward[2] = {0.0f, 0.0f};
        if (w != 0.0f) {
            const float h = score[0] - score[1], z = p.beta * h - p.margin;
            if (p.kind == ZS_PREFERENCE_SIGMOID) {
                loss = (1.0f - p.smooth) * softplus(-z) + p.smooth * softplus(z);
                dh = p.beta * (p.smooth / (1.0f + expf(-z)) - (1.0f - p.smooth) / (1.0f + expf(z)));
            } else if (p.kind == ZS_PREFERENCE_HINGE) {
                loss = z < 1.0f ? 1.0f - z : (z != z ? z : 0.0f);
                dh = z < 1.0f ? -p.beta : 0.0f;
            } else {
                const float gap = h - p.target;
                loss = gap * gap;
                dh = 2.0f * gap;
            }
            reward[0] = p.beta * score[0];
            reward[1] = p.beta * score[1];
        }
        if (threadIdx.x == 0) {
            p.loss[i] = loss;
            p.reward[2 * (int64_t)i] = reward[0];
            p.reward[2 * (int64_t)i + 1] = reward[1];
            sum[0] += (double)w * loss;
            sum[1] += reward[0] > reward[1] ? (double)w : 0.0;
            sum[2] += (double)w * ((double)reward[0] - (double)reward[1]);
        }
        if (p.dlogp == nullptr) continue;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const float d = (side ? -dh : dh) * share[side] * w;
            for (int64_t j = first[side] + threadIdx.x; j < last[side]; j += kPairThreads)
                p.dlogp[j] = p.mask != nullptr && p.mask[j] == 0 ? 0.0f : d;
        }
    }
    if (threadIdx.x == 0)
        for (int q = 0; q < ZS_PREFERENCE_TOTALS; ++q) p.work->part[blockIdx.x * ZS_PREFERENCE_TOTALS + q] = sum[q];
    if (!last_to_arrive(p.work, gridDim.x)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < ZS_PREFERENCE_TOTALS) {
        double t = 0.0;
        for (unsigned b = lane; b < gridDim.x; b += 32)
            t += *(volatile double*)&p.work->part[b * ZS_PREFERENCE_TOTALS + warp];
        t = warp_sum(t);
        if (lane == 0) s_sum[warp] = t;
    }
    __syncthreads();
    if (threadIdx.x < ZS_PREFERENCE_TOTALS) p.totals[threadIdx.x] = __double2float_rn(s_sum[threadIdx.x]);
}

}  // namespace

namespace zs {
uint64_t take_fault_preference() { return take_fault(); }
}  // namespace zs

extern "C" {

ZS_API int32_t zero_preference_loss_async(const float* logp, const float* ref_logp, const uint8_t* mask,
                                          int64_t n_tokens, const int64_t* cu_seqlens, const float* weights,
                                          int32_t n_pairs, const zs_preference* hp, float* loss, float* reward,
                                          float* dlogp, float* totals, void* work_dev, void* stream) {
    zs::NvtxRange nvtx_range("zero_preference_loss_async");
    if (n_tokens < 0 || n_pairs < 0 || hp == nullptr || !(hp->beta > 0.0) || !finite_double(hp->beta) ||
        !finite_double(hp->margin) || hp->kind < ZS_PREFERENCE_SIGMOID || hp->kind > ZS_PREFERENCE_SQUARED ||
        (hp->average != 0 && hp->average != 1) || !(hp->label_smoothing >= 0.0 && hp->label_smoothing <= 0.5) ||
        (hp->kind != ZS_PREFERENCE_SIGMOID && hp->label_smoothing != 0.0))
        return ZS_ERR_ARG;
    if (totals == nullptr || work_dev == nullptr || (n_tokens > 0 && logp == nullptr)) return ZS_ERR_ARG;
    if (n_pairs > 0 && (cu_seqlens == nullptr || loss == nullptr || reward == nullptr)) return ZS_ERR_ARG;
    if (!zs::aligned_to(cu_seqlens, 8) || !zs::aligned_to(work_dev, 8)) return ZS_ERR_ALIGN;
    const void* floats[] = {logp, ref_logp, weights, loss, reward, dlogp, totals};
    for (const void* q : floats)
        if (!zs::aligned_to(q, 4)) return ZS_ERR_ALIGN;
    const PairArgs a{logp, ref_logp, mask, n_tokens, cu_seqlens, weights,
                     n_pairs > 0 ? (float)(1.0 / (double)n_pairs) : 0.0f, n_pairs, hp->kind, hp->average,
                     (float)hp->beta, (float)hp->label_smoothing, (float)hp->margin, (float)(0.5 / hp->beta),
                     loss, reward, dlogp, totals, (Work*)work_dev};
    const int blocks = zs::persistent_blocks((const void*)preference_loss_kernel, kPairThreads,
                                             (int64_t)n_pairs * kPairThreads);
    return launch_ex(preference_loss_kernel, blocks, kPairThreads, 0, true, (cudaStream_t)stream, a,
                     "preference_loss_kernel");
}

}  // extern "C"
