// preference.cu -- the paired preference loss over packed token
// log-probabilities, with its gradient.
//
// Per pair: the two sequences' sums (or means) of logp - ref over unmasked
// tokens, one scalar loss of their difference, and a gradient that is the same
// number for every unmasked token of a sequence.  So a pair is read once for
// its sums and its gradient is written without reading the values again.
#include <stdint.h>

#include <cuda_fp16.h>

#include "cluster_counts.h"
#include "zs_internal.h"

namespace {

#include "step_common.cuh"
#include "step_end.cuh"
#include "loss_common.cuh"

[[maybe_unused]] constexpr uint32_t kSitePair = 17;

// (4096 pairs, 8.2 M tokens, in a build that dealt pairs in runs of equal tokens:
// these took 34 us, 96 threads and 10 blocks 36, 64 and 16 43, 256 and 4 47.  Dealt
// by number, as here, these take 35 and 64 and 16 took 48.)
constexpr int kPairThreads = 128, kPairWarps = kPairThreads / 32, kPairBlocks = 8;  // blocks of an SM
constexpr int kBatch = 4;  // fours that a thread loads together

struct PairArgs {
    const float *logp, *ref;
    const uint8_t* mask;
    int64_t n;
    const int64_t* cu;
    const float* weights;
    float uniform_weight;
    int32_t n_pairs, kind, average;
    float beta, smooth, margin, target;  // target = 1 / (2 beta)
    // tokens from the buffers' start to a boundary of 4 tokens in all of them
    // (0-3), or -1: there is none, tokens are taken one by one
    int32_t lead;
    float *loss, *reward, *dlogp, *totals;
    Work* work;
};

__device__ __forceinline__ float softplus(float z) { return fmaxf(z, 0.0f) + log1pf(expf(-fabsf(z))); }

// What a block has of a pair's two sequences: sums over unmasked tokens and
// their numbers.
struct PairPart {
    double sum[2];
    int64_t count[2];
};

// The tokens [lo, hi) of a sequence: whole fours [first, last) on boundaries of
// the buffers, at most three tokens before them and after them.  Without a
// common boundary all tokens come "after", and are taken one by one.
struct Range {
    int64_t lo, hi, first, last;
};
__device__ __forceinline__ Range range_of(const PairArgs& p, int64_t u, int64_t v) {
    Range r;
    r.lo = min(max(u, (int64_t)0), p.n);
    r.hi = min(max(v, r.lo), p.n);
    r.first = r.last = r.lo;
    if (p.lead >= 0) {
        // (lo + 4 keeps the dividends positive)
        r.first = min((r.lo - p.lead + 4 + 3) / 4 * 4 - 4 + p.lead, r.hi);
        r.last = max((r.hi - p.lead + 4) / 4 * 4 - 4 + p.lead, r.first);
    }
    return r;
}

// 13 bytes in and out for a token and the mask once more.  A cluster takes a
// pair: one block of it where there are many pairs, up to eight where there are
// few.  Tokens are taken four at a time; a pair of usual length gives each
// thread a few fours, so what a pair costs whatever its length (the sums' joining,
// the loss) is kept to four warps.
// Measured: 4096 pairs, 8.2 M tokens, 35 us, 3.0 TB/s of the bytes that have to
// move (147 us in the first form, token by token).  It fills neither memory (45 %)
// nor issue (2.1 of 4 slots); waiting at the barriers around a pair's serial part is
// its most frequent stall, and pairs are dealt by number, whatever their lengths.
__global__ void __launch_bounds__(kPairThreads, kPairBlocks) preference_loss_kernel(const __grid_constant__ PairArgs p) {
    __shared__ double s_sum[kPairWarps][2];
    __shared__ int64_t s_count[kPairWarps][2];
    __shared__ PairPart s_peer[2][kMaxCluster];
    __shared__ float s_grad[2];
    __shared__ double s_total[ZS_PREFERENCE_TOTALS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t ctas = (int32_t)cluster_size(), rank = (int32_t)cluster_rank();
    if (ctas > 1) cluster_arrive();  // matched by the wait below: every block of the cluster has started
    griddep_wait();
    griddep_launch_dependents();
    if (ctas > 1) cluster_wait();
    const uint32_t cluster = blockIdx.x / (uint32_t)ctas, clusters = gridDim.x / (uint32_t)ctas;
    const uint32_t n_pairs = (uint32_t)p.n_pairs;  // (up to 2^31 - 1: one cluster further still has 32 bits)
    const int32_t me = rank * kPairThreads + tid, step = ctas * kPairThreads;
    double sum[ZS_PREFERENCE_TOTALS] = {};  // of the cluster's first thread
    int par = 0;
    int64_t next_cu[3] = {0, 0, 0};
    float next_w = 0.0f;
    auto fetch = [&](uint32_t i) {  // a pair's offsets and weight, one pair ahead
        if (i >= n_pairs) return;
#pragma unroll
        for (int k = 0; k < 3; ++k) next_cu[k] = p.cu[2 * (int64_t)i + k];
        next_w = p.weights != nullptr ? p.weights[i] : p.uniform_weight;
    };
    fetch(cluster);
    for (uint32_t i = cluster; i < n_pairs; i += clusters) {
        const float w = next_w;
        const Range r0 = range_of(p, next_cu[0], next_cu[1]), r1 = range_of(p, next_cu[1], next_cu[2]);
        fetch(i + clusters);
        // the fours of both sequences as one list: four x at fours(x)
        const int32_t g0 = (int32_t)((r0.last - r0.first) / 4), groups = g0 + (int32_t)((r1.last - r1.first) / 4);
        const int64_t first1 = r1.first - 4 * (int64_t)g0;
        auto token_of = [&](int32_t x) { return (x < g0 ? r0.first : first1) + 4 * (int64_t)x; };
        // the tokens outside them: with fours there are at most three at each of
        // four places, one to a thread of the first block
        const bool lone_chosen = tid < 8;
        const int at = tid & 7;
        int64_t lone = -1;
        if (p.lead >= 0 && rank == 0 && tid < 16) {
            const int64_t t = at < 4 ? (lone_chosen ? r0.lo : r1.lo) + at : (lone_chosen ? r0.last : r1.last) + at - 4;
            if (t < (at < 4 ? (lone_chosen ? r0.first : r1.first) : (lone_chosen ? r0.hi : r1.hi))) lone = t;
        }
        Sum2 part0{0.0f, 0.0f}, part1{0.0f, 0.0f};
        int32_t count0 = 0, count1 = 0;
        uint32_t m[kBatch];      // masks of the thread's first fours
        bool lone_mask = true;   // and of its lone token
        // (loads first, all of them; a masked token's values are not used,
        // whatever they are)
        auto batch = [&](int32_t x0, uint32_t (&mask)[kBatch]) {
            float4 l[kBatch], f[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int32_t x = x0 + k * step;
                const int64_t t = token_of(x);
                mask[k] = 0u;
                l[k] = f[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (x < groups && ZS_RANGE_OK(kSitePair, t, 4, p.n)) {
                    l[k] = __ldcs(reinterpret_cast<const float4*>(p.logp + t));
                    if (p.ref != nullptr) f[k] = __ldcs(reinterpret_cast<const float4*>(p.ref + t));
                    mask[k] = p.mask != nullptr ? *reinterpret_cast<const uint32_t*>(p.mask + t) : 0x01010101u;
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const bool h0 = (mask[k] & 0xffu) != 0u, h1 = (mask[k] & 0xff00u) != 0u, h2 = (mask[k] & 0xff0000u) != 0u,
                           h3 = (mask[k] & 0xff000000u) != 0u;
                const float d = ((h0 ? l[k].x - f[k].x : 0.0f) + (h1 ? l[k].y - f[k].y : 0.0f)) +
                                ((h2 ? l[k].z - f[k].z : 0.0f) + (h3 ? l[k].w - f[k].w : 0.0f));
                const bool chosen = x0 + k * step < g0;
                part0.add(chosen ? d : 0.0f);
                part1.add(chosen ? 0.0f : d);
                const int32_t c = (h0 ? 1 : 0) + (h1 ? 1 : 0) + (h2 ? 1 : 0) + (h3 ? 1 : 0);
                count0 += chosen ? c : 0;
                count1 += chosen ? 0 : c;
            }
        };
#pragma unroll
        for (int k = 0; k < kBatch; ++k) m[k] = 0u;
        if (w != 0.0f) {
            float l = 0.0f, f = 0.0f;
            if (lone >= 0 && ZS_RANGE_OK(kSitePair, lone, 1, p.n)) {
                l = p.logp[lone];
                if (p.ref != nullptr) f = p.ref[lone];
                if (p.mask != nullptr) lone_mask = p.mask[lone] != 0;
            }
            batch(me, m);
            for (int32_t x = me + kBatch * step; x < groups; x += kBatch * step) {
                uint32_t unused[kBatch];
                batch(x, unused);
            }
            if (lone >= 0 && lone_mask) {
                part0.add(lone_chosen ? l - f : 0.0f);
                part1.add(lone_chosen ? 0.0f : l - f);
                count0 += lone_chosen ? 1 : 0;
                count1 += lone_chosen ? 0 : 1;
            }
            if (p.lead < 0) {  // one by one
                auto each = [&](const Range& r, Sum2& part, int32_t& count) {
#pragma unroll 4
                    for (int64_t t = r.lo + me; t < r.hi; t += step) {
                        if (!ZS_RANGE_OK(kSitePair, t, 1, p.n)) continue;
                        const float d = p.ref != nullptr ? p.logp[t] - p.ref[t] : p.logp[t];
                        const bool have = p.mask == nullptr || p.mask[t] != 0;
                        part.add(have ? d : 0.0f);
                        count += have ? 1 : 0;
                    }
                };
                each(r0, part0, count0);
                each(r1, part1, count1);
            }
        }
        // the warps', the block's and the cluster's sums, in a fixed order
        // (the lower half of a warp goes on with the chosen sequence, the upper
        // with the other; fp64 sums would be bound by their few units)
        {
            const bool low = lane < 16;
            Sum2 keep = low ? part0 : part1, give = low ? part1 : part0;
            keep.add(__shfl_xor_sync(0xffffffffu, give.hi, 16));
            keep.lo = __fadd_rn(keep.lo, __shfl_xor_sync(0xffffffffu, give.lo, 16));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) {
                const float hi = __shfl_xor_sync(0xffffffffu, keep.hi, o), lo = __shfl_xor_sync(0xffffffffu, keep.lo, o);
                keep.add(hi);
                keep.lo = __fadd_rn(keep.lo, lo);
            }
            if ((lane & 15) == 0) s_sum[warp][lane >> 4] = keep.value();
            if (p.average) {
                const int32_t k0 = __reduce_add_sync(0xffffffffu, count0), k1 = __reduce_add_sync(0xffffffffu, count1);
                if (lane == 0) {
                    s_count[warp][0] = k0;
                    s_count[warp][1] = k1;
                }
            } else if (lane == 0) {
                s_count[warp][0] = s_count[warp][1] = 0;
            }
        }
        __syncthreads();
        PairPart mine{{0.0, 0.0}, {0, 0}};
        if (warp == 0) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
                for (int k = 0; k < kPairWarps; ++k) {
                    mine.sum[s] += s_sum[k][s];
                    mine.count[s] += s_count[k][s];
                }
        }
        if (ctas > 1) {
            if (warp == 0 && lane < ctas) {
                uint32_t a;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(&s_peer[par][rank])), "r"(lane));
                asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(a), "d"(mine.sum[0]) : "memory");
                asm volatile("st.shared::cluster.f64 [%0+8], %1;" ::"r"(a), "d"(mine.sum[1]) : "memory");
                asm volatile("st.shared::cluster.s64 [%0+16], %1;" ::"r"(a), "l"(mine.count[0]) : "memory");
                asm volatile("st.shared::cluster.s64 [%0+24], %1;" ::"r"(a), "l"(mine.count[1]) : "memory");
            }
            cluster_arrive();
            cluster_wait();
            mine = PairPart{{0.0, 0.0}, {0, 0}};
            if (warp == 0) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    for (int k = 0; k < ctas; ++k) {
                        mine.sum[s] += s_peer[par][k].sum[s];
                        mine.count[s] += s_peer[par][k].count[s];
                    }
            }
            par ^= 1;  // the other half next: this one may still be read
        }
        if (warp == 0) {
            float score[2], share[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const double one = p.average && mine.count[s] > 0 ? 1.0 / (double)mine.count[s] : 1.0;
                score[s] = (float)(mine.sum[s] * one);
                share[s] = (float)one;
            }
            float loss = 0.0f, dh = 0.0f, reward[2] = {0.0f, 0.0f};
            if (w != 0.0f) {
                const float h = score[0] - score[1], z = p.beta * h - p.margin;
                if (p.kind == ZS_PREFERENCE_SIGMOID) {
                    loss = (1.0f - p.smooth) * softplus(-z);
                    if (p.smooth != 0.0f) loss += p.smooth * softplus(z);  // (0 times an infinite one has no value)
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
            if (lane == 0) {
                s_grad[0] = dh * share[0] * w;
                s_grad[1] = -dh * share[1] * w;
                if (rank == 0) {
                    p.loss[i] = loss;
                    p.reward[2 * (int64_t)i] = reward[0];
                    p.reward[2 * (int64_t)i + 1] = reward[1];
                    sum[0] += (double)w * loss;
                    sum[1] += reward[0] > reward[1] ? (double)w : 0.0;
                    sum[2] += (double)w * ((double)reward[0] - (double)reward[1]);
                }
            }
        }
        // (s_sum and s_grad are written again only after the next pair's first
        // and second barrier)
        __syncthreads();
        if (p.dlogp == nullptr) continue;
        const float d0 = s_grad[0], d1 = s_grad[1];
        auto write = [&](int32_t x, uint32_t mask) {
            const int64_t t = token_of(x);
            if (x >= groups || !ZS_RANGE_OK(kSitePair, t, 4, p.n)) return;
            const float g = x < g0 ? d0 : d1;
            __stcs(reinterpret_cast<float4*>(p.dlogp + t),
                   make_float4((mask & 0xffu) != 0u ? g : 0.0f, (mask & 0xff00u) != 0u ? g : 0.0f,
                               (mask & 0xff0000u) != 0u ? g : 0.0f, (mask & 0xff000000u) != 0u ? g : 0.0f));
        };
#pragma unroll
        for (int k = 0; k < kBatch; ++k) write(me + k * step, m[k]);
#pragma unroll 4
        for (int32_t x = me + kBatch * step; x < groups; x += step)
            write(x, p.mask != nullptr ? *reinterpret_cast<const uint32_t*>(p.mask + token_of(x)) : 0x01010101u);
        if (lone >= 0 && ZS_RANGE_OK(kSitePair, lone, 1, p.n)) p.dlogp[lone] = lone_mask ? (lone_chosen ? d0 : d1) : 0.0f;
        if (p.lead < 0) {
            auto each = [&](const Range& r, float g) {
#pragma unroll 4
                for (int64_t t = r.lo + me; t < r.hi; t += step)
                    if (ZS_RANGE_OK(kSitePair, t, 1, p.n)) p.dlogp[t] = p.mask != nullptr && p.mask[t] == 0 ? 0.0f : g;
            };
            each(r0, d0);
            each(r1, d1);
        }
    }
    if (rank != 0) return;
    if (tid == 0)
        for (int q = 0; q < ZS_PREFERENCE_TOTALS; ++q) p.work->part[cluster * ZS_PREFERENCE_TOTALS + q] = sum[q];
    if (!last_to_arrive(p.work, clusters)) return;
    if (warp < ZS_PREFERENCE_TOTALS) {
        double t = 0.0;
        for (uint32_t b = lane; b < clusters; b += 32) t += *(volatile double*)&p.work->part[b * ZS_PREFERENCE_TOTALS + warp];
        t = warp_sum(t);
        if (lane == 0) s_total[warp] = t;
    }
    __syncthreads();
    if (tid < ZS_PREFERENCE_TOTALS) p.totals[tid] = __double2float_rn(s_total[tid]);
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
    if (n_tokens < 0 || n_tokens > (1ll << 32) || n_pairs < 0 || hp == nullptr || !(hp->beta > 0.0) || !finite_double(hp->beta) ||
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
    PairArgs a{logp, ref_logp, mask, n_tokens, cu_seqlens, weights,
               n_pairs > 0 ? (float)(1.0 / (double)n_pairs) : 0.0f, n_pairs, hp->kind, hp->average,
               (float)hp->beta, (float)hp->label_smoothing, (float)hp->margin, (float)(0.5 / hp->beta),
               -1, loss, reward, dlogp, totals, (Work*)work_dev};
    for (int lead = 0; lead < 4 && a.lead < 0; ++lead) {
        auto at = [&](const float* q) { return q == nullptr || zs::aligned_to(q + lead, 16); };
        if (at(logp) && at(ref_logp) && at(dlogp) && (mask == nullptr || zs::aligned_to(mask + lead, 4))) a.lead = lead;
    }
    // one block to a pair, more while blocks would be idle and have a step's work
    const int full = kPairBlocks * zs::device_sm_count();
    int ctas = 1;
    const int64_t mean = n_pairs > 0 ? n_tokens / n_pairs : 0;
    while (ctas < kMaxCluster && 2ll * ctas * n_pairs <= full && mean > (int64_t)ctas * kPairThreads * 4) ctas *= 2;
    cudaError_t err = cudaSuccess;
    int clusters = active_clusters((const void*)preference_loss_kernel, kPairThreads, ctas, 0, &err);
    if (clusters < 1) return zs::cuda_fail(err, "preference_loss_kernel");
    if (clusters > n_pairs) clusters = n_pairs > 0 ? n_pairs : 1;
    return launch_clusters(preference_loss_kernel, clusters, ctas, kPairThreads, 0, (cudaStream_t)stream, a,
                           "preference_loss_kernel");
}

}  // extern "C"
