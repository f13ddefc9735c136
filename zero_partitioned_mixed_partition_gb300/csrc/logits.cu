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
//
// One kernel does all of it (rows_kernel).  A cluster of 1 to 8 CTAs takes a
// row, each CTA a slice of its 16-byte vectors.  One warp of a CTA loads the
// slice ahead into a ring of buffers in shared memory by bulk copies.  Eight
// warps compute: a first pass over the slice gives their parts of the row's
// statistics, and where a gradient is wanted a second pass writes it.  One more
// warp joins the parts, exchanges them with the cluster's other CTAs through
// distributed shared memory and turns them into the row's outputs and gradient
// coefficients; no barrier of the block is on the way.  The second pass finds the
// row in L2: so few rows are under way at once that they fit there (plan_rows).
// Forms that kept the slices in shared memory between the passes were built
// first; the best of them took 910 us in the first case below, with clusters of
// six CTAs.
//
// Measured on one GB300 (6787 GB/s copied): policy loss and gradient, 8192 x
// 131072 bf16, a tenth of the rows left out, with entropy: 683 us, 5.97 TB/s of
// the bytes that have to move; 4096 x 32000 bf16, 30 % left out, no entropy:
// 87 us, 5.1 TB/s; log-probabilities, 8192 x 50257 bf16, a quarter left out:
// 99 us, 6.2 TB/s.  Nothing is full in the first: 88 % of the copy rate, and 2.2 of 4
// issue slots a cycle (on 1024 rows; 130 instructions for 8 logits, 87 of them in
// the two passes' loops).  In the second a CTA takes its rows one at a time, so the
// turn from statistics to gradient stands open in each (an estimated 1.5 us of
// 8), and its 2867 live rows are 9.4 rounds of 304; letting the next row's first
// pass go in between was tried: 94 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <cfloat>
#include <initializer_list>

#include "cluster_counts.h"
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

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------- vectors ---

// A 16-byte vector: its values as fp32 pairs, its largest value (a NaN is
// passed over), and fp32 pairs rounded to it.
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void pairs(const uint4& r, uint64_t* x) {
        x[0] = pair(__uint_as_float(r.x), __uint_as_float(r.y));
        x[1] = pair(__uint_as_float(r.z), __uint_as_float(r.w));
    }
    static __device__ __forceinline__ float top(const uint4& r) {
        return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
    }
    static __device__ __forceinline__ uint4 pack(const uint64_t* x) {
        float a, b, c, d;
        split(x[0], a, b);
        split(x[1], c, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
};
template <> struct Vec<__half> {
    static constexpr int N = 8;
    static __device__ __forceinline__ __half2 h2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
    static __device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
    static __device__ __forceinline__ uint64_t widen(uint32_t w) {
        const float2 f = __half22float2(h2(w));
        return pair(f.x, f.y);
    }
    static __device__ __forceinline__ uint32_t narrow(float a, float b) { return bits(__floats2half2_rn(a, b)); }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return bits(__hmax2(h2(a), h2(b))); }
    static __device__ __forceinline__ uint32_t at_least(uint32_t w, uint32_t t) { return bits(__hmax2_nan(h2(w), h2(t))); }
    static __device__ __forceinline__ bool any_above(uint32_t m, uint32_t t) { return !__hble2(h2(m), h2(t)); }
    static __device__ __forceinline__ uint32_t down(float x) { return bits(__half2half2(__float2half_rd(x))); }
    static constexpr uint32_t kInfinity = 0x7c00u;
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ __nv_bfloat162 h2(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
    static __device__ __forceinline__ uint32_t bits(__nv_bfloat162 h) { return *reinterpret_cast<const uint32_t*>(&h); }
    static __device__ __forceinline__ uint64_t widen(uint32_t w) {  // bf16 is the upper half of an fp32
        return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t narrow(float a, float b) { return bits(__floats2bfloat162_rn(a, b)); }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return bits(__hmax2(h2(a), h2(b))); }
    static __device__ __forceinline__ uint32_t at_least(uint32_t w, uint32_t t) { return bits(__hmax2_nan(h2(w), h2(t))); }
    static __device__ __forceinline__ bool any_above(uint32_t m, uint32_t t) { return !__hble2(h2(m), h2(t)); }
    static __device__ __forceinline__ uint32_t down(float x) { return bits(__bfloat162bfloat162(__float2bfloat16_rd(x))); }
    static constexpr uint32_t kInfinity = 0x7f80u;
};
template <typename T>
__device__ __forceinline__ void pairs_of(const uint4& r, uint64_t* x) {
    if constexpr (sizeof(T) == 4) {
        Vec<T>::pairs(r, x);
    } else {
        x[0] = Vec<T>::widen(r.x);
        x[1] = Vec<T>::widen(r.y);
        x[2] = Vec<T>::widen(r.z);
        x[3] = Vec<T>::widen(r.w);
    }
}
template <typename T>
__device__ __forceinline__ uint4 vector_of(const uint64_t* x) {
    if constexpr (sizeof(T) == 4) {
        return Vec<T>::pack(x);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            split(x[i], a, b);
            w[i] = Vec<T>::narrow(a, b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}
template <typename T>
__device__ __forceinline__ uint32_t top2_of(const uint4& r) {
    return Vec<T>::max2(Vec<T>::max2(r.x, r.y), Vec<T>::max2(r.z, r.w));
}
// The larger of a pair of 16-bit values (a NaN is passed over).
template <typename T>
__device__ __forceinline__ float larger(uint32_t w) {
    float a, b;
    split(Vec<T>::widen(w), a, b);
    return fmaxf(a, b);
}
template <typename T>
__device__ __forceinline__ uint4 at_least(const uint4& r, uint32_t t) {
    return make_uint4(Vec<T>::at_least(r.x, t), Vec<T>::at_least(r.y, t), Vec<T>::at_least(r.z, t), Vec<T>::at_least(r.w, t));
}

// ------------------------------------------------------------ row statistics ---

// Statistics of a part of a row, in units of log2: s = sum 2^a, u = sum 2^a a
// with a = x k - c, k = it log2 e, and c = top k rounded once, the same c for
// the whole part; so a is rounded once from its exact value (one fused
// multiply-add) and c's own rounding is the same factor in every term.  top is
// not the largest logit but one that the largest exceeds by at most kSlack in
// those units: a sum is scaled to a new top only where a vector exceeds that,
// which after the first vectors hardly happens.  c's rounding moves a by up to
// half a unit of its last place, so this form serves where |c| < 2^24 (half a
// unit is 1/2 there, and an a of kSlack + 1/2 times any vocabulary is far from
// fp32's range); it would leave the range from 2^31 on.  For larger c, a vocabulary
// masked with -1e9 or below, a is (x - top) k instead.  top starts at the lowest
// finite float, so that a row of nothing but -inf keeps s = 0 and no difference of
// infinities is formed.
constexpr float kSlack = 20.0f;
constexpr float kLargeC = 0x1p24f;
// A logit this far below top, in the same units, has 2^a = 0 (ex2 flushes to 0
// below -126).  Where 2^a a is summed, such logits are raised to it (16-bit
// types, two by one instruction), or a to kLowest: 0 times -inf would be NaN.
constexpr float kFloor = 200.0f;
constexpr float kLowest = -1e4f;

struct __align__(16) Stats {
    float top, s, u;
    float x_label;  // the row's label's logit, carried along
};

// What is left of c's rounding: c - top k, exactly (0 in the slow form).
__device__ __forceinline__ float c_residue(float top, float k) {
    const float c = __fmul_rn(top, k);
    return fabsf(c) < kLargeC ? -fmaf(top, k, -c) : 0.0f;
}

// How far the sums at top a lie above those at top b: the difference of their c,
// where a slow one counts as top k.  (One expression for all: a branch for two fast
// ones took 695 us where this takes 688, in the first case above.)
__device__ __forceinline__ float top_gap(float a, float b, float k) {
    return fmaxf(fmaf(a - b, k, c_residue(a, k) - c_residue(b, k)), kLowest);
}

// How a vector's exponentials are formed, by the row's top: kSlow where c
// would be too large, kBounded with a raised to kLowest, else the 16-bit value
// that logits are raised to, twice.  (No such value has these bits: -0 and the
// negative number next to it.)
constexpr uint32_t kSlow = 0x80008000u, kBounded = 0x80018001u;
template <typename T>
__device__ __forceinline__ uint32_t floor_of(float top, float k) {
    if (!(fabsf(__fmul_rn(top, k)) < kLargeC)) return kSlow;
    if constexpr (sizeof(T) == 2) {
        const uint32_t f = Vec<T>::down(top - kFloor / k);
        return (f & Vec<T>::kInfinity) != Vec<T>::kInfinity ? f : kBounded;
    }
    return kBounded;
}

// A thread's running statistics, two columns of sums.  above: the largest
// 16-bit logit that needs no new top, twice.
template <typename T>
struct Running {
    float top, c;
    uint64_t s2, u2;
    uint32_t above, floor;
};

template <bool ENT, typename T>
__device__ __forceinline__ void set_top(Running<T>& st, float top, float k) {
    const float gap = top_gap(st.top, top, k), f = exp2_approx(gap);
    const uint64_t f2 = pair(f, f);
    if (ENT) st.u2 = mul2(f2, fma2(pair(gap, gap), st.s2, st.u2));
    st.s2 = mul2(f2, st.s2);
    st.top = top;
    st.c = __fmul_rn(top, k);
    st.floor = floor_of<T>(top, k);
    if constexpr (sizeof(T) == 2) st.above = Vec<T>::down(top + kSlack / k);
}
template <typename T>
__device__ __forceinline__ Running<T> empty_stats() {
    Running<T> st;
    st.top = st.c = -FLT_MAX;
    st.s2 = st.u2 = 0ull;
    st.floor = kSlow;
    if constexpr (sizeof(T) == 2) st.above = Vec<T>::kInfinity * 0x10001u | 0x80008000u;  // -inf: anything is above
    return st;
}

// The vector's logits raised to the floor.
template <typename T>
__device__ __forceinline__ uint4 raised(const uint4& r, uint32_t floor) {
    if constexpr (sizeof(T) == 2)
        return make_uint4(Vec<T>::at_least(r.x, floor), Vec<T>::at_least(r.y, floor), Vec<T>::at_least(r.z, floor),
                          Vec<T>::at_least(r.w, floor));
    return r;
}

// RAISED: the logits have been raised, no a needs a bound.
template <typename T, bool ENT, bool SLOW, bool RAISED, int U>
__device__ __forceinline__ void sum_vectors(Running<T>& st, const uint4 (&r)[U], float k) {
    constexpr int H = Vec<T>::N / 2;
    const uint64_t kk = pair(k, k), minus = SLOW ? pair(-st.top, -st.top) : pair(-st.c, -st.c);
    uint64_t s2[U], u2[U];  // a column of sums for each vector
#pragma unroll
    for (int g = 0; g < U; ++g) {
        uint64_t x[H];
        pairs_of<T>(RAISED && ENT ? raised<T>(r[g], st.floor) : r[g], x);
        s2[g] = u2[g] = 0ull;
#pragma unroll
        for (int j = 0; j < H; ++j) {
            float a, b;
            const uint64_t d = SLOW ? mul2(add2(x[j], minus), kk) : fma2(x[j], kk, minus);
            split(d, a, b);
            const uint64_t e = pair(exp2_approx(a), exp2_approx(b));
            s2[g] = j == 0 ? e : add2(s2[g], e);
            if (ENT) {
                const uint64_t m = RAISED ? d : pair(fmaxf(a, kLowest), fmaxf(b, kLowest));
                u2[g] = j == 0 ? mul2(e, m) : fma2(e, m, u2[g]);
            }
        }
    }
#pragma unroll
    for (int g = 0; g < U; ++g) {
        st.s2 = add2(st.s2, s2[g]);
        if (ENT) st.u2 = add2(st.u2, u2[g]);
    }
}

// U vectors at once: one test for a new top, and U independent columns of work.
template <typename T, bool ENT, int U>
__device__ __forceinline__ void add_vectors(Running<T>& st, const uint4 (&r)[U], float k) {
    if constexpr (sizeof(T) == 2) {
        uint32_t m = top2_of<T>(r[0]);
#pragma unroll
        for (int g = 1; g < U; ++g) m = Vec<T>::max2(m, top2_of<T>(r[g]));
        if (Vec<T>::any_above(m, st.above)) {
            const float top = larger<T>(m);
            if (top > st.top) set_top<ENT, T>(st, top, k);
        }
    } else {
        float top = Vec<T>::top(r[0]);
#pragma unroll
        for (int g = 1; g < U; ++g) top = fmaxf(top, Vec<T>::top(r[g]));
        if ((top - st.top) * k > kSlack) set_top<ENT, T>(st, top, k);
    }
    constexpr bool kCanRaise = sizeof(T) == 2 || !ENT;
    if (kCanRaise && st.floor != kSlow && (!ENT || st.floor != kBounded))
        sum_vectors<T, ENT, false, kCanRaise, U>(st, r, k);
    else if (st.floor != kSlow)
        sum_vectors<T, ENT, false, false, U>(st, r, k);
    else
        sum_vectors<T, ENT, true, false, U>(st, r, k);
}

template <typename T, bool ENT>
__device__ __forceinline__ void add_value(Running<T>& st, float x, float k) {
    if ((x - st.top) * k > kSlack) set_top<ENT, T>(st, x, k);
    const float a = st.floor != kSlow ? fmaf(x, k, -st.c) : (x - st.top) * k, e = exp2_approx(a);
    st.s2 = add2(st.s2, pair(e, 0.0f));
    if (ENT) st.u2 = add2(st.u2, pair(e * fmaxf(a, kLowest), 0.0f));
}

// The warp's statistics from its lanes', valid in every lane.
template <bool ENT>
__device__ __forceinline__ Stats join_warp(Stats st, float k) {
    // an order of floats as unsigned integers; top is never a NaN
    const uint32_t b = __float_as_uint(st.top), key = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    const uint32_t most = __reduce_max_sync(0xffffffffu, key);
    const float top = __uint_as_float(most ^ ((uint32_t)((int32_t)~most >> 31) | 0x80000000u));
    const float gap = top_gap(st.top, top, k), f = exp2_approx(gap);
    if (ENT) st.u = f * (st.u + gap * st.s);
    st.s *= f;
    st.top = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        st.s += __shfl_xor_sync(0xffffffffu, st.s, o);
        if (ENT) st.u += __shfl_xor_sync(0xffffffffu, st.u, o);
    }
    return st;
}

// ---------------------------------------------------------------- gradient ---

// Coefficients of a row's gradient: dx_i = p_i (c0 + c1 q_i) + cy [i = y] with
// q_i = log2 p_i = (x_i - top) k - l2; and the same in the statistics' terms,
// a = x_i k - c: dx_i = 2^a (f0 + f1 a) + cy [i = y].
struct GradCoef {
    float top, l2, c0, c1, cy;
    float c, f0, f1;
    uint32_t floor;
    int32_t write;  // 0: the row has no distribution, its gradient is 0
};

// raw: log2 of the row's s.
template <typename T>
__device__ __forceinline__ GradCoef grad_coef(float top, float lns, float raw, float c0, float c1, float cy, float k) {
    const float inv = exp2f(-raw);
    return GradCoef{top, lns * kLog2e, c0, c1, cy, __fmul_rn(top, k), (c0 - c1 * raw) * inv, c1 * inv, floor_of<T>(top, k), 1};
}

// One element; the same bits as in a vector.
template <bool ENT>
__device__ __forceinline__ float grad_value(const GradCoef& c, float k, float x) {
    if (c.floor != kSlow) {
        const float a = fmaf(x, k, -c.c);
        return __fmul_rn(exp2_approx(a), ENT ? fmaf(c.f1, fmaxf(a, kLowest), c.f0) : c.f0);
    }
    const float q = (x - c.top) * k - c.l2;
    return __fmul_rn(exp2_approx(q), ENT ? fmaf(c.c1, fmaxf(q, kLowest), c.c0) : c.c0);
}

// The gradient of U vectors, without the label's own term.  RAISED as above;
// not for a slow row.
template <typename T, bool ENT, bool RAISED, int U>
__device__ __forceinline__ void grad_vectors(const GradCoef& c, float k, uint4 (&r)[U]) {
    constexpr int H = Vec<T>::N / 2;
    const uint64_t kk = pair(k, k), minus = pair(-c.c, -c.c), f0 = pair(c.f0, c.f0), f1 = pair(c.f1, c.f1);
#pragma unroll
    for (int g = 0; g < U; ++g) {
        uint64_t x[H];
        pairs_of<T>(RAISED && ENT ? raised<T>(r[g], c.floor) : r[g], x);
#pragma unroll
        for (int j = 0; j < H; ++j) {
            float a, b;
            const uint64_t d = fma2(x[j], kk, minus);
            split(d, a, b);
            const uint64_t e = pair(exp2_approx(a), exp2_approx(b));
            x[j] = mul2(e, ENT ? fma2(f1, RAISED ? d : pair(fmaxf(a, kLowest), fmaxf(b, kLowest)), f0) : f0);
        }
        r[g] = vector_of<T>(x);
    }
}

// One vector in any form.
template <typename T, bool ENT>
__device__ __forceinline__ uint4 grad_vector(const GradCoef& c, float k, const uint4& r) {
    uint64_t x[Vec<T>::N / 2];
    pairs_of<T>(r, x);
#pragma unroll
    for (int j = 0; j < Vec<T>::N / 2; ++j) {
        float a, b;
        split(x[j], a, b);
        x[j] = pair(grad_value<ENT>(c, k, a), grad_value<ENT>(c, k, b));
    }
    return vector_of<T>(x);
}

// The 16-byte output vectors of a warp, consecutive lanes consecutive vectors,
// at an address that is `skip` elements short of a vector boundary: every lane
// takes its own elements from `skip` on and the next lane's up to it; the
// warp's first `skip` elements and its last ones go out one by one.
template <typename T>
__device__ __forceinline__ void store_shifted(T* out, const uint4& own, int skip) {
    constexpr int N = Vec<T>::N, PER = 4 / (int)sizeof(T);  // PER: elements of a word
    const int lane = threadIdx.x & 31;
    uint32_t w[8] = {own.x, own.y, own.z, own.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 + i] = __shfl_down_sync(0xffffffffu, w[i], 1);
    if (lane == 0 || lane == 31) {
        const uint32_t mine[4] = {own.x, own.y, own.z, own.w};
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (lane == 0 ? j >= skip : j < skip) continue;
            const uint32_t word = mine[j / PER];
            if constexpr (PER == 2)
                reinterpret_cast<unsigned short*>(out)[j] = (unsigned short)(word >> (16 * (j % 2)));
            else
                reinterpret_cast<uint32_t*>(out)[j] = word;
        }
    }
    const int words = skip / PER;
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = words & 2 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = words & 1 ? w[i + 1] : w[i];
    if (PER == 2 && (skip & 1)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    if (lane < 31) __stcs(reinterpret_cast<uint4*>(out + skip), make_uint4(w[0], w[1], w[2], w[3]));
}

// Zeros from out to out + n, by the whole block.
template <typename T>
__device__ __forceinline__ void zero_range(T* out, int64_t n, int threads) {
    constexpr int N = Vec<T>::N;
    int64_t head = (int64_t)(((16u - ((uintptr_t)out & 15u)) & 15u) / sizeof(T));
    if (head > n) head = n;
    const int64_t nvec = (n - head) / N, tail = head + nvec * N;
    if (threadIdx.x < head) out[threadIdx.x] = from_float<T>(0.0f);
    if (tail + threadIdx.x < n) out[tail + threadIdx.x] = from_float<T>(0.0f);
    for (int64_t i = threadIdx.x; i < nvec; i += threads)
        __stcs(reinterpret_cast<uint4*>(out + head + i * N), make_uint4(0u, 0u, 0u, 0u));
}

// ------------------------------------------------------ copies and clusters ---

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
// Whether the phase of the given parity is over; waits up to 2 us for it.
__device__ __forceinline__ bool mbar_try(uint64_t* b, uint32_t parity) {
    uint32_t done = 0;
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
template <bool RELAXED>
__device__ __forceinline__ bool mbar_wait_on(uint64_t* b, uint32_t parity, int32_t* failed) {
    const int limit = wait_limit();
#pragma unroll 1
    for (int i = 0; i < limit; ++i) {
        if (mbar_try(b, parity)) return true;
        if (*(volatile int32_t*)failed) return false;
        if (RELAXED) __nanosleep(100);
    }
    *(volatile int32_t*)failed = 1;
    return false;
}
// Waits for the phase, within the limit.  A wait that runs out sets *failed and
// returns false; so do the block's other waits from then on, at once.  RELAXED: for
// the warps that mostly wait; they leave the issue slots to the others.  (Most waits
// are over at the first try; with that in the loop, 708 us for 684 in the first case
// above.)
template <bool RELAXED = false>
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity, int32_t* failed) {
#if ZS_CHECKED
    if (wait_limit() == 0) return mbar_wait_on<RELAXED>(b, parity, failed);
#endif
    return mbar_try(b, parity) || mbar_wait_on<RELAXED>(b, parity, failed);
}
// Whether every lane of the warp may go on.
__device__ __forceinline__ bool all_lanes(bool ok) { return __all_sync(0xffffffffu, ok); }
// Waits, within the ordinary limit, until the barrier counts no copy in flight.
__device__ __forceinline__ void drain(uint64_t* b, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < kWaitLimit; ++i)
        if (mbar_try(b, parity)) return;
}
// bytes (a multiple of 16, both addresses on 16-byte boundaries) from global
// to shared memory, counted by the barrier.
__device__ __forceinline__ void copy_bulk(void* dst, const void* src, uint32_t bytes, uint64_t* b) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(dst)), "l"(src), "r"(bytes), "r"(smem_addr(b)) : "memory");
}

// Writes statistics at the same place of the shared memory of CTA `rank`, and
// counts their 16 bytes at that CTA's barrier.
__device__ __forceinline__ void store_to_peer(Stats* at, uint64_t* b, uint32_t rank, const Stats& st) {
    uint32_t a, m;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(at)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(m) : "r"(smem_addr(b)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a),
                 "f"(st.top), "f"(st.s), "f"(st.u), "f"(st.x_label), "r"(m) : "memory");
}
// ------------------------------------------------------------------- kernel ---

// What the kernel makes of a row.
enum : int {
    kLogp = 0,        // log-probability and entropy
    kLogpGrad = 1,    // their gradient, from saved statistics
    kPolicyLoss = 2,  // the policy loss without a gradient
    kPolicy = 3,      // and with it
};
constexpr bool reads_for_stats(int mode) { return mode != kLogpGrad; }
constexpr bool writes_grad(int mode) { return mode == kLogpGrad || mode == kPolicy; }

struct RowArgs {
    const void* data;
    void* out;
    int64_t rows, vocab, stride, out_stride;
    float it;
    int32_t piece;   // vectors of a buffer
    int32_t buffers;
    int32_t group;   // clusters that share out their rows by the number of live ones
    const int64_t* labels;
    const zs_ctrl* ctrl;
    float *logp, *entropy;
    float* saved_out;                                    // kLogp
    const float *saved, *dlogp, *row_entropy, *dentropy;  // kLogpGrad
    const float *old_logp, *adv, *ref_logp, *weights;    // policy
    float uniform_weight;                                // the rows' weight without `weights`
    float lo, hi, dual, kl, ent_coef;
    float *token_loss, *totals;
    Work* work;
};

// Computing threads of a block: kWide, or 128 where a row has few vectors; and
// the blocks of an SM.  Two blocks of 256 + 64 threads at 96 registers: three of
// 192 + 64 at 80 took 880 us and two of 384 + 64 at 72 took 732 us where these
// take 685 us (policy loss, 8192 x 131072 bf16 with entropy): the inner loops want
// the registers more than the warps.
constexpr int kWide = 256;
constexpr int per_sm_of(int threads) { return threads == 128 ? 4 : 2; }
constexpr int kList = 256;     // live rows that a cluster takes at a time
constexpr int kMaxGroup = 48;  // clusters of a group

// (All loads at once: none waits for another's test.)
template <int MODE>
__device__ __forceinline__ bool row_is_live(const RowArgs& p, int64_t r) {
    const int64_t y = p.labels[r];
    float w = 1.0f, lns = 0.0f;
    if (MODE == kLogpGrad) lns = p.saved[2 * r + 1];
    if (MODE >= kPolicyLoss && p.weights != nullptr) w = p.weights[r];
    return (y >= 0) & (y < p.vocab) & (w != 0.0f) & (lns != -INFINITY);
}

// What the computing warps need of a row, per buffer.
struct RowInfo {
    int64_t row;
    int32_t head;        // elements before the row's first whole vector
    int32_t v0, n;       // the CTA's slice: vectors v0 .. v0 + n of the row
    int32_t y;           // the label,
    int32_t y_vec, y_at; // its vector in the slice (else outside [0, n)), and its place there
    // the row's elements outside whole vectors, of the first CTA (0-7) and the
    // last (8-15): their places (-1: none) and values
    int32_t edge_at[16];
    float edge[16];
};
constexpr int kMaxBuffers = 8;

// The live and dead rows of a batch that a cluster takes, as numbers in the batch.
struct RowLists {
    int32_t live[kList], dead[kList];
    int32_t n_live, n_dead;
};

// Rows are dealt to groups of clusters in turn, and within a group the live
// ones to its clusters in turn, as the dead ones are: with a third of the rows
// left out, dealing them by number alone left some clusters half as much again
// to do as others.  live_before, dead_before: the group's rows before this
// batch.  Called by the whole block; the lists are complete on return.
template <int MODE, int NT>
__device__ __forceinline__ void deal_rows(const RowArgs& p, int64_t j0, int32_t batch, int32_t groups, int64_t group_first,
                                          int32_t mine, int64_t& live_before, int64_t& dead_before, RowLists& lists) {
    constexpr int kWarps = NT / 32;
    __shared__ int32_t s_scan[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t run = (batch + NT - 1) / NT, first = min(tid * run, batch), last = min(first + run, batch);
    static_assert(kList * kMaxGroup <= 64 * NT, "a thread's rows have a bit each");
    uint64_t alive = 0;
#pragma unroll 4
    for (int32_t j = first; j < last; ++j)
        alive |= (uint64_t)(row_is_live<MODE>(p, (j0 + j) * groups + group_first) ? 1 : 0) << (j - first);
    const int32_t count = __popcll(alive);
    int32_t upto = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    __syncthreads();  // the previous batch is done with the lists
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    int32_t before = upto - count, live_total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        live_total += s_scan[w];
    }
    // the n-th live row of the group goes to cluster n mod group; its place in
    // the list counts from the batch's first such row, live_skip rows in
    const int32_t live_skip = (int32_t)((mine - live_before % p.group + p.group) % p.group);
    const int32_t dead_skip = (int32_t)((mine - dead_before % p.group + p.group) % p.group);
    for (int32_t j = first; j < last; ++j) {
        const bool live = alive >> (j - first) & 1;
        const int32_t off = live ? before - live_skip : j - before - dead_skip;
        if (off >= 0 && off % p.group == 0) (live ? lists.live : lists.dead)[off / p.group] = j;
        before += live ? 1 : 0;
    }
    const int32_t dead_total = batch - live_total;
    if (tid == 0) {
        lists.n_live = live_total > live_skip ? (live_total - live_skip + p.group - 1) / p.group : 0;
        lists.n_dead = dead_total > dead_skip ? (dead_total - dead_skip + p.group - 1) / p.group : 0;
    }
    live_before += live_total;
    dead_before += dead_total;
    __syncthreads();
}

// NaN in every output of every row that the cluster takes, by the whole block:
// where one of its waits ran out.  What was written before is overwritten.
template <typename T, int MODE, int NT>
__device__ __noinline__ void fill_with_nan(const RowArgs& p, int32_t groups, int64_t group_first, int64_t group_rows,
                                           int32_t mine, RowLists& lists) {
    const uint32_t ctas = cluster_size(), rank = cluster_rank();
    int64_t live_before = 0, dead_before = 0;
    for (int64_t j0 = 0; j0 < group_rows; j0 += (int64_t)kList * p.group) {
        const int32_t batch = (int32_t)min(group_rows - j0, (int64_t)kList * p.group);
        deal_rows<MODE, NT + 64>(p, j0, batch, groups, group_first, mine, live_before, dead_before, lists);
        for (int32_t i = 0; i < lists.n_live + lists.n_dead; ++i) {
            const int32_t j = i < lists.n_live ? lists.live[i] : lists.dead[i - lists.n_live];
            const int64_t r = (j0 + j) * groups + group_first;
            if (writes_grad(MODE)) {
                const int64_t a = p.vocab * rank / ctas, b = p.vocab * (rank + 1) / ctas;
                for (int64_t e = a + threadIdx.x; e < b; e += NT + 64)
                    ((T*)p.out)[r * p.out_stride + e] = from_float<T>(NAN);
            }
            if (MODE != kLogpGrad && rank == 0 && threadIdx.x == 0) {
                p.logp[r] = NAN;
                if (p.entropy != nullptr) p.entropy[r] = NAN;
                if (MODE == kLogp && p.saved_out != nullptr) p.saved_out[2 * r] = p.saved_out[2 * r + 1] = NAN;
                if (MODE >= kPolicyLoss && p.token_loss != nullptr) p.token_loss[r] = NAN;
            }
        }
    }
}

// NT computing threads, a loading warp and a statistics warp.  plan_rows has
// the cluster and buffer sizes.
//
// Every wait is bounded.  A warp whose wait runs out takes no address from what it
// waited for and no further row, and frees no buffer; the block's other waits then
// run out at once, those of the cluster's other blocks in their own time.  At the
// end a block waits for its copies in flight and for its cluster, and if a wait of
// any of them ran out they write NaN into all of the cluster's rows.
template <typename T, int MODE, bool ENT, int NT>
__global__ void __launch_bounds__(NT + 64, per_sm_of(NT)) rows_kernel(const __grid_constant__ RowArgs p) {
    constexpr int N = Vec<T>::N, kWarps = NT / 32, kLoad = kWarps, kStat = kWarps + 1;
    constexpr bool STATS = reads_for_stats(MODE), GRAD = writes_grad(MODE), POLICY = MODE >= kPolicyLoss;
    constexpr int U = 2;  // vectors that a thread takes at once
    extern __shared__ uint4 s_buffers[];  // [buffer][vector]
    __shared__ RowLists s_rows;
    __shared__ RowInfo s_info[kMaxBuffers];
    __shared__ Stats s_warp[2][kWarps], s_peer[2][kMaxCluster];
    __shared__ GradCoef s_coef[2];
    // a buffer is filled / free; row parity's parts are there / its results are
    // (and its parts read); the cluster's parts are there
    __shared__ uint64_t s_full[kMaxBuffers], s_empty[kMaxBuffers], s_parts[2], s_done[2], s_met[2];
    __shared__ int32_t s_failed;  // a wait of the cluster ran out
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ctas = cluster_size(), rank = cluster_rank();
    if (tid == 0) {
        for (int i = 0; i < kMaxBuffers; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_parts[i], kWarps);
            mbar_init(&s_done[i], 1);
            mbar_init(&s_met[i], 1);
        }
        s_failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    cluster_arrive();  // matched by the wait below: every CTA has started and set up its barriers
    griddep_wait();
    griddep_launch_dependents();
    const float k = p.it * kLog2e, scale = GRAD ? loss_scale_of(p.ctrl) * p.it : 0.0f;
    const int32_t cluster = (int32_t)(blockIdx.x / ctas), clusters = (int32_t)(gridDim.x / ctas);
    const int32_t groups = clusters / p.group, mine = cluster % p.group;
    const int64_t group_first = cluster / p.group;
    const int64_t group_rows = group_first < p.rows ? (p.rows - group_first + groups - 1) / groups : 0;
    int64_t live_before = 0, dead_before = 0;
    double sum[ZS_POLICY_TOTALS] = {};  // the cluster's totals, in the statistics warp's first lane
    // the cursor through the buffers, and the rows' parity
    int32_t buf = 0, par = 0;
    uint32_t phase = 0, par_phase = 0;
    auto advance = [&]() {
        if (++buf == p.buffers) {
            buf = 0;
            phase ^= 1u;
        }
    };
    auto next_row = [&]() {
        par ^= 1;
        if (par == 0) par_phase ^= 1u;
    };
    cluster_wait();

    for (int64_t j0 = 0; j0 < group_rows; j0 += (int64_t)kList * p.group) {
        if (j0 > 0 && __syncthreads_or(*(volatile int32_t*)&s_failed)) break;
        const int32_t batch = (int32_t)min(group_rows - j0, (int64_t)kList * p.group);
        deal_rows<MODE, NT + 64>(p, j0, batch, groups, group_first, mine, live_before, dead_before, s_rows);
        const int32_t n_live = s_rows.n_live;
        auto row_at = [&](int32_t j) { return (j0 + j) * groups + group_first; };

        if (warp == kLoad) {
            // ---- the loading warp
            auto load_row = [&](int32_t i) {
                const int64_t r = row_at(s_rows.live[i]), y = p.labels[r];
                const T* row = (const T*)p.data + r * p.stride;
                int32_t head = (int32_t)(((16u - ((uintptr_t)row & 15u)) & 15u) / sizeof(T));
                if (head > p.vocab) head = (int32_t)p.vocab;
                const int32_t nvec = (int32_t)((p.vocab - head) / N);
                const int32_t per = (nvec + (int32_t)ctas - 1) / (int32_t)ctas;
                const int32_t v0 = min((int32_t)rank * per, nvec), n = min(per, nvec - v0);
                int32_t edge_at = -1;
                if (lane < 8 && rank == 0 && lane < head) edge_at = lane;
                const int64_t tail = head + (int64_t)nvec * N + lane - 8;
                if (lane >= 8 && lane < 16 && rank == ctas - 1 && tail < p.vocab) edge_at = (int32_t)tail;
                const float edge = edge_at >= 0 ? to_float<T>(row[edge_at]) : 0.0f;
                int32_t first = 0;
                do {
                    if (!all_lanes(mbar_wait<true>(&s_empty[buf], phase ^ 1u, &s_failed))) return false;
                    const int32_t count = min(p.piece, n - first);
                    const bool ok = count > 0 && ZS_RANGE_OK(kSiteLogits, head + (int64_t)(v0 + first) * N, (int64_t)count * N, p.vocab);
                    // the copy first: the row's label and edges may still be on
                    // their way (the barrier's phase ends with the arrival below)
                    if (lane == 0 && ok)
                        copy_bulk(s_buffers + (int64_t)buf * p.piece, row + head + (int64_t)(v0 + first) * N,
                                  (uint32_t)count * 16u, &s_full[buf]);
                    RowInfo& to = s_info[buf];
                    if (lane == 0) {
                        to.row = r;
                        to.head = head;
                        to.v0 = v0;
                        to.n = n;
                        to.y = (int32_t)y;
                        to.y_vec = y >= head ? (int32_t)((y - head) / N) - v0 : -1;
                        to.y_at = y >= head ? (int32_t)((y - head) % N) : 0;
                    }
                    if (lane < 16) {
                        to.edge_at[lane] = edge_at;
                        to.edge[lane] = edge;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_expect(&s_full[buf], ok ? (uint32_t)count * 16u : 0u);
                    advance();
                    first += p.piece;
                } while (first < n);
                return true;
            };
            for (int32_t i = 0; i < n_live; ++i)
                if (!load_row(i) || (MODE == kPolicy && !load_row(i))) break;
            continue;
        }

        if (warp == kStat) {
            // ---- the statistics warp
            for (int32_t i = 0; i < n_live; ++i) {
                const int64_t r = row_at(s_rows.live[i]);
                float x_label = 0.0f, w = 0.0f, adv = 0.0f, old_logp = 0.0f, ref_logp = 0.0f;
                if (STATS) x_label = to_float<T>(((const T*)p.data)[r * p.stride + p.labels[r]]);
                if (POLICY) {
                    w = p.weights != nullptr ? p.weights[r] : p.uniform_weight;
                    adv = p.adv[r];
                    old_logp = p.old_logp[r];
                    if (p.ref_logp != nullptr) ref_logp = p.ref_logp[r];
                }
                GradCoef g = {};
                bool ok;  // (if not: what comes of it is overwritten at the end)
                if constexpr (STATS) {
                    const Stats none{-FLT_MAX, 0.0f, 0.0f, 0.0f};
                    ok = mbar_wait<true>(&s_parts[par], par_phase, &s_failed);
                    Stats st = join_warp<ENT>(lane < kWarps ? s_warp[par][lane] : none, k);
                    if (ctas > 1) {
                        // (every CTA has read the label's logit before any can
                        // write the row's gradient in its place: it is sent)
                        st.x_label = x_label;
                        if (lane == 0) mbar_expect(&s_met[par], 16u * ctas);
                        if (lane < (int)ctas) store_to_peer(&s_peer[par][rank], &s_met[par], (uint32_t)lane, st);
                        ok = mbar_wait<true>(&s_met[par], par_phase, &s_failed) && ok;
                        st = join_warp<ENT>(lane < (int)ctas ? s_peer[par][lane] : none, k);
                    }
                    float logp = -INFINITY, ent = 0.0f, lns = -INFINITY, raw = 0.0f, loss = 0.0f;
                    const bool some = st.s != 0.0f;
                    if (some) {
                        raw = logf(st.s);
                        lns = fmaf(c_residue(st.top, k), kLn2, raw);
                        logp = (x_label - st.top) * p.it - lns;
                        if (ENT) ent = raw - st.u / st.s * kLn2;
                    } else {
                        st.top = -INFINITY;
                    }
                    if (POLICY && some) {
                        const float ratio = expf(logp - old_logp);
                        const float held = fminf(fmaxf(ratio, p.lo), p.hi);
                        // (no advantage, no loss, although the ratio may have passed fp32)
                        const float free_pg = adv == 0.0f ? 0.0f : -adv * ratio, held_pg = -adv * held;
                        bool cut = free_pg < held_pg;
                        float pg = cut ? held_pg : free_pg;
                        if (p.dual > 0.0f && adv < 0.0f && pg > -adv * p.dual) {
                            pg = -adv * p.dual;
                            cut = true;
                        }
                        if (ratio != ratio) pg = ratio;  // a NaN passes through
                        float kl = 0.0f, dlogp = cut ? 0.0f : free_pg;
                        if (p.ref_logp != nullptr) {
                            const float gap = ref_logp - logp, rise = expm1f(gap);
                            kl = rise == INFINITY ? rise : rise - gap;
                            if (p.kl != 0.0f) dlogp -= p.kl * rise;  // (0 times an infinite one has no value)
                        }
                        loss = pg;
                        if (p.kl != 0.0f) loss += p.kl * kl;
                        if (ENT) loss -= p.ent_coef * ent;
                        if (rank == 0 && lane == 0) {
                            sum[0] += (double)w * loss;
                            sum[1] += (double)w * pg;
                            sum[2] += (double)w * kl;
                            sum[3] += (double)w * ent;
                            sum[4] += cut ? (double)w : 0.0;
                        }
                        const float da = scale * w * dlogp, db = ENT ? -scale * w * p.ent_coef : 0.0f;
                        if (GRAD) g = grad_coef<T>(st.top, lns, raw * kLog2e, ENT ? -(da + db * ent) : -da, -db * kLn2, da, k);
                    }
                    if (lane == 0 && rank == 0) {
                        p.logp[r] = logp;
                        if (ENT && p.entropy != nullptr) p.entropy[r] = ent;
                        if (MODE == kLogp && p.saved_out != nullptr) {
                            p.saved_out[2 * r] = st.top;
                            p.saved_out[2 * r + 1] = lns;
                        }
                        if (POLICY && p.token_loss != nullptr) p.token_loss[r] = loss;
                    }
                } else {
                    const float a = scale * p.dlogp[r], b = ENT ? scale * p.dentropy[r] : 0.0f;
                    const float top = p.saved[2 * r], lns = p.saved[2 * r + 1];
                    g = grad_coef<T>(top, lns, fmaf(lns, kLog2e, -c_residue(top, k)),
                                     ENT ? -(a + b * p.row_entropy[r]) : -a, -b * kLn2, a, k);
                    // the coefficients of two rows before have been read
                    ok = mbar_wait<true>(&s_parts[par], par_phase ^ 1u, &s_failed);
                }
                if (lane == 0) {
                    if (GRAD) s_coef[par] = g;
                    mbar_arrive(&s_done[par]);
                }
                if (!all_lanes(ok)) break;
                next_row();
            }
            continue;
        }

        // ---- the computing warps
        // The buffer is free again, if its waits were met; false: the warp stops.  With
        // a gradient the warp agrees on that at every buffer.  Without one it agrees at a
        // row's start and end, in between a lane whose wait ran out works on whatever is
        // there, and the first lane, if it is that one, sets nothing free (scoring 8192 x
        // 50257 bf16: 99.0 us so, 100.0 with every buffer; the policy loss is better with
        // every buffer, 86.3 us for 86.7 in the second case above).
        auto release = [&](bool ok) {
            if (GRAD) {
                if (!all_lanes(ok)) return false;
            } else {
                __syncwarp();
            }
            if (lane == 0 && ok) mbar_arrive(&s_empty[buf]);
            advance();
            return true;
        };
        // first pass over the next row: its parts of the statistics (false: a wait ran out)
        auto first_pass = [&]() {
            bool ok = mbar_wait(&s_full[buf], phase, &s_failed);
            if (!GRAD && !all_lanes(ok)) return false;
            const int32_t n = ok ? s_info[buf].n : 0;
            const int32_t edge_at = tid < 16 ? s_info[buf].edge_at[tid] : -1;
            const float x_edge = tid < 16 ? s_info[buf].edge[tid] : 0.0f;
            Running<T> run = empty_stats<T>();
            for (int32_t first = 0;;) {
                const uint4* v = s_buffers + (int64_t)buf * p.piece;
                const int32_t count = min(p.piece, n - first);
                int32_t q = tid;
                for (; q + (U - 1) * NT < count; q += U * NT) {
                    uint4 x[U];
#pragma unroll
                    for (int g = 0; g < U; ++g) x[g] = v[q + g * NT];
                    add_vectors<T, ENT, U>(run, x, k);
                }
                for (; q < count; q += NT) {
                    const uint4 x[1] = {v[q]};
                    add_vectors<T, ENT, 1>(run, x, k);
                }
                if (!release(ok)) return false;
                first += p.piece;
                if (first >= n) break;
                ok = mbar_wait(&s_full[buf], phase, &s_failed) && (GRAD || ok);
            }
            if (edge_at >= 0) add_value<T, ENT>(run, x_edge, k);
            Stats st{run.top, 0.0f, 0.0f, 0.0f};
            float a, b;
            split(run.s2, a, b);
            st.s = a + b;
            if (ENT) {
                split(run.u2, a, b);
                st.u = a + b;
            }
            st = join_warp<ENT>(st, k);
            // the parts of two rows before have been read
            if (!GRAD && !all_lanes(mbar_wait(&s_done[par], par_phase ^ 1u, &s_failed) && ok)) return false;
            if (lane == 0) {
                s_warp[par][warp] = st;
                mbar_arrive(&s_parts[par]);
            }
            return true;
        };
        // second pass: its gradient
        auto second_pass = [&]() {
            bool ok = mbar_wait(&s_full[buf], phase, &s_failed);
            ok = mbar_wait(&s_done[par], par_phase, &s_failed) && ok;
            if (!all_lanes(ok)) return false;
            const GradCoef c = s_coef[par];
            if (MODE == kLogpGrad) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_parts[par]);
            }
            const RowInfo& f = s_info[buf];
            const int32_t n = f.n, y_vec = f.y_vec, y_at = f.y_at;
            T* row = (T*)p.out + f.row * p.out_stride;
            if (tid < 16 && f.edge_at[tid] >= 0) {
                float x = c.write ? grad_value<ENT>(c, k, f.edge[tid]) : 0.0f;
                if (c.write && f.edge_at[tid] == f.y) x += c.cy;
                row[f.edge_at[tid]] = from_float<T>(x);
            }
            T* out = row + f.head + (int64_t)f.v0 * N;
            const int skip = (int)(((16u - ((uintptr_t)out & 15u)) & 15u) / sizeof(T));
            constexpr bool kCanRaise = sizeof(T) == 2 || !ENT;
            const bool usual = c.write && c.floor != kSlow && !(kCanRaise && ENT && c.floor == kBounded);
            for (int32_t first = 0;;) {
                const uint4* v = s_buffers + (int64_t)buf * p.piece;
                const int32_t count = min(p.piece, n - first);
                T* to = out + (int64_t)first * N;
                auto in_row = [&](int32_t q) { return ZS_RANGE_OK(kSiteDlogits, (to - row) + (int64_t)q * N, N, p.vocab); };
                int32_t q = tid;
                if (skip == 0) {
                    uint4* to16 = reinterpret_cast<uint4*>(to);
                    if (usual) {
                        for (; q + (U - 1) * NT < count; q += U * NT) {
                            uint4 x[U];
#pragma unroll
                            for (int g = 0; g < U; ++g) x[g] = v[q + g * NT];
                            grad_vectors<T, ENT, kCanRaise, U>(c, k, x);
#pragma unroll
                            for (int g = 0; g < U; ++g)
                                if (in_row(q + g * NT)) __stcs(to16 + q + g * NT, x[g]);
                        }
                        for (; q < count; q += NT) {
                            uint4 x[1] = {v[q]};
                            grad_vectors<T, ENT, kCanRaise, 1>(c, k, x);
                            if (in_row(q)) __stcs(to16 + q, x[0]);
                        }
                    } else {
                        for (; q < count; q += NT)
                            if (in_row(q)) __stcs(to16 + q, c.write ? grad_vector<T, ENT>(c, k, v[q]) : make_uint4(0u, 0u, 0u, 0u));
                    }
                } else {
                    for (int32_t base = warp * 32; base < count; base += NT, q += NT) {
                        const bool have = q < count && in_row(q);
                        uint4 x[1] = {make_uint4(0u, 0u, 0u, 0u)};
                        if (have) x[0] = v[q];
                        if (usual)
                            grad_vectors<T, ENT, kCanRaise, 1>(c, k, x);
                        else
                            x[0] = c.write ? grad_vector<T, ENT>(c, k, x[0]) : make_uint4(0u, 0u, 0u, 0u);
                        if (__all_sync(0xffffffffu, have)) {
                            store_shifted<T>(to + (int64_t)q * N, x[0], skip);
                        } else if (have) {
                            const uint32_t w[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
#pragma unroll
                            for (int j = 0; j < N; ++j) {
                                if constexpr (sizeof(T) == 2)
                                    reinterpret_cast<unsigned short*>(to + (int64_t)q * N)[j] = (unsigned short)(w[j / 2] >> (16 * (j % 2)));
                                else
                                    reinterpret_cast<uint32_t*>(to + (int64_t)q * N)[j] = w[j];
                            }
                        }
                    }
                }
                // the label's element, once more with its own term, by the warp
                // that wrote it (after a fence: another lane may have)
                const int32_t y_here = y_vec - first;
                if (y_here >= 0 && y_here < count && (y_here / 32) % kWarps == warp) {
                    __syncwarp();
                    if (lane == 0 && c.write && in_row(y_here)) {
                        const float x = to_float<T>(reinterpret_cast<const T*>(v + y_here)[y_at]);
                        to[(int64_t)y_here * N + y_at] = from_float<T>(grad_value<ENT>(c, k, x) + c.cy);
                    }
                }
                if (!release(ok)) return false;
                first += p.piece;
                if (first >= n) break;
                ok = mbar_wait(&s_full[buf], phase, &s_failed);
            }
            return true;
        };
        // dead rows
        const int32_t n_dead = s_rows.n_dead;
        for (int32_t i = 0; i < n_dead; ++i) {
            const int64_t r = row_at(s_rows.dead[i]);
            if (GRAD) {
                const int64_t a = p.vocab * rank / ctas, b = p.vocab * (rank + 1) / ctas;
                zero_range<T>((T*)p.out + r * p.out_stride + a, b - a, NT);
            }
            if (MODE != kLogpGrad && rank == 0 && tid == 0) {
                p.logp[r] = 0.0f;
                if (ENT && p.entropy != nullptr) p.entropy[r] = 0.0f;
                if (MODE == kLogp && p.saved_out != nullptr) p.saved_out[2 * r] = p.saved_out[2 * r + 1] = 0.0f;
                if (POLICY && p.token_loss != nullptr) p.token_loss[r] = 0.0f;
            }
        }
        // live rows
        for (int32_t i = 0; i < n_live; ++i) {
            if (STATS && !first_pass()) break;
            if (GRAD && !second_pass()) break;
            next_row();
        }
    }
    // the end: no copy in flight, no CTA of the cluster that still writes to this one
    if (warp == kLoad)
        for (int32_t b = 0; b < p.buffers; ++b) drain(&s_full[b], b < buf ? phase : phase ^ 1u);
    bool failed = __syncthreads_or(*(volatile int32_t*)&s_failed) != 0;
    if (ctas > 1) {
        if (failed && tid < (int)ctas) {
            uint32_t a;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(&s_failed)), "r"(tid));
            asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(a), "r"(1) : "memory");
        }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        failed = *(volatile int32_t*)&s_failed != 0;
    }
    if (failed) {
        // (statistics on their way to a CTA that no longer waits for them)
        if (ctas > 1)
            for (int i = 0; i < 100; ++i) __nanosleep(1000);
        fill_with_nan<T, MODE, NT>(p, groups, group_first, group_rows, mine, s_rows);
        sum[0] = sum[1] = sum[2] = sum[3] = sum[4] = NAN;
    }
    if constexpr (POLICY) {
        // partial sums by cluster, then in their order by the last one to arrive
        if (rank != 0) return;
        if (warp == kStat && lane == 0) {
            for (int i = 0; i < ZS_POLICY_TOTALS; ++i) p.work->part[cluster * ZS_POLICY_TOTALS + i] = sum[i];
            __threadfence();
        }
        __syncthreads();
        if (!last_to_arrive(p.work, (uint32_t)clusters)) return;
        for (int i = warp; i < ZS_POLICY_TOTALS; i += kWarps + 2) {
            double t = 0.0;
            for (int32_t b = lane; b < clusters; b += 32) t += *(volatile double*)&p.work->part[b * ZS_POLICY_TOTALS + i];
            t = warp_sum(t);
            if (lane == 0) p.totals[i] = __double2float_rn(t);
        }
    }
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

// Calls go(T{}) with the element type of the logits.
template <typename F>
int32_t with_type(int32_t type, F go) {
    if (type == ZS_F32) return go(float{});
    if (type == ZS_F16) return go(__half{});
    return go(__nv_bfloat16{});
}

// --------------------------------------------------------------- launch plan ---

struct Plan {
    int ctas, piece, buffers;  // CTAs of a cluster; vectors of a buffer; buffers
};

// Bytes of buffers that a CTA may have so that `per_sm` of them share an SM
// (228 KB, 1 KB of it kept back for each, and some KB of other shared memory).
constexpr int buffer_bytes(int per_sm) { return 228 * 1024 / per_sm - 1024 - 5 * 1024 - 512; }
// Vectors (22.5 KB) of a buffer; four buffers.  (1024 vectors and six buffers:
// 725 us for the case above.)
constexpr int kPiece = 1440;
// Bytes of rows that may be under way at once where they are read twice.  (For
// the case above: clusters of two and 40 MB of rows 685 to 689 us, of one and
// 80 MB 887 us, of four and 20 MB 784 us.)
constexpr int64_t kRowsInL2 = 45ll << 20;

// The second pass should find its row in L2 (129 MB, which the gradient passes
// through as well): the cluster is as small as keeps the rows under way within
// kRowsInL2.  Where there are few rows, it grows until they occupy the GPU.
template <int NT>
Plan plan_rows(int64_t rows, int64_t nvec, bool twice) {
    constexpr int kPerSm = per_sm_of(NT);
    const int64_t ctas = (int64_t)kPerSm * zs::device_sm_count();
    auto slice = [&](int c) { return nvec > c ? (int)((nvec + c - 1) / c) : 1; };
    Plan pl{1, 0, kMaxBuffers};
    while (twice && pl.ctas < kMaxCluster && ctas / pl.ctas * nvec * 16 > kRowsInL2) pl.ctas *= 2;
    while (pl.ctas < kMaxCluster && rows * pl.ctas < ctas && slice(pl.ctas) > NT) pl.ctas *= 2;
    pl.piece = slice(pl.ctas) < kPiece ? slice(pl.ctas) : kPiece;
    while (pl.buffers > 2 && pl.buffers * pl.piece * 16 > buffer_bytes(kPerSm)) --pl.buffers;
    return pl;
}

template <typename T, int MODE, bool ENT, int NT>
int32_t launch_rows(RowArgs& a, cudaStream_t stream) {
    auto kernel = rows_kernel<T, MODE, ENT, NT>;
    const Plan pl = plan_rows<NT>(a.rows, a.vocab * (int64_t)sizeof(T) / 16, MODE == kPolicy);
    const int smem = pl.buffers * pl.piece * 16;
    const cudaError_t ready =
        cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, buffer_bytes(1));
    if (ready != cudaSuccess) return zs::cuda_fail(ready, "rows_kernel");
    cudaError_t err = cudaSuccess;
    int64_t clusters = active_clusters((const void*)kernel, NT + 64, pl.ctas, smem, &err);
    if (clusters < 1) return zs::cuda_fail(err, "rows_kernel");
    if (clusters > kWorkParts / ZS_POLICY_TOTALS) clusters = kWorkParts / ZS_POLICY_TOTALS;
    // groups of about 32 clusters, of one size; some clusters may be left out
    int group = 1;
    if (a.rows <= clusters) {
        clusters = a.rows > 0 ? a.rows : 1;
    } else if (clusters >= kMaxGroup) {
        group = 32;
        for (int g = 24; g <= kMaxGroup; ++g)
            if (clusters % g < clusters % group) group = g;
        clusters -= clusters % group;
    } else {
        group = (int)clusters;
    }
    a.piece = pl.piece;
    a.buffers = pl.buffers;
    a.group = group;
    return launch_clusters(kernel, (int)clusters, pl.ctas, NT + 64, smem, stream, a, "rows_kernel");
}

// Blocks of 128 threads, four to an SM, where a row has fewer vectors than 1024:
// more rows are under way and a thread has more of each.  Measured with both, us of
// scoring, its gradient, and the policy loss with its gradient:
//                     128 threads      256 threads
//   8192 x 1000 bf16  20   19   41     31   29   64
//   8192 x 8000 bf16  33   52   65     40   48   85
//   8192 x 24000 bf16 69  136  145     74  134  158
//   600 x 3001 bf16   8.2  8.6 14.4    7.4  8.2 13.3
// (Some hundred rows are better off with 256, by up to a tenth.)
template <typename T, int MODE, bool ENT>
int32_t launch_sized(RowArgs& a, cudaStream_t stream) {
    if (a.vocab * (int64_t)sizeof(T) / 16 < 1024) return launch_rows<T, MODE, ENT, 128>(a, stream);
    return launch_rows<T, MODE, ENT, kWide>(a, stream);
}
template <int MODE>
int32_t launch(const zs_logits* x, RowArgs& a, bool ent, void* stream) {
    a.data = x->data;
    a.rows = x->rows;
    a.vocab = x->vocab;
    a.stride = x->row_stride;
    a.it = (float)x->inv_temperature;
    return with_type(x->type, [&](auto t) {
        using T = decltype(t);
        return ent ? launch_sized<T, MODE, true>(a, (cudaStream_t)stream) : launch_sized<T, MODE, false>(a, (cudaStream_t)stream);
    });
}

}  // namespace

namespace zs {
uint64_t take_fault_logits() { return take_fault(); }
int32_t set_wait_limit(int32_t tries) {
#if ZS_CHECKED
    const cudaError_t err = cudaMemcpyToSymbol(g_wait_limit, &tries, sizeof(tries));
    return err == cudaSuccess ? 1 : cuda_fail(err, "zero_debug_wait_limit");
#else
    (void)tries;
    return 0;
#endif
}
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
    RowArgs a = {};
    a.labels = labels;
    a.logp = logp;
    a.entropy = entropy;
    a.saved_out = saved;
    return launch<kLogp>(x, a, entropy != nullptr, stream);
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
    RowArgs a = {};
    a.out = dlogits;
    a.out_stride = dlogits_stride;
    a.labels = labels;
    a.saved = saved;
    a.dlogp = dlogp;
    a.row_entropy = entropy;
    a.dentropy = dentropy;
    a.ctrl = ctrl_dev;
    return launch<kLogpGrad>(x, a, dentropy != nullptr, stream);
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
    RowArgs a = {};
    a.out = dlogits;
    a.out_stride = dlogits_stride;
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
    const bool ent = entropy != nullptr || hp->entropy_coef != 0.0;
    return dlogits != nullptr ? launch<kPolicy>(x, a, ent, stream) : launch<kPolicyLoss>(x, a, ent, stream);
}

}  // extern "C"
