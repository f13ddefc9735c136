// norm.cu -- layer norm and its gradient.
//
//   xh = (x - mean) rstd,   y = xh gamma + beta,
//   dx = rstd (a - mean(a) - xh mean(a xh)) with a = dy gamma,
//   dgamma = sum_rows dy xh,   dbeta = sum_rows dy.
//
// Rows are read once and written once, so memory bounds the large cases: a row lies in the
// registers of a team of warps between its sums and its output, the rows after it are on their
// way into shared memory, and the gradient keeps its columns' sums over rows in registers.
// Measured on one GB300 (6772 GB/s copied): 16384 x 1600 bf16 24.3 us, 4.3 TB/s, fp32 41.2 us, 5.1
// TB/s; gradient 16384 x 4096 bf16 71 us, 5.7 TB/s, 84 % of the copy rate.  The first issues some 0.6
// instructions a cycle and scheduler, 19 for an element, of which a fourth turn bf16 into fp32
// (three times, since the row is held as it was read; held as fp32 the rows ahead no longer fit
// the registers, 35 us): neither issue nor memory is its limit, but a row's two barriers and
// exchanges, with a third of the warps resident.  Earlier forms of the gradient: next row in
// registers instead of shared memory 87 us; team size at run time 90 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "cluster_counts.h"
#include "zs_internal.h"

namespace {

#include "step_common.cuh"
#include "step_end.cuh"
#include "loss_common.cuh"
#include "elem.cuh"
#include "launch.cuh"

[[maybe_unused]] constexpr uint32_t kSiteNormRow = 18;

constexpr int64_t kMaxWidth = 1 << 24, kMaxGroups = 1024;

struct NormArgs {
    const void *x, *gamma, *beta, *dy;
    const float* saved;
    void *y, *dx, *dgamma, *dbeta;
    float* saved_out;
    float* part;
    int64_t rows, width, x_stride, y_stride, dy_stride, dx_stride;
    float eps, inv_width, float_width;
    int32_t param_type;
};

// ------------------------------------------------------------- parameters ---

// V values of gamma or beta from k on (`missing` without one).
template <typename P, int V>
__device__ __forceinline__ void params_at(const void* p, int64_t k, float missing, float* out) {
    if (p == nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = missing;
    } else {
        unpack<P, V>(*reinterpret_cast<const Pack<P, V>*>((const P*)p + k), out);
    }
}
template <int V>
__device__ __forceinline__ void params_at(const void* p, int32_t type, int64_t k, float missing, float* out) {
    if (type == ZS_F32)
        params_at<float, V>(p, k, missing, out);
    else if (type == ZS_F16)
        params_at<__half, V>(p, k, missing, out);
    else
        params_at<__nv_bfloat16, V>(p, k, missing, out);
}
__device__ __forceinline__ void store_param(void* p, int32_t type, int64_t k, float x) {
    if (type == ZS_F32)
        ((float*)p)[k] = x;
    else if (type == ZS_F16)
        ((__half*)p)[k] = from_float<__half>(x);
    else
        ((__nv_bfloat16*)p)[k] = from_float<__nv_bfloat16>(x);
}

// ------------------------------------------------------------------- teams ---

// A team of 1 to 16 warps takes a row: C vectors of V elements to a thread, held in
// registers as they were read from the first sum to the output, so that a row is read
// once and the variance is of differences from the mean.  A block has threads / (32 warps) teams.
constexpr int kThreads = 256, kMaxThreads = 512;

template <int WARPS> struct Team {
    static constexpr int kTeamThreads = 32 * WARPS;
    static constexpr int kBlock = kTeamThreads > kThreads ? kTeamThreads : kThreads;
    static constexpr int kTeams = kBlock / kTeamThreads;
    int number, thread;  // the team of the block, the thread of the team
    uint32_t turn = 0;   // which of the places is next
    __device__ __forceinline__ Team() : number(threadIdx.x / kTeamThreads), thread(threadIdx.x % kTeamThreads) {}
    __device__ __forceinline__ void barrier() const {
        asm volatile("bar.sync %0, %1;" ::"r"(number + 1), "n"(kTeamThreads) : "memory");
    }
    // The sums over the team, in every thread.  Two places in turn, so that one barrier is
    // enough: who writes a place again has passed the barrier between, which its readers
    // reach after reading.  Every warp adds the warps' sums up anew, in one order.
    __device__ __forceinline__ float sum(float x) {
        __shared__ float s[2][kMaxThreads / 32];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if constexpr (WARPS > 1) {
            const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
            if (lane == 0) s[turn][warp] = x;
            barrier();
            x = s[turn][number * WARPS + lane % WARPS];
            turn ^= 1;
#pragma unroll
            for (int o = WARPS / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        }
        return x;
    }
    // Of two numbers: the warp's halves take one each, for half the exchanges.
    __device__ __forceinline__ float2 sum(float x, float y) {
        __shared__ float s[2][2][kMaxThreads / 32];
        const int lane = threadIdx.x % 32, half = lane / 16;
        float v = (half ? y : x) + __shfl_xor_sync(0xffffffffu, half ? x : y, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if constexpr (WARPS > 1) {
            if (lane % 16 == 0) s[turn][half][threadIdx.x / 32] = v;
            barrier();
            v = s[turn][half][number * WARPS + lane % WARPS];
            turn ^= 1;
#pragma unroll
            for (int o = WARPS / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        }
        const float w = __shfl_xor_sync(0xffffffffu, v, 16);
        return half ? make_float2(w, v) : make_float2(v, w);
    }
};

// The C vectors of a thread as C V / 2 pairs (with V = 1 of two vectors each).
template <typename T, int V, int C>
__device__ __forceinline__ void pairs_of(const Pack<T, V>* x, uint64_t* p) {
    float f[C * V];
#pragma unroll
    for (int c = 0; c < C; ++c) unpack<T, V>(x[c], f + c * V);
#pragma unroll
    for (int i = 0; i < C * V / 2; ++i) p[i] = pair(f[2 * i], f[2 * i + 1]);
}
template <int N>
__device__ __forceinline__ void split_all(const uint64_t* p, float* f) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) split(p[i], f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ float sum_of(uint64_t p) {
    float a, b;
    split(p, a, b);
    return a + b;
}

__device__ __forceinline__ float not_below_0(float x) { return x < 0.0f ? 0.0f : x; }  // (NaN stays)

// --------------------------------------------------------------- rows ahead ---

// A thread's vectors of the rows that its team takes next, copied ahead into shared
// memory: DEPTH rows of EACH 16-byte vectors.  A thread reads only what it copied itself,
// so nothing but its own copies has to be waited for.
template <int EACH, int DEPTH, int THREADS>
struct Ahead {
    static constexpr uint32_t stride = THREADS * 16, row_bytes = EACH * stride;
    uint32_t base, in, out;  // in, out: the rows copied and read next
    __device__ __forceinline__ Ahead(const void* shared) {
        base = in = out = (uint32_t)__cvta_generic_to_shared(shared) + threadIdx.x * 16;
    }
    __device__ __forceinline__ void copy(int i, const void* from) const {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(in + i * stride), "l"(from) : "memory");
    }
    __device__ __forceinline__ uint32_t next(uint32_t at) const {
        return at == base + (DEPTH - 1) * row_bytes ? base : at + row_bytes;
    }
    __device__ __forceinline__ void copied() {
        asm volatile("cp.async.commit_group;" ::: "memory");
        in = next(in);
    }
    // Until all but the last DEPTH - 1 rows have come.
    __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory"); }
    __device__ __forceinline__ uint4 get(int i) const {
        uint4 x;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(out + i * stride) : "memory");
        return x;
    }
    __device__ __forceinline__ void read() { out = next(out); }
};
// Rows ahead: as many as some 64 KB of a block of 256 threads hold.
constexpr int depth_of(int each) { return each >= 8 ? 2 : each >= 4 ? 4 : 6; }
constexpr size_t ahead_bytes(int each, int threads) { return (size_t)depth_of(each) * each * threads * 16; }

template <typename T, typename P, int V, int C, int WARPS>
__global__ void __launch_bounds__(Team<WARPS>::kBlock, 1024 / Team<WARPS>::kBlock) norm_rows_kernel(const __grid_constant__ NormArgs a) {
    constexpr bool kRing = V * sizeof(T) == 16;
    extern __shared__ uint4 s_ahead[];
    Team<WARPS> t;
    constexpr int kTeam = Team<WARPS>::kTeamThreads;
    const int32_t vectors = (int32_t)(a.width / V);
    const int64_t step = (int64_t)gridDim.x * Team<WARPS>::kTeams;
    Ahead<C, depth_of(C), Team<WARPS>::kBlock> ahead(s_ahead);
    int64_t r = (int64_t)blockIdx.x * Team<WARPS>::kTeams + t.number, rc = r;
    bool in[C];
#pragma unroll
    for (int c = 0; c < C; ++c) in[c] = t.thread + c * kTeam < vectors;
    const int64_t x_step = step * a.x_stride, y_step = step * a.y_stride;
    const T* x = (const T*)a.x + r * a.x_stride + t.thread * V;  // of the row to copy (to load) next
    T* y = (T*)a.y + r * a.y_stride + t.thread * V;
    griddep_wait();
    auto copy_row = [&]() {
        if (rc < a.rows) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (in[c]) ahead.copy(c, x + c * kTeam * V);
        }
        ahead.copied();
        rc += step;
        x += x_step;
    };
    if (kRing)
        for (int i = 0; i < depth_of(C) - 1; ++i) copy_row();
    for (; r < a.rows; r += step, y += y_step) {
        Pack<T, V> raw[C];
        if constexpr (kRing) {
            copy_row();
            ahead.wait();
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            raw[c] = Pack<T, V>{};
            if (in[c]) {
                if constexpr (kRing)
                    raw[c].raw = ahead.get(c);
                else
                    raw[c] = *reinterpret_cast<const Pack<T, V>*>(x + c * kTeam * V);
            }
        }
        if constexpr (kRing)
            ahead.read();
        else
            x += x_step;
        uint64_t s[2] = {0, 0};
        constexpr int G = V == 1 ? C : V;  // elements taken together
#pragma unroll
        for (int c = 0; c < C * V / G; ++c) {
            uint64_t part[G / 2];
            pairs_of<T, V, G / V>(raw + c * (G / V), part);
#pragma unroll
            for (int i = 0; i < G / 2; ++i) s[i & 1] = add2(s[i & 1], part[i]);
        }
        // The mean.  In a constant row of 16-bit numbers every sum is exact (11 bits of the number,
        // 13 of their count; rows of more than 8192 come in eights), and so is the quotient.  Sums of
        // fp32 numbers are some units off: there the differences from the first mean are summed as
        // well as their squares, and correct it.  In a constant row the difference d is a few units,
        // both sums, w d and w d^2, and the quotient are exact, and the deviation is 0.  (Correcting
        // 16-bit rows too took 31.4 us for 29.3 at 16384 x 1600; fp32 takes 47 for 43.7.)
        constexpr bool kCorrect = sizeof(T) == 4;
        const float sum = t.sum(sum_of(add2(s[0], s[1])));
        const float near = kCorrect ? __fmul_rn(sum, a.inv_width) : __fdiv_rn(sum, a.float_width);
        const uint64_t n2 = pair(-near, -near);
        uint64_t e = 0;
        s[0] = s[1] = 0;
        if constexpr (V == 1) {
            uint64_t v[C / 2];
            pairs_of<T, V, C>(raw, v);
#pragma unroll
            for (int i = 0; i < C / 2; ++i) {
                const uint64_t d = add2(v[i], pair(in[2 * i] ? -near : 0.0f, in[2 * i + 1] ? -near : 0.0f));
                if (kCorrect) e = add2(e, d);
                s[i & 1] = fma2(d, d, s[i & 1]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (!in[c]) continue;
                uint64_t part[V / 2];
                pairs_of<T, V, 1>(raw + c, part);
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    part[i] = add2(part[i], n2);
                    s[i & 1] = fma2(part[i], part[i], s[i & 1]);
                }
                if (kCorrect) e = add2(e, V == 4 ? add2(part[0], part[V / 2 - 1]) : part[0]);
            }
        }
        float mean = near, squares;
        if constexpr (kCorrect) {
            const float2 sums = t.sum(sum_of(e), sum_of(add2(s[0], s[1])));
            const float off = __fdiv_rn(sums.x, a.float_width);
            mean = __fadd_rn(near, off);
            squares = not_below_0(fmaf(-off, sums.x, sums.y));
        } else {
            squares = t.sum(sum_of(add2(s[0], s[1])));
        }
        const uint64_t m2 = kCorrect ? pair(-mean, -mean) : n2;
        // (the hardware's reciprocal root is off by some 2^-22.9 of itself)
        const float rstd = rsqrtf(fmaf(squares, a.inv_width, a.eps));
        const uint64_t r2 = pair(rstd, rstd);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!in[c]) continue;
            const int32_t k = (t.thread + c * kTeam) * V;
            float f[V], g[V], b[V];
            unpack<T, V>(raw[c], f);
            params_at<P, V>(a.gamma, k, 1.0f, g);
            params_at<P, V>(a.beta, k, 0.0f, b);
            if constexpr (V == 1) {
                f[0] = fmaf((f[0] - mean) * rstd, g[0], b[0]);
            } else {
#pragma unroll
                for (int i = 0; i < V; i += 2)
                    split(fma2(mul2(add2(pair(f[i], f[i + 1]), m2), r2), pair(g[i], g[i + 1]), pair(b[i], b[i + 1])), f[i], f[i + 1]);
            }
            if (ZS_RANGE_OK(kSiteNormRow, k, V, a.width))
                *reinterpret_cast<Pack<T, V>*>(y + c * kTeam * V) = pack<T, V>(f);
        }
        if (t.thread == 0 && a.saved_out != nullptr) {
            a.saved_out[2 * r] = mean;
            a.saved_out[2 * r + 1] = rstd;
        }
    }
}

// The gradient in one pass over dy and x: a team keeps its columns' parts of dgamma and
// dbeta in registers from row to row.  A block's teams add their parts up in shared
// memory, in their order; a block leaves one row of parts.
template <typename T, int V, int C, int WARPS, bool PARAMS>
__global__ void __launch_bounds__(Team<WARPS>::kBlock, 512 / Team<WARPS>::kBlock) norm_grad_kernel(const __grid_constant__ NormArgs a) {
    constexpr bool kRing = V * sizeof(T) == 16;
    constexpr int N = C * V, H = N / 2;
    extern __shared__ uint4 s_ahead[];  // rows ahead; with several teams, [2][width] of parts after them
    float* const s_part = reinterpret_cast<float*>(s_ahead + (kRing ? ahead_bytes(2 * C, Team<WARPS>::kBlock) / 16 : 0));
    Team<WARPS> t;
    constexpr int kTeam = Team<WARPS>::kTeamThreads;
    const int32_t vectors = (int32_t)(a.width / V);
    const int64_t step = (int64_t)gridDim.x * Team<WARPS>::kTeams;
    Ahead<2 * C, depth_of(2 * C), Team<WARPS>::kBlock> ahead(s_ahead);
    int64_t r = (int64_t)blockIdx.x * Team<WARPS>::kTeams + t.number, rc = r;
    bool in[C];
#pragma unroll
    for (int c = 0; c < C; ++c) in[c] = t.thread + c * kTeam < vectors;
    const int64_t x_step = step * a.x_stride, dy_step = step * a.dy_stride, dx_step = step * a.dx_stride;
    const T* px = (const T*)a.x + r * a.x_stride + t.thread * V;
    const T* pd = (const T*)a.dy + r * a.dy_stride + t.thread * V;
    T* dx = (T*)a.dx + r * a.dx_stride + t.thread * V;
    const float* saved = a.saved + 2 * r;
    griddep_wait();
    auto copy_row = [&]() {
        if (rc < a.rows) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (in[c]) {
                    ahead.copy(2 * c, px + c * kTeam * V);
                    ahead.copy(2 * c + 1, pd + c * kTeam * V);
                }
        }
        ahead.copied();
        rc += step;
        px += x_step;
        pd += dy_step;
    };
    if (kRing)
        for (int i = 0; i < depth_of(2 * C) - 1; ++i) copy_row();
    uint64_t g[H], dg[H], db[H];
    {
        float f[N];
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[c * V + i] = 0.0f;
            if (in[c]) params_at<V>(a.gamma, a.param_type, (t.thread + c * kTeam) * V, 1.0f, f + c * V);
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
            g[i] = pair(f[2 * i], f[2 * i + 1]);
            dg[i] = db[i] = 0;
        }
    }
    Pack<T, V> x[C], dy[C];
    float mean = 0.0f, rstd = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = dy[c] = Pack<T, V>{};
    // (without the ring a row's vectors are loaded one row ahead, into registers)
    auto load = [&]() {
        mean = saved[0];
        rstd = saved[1];
        saved += 2 * step;
        if constexpr (!kRing) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (in[c]) {
                    x[c] = *reinterpret_cast<const Pack<T, V>*>(px + c * kTeam * V);
                    dy[c] = *reinterpret_cast<const Pack<T, V>*>(pd + c * kTeam * V);
                }
            px += x_step;
            pd += dy_step;
        }
    };
    if (r < a.rows) load();
    for (; r < a.rows; r += step, dx += dx_step) {
        if constexpr (kRing) {
            copy_row();
            ahead.wait();
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (in[c]) {
                    x[c].raw = ahead.get(2 * c);
                    dy[c].raw = ahead.get(2 * c + 1);
                }
            ahead.read();
        }
        uint64_t xh[H], e[H], s = 0, u = 0;
        const uint64_t r2 = pair(rstd, rstd), m2 = pair(-mean, -mean);
        pairs_of<T, V, C>(x, xh);
        pairs_of<T, V, C>(dy, e);
        // (vectors outside the row have x = 0, dy = 0 and gamma = 0, so xh's value there, -mean rstd,
        // is of no account as long as it is finite)
#pragma unroll
        for (int i = 0; i < H; ++i) {
            xh[i] = mul2(add2(xh[i], m2), r2);
            if (PARAMS) {
                dg[i] = fma2(e[i], xh[i], dg[i]);
                db[i] = add2(db[i], e[i]);
            }
            e[i] = mul2(e[i], g[i]);
            s = add2(s, e[i]);
            u = fma2(e[i], xh[i], u);
        }
        // (it passes fp32 in constant rows of large numbers alone, in others it stays below some
        // 2^24 sqrt(width): all of xh is 0 then.  Masking the vectors instead took 505 us for 277 at
        // 23986 x 2375 bf16.)
        if (fabsf(mean * rstd) > 3.402823466e38f) u = 0;
        if (r + step < a.rows) load();
        if (a.dx == nullptr) continue;
        const float2 sums = t.sum(sum_of(s), sum_of(u));
        const float m = -sums.x * a.inv_width, n = -sums.y * a.inv_width;
        const uint64_t mm = pair(m, m), nn = pair(n, n);
        float f[N];
#pragma unroll
        for (int i = 0; i < H; ++i) split(mul2(fma2(xh[i], nn, add2(e[i], mm)), r2), f[2 * i], f[2 * i + 1]);
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (in[c] && ZS_RANGE_OK(kSiteNormRow, (int64_t)(t.thread + c * kTeam) * V, V, a.width))
                *reinterpret_cast<Pack<T, V>*>(dx + c * kTeam * V) = pack<T, V>(f + c * V);
    }
    if (!PARAMS) return;
    float* const out = a.part + 2 * (int64_t)blockIdx.x * a.width;
    float pg[N], pb[N];
    split_all<N>(dg, pg);
    split_all<N>(db, pb);
    for (int n = 0; n < Team<WARPS>::kTeams; ++n) {
        if (n == t.number) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (!in[c]) continue;
                const int32_t k = (t.thread + c * kTeam) * V;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (n > 0) pg[c * V + i] += s_part[k + i], pb[c * V + i] += s_part[a.width + k + i];
                    if (n + 1 < Team<WARPS>::kTeams) {
                        s_part[k + i] = pg[c * V + i];
                        s_part[a.width + k + i] = pb[c * V + i];
                    }
                }
                if (n + 1 == Team<WARPS>::kTeams) {
                    *reinterpret_cast<Pack<float, V>*>(out + k) = pack<float, V>(pg + c * V);
                    *reinterpret_cast<Pack<float, V>*>(out + a.width + k) = pack<float, V>(pb + c * V);
                }
            }
        }
        if (Team<WARPS>::kTeams > 1) __syncthreads();
    }
}

// Adds up the blocks' parts: 32 columns to a block, 16 threads to a column.
__global__ void __launch_bounds__(512) norm_param_kernel(const __grid_constant__ NormArgs a, int32_t groups) {
    __shared__ float s[2][16][33];
    const int column = threadIdx.x % 32, lane = threadIdx.x / 32;
    const int64_t k = (int64_t)blockIdx.x * 32 + column;
    griddep_wait();
    float g = 0.0f, b = 0.0f;
    if (k < a.width) {
#pragma unroll 4
        for (int32_t q = lane; q < groups; q += 16) {
            g += a.part[2 * (int64_t)q * a.width + k];
            b += a.part[(2 * (int64_t)q + 1) * a.width + k];
        }
    }
    s[0][lane][column] = g;
    s[1][lane][column] = b;
    __syncthreads();
    if (lane > 1 || k >= a.width) return;
    float sum = 0.0f;
    for (int q = 0; q < 16; ++q) sum += s[lane][q][column];
    void* const out = lane == 0 ? a.dgamma : a.dbeta;
    if (out != nullptr) store_param(out, a.param_type, k, sum);
}

// ----------------------------------------------------------------- long rows ---

// Rows that a team's registers do not hold (and forward those with gamma and beta of the
// other 16-bit type, or of a 16-bit type next to fp32 rows) are read once for each sum, from
// L2 after the first: a block to a row.  The mean is corrected as fp32's above; a thread's first
// sum is held in two parts, so that the mean stays within a few units over any width.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads, 3) norm_long_kernel(const __grid_constant__ NormArgs a) {
    Team<kMaxThreads / 32> t;
    griddep_wait();
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = (const T*)a.x + r * a.x_stride;
        T* y = (T*)a.y + r * a.y_stride;
        Sum2 first = {0.0f, 0.0f};
#pragma unroll 4
        for (int64_t k = threadIdx.x; k < a.width; k += kMaxThreads) first.add(to_float(x[k]));
        const float near = __fmul_rn(t.sum(__fadd_rn(first.hi, first.lo)), a.inv_width);
        float e = 0.0f, s = 0.0f;
#pragma unroll 4
        for (int64_t k = threadIdx.x; k < a.width; k += kMaxThreads) {
            const float d = to_float(x[k]) - near;
            e += d;
            s = fmaf(d, d, s);
        }
        const float2 sums = t.sum(e, s);
        const float off = __fdiv_rn(sums.x, a.float_width), mean = __fadd_rn(near, off);
        const float rstd = rsqrtf(fmaf(not_below_0(fmaf(-off, sums.x, sums.y)), a.inv_width, a.eps));
#pragma unroll 4
        for (int64_t k = threadIdx.x; k < a.width; k += kMaxThreads) {
            float g, b;
            params_at<1>(a.gamma, a.param_type, k, 1.0f, &g);
            params_at<1>(a.beta, a.param_type, k, 0.0f, &b);
            y[k] = from_float<T>(fmaf((to_float(x[k]) - mean) * rstd, g, b));
        }
        if (threadIdx.x == 0 && a.saved_out != nullptr) {
            a.saved_out[2 * r] = mean;
            a.saved_out[2 * r + 1] = rstd;
        }
    }
}
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) norm_long_dx_kernel(const __grid_constant__ NormArgs a) {
    Team<kMaxThreads / 32> t;
    griddep_wait();
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *x = (const T*)a.x + r * a.x_stride, *dy = (const T*)a.dy + r * a.dy_stride;
        const float mean = a.saved[2 * r], rstd = a.saved[2 * r + 1];
        float s = 0.0f, u = 0.0f, g;
#pragma unroll 4
        for (int64_t k = threadIdx.x; k < a.width; k += kMaxThreads) {
            params_at<1>(a.gamma, a.param_type, k, 1.0f, &g);
            g *= to_float(dy[k]);
            s += g;
            u = fmaf(g, (to_float(x[k]) - mean) * rstd, u);
        }
        const float2 sums = t.sum(s, u);
        const float m = sums.x * a.inv_width, n = sums.y * a.inv_width;
#pragma unroll 4
        for (int64_t k = threadIdx.x; k < a.width; k += kMaxThreads) {
            params_at<1>(a.gamma, a.param_type, k, 1.0f, &g);
            const float xh = (to_float(x[k]) - mean) * rstd;
            ((T*)a.dx)[r * a.dx_stride + k] = from_float<T>(rstd * (g * to_float(dy[k]) - fmaf(xh, n, m)));
        }
    }
}
// Parts of dgamma and dbeta: a thread to a column, blocks of rows.
template <typename T>
__global__ void __launch_bounds__(256) norm_long_part_kernel(const __grid_constant__ NormArgs a) {
    griddep_wait();
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= a.width) return;
    float g = 0.0f, b = 0.0f;
#pragma unroll 4
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float dy = to_float(((const T*)a.dy)[r * a.dy_stride + k]);
        g = fmaf(dy, (to_float(((const T*)a.x)[r * a.x_stride + k]) - a.saved[2 * r]) * a.saved[2 * r + 1], g);
        b += dy;
    }
    a.part[2 * (int64_t)blockIdx.y * a.width + k] = g;
    a.part[(2 * (int64_t)blockIdx.y + 1) * a.width + k] = b;
}

// ------------------------------------------------------------------ launches ---

int64_t groups_of(int64_t rows) { return rows < kMaxGroups ? (rows > 0 ? rows : 1) : kMaxGroups; }

// How a row is dealt to a team: c vectors of v elements to a thread, `most` at most, with
// as few warps as that takes; warps = 0: the row is too long.
struct Shape {
    int c, warps;
};
constexpr int kElements = 16;  // of a thread, where rows are taken element by element
Shape shape_of(int64_t width, int v, int most) {
    const int64_t vectors = width / v;
    for (int warps = 1; warps <= kMaxThreads / 32; warps *= 2)
        if (vectors <= 32ll * warps * most) return {(int)((vectors + 32 * warps - 1) / (32 * warps)), warps};
    return {0, 0};
}
// Calls f with the number of warps as a constant.
template <typename F>
int32_t with_warps(int warps, F f) {
    switch (warps) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    default: return f(std::integral_constant<int, 16>());
    }
}
// Whether rows of these matrices (row strides in elements) can be accessed as vectors of v
// elements, and the parameters next to them.
template <typename... M>
bool vectors_fit(int v, int64_t width, int64_t size, const void* gamma, const void* beta, M... matrices) {
    const uintptr_t bytes = (uintptr_t)(v * size);
    if (width % v != 0 || !zs::aligned_to(gamma, 16) || !zs::aligned_to(beta, 16)) return false;
    auto fits = [&](const void* p, int64_t stride) { return zs::aligned_to(p, bytes) && stride % v == 0; };
    return (fits(matrices.first, matrices.second) && ...);
}
struct Matrix {
    const void* first;
    int64_t second;
};

template <typename T, typename P, int V, int C, int WARPS>
int32_t launch_rows(const NormArgs& a, cudaStream_t stream) {
    constexpr int threads = Team<WARPS>::kBlock, teams = Team<WARPS>::kTeams;
    constexpr size_t shared = V * sizeof(T) == 16 ? ahead_bytes(C, threads) : 0;
    const auto kernel = norm_rows_kernel<T, P, V, C, WARPS>;
    const unsigned grid = grid_of((const void*)kernel, threads, shared, (a.rows + teams - 1) / teams);
    if (grid == 0) return ZS_ERR_CUDA;
    return launch_shared(kernel, dim3(grid), threads, shared, stream, "norm_rows_kernel", a);
}
template <typename T>
int32_t launch_long(const NormArgs& a, cudaStream_t stream, T) {
    const unsigned grid = grid_of((const void*)norm_long_kernel<T>, kMaxThreads, 0, a.rows);
    if (grid == 0) return ZS_ERR_CUDA;
    return launch(norm_long_kernel<T>, dim3(grid), kMaxThreads, stream, "norm_long_kernel", a);
}
template <typename T, typename P>
int32_t launch_forward(const NormArgs& a, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T), M = 4;
    auto fit = [&](int v) { return vectors_fit(v, a.width, sizeof(T), a.gamma, a.beta, Matrix{a.x, a.x_stride}, Matrix{a.y, a.y_stride}); };
    const bool wide = fit(V);
    const Shape s = shape_of(a.width, wide ? V : 1, wide ? M : kElements);
    if (s.warps == 0) return launch_long(a, stream, T());
    if (!wide)
        return with_warps(s.warps, [&](auto w) {
            // (rows on boundaries of two elements: two to an access)
            if (fit(2)) return launch_rows<T, P, 2, kElements / 2, decltype(w)::value>(a, stream);
            return launch_rows<T, P, 1, kElements, decltype(w)::value>(a, stream);
        });
    if (s.c == 1) return launch_rows<T, P, V, 1, 1>(a, stream);
    if (s.c == 2) return launch_rows<T, P, V, 2, 1>(a, stream);
    return with_warps(s.warps, [&](auto w) { return launch_rows<T, P, V, M, decltype(w)::value>(a, stream); });
}

int32_t launch_params(const NormArgs& a, int64_t groups, cudaStream_t stream) {
    return launch(norm_param_kernel, dim3((unsigned)((a.width + 31) / 32)), 512, stream, "norm_param_kernel", a, (int32_t)groups);
}
template <typename T, int V, int C, int WARPS>
int32_t launch_grad_rows(const NormArgs& a, cudaStream_t stream) {
    const bool params = a.dgamma != nullptr || a.dbeta != nullptr;
    constexpr int threads = Team<WARPS>::kBlock, teams = Team<WARPS>::kTeams;
    const size_t shared = (V * sizeof(T) == 16 ? ahead_bytes(2 * C, threads) : 0) + (params && teams > 1 ? 8 * (size_t)a.width : 0);
    auto go = [&](auto kernel) {
        unsigned grid = grid_of((const void*)kernel, threads, shared, (a.rows + teams - 1) / teams);
        if (grid == 0) return (int32_t)ZS_ERR_CUDA;
        if (grid > kMaxGroups) grid = kMaxGroups;
        const int32_t rc = launch_shared(kernel, dim3(grid), threads, shared, stream, "norm_grad_kernel", a);
        return rc != ZS_OK || !params ? rc : launch_params(a, grid, stream);
    };
    return params ? go(norm_grad_kernel<T, V, C, WARPS, true>) : go(norm_grad_kernel<T, V, C, WARPS, false>);
}
template <typename T>
int32_t launch_grad(const NormArgs& a, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T), M = 16 / V;
    const bool params = a.dgamma != nullptr || a.dbeta != nullptr;
    auto fit = [&](int v) {
        return vectors_fit(v, a.width, sizeof(T), a.gamma, nullptr, Matrix{a.x, a.x_stride}, Matrix{a.dy, a.dy_stride},
                           Matrix{a.dx, a.dx_stride});
    };
    const bool wide = fit(V);
    const Shape s = shape_of(a.width, wide ? V : 1, wide ? M : kElements);
    if (s.warps == 0) {
        if (params) {
            // (before dx, which may take dy's or x's place)
            const int64_t groups = a.rows < 64 ? groups_of(a.rows) : 64;
            ZS_TRY(launch(norm_long_part_kernel<T>, dim3((unsigned)((a.width + 255) / 256), (unsigned)groups), 256, stream,
                          "norm_long_part_kernel", a));
            ZS_TRY(launch_params(a, groups, stream));
        }
        if (a.dx == nullptr) return ZS_OK;
        const unsigned grid = grid_of((const void*)norm_long_dx_kernel<T>, kMaxThreads, 0, a.rows);
        if (grid == 0) return ZS_ERR_CUDA;
        return launch(norm_long_dx_kernel<T>, dim3(grid), kMaxThreads, stream, "norm_long_dx_kernel", a);
    }
    if (!wide)
        return with_warps(s.warps, [&](auto w) {
            if (fit(2)) return launch_grad_rows<T, 2, kElements / 2, decltype(w)::value>(a, stream);
            return launch_grad_rows<T, 1, kElements, decltype(w)::value>(a, stream);
        });
    if (s.c == 1) return launch_grad_rows<T, V, 1, 1>(a, stream);
    return with_warps(s.warps, [&](auto w) { return launch_grad_rows<T, V, M, decltype(w)::value>(a, stream); });
}

bool valid_sizes(int64_t rows, int64_t width) {
    return rows >= 0 && rows <= 0x7fffffffll && width >= 1 && width <= kMaxWidth;
}
bool valid_type(int32_t t) { return t == ZS_F32 || t == ZS_F16 || t == ZS_BF16; }
bool valid_stride(int64_t rows, int64_t width, int64_t stride) {
    return rows <= 1 || (stride >= width && stride <= 1ll << 40);
}

int32_t check_norm(const zs_norm* n) {
    if (n == nullptr || !valid_sizes(n->rows, n->width) || !valid_type(n->type) || !valid_type(n->param_type) ||
        !(n->eps >= 0.0 && n->eps <= 1e30) || (n->rows > 0 && n->x == nullptr) || !valid_stride(n->rows, n->width, n->x_stride))
        return ZS_ERR_ARG;
    const uintptr_t e = (uintptr_t)elem_size(n->type), p = (uintptr_t)elem_size(n->param_type);
    if (!zs::aligned_to(n->x, e) || !zs::aligned_to(n->gamma, p) || !zs::aligned_to(n->beta, p)) return ZS_ERR_ALIGN;
    return ZS_OK;
}
NormArgs args_of(const zs_norm* n) {
    NormArgs a = {};
    a.x = n->x;
    a.gamma = n->gamma;
    a.beta = n->beta;
    a.param_type = n->param_type;
    a.rows = n->rows;
    a.width = n->width;
    a.x_stride = n->rows > 1 ? n->x_stride : n->width;
    a.eps = (float)n->eps;
    a.inv_width = (float)(1.0 / (double)n->width);
    a.float_width = (float)n->width;  // (exact: up to 2^24)
    return a;
}

}  // namespace

namespace zs {
uint64_t take_fault_norm() { return take_fault(); }
}  // namespace zs

extern "C" {

ZS_API int32_t zero_layer_norm_async(const zs_norm* n, void* y, int64_t y_stride, float* saved, void* stream) {
    zs::NvtxRange nvtx_range("zero_layer_norm_async");
    ZS_TRY(check_norm(n));
    if (n->rows == 0) return ZS_OK;
    if (y == nullptr || !valid_stride(n->rows, n->width, y_stride)) return ZS_ERR_ARG;
    if (!zs::aligned_to(y, (uintptr_t)elem_size(n->type)) || !zs::aligned_to(saved, 4)) return ZS_ERR_ALIGN;
    NormArgs a = args_of(n);
    a.y = y;
    a.y_stride = n->rows > 1 ? y_stride : n->width;
    a.saved_out = saved;
    return with_elem(n->type, [&](auto t) {
        using T = decltype(t);
        return n->param_type == n->type ? launch_forward<T, T>(a, (cudaStream_t)stream)
               : n->param_type == ZS_F32 ? launch_forward<T, float>(a, (cudaStream_t)stream)
                                         : launch_long(a, (cudaStream_t)stream, t);
    });
}

ZS_API int64_t zero_layer_norm_work_bytes(int64_t rows, int64_t width) {
    if (!valid_sizes(rows, width)) return ZS_ERR_ARG;
    return 8 * groups_of(rows) * ((width + 3) / 4 * 4);
}

ZS_API int32_t zero_layer_norm_grad_async(const zs_norm* n, const void* dy, int64_t dy_stride, const float* saved,
                                          void* dx, int64_t dx_stride, void* dgamma, void* dbeta, void* work_dev,
                                          int64_t work_bytes, void* stream) {
    zs::NvtxRange nvtx_range("zero_layer_norm_grad_async");
    ZS_TRY(check_norm(n));
    const bool params = dgamma != nullptr || dbeta != nullptr;
    if (!params && dx == nullptr) return ZS_ERR_ARG;
    if (n->rows > 0 && (dy == nullptr || saved == nullptr)) return ZS_ERR_ARG;
    if (!valid_stride(n->rows, n->width, dy_stride) || (dx != nullptr && !valid_stride(n->rows, n->width, dx_stride)))
        return ZS_ERR_ARG;
    if (params && (work_dev == nullptr || work_bytes < zero_layer_norm_work_bytes(n->rows, n->width))) return ZS_ERR_ARG;
    const uintptr_t e = (uintptr_t)elem_size(n->type), q = (uintptr_t)elem_size(n->param_type);
    if (!zs::aligned_to(dy, e) || !zs::aligned_to(dx, e) || !zs::aligned_to(saved, 4) || !zs::aligned_to(dgamma, q) ||
        !zs::aligned_to(dbeta, q) || !zs::aligned_to(work_dev, 16))
        return ZS_ERR_ALIGN;
    if (n->rows == 0 && !params) return ZS_OK;
    NormArgs a = args_of(n);
    a.dy = dy;
    a.dy_stride = n->rows > 1 ? dy_stride : n->width;
    a.saved = saved;
    a.dx = dx;
    a.dx_stride = n->rows > 1 ? dx_stride : n->width;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.part = (float*)work_dev;
    return with_elem(n->type, [&](auto t) { return launch_grad<decltype(t)>(a, (cudaStream_t)stream); });
}

}  // extern "C"
