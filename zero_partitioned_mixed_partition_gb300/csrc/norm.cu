// norm.cu -- layer norm and its gradient.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "cluster_counts.h"
#include "zs_internal.h"

namespace {

#include "step_common.cuh"
#include "step_end.cuh"
#include "elem.cuh"
#include "packed.cuh"
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
    float eps, inv_width;
    int32_t param_type;
};

// ------------------------------------------------------------- parameters ---

// V values of gamma or beta from k on (`missing` without one).  Their type is a run-time
// choice: one branch, the same for all threads, for a load from L1.
template <int V>
__device__ __forceinline__ void params_at(const void* p, int32_t type, int64_t k, float missing, float* out) {
    if (p == nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = missing;
    } else if (type == ZS_F32) {
        constexpr int N = V < 4 ? V : 4;
#pragma unroll
        for (int i = 0; i < V; i += N)
            unpack<float, N>(*reinterpret_cast<const Pack<float, N>*>((const float*)p + k + i), out + i);
    } else if (type == ZS_F16) {
        unpack<__half, V>(*reinterpret_cast<const Pack<__half, V>*>((const __half*)p + k), out);
    } else {
        unpack<__nv_bfloat16, V>(*reinterpret_cast<const Pack<__nv_bfloat16, V>*>((const __nv_bfloat16*)p + k), out);
    }
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

struct Team {
    int warps, number, teams, thread, threads;  // thread: of the team
};
__device__ __forceinline__ Team team_of(int warps) {
    Team t;
    t.warps = warps;
    t.threads = 32 * warps;
    t.number = threadIdx.x / t.threads;
    t.teams = blockDim.x / t.threads;
    t.thread = threadIdx.x % t.threads;
    return t;
}
// The sums of x and y over the team, in every thread.  `turn` numbers the team's
// calls: two places in turn, so that one barrier is enough (who writes a place again has
// passed the barrier between, which its readers reach after reading).
__device__ __forceinline__ float2 team_sum(const Team& t, uint32_t turn, float x, float y) {
    __shared__ float2 s[2][kMaxThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        y += __shfl_xor_sync(0xffffffffu, y, o);
    }
    if (t.warps == 1) return make_float2(x, y);
    float2* const place = s[turn & 1] + t.number * t.warps;
    if (t.thread % 32 == 0) place[t.thread / 32] = make_float2(x, y);
    asm volatile("bar.sync %0, %1;" ::"r"(t.number + 1), "r"(t.threads) : "memory");
    x = y = 0.0f;
    for (int w = 0; w < t.warps; ++w) {
        x += place[w].x;
        y += place[w].y;
    }
    return make_float2(x, y);
}

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
// For elements one by one: a value for those of the thread's that are in the row, 0 for
// the others.
template <int C>
__device__ __forceinline__ void where_in(const Team& t, int32_t width, float value, uint64_t* p) {
#pragma unroll
    for (int i = 0; i < C / 2; ++i)
        p[i] = pair(t.thread + 2 * i * t.threads < width ? value : 0.0f, t.thread + (2 * i + 1) * t.threads < width ? value : 0.0f);
}
__device__ __forceinline__ float sum_of(uint64_t p) {
    float a, b;
    split(p, a, b);
    return a + b;
}

// --------------------------------------------------------------- rows ahead ---

// A thread's vectors of the rows that its team takes next, copied ahead into shared
// memory: `DEPTH` rows of `EACH` 16-byte vectors.  A thread reads only what it copied
// itself, so nothing but its own copies has to be waited for.
template <int EACH, int DEPTH>
struct Ahead {
    uint32_t base, stride;  // of the thread's first vector; from one vector to the next
    __device__ __forceinline__ Ahead(const void* shared) {
        stride = blockDim.x * 16;
        base = (uint32_t)__cvta_generic_to_shared(shared) + threadIdx.x * 16;
    }
    __device__ __forceinline__ uint32_t at(uint32_t row, int i) const { return base + ((row % DEPTH) * EACH + i) * stride; }
    __device__ __forceinline__ void copy(uint32_t row, int i, const void* from) const {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at(row, i)), "l"(from) : "memory");
    }
    __device__ __forceinline__ void done_row() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // Until all but the last DEPTH - 1 rows have come.
    __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory"); }
    template <typename P>
    __device__ __forceinline__ P get(uint32_t row, int i) const {
        uint4 x;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at(row, i)) : "memory");
        return *reinterpret_cast<P*>(&x);
    }
};
// Rows ahead: as many as some 64 KB of a block of 256 threads hold.
constexpr int depth_of(int each) { return each >= 8 ? 2 : each >= 4 ? 4 : 6; }
constexpr size_t ahead_bytes(int each, int threads) { return (size_t)depth_of(each) * each * threads * 16; }

template <typename T, int V, int C>
__global__ void __launch_bounds__(kMaxThreads, 2) norm_rows_kernel(const __grid_constant__ NormArgs a, int32_t warps) {
    constexpr bool kRing = V * sizeof(T) == 16;
    constexpr int D = depth_of(C);
    extern __shared__ uint4 s_ahead[];
    const Team t = team_of(warps);
    const int32_t vectors = (int32_t)(a.width / V);
    const int64_t step = (int64_t)gridDim.x * t.teams;
    const Ahead<C, D> ahead(s_ahead);
    int64_t r = (int64_t)blockIdx.x * t.teams + t.number, rc = r;
    uint32_t turn = 0, row = 0, row_copied = 0;
    griddep_wait();
    auto copy_row = [&]() {
        if (rc < a.rows) {
            const Pack<T, V>* x = reinterpret_cast<const Pack<T, V>*>((const T*)a.x + rc * a.x_stride);
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (t.thread + c * t.threads < vectors) ahead.copy(row_copied, c, x + t.thread + c * t.threads);
        }
        ahead.done_row();
        rc += step;
        ++row_copied;
    };
    if (kRing)
        for (int i = 0; i < D - 1; ++i) copy_row();
    for (; r < a.rows; r += step, ++row) {
        Pack<T, V>* y = reinterpret_cast<Pack<T, V>*>((T*)a.y + r * a.y_stride);
        Pack<T, V> raw[C];
        if constexpr (kRing) {
            copy_row();
            ahead.wait();
        }
        const Pack<T, V>* x = reinterpret_cast<const Pack<T, V>*>((const T*)a.x + r * a.x_stride);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            raw[c] = Pack<T, V>{};
            if (t.thread + c * t.threads < vectors) {
                if constexpr (kRing)
                    raw[c] = ahead.template get<Pack<T, V>>(row, c);
                else
                    raw[c] = x[t.thread + c * t.threads];
            }
        }
        uint64_t s[2] = {0, 0};
        constexpr int G = V == 1 ? C : V;  // elements taken together
#pragma unroll
        for (int c = 0; c < C * V / G; ++c) {
            uint64_t part[G / 2];
            pairs_of<T, V, G / V>(raw + c * (G / V), part);
#pragma unroll
            for (int i = 0; i < G / 2; ++i) s[i & 1] = add2(s[i & 1], part[i]);
        }
        const float mean = team_sum(t, turn++, sum_of(add2(s[0], s[1])), 0.0f).x * a.inv_width;
        const uint64_t m2 = pair(-mean, -mean);
        s[0] = s[1] = 0;
        if constexpr (V == 1) {
            uint64_t minus[C / 2], v[C / 2];
            where_in<C>(t, vectors, -mean, minus);
            pairs_of<T, V, C>(raw, v);
#pragma unroll
            for (int i = 0; i < C / 2; ++i) {
                const uint64_t d = add2(v[i], minus[i]);
                s[i & 1] = fma2(d, d, s[i & 1]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (t.thread + c * t.threads >= vectors) break;
                uint64_t part[V / 2];
                pairs_of<T, V, 1>(raw + c, part);
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const uint64_t d = add2(part[i], m2);
                    s[i & 1] = fma2(d, d, s[i & 1]);
                }
            }
        }
        const float rstd = 1.0f / sqrtf(team_sum(t, turn++, sum_of(add2(s[0], s[1])), 0.0f).x * a.inv_width + a.eps);
        const uint64_t r2 = pair(rstd, rstd);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int32_t q = t.thread + c * t.threads;
            if (q >= vectors) break;
            float f[V], g[V], b[V];
            unpack<T, V>(raw[c], f);
            params_at<V>(a.gamma, a.param_type, (int64_t)q * V, 1.0f, g);
            params_at<V>(a.beta, a.param_type, (int64_t)q * V, 0.0f, b);
            if constexpr (V == 1) {
                f[0] = fmaf((f[0] - mean) * rstd, g[0], b[0]);
            } else {
#pragma unroll
                for (int i = 0; i < V; i += 2)
                    split(fma2(mul2(add2(pair(f[i], f[i + 1]), m2), r2), pair(g[i], g[i + 1]), pair(b[i], b[i + 1])), f[i], f[i + 1]);
            }
            if (ZS_RANGE_OK(kSiteNormRow, (int64_t)q * V, V, a.width)) y[q] = pack<T, V>(f);
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
template <typename T, int V, int C, bool PARAMS>
__global__ void __launch_bounds__(kMaxThreads) norm_grad_kernel(const __grid_constant__ NormArgs a, int32_t warps) {
    constexpr bool kRing = V * sizeof(T) == 16;
    constexpr int N = C * V, H = N / 2, D = depth_of(2 * C);
    extern __shared__ uint4 s_ahead[];  // rows ahead; with several teams, [2][width] of parts after them
    float* const s_part = reinterpret_cast<float*>(s_ahead + (kRing ? ahead_bytes(2 * C, blockDim.x) / 16 : 0));
    const Team t = team_of(warps);
    const int32_t vectors = (int32_t)(a.width / V);
    const int64_t step = (int64_t)gridDim.x * t.teams;
    const Ahead<2 * C, D> ahead(s_ahead);
    int64_t r = (int64_t)blockIdx.x * t.teams + t.number, rc = r;
    uint32_t turn = 0, row = 0, row_copied = 0;
    griddep_wait();
    auto copy_row = [&]() {
        if (rc < a.rows) {
            const Pack<T, V>* px = reinterpret_cast<const Pack<T, V>*>((const T*)a.x + rc * a.x_stride);
            const Pack<T, V>* pd = reinterpret_cast<const Pack<T, V>*>((const T*)a.dy + rc * a.dy_stride);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int32_t q = t.thread + c * t.threads;
                if (q < vectors) {
                    ahead.copy(row_copied, 2 * c, px + q);
                    ahead.copy(row_copied, 2 * c + 1, pd + q);
                }
            }
        }
        ahead.done_row();
        rc += step;
        ++row_copied;
    };
    if (kRing)
        for (int i = 0; i < D - 1; ++i) copy_row();
    uint64_t g[H], dg[H], db[H];
    {
        float f[N];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int32_t q = t.thread + c * t.threads;
#pragma unroll
            for (int i = 0; i < V; ++i) f[c * V + i] = 0.0f;
            if (q < vectors) params_at<V>(a.gamma, a.param_type, (int64_t)q * V, 1.0f, f + c * V);
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
    auto load = [&](int64_t i) {
        mean = a.saved[2 * i];
        rstd = a.saved[2 * i + 1];
        if constexpr (!kRing) {
            const Pack<T, V>* px = reinterpret_cast<const Pack<T, V>*>((const T*)a.x + i * a.x_stride);
            const Pack<T, V>* pd = reinterpret_cast<const Pack<T, V>*>((const T*)a.dy + i * a.dy_stride);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int32_t q = t.thread + c * t.threads;
                if (q < vectors) {
                    x[c] = px[q];
                    dy[c] = pd[q];
                }
            }
        }
    };
    if (r < a.rows) load(r);
    for (; r < a.rows; r += step, ++row) {
        if constexpr (kRing) {
            copy_row();
            ahead.wait();
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (t.thread + c * t.threads < vectors) {
                    x[c] = ahead.template get<Pack<T, V>>(row, 2 * c);
                    dy[c] = ahead.template get<Pack<T, V>>(row, 2 * c + 1);
                }
        }
        uint64_t xh[H], e[H], s = 0, u = 0;
        const uint64_t r2 = pair(rstd, rstd), m2 = pair(-mean, -mean);
        pairs_of<T, V, C>(x, xh);
        pairs_of<T, V, C>(dy, e);
        // (vectors outside the row have dy = 0 and gamma = 0, so xh's value there is of no
        // account as long as it is finite, and it is wherever the row's is)
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
        if (r + step < a.rows) load(r + step);
        if (a.dx == nullptr) continue;
        const float2 sums = team_sum(t, turn++, sum_of(s), sum_of(u));
        const float m = -sums.x * a.inv_width, n = -sums.y * a.inv_width;
        const uint64_t mm = pair(m, m), nn = pair(n, n);
        Pack<T, V>* dx = reinterpret_cast<Pack<T, V>*>((T*)a.dx + r * a.dx_stride);
        float f[N];
#pragma unroll
        for (int i = 0; i < H; ++i) split(mul2(fma2(xh[i], nn, add2(e[i], mm)), r2), f[2 * i], f[2 * i + 1]);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int32_t q = t.thread + c * t.threads;
            if (q < vectors && ZS_RANGE_OK(kSiteNormRow, (int64_t)q * V, V, a.width)) dx[q] = pack<T, V>(f + c * V);
        }
    }
    if (!PARAMS) return;
    float* const out = a.part + 2 * (int64_t)blockIdx.x * a.width;
    float pg[N], pb[N];
    split_all<N>(dg, pg);
    split_all<N>(db, pb);
    for (int n = 0; n < t.teams; ++n) {
        if (n == t.number) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int32_t q = t.thread + c * t.threads;
                if (q >= vectors) break;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int32_t k = q * V + i;
                    float p = pg[c * V + i], b = pb[c * V + i];
                    if (n > 0) p += s_part[k], b += s_part[a.width + k];
                    if (n + 1 < t.teams) {
                        s_part[k] = p;
                        s_part[a.width + k] = b;
                    } else {
                        out[k] = p;
                        out[a.width + k] = b;
                    }
                }
            }
        }
        if (t.teams > 1) __syncthreads();
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

// Rows that a team's registers do not hold are read once for each sum, from L2 after
// the first: a block to a row.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) norm_long_kernel(const __grid_constant__ NormArgs a) {
    const Team t = team_of(kMaxThreads / 32);
    uint32_t turn = 0;
    griddep_wait();
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = (const T*)a.x + r * a.x_stride;
        T* y = (T*)a.y + r * a.y_stride;
        float s = 0.0f;
#pragma unroll 4
        for (int64_t k = threadIdx.x; k < a.width; k += kMaxThreads) s += to_float(x[k]);
        const float mean = team_sum(t, turn++, s, 0.0f).x * a.inv_width;
        s = 0.0f;
#pragma unroll 4
        for (int64_t k = threadIdx.x; k < a.width; k += kMaxThreads) {
            const float d = to_float(x[k]) - mean;
            s = fmaf(d, d, s);
        }
        const float rstd = 1.0f / sqrtf(team_sum(t, turn++, s, 0.0f).x * a.inv_width + a.eps);
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
    const Team t = team_of(kMaxThreads / 32);
    uint32_t turn = 0;
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
        const float2 sums = team_sum(t, turn++, s, u);
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

// How a row is dealt to a team: V elements to a vector, C vectors to a thread.  c = 0: the
// row is too long.
struct Shape {
    int v, c, warps;
};
Shape shape_of(int64_t width, int v, int most) {
    const int64_t vectors = width / v;
    const int per_thread = v == 1 ? 16 : most / v;
    for (int warps = 1; warps <= kMaxThreads / 32; warps *= 2) {
        if (vectors > 32ll * warps * per_thread) continue;
        const int c = (int)((vectors + 32 * warps - 1) / (32 * warps));
        return {v, v == 1 ? (c <= 4 ? 4 : 16) : c, warps};
    }
    return {v, 0, kMaxThreads / 32};
}
// Whether rows of these matrices (row strides in elements) and the parameters can be
// accessed as 16-byte vectors.
template <typename... M>
bool vectors_fit(int64_t width, int64_t size, const void* gamma, const void* beta, M... matrices) {
    const int64_t v = 16 / size;
    if (width % v != 0 || !zs::aligned_to(gamma, 16) || !zs::aligned_to(beta, 16)) return false;
    auto fits = [&](const void* p, int64_t stride) { return zs::aligned_to(p, 16) && stride % v == 0; };
    return (fits(matrices.first, matrices.second) && ...);
}
struct Matrix {
    const void* first;
    int64_t second;
};

template <typename T, int V, int C>
int32_t launch_rows(const NormArgs& a, int warps, cudaStream_t stream) {
    const int threads = warps > kThreads / 32 ? 32 * warps : kThreads, teams = threads / (32 * warps);
    const size_t shared = V * sizeof(T) == 16 ? ahead_bytes(C, threads) : 0;
    const unsigned grid = grid_of((const void*)norm_rows_kernel<T, V, C>, threads, shared, (a.rows + teams - 1) / teams);
    if (grid == 0) return ZS_ERR_CUDA;
    return launch_shared(norm_rows_kernel<T, V, C>, dim3(grid), threads, shared, stream, "norm_rows_kernel", a, warps);
}
template <typename T>
int32_t launch_forward(const NormArgs& a, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const bool wide = vectors_fit(a.width, sizeof(T), a.gamma, a.beta, Matrix{a.x, a.x_stride}, Matrix{a.y, a.y_stride});
    const Shape s = shape_of(a.width, wide ? V : 1, 4 * V);
    if (s.c == 0) {
        const unsigned grid = grid_of((const void*)norm_long_kernel<T>, kMaxThreads, 0, a.rows);
        if (grid == 0) return ZS_ERR_CUDA;
        return launch(norm_long_kernel<T>, dim3(grid), kMaxThreads, stream, "norm_long_kernel", a);
    }
    if (!wide) return s.c == 4 ? launch_rows<T, 1, 4>(a, s.warps, stream) : launch_rows<T, 1, 16>(a, s.warps, stream);
    if (s.c == 1) return launch_rows<T, V, 1>(a, s.warps, stream);
    return s.c == 2 ? launch_rows<T, V, 2>(a, s.warps, stream) : launch_rows<T, V, 4>(a, s.warps, stream);
}

int32_t launch_params(const NormArgs& a, int64_t groups, cudaStream_t stream) {
    return launch(norm_param_kernel, dim3((unsigned)((a.width + 31) / 32)), 512, stream, "norm_param_kernel", a, (int32_t)groups);
}
template <typename T, int V, int C>
int32_t launch_grad_rows(const NormArgs& a, int warps, cudaStream_t stream) {
    const bool params = a.dgamma != nullptr || a.dbeta != nullptr;
    const int threads = warps > kThreads / 32 ? 32 * warps : kThreads, teams = threads / (32 * warps);
    const size_t shared = (V * sizeof(T) == 16 ? ahead_bytes(2 * C, threads) : 0) + (params && teams > 1 ? 8 * (size_t)a.width : 0);
    auto go = [&](auto kernel) {
        unsigned grid = grid_of((const void*)kernel, threads, shared, (a.rows + teams - 1) / teams);
        if (grid == 0) return (int32_t)ZS_ERR_CUDA;
        if (grid > kMaxGroups) grid = kMaxGroups;
        const int32_t rc = launch_shared(kernel, dim3(grid), threads, shared, stream, "norm_grad_kernel", a, warps);
        return rc != ZS_OK || !params ? rc : launch_params(a, grid, stream);
    };
    return params ? go(norm_grad_kernel<T, V, C, true>) : go(norm_grad_kernel<T, V, C, false>);
}
template <typename T>
int32_t launch_grad(const NormArgs& a, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const bool params = a.dgamma != nullptr || a.dbeta != nullptr;
    const bool wide = vectors_fit(a.width, sizeof(T), a.gamma, nullptr, Matrix{a.x, a.x_stride}, Matrix{a.dy, a.dy_stride},
                                  Matrix{a.dx, a.dx_stride});
    const Shape s = shape_of(a.width, wide ? V : 1, 16);
    if (s.c == 0) {
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
    if (!wide) return s.c == 4 ? launch_grad_rows<T, 1, 4>(a, s.warps, stream) : launch_grad_rows<T, 1, 16>(a, s.warps, stream);
    if (s.c == 1) return launch_grad_rows<T, V, 1>(a, s.warps, stream);
    if (V == 8 || s.c == 2) return launch_grad_rows<T, V, 2>(a, s.warps, stream);
    return launch_grad_rows<T, V, 16 / V>(a, s.warps, stream);
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
    return with_elem(n->type, [&](auto t) { return launch_forward<decltype(t)>(a, (cudaStream_t)stream); });
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
