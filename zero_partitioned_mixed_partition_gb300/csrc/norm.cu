// norm.cu -- layer norm and its gradient.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "zs_internal.h"

namespace {

#include "step_common.cuh"
#include "step_end.cuh"
#include "elem.cuh"
#include "launch.cuh"

constexpr int64_t kMaxWidth = 1 << 24, kMaxGroups = 1024;

struct NormArgs {
    const void *x, *gamma, *beta, *dy;
    const float* saved;
    void *y, *dx, *dgamma, *dbeta;
    float* saved_out;
    float* part;
    int64_t rows, width, x_stride, y_stride, dy_stride, dx_stride;
    float eps, inv_width;
};

// Sum over the block, in every thread.
__device__ float block_sum(float x) {
    __shared__ float s[32];
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = x;
    __syncthreads();
    float t = 0.0f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) t += s[w];
    return t;
}

template <typename T, typename P>
__global__ void __launch_bounds__(256) norm_kernel(const __grid_constant__ NormArgs a) {
    griddep_wait();
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = (const T*)a.x + r * a.x_stride;
        T* y = (T*)a.y + r * a.y_stride;
        float s = 0.0f;
        for (int64_t k = threadIdx.x; k < a.width; k += blockDim.x) s += to_float(x[k]);
        const float mean = block_sum(s) * a.inv_width;
        s = 0.0f;
        for (int64_t k = threadIdx.x; k < a.width; k += blockDim.x) {
            const float d = to_float(x[k]) - mean;
            s = fmaf(d, d, s);
        }
        const float rstd = 1.0f / sqrtf(block_sum(s) * a.inv_width + a.eps);
        for (int64_t k = threadIdx.x; k < a.width; k += blockDim.x) {
            const float g = a.gamma != nullptr ? to_float(((const P*)a.gamma)[k]) : 1.0f;
            const float b = a.beta != nullptr ? to_float(((const P*)a.beta)[k]) : 0.0f;
            y[k] = from_float<T>(fmaf((to_float(x[k]) - mean) * rstd, g, b));
        }
        if (threadIdx.x == 0 && a.saved_out != nullptr) {
            a.saved_out[2 * r] = mean;
            a.saved_out[2 * r + 1] = rstd;
        }
    }
}

template <typename T, typename P>
__global__ void __launch_bounds__(256) norm_dx_kernel(const __grid_constant__ NormArgs a) {
    griddep_wait();
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *x = (const T*)a.x + r * a.x_stride, *dy = (const T*)a.dy + r * a.dy_stride;
        const float mean = a.saved[2 * r], rstd = a.saved[2 * r + 1];
        float s = 0.0f, t = 0.0f;
        for (int64_t k = threadIdx.x; k < a.width; k += blockDim.x) {
            const float g = to_float(dy[k]) * (a.gamma != nullptr ? to_float(((const P*)a.gamma)[k]) : 1.0f);
            s += g;
            t = fmaf(g, (to_float(x[k]) - mean) * rstd, t);
        }
        s = block_sum(s) * a.inv_width;
        t = block_sum(t) * a.inv_width;
        for (int64_t k = threadIdx.x; k < a.width; k += blockDim.x) {
            const float g = to_float(dy[k]) * (a.gamma != nullptr ? to_float(((const P*)a.gamma)[k]) : 1.0f);
            const float xh = (to_float(x[k]) - mean) * rstd;
            ((T*)a.dx)[r * a.dx_stride + k] = from_float<T>(rstd * (g - s - xh * t));
        }
    }
}

// Sums over the rows of a group, a thread to a column; and over the groups.
template <typename T>
__global__ void __launch_bounds__(256) norm_part_kernel(const __grid_constant__ NormArgs a) {
    griddep_wait();
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= a.width) return;
    float g = 0.0f, b = 0.0f;
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float dy = to_float(((const T*)a.dy)[r * a.dy_stride + k]);
        g = fmaf(dy, (to_float(((const T*)a.x)[r * a.x_stride + k]) - a.saved[2 * r]) * a.saved[2 * r + 1], g);
        b += dy;
    }
    a.part[2 * (int64_t)blockIdx.y * a.width + k] = g;
    a.part[(2 * (int64_t)blockIdx.y + 1) * a.width + k] = b;
}
template <typename P>
__global__ void __launch_bounds__(256) norm_param_kernel(const __grid_constant__ NormArgs a, int64_t groups) {
    griddep_wait();
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= a.width) return;
    float g = 0.0f, b = 0.0f;
    for (int64_t q = 0; q < groups; ++q) {
        g += a.part[2 * q * a.width + k];
        b += a.part[(2 * q + 1) * a.width + k];
    }
    if (a.dgamma != nullptr) ((P*)a.dgamma)[k] = from_float<P>(g);
    if (a.dbeta != nullptr) ((P*)a.dbeta)[k] = from_float<P>(b);
}

int64_t groups_of(int64_t rows) { return rows < 64 ? (rows > 0 ? rows : 1) : 64; }

unsigned blocks_for(int64_t rows) {
    const int64_t most = 8 * zs::device_sm_count();
    return (unsigned)(rows < most ? rows : most);
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
    a.rows = n->rows;
    a.width = n->width;
    a.x_stride = n->rows > 1 ? n->x_stride : n->width;
    a.eps = (float)n->eps;
    a.inv_width = (float)(1.0 / (double)n->width);
    return a;
}

template <typename T, typename P>
int32_t launch_grad(const NormArgs& a, cudaStream_t stream) {
    if (a.dgamma != nullptr || a.dbeta != nullptr) {
        // (before dx, which may take dy's or x's place)
        const int64_t groups = groups_of(a.rows);
        const unsigned wide = (unsigned)((a.width + 255) / 256);
        ZS_TRY(launch(norm_part_kernel<T>, dim3(wide, (unsigned)groups), 256, stream, "norm_part_kernel", a));
        ZS_TRY(launch(norm_param_kernel<P>, dim3(wide), 256, stream, "norm_param_kernel", a, groups));
    }
    if (a.dx == nullptr || a.rows == 0) return ZS_OK;
    return launch(norm_dx_kernel<T, P>, dim3(blocks_for(a.rows)), 256, stream, "norm_dx_kernel", a);
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
        return with_elem(n->param_type, [&](auto p) {
            return launch(norm_kernel<decltype(t), decltype(p)>, dim3(blocks_for(a.rows)), 256, (cudaStream_t)stream,
                          "norm_kernel", a);
        });
    });
}

ZS_API int64_t zero_layer_norm_work_bytes(int64_t rows, int64_t width) {
    if (!valid_sizes(rows, width)) return ZS_ERR_ARG;
    const int64_t groups = rows < 1 ? 1 : rows < kMaxGroups ? rows : kMaxGroups;
    return 8 * groups * ((width + 3) / 4 * 4);
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
    return with_elem(n->type, [&](auto t) {
        return with_elem(n->param_type,
                         [&](auto p) { return launch_grad<decltype(t), decltype(p)>(a, (cudaStream_t)stream); });
    });
}

}  // extern "C"
