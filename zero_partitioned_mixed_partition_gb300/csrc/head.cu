// head.cu -- token log-probabilities from hidden states and the vocabulary
// matrix, and their gradient, without keeping the logits.
//
// With x = H W^T, t near a row's largest logit and lnS = ln sum_j exp((x_j - t) it):
//   logp = (x_y - t) it - lnS,      d_ij = c_i (1[j = y_i] - p_ij),
//   dH = d W,   dW = d^T H,         c_i = L it dlogp_i.
// Rows that are left out (ignored labels, dlogp = 0) are taken out first: the
// live rows' hidden states are copied together, so that prompts cost nothing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <initializer_list>

#include "cluster_counts.h"
#include "zs_internal.h"

namespace {

#include "step_common.cuh"
#include "step_end.cuh"
#include "loss_common.cuh"
#include "elem.cuh"
#include "launch.cuh"

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLowestFloat = -3.402823466e38f;

constexpr int64_t kTile = 256;  // rows, and entries of the vocabulary, that a block's sums cover
constexpr int64_t kMaxRows = 1 << 24, kMaxVocab = 1 << 24, kMaxWidth = 1 << 16;
constexpr int64_t kPieceBytes = 1ll << 30;  // of a piece's gradient, where the caller leaves the choice

constexpr int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// ------------------------------------------------------------------ scratch ---

// What the rows kernel leaves for the others.
struct Counts {
    int32_t live;     // rows that are not left out
    float scale;      // d's power of 2
    float unscale;    // its inverse
};
// A live row.
struct __align__(16) Row {
    float top, log_sum;  // t, lnS
    float coef;          // c times d's scale
    int32_t label;
};

// The parts of the scratch buffer, as offsets from its start.
struct Plan {
    int64_t rows_pad, tiles, piece;
    int64_t index, row, hidden, part, label_logit, d, total;
};
Plan plan_of(int64_t rows, int64_t width, int64_t vocab, int64_t piece, bool gradient) {
    Plan p = {};
    p.rows_pad = round_up(rows > 0 ? rows : 1, kTile);
    p.tiles = round_up(vocab, kTile) / kTile;
    int64_t at = 128;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += round_up(bytes, 128);
        return here;
    };
    p.index = take(4 * p.rows_pad);
    p.row = take((int64_t)sizeof(Row) * p.rows_pad);
    p.hidden = take(2 * p.rows_pad * width);
    if (gradient) {
        if (piece <= 0) piece = kPieceBytes / (2 * p.rows_pad);
        p.piece = piece < kTile ? kTile : round_up(piece, kTile);
        if (p.piece > p.tiles * kTile) p.piece = p.tiles * kTile;
        p.part = take(4 * p.rows_pad * width);
        p.d = take(2 * p.rows_pad * p.piece);
    } else {
        p.part = take(8 * p.rows_pad * p.tiles);
        p.label_logit = take(4 * p.rows_pad);
    }
    p.total = at;
    return p;
}
bool valid_sizes(int64_t rows, int64_t width, int64_t vocab) {
    return rows >= 0 && rows <= kMaxRows && vocab >= 1 && vocab <= kMaxVocab && width >= 8 && width <= kMaxWidth &&
           width % 8 == 0;
}
// The plan with the largest piece that fits; total = 0: none does.
Plan plan_within(int64_t rows, int64_t width, int64_t vocab, int64_t bytes) {
    Plan p = plan_of(rows, width, vocab, kTile, true);
    const int64_t more = (bytes - p.total) / (2 * p.rows_pad * kTile);
    if (bytes < p.total) {
        p.total = 0;
        return p;
    }
    return plan_of(rows, width, vocab, (more + 1) * kTile, true);
}

// ------------------------------------------------------------- live rows ---

struct HeadArgs {
    const void *hidden, *weight;
    int64_t rows, vocab, width, hidden_stride, weight_stride;
    float it;
    const int64_t* labels;
    const float *saved, *dlogp;  // gradient: else NULL
    const zs_ctrl* ctrl;
    float *logp, *saved_out;     // forward
    uint16_t* dhidden;
    int64_t dhidden_stride;
    uint16_t* dweight;
    int64_t dweight_stride;
    Counts* counts;
    int32_t* index;
    Row* row;
    uint16_t* compact;           // [rows_pad][width]
    void* part;
    float* label_logit;
    uint16_t* d;                 // [rows_pad][piece]
    int64_t rows_pad, tiles, piece;
};

__device__ __forceinline__ bool is_live(const HeadArgs& a, int64_t i) {
    const int64_t y = a.labels[i];
    return y >= 0 && y < a.vocab && (a.dlogp == nullptr || a.dlogp[i] != 0.0f);
}

constexpr int kRowThreads = 1024;

// Numbers the live rows in their order, and finds the power of 2 by which d is
// scaled.  One block: the numbers depend on all rows before.
__global__ void __launch_bounds__(kRowThreads) head_rows_kernel(const __grid_constant__ HeadArgs a) {
    __shared__ int32_t s_count[kRowThreads / 32];
    __shared__ float s_top[kRowThreads / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    griddep_wait();
    int32_t base = 0;
    float top = 0.0f;
    const float factor = loss_scale_of(a.ctrl) * a.it;
    for (int64_t from = 0; from < a.rows; from += kRowThreads) {
        const int64_t i = from + threadIdx.x;
        const bool live = i < a.rows && is_live(a, i);
        const uint32_t votes = __ballot_sync(0xffffffffu, live);
        if (lane == 0) s_count[warp] = __popc(votes);
        __syncthreads();
        int32_t before = base, all = 0;
        for (int w = 0; w < kRowThreads / 32; ++w) {
            before += w < warp ? s_count[w] : 0;
            all += s_count[w];
        }
        __syncthreads();
        base += all;
        if (live) {
            const int32_t r = before + __popc(votes & ((1u << lane) - 1u));
            Row row = {0.0f, 0.0f, 0.0f, (int32_t)a.labels[i]};
            if (a.dlogp != nullptr) {
                row.top = a.saved[2 * i];
                row.log_sum = a.saved[2 * i + 1];
                // (a row of nothing but -inf has no gradient)
                row.coef = row.log_sum == -__int_as_float(0x7f800000) ? 0.0f : factor * a.dlogp[i];
                // (a NaN counts as infinite)
                const float size = fabsf(row.coef);
                top = fmaxf(top, size <= 3.402823466e38f ? size : __int_as_float(0x7f800000));
            }
            a.index[r] = (int32_t)i;
            a.row[r] = row;
        }
    }
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 0; w < kRowThreads / 32; ++w) top = fmaxf(top, s_top[w]);
        // the largest |c| goes to [2^14, 2^15)
        int e = top > 0.0f && top <= 3.402823466e38f ? 14 - ilogbf(top) : 0;
        e = e > 120 ? 120 : e < -120 ? -120 : e;
        *a.counts = Counts{base, scalbnf(1.0f, e), scalbnf(1.0f, -e)};
    }
}

// Copies the live rows' hidden states together, with zeros up to a whole tile,
// and writes the outputs of the rows that are left out.
__global__ void __launch_bounds__(256) head_gather_kernel(const __grid_constant__ HeadArgs a) {
    griddep_wait();
    const int64_t vectors = a.width / 8;
    const int32_t live = a.counts->live;
    const int64_t pad = round_up(live, kTile);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t r = blockIdx.x; r < pad; r += gridDim.x) {
        const uint4* src = r < live ? reinterpret_cast<const uint4*>((const uint16_t*)a.hidden + a.index[r] * a.hidden_stride)
                                    : nullptr;
        uint4* dst = reinterpret_cast<uint4*>(a.compact + r * a.width);
        for (int64_t k = threadIdx.x; k < vectors; k += blockDim.x) dst[k] = r < live ? src[k] : zero;
        if (threadIdx.x == 0) {
            if (r >= live) a.row[r] = Row{0.0f, 0.0f, 0.0f, -1};
            else if (a.dlogp != nullptr) a.row[r].coef *= a.counts->scale;
        }
    }
    for (int64_t i = blockIdx.x; i < a.rows; i += gridDim.x) {
        if (is_live(a, i)) continue;
        if (a.dhidden != nullptr)
            for (int64_t k = threadIdx.x; k < vectors; k += blockDim.x)
                reinterpret_cast<uint4*>(a.dhidden + i * a.dhidden_stride)[k] = zero;
        if (threadIdx.x == 0 && a.logp != nullptr) a.logp[i] = 0.0f;
        if (threadIdx.x < 2 && a.saved_out != nullptr) a.saved_out[2 * i + threadIdx.x] = 0.0f;
    }
}

// ---------------------------------------------------------------- products ---

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// d of a live row's logit, scaled.
__device__ __forceinline__ float d_of(const Row& row, float x, int32_t j, float k) {
    const float p = exp2_approx((x - row.top) * k - row.log_sum * kLog2e);
    return j == row.label ? row.coef * (1.0f - p) : -row.coef * p;
}

constexpr int kBlockRows = 16;

enum { kLogits, kGrad, kDHidden, kDWeight };

// A block makes kBlockRows x 256 sums, a thread those of one column.
//   kLogits    rows of H and of W: statistics of each row over the block's columns
//   kGrad      the same logits of one piece: d
//   kDHidden   d of one piece times W: added to fp32 sums, or the output
//   kDWeight   d^T H: rows of dW
template <typename T, int MODE>
__global__ void __launch_bounds__(256) head_product_kernel(const __grid_constant__ HeadArgs a, int64_t first, int64_t count,
                                                           int last) {
    __shared__ float s_a[kBlockRows][33];
    __shared__ float s_x[kBlockRows][256];
    griddep_wait();
    const int32_t live = a.counts->live;
    const int64_t m0 = (int64_t)blockIdx.x * kBlockRows, n0 = (int64_t)blockIdx.y * 256;
    const int64_t n = n0 + threadIdx.x;
    const T* hidden = (const T*)a.compact;
    const T* weight = (const T*)a.weight + first * a.weight_stride;
    const T* d = (const T*)a.d;
    int64_t inner;
    if (MODE == kLogits || MODE == kGrad) {
        if (m0 >= round_up(live, kTile)) return;
        inner = a.width;
    } else if (MODE == kDHidden) {
        if (m0 >= live) return;
        inner = count;
    } else {
        inner = live;
    }
    float sum[kBlockRows] = {};
    for (int64_t k0 = 0; k0 < inner; k0 += 32) {
        for (int q = threadIdx.x; q < kBlockRows * 32; q += 256) {
            const int m = MODE == kDWeight ? q % kBlockRows : q / 32, k = MODE == kDWeight ? q / kBlockRows : q % 32;
            float x = 0.0f;
            if (k0 + k < inner) {
                if (MODE == kLogits || MODE == kGrad) x = to_float(hidden[(m0 + m) * a.width + k0 + k]);
                if (MODE == kDHidden) x = to_float(d[(m0 + m) * a.piece + k0 + k]);
                if (MODE == kDWeight) x = to_float(d[(k0 + k) * a.piece + m0 + m]);
            }
            s_a[m][k] = x;
        }
        __syncthreads();
        const int lim = inner - k0 < 32 ? (int)(inner - k0) : 32;
        for (int k = 0; k < lim; ++k) {
            float y = 0.0f;
            if (MODE == kLogits || MODE == kGrad) y = n < count ? to_float(weight[n * a.weight_stride + k0 + k]) : 0.0f;
            if (MODE == kDHidden) y = n < a.width ? to_float(weight[(k0 + k) * a.weight_stride + n]) : 0.0f;
            if (MODE == kDWeight) y = n < a.width ? to_float(hidden[(k0 + k) * a.width + n]) : 0.0f;
#pragma unroll
            for (int m = 0; m < kBlockRows; ++m) sum[m] = fmaf(s_a[m][k], y, sum[m]);
        }
        __syncthreads();
    }
    const float k = a.it * kLog2e;
    if (MODE == kLogits) {
#pragma unroll
        for (int m = 0; m < kBlockRows; ++m) s_x[m][threadIdx.x] = n < count ? sum[m] : -__int_as_float(0x7f800000);
        __syncthreads();
        if (threadIdx.x < kBlockRows) {
            const int m = threadIdx.x;
            float top = kLowestFloat, s = 0.0f;
            for (int j = 0; j < 256; ++j) top = fmaxf(top, s_x[m][j]);
            for (int j = 0; j < 256; ++j) s += exp2_approx((s_x[m][j] - top) * k);
            const int32_t y = a.row[m0 + m].label;
            if (y >= n0 && y < n0 + 256) a.label_logit[m0 + m] = s_x[m][y - n0];
            ((float2*)a.part)[blockIdx.y * a.rows_pad + m0 + m] = make_float2(top, s);
        }
    }
    for (int m = 0; m < kBlockRows; ++m) {
        if (MODE == kGrad) {
            const Row row = a.row[m0 + m];
            const float v = n < count && row.coef != 0.0f ? d_of(row, sum[m], (int32_t)(first + n), k) : 0.0f;
            ((T*)a.d)[(m0 + m) * a.piece + n] = from_float<T>(v);
        }
        if (MODE == kDHidden && n < a.width && m0 + m < live) {
            float* acc = (float*)a.part + (m0 + m) * a.width + n;
            const float v = first > 0 ? *acc + sum[m] : sum[m];
            if (last) {
                ((T*)a.dhidden)[a.index[m0 + m] * a.dhidden_stride + n] = from_float<T>(v * a.counts->unscale);
            } else {
                *acc = v;
            }
        }
        if (MODE == kDWeight && n < a.width && m0 + m < count)
            ((T*)a.dweight)[(first + m0 + m) * a.dweight_stride + n] = from_float<T>(sum[m] * a.counts->unscale);
    }
}

// Joins the statistics of a row's tiles: a warp to a row.
__global__ void __launch_bounds__(256) head_join_kernel(const __grid_constant__ HeadArgs a) {
    griddep_wait();
    const int lane = threadIdx.x % 32;
    const int64_t r = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (r >= a.counts->live) return;
    const float2* part = (const float2*)a.part + r;
    const float k = a.it * kLog2e;
    float top = kLowestFloat, s = 0.0f;
    for (int64_t t = lane; t < a.tiles; t += 32) top = fmaxf(top, part[t * a.rows_pad].x);
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    for (int64_t t = lane; t < a.tiles; t += 32) {
        const float2 q = part[t * a.rows_pad];
        s += q.y * exp2_approx((q.x - top) * k);
    }
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
        const int64_t i = a.index[r];
        const float log_sum = logf(s);
        a.logp[i] = s == 0.0f ? log_sum : (a.label_logit[r] - top) * a.it - log_sum;
        if (a.saved_out != nullptr) {
            a.saved_out[2 * i] = top;
            a.saved_out[2 * i + 1] = log_sum;
        }
    }
}

// ------------------------------------------------------------------- launches ---

bool valid_stride(int64_t rows, int64_t width, int64_t stride) {
    return rows <= 1 || (stride >= width && stride <= 1ll << 40);
}

int32_t check_head(const zs_head* h) {
    if (h == nullptr || !valid_sizes(h->rows, h->width, h->vocab) || (h->type != ZS_F16 && h->type != ZS_BF16) ||
        h->reserved != 0 || !(h->inv_temperature >= 1e-6 && h->inv_temperature <= 1e6))
        return ZS_ERR_ARG;
    if (h->weight == nullptr || (h->rows > 0 && h->hidden == nullptr)) return ZS_ERR_ARG;
    if (!valid_stride(h->rows, h->width, h->hidden_stride) || !valid_stride(h->vocab, h->width, h->weight_stride))
        return ZS_ERR_ARG;
    if (!zs::aligned_to(h->hidden, 16) || !zs::aligned_to(h->weight, 16) || (h->rows > 1 && h->hidden_stride % 8 != 0) ||
        (h->vocab > 1 && h->weight_stride % 8 != 0))
        return ZS_ERR_ALIGN;
    return ZS_OK;
}

HeadArgs args_of(const zs_head* h, const Plan& p, void* work) {
    HeadArgs a = {};
    char* base = (char*)work;
    a.hidden = h->hidden;
    a.weight = h->weight;
    a.rows = h->rows;
    a.vocab = h->vocab;
    a.width = h->width;
    a.hidden_stride = h->rows > 1 ? h->hidden_stride : h->width;
    a.weight_stride = h->vocab > 1 ? h->weight_stride : h->width;
    a.it = (float)h->inv_temperature;
    a.counts = (Counts*)base;
    a.index = (int32_t*)(base + p.index);
    a.row = (Row*)(base + p.row);
    a.compact = (uint16_t*)(base + p.hidden);
    a.part = base + p.part;
    a.label_logit = (float*)(base + p.label_logit);
    a.d = (uint16_t*)(base + p.d);
    a.rows_pad = p.rows_pad;
    a.tiles = p.tiles;
    a.piece = p.piece;
    return a;
}

int32_t launch_rows(const HeadArgs& a, cudaStream_t stream) {
    ZS_TRY(launch(head_rows_kernel, dim3(1), kRowThreads, stream, "head_rows_kernel", a));
    const int64_t most = 8 * zs::device_sm_count();
    return launch(head_gather_kernel, dim3((unsigned)(a.rows_pad < most ? a.rows_pad : most)), 256, stream,
                  "head_gather_kernel", a);
}

template <typename T>
int32_t launch_logp(const HeadArgs& a, cudaStream_t stream) {
    ZS_TRY(launch_rows(a, stream));
    ZS_TRY(launch(head_product_kernel<T, kLogits>, dim3((unsigned)(a.rows_pad / kBlockRows), (unsigned)a.tiles), 256, stream,
                  "head_product_kernel", a, (int64_t)0, a.vocab, 0));
    return launch(head_join_kernel, dim3((unsigned)(round_up(a.rows, 8) / 8)), 256, stream, "head_join_kernel", a);
}

template <typename T>
int32_t launch_grad(const HeadArgs& a, cudaStream_t stream) {
    ZS_TRY(launch_rows(a, stream));
    const unsigned wide = (unsigned)(round_up(a.width, 256) / 256), rows = (unsigned)(a.rows_pad / kBlockRows);
    for (int64_t first = 0; first < a.vocab; first += a.piece) {
        const int64_t count = a.vocab - first < a.piece ? a.vocab - first : a.piece;
        const int last = first + count == a.vocab;
        ZS_TRY(launch(head_product_kernel<T, kGrad>, dim3(rows, (unsigned)(round_up(count, 256) / 256)), 256, stream,
                      "head_product_kernel", a, first, count, last));
        if (a.dhidden != nullptr)
            ZS_TRY(launch(head_product_kernel<T, kDHidden>, dim3(rows, wide), 256, stream, "head_product_kernel", a, first,
                          count, last));
        if (a.dweight != nullptr)
            ZS_TRY(launch(head_product_kernel<T, kDWeight>, dim3((unsigned)(round_up(count, kBlockRows) / kBlockRows), wide),
                          256, stream, "head_product_kernel", a, first, count, last));
    }
    return ZS_OK;
}

}  // namespace

namespace zs {
uint64_t take_fault_head() { return take_fault(); }
}  // namespace zs

extern "C" {

ZS_API int64_t zero_head_work_bytes(int64_t rows, int64_t width, int64_t vocab, int64_t piece, int32_t gradient) {
    if (!valid_sizes(rows, width, vocab) || piece < 0 || (gradient != 0 && gradient != 1)) return ZS_ERR_ARG;
    return plan_of(rows, width, vocab, piece, gradient == 1).total;
}

ZS_API int32_t zero_head_logp_async(const zs_head* h, const int64_t* labels, float* logp, float* saved,
                                    void* work_dev, int64_t work_bytes, void* stream) {
    zs::NvtxRange nvtx_range("zero_head_logp_async");
    ZS_TRY(check_head(h));
    if (h->rows == 0) return ZS_OK;
    if (labels == nullptr || logp == nullptr || work_dev == nullptr) return ZS_ERR_ARG;
    if (!zs::aligned_to(labels, 8) || !zs::aligned_to(logp, 4) || !zs::aligned_to(saved, 4) || !zs::aligned_to(work_dev, 128))
        return ZS_ERR_ALIGN;
    const Plan p = plan_of(h->rows, h->width, h->vocab, 0, false);
    if (work_bytes < p.total) return ZS_ERR_ARG;
    HeadArgs a = args_of(h, p, work_dev);
    a.labels = labels;
    a.logp = logp;
    a.saved_out = saved;
    return h->type == ZS_F16 ? launch_logp<__half>(a, (cudaStream_t)stream) : launch_logp<__nv_bfloat16>(a, (cudaStream_t)stream);
}

ZS_API int32_t zero_head_logp_grad_async(const zs_head* h, const int64_t* labels, const float* saved,
                                         const float* dlogp, const zs_ctrl* ctrl_dev, void* dhidden,
                                         int64_t dhidden_stride, void* dweight, int64_t dweight_stride,
                                         void* work_dev, int64_t work_bytes, void* stream) {
    zs::NvtxRange nvtx_range("zero_head_logp_grad_async");
    ZS_TRY(check_head(h));
    if (work_dev == nullptr || (dhidden == nullptr && dweight == nullptr)) return ZS_ERR_ARG;
    if (h->rows > 0 && (labels == nullptr || saved == nullptr || dlogp == nullptr)) return ZS_ERR_ARG;
    if ((dhidden != nullptr && !valid_stride(h->rows, h->width, dhidden_stride)) ||
        (dweight != nullptr && !valid_stride(h->vocab, h->width, dweight_stride)))
        return ZS_ERR_ARG;
    if (!zs::aligned_to(labels, 8) || !zs::aligned_to(saved, 4) || !zs::aligned_to(dlogp, 4) || !zs::aligned_to(ctrl_dev, 8) ||
        !zs::aligned_to(dhidden, 16) || !zs::aligned_to(dweight, 16) || !zs::aligned_to(work_dev, 128) ||
        (dhidden != nullptr && h->rows > 1 && dhidden_stride % 8 != 0) ||
        (dweight != nullptr && h->vocab > 1 && dweight_stride % 8 != 0))
        return ZS_ERR_ALIGN;
    const Plan p = plan_within(h->rows, h->width, h->vocab, work_bytes);
    if (p.total == 0) return ZS_ERR_ARG;
    if (h->rows == 0 && dweight == nullptr) return ZS_OK;
    HeadArgs a = args_of(h, p, work_dev);
    a.labels = labels;
    a.saved = saved;
    a.dlogp = dlogp;
    a.ctrl = ctrl_dev;
    a.dhidden = (uint16_t*)dhidden;
    a.dhidden_stride = h->rows > 1 ? dhidden_stride : h->width;
    a.dweight = (uint16_t*)dweight;
    a.dweight_stride = h->vocab > 1 ? dweight_stride : h->width;
    return h->type == ZS_F16 ? launch_grad<__half>(a, (cudaStream_t)stream) : launch_grad<__nv_bfloat16>(a, (cudaStream_t)stream);
}

}  // extern "C"
