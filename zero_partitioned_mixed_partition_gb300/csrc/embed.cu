// embed.cu -- embedding lookup with scaling, and the gradient of its table.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "zs_internal.h"

namespace {

#include "step_common.cuh"
#include "step_end.cuh"
#include "elem.cuh"
#include "launch.cuh"

constexpr int64_t kMaxTokens = 1 << 28, kMaxVocab = 1 << 30, kMaxWidth = 1 << 24;

struct EmbedArgs {
    const void* table;
    const int64_t* ids;
    int64_t tokens, vocab, width, table_stride;
    float scale;
    void* out;
    int64_t out_stride;
    const void* dout;
    int64_t dout_stride;
    void* dtable;
    int64_t dtable_stride;
    int32_t accumulate;
};

template <typename T>
__global__ void __launch_bounds__(256) embed_kernel(const __grid_constant__ EmbedArgs a) {
    griddep_wait();
    for (int64_t i = blockIdx.x; i < a.tokens; i += gridDim.x) {
        const int64_t v = a.ids[i];
        const bool inside = v >= 0 && v < a.vocab;
        const T* row = (const T*)a.table + (inside ? v : 0) * a.table_stride;
        T* out = (T*)a.out + i * a.out_stride;
        for (int64_t k = threadIdx.x; k < a.width; k += blockDim.x)
            out[k] = inside ? from_float<T>(to_float(row[k]) * a.scale) : from_float<T>(0.0f);
    }
}

// A block to a row of the table: looks through the tokens in their order.
template <typename T, typename G>
__global__ void __launch_bounds__(256) embed_grad_kernel(const __grid_constant__ EmbedArgs a) {
    griddep_wait();
    for (int64_t v = blockIdx.x; v < a.vocab; v += gridDim.x) {
        G* row = (G*)a.dtable + v * a.dtable_stride;
        for (int64_t k0 = 0; k0 < a.width; k0 += 256) {
            const int64_t k = k0 + threadIdx.x;
            float s = 0.0f;
            bool any = false;
            for (int64_t from = 0; from < a.tokens; from += 256) {
                const int64_t i = from + threadIdx.x;
                const bool hit = i < a.tokens && a.ids[i] == v;
                if (!__syncthreads_or(hit)) continue;
                any = true;
                for (int64_t j = from; j < from + 256 && j < a.tokens; ++j)
                    if (a.ids[j] == v && k < a.width) s += to_float(((const T*)a.dout)[j * a.dout_stride + k]);
            }
            if (k >= a.width) continue;
            s *= a.scale;
            if (!a.accumulate)
                row[k] = from_float<G>(s);
            else if (any)
                row[k] = from_float<G>(to_float(row[k]) + s);
        }
    }
}

unsigned blocks_for(int64_t rows) {
    const int64_t most = 8 * zs::device_sm_count();
    return (unsigned)(rows < most ? rows : most);
}

bool valid_stride(int64_t rows, int64_t width, int64_t stride) {
    return rows <= 1 || (stride >= width && stride <= 1ll << 40);
}

int32_t check_embed(const zs_embed* e) {
    if (e == nullptr || e->tokens < 0 || e->tokens > kMaxTokens || e->vocab < 1 || e->vocab > kMaxVocab || e->width < 1 ||
        e->width > kMaxWidth || (e->type != ZS_F32 && e->type != ZS_F16 && e->type != ZS_BF16) || e->reserved != 0 ||
        !(e->scale >= -1e30 && e->scale <= 1e30) || (e->tokens > 0 && e->ids == nullptr))
        return ZS_ERR_ARG;
    return zs::aligned_to(e->ids, 8) ? ZS_OK : ZS_ERR_ALIGN;
}
EmbedArgs args_of(const zs_embed* e) {
    EmbedArgs a = {};
    a.table = e->table;
    a.ids = e->ids;
    a.tokens = e->tokens;
    a.vocab = e->vocab;
    a.width = e->width;
    a.table_stride = e->vocab > 1 ? e->table_stride : e->width;
    a.scale = (float)e->scale;
    return a;
}

}  // namespace

namespace zs {
uint64_t take_fault_embed() { return take_fault(); }
}  // namespace zs

extern "C" {

ZS_API int32_t zero_embed_async(const zs_embed* e, void* out, int64_t out_stride, void* stream) {
    zs::NvtxRange nvtx_range("zero_embed_async");
    ZS_TRY(check_embed(e));
    if (e->tokens == 0) return ZS_OK;
    if (e->table == nullptr || out == nullptr || !valid_stride(e->vocab, e->width, e->table_stride) ||
        !valid_stride(e->tokens, e->width, out_stride))
        return ZS_ERR_ARG;
    const uintptr_t size = (uintptr_t)elem_size(e->type);
    if (!zs::aligned_to(e->table, size) || !zs::aligned_to(out, size)) return ZS_ERR_ALIGN;
    EmbedArgs a = args_of(e);
    a.out = out;
    a.out_stride = e->tokens > 1 ? out_stride : e->width;
    return with_elem(e->type, [&](auto t) {
        return launch(embed_kernel<decltype(t)>, dim3(blocks_for(a.tokens)), 256, (cudaStream_t)stream, "embed_kernel", a);
    });
}

ZS_API int64_t zero_embed_work_bytes(int64_t tokens, int64_t width) {
    if (tokens < 0 || tokens > kMaxTokens || width < 1 || width > kMaxWidth) return ZS_ERR_ARG;
    return 128;
}

ZS_API int32_t zero_embed_grad_async(const zs_embed* e, const void* dout, int64_t dout_stride, void* dtable,
                                     int64_t dtable_stride, int32_t dtable_type, int32_t accumulate, void* work_dev,
                                     int64_t work_bytes, void* stream) {
    zs::NvtxRange nvtx_range("zero_embed_grad_async");
    ZS_TRY(check_embed(e));
    if (dtable == nullptr || work_dev == nullptr || (dtable_type != e->type && dtable_type != ZS_F32) ||
        (accumulate != 0 && accumulate != 1) || (e->tokens > 0 && dout == nullptr) ||
        !valid_stride(e->tokens, e->width, dout_stride) || !valid_stride(e->vocab, e->width, dtable_stride) ||
        work_bytes < zero_embed_work_bytes(e->tokens, e->width))
        return ZS_ERR_ARG;
    if (!zs::aligned_to(dout, (uintptr_t)elem_size(e->type)) || !zs::aligned_to(dtable, (uintptr_t)elem_size(dtable_type)) ||
        !zs::aligned_to(work_dev, 16))
        return ZS_ERR_ALIGN;
    EmbedArgs a = args_of(e);
    a.dout = dout;
    a.dout_stride = e->tokens > 1 ? dout_stride : e->width;
    a.dtable = dtable;
    a.dtable_stride = e->vocab > 1 ? dtable_stride : e->width;
    a.accumulate = accumulate;
    return with_elem(e->type, [&](auto t) {
        using T = decltype(t);
        auto go = [&](auto kernel) {
            return launch(kernel, dim3(blocks_for(a.vocab)), 256, (cudaStream_t)stream, "embed_grad_kernel", a);
        };
        return dtable_type == ZS_F32 ? go(embed_grad_kernel<T, float>) : go(embed_grad_kernel<T, T>);
    });
}

}  // extern "C"
