// elem.cuh -- element types of the head, norm and embedding kernels: their
// conversions, and 16-byte vectors of them.  Included inside an anonymous
// namespace, after <cuda_fp16.h> and <cuda_bf16.h>.
#pragma once

template <typename T> __device__ __forceinline__ float to_float(T x);
template <> __device__ __forceinline__ float to_float<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Two values rounded to a 16-bit type, the first in the lower half.
template <typename T> __device__ __forceinline__ uint32_t narrow2(float a, float b);
template <> __device__ __forceinline__ uint32_t narrow2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t narrow2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T> __device__ __forceinline__ float2 widen2(uint32_t w);
template <> __device__ __forceinline__ float2 widen2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <> __device__ __forceinline__ float2 widen2<__nv_bfloat16>(uint32_t w) {  // the upper half of an fp32
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// V values of a type, as accesses of up to 16 bytes (V = 1: an element).
template <typename T, int V> struct alignas(V * sizeof(T) < 16 ? V * sizeof(T) : 16) Pack {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V>& p, float* x) {
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 f = widen2<T>(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = to_float<T>(p.v[i]);
    }
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> pack(const float* x) {
    Pack<T, V> p;
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&p);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = narrow2<T>(x[2 * i], x[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p.v[i] = from_float<T>(x[i]);
    }
    return p;
}

// Calls f with a value of the element type.
template <typename F>
int32_t with_elem(int32_t type, F f) {
    return type == ZS_F32 ? f(float()) : type == ZS_F16 ? f(__half()) : f(__nv_bfloat16());
}
inline int64_t elem_size(int32_t type) { return type == ZS_F32 ? 4 : 2; }
