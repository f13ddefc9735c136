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
template <int BYTES> struct RawOf;
template <> struct RawOf<2> { using type = uint16_t; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = uint4; };
struct alignas(16) Raw32 {
    uint4 a, b;
};
template <> struct RawOf<32> { using type = Raw32; };
template <typename T, int V> struct Pack {
    typename RawOf<V * sizeof(T)>::type raw;
};
template <typename T, int V>
__device__ __forceinline__ void unpack(Pack<T, V> p, float* x) {  // (by value: one load where p is in memory)
    if constexpr (V == 1 && sizeof(T) == 2) {
        x[0] = to_float<T>(*reinterpret_cast<const T*>(&p.raw));
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&p.raw);
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 f = widen2<T>(w[i]);
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = __uint_as_float(w[i]);
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> pack(const float* x) {
    Pack<T, V> p;
    if constexpr (V == 1 && sizeof(T) == 2) {
        const T t = from_float<T>(x[0]);
        p.raw = *reinterpret_cast<const uint16_t*>(&t);
    } else {
        uint32_t* w = reinterpret_cast<uint32_t*>(&p.raw);
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) w[i] = narrow2<T>(x[2 * i], x[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(x[i]);
        }
    }
    return p;
}

// Calls f with a value of the element type.
template <typename F>
int32_t with_elem(int32_t type, F f) {
    return type == ZS_F32 ? f(float()) : type == ZS_F16 ? f(__half()) : f(__nv_bfloat16());
}
inline int64_t elem_size(int32_t type) { return type == ZS_F32 ? 4 : 2; }
