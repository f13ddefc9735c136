// Exhaustive GPU checks of the packed arithmetic of the AdamW step over a list
// of tensors (csrc/tensors_math.cuh), run by tests/test_gpu_tensors_math.py:
//
//  1. sqrt2 against __fsqrt_rn, for every float in [2^-80, 2^80];
//  2. reciprocal2 against __frcp_rn, for every float in [2^-64, 2^64];
//  3. div2 against __fdiv_rn, for 40 divisors over [2^-40, 2^40] and every
//     float x with 2^-80 <= |x| <= 2^80 (one sign in each half of the pair);
//  4. div2_by_constant against __fdiv_rn, for 10 divisors in (0, 1] and the
//     same x.
//
// Bit for bit.  Every loop is a grid-stride loop over a fixed range; nothing
// waits.  Prints one line per check and exits 1 if any value differs.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <cmath>

namespace {

#include "packed.cuh"
#include "tensors_math.cuh"

__device__ unsigned long long g_bad;

__device__ __forceinline__ bool same(float a, float b) { return __float_as_uint(a) == __float_as_uint(b); }

enum { kSqrt, kReciprocal, kDivide, kConstant };

// Bit patterns [lo, hi].
template <int WHAT>
__global__ void check(uint32_t lo, uint32_t hi, float d) {
    unsigned long long bad = 0;
    for (uint64_t i = lo + (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i <= hi; i += (uint64_t)gridDim.x * blockDim.x) {
        const float x = __uint_as_float((uint32_t)i);
        float a, b;
        if (WHAT == kSqrt) {
            split(sqrt2(pair(x, x)), a, b);
            bad += !same(a, __fsqrt_rn(x)) || !same(b, __fsqrt_rn(x));
        } else if (WHAT == kReciprocal) {
            split(reciprocal2(pair(x, x)), a, b);
            bad += !same(a, __frcp_rn(x)) || !same(b, __frcp_rn(x));
        } else {
            split(WHAT == kDivide ? div2(pair(x, -x), pair(d, d)) : div2_by_constant(pair(x, -x), d, __frcp_rn(d)), a, b);
            bad += !same(a, __fdiv_rn(x, d)) || !same(b, __fdiv_rn(-x, d));
        }
    }
    if (bad) atomicAdd(&g_bad, bad);
}

uint32_t bits_of_power(int e) { return (uint32_t)(127 + e) << 23; }

int total_bad = 0;

template <int WHAT>
void run(const char* name, int lo, int hi, float d) {
    unsigned long long zero = 0, bad = 0;
    cudaMemcpyToSymbol(g_bad, &zero, sizeof(zero));
    check<WHAT><<<1216, 256>>>(bits_of_power(lo), bits_of_power(hi), d);
    cudaMemcpyFromSymbol(&bad, g_bad, sizeof(bad));
    printf("%s d = %.9g: %llu mismatches\n", name, d, bad);
    total_bad += bad != 0;
}

}  // namespace

int main() {
    run<kSqrt>("sqrt2", -80, 80, 1.0f);
    run<kReciprocal>("reciprocal2", -64, 64, 1.0f);
    uint32_t s = 12345u;
    for (int i = 0; i < 40; ++i) {
        s = s * 1664525u + 1013904223u;
        const float f = 1.0f + (float)(s >> 9) / 8388608.0f;
        const float d = i == 0 ? 1.0f : i == 1 ? std::nextafterf(2.0f, 1.0f) : i == 2 ? std::nextafterf(1.0f, 2.0f) : f;
        run<kDivide>("div2", -80, 80, std::ldexp(d, i < 3 ? 0 : 2 * i - 40));
    }
    double p = 1.0;
    for (int t = 1; t <= 10; ++t) {
        p *= t < 6 ? 0.9 : 0.999;
        run<kConstant>("div2_by_constant", -80, 80, (float)(1.0 - p));
    }
    const cudaError_t err = cudaDeviceSynchronize();
    if (err != cudaSuccess) {
        printf("CUDA error: %s\n", cudaGetErrorString(err));
        return 1;
    }
    printf(total_bad ? "differences\n" : "all equal\n");
    return total_bad ? 1 : 0;
}
