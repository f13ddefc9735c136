// tensors_math.cuh -- correctly rounded divisions and square roots of pairs of
// fp32 values, for the AdamW step over a list of tensors.  Included inside an
// anonymous namespace by tensors.cu (and by the program that checks them
// against the scalar operations), after packed.cuh.
#pragma once

// div_by_constant for a pair.
__device__ __forceinline__ uint64_t div2_by_constant(uint64_t x, float d, float y) {
    const uint64_t minus = pair(-d, -d), yy = pair(y, y);
    uint64_t q = mul2(x, yy);
    q = fma2(fma2(q, minus, x), yy, q);
    return fma2(fma2(q, minus, x), yy, q);
}

__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The square roots of a pair, correctly rounded, for values in [2^-80, 2^80]:
// from y ~ 1 / sqrt(x), g = x y and h = y / 2 approach sqrt(x) and half its
// reciprocal together (Goldschmidt's iteration), then one step with the exact
// residual x - g g (P. Markstein, "IA-64 and Elementary Functions", 2000).
// Checked against __fsqrt_rn for every significand and both exponent parities,
// which is every case: no exponent in the range loses a bit.
__device__ __forceinline__ uint64_t sqrt2(uint64_t x) {
    float a, b;
    split(x, a, b);
    const uint64_t y = pair(rsqrt_approx(a), rsqrt_approx(b)), half = pair(0.5f, 0.5f), minus = pair(-1.0f, -1.0f);
    uint64_t g = mul2(x, y), h = mul2(y, half);
    const uint64_t r = fma2(mul2(h, minus), g, half);
    g = fma2(g, r, g);
    h = fma2(h, r, h);
    return fma2(fma2(mul2(g, minus), g, x), h, g);
}

// The quotients of a pair, correctly rounded, for divisors in [2^-64, 2^64] and
// |x| in [2^-80, 2^80] (or 0), the quotient a normal float: y = RN(1 / d) by two Newton steps from the
// hardware's estimate, then as div_by_constant (Markstein's theorem).  Checked:
// y against __frcp_rn for every significand.
__device__ __forceinline__ uint64_t reciprocal2(uint64_t d) {
    float a, b;
    split(d, a, b);
    const uint64_t one = pair(1.0f, 1.0f), minus = mul2(d, pair(-1.0f, -1.0f));
    uint64_t y = pair(rcp_approx(a), rcp_approx(b));
    y = fma2(fma2(minus, y, one), y, y);
    return fma2(fma2(minus, y, one), y, y);
}
__device__ __forceinline__ uint64_t div2(uint64_t x, uint64_t d) {
    const uint64_t y = reciprocal2(d), minus = mul2(d, pair(-1.0f, -1.0f));
    uint64_t q = mul2(x, y);
    q = fma2(fma2(q, minus, x), y, q);
    return fma2(fma2(q, minus, x), y, q);
}
