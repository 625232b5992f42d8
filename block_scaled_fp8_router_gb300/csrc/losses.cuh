// losses.cuh -- device helpers shared by the loss kernels (losses.cu,
// router_dense.cu): the hardware exponential, reciprocal, and sums in two
// fp32 numbers.
#pragma once

#include "common.cuh"

namespace moe {

constexpr float LN2 = 0.693147180559945309f;
constexpr float LOG2E = 1.44269504088896341f;

// 2^x, relative error 2^-22, results below the smallest normal flushed to 0
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / x to within a unit in the last place (1 / inf = 0)
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2 x, absolute error 2^-22 near 1
__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a / b for b in [2^-100, 2^126]: the reciprocal's quotient and one step of its
// exact residual (Markstein), in general the correctly rounded quotient
__device__ __forceinline__ float div1(float a, float b)
{
    const float r = rcp(b), q = a * r;
    return fmaf(fmaf(-q, b, a), r, q);
}

// ---- two fp32 at a time ----
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// a sum in two fp32 numbers (Knuth's exact sum of two, the error carried along):
// about 48 bits, without the fp64 units, which are slow here
struct Sum2 {
    float hi, lo;
};
__device__ __forceinline__ void add(Sum2 &s, float v)
{
    const float t = __fadd_rn(s.hi, v), z = __fsub_rn(t, s.hi);
    const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, z)), __fsub_rn(v, z));
    s.hi = t;
    s.lo = __fadd_rn(s.lo, e);
}
__device__ __forceinline__ void add(Sum2 &s, const Sum2 &o)
{
    add(s, o.hi);
    s.lo = __fadd_rn(s.lo, o.lo);
}
// the sum: infinite (not NaN, as the error term then is) where it is beyond fp32
__device__ __forceinline__ float total(const Sum2 &s)
{
    const float t = s.hi + s.lo;
    return t == t ? t : s.hi;
}
__device__ __forceinline__ void warp_sum2(Sum2 &s)
{
    for (int o = 16; o; o >>= 1) {
        Sum2 b;
        b.hi = __shfl_xor_sync(0xFFFFFFFFu, s.hi, o);
        b.lo = __shfl_xor_sync(0xFFFFFFFFu, s.lo, o);
        add(s, b);
    }
}

} // namespace moe
