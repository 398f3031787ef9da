// ssu_math.cuh -- packed fp32 arithmetic and fast elementary functions of the convolution and
// the per-channel scan.
#pragma once

#include "ssu_common.cuh"

namespace ssu {

// 2^v by the special-function unit (relative error about 2^-22.5); 2^-inf = 0.
__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ float rcp_fast(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// silu(v) = v / (1 + e^-v) of two values by the special-function unit's exponential and
// reciprocal. Relative error below (4 + |v|) 2^-23, from the rounding of v log2(e); a 16-bit
// output's rounding (2^-8 or 2^-11) hides it. The reciprocal flushes what is below 2^-126, so
// that results beyond v = -87.3, where silu is -2^-119, are 0: for 16-bit outputs that is left
// so (numerator and denominator both times 2^-7 would keep them, for one more product: 16 full
// rows of 512 tokens of the scan 271 us instead of 265, of the convolution 39.8 instead of
// 38.9). With kExact, for fp32 outputs, the product's rounding error is carried along
// (6 * 2^-24), and far below zero numerator and denominator are 2^-32 of theirs (the exponent
// less 32 is exact), which keeps every result, the subnormal ones too.
template <bool kExact> __device__ __forceinline__ float2 silu2(float2 v)
{
    const float kLog2e = 1.44269504f, kLog2eLo = 1.92596e-8f, kLn2 = 0.693147181f;
    float2 e;
    if constexpr (kExact) {
        const float2 c = make_float2(fminf(fmaxf(v.x, -126.f), 126.f),
                                     fminf(fmaxf(v.y, -126.f), 126.f));
        const float2 hi = mul2(c, both(-kLog2e));
        const float2 lo = fma2(c, both(-kLog2eLo), fma2(c, both(-kLog2e), make_float2(-hi.x, -hi.y)));
        const bool fx = v.x < -64.f, fy = v.y < -64.f;      // (1 + e^-v is e^-v there)
        const float2 m = add2(hi, make_float2(fx ? -32.f : 0.f, fy ? -32.f : 0.f));
        v = mul2(v, make_float2(fx ? 0x1p-32f : 1.f, fy ? 0x1p-32f : 1.f));
        e = mul2(make_float2(exp2_fast(m.x), exp2_fast(m.y)), fma2(lo, both(kLn2), both(1.f)));
    } else {
        const float2 m = mul2(v, both(-kLog2e));
        e = make_float2(exp2_fast(m.x), exp2_fast(m.y));
    }
    e = add2(e, both(1.f));
    return mul2(v, make_float2(rcp_fast(e.x), rcp_fast(e.y)));
}

}  // namespace ssu
