// ssu_scan.cuh -- shared pieces of the per-channel selective scan (ssu_scan_prefill.cu,
// ssu_scan_decode.cu).
#pragma once

#include "ssu_common.cuh"

namespace ssu {
namespace scan {

// How the N states of a channel are spread over lanes: kStates per lane, kLanes lanes.
template <int N> struct Geo {
    static constexpr int kStates = N > 128 ? N / 32 : 4;
    static constexpr int kLanes = N / kStates;          // 2, 4, 8, 16, 32, 32
    static constexpr int kPerWarp = 32 / kLanes;        // channels of a warp
};

// 2^v by the special-function unit (relative error about 2^-22.5); 2^-inf = 0.
__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// log(1 + e^v) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1]. log1p by Gregory's series
// log1p(e) = 2 (s + s^3/3 + s^5/5 + ...) with s = e / (2 + e) <= 1/3, cut where the next
// term is below 2^-25 of the sum; it keeps full relative accuracy for the small steps
// (e << 1) that a log of 1 + e would lose. exp(-|v|) = 2^(hi + lo) with the product's
// rounding error carried in lo.
__device__ __forceinline__ float softplus_scan(float v)
{
    const float kLog2e = 1.44269504f, kLog2eLo = 1.92596e-8f, kLn2 = 0.693147181f;
    const float a = fmaxf(-fabsf(v), -104.f);           // e^-104 is 0 in fp32
    const float hi = a * kLog2e;
    const float lo = fmaf(a, kLog2e, -hi) + a * kLog2eLo;
    const float e = exp2_fast(hi) * fmaf(lo, kLn2, 1.f);
    const float s = __fdividef(e, 2.f + e), q = s * s;
    float p = 1.f / 13.f;
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    return fmaf(2.f * s, p, v < 0.f ? 0.f : v);         // a NaN stays one
}

// silu with the approximate exponential and division: relative error below 2^-20 for
// |z| < 20, which a 16-bit output's rounding (2^-9 or 2^-11) hides; fp32 outputs take the
// accurate one.
__device__ __forceinline__ float gate(float z, int out_dtype)
{
    return out_dtype == SSU_F32 ? silu_f(z) : __fdividef(z, 1.f + __expf(-z));
}

// kS consecutive states (4, or 8) of a channel, in the pool's type. The element offset is
// a multiple of 4, so that every access is aligned to its size.
template <int kS>
__device__ __forceinline__ void load_states(const void *pool, int dtype, int64_t at, float (&h)[kS])
{
#pragma unroll
    for (int i = 0; i < kS; i += 4) {
        float4 v;
        if (dtype == SSU_F32)
            v = Quad<float>::load(static_cast<const float *>(pool) + at + i);
        else if (dtype == SSU_F16)
            v = Quad<__half>::load(static_cast<const __half *>(pool) + at + i);
        else
            v = Quad<__nv_bfloat16>::load(static_cast<const __nv_bfloat16 *>(pool) + at + i);
        h[i] = v.x;
        h[i + 1] = v.y;
        h[i + 2] = v.z;
        h[i + 3] = v.w;
    }
}

template <int kS>
__device__ __forceinline__ void store_states(void *pool, int dtype, int64_t at, const float (&h)[kS])
{
#pragma unroll
    for (int i = 0; i < kS; i += 4) {
        const float4 v = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
        if (dtype == SSU_F32)
            Quad<float>::store(static_cast<float *>(pool) + at + i, v);
        else if (dtype == SSU_F16)
            Quad<__half>::store(static_cast<__half *>(pool) + at + i, v);
        else
            Quad<__nv_bfloat16>::store(static_cast<__nv_bfloat16 *>(pool) + at + i, v);
    }
}

// The rows A[d, :] times log2(e), so that a decay is one exp2 of a product.
template <int kS>
__device__ __forceinline__ void load_decay_rates(const float *A, int64_t at, float (&r)[kS])
{
    const float kLog2e = 1.44269504f;
#pragma unroll
    for (int i = 0; i < kS; i += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(A + at + i);
        r[i] = v.x * kLog2e;
        r[i + 1] = v.y * kLog2e;
        r[i + 2] = v.z * kLog2e;
        r[i + 3] = v.w * kLog2e;
    }
}

}  // namespace scan
}  // namespace ssu
