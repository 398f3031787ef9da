// ssu_scan.cuh -- shared pieces of the per-channel selective scan (ssu_scan_prefill.cu,
// ssu_scan_decode.cu).
#pragma once

#include "ssu_math.cuh"

namespace ssu {
namespace scan {

// How the N states of a channel are spread over lanes: kStates per lane, kLanes lanes.
template <int N> struct Geo {
    static constexpr int kStates = N > 128 ? N / 32 : 4;
    static constexpr int kLanes = N / kStates;          // 2, 4, 8, 16, 32, 32
    static constexpr int kPerWarp = 32 / kLanes;        // channels of a warp
};

// The decays 2^(s r) of two states over a step s (twice), r = A log2(e). The unit's result is
// low on average (measured: by 5e-9 for exponents around -1/2000, by 2e-8 from -1/1000 to
// -1/2), which a state that remembers hundreds of tokens would gather; 2^-26 added to the
// exponent, in the product's own instruction, leaves at most 1.3e-8 either way. A step of 0
// still gives exactly 1.
__device__ __forceinline__ float2 decay2(float2 s, float2 r)
{
    const float2 v = fma2(s, r, both(0x1p-26f));
    return make_float2(exp2_fast(v.x), exp2_fast(v.y));
}

// log(1 + e^v) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1], for two values. log1p(e) = e
// times the minimax polynomial of degree 8 in e that starts with 1 (relative error 2^-24.8):
// it keeps full relative accuracy for the small steps (e << 1) that a log of 1 + e would
// lose, and leaves the special-function unit, which the scan waits for, one operation (16 full
// rows of 512 tokens 263 us; as 2 atanh(e / (2 + e)), with a reciprocal, 265).
// exp(-|v|) = 2^(hi + lo) with the product's rounding error carried in lo.
__device__ __forceinline__ float2 softplus2(float2 v)
{
    const float kLog2e = 1.44269504f, kLog2eLo = 1.92596e-8f, kLn2 = 0.693147181f;
    const float2 a = make_float2(fmaxf(-fabsf(v.x), -104.f),       // 0 from e^-87.3 on
                                 fmaxf(-fabsf(v.y), -104.f));
    const float2 hi = mul2(a, both(kLog2e));
    const float2 lo = fma2(a, both(kLog2eLo), fma2(a, both(kLog2e), make_float2(-hi.x, -hi.y)));
    const float2 e = mul2(make_float2(exp2_fast(hi.x), exp2_fast(hi.y)),
                          fma2(lo, both(kLn2), both(1.f)));
    float2 p = both(0.00536482083f);
    p = fma2(p, e, both(-0.0300657805f));
    p = fma2(p, e, both(0.0792045146f));
    p = fma2(p, e, both(-0.137538016f));
    p = fma2(p, e, both(0.191536546f));
    p = fma2(p, e, both(-0.248571634f));
    p = fma2(p, e, both(0.33321324f));
    p = fma2(p, e, both(-0.499996483f));
    p = fma2(p, e, both(1.f));
    // max(v, 0), but a NaN stays one
    return fma2(e, p, make_float2(v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y));
}

// silu of two gate values, for outputs of type `out_dtype`.
__device__ __forceinline__ float2 gate2(float2 z, int out_dtype)
{
    return out_dtype == SSU_F32 ? silu2<true>(z) : silu2<false>(z);
}

// The lanes of a channel share out four items (tokens of a prompt, rows of a batch): a lane
// forms the scalars of its own, hands them to the others and gets back their sums.

// Of four items, the i-th that lane ln of a channel owns (lanes beyond the fourth repeat).
template <int kL> __device__ __forceinline__ int own(int ln, int i)
{
    return kL == 1 ? i : kL == 2 ? ln + 2 * i : ln & 3;
}

// Value of item u (of four) and channel c from the lane that owns it; v: this lane's own.
template <int kL, int CH, int kPr>
__device__ __forceinline__ float of_item(const float2 (&v)[kPr], int u, int c)
{
    const int i = kL == 1 ? u : kL == 2 ? u >> 1 : 0;       // its index at the owner
    const float w = CH == 2 ? (c ? v[i].y : v[i].x) : (i & 1 ? v[i >> 1].y : v[i >> 1].x);
    return kL == 1 ? w : __shfl_sync(~0u, w, kL == 2 ? u & 1 : u, kL);
}

// Sums over the lanes of a channel of four values (four items) of CH channels: each lane
// gets those of its own items. At each of the first two steps a lane hands half of its
// values to its partner.
template <int kL, int CH, int kPr>
__device__ __forceinline__ void sum_own(const float (&v)[CH][4], float2 (&s)[kPr], int ln)
{
    float own[CH][4];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if constexpr (kL == 1) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                own[c][u] = v[c][u];
        } else {
            const bool hi = ln & 1;                         // odd items
            const float g0 = __shfl_xor_sync(~0u, hi ? v[c][0] : v[c][1], 1);
            const float g1 = __shfl_xor_sync(~0u, hi ? v[c][2] : v[c][3], 1);
            own[c][0] = (hi ? v[c][1] : v[c][0]) + g0;
            own[c][1] = (hi ? v[c][3] : v[c][2]) + g1;
            if constexpr (kL >= 4) {
                const bool h2 = ln & 2;                     // items 2, 3
                const float g = __shfl_xor_sync(~0u, h2 ? own[c][0] : own[c][1], 2);
                own[c][0] = (h2 ? own[c][1] : own[c][0]) + g;
#pragma unroll
                for (int o = 4; o < kL; o <<= 1)
                    own[c][0] += __shfl_xor_sync(~0u, own[c][0], o);
            }
        }
    }
#pragma unroll
    for (int p = 0; p < kPr; ++p)
        s[p] = CH == 2 ? make_float2(own[0][p], own[CH - 1][p])
                       : make_float2(own[0][2 * p], own[0][kL >= 4 ? 0 : 2 * p + 1]);
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

// The rows A[d, :] times log2(e), so that a decay is one exp2 of a product. A rate of -inf (a
// state that forgets at once) becomes the lowest finite one: it decays by the same 0 over any
// step, and a step of 0, which tokens behind the row's last one are given, is no NaN.
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
#pragma unroll
        for (int e = i; e < i + 4; ++e)
            r[e] = r[e] < -3.402823466e38f ? -3.402823466e38f : r[e];      // (a NaN stays one)
    }
}

}  // namespace scan
}  // namespace ssu
