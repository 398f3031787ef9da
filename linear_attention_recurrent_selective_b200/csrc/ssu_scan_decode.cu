// ssu_scan_decode.cu -- one token of the per-channel selective scan.
//
// For channel d of a row (group g = d / (D / G)) and state n:
//     dt = softplus(dt + dt_bias[d]);  h[d,n] = exp(dt A[d,n]) h[d,n] + dt x[d] B[g,n]
//     out[d] = (sum_n h[d,n] C[g,n] + D[d] x[d]) * silu(z[d])
//
// Bound: memory. The state is read and written once (2 D N elements a row) for one
// exponential and four multiply-adds per state; x, dt, z and out are 1/N of it each.
//
// Layout: a lane holds 4 states of a channel (one 16- or 8-byte access), kLanes lanes a
// channel, and takes kRows batch rows of that channel at a time: A's row (as large as a
// row's fp32 state, but shared by the batch) is read once, kRows independent state loads
// are in flight, and the step sizes -- a softplus each, equal in all lanes of a channel --
// are computed one row per lane and exchanged by shuffles.
#include "ssu_scan.cuh"

namespace ssu {
namespace {

using namespace scan;

constexpr int kThreads = 128;
constexpr int kRows = 4;

template <int N>
__global__ void __launch_bounds__(kThreads)
scan_decode_kernel(const __grid_constant__ ScanArgs a, const int blocks)
{
    using G = Geo<N>;
    constexpr int kS = G::kStates, kL = G::kLanes;
    const int lane = threadIdx.x & 31;
    const int ln = lane % kL;
    const int d = (blockIdx.x % blocks) * (kThreads / kL) + threadIdx.x / kL;
    const int b0 = (blockIdx.x / blocks) * kRows;
    const bool in = d < a.D;                      // whole lanes of a channel drop out together
    const int dc = in ? d : a.D - 1;
    const int n0 = ln * kS;
    const int g = dc / (a.D / a.G);

    int slot[kRows];
    float h[kRows][kS];
    bool live[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int b = b0 + r;
        slot[r] = b < a.active ? (a.idx ? a.idx[b] : b) : -1;
        live[r] = in && slot[r] >= 0 && slot[r] < a.P;
        if (slot[r] >= a.P && d == 0 && ln == 0 && a.err)   // caller bug: skip and report
            atomicOr(a.err, SSU_FLAG_INDEX_RANGE);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        if (live[r])
            load_states<kS>(a.state, a.state_dtype,
                            (int64_t)slot[r] * a.slot_stride + (int64_t)d * N + n0, h[r]);
    float rate[kS];
    load_decay_rates<kS>(a.A, (int64_t)dc * N + n0, rate);
    const float bias = a.dt_bias ? a.dt_bias[dc] : 0.f;
    const float skip = a.Dp ? a.Dp[dc] : 0.f;

    // the step sizes: with at least kRows lanes a channel, lane r of the channel takes row r
    float dt[kRows], x[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        x[r] = live[r] ? ld_f32(a.x, a.x_dtype, (int64_t)(b0 + r) * a.ldx + d) : 0.f;
    if constexpr (kL >= kRows) {
        const int r = ln % kRows;
        float v = b0 + r < a.active ? ld_f32(a.dt, a.dt_dtype, (int64_t)(b0 + r) * a.lddt + dc) : 0.f;
        v += bias;
        v = a.softplus ? softplus_scan(v) : v;
#pragma unroll
        for (int q = 0; q < kRows; ++q)
            dt[q] = __shfl_sync(~0u, v, q, kL);
    } else {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float v = b0 + r < a.active ? ld_f32(a.dt, a.dt_dtype, (int64_t)(b0 + r) * a.lddt + dc)
                                        : 0.f;
            v += bias;
            dt[r] = a.softplus ? softplus_scan(v) : v;
        }
    }

    float y[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        y[r] = 0.f;
        if (live[r]) {
            const int64_t bo = (int64_t)(b0 + r) * a.ldb + (int64_t)g * N + n0;
            const int64_t co = (int64_t)(b0 + r) * a.ldc + (int64_t)g * N + n0;
            const float dtx = dt[r] * x[r];
#pragma unroll
            for (int i = 0; i < kS; ++i) {
                h[r][i] = fmaf(h[r][i], exp2_fast(dt[r] * rate[i]),
                               dtx * ld_f32(a.B, a.bc_dtype, bo + i));
                y[r] = fmaf(h[r][i], ld_f32(a.C, a.bc_dtype, co + i), y[r]);
            }
            store_states<kS>(a.state, a.state_dtype,
                             (int64_t)slot[r] * a.slot_stride + (int64_t)d * N + n0, h[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int o = kL / 2; o > 0; o >>= 1)
            y[r] += __shfl_xor_sync(~0u, y[r], o);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int b = b0 + r;
        if (ln != r % kL || !in || b >= a.active || slot[r] >= a.P)
            continue;
        float v = 0.f;                              // padding row: zero
        if (slot[r] >= 0) {
            v = fmaf(skip, x[r], y[r]);
            if (a.z)
                v *= gate(ld_f32(a.z, a.x_dtype, (int64_t)b * a.ldz + d), a.x_dtype);
        }
        st_f32(a.out, a.x_dtype, (int64_t)b * a.D + d, v);
    }
}

template <int N> int launch_n(const ScanArgs &a, cudaStream_t s)
{
    const int per = kThreads / Geo<N>::kLanes;
    const int blocks = (a.D + per - 1) / per;
    const int64_t grid = (int64_t)blocks * ((a.active + kRows - 1) / kRows);
    if (grid > 0x7fffffffLL)
        return SSU_ERR_SHAPE;
    return launch_kernel(scan_decode_kernel<N>, (unsigned)grid, kThreads, 0, s, a, blocks);
}

}  // namespace

int launch_scan_decode(const ScanArgs &a, cudaStream_t s)
{
    switch (a.N) {
    case 8: return launch_n<8>(a, s);
    case 16: return launch_n<16>(a, s);
    case 32: return launch_n<32>(a, s);
    case 64: return launch_n<64>(a, s);
    case 128: return launch_n<128>(a, s);
    case 256: return launch_n<256>(a, s);
    default: return SSU_ERR_UNSUPPORTED;
    }
}

}  // namespace ssu
