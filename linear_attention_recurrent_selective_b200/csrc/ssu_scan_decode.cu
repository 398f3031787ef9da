// ssu_scan_decode.cu -- one token of the per-channel selective scan.
//
// For channel d of a row (group g = d / (D / G)) and state n:
//     dt = softplus(dt + dt_bias[d]);  h[d,n] = exp(dt A[d,n]) h[d,n] + dt x[d] B[g,n]
//     out[d] = (sum_n h[d,n] C[g,n] + D[d] x[d]) * silu(z[d])
//
// Bound: memory. The state is read and written once (2 D N elements a row) for one
// exponential and four multiply-adds per state; x, dt, z and out are 1/N of it each.
//
// Measured (B200, 256 rows of 5120 channels, 16 states, fp32 pool, bfloat16 inputs): 33.3 us,
// 0.83 of the copy rate; issue slots are 79 % busy, the conversions of B and C and the
// exchange between lanes ahead of the recurrence itself. Loading each operand where it is
// used, element by element, took 71 us.
//
// Layout: a lane holds 4 states of a channel (one 16- or 8-byte access; 8 at N = 256), kL
// lanes a channel, and takes four batch rows of that channel at a time: A's row (as large as
// a row's fp32 state, but shared by the batch) is read once, and every load of the four rows
// is issued before the first is used. The lanes of a channel share out the four rows: a lane
// loads x, dt and z of its own, forms the step (a softplus), hands it to the others by
// shuffles, gets back the sum over all states from a transposing butterfly, and stores the
// output.
#include "ssu_scan.cuh"

namespace ssu {
namespace {

using namespace scan;

constexpr int kThreads = 128;
constexpr int kRows = 4;

// kS neighbouring elements of B or C as raw bits: one or two accesses where `vec` (groups
// of four are aligned to their size).
template <int kS> struct RawBC {
    uint32_t w[kS];                   // 16-bit types: packed in the first half
};

template <int kS>
__device__ __forceinline__ void load_raw(RawBC<kS> &r, const void *p, int dtype, int64_t at, bool vec)
{
    if (dtype == SSU_F32) {
        const uint32_t *const q = static_cast<const uint32_t *>(p) + at;
#pragma unroll
        for (int i = 0; i < kS; i += 4) {
            if (vec) {
                const uint4 v = *reinterpret_cast<const uint4 *>(q + i);
                r.w[i] = v.x, r.w[i + 1] = v.y, r.w[i + 2] = v.z, r.w[i + 3] = v.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    r.w[i + e] = q[i + e];
            }
        }
    } else {
        const uint16_t *const q = static_cast<const uint16_t *>(p) + at;
#pragma unroll
        for (int i = 0; i < kS; i += 4) {
            if (vec) {
                const uint2 v = *reinterpret_cast<const uint2 *>(q + i);
                r.w[i / 2] = v.x, r.w[i / 2 + 1] = v.y;
            } else {
                r.w[i / 2] = q[i] | (uint32_t)q[i + 1] << 16;
                r.w[i / 2 + 1] = q[i + 2] | (uint32_t)q[i + 3] << 16;
            }
        }
    }
}

template <int kS> __device__ __forceinline__ float2 pair_of(const RawBC<kS> &r, int dtype, int i)
{
    if (dtype == SSU_F32)
        return make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    if (dtype == SSU_BF16)
        return make_float2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xffff0000u));
    __half2 h;
    memcpy(&h, &r.w[i], 4);
    return __half22float2(h);
}

// DT: the type of x, dt, z, B and C where they share it, else -1; ST: fp32 states, else -1.
template <int N, int DT, int ST>
__global__ void __launch_bounds__(kThreads)
scan_decode_kernel(const __grid_constant__ ScanArgs a, const int blocks)
{
    using G = Geo<N>;
    constexpr int kS = G::kStates, kL = G::kLanes, kP = kS / 2;
    constexpr int kOwn = kL >= 4 ? 1 : 4 / kL, kPr = (kOwn + 1) / 2;
    const int xt = DT < 0 ? a.x_dtype : DT, dtt = DT < 0 ? a.dt_dtype : DT;
    const int bct = DT < 0 ? a.bc_dtype : DT, stt = ST < 0 ? a.state_dtype : ST;
    const int ln = threadIdx.x % kL;
    const int d = (blockIdx.x % blocks) * (kThreads / kL) + threadIdx.x / kL;
    const int b0 = (blockIdx.x / blocks) * kRows;
    const bool in = d < a.D;                      // whole lanes of a channel drop out together
    const int dc = in ? d : a.D - 1;
    const int n0 = ln * kS;
    const int64_t at = (int64_t)dc * N + n0, gn = (int64_t)(dc / (a.D / a.G)) * N + n0;

    int slot[kRows];
    bool live[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        slot[r] = b0 + r < a.active ? (a.idx ? a.idx[b0 + r] : b0 + r) : -1;
    // this lane's own rows, in pairs: x, dt and z; rows beyond the batch read the last one's
    const auto row_of = [&](int i) { return min(b0 + own<kL>(ln, i), a.active - 1); };
    float2 x[kPr], dt[kPr], z[kPr];
    const auto two = [&](const void *p, int type, int64_t ld, int i) {
        const int64_t ra = row_of(2 * i), rb = row_of(kOwn > 1 ? 2 * i + 1 : 0);
        const float v = ld_f32(p, type, ra * ld + dc);
        return make_float2(v, kOwn > 1 ? ld_f32(p, type, rb * ld + dc) : v);
    };
#pragma unroll
    for (int p = 0; p < kPr; ++p) {
        x[p] = two(a.x, xt, a.ldx, p);
        dt[p] = two(a.dt, dtt, a.lddt, p);
        if (a.z)
            z[p] = two(a.z, xt, a.ldz, p);
    }
    float h[kRows][kS], rate[kS];
    RawBC<kS> rB[kRows], rC[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        live[r] = slot[r] >= 0 && slot[r] < a.P;
        if (live[r]) {
            load_states<kS>(a.state, stt, (int64_t)slot[r] * a.slot_stride + at, h[r]);
            load_raw<kS>(rB[r], a.B, bct, (int64_t)(b0 + r) * a.ldb + gn, a.vec & 1);
            load_raw<kS>(rC[r], a.C, bct, (int64_t)(b0 + r) * a.ldc + gn, a.vec & 2);
        }
    }
    load_decay_rates<kS>(a.A, at, rate);
    const float bias = a.dt_bias ? a.dt_bias[dc] : 0.f;
    const float skip = a.Dp ? a.Dp[dc] : 0.f;

    float2 dx[kPr];
#pragma unroll
    for (int p = 0; p < kPr; ++p) {
        dt[p] = add2(dt[p], both(bias));
        if (a.softplus)
            dt[p] = softplus2(dt[p]);
        dx[p] = mul2(dt[p], x[p]);
    }
    float y[1][kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const float2 d2 = both(of_item<kL, 1, kPr>(dt, r, 0)), x2 = both(of_item<kL, 1, kPr>(dx, r, 0));
        float2 acc = make_float2(0.f, 0.f);
        if (live[r]) {
#pragma unroll
            for (int i = 0; i < kP; ++i) {
                const float2 e = decay2(d2, make_float2(rate[2 * i], rate[2 * i + 1]));
                const float2 s = fma2(make_float2(h[r][2 * i], h[r][2 * i + 1]), e,
                                      mul2(x2, pair_of<kS>(rB[r], bct, i)));
                acc = fma2(s, pair_of<kS>(rC[r], bct, i), acc);
                h[r][2 * i] = s.x;
                h[r][2 * i + 1] = s.y;
            }
            if (in)
                store_states<kS>(a.state, stt, (int64_t)slot[r] * a.slot_stride + at, h[r]);
        }
        y[0][r] = acc.x + acc.y;
    }
    float2 o[kPr];
    sum_own<kL, 1, kPr>(y, o, ln);
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int r = own<kL>(ln, i), b = b0 + r;
        const int sl = kL >= 4 ? (r & 2 ? (r & 1 ? slot[3] : slot[2]) : (r & 1 ? slot[1] : slot[0]))
                     : kL == 2 ? (ln ? slot[2 * i + 1] : slot[2 * i]) : slot[i];
        if (!in || b >= a.active || (kL > 4 && ln >= 4))
            continue;
        if (sl >= a.P) {                            // caller bug: skip and report
            if (d == 0 && a.err)
                atomicOr(a.err, SSU_FLAG_INDEX_RANGE);
            continue;
        }
        const bool second = i & 1;
        float v = 0.f;                              // padding row: zero
        if (sl >= 0) {
            v = second ? o[i / 2].y : o[i / 2].x;
            if (a.Dp)                               // (0 times an infinite x would be a NaN)
                v = fmaf(skip, second ? x[i / 2].y : x[i / 2].x, v);
            if (a.z)
                v *= gate2(both(second ? z[i / 2].y : z[i / 2].x), xt).x;
        }
        st_f32(a.out, xt, (int64_t)b * a.D + d, v);
    }
}

template <int N, int DT, int ST> int launch_n(const ScanArgs &a, cudaStream_t s)
{
    const int per = kThreads / Geo<N>::kLanes;
    const int blocks = (a.D + per - 1) / per;
    const int64_t grid = (int64_t)blocks * ((a.active + kRows - 1) / kRows);
    if (grid > 0x7fffffffLL)
        return SSU_ERR_SHAPE;
    return launch_kernel(scan_decode_kernel<N, DT, ST>, (unsigned)grid, kThreads, 0, s, a, blocks);
}

template <int N, int DT> int launch_st(const ScanArgs &a, cudaStream_t s)
{
    return a.state_dtype == SSU_F32 ? launch_n<N, DT, SSU_F32>(a, s) : launch_n<N, DT, -1>(a, s);
}

// A type that x, dt, z, B and C share is compiled in.
template <int N> int launch_dt(const ScanArgs &a, cudaStream_t s)
{
    if (a.x_dtype == a.dt_dtype && a.x_dtype == a.bc_dtype) {
        switch (a.x_dtype) {
        case SSU_F32: return launch_st<N, SSU_F32>(a, s);
        case SSU_F16: return launch_st<N, SSU_F16>(a, s);
        case SSU_BF16: return launch_st<N, SSU_BF16>(a, s);
        }
    }
    return launch_st<N, -1>(a, s);
}

}  // namespace

int launch_scan_decode(ScanArgs a, cudaStream_t s)
{
    const int quad = 4 * (a.bc_dtype == SSU_F32 ? 4 : 2);
    const auto quads = [&](const void *p, int64_t ld) {
        return reinterpret_cast<uintptr_t>(p) % quad == 0 && ld % 4 == 0;
    };
    a.vec = (quads(a.B, a.ldb) ? 1 : 0) | (quads(a.C, a.ldc) ? 2 : 0);
    switch (a.N) {
    case 8: return launch_dt<8>(a, s);
    case 16: return launch_dt<16>(a, s);
    case 32: return launch_dt<32>(a, s);
    case 64: return launch_dt<64>(a, s);
    case 128: return launch_dt<128>(a, s);
    case 256: return launch_dt<256>(a, s);
    default: return SSU_ERR_UNSUPPORTED;
    }
}

}  // namespace ssu
