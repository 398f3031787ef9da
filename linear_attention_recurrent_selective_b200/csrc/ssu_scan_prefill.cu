// ssu_scan_prefill.cu -- the per-channel selective scan over the tokens of a prompt.
//
// The recurrence of ssu_scan_decode.cu run over t < L_b with the state held in registers:
//     h[d,n] = exp(dt[t,d] A[d,n]) h[d,n] + dt[t,d] x[t,d] B[t,n]
//     out[t,d] = (sum_n h[d,n] C[t,n] + D[d] x[t,d]) * silu(z[t,d])
// The decay differs for every (channel, state), so there is no product of matrices in it:
// N exponentials and 4 N multiply-adds per (token, channel).
//
// Bound: the special-function unit (16 exponentials a clock and SM, so one clock per
// (token, channel) and SM at N = 16), ahead of memory (x, dt, z, out: 8 bytes).
//
// Layout: a lane holds 4 states (8 at N = 256) of kChan neighbouring channels; a CTA of 4
// warps takes a block of channels of one row and walks its tokens in chunks of TC. Per
// chunk the threads compute dt and dt*x of every (token, channel) once into shared memory
// (a softplus each) with B and C widened beside them; then each warp runs its channels
// through the chunk, reading B and C as 16-byte broadcasts shared by kChan channels; the
// N-sums of 4 tokens are formed together by a transposing butterfly (3 shuffles instead of
// 8 at N = 16); sums go back through shared memory in place of dt, and the threads that
// staged x finish the outputs with 16-byte stores. The next chunk's inputs are loaded into
// registers while the current one is computed. Rows run longest first.
#include "ssu_scan.cuh"

namespace ssu {
namespace {

using namespace scan;

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kChan = 2;

template <int N> struct Tile {
    static constexpr int kCh = kWarps * Geo<N>::kPerWarp * kChan;       // channels of a CTA
    static constexpr int kTok = N <= 64 ? 32 : (N == 128 ? 16 : 8);     // tokens of a chunk
    static constexpr int kVpt = (kTok * kCh / 8 + kThreads - 1) / kThreads;  // 8-vectors a thread
    static constexpr int kBc = kTok * N / 4;                            // B (or C) 4-vectors
    static constexpr int kBpt = (kBc + kThreads - 1) / kThreads;
    static constexpr int kSmem = kTok * kCh * 8 + 2 * kTok * N * 4;
};

// Eight neighbouring elements of a row, as raw bits: two 16-byte loads at most where
// `vec` (the row is 16-byte aligned and all eight exist), else element by element with
// zeros beyond `n`.
struct Raw8 {
    uint4 lo, hi;
};

__device__ __forceinline__ Raw8 load8(const void *p, int dtype, int64_t at, int n, bool vec)
{
    Raw8 r;
    r.lo = make_uint4(0, 0, 0, 0);
    r.hi = r.lo;
    if (n <= 0)
        return r;
    if (dtype == SSU_F32) {
        const float *q = static_cast<const float *>(p) + at;
        if (vec && n >= 8) {
            r.lo = *reinterpret_cast<const uint4 *>(q);
            r.hi = *reinterpret_cast<const uint4 *>(q + 4);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = i < n ? __float_as_uint(q[i]) : 0u;
            r.lo = make_uint4(w[0], w[1], w[2], w[3]);
            r.hi = make_uint4(w[4], w[5], w[6], w[7]);
        }
    } else {
        const uint16_t *q = static_cast<const uint16_t *>(p) + at;
        if (vec && n >= 8) {
            r.lo = *reinterpret_cast<const uint4 *>(q);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = i < n ? q[i] : 0u;
            r.lo = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16,
                              w[6] | w[7] << 16);
        }
    }
    return r;
}

__device__ __forceinline__ void widen8(const Raw8 &r, int dtype, float (&f)[8])
{
    if (dtype == SSU_F32) {
        Vec16<float>::unpack(r.lo, f);
        Vec16<float>::unpack(r.hi, f + 4);
    } else if (dtype == SSU_F16) {
        Vec16<__half>::unpack(r.lo, f);
    } else {
        Vec16<__nv_bfloat16>::unpack(r.lo, f);
    }
}

__device__ __forceinline__ void store8(void *p, int dtype, int64_t at, int n, bool vec,
                                       const float (&f)[8])
{
    if (vec && n >= 8) {
        if (dtype == SSU_F32) {
            uint4 *q = reinterpret_cast<uint4 *>(static_cast<float *>(p) + at);
            q[0] = Vec16<float>::pack(f);
            q[1] = Vec16<float>::pack(f + 4);
        } else if (dtype == SSU_F16) {
            *reinterpret_cast<uint4 *>(static_cast<__half *>(p) + at) = Vec16<__half>::pack(f);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + at) =
                Vec16<__nv_bfloat16>::pack(f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                st_f32(p, dtype, at + i, f[i]);
    }
}

// Sums over the kL lanes of a channel of four values (four tokens), transposing: at each
// of the first two steps a lane hands half of its values to its partner. On return v[0]
// (and v[1] with two lanes) are the sums of the tokens the lane owns; own_token() names
// the first of them.
template <int kL> __device__ __forceinline__ void sum4(float (&v)[4], int ln)
{
    const bool hi = ln & 1;
    const float s0 = hi ? v[0] : v[2], s1 = hi ? v[1] : v[3];
    const float r0 = __shfl_xor_sync(~0u, s0, 1), r1 = __shfl_xor_sync(~0u, s1, 1);
    v[0] = (hi ? v[2] : v[0]) + r0;                 // lane bit 0 set: tokens 2, 3
    v[1] = (hi ? v[3] : v[1]) + r1;
    if constexpr (kL >= 4) {
        const bool h2 = ln & 2;
        const float s = h2 ? v[0] : v[1];
        v[0] = (h2 ? v[1] : v[0]) + __shfl_xor_sync(~0u, s, 2);
#pragma unroll
        for (int o = 4; o < kL; o <<= 1)
            v[0] += __shfl_xor_sync(~0u, v[0], o);
    }
}

template <int kL> __device__ __forceinline__ int own_token(int ln)
{
    return kL >= 4 ? ((ln & 1) << 1) + ((ln >> 1) & 1) : (ln & 1) << 1;
}

// Length used to order the rows: padding and out-of-range rows do (almost) no work.
__device__ __forceinline__ int sched_len(const ScanArgs &a, int b)
{
    const int slot = a.idx ? a.idx[b] : b;
    if (slot < 0 || slot >= a.P)
        return 0;
    const int L = a.ctx ? a.ctx[b] : a.T;
    return L < 0 ? 0 : (L > a.T ? a.T : L);
}

// The row of rank `rank` by decreasing length (ties by index), for up to kRankMax rows.
__device__ __forceinline__ int ranked_row(const ScanArgs &a, int rank, int *s_len, int *s_row)
{
    if (!a.ctx || a.active > kRankMax)
        return rank;
    const int tid = threadIdx.x;
    if (tid < a.active)
        s_len[tid] = sched_len(a, tid);
    __syncthreads();
    if (tid < a.active) {
        const int mine = s_len[tid];
        int r = 0;
        for (int o = 0; o < a.active; ++o)
            r += (s_len[o] > mine) || (s_len[o] == mine && o < tid);
        if (r == rank)
            *s_row = tid;
    }
    __syncthreads();
    return *s_row;
}

template <int N>
__global__ void __launch_bounds__(kThreads)
scan_prefill_kernel(const __grid_constant__ ScanArgs a, const int blocks)
{
    using G = Geo<N>;
    using T = Tile<N>;
    constexpr int kS = G::kStates, kL = G::kLanes, kTok = T::kTok, kCh = T::kCh;
    extern __shared__ __align__(16) uint8_t smem[];
    float2 *const s_dt = reinterpret_cast<float2 *>(smem);              // [kTok][kCh] dt, dt x
    float *const s_B = reinterpret_cast<float *>(smem + kTok * kCh * 8);    // [kTok][N]
    float *const s_C = s_B + kTok * N;
    __shared__ int s_len[kRankMax], s_row;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = ranked_row(a, blockIdx.x / blocks, s_len, &s_row);
    const int d0 = (blockIdx.x % blocks) * kCh;             // the CTA's first channel
    const int per = a.D / a.G;                              // channels of a group
    const int slot = a.idx ? a.idx[b] : b;
    const bool first = blockIdx.x % blocks == 0 && tid == 0;
    if (slot >= a.P) {                                      // caller bug: skip and report
        if (first && a.err)
            atomicOr(a.err, SSU_FLAG_INDEX_RANGE);
        return;
    }
    const int64_t row = (int64_t)b * a.T;                   // the row's first token
    const bool vo = a.vec & 8;
    if (slot < 0) {                                         // padding row: zeros
        if (a.out) {
            const float zero[8] = {};
            for (int64_t v = tid; v < (int64_t)a.T * (kCh / 8); v += kThreads) {
                const int c = d0 + (int)(v % (kCh / 8)) * 8;
                store8(a.out, a.x_dtype, (row + v / (kCh / 8)) * a.D + c, a.D - c, vo, zero);
            }
        }
        return;
    }
    int L = a.T;
    if (a.ctx) {
        L = a.ctx[b];
        if (first && a.err && (L < 0 || L > a.T))
            atomicOr(a.err, L < 0 ? SSU_FLAG_NEGATIVE_LENGTH : SSU_FLAG_CONTEXT_RANGE);
        L = L < 0 ? 0 : (L > a.T ? a.T : L);
    }
    if (L == 0)
        return;

    // the lane's states and decay rates: channels ch, ch + 1 of the CTA, states n0 ..
    const int ln = lane % kL, n0 = ln * kS;
    const int ch = (warp * G::kPerWarp + lane / kL) * kChan;
    float h[kChan][kS], rate[kChan][kS];
#pragma unroll
    for (int c = 0; c < kChan; ++c) {
        const int d = min(d0 + ch + c, a.D - 1);
        load_states<kS>(a.state, a.state_dtype,
                        (int64_t)slot * a.slot_stride + (int64_t)d * N + n0, h[c]);
        load_decay_rates<kS>(a.A, (int64_t)d * N + n0, rate[c]);
    }
    // channels of one CTA may belong to two groups: B and C are staged for the group of
    // its first channel, and a channel of another group reads them from memory (rare: only
    // where a group's channel count is no multiple of kCh)
    const int g0 = d0 / per;
    const bool one_group = (min(d0 + kCh, a.D) - 1) / per == g0;

    // this thread's vectors of a chunk: tokens tv + i * kStep, always the same 8 channels
    constexpr int kStep = kThreads / (kCh / 8);
    const int tv = tid / (kCh / 8), cv = tid % (kCh / 8) * 8, c8 = d0 + cv, left = a.D - c8;
    float bias[8], skip[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        bias[e] = a.dt_bias && e < left ? a.dt_bias[c8 + e] : 0.f;
        skip[e] = a.Dp && e < left ? a.Dp[c8 + e] : 0.f;
    }
    Raw8 rx[T::kVpt], rd[T::kVpt];
    uint4 rB[T::kBpt], rC[T::kBpt];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < T::kVpt; ++i) {
            const int tc = tv + i * kStep, t = t0 + tc;
            const int n = tc < kTok && t < L ? left : 0;
            rx[i] = load8(a.x, a.x_dtype, (row + t) * a.ldx + c8, n, a.vec & 1);
            rd[i] = load8(a.dt, a.dt_dtype, (row + t) * a.lddt + c8, n, a.vec & 2);
        }
#pragma unroll
        for (int i = 0; i < T::kBpt; ++i) {
            const int v = tid + i * kThreads, t = t0 + v / (N / 4), n = (v % (N / 4)) * 4;
            float f[4] = {}, q[4] = {};
            if (v < T::kBc && t < L) {
                const int64_t ob = (row + t) * a.ldb + (int64_t)g0 * N + n;
                const int64_t oc = (row + t) * a.ldc + (int64_t)g0 * N + n;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[e] = ld_f32(a.B, a.bc_dtype, ob + e);
                    q[e] = a.out ? ld_f32(a.C, a.bc_dtype, oc + e) : 0.f;
                }
            }
            rB[i] = Vec16<float>::pack(f);
            rC[i] = Vec16<float>::pack(q);
        }
    };

    fetch(0);
    for (int t0 = 0; t0 < L; t0 += kTok) {
        // ---- stage: dt, dt x, B, C of the chunk; zero steps beyond the row's end
        Raw8 xs[T::kVpt], zs[T::kVpt];
#pragma unroll
        for (int i = 0; i < T::kVpt; ++i) {
            const int tc = tv + i * kStep, t = t0 + tc;
            xs[i] = rx[i];
            if (tc < kTok) {
                float x[8], dt[8];
                widen8(rx[i], a.x_dtype, x);
                widen8(rd[i], a.dt_dtype, dt);
                float4 *const to = reinterpret_cast<float4 *>(s_dt + tc * kCh + cv);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dt[e] += bias[e];
                    dt[e] = a.softplus ? softplus_scan(dt[e]) : dt[e];
                    dt[e] = t < L && e < left ? dt[e] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    to[e / 2] = make_float4(dt[e], dt[e] * x[e], dt[e + 1], dt[e + 1] * x[e + 1]);
                if (a.z)
                    zs[i] = load8(a.z, a.x_dtype, (row + t) * a.ldz + c8, t < L ? left : 0,
                                  a.vec & 4);
            }
        }
#pragma unroll
        for (int i = 0; i < T::kBpt; ++i) {
            const int v = tid + i * kThreads;
            if (v < T::kBc) {
                reinterpret_cast<uint4 *>(s_B)[v] = rB[i];
                reinterpret_cast<uint4 *>(s_C)[v] = rC[i];
            }
        }
        __syncthreads();
        if (t0 + kTok < L)
            fetch(t0 + kTok);

        // ---- run the chunk, four tokens at a time
#pragma unroll 1
        for (int t = 0; t < kTok; t += 4) {
            float y[kChan][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 sd = *reinterpret_cast<const float4 *>(s_dt + (t + u) * kCh + ch);
                const float dt[kChan] = {sd.x, sd.z}, dtx[kChan] = {sd.y, sd.w};
                float Bv[kS], Cv[kS];
#pragma unroll
                for (int i = 0; i < kS; i += 4) {
                    const float4 vb = *reinterpret_cast<const float4 *>(s_B + (t + u) * N + n0 + i);
                    const float4 vc = *reinterpret_cast<const float4 *>(s_C + (t + u) * N + n0 + i);
                    Bv[i] = vb.x, Bv[i + 1] = vb.y, Bv[i + 2] = vb.z, Bv[i + 3] = vb.w;
                    Cv[i] = vc.x, Cv[i + 1] = vc.y, Cv[i + 2] = vc.z, Cv[i + 3] = vc.w;
                }
#pragma unroll
                for (int c = 0; c < kChan; ++c) {
                    if (!one_group) {
                        const int g = min(d0 + ch + c, a.D - 1) / per;
                        const bool ok = t0 + t + u < L;
#pragma unroll
                        for (int i = 0; i < kS; ++i) {
                            Bv[i] = ok ? ld_f32(a.B, a.bc_dtype, (row + t0 + t + u) * a.ldb +
                                                                     (int64_t)g * N + n0 + i)
                                       : 0.f;
                            Cv[i] = ok && a.out
                                        ? ld_f32(a.C, a.bc_dtype, (row + t0 + t + u) * a.ldc +
                                                                      (int64_t)g * N + n0 + i)
                                        : 0.f;
                        }
                    }
                    float acc = 0.f;
#pragma unroll
                    for (int i = 0; i < kS; ++i) {
                        h[c][i] = fmaf(h[c][i], exp2_fast(dt[c] * rate[c][i]), dtx[c] * Bv[i]);
                        acc = fmaf(h[c][i], Cv[i], acc);
                    }
                    y[c][u] = acc;
                }
            }
#pragma unroll
            for (int c = 0; c < kChan; ++c)
                sum4<kL>(y[c], ln);
            __syncwarp();               // the channels' steps are read: the sums replace them
#pragma unroll
            for (int c = 0; c < kChan; ++c) {
                const int u = own_token<kL>(ln);
                if (kL <= 4 || ln < 4)
                    s_dt[(t + u) * kCh + ch + c].x = y[c][0];
                if (kL == 2)
                    s_dt[(t + u + 1) * kCh + ch + c].x = y[c][1];
            }
        }
        __syncthreads();

        // ---- the outputs, by the threads that staged the same (token, channels)
        if (a.out) {
#pragma unroll
            for (int i = 0; i < T::kVpt; ++i) {
                const int tc = tv + i * kStep, t = t0 + tc;
                if (tc < kTok && t < L && left > 0) {
                    float x[8], z[8], o[8];
                    widen8(xs[i], a.x_dtype, x);
                    if (a.z)
                        widen8(zs[i], a.x_dtype, z);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        o[e] = fmaf(skip[e], x[e], s_dt[tc * kCh + cv + e].x);
                        if (a.z)
                            o[e] *= gate(z[e], a.x_dtype);
                    }
                    store8(a.out, a.x_dtype, (row + t) * a.D + c8, left, vo, o);
                }
            }
        }
    }

    if (a.update) {
#pragma unroll
        for (int c = 0; c < kChan; ++c)
            if (d0 + ch + c < a.D)
                store_states<kS>(a.state, a.state_dtype,
                                 (int64_t)slot * a.slot_stride + (int64_t)(d0 + ch + c) * N + n0,
                                 h[c]);
    }
}

template <int N> int launch_n(const ScanArgs &a, cudaStream_t s)
{
    using T = Tile<N>;
    const int blocks = (a.D + T::kCh - 1) / T::kCh;
    const int64_t grid = (int64_t)blocks * a.active;
    if (grid > 0x7fffffffLL)
        return SSU_ERR_SHAPE;
    return launch_kernel(scan_prefill_kernel<N>, (unsigned)grid, kThreads, T::kSmem, s, a, blocks);
}

bool rows16(const void *p, int dtype, int64_t ld)
{
    const int e = dtype == SSU_F32 ? 4 : 2;
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * e) % 16 == 0;
}

}  // namespace

int launch_scan_prefill(ScanArgs a, cudaStream_t s)
{
    a.vec = (rows16(a.x, a.x_dtype, a.ldx) ? 1 : 0) | (rows16(a.dt, a.dt_dtype, a.lddt) ? 2 : 0) |
            (a.z && rows16(a.z, a.x_dtype, a.ldz) ? 4 : 0) |
            (a.out && rows16(a.out, a.x_dtype, a.D) ? 8 : 0);
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
