// ssu_scan_prefill.cuh -- the per-channel selective scan over the tokens of a prompt.
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
// Measured (B200, bfloat16, 5120 channels, 16 states): 16 full rows of 512 tokens 265 us, 16
// ragged ones 126 to 155 us by their lengths, against 88 us (full: 174) for the special-function
// operations alone (16 decays, 1 for the softplus, 2 for the gate); that unit is 69 % busy and
// issue slots 65 %. The ragged rows with 8 states 110 us, with 32 250 us; of 2048 channels with
// 64 states 214 us, with 128 337 us. 64 rows of 5 drafted tokens 73 us: a chunk's groups behind
// the row's end are run as well.
// Without the decays' exponentials the full rows take 253 of then 286 us, without softplus
// and gate 233, without the exchanges between lanes 251, and B and C cost nothing: what
// bounds it is the sum of what a warp issues. One row of 4099 tokens of 1000 channels: 79 us
// in 32 segments (770 us in one).
//
// Layout: a lane holds 8 states of a channel, kL = N / 8 lanes a channel; a CTA takes a block
// of neighbouring channels of one row and walks its tokens in chunks of kTok, whose raw
// inputs arrive in shared memory by cp.async one chunk ahead (plain loads where rows are not
// 16-byte aligned), with B and C widened to fp32 beside them: one barrier a chunk. A warp runs
// its channels four tokens at a time. The lanes of a channel share out the four tokens: a
// lane forms the steps dt and dt*x of its own (packed in pairs), hands them to the others by
// shuffles, gets back the sums over all states of its own tokens from a transposing
// butterfly, and finishes and stores their outputs. The next group's steps are formed while
// this one runs. Rows run longest first.
//
// Few rows leave most of the card idle, so a long row may be cut into segments of tokens for
// the CTAs of a cluster and the warps of each. The recurrence is linear in the state: a
// segment started from zero ends in h0, and started from h in exp(A sum dt) h + h0. So every
// team but the first runs its segment from zero without outputs (about 2/3 of the work), the
// ends are exchanged (through distributed shared memory between CTAs), each team folds those
// before it into its true start, and runs its segment again with outputs. The first team
// starts from the true state and runs once; its segment is 2/3 as long, so that the teams
// meet in time.
#pragma once

#include <cooperative_groups.h>

#include "ssu_scan.cuh"

namespace ssu {
namespace {

using namespace scan;
namespace cg = cooperative_groups;

constexpr int kStates = 8;            // of a lane
constexpr int kMinWarps = 16;         // of an SM: at most 128 registers a thread
// Most warps that cutting rows into segments may make, a little above the 2368 that the card
// holds at a time (148 SMs of kMinWarps). A row of 4096 tokens of 5120 channels takes 353 us in
// 2560 warps and 422 in half as many, one of 2560 channels 186 and 210. Twice the warps lose:
// 4099 tokens of 1000 channels 164 us in 4096 against 79, two rows of 2048 tokens of 2048
// channels 135 against 131, four of 5120 channels 541 cut into 5120 warps against 369 uncut
// (but the one row of 5120 channels 322 against 353).
constexpr int kFill = 2700;
constexpr int kMaxParts = 16;         // CTAs of a cluster (above 8 by opt-in)

// CH: neighbouring channels of a lane, 1 or 2. TM: teams of a CTA, each with a segment of the
// row's tokens; one team is the whole CTA, more are a warp each.
template <int N, int CH, int TM> struct Tile {
    static constexpr int kL = N / kStates;                              // lanes of a channel
    static constexpr int kWarps = TM > 1 ? 1 : N == 256 ? 8 / CH : (N >= 32 ? 4 : 4 / CH);
    static constexpr int kThreads = 32 * kWarps;                        // of a team
    // channels of a CTA: a multiple of 8, so that a row of them is whole 16-byte units
    static constexpr int kCh = kThreads / kL * CH;
    static constexpr int kTok = N <= 64 && TM == 1 ? 32 : N <= 128 ? 16 : 8;   // of a chunk
    static constexpr int kOwn = kL >= 4 ? 1 : 4 / kL;                   // tokens of a lane, of 4
    // the lane's values of a group as packed pairs: of its two channels, or of two tokens
    static constexpr int kPr = CH == 2 ? kOwn : (kOwn + 1) / 2;
    // shared memory of a team: B and C widened, two stages of [2][kTok][N]; two stages of raw
    // x, dt, z, B, C. Behind the teams', where rows are split: the end state [kCh][N] and sum
    // of steps [kCh] of each team's segment, and of the CTA's where it has several
    static constexpr int kWide = 2 * kTok * N * 4;
    static constexpr int kFixed = 2 * kWide;
    static constexpr int kEnd = kCh * N + kCh;                          // floats of one end
    static constexpr int kEnds = (TM > 1 ? TM + 1 : 1) * kEnd * 4;
    static_assert(kCh % 8 == 0, "");
};

__host__ __device__ __forceinline__ int esize(int dtype) { return dtype == SSU_F32 ? 4 : 2; }

// Byte offsets of the raw inputs of one chunk.
struct Raw {
    int x, dt, z, B, C, bytes;
};

template <int N, int CH, int TM>
__host__ __device__ __forceinline__ Raw raw_layout(int ex, int ed, int eb, bool z)
{
    using T = Tile<N, CH, TM>;
    Raw r;
    r.x = 0;
    r.dt = T::kTok * T::kCh * ex;
    r.z = r.dt + T::kTok * T::kCh * ed;
    r.B = r.z + (z ? T::kTok * T::kCh * ex : 0);
    r.C = r.B + T::kTok * N * eb;
    r.bytes = r.C + T::kTok * N * eb;
    return r;
}

__device__ __forceinline__ void copy16(void *dst, const void *src, int bytes)
{
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes)
                 : "memory");
}

constexpr int log2_of(int n) { return n <= 1 ? 0 : 1 + log2_of(n / 2); }

// Bring kTok rows of kRow (a power of two) elements (of which the first `left` exist) of
// tokens t0.. into shared memory, zeros beyond token t1 and element `left`. Row t starts at
// element t * ld of src.
template <int kThreads, int kTok, int kRow>
__device__ __forceinline__ void fetch_rows(uint8_t *dst, const void *src, int es, int64_t ld,
                                           int left, int t0, int t1, bool vec, int tid)
{
    const char *const p = static_cast<const char *>(src);
    if (vec) {
        const int lg = es == 4 ? 2 : 3, lp = log2_of(kRow) - lg;        // 2^lp units of a row
        for (int u = tid; u < kTok << lp; u += kThreads) {
            const int t = u >> lp, e = (u & ((1 << lp) - 1)) << lg;
            const int n = t0 + t < t1 ? min(max(left - e, 0), 1 << lg) * es : 0;
            copy16(dst + u * 16, n ? p + ((t0 + t) * ld + e) * es : p, n);
        }
    } else {
        for (int u = tid; u < kTok * kRow; u += kThreads) {
            const int t = u / kRow, e = u % kRow;
            const bool in = t0 + t < t1 && e < left;
            if (es == 4)
                reinterpret_cast<uint32_t *>(dst)[u] =
                    in ? reinterpret_cast<const uint32_t *>(p)[(t0 + t) * ld + e] : 0u;
            else
                reinterpret_cast<uint16_t *>(dst)[u] =
                    in ? reinterpret_cast<const uint16_t *>(p)[(t0 + t) * ld + e] : (uint16_t)0;
        }
    }
}

// Element i of a raw array in shared memory.
__device__ __forceinline__ float elem_at(const uint8_t *raw, int dtype, int i)
{
    if (dtype == SSU_F32)
        return reinterpret_cast<const float *>(raw)[i];
    if (dtype == SSU_F16)
        return __half2float(reinterpret_cast<const __half *>(raw)[i]);
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(raw)[i]);
}

// Elements i and j of a raw array (i even and j = i + 1 where kAdjacent).
template <bool kAdjacent>
__device__ __forceinline__ float2 elems_at(const uint8_t *raw, int dtype, int i, int j)
{
    if constexpr (kAdjacent) {
        if (dtype == SSU_F32)
            return reinterpret_cast<const float2 *>(raw)[i >> 1];
        if (dtype == SSU_F16)
            return __half22float2(reinterpret_cast<const __half2 *>(raw)[i >> 1]);
        return __bfloat1622float2(reinterpret_cast<const __nv_bfloat162 *>(raw)[i >> 1]);
    } else {
        const float v = elem_at(raw, dtype, i);
        return make_float2(v, i == j ? v : elem_at(raw, dtype, j));
    }
}

// Outputs of two neighbouring channels, as one access where `vec` (both exist and the pair
// is aligned).
__device__ __forceinline__ void store_pair(void *p, int dtype, int64_t at, bool two, bool vec,
                                           float2 o)
{
    if (vec && two) {
        if (dtype == SSU_F32)
            *reinterpret_cast<float2 *>(static_cast<float *>(p) + at) = o;
        else if (dtype == SSU_F16)
            *reinterpret_cast<__half2 *>(static_cast<__half *>(p) + at) =
                __floats2half2_rn(o.x, o.y);
        else
            *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p) + at) =
                __floats2bfloat162_rn(o.x, o.y);
    } else {
        st_f32(p, dtype, at, o.x);
        if (two)
            st_f32(p, dtype, at + 1, o.y);
    }
}

// Widen kAll raw elements to fp32; a thread takes what it brought by fetch_rows, so that it
// needs to wait for its own copies only.
template <int kThreads, int kAll>
__device__ __forceinline__ void widen_rows(float *dst, const uint8_t *raw, int dtype, bool vec,
                                           int tid)
{
    if (!vec) {
        for (int u = tid; u < kAll; u += kThreads)
            dst[u] = elem_at(raw, dtype, u);
    } else if (dtype == SSU_F32) {
        for (int u = tid; u < kAll / 4; u += kThreads)
            reinterpret_cast<uint4 *>(dst)[u] = reinterpret_cast<const uint4 *>(raw)[u];
    } else {
        for (int u = tid; u < kAll / 8; u += kThreads) {
            float f[8];
            if (dtype == SSU_F16)
                Vec16<__half>::unpack(reinterpret_cast<const uint4 *>(raw)[u], f);
            else
                Vec16<__nv_bfloat16>::unpack(reinterpret_cast<const uint4 *>(raw)[u], f);
            reinterpret_cast<uint4 *>(dst)[2 * u] = Vec16<float>::pack(f);
            reinterpret_cast<uint4 *>(dst)[2 * u + 1] = Vec16<float>::pack(f + 4);
        }
    }
}

// Length used to order the rows: padding and out-of-range rows do (almost) no work.
__device__ __forceinline__ int sched_len(const ScanArgs &a, int b)
{
    const int L = a.ctx ? a.ctx[b] : a.T;           // (one round trip for both)
    const int slot = a.idx ? a.idx[b] : b;
    if (slot < 0 || slot >= a.P)
        return 0;
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

// What a lane keeps of its channels: states and decay rates as pairs of neighbours.
template <int CH> struct Lane {
    float2 h[CH][kStates / 2], rate[CH][kStates / 2];
    float sum[CH];                              // steps since the segment's start
};

// The CTA's block of channels: all of one group.
struct Block {
    int g, d0, n;                               // group, first channel, channels
};

// Run tokens [t_begin, t_end) of the row through the lane's states; kOut: form the outputs.
// DT: the type of x, dt, z, B and C where they share it and it was compiled in, else -1.
template <int N, int CH, int TM, int DT, bool kOut>
__device__ __forceinline__ void run_tokens(const ScanArgs &a, Lane<CH> &st, uint8_t *smem, int b,
                                           const Block blk, int t_begin, int t_end)
{
    using T = Tile<N, CH, TM>;
    constexpr int kL = T::kL, kTok = T::kTok, kCh = T::kCh, kOwn = T::kOwn, kPr = T::kPr;
    constexpr int kP = kStates / 2, kThreads = T::kThreads;
    const int tid = TM > 1 ? threadIdx.x % kThreads : threadIdx.x;      // in the team
    const int ln = tid % kL, n0 = ln * kStates, ch = tid / kL * CH;
    const int64_t row = (int64_t)b * a.T;

    // rows of this CTA's channels, from token 0 of the row
    const int xt = DT < 0 ? a.x_dtype : DT, dtt = DT < 0 ? a.dt_dtype : DT;
    const int bct = DT < 0 ? a.bc_dtype : DT;
    const int ex = esize(xt), ed = esize(dtt), eb = esize(bct);
    const bool gated = kOut && a.z, skips = kOut && a.Dp, softplus = a.softplus;
    const Raw lay = raw_layout<N, CH, TM>(ex, ed, eb, a.z);
    uint8_t *const raw0 = smem + T::kFixed;
    const char *const gx = static_cast<const char *>(a.x) + (row * a.ldx + blk.d0) * ex;
    const char *const gd = static_cast<const char *>(a.dt) + (row * a.lddt + blk.d0) * ed;
    const char *const gz = static_cast<const char *>(a.z) + (row * a.ldz + blk.d0) * ex;
    const char *const gB = static_cast<const char *>(a.B) + (row * a.ldb + (int64_t)blk.g * N) * eb;
    const char *const gC = static_cast<const char *>(a.C) + (row * a.ldc + (int64_t)blk.g * N) * eb;

    // the lane's channels and, in pairs, its own values of a group: the tokens at 2 p and
    // 2 p + 1 of its list of one channel, or token p of both channels
    const bool live = ch < blk.n, live1 = CH == 2 ? ch + 1 < blk.n : live;
    const int d = blk.d0 + ch;
    float2 bias = make_float2(0.f, 0.f), skip = bias;
    if (a.dt_bias) {
        bias.x = live ? a.dt_bias[d] : 0.f;
        bias.y = CH == 1 ? bias.x : live1 ? a.dt_bias[d + 1] : 0.f;
    }
    const uint32_t keep = skips ? ~0u : 0u;
    if (skips) {
        skip.x = live ? a.Dp[d] : 0.f;
        skip.y = CH == 1 ? skip.x : live1 ? a.Dp[d + 1] : 0.f;
    }
    const auto first_of = [&](int p) { return own<kL>(ln, CH == 2 ? p : 2 * p); };
    const auto second_of = [&](int p) {
        return CH == 2 ? own<kL>(ln, p) : own<kL>(ln, kOwn > 1 ? 2 * p + 1 : 0);
    };

    // (Options are taken by selection: a branch would keep the four stages of a group --
    // steps of the next, scan, sums, outputs -- from being interleaved.)
    // one round ahead of the first chunk only fetches it
    int stage = 1;
    for (int t0 = t_begin - kTok; t0 < t_end; t0 += kTok, stage ^= 1) {
        const uint8_t *const r = raw0 + stage * lay.bytes;
        float *const s_B = reinterpret_cast<float *>(smem + stage * T::kWide);
        float *const s_C = s_B + kTok * N;
        if (t0 >= t_begin) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            widen_rows<kThreads, kTok * N>(s_B, r + lay.B, bct, a.vec & 16, tid);
            if (kOut)
                widen_rows<kThreads, kTok * N>(s_C, r + lay.C, bct, a.vec & 32, tid);
            if (TM > 1)
                __syncwarp();           // the chunk is here, the other stage is free
            else
                __syncthreads();
        }
        if (const int t1 = t0 + kTok; t1 < t_end) {
            uint8_t *const to = raw0 + (stage ^ 1) * lay.bytes;
            fetch_rows<kThreads, kTok, kCh>(to + lay.x, gx, ex, a.ldx, blk.n, t1, t_end, a.vec & 1,
                                            tid);
            fetch_rows<kThreads, kTok, kCh>(to + lay.dt, gd, ed, a.lddt, blk.n, t1, t_end,
                                            a.vec & 2, tid);
            fetch_rows<kThreads, kTok, N>(to + lay.B, gB, eb, a.ldb, N, t1, t_end, a.vec & 16, tid);
            if (gated)
                fetch_rows<kThreads, kTok, kCh>(to + lay.z, gz, ex, a.ldz, blk.n, t1, t_end,
                                                a.vec & 4, tid);
            if (kOut)
                fetch_rows<kThreads, kTok, N>(to + lay.C, gC, eb, a.ldc, N, t1, t_end, a.vec & 32,
                                              tid);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        if (t0 < t_begin)
            continue;
        // the lane's own tokens of the group at t: inputs and steps; none beyond the end
        const auto steps = [&](int t, float2 (&x)[kPr], float2 (&dt)[kPr], float2 (&dx)[kPr]) {
#pragma unroll
            for (int p = 0; p < kPr; ++p) {
                const int ta = t + first_of(p), tb = t + second_of(p);
                const int ia = ta * kCh + ch, ib = tb * kCh + ch + CH - 1;
                x[p] = elems_at<CH == 2>(r + lay.x, xt, ia, ib);
                dt[p] = add2(elems_at<CH == 2>(r + lay.dt, dtt, ia, ib), bias);
                const float2 sp = softplus2(dt[p]);
                dt[p].x = softplus ? sp.x : dt[p].x;
                dt[p].y = softplus ? sp.y : dt[p].y;
                dt[p].x = t0 + ta < t_end ? dt[p].x : 0.f;
                dt[p].y = t0 + tb < t_end ? dt[p].y : 0.f;
                dx[p] = mul2(dt[p], x[p]);
                // for D x; without D 0, which an infinite x times a zero D would not be
                x[p].x = __uint_as_float(__float_as_uint(x[p].x) & keep);
                x[p].y = __uint_as_float(__float_as_uint(x[p].y) & keep);
            }
        };
        float2 x[kPr], dt[kPr], dx[kPr];
        steps(0, x, dt, dx);

#pragma unroll 1
        for (int t = 0; t < kTok; t += 4) {
            float y[CH][4];
            float2 xn[kPr], dtn[kPr], dxn[kPr];
            steps((t + 4) & (kTok - 1), xn, dtn, dxn);      // (the last one's are not used)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float2 Bv[kP], Cv[kP];
#pragma unroll
                for (int i = 0; i < kP; i += 2) {
                    const float4 v = *reinterpret_cast<const float4 *>(s_B + (t + u) * N + n0 + 2 * i);
                    Bv[i] = make_float2(v.x, v.y);
                    Bv[i + 1] = make_float2(v.z, v.w);
                    if (kOut) {
                        const float4 w =
                            *reinterpret_cast<const float4 *>(s_C + (t + u) * N + n0 + 2 * i);
                        Cv[i] = make_float2(w.x, w.y);
                        Cv[i + 1] = make_float2(w.z, w.w);
                    }
                }
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const float2 d2 = both(of_item<kL, CH, kPr>(dt, u, c));
                    const float2 x2 = both(of_item<kL, CH, kPr>(dx, u, c));
                    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < kP; ++i) {
                        const float2 e = decay2(d2, st.rate[c][i]);
                        st.h[c][i] = fma2(st.h[c][i], e, mul2(x2, Bv[i]));
                        if (kOut)
                            acc = i ? fma2(st.h[c][i], Cv[i], acc) : mul2(st.h[c][i], Cv[i]);
                    }
                    if (kOut)
                        y[c][u] = acc.x + acc.y;
                    else
                        st.sum[c] += d2.x;
                }
            }
            if (kOut) {
                float2 o[kPr];
                sum_own<kL, CH, kPr>(y, o, ln);
#pragma unroll
                for (int p = 0; p < kPr; ++p) {
                    const int ta = t + first_of(p), tb = t + second_of(p);
                    o[p] = fma2(skip, x[p], o[p]);
                    // (without a gate this reads x, a tile of the same size, and drops the product)
                    const float2 z = elems_at<CH == 2>(r + (gated ? lay.z : lay.x), xt,
                                                       ta * kCh + ch, tb * kCh + ch + CH - 1);
                    const float2 go = mul2(o[p], gate2(z, xt));
                    o[p].x = gated ? go.x : o[p].x;
                    o[p].y = gated ? go.y : o[p].y;
                    if (live && (kL <= 4 || ln < 4) && t0 + ta < t_end) {
                        const int64_t at = (row + t0 + ta) * a.D + d;
                        if constexpr (CH == 2) {
                            store_pair(a.out, xt, at, live1, a.vec & 8, o[p]);
                        } else {
                            st_f32(a.out, xt, at, o[p].x);
                            if (kOwn > 1 && t0 + tb < t_end)
                                st_f32(a.out, xt, at + (int64_t)(tb - ta) * a.D, o[p].y);
                        }
                    }
                }
            }
#pragma unroll
            for (int p = 0; p < kPr; ++p) {
                x[p] = xn[p];
                dt[p] = dtn[p];
                dx[p] = dxn[p];
            }
        }
    }
}

template <int N, int CH, int TM, int DT>
__global__ void __launch_bounds__(Tile<N, CH, TM>::kThreads * TM,
                                  kMinWarps / (Tile<N, CH, TM>::kWarps * TM))
scan_prefill_kernel(const __grid_constant__ ScanArgs a, const int blocks, const int parts)
{
    using T = Tile<N, CH, TM>;
    constexpr int S = kStates, kP = S / 2, kL = T::kL, kCh = T::kCh, kThreads = T::kThreads;
    constexpr int kEnd = T::kEnd;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_len[kRankMax], s_row;

    const int team = TM > 1 ? threadIdx.x / kThreads : 0;
    const int tid = TM > 1 ? threadIdx.x % kThreads : threadIdx.x;      // in the team
    const int part = blockIdx.x % parts, unit = blockIdx.x / parts;
    const int b = ranked_row(a, unit / blocks, s_len, &s_row);
    const int per = a.D / a.G, of_group = blocks / a.G;     // channels, blocks of a group
    Block blk;
    blk.g = unit % blocks / of_group;
    blk.d0 = blk.g * per + unit % blocks % of_group * kCh;
    blk.n = min(kCh, (blk.g + 1) * per - blk.d0);
    const int len = a.ctx ? a.ctx[b] : a.T;                 // (in one round trip with the slot)
    const int slot = a.idx ? a.idx[b] : b;
    const bool first = unit % blocks == 0 && part == 0 && threadIdx.x == 0;
    if (slot >= a.P) {                                      // caller bug: skip and report
        if (first && a.err)
            atomicOr(a.err, SSU_FLAG_INDEX_RANGE);
        return;
    }
    if (slot < 0) {                                         // padding row: zeros
        if (a.out && part == 0) {
            for (int64_t v = threadIdx.x; v < (int64_t)a.T * kCh; v += kThreads * TM)
                if (v % kCh < blk.n)
                    st_f32(a.out, a.x_dtype, ((int64_t)b * a.T + v / kCh) * a.D + blk.d0 + v % kCh,
                           0.f);
        }
        return;
    }
    if (first && a.err && (len < 0 || len > a.T))
        atomicOr(a.err, len < 0 ? SSU_FLAG_NEGATIVE_LENGTH : SSU_FLAG_CONTEXT_RANGE);
    const int L = len < 0 ? 0 : (len > a.T ? a.T : len);
    if (L == 0)
        return;

    // the lane's states and decay rates
    const int ln = tid % kL, n0 = ln * S, ch = tid / kL * CH;
    const int64_t pool0 = (int64_t)slot * a.slot_stride;
    Lane<CH> s;
    const int seg = part * TM + team, segs = parts * TM;    // this team's segment, of so many
    const bool last = seg + 1 == segs;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int64_t at = ((int64_t)blk.d0 + min(ch + c, blk.n - 1)) * N + n0;
        float h[S] = {}, rate[S];
        load_decay_rates<S>(a.A, at, rate);
        if (seg == 0)
            load_states<S>(a.state, a.state_dtype, pool0 + at, h);
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            s.h[c][i] = make_float2(h[2 * i], h[2 * i + 1]);
            s.rate[c][i] = make_float2(rate[2 * i], rate[2 * i + 1]);
        }
        s.sum[c] = 0.f;
    }

    // segments in units of a chunk: the first 2 shares, the others 3
    cg::cluster_group cluster = cg::this_cluster();
    const int chunks = (L + T::kTok - 1) / T::kTok, shares = 3 * segs - 1;
    const auto bound = [&](int p) {
        return p == 0 ? 0 : min((int)((int64_t)chunks * (3 * p - 1) / shares) * T::kTok, L);
    };
    const int t0 = bound(seg), t1 = last ? L : bound(seg + 1);
    const Raw lay =
        raw_layout<N, CH, TM>(esize(a.x_dtype), esize(a.dt_dtype), esize(a.bc_dtype), a.z);
    const int team_bytes = T::kFixed + 2 * lay.bytes;
    float *const ends = reinterpret_cast<float *>(smem + TM * team_bytes);  // [TM (+ 1)][kEnd]
    const int end_at = ch * N + n0, sum_at = kCh * N + ch;                  // this lane's, in one
    float *const cta_end = TM > 1 ? ends + TM * kEnd : ends;
    const auto put_end = [&](float *end) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
#pragma unroll
            for (int i = 0; i < kP; ++i)
                *reinterpret_cast<float2 *>(end + end_at + c * N + 2 * i) = s.h[c][i];
            if (ln == 0)
                end[sum_at + c] = s.sum[c];
        }
    };
    // the state behind a segment that ends in `end`: `first` replaces it, others let it decay
    // over their steps and add what they end in from zero (one exponential a segment: its mean
    // error, which the decays of single tokens are corrected for, does not gather)
    const auto fold = [&](const float *end, bool replace) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const float sum = end[sum_at + c];
#pragma unroll
            for (int i = 0; i < kP; ++i) {
                const float2 e = *reinterpret_cast<const float2 *>(end + end_at + c * N + 2 * i);
                const float2 f = make_float2(exp2_fast(sum * s.rate[c][i].x),
                                             exp2_fast(sum * s.rate[c][i].y));
                s.h[c][i] = replace ? e : fma2(s.h[c][i], f, e);
            }
            s.sum[c] += sum;
        }
    };
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        if (pass == 1) {
            if (segs == 1)
                break;
            put_end(ends + team * kEnd);
            if (TM > 1) {
                __syncthreads();
                if (team == 0 && part + 1 < parts) {        // the whole CTA's end
                    const Lane<CH> mine = s;
                    for (int q = 1; q < TM; ++q)
                        fold(ends + q * kEnd, false);
                    put_end(cta_end);
                    s = mine;
                }
            }
            if (parts > 1)
                cluster.sync();
            // every end is there: fold those before this segment into its start
            if (seg > 0) {
#pragma unroll 4
                for (int q = 0; q < part; ++q)
                    fold(cluster.map_shared_rank(cta_end, q), q == 0);
                for (int q = 0; q < team; ++q)
                    fold(ends + q * kEnd, part == 0 && q == 0);
            }
            if (parts > 1)
                cluster.barrier_arrive();                   // the others' ends are read
            if (seg == 0)
                break;
        }
        // the first segment starts from the true state and runs once, with outputs; of the
        // others the last needs no end, and all run with outputs in the second pass
        uint8_t *const own_smem = smem + team * team_bytes;
        if (a.out && (pass == 1 || seg == 0))
            run_tokens<N, CH, TM, DT, true>(a, s, own_smem, b, blk, t0, t1);
        else if (pass == 0 ? !last || segs == 1 : last)
            run_tokens<N, CH, TM, DT, false>(a, s, own_smem, b, blk, t0, t1);
    }
    if (parts > 1)
        cluster.barrier_wait();                 // no CTA leaves while its end may be read

    if (a.update && last) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (ch + c < blk.n) {
                float h[S];
#pragma unroll
                for (int i = 0; i < kP; ++i) {
                    h[2 * i] = s.h[c][i].x;
                    h[2 * i + 1] = s.h[c][i].y;
                }
                store_states<S>(a.state, a.state_dtype,
                                pool0 + ((int64_t)blk.d0 + ch + c) * N + n0, h);
            }
    }
}

// How many segments a row is cut into: while that leaves at most kFill warps and every
// segment 64 tokens. s segments cost (5 s - 2) / (3 s - 1) of a row's work (1.6 for 4 and
// more) but run s times as wide, in 6 / (3 s - 1) of its steps, so fewer than four gain
// nothing. `warps`: of the call with one segment a row; `most`: that the form can take.
int segments_of(int64_t warps, int T, int most)
{
    int s = 1;
    while (s < most && warps * s * 2 <= kFill && T >= 128 * s)
        s *= 2;
    return s < 4 ? 1 : s;
}

// Clusters of more than 8 CTAs need the kernel's consent, given once per device.
template <auto kernel> bool wide_clusters()
{
    static std::once_flag once[kMaxDevices];
    static bool ok[kMaxDevices];
    const int dev = current_device();
    if (dev < 0)
        return false;
    std::call_once(once[dev], [&] {
        ok[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                  cudaSuccess;
    });
    return ok[dev];
}

template <int N, int CH, int TM> int64_t blocks_of(const ScanArgs &a)
{
    constexpr int kCh = Tile<N, CH, TM>::kCh;
    return (int64_t)a.G * ((a.D / a.G + kCh - 1) / kCh);
}

// `segs` segments a row, a multiple of TM.
template <int N, int CH, int TM, int DT>
int launch_c(const ScanArgs &a, int segs, cudaStream_t s)
{
    using T = Tile<N, CH, TM>;
    const int64_t blocks = blocks_of<N, CH, TM>(a), units = blocks * a.active;
    const int parts = segs / TM;
    const int64_t grid = units * parts;
    if (blocks > 0x7fffffffLL || grid > 0x7fffffffLL)
        return SSU_ERR_SHAPE;
    const Raw lay = raw_layout<N, CH, TM>(esize(a.x_dtype), esize(a.dt_dtype), esize(a.bc_dtype), a.z);
    // the largest layout (fp32 inputs) sets the kernel's shared-memory limit
    constexpr int kMost =
        TM * (T::kFixed + 2 * (T::kTok * T::kCh * 12 + T::kTok * N * 8)) + T::kEnds;
    const KernelFacts *f = kernel_facts<scan_prefill_kernel<N, CH, TM, DT>>(T::kThreads * TM, kMost);
    if (!f || f->status != SSU_OK)
        return SSU_ERR_CUDA;
    if (parts > 8 && !wide_clusters<scan_prefill_kernel<N, CH, TM, DT>>())
        return SSU_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(T::kThreads * TM);
    cfg.dynamicSmemBytes = TM * (T::kFixed + 2 * lay.bytes) + (segs > 1 ? T::kEnds : 0);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = parts > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, scan_prefill_kernel<N, CH, TM, DT>, a, (int)blocks, parts) ==
                   cudaSuccess
               ? SSU_OK
               : SSU_ERR_CUDA;
}

// Two channels a lane halve the exchanges between lanes and the reads of B and C, at twice
// the registers: better from 64 states on (8 lanes a channel), where that leaves every SM
// eight warps; one channel a lane is better below. Segments go to the CTAs of a cluster, and
// up to 32 states (where a warp's channels still make whole 16-byte units of a row) to the
// four warps of each.
template <int N, int DT> int launch_n(const ScanArgs &a, cudaStream_t s)
{
    const int64_t one = blocks_of<N, 1, 1>(a) * Tile<N, 1, 1>::kWarps;
    if (one > 0x7fffffffLL)
        return SSU_ERR_SHAPE;
    if constexpr (N >= 64) {
        const int64_t two = blocks_of<N, 2, 1>(a) * Tile<N, 2, 1>::kWarps;
        if (two * a.active >= kFill / 2)
            return launch_c<N, 2, 1, DT>(a, 1, s);
    }
    const int64_t warps = one * a.active;
    if constexpr (N <= 32) {
        const int segs = segments_of(warps, a.T, 4 * kMaxParts);
        if (segs > 1)
            return launch_c<N, 1, 4, DT>(a, segs, s);
        return launch_c<N, 1, 1, DT>(a, 1, s);
    }
    return launch_c<N, 1, 1, DT>(a, segments_of(warps, a.T, kMaxParts), s);
}

template <int DT> int launch_dt(const ScanArgs &a, cudaStream_t s)
{
    switch (a.N) {
    case 8: return launch_n<8, DT>(a, s);
    case 16: return launch_n<16, DT>(a, s);
    case 32: return launch_n<32, DT>(a, s);
    case 64: return launch_n<64, DT>(a, s);
    case 128: return launch_n<128, DT>(a, s);
    case 256: return launch_n<256, DT>(a, s);
    default: return SSU_ERR_UNSUPPORTED;
    }
}

}  // namespace
}  // namespace ssu
