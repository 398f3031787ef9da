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
// Layout: a lane holds 4 states (8 at N = 256) of one or two neighbouring channels; a CTA of 4
// warps takes a block of channels of one row and walks its tokens in chunks of kTok, whose
// raw inputs arrive by cp.async one chunk ahead (plain loads where rows are not 16-byte
// aligned). Per chunk the threads compute dt and dt*x of every (token, channel) once into
// shared memory (a softplus each), with B and C widened beside them; each warp runs its
// channels through the chunk, reading B and C as 16-byte broadcasts; the N-sums of 4 tokens are formed together by a transposing butterfly (3
// shuffles instead of 8 at N = 16) and go back in place of dt, from where the outputs are
// finished. Rows run longest first.
//
// Few rows leave most of the card idle, so a long row may be split over a cluster of CTAs,
// each taking a segment of its tokens. The recurrence is linear in the state: a segment
// started from zero ends in h0, and started from h in exp(A sum dt) h + h0. So every CTA
// but the first runs its segment from zero without outputs (about 2/3 of the work), the
// ends are exchanged through distributed shared memory, each CTA folds those before it into
// its true start, and runs its segment again with outputs. The first CTA starts from the
// true state and runs once; its segment is 2/3 as long, so that the CTAs meet in time.
#include <cooperative_groups.h>

#include "ssu_scan.cuh"

namespace ssu {
namespace {

using namespace scan;
namespace cg = cooperative_groups;

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kFill = 592;            // CTAs that give 148 SMs four each
constexpr int kMaxParts = 16;         // CTAs of a cluster (above 8 by opt-in)

// CH: channels of a lane, 1 or 2.
template <int N, int CH> struct Tile {
    // (a multiple of 8, so that a row of the block is whole 16-byte units)
    static constexpr int kCh = kWarps * Geo<N>::kPerWarp * CH;          // channels of a CTA
    static constexpr int kTok = N <= 128 ? 16 : 8;                      // tokens of a chunk
    static constexpr int kPoly = CH == 2 ? 1 : 0;   // pairs of exponentials by polynomial
    static constexpr int kPairs = kCh / 2;                              // channel pairs of a token
    static constexpr int kItems = (kTok * kPairs + kThreads - 1) / kThreads;  // of a thread
    // shared memory: dt and dt x [kTok][kCh], B and C widened [kTok][N], the segment's end
    // state [kCh][N] and step sum [kCh], then two stages of raw x, dt, z, B, C
    static constexpr int kSteps = kTok * kCh * 8;
    static constexpr int kWide = kTok * N * 4;
    static constexpr int kEnds = kCh * N * 4 + kCh * 4;
    static constexpr int kFixed = kSteps + 2 * kWide + kEnds;
};

__host__ __device__ __forceinline__ int esize(int dtype) { return dtype == SSU_F32 ? 4 : 2; }

// Byte offsets of the raw inputs of one chunk.
struct Raw {
    int x, dt, z, B, C, bytes;
};

template <int N, int CH> __host__ __device__ __forceinline__ Raw raw_layout(const ScanArgs &a)
{
    using T = Tile<N, CH>;
    Raw r;
    r.x = 0;
    r.dt = T::kTok * T::kCh * esize(a.x_dtype);
    r.z = r.dt + T::kTok * T::kCh * esize(a.dt_dtype);
    r.B = r.z + (a.z ? T::kTok * T::kCh * esize(a.x_dtype) : 0);
    r.C = r.B + T::kTok * N * esize(a.bc_dtype);
    r.bytes = r.C + T::kTok * N * esize(a.bc_dtype);
    return r;
}

__device__ __forceinline__ void copy16(void *dst, const void *src, int bytes)
{
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes)
                 : "memory");
}

// Bring kTok rows of kRow elements (of which the first `left` exist) of tokens t0.. into
// shared memory, zeros beyond token t1 and element `left`. Row t starts at element
// t * ld of src.
template <int kTok, int kRow>
__device__ __forceinline__ void fetch_rows(uint8_t *dst, const void *src, int es, int64_t ld,
                                           int left, int t0, int t1, bool vec, int tid)
{
    const char *const p = static_cast<const char *>(src);
    if (vec) {
        const int lg = es == 4 ? 2 : 3, per = kRow >> lg;       // 16-byte units of a row
        for (int u = tid; u < kTok * per; u += kThreads) {
            const int t = u / per, e = (u % per) << lg;
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

// Elements 2i and 2i + 1 of a raw array in shared memory.
__device__ __forceinline__ float2 pair_at(const uint8_t *raw, int dtype, int i)
{
    if (dtype == SSU_F32)
        return reinterpret_cast<const float2 *>(raw)[i];
    if (dtype == SSU_F16)
        return __half22float2(reinterpret_cast<const __half2 *>(raw)[i]);
    return __bfloat1622float2(reinterpret_cast<const __nv_bfloat162 *>(raw)[i]);
}

// Outputs of two neighbouring channels, as one access where `vec` (both exist and the pair
// is aligned).
__device__ __forceinline__ void store_pair(void *p, int dtype, int64_t at, bool both, bool vec,
                                           float2 o)
{
    if (vec && both) {
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
        if (both)
            st_f32(p, dtype, at + 1, o.y);
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

// What a lane keeps of its channels: states and decay rates as pairs of neighbours.
template <int N, int CH> struct Lane {
    static constexpr int kP = Geo<N>::kStates / 2;
    float2 h[CH][kP], rate[CH][kP];
    float sum[CH];                              // steps since the segment's start
};

// The CTA's block of channels: all of one group.
struct Block {
    int g, d0, n;                               // group, first channel, channels
};

// Run tokens [t_begin, t_end) of the row through the lane's states; kOut: form the outputs.
template <int N, int CH, bool kOut>
__device__ __forceinline__ void run_tokens(const ScanArgs &a, Lane<N, CH> &s, uint8_t *smem, int b,
                                           const Block blk, int t_begin, int t_end)
{
    using G = Geo<N>;
    using T = Tile<N, CH>;
    constexpr int kS = G::kStates, kP = Lane<N, CH>::kP, kL = G::kLanes;
    constexpr int kTok = T::kTok, kCh = T::kCh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float2 *const s_dt = reinterpret_cast<float2 *>(smem);
    float *const s_B = reinterpret_cast<float *>(smem + T::kSteps);
    float *const s_C = s_B + kTok * N;
    uint8_t *const raw0 = smem + T::kFixed;
    const Raw lay = raw_layout<N, CH>(a);
    const int ln = lane % kL, n0 = ln * kS;
    const int ch = (warp * G::kPerWarp + lane / kL) * CH;
    const int64_t row = (int64_t)b * a.T;

    // rows of this CTA's channels, from token 0 of the row
    const int ex = esize(a.x_dtype), ed = esize(a.dt_dtype), eb = esize(a.bc_dtype);
    const char *const gx = static_cast<const char *>(a.x) + (row * a.ldx + blk.d0) * ex;
    const char *const gd = static_cast<const char *>(a.dt) + (row * a.lddt + blk.d0) * ed;
    const char *const gz = static_cast<const char *>(a.z) + (row * a.ldz + blk.d0) * ex;
    const char *const gB = static_cast<const char *>(a.B) + (row * a.ldb + (int64_t)blk.g * N) * eb;
    const char *const gC = static_cast<const char *>(a.C) + (row * a.ldc + (int64_t)blk.g * N) * eb;

    // this thread's items of a chunk: always the same pair of channels, of tokens
    // tp + i * kStep
    constexpr int kStep = kThreads / T::kPairs;
    const int tp = tid / T::kPairs, pr = tid % T::kPairs, c2 = blk.d0 + 2 * pr;
    const bool in0 = 2 * pr < blk.n, in1 = 2 * pr + 1 < blk.n;
    float2 bias = make_float2(0.f, 0.f), skip = bias;
    if (a.dt_bias) {
        bias.x = in0 ? a.dt_bias[c2] : 0.f;
        bias.y = in1 ? a.dt_bias[c2 + 1] : 0.f;
    }
    if (kOut && a.Dp) {
        skip.x = in0 ? a.Dp[c2] : 0.f;
        skip.y = in1 ? a.Dp[c2 + 1] : 0.f;
    }

    // one round ahead of the first chunk only fetches it
    int stage = 1;
    for (int t0 = t_begin - kTok; t0 < t_end; t0 += kTok, stage ^= 1) {
        if (t0 >= t_begin) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();            // the chunk is here, the other stage is free
        }
        if (const int t1 = t0 + kTok; t1 < t_end) {
            uint8_t *const r = raw0 + (stage ^ 1) * lay.bytes;
            fetch_rows<kTok, kCh>(r + lay.x, gx, ex, a.ldx, blk.n, t1, t_end, a.vec & 1, tid);
            fetch_rows<kTok, kCh>(r + lay.dt, gd, ed, a.lddt, blk.n, t1, t_end, a.vec & 2, tid);
            fetch_rows<kTok, N>(r + lay.B, gB, eb, a.ldb, N, t1, t_end, a.vec & 16, tid);
            if (kOut) {
                if (a.z)
                    fetch_rows<kTok, kCh>(r + lay.z, gz, ex, a.ldz, blk.n, t1, t_end, a.vec & 4,
                                          tid);
                fetch_rows<kTok, N>(r + lay.C, gC, eb, a.ldc, N, t1, t_end, a.vec & 32, tid);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        if (t0 < t_begin)
            continue;
        const uint8_t *const r = raw0 + stage * lay.bytes;

        // ---- steps, and B and C in fp32; zero steps beyond the end
#pragma unroll
        for (int i = 0; i < T::kItems; ++i) {
            const int t = tp + i * kStep;
            if (t < kTok) {
                const float2 x = pair_at(r + lay.x, a.x_dtype, t * T::kPairs + pr);
                float2 dt = add2(pair_at(r + lay.dt, a.dt_dtype, t * T::kPairs + pr), bias);
                if (a.softplus)
                    dt = softplus2(dt);
                dt.x = t0 + t < t_end && in0 ? dt.x : 0.f;
                dt.y = t0 + t < t_end && in1 ? dt.y : 0.f;
                reinterpret_cast<float4 *>(s_dt)[t * T::kPairs + pr] =
                    make_float4(dt.x, dt.x * x.x, dt.y, dt.y * x.y);
            }
        }
        for (int i = tid; i < kTok * N / 2; i += kThreads) {
            reinterpret_cast<float2 *>(s_B)[i] = pair_at(r + lay.B, a.bc_dtype, i);
            if (kOut)
                reinterpret_cast<float2 *>(s_C)[i] = pair_at(r + lay.C, a.bc_dtype, i);
        }
        __syncthreads();

        // ---- run the chunk, four tokens at a time
#pragma unroll 1
        for (int t = 0; t < kTok; t += 4) {
            float y[CH][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float2 sd[CH];                  // dt, dt x
                if constexpr (CH == 2) {
                    const float4 v = *reinterpret_cast<const float4 *>(s_dt + (t + u) * kCh + ch);
                    sd[0] = make_float2(v.x, v.y);
                    sd[1] = make_float2(v.z, v.w);
                } else {
                    sd[0] = s_dt[(t + u) * kCh + ch];
                }
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
                    const float2 dt2 = both(sd[c].x), dx2 = both(sd[c].y);
                    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < kP; ++i) {
                        const float2 v = mul2(dt2, s.rate[c][i]);
                        const float2 e = c * kP + i < T::kPoly
                                             ? exp2_poly2(v)
                                             : make_float2(exp2_fast(v.x), exp2_fast(v.y));
                        s.h[c][i] = fma2(s.h[c][i], e, mul2(dx2, Bv[i]));
                        if (kOut)
                            acc = i ? fma2(s.h[c][i], Cv[i], acc) : mul2(s.h[c][i], Cv[i]);
                    }
                    if (kOut)
                        y[c][u] = acc.x + acc.y;
                    else
                        s.sum[c] += sd[c].x;
                }
            }
            if (kOut) {
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    sum4<kL>(y[c], ln);
                __syncwarp();           // the channels' steps are read: the sums replace them
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const int u = own_token<kL>(ln);
                    if (kL <= 4 || ln < 4)
                        s_dt[(t + u) * kCh + ch + c].x = y[c][0];
                    if (kL == 2)
                        s_dt[(t + u + 1) * kCh + ch + c].x = y[c][1];
                }
            }
        }
        __syncthreads();

        // ---- the outputs, by the threads that formed the same steps
        if (kOut) {
#pragma unroll
            for (int i = 0; i < T::kItems; ++i) {
                const int t = tp + i * kStep;
                if (t < kTok && t0 + t < t_end && in0) {
                    const float4 v = reinterpret_cast<const float4 *>(s_dt)[t * T::kPairs + pr];
                    const float2 x = pair_at(r + lay.x, a.x_dtype, t * T::kPairs + pr);
                    float2 o = fma2(skip, x, make_float2(v.x, v.z));
                    if (a.z) {
                        const float2 z = pair_at(r + lay.z, a.x_dtype, t * T::kPairs + pr);
                        o = mul2(o, make_float2(gate(z.x, a.x_dtype), gate(z.y, a.x_dtype)));
                    }
                    store_pair(a.out, a.x_dtype, (row + t0 + t) * a.D + c2, in1, a.vec & 8, o);
                }
            }
        }
    }
}

template <int N, int CH>
__global__ void __launch_bounds__(kThreads, 4)
scan_prefill_kernel(const __grid_constant__ ScanArgs a, const int blocks, const int parts)
{
    using G = Geo<N>;
    using T = Tile<N, CH>;
    constexpr int kS = G::kStates, kP = Lane<N, CH>::kP, kL = G::kLanes, kCh = T::kCh;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_len[kRankMax], s_row;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int part = blockIdx.x % parts, unit = blockIdx.x / parts;
    const int b = ranked_row(a, unit / blocks, s_len, &s_row);
    const int per = a.D / a.G, of_group = blocks / a.G;     // channels, blocks of a group
    Block blk;
    blk.g = unit % blocks / of_group;
    blk.d0 = blk.g * per + unit % blocks % of_group * kCh;
    blk.n = min(kCh, (blk.g + 1) * per - blk.d0);
    const int slot = a.idx ? a.idx[b] : b;
    const bool first = unit % blocks == 0 && part == 0 && tid == 0;
    if (slot >= a.P) {                                      // caller bug: skip and report
        if (first && a.err)
            atomicOr(a.err, SSU_FLAG_INDEX_RANGE);
        return;
    }
    if (slot < 0) {                                         // padding row: zeros
        if (a.out && part == 0) {
            for (int64_t v = tid; v < (int64_t)a.T * T::kPairs; v += kThreads) {
                const int c = (int)(v % T::kPairs) * 2;
                if (c < blk.n)
                    store_pair(a.out, a.x_dtype,
                               ((int64_t)b * a.T + v / T::kPairs) * a.D + blk.d0 + c,
                               c + 1 < blk.n, a.vec & 8, make_float2(0.f, 0.f));
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

    // the lane's states and decay rates: channels ch .. of the block, states n0 ..
    const int ln = lane % kL, n0 = ln * kS;
    const int ch = (warp * G::kPerWarp + lane / kL) * CH;
    const int64_t pool0 = (int64_t)slot * a.slot_stride + (int64_t)blk.d0 * N + n0;
    Lane<N, CH> s;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int64_t at = (int64_t)min(ch + c, blk.n - 1) * N;
        float h[kS], rate[kS];
        load_decay_rates<kS>(a.A, (int64_t)blk.d0 * N + n0 + at, rate);
        if (part == 0) {
            load_states<kS>(a.state, a.state_dtype, pool0 + at, h);
        } else {
#pragma unroll
            for (int i = 0; i < kS; ++i)
                h[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            s.h[c][i] = make_float2(h[2 * i], h[2 * i + 1]);
            s.rate[c][i] = make_float2(rate[2 * i], rate[2 * i + 1]);
        }
        s.sum[c] = 0.f;
    }

    // this CTA's tokens: segments in units of a chunk, the first 2 shares, the others 3
    cg::cluster_group cluster = cg::this_cluster();
    const int chunks = (L + T::kTok - 1) / T::kTok, shares = 3 * parts - 1;
    const auto bound = [&](int p) {
        return p == 0 ? 0 : min((int)((int64_t)chunks * (3 * p - 1) / shares) * T::kTok, L);
    };
    const int t0 = bound(part), t1 = part + 1 == parts ? L : bound(part + 1);
    const bool last = part + 1 == parts;
    float *const s_end = reinterpret_cast<float *>(smem + T::kSteps + 2 * T::kWide);
    float *const s_sum = s_end + kCh * N;
#pragma unroll 1
    for (int pass = part > 0 && last ? 1 : 0; pass < (part ? 2 : 1); ++pass) {
        if (pass == 1) {
            // every end is there: fold those before this segment into its start
            cluster.sync();
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                for (int q = 0; q < part; ++q) {
                    const float *const end = cluster.map_shared_rank(s_end, q);
                    const float sum = q ? *cluster.map_shared_rank(s_sum + ch + c, q) : 0.f;
#pragma unroll
                    for (int i = 0; i < kP; ++i) {
                        const float2 e =
                            *reinterpret_cast<const float2 *>(end + (ch + c) * N + n0 + 2 * i);
                        float2 &h = s.h[c][i];
                        const float2 d = make_float2(exp2_fast(sum * s.rate[c][i].x),
                                                     exp2_fast(sum * s.rate[c][i].y));
                        h = q ? fma2(h, d, e) : e;
                    }
                }
            }
            cluster.barrier_arrive();           // the others' ends are read
        }
        if (a.out && (pass == 1 || part == 0))
            run_tokens<N, CH, true>(a, s, smem, b, blk, t0, t1);
        else if (pass == 0 || last)
            run_tokens<N, CH, false>(a, s, smem, b, blk, t0, t1);
        if (pass == 0 && parts > 1) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
#pragma unroll
                for (int i = 0; i < kP; ++i)
                    *reinterpret_cast<float2 *>(s_end + (ch + c) * N + n0 + 2 * i) = s.h[c][i];
                if (ln == 0)
                    s_sum[ch + c] = s.sum[c];
            }
        }
    }
    if (parts > 1) {
        if (part == 0) {
            cluster.sync();
            cluster.barrier_arrive();
        }
        cluster.barrier_wait();                 // no CTA leaves while its end may be read
    }

    if (a.update && last) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (ch + c < blk.n) {
                float h[kS];
#pragma unroll
                for (int i = 0; i < kP; ++i) {
                    h[2 * i] = s.h[c][i].x;
                    h[2 * i + 1] = s.h[c][i].y;
                }
                store_states<kS>(a.state, a.state_dtype, pool0 + (int64_t)(ch + c) * N, h);
            }
    }
}

// How a call is spread. A lane takes two channels (it reads B and C once for both and mixes
// in polynomial exponentials) where that leaves every SM at least two CTAs, else one. Rows
// are split into p parts while the CTAs fill less than half of the card's room for them
// and every part keeps at least 64 tokens: that costs (3 p + 2) / (3 p - 1) of a row's work
// and runs it p times as wide, so two parts gain nothing.
int parts_of(int64_t units, int T)
{
    int p = 1;
    while (p < kMaxParts && units * p * 2 <= kFill && T >= 128 * p)
        p *= 2;
    return p < 4 ? 1 : p;
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

template <int N, int CH> int launch_c(const ScanArgs &a, int blocks, cudaStream_t s)
{
    using T = Tile<N, CH>;
    const int64_t units = (int64_t)blocks * a.active;
    const int parts = parts_of(units, a.T);
    if (units * parts > 0x7fffffffLL)
        return SSU_ERR_SHAPE;
    // the largest layout (fp32 inputs) sets the kernel's shared-memory limit
    constexpr int kMost = T::kFixed + 2 * (T::kTok * T::kCh * 12 + T::kTok * N * 8);
    const KernelFacts *f = kernel_facts<scan_prefill_kernel<N, CH>>(kThreads, kMost);
    if (!f || f->status != SSU_OK)
        return SSU_ERR_CUDA;
    if (parts > 8 && !wide_clusters<scan_prefill_kernel<N, CH>>())
        return SSU_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = T::kFixed + 2 * raw_layout<N, CH>(a).bytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = parts > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, scan_prefill_kernel<N, CH>, a, blocks, parts) == cudaSuccess
               ? SSU_OK
               : SSU_ERR_CUDA;
}

template <int N> int launch_n(const ScanArgs &a, cudaStream_t s)
{
    const auto blocks = [&](int ch) { return (int64_t)a.G * ((a.D / a.G + ch - 1) / ch); };
    const int64_t two = blocks(Tile<N, 2>::kCh);
    if (two > 0x3fffffffLL)
        return SSU_ERR_SHAPE;
    // (above 64 states one channel a lane would leave a CTA's rows shorter than 16 bytes)
    if constexpr (N <= 64)
        if (two * a.active < kFill / 2)
            return launch_c<N, 1>(a, (int)blocks(Tile<N, 1>::kCh), s);
    return launch_c<N, 2>(a, (int)two, s);
}

// Whether a row of elements starts and steps on 16 bytes. With `first` (elements), so does
// every further block of that many.
bool rows16(const void *p, int dtype, int64_t ld, int64_t first = 0)
{
    const int e = esize(dtype);
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * e) % 16 == 0 && (first * e) % 16 == 0;
}

}  // namespace

int launch_scan_prefill(ScanArgs a, cudaStream_t s)
{
    if (!a.out)
        a.z = nullptr;
    // a CTA's channels start at a multiple of 8 within their group
    const int64_t per = a.G > 1 ? a.D / a.G : 0;
    const bool pairs = a.out && a.D % 2 == 0 && per % 2 == 0 &&
                       reinterpret_cast<uintptr_t>(a.out) % (2 * esize(a.x_dtype)) == 0;
    a.vec = (rows16(a.x, a.x_dtype, a.ldx, per) ? 1 : 0) |
            (rows16(a.dt, a.dt_dtype, a.lddt, per) ? 2 : 0) |
            (a.z && rows16(a.z, a.x_dtype, a.ldz, per) ? 4 : 0) | (pairs ? 8 : 0) |
            (rows16(a.B, a.bc_dtype, a.ldb, a.N) ? 16 : 0) |
            (a.out && rows16(a.C, a.bc_dtype, a.ldc, a.N) ? 32 : 0);
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
