// ssu_conv_prefill.cu -- the causal conv1d of the raw xBC channels over whole prompts and
// over draft trees, and the commit of the accepted tokens to the conv windows.
//
// The convolution is the one of ssu_conv.cu (Selective State Update page, convState; the
// causal conv1d of the FlashInfer page flashinfer.gdn_fused_decode_step), run over T
// tokens of a row. With in[t] the raw input of token t and in[-1], in[-2], ... the slot's
// window from its newest tap backwards:
//     v[t, c] = bias[c] + sum_k w[c, k] * in[t - (W-1) + k, c],   out = v * sigmoid(v)
// and the window becomes the last W-1 of (window, tokens). Over a draft tree the inputs
// before node t are its ancestors, then the window, which is only read.
//
// Bound: memory. A prompt token moves 2 elements per channel (one read, one written) for
// W + 3 multiply-adds and two special-function operations (the sigmoid); windows are
// touched once per row.
//
// Measured (B200, bfloat16, 5376 channels, width 4; the inputs of a call not in L2): 16 ragged
// rows of up to 512 tokens 24 to 28 us by their lengths, 16 full ones 38.5 us (0.71 of the copy
// rate; DRAM 40 %, the special-function unit 58 % and issue slots 45 % busy: 16 warps an SM,
// whose strips end in waves); one token of each of 256 rows 8.7 us (0.39; 5.7 where the windows
// are in L2); 64 rows of 5 drafted tokens 7.8 us; draft trees of 16 x 128 nodes in half
// precision 18.5 us (0.37: a CTA loads, walks, computes and stores one after the other, in
// little over one wave); the commit of 64 rows 4.5 us (3.1 in L2), of which a launch alone is
// about 2.5. The full rows again: in fp32 62 us (0.89), at width 5 52 us, at 8 76 us, at 16
// 816 us (tap by tap), with channels that are not on 16 bytes 80 us.
//
// Layout: a thread owns VEC neighbouring channels (one access of a row; one channel where
// rows or segments are not aligned) over a strip of up to kStrip tokens, and slides the
// last W-1 inputs through registers, so each input is read once per strip plus W-1 at the
// strip's start. The next tokens' inputs are loaded before the current ones are used. The thread of a row's first strip also owns the window of its channels:
// it alone reads the old taps (a later strip starts at t >= kStrip >= W-1) and it alone
// writes the new ones, after its reads, so the update needs no second launch.
//
// Over a tree the inputs of a node lie anywhere among the row's nodes: a CTA brings all
// nodes' rows of 128 bytes of channels to shared memory, with the window's taps as rows
// before them, so that each input is read from memory once; a thread per node walks its
// ancestors into a list of rows, and the outputs gather by it.
#include "ssu_math.cuh"

namespace ssu {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxNodes = 128;        // nodes of a draft tree
constexpr int kBad = 255;             // in a node's list of rows: it is malformed
constexpr int kStages = 2, kGroup = 8;  // of a thread's ring
constexpr int kStrip = 32;            // tokens of a strip, >= the widest window (16) - 1

template <typename E, int VEC> struct alignas(sizeof(E) * VEC) Chunk {
    E v[VEC];
};

template <typename E, int VEC>
__device__ __forceinline__ Chunk<E, VEC> load_chunk(const void *p, int64_t i)
{
    return *reinterpret_cast<const Chunk<E, VEC> *>(static_cast<const E *>(p) + i);
}

template <typename E> __device__ __forceinline__ float widen(E v);
template <> __device__ __forceinline__ float widen(float v) { return v; }
template <> __device__ __forceinline__ float widen(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

// Two neighbouring 16-bit values.
template <typename E> __device__ __forceinline__ float2 widen_pair(uint32_t w);
template <> __device__ __forceinline__ float2 widen_pair<__half>(uint32_t w)
{
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
}
template <> __device__ __forceinline__ float2 widen_pair<__nv_bfloat16>(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <typename E> __device__ __forceinline__ uint32_t narrow_pair(float a, float b);
template <> __device__ __forceinline__ uint32_t narrow_pair<__half>(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}
template <> __device__ __forceinline__ uint32_t narrow_pair<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}

template <typename E, int VEC>
__device__ __forceinline__ void widen_chunk(const Chunk<E, VEC> &c, float *f)
{
    if constexpr (VEC % 2 == 0 && sizeof(E) == 2) {
        uint32_t w[VEC / 2];
        memcpy(w, &c, sizeof c);
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const float2 v = widen_pair<E>(w[e / 2]);
            f[e] = v.x;
            f[e + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            f[e] = widen<E>(c.v[e]);
    }
}

template <typename E> __device__ __forceinline__ E narrow(float v);
template <> __device__ __forceinline__ float narrow(float v) { return v; }
template <> __device__ __forceinline__ __half narrow(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 narrow(float v)
{
    return __float2bfloat16_rn(v);
}

template <typename E, int VEC>
__device__ __forceinline__ void store_floats(E *p, const float *f)
{
    Chunk<E, VEC> c;
    if constexpr (VEC % 2 == 0 && sizeof(E) == 2) {
        uint32_t w[VEC / 2];
#pragma unroll
        for (int e = 0; e < VEC; e += 2)
            w[e / 2] = narrow_pair<E>(f[e], f[e + 1]);
        memcpy(&c, w, sizeof c);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            c.v[e] = narrow<E>(f[e]);
    }
    *reinterpret_cast<Chunk<E, VEC> *>(p) = c;
}

// v * sigmoid(v) for an output of type E.
template <typename E> __device__ __forceinline__ float conv_silu(float v)
{
    return silu2<sizeof(E) == 4>(both(v)).x;
}

template <typename E, int VEC> __device__ __forceinline__ void silu_vec(float (&v)[VEC])
{
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const float2 r = silu2<sizeof(E) == 4>(make_float2(v[e], v[e + 1]));
            v[e] = r.x;
            v[e + 1] = r.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            v[e] = conv_silu<E>(v[e]);
    }
}

// acc += w * f over VEC channels (packed in pairs).
template <int VEC>
__device__ __forceinline__ void fma_vec(float (&acc)[VEC], const float (&w)[VEC], const float *f)
{
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const float2 r = fma2(make_float2(w[e], w[e + 1]), make_float2(f[e], f[e + 1]),
                                  make_float2(acc[e], acc[e + 1]));
            acc[e] = r.x;
            acc[e + 1] = r.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            acc[e] = fmaf(w[e], f[e], acc[e]);
    }
}

// The widest access (at most 16 bytes) that whole runs of `bytes` contiguous bytes from one
// multiple of `bytes` to the next can be cut into.
constexpr int access(int bytes) { return bytes % 16 == 0 ? 16 : bytes % 8 == 0 ? 8 : bytes % 4 == 0 ? 4 : 2; }

// The window taps of VEC channels from channel c0: every tap in registers, oldest first.
// mode 1: channel-major windows (stride_c = W-1, stride_k = 1), the VEC * (W-1) elements
// contiguous and 16-byte aligned; mode 2: tap-major (stride_c = 1), a vector per tap;
// mode 0: element by element.
template <typename E, int VEC, int W>
__device__ __forceinline__ void load_taps(const ConvPrefillArgs &a, int64_t at, E (&tap)[W - 1][VEC])
{
    const E *p = static_cast<const E *>(a.cstate) + at;
    if (a.win_mode == 1) {
        constexpr int kAll = VEC * (W - 1), kC = access(kAll * sizeof(E)) / sizeof(E);
        Chunk<E, kC> raw[kAll / kC];
#pragma unroll
        for (int j = 0; j < kAll / kC; ++j)
            raw[j] = load_chunk<E, kC>(p, j * kC);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                tap[k][e] = raw[(e * (W - 1) + k) / kC].v[(e * (W - 1) + k) % kC];
    } else if (a.win_mode == 2) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const Chunk<E, VEC> c = load_chunk<E, VEC>(p, k * a.ck);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                tap[k][e] = c.v[e];
        }
    } else {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                tap[k][e] = p[e * a.cc + k * a.ck];
    }
}

template <typename E, int VEC, int W>
__device__ __forceinline__ void store_taps(const ConvPrefillArgs &a, int64_t at,
                                           const E (&tap)[W - 1][VEC])
{
    E *p = static_cast<E *>(a.cstate) + at;
    if (a.win_mode == 1) {
        constexpr int kAll = VEC * (W - 1), kC = access(kAll * sizeof(E)) / sizeof(E);
        Chunk<E, kC> raw[kAll / kC];
#pragma unroll
        for (int e = 0; e < VEC; ++e)
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                raw[(e * (W - 1) + k) / kC].v[(e * (W - 1) + k) % kC] = tap[k][e];
#pragma unroll
        for (int j = 0; j < kAll / kC; ++j)
            *reinterpret_cast<Chunk<E, kC> *>(p + j * kC) = raw[j];
    } else if (a.win_mode == 2) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            Chunk<E, VEC> c;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                c.v[e] = tap[k][e];
            *reinterpret_cast<Chunk<E, VEC> *>(p + k * a.ck) = c;
        }
    } else {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                p[e * a.cc + k * a.ck] = tap[k][e];
    }
}

// The weights of VEC channels from channel c0 (contiguous), tap by tap.
template <typename E, int VEC, int W>
__device__ __forceinline__ void load_weights(const ConvPrefillArgs &a, int c0, float (&w)[W][VEC])
{
    // (single channels are the form for unaligned rows, the weights' among them)
    constexpr int kAll = VEC * W, kC = VEC == 1 ? 1 : access(kAll * sizeof(E)) / sizeof(E);
    Chunk<E, kC> raw[kAll / kC];
#pragma unroll
    for (int j = 0; j < kAll / kC; ++j)
        raw[j] = load_chunk<E, kC>(a.w, (int64_t)c0 * W + j * kC);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
#pragma unroll
        for (int k = 0; k < W; ++k)
            w[k][e] = widen<E>(raw[(e * W + k) / kC].v[(e * W + k) % kC]);
}

// The window after n inputs have passed through it: the last W-1 of (old taps, inputs).
template <typename E, int VEC, int W, typename Input>
__device__ __forceinline__ void new_taps(const E (&old)[W - 1][VEC], E (&nw)[W - 1][VEC], int n,
                                         const Input &input)
{
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int t = n + j - (W - 1);          // < 0: still an old tap
        if (t >= 0) {
            const Chunk<E, VEC> c = input(t);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                nw[j][e] = c.v[e];
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
#pragma unroll
                for (int o = 0; o < W - 1; ++o)
                    if (o == n + j)
                        nw[j][e] = old[o][e];
        }
    }
}

// Where a channel's outputs go: x, B and C are separate dense [batch, T, dim] tensors.
template <typename E> struct OutSeg {
    E *p;               // element (b, t = 0, this channel)
    int64_t ld;
};

template <typename E>
__device__ __forceinline__ OutSeg<E> out_seg(const ConvPrefillArgs &a, int64_t b, int ch)
{
    void *base = a.x;
    int dim = a.x_dim, c = ch;
    if (ch >= a.x_dim) {
        c -= a.x_dim;
        dim = a.bc_dim;
        base = a.B;
        if (c >= a.bc_dim) {
            c -= a.bc_dim;
            base = a.C;
        }
    }
    return OutSeg<E>{static_cast<E *>(base) + b * a.T * dim + c, dim};
}

// A row's length as given, asked for before its slot is looked at so that the two loads share
// one round trip; then clamped, where the row's first thread reports one outside [0, T].
__device__ __forceinline__ int given_length(const int32_t *len, int64_t b, int T)
{
    return len ? len[b] : T;
}
__device__ __forceinline__ int row_length(int L, int T, int over_flag, bool report, int32_t *err)
{
    if (report && err && (L < 0 || L > T))
        atomicOr(err, L < 0 ? SSU_FLAG_NEGATIVE_LENGTH : over_flag);
    return L < 0 ? 0 : (L > T ? T : L);
}

// One thread per (row, strip, vector of channels), widths 2..8; U: tokens loaded together.
template <typename E, int VEC, int W, int U>
__global__ void __launch_bounds__(kThreads)
conv_prefill_kernel(const __grid_constant__ ConvPrefillArgs a, const int groups, const int strips)
{
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int g = (int)(id % groups);
    const int64_t rs = id / groups;
    const int strip = (int)(rs % strips);
    const int64_t b = rs / strips;
    if (b >= a.active)
        return;
    const int c0 = g * VEC, t0 = strip * kStrip;
    const bool first = strip == 0 && g == 0;
    const int len = given_length(a.ctx, b, a.T);
    const int slot = a.idx ? a.idx[b] : (int)b;
    if (slot >= a.P) {                          // caller bug: skip the row and report it
        if (first && a.err)
            atomicOr(a.err, SSU_FLAG_INDEX_RANGE);
        return;
    }
    const OutSeg<E> out = out_seg<E>(a, b, c0);
    if (slot < 0) {                             // padding row: zeros at every token
        float zero[VEC] = {};
        for (int t = t0; t < min(t0 + kStrip, a.T); ++t)
            store_floats<E, VEC>(out.p + t * out.ld, zero);
        return;
    }
    const int L = row_length(len, a.T, SSU_FLAG_CONTEXT_RANGE, first, a.err);
    const int t1 = min(t0 + kStrip, L);
    if (t0 >= L)
        return;

    float w[W][VEC], bias[VEC];
    {
        load_weights<E, VEC, W>(a, c0, w);
        Chunk<E, VEC> rb;
        if (a.bias)
            rb = load_chunk<E, VEC>(a.bias, c0);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            bias[e] = a.bias ? widen<E>(rb.v[e]) : 0.f;
    }
    const E *in = static_cast<const E *>(a.xbc) + b * a.T * a.ldx + c0;
    const int64_t tap_at = (int64_t)slot * a.cslot + (int64_t)c0 * a.cc;

    float win[W - 1][VEC];                      // in[t - (W-1)] .. in[t - 1]
    E old[W - 1][VEC];
    if (strip == 0) {
        load_taps<E, VEC, W>(a, tap_at, old);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                win[j][e] = widen<E>(old[j][e]);
    } else {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            widen_chunk<E, VEC>(load_chunk<E, VEC>(in, (t0 - (W - 1) + j) * a.ldx), win[j]);
    }

    const auto token = [&](const Chunk<E, VEC> &raw, int t) {
        float f[VEC], acc[VEC];
        widen_chunk<E, VEC>(raw, f);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            acc[e] = bias[e];
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            fma_vec<VEC>(acc, w[k], win[k]);
        fma_vec<VEC>(acc, w[W - 1], f);
        if (a.silu)
            silu_vec<E, VEC>(acc);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
#pragma unroll
            for (int k = 0; k + 1 < W - 1; ++k)
                win[k][e] = win[k + 1][e];
            win[W - 2][e] = f[e];
        }
        store_floats<E, VEC>(out.p + t * out.ld, acc);
    };
    int t = t0;
    if constexpr (U > 1) {                      // groups of U tokens, loaded a round ahead
        Chunk<E, VEC> raw[U], next[U];
        if (t + U <= t1) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                raw[u] = load_chunk<E, VEC>(in, (t + u) * a.ldx);
        }
        for (; t + U <= t1; t += U) {
            if (t + 2 * U <= t1) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    next[u] = load_chunk<E, VEC>(in, (t + U + u) * a.ldx);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                token(raw[u], t + u);
#pragma unroll
            for (int u = 0; u < U; ++u)
                raw[u] = next[u];
        }
    }
    for (; t < t1; ++t)
        token(load_chunk<E, VEC>(in, t * a.ldx), t);

    if (strip == 0 && a.update) {
        E nw[W - 1][VEC];
        new_taps<E, VEC, W>(old, nw, L, [&](int p) { return load_chunk<E, VEC>(in, p * a.ldx); });
        store_taps<E, VEC, W>(a, tap_at, nw);
    }
}

// The same for whole 16-byte vectors and long rows: each thread streams its vectors of the
// strip through a ring of its own in shared memory by cp.async, kStages - 1 groups of kGroup
// tokens ahead, so that what is in flight does not take registers (a register prefetch of
// one group kept 14 KB an SM in flight: 60 us for 16 rows of 512 tokens of 5376 channels in
// bfloat16, against 39 us this way, DRAM 38 % busy). Only its own copies are waited for: no barrier.
template <typename E, int W>
__global__ void __launch_bounds__(kThreads, 4)
conv_stream_kernel(const __grid_constant__ ConvPrefillArgs a, const int groups, const int strips)
{
    constexpr int VEC = Vec16<E>::kElems;
    __shared__ Chunk<E, VEC> ring[kStages * kGroup][kThreads];
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int g = (int)(id % groups);
    const int64_t rs = id / groups;
    const int strip = (int)(rs % strips);
    const int64_t b = rs / strips;
    if (b >= a.active)
        return;
    const int c0 = g * VEC, t0 = strip * kStrip;
    const bool first = strip == 0 && g == 0;
    const int len = given_length(a.ctx, b, a.T);
    const int slot = a.idx ? a.idx[b] : (int)b;
    if (slot >= a.P) {                          // caller bug: skip the row and report it
        if (first && a.err)
            atomicOr(a.err, SSU_FLAG_INDEX_RANGE);
        return;
    }
    const OutSeg<E> out = out_seg<E>(a, b, c0);
    if (slot < 0) {                             // padding row: zeros at every token
        float zero[VEC] = {};
        for (int t = t0; t < min(t0 + kStrip, a.T); ++t)
            store_floats<E, VEC>(out.p + t * out.ld, zero);
        return;
    }
    const int L = row_length(len, a.T, SSU_FLAG_CONTEXT_RANGE, first, a.err);
    const int t1 = min(t0 + kStrip, L);
    if (t0 >= L)
        return;

    const E *in = static_cast<const E *>(a.xbc) + b * a.T * a.ldx + c0;
    const uint32_t mine = (uint32_t)__cvta_generic_to_shared(&ring[0][threadIdx.x]);
    const auto fetch = [&](int t, int stage) {  // tokens t .. t + kGroup - 1 of the strip
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
            if (t + u < t1)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 mine + (stage * kGroup + u) * (kThreads * 16)),
                             "l"(in + (t + u) * a.ldx)
                             : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s)
        fetch(t0 + s * kGroup, s);

    float w[W][VEC], bias[VEC], win[W - 1][VEC];
    load_weights<E, VEC, W>(a, c0, w);
    Chunk<E, VEC> rb;
    if (a.bias)
        rb = load_chunk<E, VEC>(a.bias, c0);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        bias[e] = a.bias ? widen<E>(rb.v[e]) : 0.f;
    const int64_t tap_at = (int64_t)slot * a.cslot + (int64_t)c0 * a.cc;
    if (strip == 0) {
        E old[W - 1][VEC];
        load_taps<E, VEC, W>(a, tap_at, old);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                win[j][e] = widen<E>(old[j][e]);
        // the window's new taps: the last W-1 of (old taps, tokens)
        if (a.update) {
            E nw[W - 1][VEC];
            new_taps<E, VEC, W>(old, nw, L, [&](int t) {
                return load_chunk<E, VEC>(in, t * a.ldx);
            });
            store_taps<E, VEC, W>(a, tap_at, nw);
        }
    } else {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            widen_chunk<E, VEC>(load_chunk<E, VEC>(in, (t0 - (W - 1) + j) * a.ldx), win[j]);
    }

    const auto token = [&](const Chunk<E, VEC> &raw, int t) {
        float f[VEC], acc[VEC];
        widen_chunk<E, VEC>(raw, f);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            acc[e] = bias[e];
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            fma_vec<VEC>(acc, w[k], win[k]);
        fma_vec<VEC>(acc, w[W - 1], f);
        if (a.silu)
            silu_vec<E, VEC>(acc);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
#pragma unroll
            for (int k = 0; k + 1 < W - 1; ++k)
                win[k][e] = win[k + 1][e];
            win[W - 2][e] = f[e];
        }
        store_floats<E, VEC>(out.p + t * out.ld, acc);
    };
    int stage = 0, t = t0;
    for (; t < t1; t += kGroup) {
        fetch(t + (kStages - 1) * kGroup, stage == 0 ? kStages - 1 : stage - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        if (t + kGroup <= t1) {                 // (whole groups: the window moves by renaming)
#pragma unroll
            for (int u = 0; u < kGroup; ++u)
                token(ring[stage * kGroup + u][threadIdx.x], t + u);
        } else {
#pragma unroll 1
            for (int u = 0; t + u < t1; ++u)
                token(ring[stage * kGroup + u][threadIdx.x], t + u);
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// One token a row (T = 1), half vectors: a thread takes the same channels of kRows rows, so
// that their weights are read once, with every load of both rows issued before the first is
// used and few enough registers for one wave of 256 rows of 5376 channels. The windows are
// most of the traffic.
template <typename E, int VEC, int W>
__global__ void __launch_bounds__(kThreads, 6)
conv_token_kernel(const __grid_constant__ ConvPrefillArgs a, const int groups)
{
    constexpr int kRows = 2;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int g = (int)(id % groups), c0 = g * VEC;
    const int64_t b0 = id / groups * kRows;
    if (b0 >= a.active)
        return;
    int slot[kRows], len[kRows];
    bool live[kRows];
    Chunk<E, VEC> x[kRows];
    E tap[kRows][W - 1][VEC];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int64_t b = b0 + r;
        len[r] = b < a.active ? given_length(a.ctx, b, 1) : 0;
        slot[r] = b < a.active ? (a.idx ? a.idx[b] : (int)b) : a.P;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int64_t b = b0 + r;
        live[r] = slot[r] >= 0 && slot[r] < a.P;
        if (live[r])
            live[r] = row_length(len[r], 1, SSU_FLAG_CONTEXT_RANGE, g == 0, a.err) == 1;
        else if (b < a.active && slot[r] >= 0 && g == 0 && a.err)
            atomicOr(a.err, SSU_FLAG_INDEX_RANGE);      // caller bug: skip and report
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        if (live[r]) {
            x[r] = load_chunk<E, VEC>(a.xbc, (b0 + r) * a.ldx + c0);
            load_taps<E, VEC, W>(a, (int64_t)slot[r] * a.cslot + (int64_t)c0 * a.cc, tap[r]);
        }
    float w[W][VEC], bias[VEC];
    load_weights<E, VEC, W>(a, c0, w);
    Chunk<E, VEC> rb;
    if (a.bias)
        rb = load_chunk<E, VEC>(a.bias, c0);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        bias[e] = a.bias ? widen<E>(rb.v[e]) : 0.f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (!live[r] && slot[r] >= 0)           // past the batch or the pool, or length 0
            continue;
        float acc[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            acc[e] = slot[r] < 0 ? 0.f : bias[e];       // padding row: zero
        if (live[r]) {
            float f[VEC];
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    f[e] = widen<E>(tap[r][k][e]);
                fma_vec<VEC>(acc, w[k], f);
            }
            widen_chunk<E, VEC>(x[r], f);
            fma_vec<VEC>(acc, w[W - 1], f);
            if (a.silu)
                silu_vec<E, VEC>(acc);
            if (a.update) {
                E nw[W - 1][VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
#pragma unroll
                    for (int k = 0; k + 1 < W - 1; ++k)
                        nw[k][e] = tap[r][k + 1][e];
                    nw[W - 2][e] = x[r].v[e];
                }
                store_taps<E, VEC, W>(a, (int64_t)slot[r] * a.cslot + (int64_t)c0 * a.cc, nw);
            }
        }
        const OutSeg<E> out = out_seg<E>(a, b0 + r, c0);
        store_floats<E, VEC>(out.p, acc);
    }
}

// Every other width (1, 9..16): a thread per (row, strip, channel) that reads each tap
// where it lies. Same ownership of the windows.
template <typename E>
__global__ void __launch_bounds__(kThreads)
conv_prefill_any_kernel(const __grid_constant__ ConvPrefillArgs a, const int channels,
                        const int strips)
{
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int c = (int)(id % channels);
    const int64_t rs = id / channels;
    const int strip = (int)(rs % strips);
    const int64_t b = rs / strips;
    if (b >= a.active)
        return;
    const int t0 = strip * kStrip, W = a.width;
    const bool first = strip == 0 && c == 0;
    const int len = given_length(a.ctx, b, a.T);
    const int slot = a.idx ? a.idx[b] : (int)b;
    if (slot >= a.P) {
        if (first && a.err)
            atomicOr(a.err, SSU_FLAG_INDEX_RANGE);
        return;
    }
    const OutSeg<E> out = out_seg<E>(a, b, c);
    if (slot < 0) {
        for (int t = t0; t < min(t0 + kStrip, a.T); ++t)
            out.p[t * out.ld] = narrow<E>(0.f);
        return;
    }
    const int L = row_length(len, a.T, SSU_FLAG_CONTEXT_RANGE, first, a.err);
    const int t1 = min(t0 + kStrip, L);
    if (t0 >= L)
        return;
    const E *in = static_cast<const E *>(a.xbc) + b * a.T * a.ldx + c;
    const E *w = static_cast<const E *>(a.w) + (int64_t)c * W;
    const float bias = a.bias ? widen<E>(static_cast<const E *>(a.bias)[c]) : 0.f;
    E *tap = static_cast<E *>(a.cstate) + (int64_t)slot * a.cslot + (int64_t)c * a.cc;
    for (int t = t0; t < t1; ++t) {
        float acc = bias;
        for (int k = W - 1, at = t; k >= 0; --k, --at)
            acc = fmaf(widen<E>(w[k]),
                       at >= 0 ? widen<E>(in[at * a.ldx]) : widen<E>(tap[(at + W - 1) * a.ck]), acc);
        out.p[t * out.ld] = narrow<E>(a.silu ? conv_silu<E>(acc) : acc);
    }
    if (strip == 0 && a.update)
        for (int j = 0; j < W - 1; ++j) {       // ascending: a tap is read before it is replaced
            const int t = L + j - (W - 1);
            tap[j * a.ck] = t >= 0 ? in[t * a.ldx] : tap[(L + j) * a.ck];
        }
}

// A CTA per (row, 128 bytes of channels) of a draft tree of up to kMaxNodes nodes. W: the
// width, or 0 for any.
template <typename E, int W>
__global__ void __launch_bounds__(kThreads, 7)
conv_tree_kernel(const __grid_constant__ ConvPrefillArgs a, const int blocks, const bool vec)
{
    constexpr int V = Vec16<E>::kElems, kUnits = 8, kCh = kUnits * V;
    constexpr int kMaxW = W ? W : 16;
    __shared__ __align__(16) E s_in[(kMaxNodes + kMaxW - 1) * kCh];
    constexpr int kRowB = W && W <= 4 ? 4 : 16;
    __shared__ __align__(4) uint8_t s_row[kMaxNodes][kRowB];    // rows of the inputs, newest first
    __shared__ int s_par[kMaxNodes];
    const int width = W ? W : a.width, taps = width - 1;
    const int b = blockIdx.x / blocks, tid = threadIdx.x;
    const int c0 = (blockIdx.x % blocks) * kCh, channels = a.x_dim + 2 * a.bc_dim;
    const bool first = blockIdx.x % blocks == 0 && tid == 0;
    const int len = given_length(a.ctx, b, a.T);
    const int slot = a.idx ? a.idx[b] : b;
    if (slot >= a.P) {                          // caller bug: skip the row and report it
        if (first && a.err)
            atomicOr(a.err, SSU_FLAG_INDEX_RANGE);
        return;
    }
    // this thread's unit of V channels, and where its outputs go
    const int u = tid % kUnits, cu = c0 + u * V;
    const OutSeg<E> seg = out_seg<E>(a, b, min(cu, channels - 1));
    const auto store = [&](int t, const float (&f)[V]) {
        if (vec) {                              // whole and inside one segment
            if (cu < channels)
                store_floats<E, V>(seg.p + t * seg.ld, f);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (cu + e < channels) {
                    const OutSeg<E> o = out_seg<E>(a, b, cu + e);
                    o.p[t * o.ld] = narrow<E>(f[e]);
                }
        }
    };
    if (slot < 0) {                             // padding row: zeros
        const float zero[V] = {};
        for (int t = tid / kUnits; t < a.T; t += kThreads / kUnits)
            store(t, zero);
        return;
    }
    const int L = row_length(len, a.T, SSU_FLAG_CONTEXT_RANGE, first, a.err);
    if (L == 0)
        return;

    const E *const in = static_cast<const E *>(a.xbc) + (int64_t)b * a.T * a.ldx + c0;
    const int left = min(kCh, channels - c0);
    if (vec) {
        for (int i = tid; i < L * kUnits; i += kThreads) {
            const int t = i / kUnits, e = i % kUnits * V;
            if (e < left) {
                const uint32_t d = (uint32_t)__cvta_generic_to_shared(s_in + (taps + t) * kCh + e);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d),
                             "l"(in + t * a.ldx + e)
                             : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    } else {
        for (int i = tid; i < L * kCh; i += kThreads)
            if (i % kCh < left)
                s_in[(taps + i / kCh) * kCh + i % kCh] = in[i / kCh * a.ldx + i % kCh];
    }
    const E *const tap = static_cast<const E *>(a.cstate) + (int64_t)slot * a.cslot +
                         (int64_t)c0 * a.cc;
    for (int i = tid; i < taps * kCh; i += kThreads)
        if (i % kCh < left)
            s_in[i] = tap[i % kCh * a.cc + i / kCh * a.ck];
    if (tid < L)
        s_par[tid] = a.parents[(int64_t)b * a.T + tid];

    float w[W ? W : 1][V], bias[V];
    if (vec) {                                  // (a unit beyond the last repeats it)
        const int c = min(cu, channels - V);
        Chunk<E, V> rb;
        if (a.bias)
            rb = load_chunk<E, V>(a.bias, c);
#pragma unroll
        for (int e = 0; e < V; ++e)
            bias[e] = a.bias ? widen<E>(rb.v[e]) : 0.f;
        if constexpr (W > 0)
            load_weights<E, V, W>(a, c, w);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = min(cu + e, channels - 1);
            bias[e] = a.bias ? widen<E>(static_cast<const E *>(a.bias)[c]) : 0.f;
            if constexpr (W > 0) {
#pragma unroll
                for (int k = 0; k < W; ++k)
                    w[k][e] = widen<E>(static_cast<const E *>(a.w)[(int64_t)c * W + k]);
            }
        }
    }
    __syncthreads();
    // the rows of a node's inputs: nodes from row `taps` on, taps before them (so a parent of
    // -1 is the newest tap). A parent outside [-1, L) marks the node as malformed; the walk
    // takes width - 1 steps whatever the parents hold.
    if (tid < L) {
        int at = tid;
        bool bad = false;
        for (int k = 0; k < width; ++k) {
            s_row[tid][k] = (uint8_t)(at + taps);
            if (k + 1 < width) {
                if (at >= 0) {
                    at = s_par[at];
                    if (at < -1 || at >= L) {
                        bad = true;
                        at = -1;
                    }
                } else {
                    --at;
                }
            }
        }
        if (bad)
            s_row[tid][0] = kBad;               // (no row has this number)
        if (bad && c0 == 0 && a.err)
            atomicOr(a.err, SSU_FLAG_TREE);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();

    for (int t = tid / kUnits; t < L; t += kThreads / kUnits) {
        float acc[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            acc[e] = bias[e];
        const auto add = [&](int row, const float (&wk)[V]) {
            float f[V];
            widen_chunk<E, V>(load_chunk<E, V>(s_in, row * kCh + u * V), f);
            fma_vec<V>(acc, wk, f);
        };
        const uint32_t rows = *reinterpret_cast<const uint32_t *>(s_row[t]);
        if ((rows & 255) == kBad) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                acc[e] = 0.f;
            store(t, acc);
            continue;
        }
        if constexpr (W > 0) {
#pragma unroll
            for (int k = 0; k < W; ++k)
                add(rows >> (8 * (W - 1 - k)) & 255, w[k]);
        } else {
            for (int k = 0; k < width; ++k) {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    w[0][e] = widen<E>(
                        static_cast<const E *>(a.w)[(int64_t)min(cu + e, channels - 1) * width + k]);
                add(s_row[t][width - 1 - k], w[0]);
            }
        }
        if (a.silu)
            silu_vec<E, V>(acc);
        store(t, acc);
    }
}

// Commit: the window becomes the last W-1 of (window, first k_b accepted tokens). A block
// covers kThreads vectors of one row's channels; all its threads check the row's ids.
template <typename E, int VEC, int W>
__global__ void __launch_bounds__(kThreads)
conv_replay_kernel(const __grid_constant__ ConvPrefillArgs a, const int groups, const int blocks)
{
    const int b = blockIdx.x / blocks, part = blockIdx.x % blocks;
    const bool first = part == 0 && threadIdx.x == 0;
    const int most = a.nodes ? a.max_accept : a.T;
    const int len = given_length(a.ctx, b, most);
    const int slot = a.idx ? a.idx[b] : b;
    if (slot < 0)
        return;
    if (slot >= a.P) {
        if (first && a.err)
            atomicOr(a.err, SSU_FLAG_INDEX_RANGE);
        return;
    }
    const int k = row_length(len, most, SSU_FLAG_ACCEPTED_RANGE, first, a.err);
    if (k == 0)
        return;
    const int32_t *ids = a.nodes ? a.nodes + (int64_t)b * a.max_accept : nullptr;
    if (ids) {
        bool bad = false;
        for (int i = threadIdx.x; i < k; i += kThreads)
            bad |= ids[i] < 0 || ids[i] >= a.T;
        if (__syncthreads_or(bad)) {
            if (first && a.err)
                atomicOr(a.err, SSU_FLAG_TREE);
            return;
        }
    }
    const int g = part * kThreads + threadIdx.x;
    if (g >= groups)
        return;
    const int c0 = g * VEC;
    const E *in = static_cast<const E *>(a.xbc) + (int64_t)b * a.T * a.ldx + c0;
    const int64_t tap_at = (int64_t)slot * a.cslot + (int64_t)c0 * a.cc;
    if constexpr (W > 0) {
        E old[W - 1][VEC], nw[W - 1][VEC];
        if (k < W - 1)
            load_taps<E, VEC, W>(a, tap_at, old);
        new_taps<E, VEC, W>(old, nw, k, [&](int t) {
            return load_chunk<E, VEC>(in, (ids ? ids[t] : t) * a.ldx);
        });
        store_taps<E, VEC, W>(a, tap_at, nw);
    } else {
        E *tap = static_cast<E *>(a.cstate) + tap_at;
        const int w1 = a.width - 1;
        for (int j = 0; j < w1; ++j) {          // ascending: a tap is read before it is replaced
            const int t = k + j - w1;
            tap[j * a.ck] = t >= 0 ? in[(ids ? ids[t] : t) * a.ldx] : tap[(k + j) * a.ck];
        }
    }
}

bool aligned(const void *p, int n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// Whether whole 16-byte vectors of channels can be used: every row of the input, the
// weights and each output segment start and step on 16 bytes.
template <typename E> bool vector_rows(const ConvPrefillArgs &a)
{
    constexpr int V = Vec16<E>::kElems;
    return a.x_dim % V == 0 && a.bc_dim % V == 0 && a.ldx % V == 0 && aligned(a.xbc, 16) &&
           (!a.w || aligned(a.w, 16)) && (!a.bias || aligned(a.bias, 16)) &&
           (!a.x || aligned(a.x, 16)) && (!a.B || aligned(a.B, 16)) && (!a.C || aligned(a.C, 16));
}

template <typename E> int window_mode(const ConvPrefillArgs &a)
{
    constexpr int V = Vec16<E>::kElems;
    if (a.width < 2 || !aligned(a.cstate, 16) || a.cslot % V != 0)
        return 0;
    if (a.cc == a.width - 1 && a.ck == 1)
        return 1;
    if (a.cc == 1 && (a.ck % V == 0 || a.width == 2))
        return 2;
    return 0;
}

template <typename E, int VEC, int W>
int launch_w(const ConvPrefillArgs &a, cudaStream_t s)
{
    const int groups = (a.x_dim + 2 * a.bc_dim) / VEC;
    const int strips = (a.T + kStrip - 1) / kStrip;
    const int64_t blocks = ((int64_t)groups * strips * a.active + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL)
        return SSU_ERR_SHAPE;
    // few tokens want few registers: one at a time (whole vectors of 2 to 4 taps come here for
    // few tokens only)
    constexpr int U = VEC == 1 ? 8 : W <= 4 ? 1 : 4;
    if constexpr (W == 0) {
        return launch_kernel(conv_prefill_any_kernel<E>, (unsigned)blocks, kThreads, 0, s, a, groups,
                             strips);
    } else {
        const auto kernel =
            a.T < 8 ? conv_prefill_kernel<E, VEC, W, 1> : conv_prefill_kernel<E, VEC, W, U>;
        return launch_kernel(kernel, (unsigned)blocks, kThreads, 0, s, a, groups, strips);
    }
}

template <typename E, int W> int launch_token(const ConvPrefillArgs &a, cudaStream_t s)
{
    constexpr int VEC = Vec16<E>::kElems / 2;
    const int groups = (a.x_dim + 2 * a.bc_dim) / VEC;
    const int64_t blocks = ((int64_t)groups * ((a.active + 1) / 2) + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL)
        return SSU_ERR_SHAPE;
    return launch_kernel(conv_token_kernel<E, VEC, W>, (unsigned)blocks, kThreads, 0, s, a, groups);
}

template <typename E, int W> int launch_stream(const ConvPrefillArgs &a, cudaStream_t s)
{
    const int groups = (a.x_dim + 2 * a.bc_dim) / Vec16<E>::kElems;
    const int strips = (a.T + kStrip - 1) / kStrip;
    const int64_t blocks = ((int64_t)groups * strips * a.active + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL)
        return SSU_ERR_SHAPE;
    return launch_kernel(conv_stream_kernel<E, W>, (unsigned)blocks, kThreads, 0, s, a, groups,
                         strips);
}

template <typename E, int W> int launch_tree(const ConvPrefillArgs &a, bool vec, cudaStream_t s)
{
    const int per = 8 * Vec16<E>::kElems;           // channels of a CTA
    const int blocks = (a.x_dim + 2 * a.bc_dim + per - 1) / per;
    if ((int64_t)blocks * a.active > 0x7fffffffLL)
        return SSU_ERR_SHAPE;
    return launch_kernel(conv_tree_kernel<E, W>, (unsigned)(blocks * a.active), kThreads, 0, s, a,
                         blocks, vec);
}

template <typename E, int VEC>
int launch_v(const ConvPrefillArgs &a, cudaStream_t s)
{
    switch (a.width) {
    case 2: return launch_w<E, VEC, 2>(a, s);
    case 3: return launch_w<E, VEC, 3>(a, s);
    case 4: return launch_w<E, VEC, 4>(a, s);
    case 5: return launch_w<E, VEC, 5>(a, s);
    case 6: return launch_w<E, VEC, 6>(a, s);
    case 7: return launch_w<E, VEC, 7>(a, s);
    case 8: return launch_w<E, VEC, 8>(a, s);
    default: return launch_w<E, 1, 0>(a, s);
    }
}

template <typename E> int launch_e(ConvPrefillArgs a, cudaStream_t s)
{
    const bool vec = vector_rows<E>(a);
    if (a.parents) {
        switch (a.width) {
        case 2: return launch_tree<E, 2>(a, vec, s);
        case 3: return launch_tree<E, 3>(a, vec, s);
        case 4: return launch_tree<E, 4>(a, vec, s);
        default: return launch_tree<E, 0>(a, vec, s);
        }
    }
    if (!vec)
        return launch_v<E, 1>(a, s);
    a.win_mode = window_mode<E>(a);
    if (a.T >= 8) {
        switch (a.width) {
        case 2: return launch_stream<E, 2>(a, s);
        case 3: return launch_stream<E, 3>(a, s);
        case 4: return launch_stream<E, 4>(a, s);
        }
    }
    if (a.T == 1) {
        switch (a.width) {
        case 2: return launch_token<E, 2>(a, s);
        case 3: return launch_token<E, 3>(a, s);
        case 4: return launch_token<E, 4>(a, s);
        }
    }
    // half vectors: fewer registers a thread and twice the threads, for few tokens and for
    // windows of 5 to 8
    return launch_v<E, Vec16<E>::kElems / 2>(a, s);
}

template <typename E, int VEC, int W>
int launch_replay_w(const ConvPrefillArgs &a, cudaStream_t s)
{
    const int groups = a.x_dim / VEC;
    const int blocks = (groups + kThreads - 1) / kThreads;
    if ((int64_t)blocks * a.active > 0x7fffffffLL)
        return SSU_ERR_SHAPE;
    return launch_kernel(conv_replay_kernel<E, VEC, W>, (unsigned)(blocks * a.active), kThreads,
                         0, s, a, groups, blocks);
}

template <typename E, int VEC>
int launch_replay_v(const ConvPrefillArgs &a, cudaStream_t s)
{
    switch (a.width) {
    case 2: return launch_replay_w<E, VEC, 2>(a, s);
    case 3: return launch_replay_w<E, VEC, 3>(a, s);
    case 4: return launch_replay_w<E, VEC, 4>(a, s);
    default: return launch_replay_w<E, 1, 0>(a, s);
    }
}

template <typename E> int launch_replay_e(ConvPrefillArgs a, cudaStream_t s)
{
    if (!vector_rows<E>(a))
        return launch_replay_v<E, 1>(a, s);
    a.win_mode = window_mode<E>(a);
    return launch_replay_v<E, Vec16<E>::kElems>(a, s);
}

}  // namespace

int launch_conv_prefill(const ConvPrefillArgs &a, int x_dtype, cudaStream_t s)
{
    switch (x_dtype) {
    case SSU_F32: return launch_e<float>(a, s);
    case SSU_F16: return launch_e<__half>(a, s);
    case SSU_BF16: return launch_e<__nv_bfloat16>(a, s);
    default: return SSU_ERR_DTYPE;
    }
}

int launch_conv_replay(const ConvPrefillArgs &a, int x_dtype, cudaStream_t s)
{
    switch (x_dtype) {
    case SSU_F32: return launch_replay_e<float>(a, s);
    case SSU_F16: return launch_replay_e<__half>(a, s);
    case SSU_BF16: return launch_replay_e<__nv_bfloat16>(a, s);
    default: return SSU_ERR_DTYPE;
    }
}

}  // namespace ssu
