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
// Layout: a thread owns one 16-byte vector of channels (VEC = 8 or 4; 1 where rows or
// segments are not 16-byte aligned) over a strip of up to kStrip tokens, and slides the
// last W-1 inputs through registers, so each input is read once per strip plus W-1 at the
// strip's start. The thread of a row's first strip also owns the window of its channels:
// it alone reads the old taps (a later strip starts at t >= kStrip >= W-1) and it alone
// writes the new ones, after its reads, so the update needs no second launch.
#include "ssu_common.cuh"

namespace ssu {
namespace {

constexpr int kThreads = 128;
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

template <typename E, int VEC>
__device__ __forceinline__ void widen_chunk(const Chunk<E, VEC> &c, float *f)
{
    if constexpr (VEC == Vec16<E>::kElems) {
        uint4 r;
        memcpy(&r, &c, 16);
        Vec16<E>::unpack(r, f);
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
    if constexpr (VEC == Vec16<E>::kElems) {
        *reinterpret_cast<uint4 *>(p) = Vec16<E>::pack(f);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            p[e] = narrow<E>(f[e]);
    }
}

// v * sigmoid(v). 16-bit outputs take the approximate exponential and division, whose
// error (a few 2^-22) is far below the 2^-9 of the rounding that follows; fp32 outputs
// take the accurate ones.
template <typename E> __device__ __forceinline__ float conv_silu(float v)
{
    if constexpr (sizeof(E) == 4)
        return silu_f(v);
    else
        return __fdividef(v, 1.f + __expf(-v));
}

// The window taps of VEC channels from channel c0: every tap in registers, oldest first.
// mode 1: channel-major windows (stride_c = W-1, stride_k = 1), the VEC * (W-1) elements
// contiguous and 16-byte aligned; mode 2: tap-major (stride_c = 1), a vector per tap;
// mode 0: element by element.
template <typename E, int VEC, int W>
__device__ __forceinline__ void load_taps(const ConvPrefillArgs &a, int64_t at, E (&tap)[W - 1][VEC])
{
    const E *p = static_cast<const E *>(a.cstate) + at;
    if (a.win_mode == 1) {
        Chunk<E, VEC> raw[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            raw[j] = load_chunk<E, VEC>(p, j * VEC);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                tap[k][e] = raw[(e * (W - 1) + k) / VEC].v[(e * (W - 1) + k) % VEC];
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
        Chunk<E, VEC> raw[W - 1];
#pragma unroll
        for (int e = 0; e < VEC; ++e)
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                raw[(e * (W - 1) + k) / VEC].v[(e * (W - 1) + k) % VEC] = tap[k][e];
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            *reinterpret_cast<Chunk<E, VEC> *>(p + j * VEC) = raw[j];
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

// A row's clamped length; the row's first thread reports a length outside [0, T].
__device__ __forceinline__ int row_length(const int32_t *len, int b, int T, int over_flag,
                                          bool report, int32_t *err)
{
    if (!len)
        return T;
    const int L = len[b];
    if (report && err && (L < 0 || L > T))
        atomicOr(err, L < 0 ? SSU_FLAG_NEGATIVE_LENGTH : over_flag);
    return L < 0 ? 0 : (L > T ? T : L);
}

// The parent of a tree node, -1 at a root. One outside [-1, L) marks the node as malformed;
// the W-1 steps of a node's walk end whatever the parents hold.
__device__ __forceinline__ int parent_of(const int32_t *par, int at, int L, bool &bad)
{
    const int up = par[at];
    if (up >= -1 && up < L)
        return up;
    bad = true;
    return -1;
}

// One thread per (row, strip, vector of channels), widths 2..4.
template <typename E, int VEC, int W, bool TREE>
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
    const int L = row_length(a.ctx, (int)b, a.T, SSU_FLAG_CONTEXT_RANGE, first, a.err);
    const int t1 = min(t0 + kStrip, L);
    if (t0 >= L)
        return;

    float w[W][VEC], bias[VEC];
    {
        Chunk<E, VEC> raw[W];                   // VEC channels' weights are contiguous
#pragma unroll
        for (int j = 0; j < W; ++j)
            raw[j] = load_chunk<E, VEC>(a.w, (int64_t)c0 * W + j * VEC);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
#pragma unroll
            for (int k = 0; k < W; ++k)
                w[k][e] = widen<E>(raw[(e * W + k) / VEC].v[(e * W + k) % VEC]);
        Chunk<E, VEC> rb;
        if (a.bias)
            rb = load_chunk<E, VEC>(a.bias, c0);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            bias[e] = a.bias ? widen<E>(rb.v[e]) : 0.f;
    }
    const E *in = static_cast<const E *>(a.xbc) + b * a.T * a.ldx + c0;
    const int64_t tap_at = (int64_t)slot * a.cslot + (int64_t)c0 * a.cc;

    if constexpr (TREE) {
        const int32_t *par = a.parents + b * a.T;
        E old[W - 1][VEC];
        load_taps<E, VEC, W>(a, tap_at, old);
        for (int t = t0; t < t1; ++t) {
            float acc[VEC];
            int at = t;                         // >= 0: a node; -1 - j: j taps back
            bool bad = false;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                acc[e] = bias[e];
#pragma unroll
            for (int k = W - 1; k >= 0; --k) {
                float f[VEC];
                if (at >= 0) {
                    widen_chunk<E, VEC>(load_chunk<E, VEC>(in, at * a.ldx), f);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        f[e] = 0.f;
#pragma unroll
                        for (int j = 0; j < W - 1; ++j)
                            if (at == j - (W - 1))
                                f[e] = widen<E>(old[j][e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    acc[e] = fmaf(w[k][e], f[e], acc[e]);
                if (k > 0)
                    at = at >= 0 ? parent_of(par, at, L, bad) : at - 1;
            }
            if (bad && g == 0 && a.err)
                atomicOr(a.err, SSU_FLAG_TREE);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                acc[e] = bad ? 0.f : (a.silu ? conv_silu<E>(acc[e]) : acc[e]);
            store_floats<E, VEC>(out.p + t * out.ld, acc);
        }
        return;
    }

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

    constexpr int U = 4;                        // tokens loaded together
    for (int t = t0; t < t1; t += U) {
        Chunk<E, VEC> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < t1)
                raw[u] = load_chunk<E, VEC>(in, (t + u) * a.ldx);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= t1)
                break;
            float f[VEC], acc[VEC];
            widen_chunk<E, VEC>(raw[u], f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                acc[e] = bias[e];
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
                    acc[e] = fmaf(w[k][e], win[k][e], acc[e]);
                acc[e] = fmaf(w[W - 1][e], f[e], acc[e]);
                if (a.silu)
                    acc[e] = conv_silu<E>(acc[e]);
#pragma unroll
                for (int k = 0; k + 1 < W - 1; ++k)
                    win[k][e] = win[k + 1][e];
                win[W - 2][e] = f[e];
            }
            store_floats<E, VEC>(out.p + (t + u) * out.ld, acc);
        }
    }

    if (strip == 0 && a.update) {               // the last W-1 of (old taps, tokens)
        E nw[W - 1][VEC];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int t = L + j - (W - 1);      // < 0: still an old tap
            if (t >= 0) {
                const Chunk<E, VEC> c = load_chunk<E, VEC>(in, t * a.ldx);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    nw[j][e] = c.v[e];
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
#pragma unroll
                    for (int o = 0; o < W - 1; ++o)
                        if (o == L + j)
                            nw[j][e] = old[o][e];
            }
        }
        store_taps<E, VEC, W>(a, tap_at, nw);
    }
}

// Every other width (1, 5..16): a thread per (row, strip, channel) that reads each tap
// where it lies. Same ownership of the windows.
template <typename E, bool TREE>
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
    const int L = row_length(a.ctx, (int)b, a.T, SSU_FLAG_CONTEXT_RANGE, first, a.err);
    const int t1 = min(t0 + kStrip, L);
    if (t0 >= L)
        return;
    const E *in = static_cast<const E *>(a.xbc) + b * a.T * a.ldx + c;
    const E *w = static_cast<const E *>(a.w) + (int64_t)c * W;
    const float bias = a.bias ? widen<E>(static_cast<const E *>(a.bias)[c]) : 0.f;
    E *tap = static_cast<E *>(a.cstate) + (int64_t)slot * a.cslot + (int64_t)c * a.cc;
    const int32_t *par = TREE ? a.parents + b * a.T : nullptr;
    for (int t = t0; t < t1; ++t) {
        float acc = bias;
        int at = t;
        bool bad = false;
        for (int k = W - 1; k >= 0; --k) {
            const float f = at >= 0 ? widen<E>(in[at * a.ldx]) : widen<E>(tap[(at + W - 1) * a.ck]);
            acc = fmaf(widen<E>(w[k]), f, acc);
            if (k > 0)
                at = TREE && at >= 0 ? parent_of(par, at, L, bad) : at - 1;
        }
        if (bad && c == 0 && a.err)
            atomicOr(a.err, SSU_FLAG_TREE);
        out.p[t * out.ld] = narrow<E>(bad ? 0.f : (a.silu ? conv_silu<E>(acc) : acc));
    }
    if (!TREE && strip == 0 && a.update)
        for (int j = 0; j < W - 1; ++j) {       // ascending: a tap is read before it is replaced
            const int t = L + j - (W - 1);
            tap[j * a.ck] = t >= 0 ? in[t * a.ldx] : tap[(L + j) * a.ck];
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
    const int slot = a.idx ? a.idx[b] : b;
    if (slot < 0)
        return;
    if (slot >= a.P) {
        if (first && a.err)
            atomicOr(a.err, SSU_FLAG_INDEX_RANGE);
        return;
    }
    const int most = a.nodes ? a.max_accept : a.T;
    const int k = row_length(a.ctx, b, most, SSU_FLAG_ACCEPTED_RANGE, first, a.err);
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
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int t = k + j - (W - 1);
            if (t >= 0) {
                const Chunk<E, VEC> c = load_chunk<E, VEC>(in, (ids ? ids[t] : t) * a.ldx);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    nw[j][e] = c.v[e];
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
#pragma unroll
                    for (int o = 0; o < W - 1; ++o)
                        if (o == k + j)
                            nw[j][e] = old[o][e];
            }
        }
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
    if constexpr (W == 0) {
        return a.parents ? launch_kernel(conv_prefill_any_kernel<E, true>, (unsigned)blocks,
                                         kThreads, 0, s, a, groups, strips)
                         : launch_kernel(conv_prefill_any_kernel<E, false>, (unsigned)blocks,
                                         kThreads, 0, s, a, groups, strips);
    } else {
        return a.parents ? launch_kernel(conv_prefill_kernel<E, VEC, W, true>, (unsigned)blocks,
                                         kThreads, 0, s, a, groups, strips)
                         : launch_kernel(conv_prefill_kernel<E, VEC, W, false>, (unsigned)blocks,
                                         kThreads, 0, s, a, groups, strips);
    }
}

template <typename E, int VEC>
int launch_v(const ConvPrefillArgs &a, cudaStream_t s)
{
    switch (a.width) {
    case 2: return launch_w<E, VEC, 2>(a, s);
    case 3: return launch_w<E, VEC, 3>(a, s);
    case 4: return launch_w<E, VEC, 4>(a, s);
    default: return launch_w<E, 1, 0>(a, s);
    }
}

template <typename E> int launch_e(ConvPrefillArgs a, cudaStream_t s)
{
    if (!vector_rows<E>(a))
        return launch_v<E, 1>(a, s);
    a.win_mode = window_mode<E>(a);
    return launch_v<E, Vec16<E>::kElems>(a, s);
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
