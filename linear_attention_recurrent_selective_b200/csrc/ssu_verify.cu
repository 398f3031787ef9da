// ssu_verify.cu -- verification of drafted tokens against the target's probabilities.
//
// Chain (position t holds token x_t; x_0 is already decided, the others were drafted): for
// t = 0, 1, ... the token x = x_{t+1} is accepted while u_t q_t(x) < p_t(x), which accepts
// with probability min(1, p/q) (q = 1 where the drafts carry no distribution). With n
// tokens accepted, the next one is drawn from row n-1: from max(p - q, 0) after a rejection
// (p without the rejected token where there is no q), from p when every token was accepted.
// Tree: at a node (from the root, the first node without a parent) the children are taken
// in node order and the first whose running sum of p(token) exceeds u of that node is
// accepted; where none is, the next token is drawn from p without the children's tokens.
// Either way the token stream is distributed as the target's.
//
// A token is drawn by inverse CDF: the first one whose running sum of masses exceeds
// u_sample times their total. Sums run in 64 bits: with 32, about one draw in a hundred
// over a vocabulary of 2^17 would fall on the other side of a border by rounding alone.
// What is not a positive finite number has no mass.
//
// Bound: memory for many rows (one row of p and at most one of q per sequence), latency
// for one: a few dependent loads find the row, then it is streamed once.
//
// Layout: a cluster of CTAs per sequence. Every CTA walks the chain or tree itself (a few
// gathers), then each warp sums one contiguous region of the row; the CTAs exchange their
// sums through distributed shared memory (one cluster barrier), every CTA finds the region
// that holds the border, and the warp that owns it scans it again from L2.
#include <cooperative_groups.h>

#include "ssu_common.cuh"

namespace ssu {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxTree = 128;         // nodes of a tree (the verify budget of ssu_ddtree)

template <typename E> __device__ __forceinline__ float to_f32(E v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ float mass_of(float v)
{
    return v > 0.f && v < __int_as_float(0x7f800000) ? v : 0.f;
}

struct Shared {
    int parent[kMaxTree], token[kMaxTree], first_child[kMaxTree], path[kMaxTree];
    double child_mass[kMaxTree];
    int drop[kMaxTree];               // tokens without mass in the row to draw from
    int ndrop, stop, root, n, end;
    double warp_sum[kWarps];
    double cta_sum[2][kMaxCluster];   // one set per attempt
};

// The row a token is drawn from, and what of it carries mass.
template <typename E> struct Row {
    const E *p, *q;                   // q: subtracted where present
    const int *drop;
    int ndrop, V;

    __device__ __forceinline__ double mass(int i, float pv, float qv) const
    {
        const float a = mass_of(pv), b = mass_of(qv);
        // the difference of two floats in double: exact unless they are 2^29 apart
        return a > b ? (double)a - (double)b : 0.0;
    }
};

// VEC neighbouring masses from element i (elements at or beyond `end` have none).
// `dropped`: some dropped token lies among them.
template <typename E, int VEC>
__device__ __forceinline__ void masses(const Row<E> &r, int i, int end, const float (&pv)[VEC],
                                       const float (&qv)[VEC], bool dropped, double (&m)[VEC])
{
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        m[e] = i + e < end ? r.mass(i + e, pv[e], qv[e]) : 0.0;
        if (dropped)
            for (int k = 0; k < r.ndrop; ++k)
                if (r.drop[k] == i + e)
                    m[e] = 0.0;
    }
}

template <typename E, int VEC>
__device__ __forceinline__ void load_probs(const E *p, int i, int end, float (&f)[VEC])
{
    if constexpr (VEC > 1) {
        if (i + VEC <= end) {
            Vec16<E>::unpack(*reinterpret_cast<const uint4 *>(p + i), f);
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        f[e] = i + e < end ? to_f32<E>(p[i + e]) : 0.f;
}

// Whether a dropped token lies in [lo, hi); the same answer in every lane.
template <typename E>
__device__ __forceinline__ bool any_dropped(const Row<E> &r, int lo, int hi, int lane)
{
    bool any = false;
    for (int k = lane; k < r.ndrop; k += 32)
        any |= r.drop[k] >= lo && r.drop[k] < hi;
    return __any_sync(~0u, any);
}

// The sum of the masses of [lo, hi), in every lane.
template <typename E, int VEC>
__device__ double region_sum(const Row<E> &r, int lo, int hi, int lane)
{
    constexpr int kStep = 32 * VEC, kUnroll = 4;
    const bool dropped = any_dropped(r, lo, hi, lane);
    double sum = 0.0;
    for (int i0 = lo; i0 < hi; i0 += kStep * kUnroll) {
        float pv[kUnroll][VEC], qv[kUnroll][VEC];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kStep + lane * VEC;
            load_probs<E, VEC>(r.p, i, hi, pv[u]);
            if (r.q) {
                load_probs<E, VEC>(r.q, i, hi, qv[u]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    qv[u][e] = 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            double m[VEC];
            masses<E, VEC>(r, i0 + u * kStep + lane * VEC, hi, pv[u], qv[u], dropped, m);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                sum += m[e];
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(~0u, sum, o);
    return sum;
}

// The first token of [lo, hi) with mass at which `before` plus the running sum exceeds thr;
// the region's last token with mass where rounding leaves none.
template <typename E, int VEC>
__device__ int region_find(const Row<E> &r, int lo, int hi, double before, double thr, int lane)
{
    const bool dropped = any_dropped(r, lo, hi, lane);
    int last = -1;
    for (int i0 = lo; i0 < hi; i0 += 32 * VEC) {
        const int i = i0 + lane * VEC;
        float pv[VEC], qv[VEC];
        load_probs<E, VEC>(r.p, i, hi, pv);
        if (r.q) {
            load_probs<E, VEC>(r.q, i, hi, qv);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                qv[e] = 0.f;
        }
        double m[VEC], mine = 0.0;
        masses<E, VEC>(r, i, hi, pv, qv, dropped, m);
        int tail = -1;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            mine += m[e];
            tail = m[e] > 0.0 ? i + e : tail;
        }
        double incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double up = __shfl_up_sync(~0u, incl, o);
            incl += lane >= o ? up : 0.0;
        }
        const unsigned hit = __ballot_sync(~0u, mine > 0.0 && before + incl > thr);
        if (hit) {
            const int src = __ffs(hit) - 1;
            double run = __shfl_up_sync(~0u, incl, 1);
            run = before + (lane ? run : 0.0);
            int at = tail;
#pragma unroll
            for (int e = VEC - 1; e >= 0; --e) {     // backwards: the first hit stays
                double upto = run;
#pragma unroll
                for (int f = 0; f <= e; ++f)
                    upto += m[f];
                if (m[e] > 0.0 && upto > thr)
                    at = i + e;
            }
            return __shfl_sync(~0u, at, src);
        }
        before += __shfl_sync(~0u, incl, 31);
        const unsigned some = __ballot_sync(~0u, tail >= 0);
        if (some)
            last = __shfl_sync(~0u, tail, 31 - __clz(some));
    }
    return last;
}

template <typename E, int VEC>
__global__ void __launch_bounds__(kThreads)
verify_kernel(const __grid_constant__ VerifyArgs a)
{
    __shared__ Shared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool report = rank == 0 && a.err;
    cluster.barrier_arrive();         // waited for before another CTA's memory is written

    const bool pad = a.idx && a.idx[b] < 0;
    int L = a.T;
    if (a.ctx && !pad) {
        L = a.ctx[b];
        if (report && tid == 0 && (L < 0 || L > a.T))
            atomicOr(a.err, L < 0 ? SSU_FLAG_NEGATIVE_LENGTH : SSU_FLAG_CONTEXT_RANGE);
        L = L < 0 ? 0 : (L > a.T ? a.T : L);
    }
    const E *const rows = static_cast<const E *>(a.p) + (int64_t)b * a.T * a.ldp;
    const E *const drafts =
        a.q ? static_cast<const E *>(a.q) + (int64_t)b * (a.T - 1) * a.ldq : nullptr;
    const int32_t *const tokens = a.tokens + (int64_t)b * a.T;
    const float *const u = a.u + (int64_t)b * a.T;
    const float us = a.u_sample[b];
    const int most = a.nodes ? a.max_accept : a.T;

    // ---- which tokens are accepted
    if (tid == 0) {
        s.stop = L;                    // chain: accepted tokens
        s.root = kMaxTree;
        s.ndrop = 0;
        s.n = 0;
    }
    __syncthreads();
    if (!pad && L > 0 && !a.parents) {
        for (int t = tid; t + 1 < L; t += kThreads) {
            const int x = tokens[t + 1];
            const bool in = x >= 0 && x < a.V;
            bool ok = false;
            if (in) {
                const float p = mass_of(to_f32<E>(rows[t * a.ldp + x]));
                const float q = drafts ? mass_of(to_f32<E>(drafts[t * a.ldq + x])) : 1.f;
                ok = (double)u[t] * (double)q < (double)p;
            } else if (report) {
                atomicOr(a.err, SSU_FLAG_TOKEN);
            }
            if (!ok)
                atomicMin(&s.stop, t + 1);
        }
        __syncthreads();
        if (tid == 0) {
            s.n = s.stop;
            s.end = s.n - 1;
            if (s.n < L && !drafts) {
                s.drop[0] = tokens[s.n];
                s.ndrop = 1;
            }
        }
    } else if (!pad && L > 0) {
        const int32_t *const par = a.parents + (int64_t)b * a.T;
        int up = -1, x = 0;
        float p = 0.f;
        if (tid < L) {
            up = par[tid];
            x = tokens[tid];
            const bool child = up >= 0 && up < L;
            if (up == -1)
                atomicMin(&s.root, tid);
            else if (!child && report)
                atomicOr(a.err, SSU_FLAG_TREE);
            if (child) {
                if (x >= 0 && x < a.V)
                    p = mass_of(to_f32<E>(rows[up * a.ldp + x]));
                else if (report)
                    atomicOr(a.err, SSU_FLAG_TOKEN);
            }
            s.parent[tid] = child ? up : -1;
            s.token[tid] = x;
            s.first_child[tid] = kMaxTree;
        }
        __syncthreads();
        if (tid < L && s.parent[tid] >= 0) {    // a token that an earlier sibling has: no mass
            for (int j = 0; j < tid; ++j)
                if (s.parent[j] == up && s.token[j] == x)
                    p = 0.f;
        }
        if (tid < L)
            s.child_mass[tid] = p;
        __syncthreads();
        if (tid < L && s.parent[tid] >= 0 && p > 0.f) {
            double run = 0.0;
            for (int j = 0; j <= tid; ++j)
                if (s.parent[j] == up)
                    run += s.child_mass[j];
            if ((double)u[up] < run)
                atomicMin(&s.first_child[up], tid);
        }
        __syncthreads();
        if (tid == 0 && s.root < kMaxTree) {
            int at = s.root, n = 1;
            s.path[0] = at;
            while (n < most && s.first_child[at] < kMaxTree) {   // at most T steps: children
                at = s.first_child[at];                          // of distinct nodes
                s.path[n++] = at;
            }
            s.n = n;
            s.end = at;
        } else if (tid == 0 && report) {
            atomicOr(a.err, SSU_FLAG_TREE);
        }
        __syncthreads();
        if (tid < L && s.n > 0 && s.n < most && s.parent[tid] == s.end)
            s.drop[atomicAdd(&s.ndrop, 1)] = x;
    }
    cluster.barrier_wait();           // every CTA of the cluster has started
    __syncthreads();
    const int n = s.n;
    if (rank == 0) {
        if (tid == 0)
            a.accepted[b] = n;
        if (a.nodes)
            for (int i = tid; i < a.max_accept; i += kThreads)
                a.nodes[(int64_t)b * a.max_accept + i] = i < n ? s.path[i] : -1;
        if (n == 0 && tid == 0)
            a.next[b] = -1;
    }
    if (n == 0)                                 // the same in every CTA of the cluster
        return;

    // ---- the next token
    const bool rejected = !a.parents && n < L;
    Row<E> r;
    r.p = rows + s.end * a.ldp;
    r.q = rejected && drafts ? drafts + s.end * a.ldq : nullptr;
    r.drop = s.drop;
    r.ndrop = s.ndrop;
    r.V = a.V;
    constexpr int kStep = 32 * VEC;
    const int regions = C * kWarps;
    const int len = ((a.V + regions - 1) / regions + kStep - 1) / kStep * kStep;
    const int64_t lo64 = (int64_t)(rank * kWarps + warp) * len;
    const int lo = (int)min(lo64, (int64_t)a.V), hi = (int)min(lo64 + len, (int64_t)a.V);

    // A residual without mass (p <= q wherever p has any, or a rejected token that held it
    // all) can only come from rounding: the draw is then from p itself.
    for (int attempt = 0; attempt < 2; ++attempt) {
        const double mine = region_sum<E, VEC>(r, lo, hi, lane);
        if (lane == 0)
            s.warp_sum[warp] = mine;
        __syncthreads();
        if (tid < C) {
            double sum = 0.0;
            for (int w = 0; w < kWarps; ++w)
                sum += s.warp_sum[w];
            *cluster.map_shared_rank(&s.cta_sum[attempt][rank], tid) = sum;
        }
        cluster.sync();
        double total = 0.0;
        for (int c = 0; c < C; ++c)
            total += s.cta_sum[attempt][c];
        if (total > 0.0) {
            // the CTA, then its warp, whose running sum first exceeds thr (sums of
            // non-negative numbers in one order never decrease); the last one with any
            // mass where none does
            const double thr = (double)us * total;
            int owner = -1, last = -1;
            double run = 0.0, before = 0.0;
            for (int c = 0; c < C; ++c) {
                const double v = s.cta_sum[attempt][c];
                if (v > 0.0) {
                    last = c;
                    if (owner < 0 && run + v > thr) {
                        owner = c;
                        before = run;
                    }
                }
                run += v;
            }
            const bool beyond = owner < 0;
            if (beyond)
                owner = last;
            if (rank != owner)
                return;
            int w_owner = -1, w_last = -1;
            double w_run = before, w_before = 0.0;
            for (int w = 0; w < kWarps; ++w) {
                const double v = s.warp_sum[w];
                if (v > 0.0) {
                    w_last = w;
                    if (!beyond && w_owner < 0 && w_run + v > thr) {
                        w_owner = w;
                        w_before = w_run;
                    }
                }
                w_run += v;
            }
            const bool tail = w_owner < 0;
            if (tail)
                w_owner = w_last;
            if (warp == w_owner) {
                const double inf = __longlong_as_double(0x7ff0000000000000LL);
                const int at = region_find<E, VEC>(r, lo, hi, w_before, tail ? inf : thr, lane);
                if (lane == 0)
                    a.next[b] = at;
            }
            return;
        }
        r.q = nullptr;
        r.ndrop = 0;
        __syncthreads();                        // warp_sum is written again
    }
    if (rank == 0 && tid == 0) {                // no mass at all
        a.next[b] = -1;
        if (a.err)
            atomicOr(a.err, SSU_FLAG_NO_MASS);
    }
}

template <typename E, int VEC> int launch_v(const VerifyArgs &a, cudaStream_t s)
{
    // CTAs of a sequence: as many as fill the card once, and no more than leave each warp
    // one step of 32 vectors
    int c = 1;
    while (c < kMaxCluster && (int64_t)a.active * c < 296 && a.V > c * kWarps * 32 * VEC)
        c *= 2;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    if ((int64_t)a.active * c > 0x7fffffffLL)
        return SSU_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.active * c));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel<E, VEC>, a) == cudaSuccess ? SSU_OK
                                                                             : SSU_ERR_CUDA;
}

template <typename E> int launch_e(const VerifyArgs &a, cudaStream_t s)
{
    constexpr int V = Vec16<E>::kElems;
    const auto ok = [](const void *p, int64_t ld) {
        return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % V == 0;
    };
    return ok(a.p, a.ldp) && (!a.q || ok(a.q, a.ldq)) ? launch_v<E, V>(a, s) : launch_v<E, 1>(a, s);
}

}  // namespace

int launch_verify(const VerifyArgs &a, int p_dtype, cudaStream_t s)
{
    switch (p_dtype) {
    case SSU_F32: return launch_e<float>(a, s);
    case SSU_F16: return launch_e<__half>(a, s);
    case SSU_BF16: return launch_e<__nv_bfloat16>(a, s);
    default: return SSU_ERR_DTYPE;
    }
}

}  // namespace ssu
