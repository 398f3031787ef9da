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
// Measured (B200, where the distributions are not in L2): 64 sequences of 4 drafted tokens over
// 2^17 tokens in fp32 19.1 us, of which the rows' sums are 12.5 (0.79 of the copy rate), finding
// the row and the clusters' meeting 4.7 (6.2 where a length or an index was waited for before
// the tokens) and the drawn token 1.7; over 151936 tokens 23.0 us, over 50001, where p and q
// start at different offsets from 16 bytes, 13.9 us; one sequence over 65537 tokens in bfloat16
// 7.8 us; 16 trees of 128 nodes over 32768 tokens 11.5 us. Sums as pairs of floats instead of doubles: 33.7 us against 27.3 for the same loop.
//
// Layout: a cluster of CTAs per sequence. Every CTA walks the chain or tree itself (a few
// gathers), then each warp sums one contiguous region of the row in kChunks chunks, whose
// lane sums stay in shared memory; the CTAs exchange their sums through distributed shared
// memory (one cluster barrier) and every CTA finds the region that holds the border. The
// warp that owns it finds the chunk from the lane sums and scans only that again (from L2).
#include <cooperative_groups.h>

#include "ssu_common.cuh"

namespace ssu {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kFill = 592;            // CTAs that give 148 SMs four each
constexpr int kChunks = 16;           // of a warp's region
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
    float u[kMaxTree];
    int drop[kMaxTree];               // tokens without mass in the row to draw from
    int ndrop, stop, root, n, end;
    double warp_sum[kWarps];
    double cta_sum[2][kMaxCluster];   // one set per attempt
    double lane_sum[kWarps][kChunks][32];
};

// The row a token is drawn from, and what of it carries mass. Elements are numbered from
// -first >= 0 on, so that element 0 modulo VEC starts on 16 bytes.
template <typename E> struct Row {
    const E *p, *q;                   // element 0; q: subtracted (read with kQ only)
    const int *drop;
    int ndrop, first, end;            // elements [-first, end) exist: token = first + element
};

// VEC neighbouring elements as raw bits: one access, or with kEdge those of [lo, hi) one by
// one and zeros beyond.
template <typename E, int VEC, bool kEdge>
__device__ __forceinline__ void load_probs(const E *p, int i, int lo, int hi, uint32_t (&w)[4])
{
    if constexpr (VEC > 1 && !kEdge) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p + i);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (VEC > 1) {
        E e[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            e[k] = i + k >= lo && i + k < hi ? p[i + k] : E(0.f);
        memcpy(w, e, 16);
    } else {
        w[0] = !kEdge || (i >= lo && i < hi) ? __float_as_uint(to_f32<E>(p[i])) : 0u;
    }
}

template <typename E, int VEC>
__device__ __forceinline__ void unpack_probs(const uint32_t (&w)[4], float (&f)[VEC])
{
    if constexpr (VEC > 1)
        Vec16<E>::unpack(make_uint4(w[0], w[1], w[2], w[3]), f);
    else
        f[0] = __uint_as_float(w[0]);
}

// The masses of VEC neighbouring elements from i on. `dropped`: some of the dropped tokens
// may be among them.
template <typename E, int VEC, bool kQ>
__device__ __forceinline__ void masses(const Row<E> &r, int i, const uint32_t (&pw)[4],
                                       const uint32_t (&qw)[4], bool dropped, double (&m)[VEC])
{
    float pv[VEC], qv[VEC];
    unpack_probs<E, VEC>(pw, pv);
    if (kQ)
        unpack_probs<E, VEC>(qw, qv);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const float v = mass_of(pv[e]);
        m[e] = (double)v;
        if (kQ) {       // max(p - q, 0); the difference is exact unless they are 2^29 apart
            const float q = mass_of(qv[e]);
            m[e] -= (double)(v > q ? q : v);
        }
    }
    if (dropped) {
        for (int k = 0; k < r.ndrop; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (r.drop[k] - r.first == i + e)
                    m[e] = 0.0;
    }
}

template <int VEC> __device__ __forceinline__ double sum_of(const double (&m)[VEC])
{
    double s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        s[e] = m[e];
#pragma unroll
    for (int d = VEC / 2; d > 0; d /= 2)
#pragma unroll
        for (int e = 0; e < d; ++e)
            s[e] += s[e + d];
    return s[0];
}

// Whether a dropped token lies in elements [lo, hi); the same answer in every lane.
template <typename E>
__device__ __forceinline__ bool any_dropped(const Row<E> &r, int lo, int hi, int lane)
{
    bool any = false;
    for (int k = lane; k < r.ndrop; k += 32)
        any |= r.drop[k] - r.first >= lo && r.drop[k] - r.first < hi;
    return __any_sync(~0u, any);
}

// Sums of the masses of [lo, hi) by lane for every chunk of `per` elements (a multiple of
// 32 VEC), into out[chunk][lane]; returns the whole sum, in every lane.
template <typename E, int VEC, bool kQ>
__device__ __forceinline__ double region_sum(const Row<E> &r, int lo, int hi, int per, int lane,
                                             double (*out)[32])
{
    constexpr int kStep = 32 * VEC, kUnroll = VEC == 1 ? 8 : 16 / VEC;
    const bool dropped = any_dropped(r, lo, hi, lane);
    const int from = -r.first, to = min(hi, r.end);
    double all = 0.0, sum = 0.0;
    int chunk = 0, next = lo + per;                 // end of the current chunk
    uint32_t pw[kUnroll][4], qw[kUnroll][4];
    const auto step = [&](int at, const uint32_t (&p)[4], const uint32_t (&q)[4]) {
        double m[VEC];
        masses<E, VEC, kQ>(r, at + lane * VEC, p, q, dropped, m);
        sum += sum_of<VEC>(m);
        if (at + kStep == next || at + kStep >= hi) {
            out[chunk++][lane] = sum;
            all += sum;
            sum = 0.0;
            next += per;
        }
    };
    int at = lo;
    while (at < hi) {
        if (at >= from && at + kStep * kUnroll <= to) {     // a batch of whole steps
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                load_probs<E, VEC, false>(r.p, at + u * kStep + lane * VEC, from, to, pw[u]);
                if (kQ)
                    load_probs<E, VEC, false>(r.q, at + u * kStep + lane * VEC, from, to, qw[u]);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                step(at + u * kStep, pw[u], qw[u]);
            at += kStep * kUnroll;
        } else {                                            // a step at the row's ends
            load_probs<E, VEC, true>(r.p, at + lane * VEC, from, to, pw[0]);
            if (kQ)
                load_probs<E, VEC, true>(r.q, at + lane * VEC, from, to, qw[0]);
            step(at, pw[0], qw[0]);
            at += kStep;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        all += __shfl_xor_sync(~0u, all, o);
    return all;
}

// An inclusive running sum over the lanes.
__device__ __forceinline__ double running(double v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(~0u, v, o);
        v += lane >= o ? up : 0.0;
    }
    return v;
}

// The token at the first element of [lo, hi) with mass at which `before` plus the running
// sum exceeds thr; the last one with mass where rounding leaves none.
template <typename E, int VEC, bool kQ>
__device__ __noinline__ int find_in(const Row<E> r, int lo, int hi, double before, double thr,
                                    int lane)
{
    const bool dropped = any_dropped(r, lo, hi, lane);
    const int from = -r.first, to = min(hi, r.end);
    int last = -1;
    for (int i0 = lo; i0 < hi; i0 += 32 * VEC) {
        const int i = i0 + lane * VEC;
        uint32_t pw[4], qw[4];
        load_probs<E, VEC, true>(r.p, i, from, to, pw);
        if (kQ)
            load_probs<E, VEC, true>(r.q, i, from, to, qw);
        double m[VEC];
        masses<E, VEC, kQ>(r, i, pw, qw, dropped, m);
        const double mine = sum_of<VEC>(m);
        int tail = -1;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            tail = m[e] > 0.0 ? i + e : tail;
        const double incl = running(mine, lane);
        const unsigned hit = __ballot_sync(~0u, mine > 0.0 && before + incl > thr);
        double run = __shfl_up_sync(~0u, incl, 1);
        run = before + (lane ? run : 0.0);
        if (hit) {
            int at = -1;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                run += m[e];
                if (m[e] > 0.0 && (run > thr || i + e == tail) && at < 0)
                    at = i + e;
            }
            return r.first + __shfl_sync(~0u, at, __ffs(hit) - 1);
        }
        before += __shfl_sync(~0u, incl, 31);
        const unsigned some = __ballot_sync(~0u, tail >= 0);
        if (some)
            last = __shfl_sync(~0u, tail, 31 - __clz(some));
    }
    return r.first + last;
}

// The same over a warp's whole region, from its lane sums: the chunk first.
template <typename E, int VEC, bool kQ>
__device__ __forceinline__ int region_find(const Row<E> &r, int lo, int hi, int per, double before,
                                           double thr, int lane, const double (*sums)[32])
{
    static_assert(kChunks == 16, "two lanes a chunk");
    const int chunks = (hi - lo + per - 1) / per, c = lane >> 1;
    double part[4] = {};
    if (c < chunks)
#pragma unroll
        for (int k = 0; k < 16; ++k)                // (rotated: lanes on different banks)
            part[k & 3] += sums[c][(lane & 1) * 16 + ((k + lane) & 15)];
    double mine = sum_of<4>(part);
    mine += __shfl_xor_sync(~0u, mine, 1);          // the chunk's sum, in both of its lanes
    const bool odd = lane & 1;
    const double incl = running(odd ? mine : 0.0, lane);    // odd lanes: up to their chunk
    const unsigned some = __ballot_sync(~0u, odd && mine > 0.0);
    const unsigned hit = __ballot_sync(~0u, odd && mine > 0.0 && before + incl > thr);
    // (some is not empty: the region's sum is positive)
    const int at = hit ? __ffs(hit) - 1 : 31 - __clz(some);
    const double upto = __shfl_sync(~0u, incl - mine, at);
    const int from = lo + (at >> 1) * per;
    const double inf = __longlong_as_double(0x7ff0000000000000LL);
    return find_in<E, VEC, kQ>(r, from, min(from + per, hi), before + upto, hit ? thr : inf, lane);
}

// Draw row b's next token from the masses of `row` (less `sub`, without the dropped tokens),
// whose element 0 lies `skew` elements behind a 16-byte boundary.
template <typename E, int VEC>
__device__ __forceinline__ void draw(const VerifyArgs &a, Shared &s, cg::cluster_group &cluster,
                                     int b, const E *row, const E *sub, int skew, float us)
{
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Row<E> r;
    r.first = -skew;
    r.end = a.V + skew;
    r.p = row - skew;
    r.q = sub ? sub - skew : nullptr;
    r.drop = s.drop;
    r.ndrop = s.ndrop;
    // warps take contiguous regions of at most kChunks chunks of `per` elements
    constexpr int kStep = 32 * VEC;
    const int regions = C * kWarps;
    const int steps = ((r.end + regions - 1) / regions + kStep - 1) / kStep;
    const int per = (steps + kChunks - 1) / kChunks * kStep;
    const int64_t lo64 = (int64_t)(rank * kWarps + warp) * steps * kStep;
    const int lo = (int)min(lo64, (int64_t)r.end);
    const int hi = (int)min(lo64 + (int64_t)steps * kStep, (int64_t)r.end);

    // A residual without mass (p <= q wherever p has any, or a rejected token that held it
    // all) can only come from rounding: the draw is then from p itself.
    for (int attempt = 0; attempt < 2; ++attempt) {
        const double mine = r.q ? region_sum<E, VEC, true>(r, lo, hi, per, lane, s.lane_sum[warp])
                                : region_sum<E, VEC, false>(r, lo, hi, per, lane, s.lane_sum[warp]);
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
            if (rank != (beyond ? last : owner))
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
            if (warp == (tail ? w_last : w_owner)) {
                __syncwarp();
                const double inf = __longlong_as_double(0x7ff0000000000000LL);
                const double t = tail ? inf : thr;
                const int at = r.q ? region_find<E, VEC, true>(r, lo, hi, per, w_before, t, lane,
                                                               s.lane_sum[warp])
                                   : region_find<E, VEC, false>(r, lo, hi, per, w_before, t, lane,
                                                                s.lane_sum[warp]);
                if (lane == 0)
                    a.next[b] = at;
            }
            return;
        }
        r.q = nullptr;
        r.ndrop = 0;
        __syncthreads();                        // the sums are written again
    }
    if (rank == 0 && tid == 0) {                // no mass at all
        a.next[b] = -1;
        if (a.err)
            atomicOr(a.err, SSU_FLAG_NO_MASS);
    }
}

template <typename E>
__global__ void __launch_bounds__(kThreads, 4)
verify_kernel(const __grid_constant__ VerifyArgs a)
{
    __shared__ Shared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / C;
    const int tid = threadIdx.x;
    const bool report = rank == 0 && a.err;
    cluster.barrier_arrive();         // waited for before another CTA's memory is written

    const E *const rows = static_cast<const E *>(a.p) + (int64_t)b * a.T * a.ldp;
    const E *const drafts =
        a.q ? static_cast<const E *>(a.q) + (int64_t)b * (a.T - 1) * a.ldq : nullptr;
    const int32_t *const tokens = a.tokens + (int64_t)b * a.T;
    const float *const u = a.u + (int64_t)b * a.T;
    const int32_t *const par = a.parents ? a.parents + (int64_t)b * a.T : nullptr;
    // all loads that depend on no other are in flight before the first is waited for
    const int slot = a.idx ? a.idx[b] : 0;
    const int len = a.ctx ? a.ctx[b] : a.T;
    const float us = a.u_sample[b];
    const int most = a.nodes ? a.max_accept : a.T;
    const int ahead = par ? 0 : 1;                      // a chain's position t checks token t + 1
    const bool mine = tid + ahead < a.T;
    const int x0 = mine ? tokens[tid + ahead] : 0;
    const int up0 = mine && par ? par[tid] : -1;
    const float u0 = mine ? u[tid] : 0.f;
    const bool pad = slot < 0;
    if (report && tid == 0 && !pad && (len < 0 || len > a.T))
        atomicOr(a.err, len < 0 ? SSU_FLAG_NEGATIVE_LENGTH : SSU_FLAG_CONTEXT_RANGE);
    const int L = len < 0 ? 0 : (len > a.T ? a.T : len);

    // ---- which tokens are accepted
    if (tid == 0) {
        s.stop = L;                    // chain: accepted tokens
        s.root = kMaxTree;
        s.ndrop = 0;
        s.n = 0;
    }
    __syncthreads();
    if (!pad && L > 0 && !par) {
        for (int t = tid; t + 1 < L; t += kThreads) {
            const int x = t == tid ? x0 : tokens[t + 1];
            const float ut = t == tid ? u0 : u[t];
            const bool in = x >= 0 && x < a.V;
            bool ok = false;
            if (in) {
                const float p = mass_of(to_f32<E>(rows[t * a.ldp + x]));
                const float q = drafts ? mass_of(to_f32<E>(drafts[t * a.ldq + x])) : 1.f;
                ok = (double)ut * (double)q < (double)p;
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
        const int up = up0, x = x0;
        float p = 0.f;
        if (tid < L) {
            s.u[tid] = u0;
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
            if ((double)s.u[up] < run)
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

    // ---- the next token, by whole vectors where both rows allow it
    constexpr int V = Vec16<E>::kElems;
    const bool rejected = !par && n < L;
    const E *const row = rows + s.end * a.ldp;
    const E *const sub = rejected && drafts ? drafts + s.end * a.ldq : nullptr;
    const int skew = (int)(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(E));
    if (!sub || (int)(reinterpret_cast<uintptr_t>(sub) % 16 / sizeof(E)) == skew)
        draw<E, V>(a, s, cluster, b, row, sub, skew, us);
    else
        draw<E, 1>(a, s, cluster, b, row, sub, 0, us);
}

template <typename E> int launch_e(const VerifyArgs &a, cudaStream_t s)
{
    // CTAs of a sequence: as many as the card holds at once (four an SM), and no more than
    // leave each warp one step of 32 vectors
    int c = 1;
    while (c < kMaxCluster && (int64_t)a.active * c * 2 <= kFill &&
           a.V > c * kWarps * 32 * Vec16<E>::kElems)
        c *= 2;
    if ((int64_t)a.active * c > 0x7fffffffLL)
        return SSU_ERR_SHAPE;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.active * c));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel<E>, a) == cudaSuccess ? SSU_OK : SSU_ERR_CUDA;
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
