// verify.cuh -- verification of drafted tokens against the target's probabilities, from
// random numbers that the caller draws (speculative sampling).
//
// For a sequence with drafts x_0 .. x_{m-1}, target probabilities p_i and draft probabilities
// q_i (a point draft: q_i = 1 at x_i), draft i is accepted while
//     u_i q_i(x_i) < p_i(x_i)
// (the probability min(1, p / q) for uniform u_i).  At the first refusal n the next token is drawn
// from the residual r = max(p_n - q_n, 0); with every draft accepted (n = m) from r = p_m;
// where the residual is zero everywhere (the draft covers the target), from p_n.  The draw
// inverts the distribution function: the first v with  sum_{w <= v} r_w > u' sum_w r_w.
// Accepted tokens and the drawn one are then distributed as if the target had been sampled
// token by token.
//
// Products and sums are taken in 64 bits: a vocabulary of 10^5 has as many borders of its
// distribution function, and 32-bit sums (off by ~1e-6 of the total) would move some of
// them across u' in about every tenth draw; 64-bit sums of any order agree but for a chance
// of ~1e-11 a draw.  p u and q u of 32-bit factors are exact in 64 bits.
//
// A cluster of up to eight CTAs takes a sequence, each CTA a consecutive part of the one row
// (pair) that is drawn from -- the other rows are only gathered from.  Every warp sums a
// consecutive piece; the pieces' sums meet through distributed shared memory, and the piece
// that the target falls in is read again (from L2) by its CTA to find the token.  One launch;
// bound by the row's bytes for a large batch, by the chain of dependent reads for a small one.
#pragma once
#include <climits>

#include "common.cuh"
#include "tc05.cuh"

namespace kvattn {

struct VerifyParams {
    const void *p;                 // [B, L + 1, V] fp32 or bf16
    const void *q;                 // [B, L, V] same type, or null (point drafts)
    const int32_t *drafts;         // [B, L]
    const int32_t *lens;           // [B] drafts of each sequence, or null (all L)
    const float *u_accept;         // [B, L]
    const float *u_sample;         // [B]
    int32_t *accepted;             // [B]
    int32_t *tokens;               // [B, L + 1]
    long long p_b, p_l, q_b, q_l;  // element strides of the batch and position axes
    int B, L, V;
    int vec;                       // every row 16-byte aligned
};

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 8;
constexpr int kVerifyPerSm = 4;       // CTAs resident on an SM

template <typename T> struct ProbVec;
template <> struct ProbVec<float> { static constexpr int N = 4; };
template <> struct ProbVec<__nv_bfloat16> { static constexpr int N = 8; };

__device__ __forceinline__ float prob_f32(float x) { return x; }
__device__ __forceinline__ float prob_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void prob_unpack(const uint4 &w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y); v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void prob_unpack(const uint4 &w, float (&v)[8]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int t = 0; t < 4; ++t) { v[2 * t] = bf16_lo(a[t]); v[2 * t + 1] = bf16_hi(a[t]); }
}

// Draft entries: those below zero count as zero, so that no target entry of zero or less is accepted or
// drawn (NaN stays NaN).
__device__ __forceinline__ float draft_f32(float x) {
    float m;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(m) : "f"(x));
    return m;
}
__device__ __forceinline__ float draft_f32(__nv_bfloat16 x) { return draft_f32(__bfloat162float(x)); }
__device__ __forceinline__ void draft_unpack(const uint4 &w, float (&v)[4]) {
    prob_unpack(w, v);
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = draft_f32(v[t]);
}
__device__ __forceinline__ void draft_unpack(const uint4 &w, float (&v)[8]) {
    uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int t = 0; t < 4; ++t) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a[t]) : "r"(0u));
    prob_unpack(make_uint4(a[0], a[1], a[2], a[3]), v);
}

// The row that is drawn from: r(v) = max(p(v) - q(v), 0), or max(p(v), 0) without q; a point
// draft is a q of 1 at its token.  The comparison is exact in fp32 and false for NaN, so such an
// entry is never drawn; the difference is taken in 64 bits.
template <typename T>
struct ResidualRow {
    const T *p, *q;
    int point;       // the point draft's token, or -1
    __device__ __forceinline__ double value(float pv, float qv, int v) const {
        const float y = v == point ? 1.f : qv;
        return pv > y ? (double)pv - (double)y : 0.0;
    }
    __device__ __forceinline__ double at(int v) const {
        return value(prob_f32(p[v]), q != nullptr ? draft_f32(q[v]) : 0.f, v);
    }
};

// Sum of r over [v0, v1) by one warp (v0 and v1 multiples of the vector width when VEC,
// but for the row's end).
template <typename T, bool VEC>
__device__ __forceinline__ double residual_sum(const ResidualRow<T> &r, int v0, int v1, int lane) {
    constexpr int N = ProbVec<T>::N;
    double s0 = 0.0, s1 = 0.0;
    if (VEC) {
        constexpr int U = 4;
        for (int v = v0 + lane * N; v + N <= v1; v += 32 * N * U) {
            uint4 a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int w = v + u * 32 * N;
                a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);     // (past the piece: nothing)
                if (w + N <= v1) {
                    a[u] = __ldg(reinterpret_cast<const uint4 *>(r.p + w));
                    if (r.q != nullptr) b[u] = __ldg(reinterpret_cast<const uint4 *>(r.q + w));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[N], y[N];
                prob_unpack(a[u], x);
                draft_unpack(b[u], y);
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    const int w = v + u * 32 * N + e;
                    s0 += r.value(x[e], y[e], w);
                    s1 += r.value(x[e + 1], y[e + 1], w + 1);
                }
            }
        }
        // the row's last elements, fewer than a vector
        const int tail = v1 - (v1 - v0) % N;
        if (lane < v1 - tail) s0 += r.at(tail + lane);
    } else {
        constexpr int U = 8;
        for (int v = v0 + lane; v < v1; v += 32 * U) {
            float x[U], y[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int w = v + 32 * u;
                x[u] = w < v1 ? prob_f32(r.p[w]) : 0.f;
                y[u] = w < v1 && r.q != nullptr ? draft_f32(r.q[w]) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < U; u += 2) {
                s0 += r.value(x[u], y[u], v + 32 * u);
                s1 += r.value(x[u + 1], y[u + 1], v + 32 * (u + 1));
            }
        }
    }
    double s = s0 + s1;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    return s;
}

__device__ __forceinline__ double warp_scan(double c, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double n = __shfl_up_sync(0xffffffffu, c, off);
        if (lane >= off) c += n;
    }
    return c;
}

struct FindShared {
    double warp[kVerifyWarps];
    int hit, last;
};
// First v in [v0, v1) with base + sum_{w = v0 .. v} r_w > target, by the whole CTA; where rounding
// leaves none, the last v of the piece with r_v > 0.  A thread takes a vector's worth of
// consecutive entries: their sum, a scan over the CTA, and the thread whose range the target falls
// in looks at its entries one by one.  (A warp alone, row by row, took 16 us for the 2000 entries of
// a piece: one long chain of reads, conversions and shuffles.)
template <typename T>
__device__ __forceinline__ int residual_find(const ResidualRow<T> &r, int v0, int v1, double base, double target, bool vec,
                                             FindShared &s) {
    constexpr int E = ProbVec<T>::N;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        s.hit = INT_MAX;
        s.last = -1;
    }
    double run = base;
    for (int b = v0; b < v1; b += E * kVerifyThreads) {
        const int w0 = b + (int)threadIdx.x * E;
        float x[E], y[E];
        if (vec && w0 + E <= v1) {
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(r.p + w0));
            uint4 c = make_uint4(0u, 0u, 0u, 0u);
            if (r.q != nullptr) c = __ldg(reinterpret_cast<const uint4 *>(r.q + w0));
            prob_unpack(a, x);
            draft_unpack(c, y);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                x[e] = w0 + e < v1 ? prob_f32(r.p[w0 + e]) : 0.f;
                y[e] = w0 + e < v1 && r.q != nullptr ? draft_f32(r.q[w0 + e]) : 0.f;
            }
        }
        double mine = 0.0;
        int last = -1;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const double z = r.value(x[e], y[e], w0 + e);
            if (z > 0.0) last = w0 + e;
            mine += z;
        }
        const double incl = warp_scan(mine, lane);
        __syncthreads();                 // (the values of the turn before are read)
        if (lane == 31) s.warp[warp] = incl;
        __syncthreads();
        double before = run;
#pragma unroll
        for (int k = 0; k < kVerifyWarps; ++k) {
            if (k < warp) before += s.warp[k];
            run += s.warp[k];
        }
        double c = before + incl - mine;
        if (last >= 0) {
            if (c + mine > target) {
                int v = last;
                bool found = false;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const double z = r.value(x[e], y[e], w0 + e);
                    c += z;
                    if (!found && z > 0.0 && c > target) {
                        v = w0 + e;
                        found = true;
                    }
                }
                atomicMin(&s.hit, v);
            }
            atomicMax(&s.last, last);
        }
        __syncthreads();
        if (s.hit != INT_MAX) break;
    }
    return s.hit != INT_MAX ? s.hit : s.last;
}

__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, kVerifyPerSm) verify_kernel(const VerifyParams a) {
    __shared__ double s_sum[kVerifyWarps];
    __shared__ int s_n, s_len;
    __shared__ FindShared s_find;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t ncta;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncta));
    const int C = (int)ncta, rank = (int)cluster_ctarank();
    const int b = blockIdx.x / C;
    const T *p = static_cast<const T *>(a.p) + (long long)b * a.p_b;
    const T *q = a.q != nullptr ? static_cast<const T *>(a.q) + (long long)b * a.q_b : nullptr;
    // ---- drafts accepted before the first refusal (every CTA of the cluster finds it itself; the
    //      first 32 drafts and their numbers are read while the length is on its way)
    const float u_draw = __ldg(a.u_sample + b);
    if (warp == 0) {
        int x = lane < a.L ? __ldg(a.drafts + (long long)b * a.L + lane) : -1;
        float u = lane < a.L ? __ldg(a.u_accept + (long long)b * a.L + lane) : 0.f;
        int len = a.lens != nullptr ? __ldg(a.lens + b) : a.L;
        len = len < 0 ? 0 : (len > a.L ? a.L : len);
        int n = len;
        for (int i0 = 0; i0 < len && n == len; i0 += 32) {
            const int i = i0 + lane;
            if (i0 > 0 && i < len) {
                x = __ldg(a.drafts + (long long)b * a.L + i);
                u = __ldg(a.u_accept + (long long)b * a.L + i);
            }
            bool refuse = i < len;                // also for a token outside the vocabulary, and for NaN
            if (i < len && x >= 0 && x < a.V) {
                const double px = (double)prob_f32(p[(long long)i * a.p_l + x]);
                const double qx = q != nullptr ? (double)draft_f32(q[(long long)i * a.q_l + x]) : 1.0;
                refuse = !((double)u * qx < px);
            }
            const unsigned m = __ballot_sync(0xffffffffu, refuse);
            if (m) n = i0 + __ffs(m) - 1;
        }
        if (lane == 0) {
            s_n = n;
            s_len = len;
        }
    }
    __syncthreads();
    const int n = s_n, len = s_len;
    if (rank == 0) {
        if (threadIdx.x == 0) a.accepted[b] = n;
        for (int i = threadIdx.x; i <= a.L; i += kVerifyThreads)
            if (i != n) a.tokens[(long long)b * (a.L + 1) + i] = i < n ? __ldg(a.drafts + (long long)b * a.L + i) : -1;
    }

    ResidualRow<T> r;
    r.p = p + (long long)n * a.p_l;
    r.q = n < len && q != nullptr ? q + (long long)n * a.q_l : nullptr;
    r.point = n < len && q == nullptr ? __ldg(a.drafts + (long long)b * a.L + n) : -1;
    // consecutive pieces, one per warp of the cluster, in whole vectors
    constexpr int N = ProbVec<T>::N;
    const int vecs = (a.V + N - 1) / N;
    const int per = (vecs + C * kVerifyWarps - 1) / (C * kVerifyWarps);
    const int piece = rank * kVerifyWarps + warp;
    const long long lo = (long long)piece * per * N;
    const int v0 = lo < a.V ? (int)lo : a.V;
    const int v1 = lo + (long long)per * N < a.V ? (int)(lo + (long long)per * N) : a.V;

    bool drawn = false;
    for (int pass = 0; pass < 2 && !drawn; ++pass) {
        const double s = a.vec ? residual_sum<T, true>(r, v0, v1, lane) : residual_sum<T, false>(r, v0, v1, lane);
        if (lane == 0) s_sum[warp] = s;
        cluster_sync_all();
        // every warp of the cluster takes all the pieces' sums, in order, four a lane
        constexpr int K = kVerifyMaxCluster * kVerifyWarps / 32;
        double at[K], lane_sum = 0.0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = K * lane + k;
            at[k] = i < C * kVerifyWarps
                        ? ld_cluster_f64(map_to_rank(smem_u32(&s_sum[i % kVerifyWarps]), (uint32_t)(i / kVerifyWarps)))
                        : 0.0;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) lane_sum += at[k];
        const double upto = warp_scan(lane_sum, lane);
        const double total = __shfl_sync(0xffffffffu, upto, 31);
        // (the sums are read: they may be overwritten, or their CTA gone, after this)
        cluster_sync_all();
        if (total > 0.0) {
            drawn = true;
            const double target = (double)u_draw * total;
            // the piece the target falls in, else the last non-empty one
            double run = upto - lane_sum, before = 0.0;
            int first = -1, last = -1;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (at[k] > 0.0) {
                    last = K * lane + k;
                    if (first < 0 && run + at[k] > target) {
                        first = K * lane + k;
                        before = run;
                    }
                }
                run += at[k];
            }
            const unsigned hit = __ballot_sync(0xffffffffu, first >= 0), some = __ballot_sync(0xffffffffu, last >= 0);
            int owner;
            if (hit) {
                owner = __shfl_sync(0xffffffffu, first, __ffs(hit) - 1);
                before = __shfl_sync(0xffffffffu, before, __ffs(hit) - 1);
            } else {
                owner = __shfl_sync(0xffffffffu, last, 31 - __clz(some));
                before = 0.0;
            }
            if (owner / kVerifyWarps == rank) {
                const long long o0 = (long long)owner * per * N, o1 = o0 + (long long)per * N;
                const int v = residual_find<T>(r, o0 < a.V ? (int)o0 : a.V, o1 < a.V ? (int)o1 : a.V, before,
                                               hit ? target : 1e300, a.vec != 0, s_find);
                if (threadIdx.x == 0) a.tokens[(long long)b * (a.L + 1) + n] = v;
            }
        }
        // nothing left after the subtraction: draw from the target's own row
        r.q = nullptr;
        r.point = -1;
    }
    if (!drawn && rank == 0 && threadIdx.x == 0) a.tokens[(long long)b * (a.L + 1) + n] = -1;
}

}  // namespace kvattn
