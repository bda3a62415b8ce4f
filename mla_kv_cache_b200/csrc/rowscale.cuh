// rowscale.cuh -- a paged E4M3 KV cache with one scale per cached row (token and KV head):
// the write of new tokens (with their rotary embedding) and the read back to bf16.
//
// A row's scale comes from the row itself, so a cache can be quantised as it is written: no
// calibration pass, and an outlier token costs no other token precision.  For a row y (a
// rotated key or a value, fp32):
//     a = max(max_i |y_i|, 2^-55), at most FLT_MAX (NaN elements are passed over)
//     scale = a / 448,   code_i = E4M3(y_i * (448 / a))      (nearest, ties to even, saturated)
// and the cached value is code_i * scale: off by at most half an E4M3 step of the row's own
// size.  A NaN element becomes the NaN code and leaves its row's other elements alone.
#pragma once
#include "common.cuh"

namespace kvattn {

constexpr float kRowAmaxMin = 2.7755575615628914e-17f;   // 2^-55: 448 / a stays finite, 1 / scale too
constexpr float kRowAmaxMax = 3.4028234663852886e38f;

// ------------------------------------------------------------------------------- the write
struct RowAppendParams {
    const __nv_bfloat16 *q;        // [N, n_q, d], tokens q_stride elements apart (null: no query)
    __nv_bfloat16 *q_out;          // [N, n_q, d], tokens q_out_stride apart (may be q itself)
    const __nv_bfloat16 *k_new;    // [N, n_kv, d], tokens k_stride apart
    const __nv_bfloat16 *v_new;    // [N, n_kv, d], tokens v_stride apart
    const int32_t *positions;      // [N] (read only when rotating)
    const long long *slots;        // [N] page * page_size + row; outside the pool: not written
    uint8_t *k_pages, *v_pages;    // [num_pages, n_kv, page_size, d] codes
    float *k_scales, *v_scales;    // [num_pages, n_kv, page_size]
    long long q_stride, q_out_stride, k_stride, v_stride;
    int N, n_q, n_kv, d, page_size;
    long long n_slots;             // num_pages * page_size
    double turn_lo[16], turn_hi[8];   // turns per position of pair 16 h + l: turn_hi[h] * turn_lo[l]
    int rotate, interleaved;
    int parts, rows_per_part;      // a token's rows (heads of q, then k, then v) are shared out over warps
};

constexpr int kRowThreads = 128;

// cos and sin of position * base^(-2i/d) for pair i.  The angle is formed in turns in fp64
// (a position of 10^6 leaves it good to ~1e-10 of a turn) and only its fraction of a turn is
// taken to fp32, so no reduction of a large argument is left to the fp32 functions; their
// results are off by ~2e-7 at most, against 2^-8 of the bf16 rounding and 2^-4 of E4M3.  A pair's
// turns per position are a product of two of the 24 powers that come with the launch.
__device__ __forceinline__ float2 rope_turn(const RowAppendParams &p, int pos, int i) {
    const double turns = (double)pos * (p.turn_hi[i >> 4] * p.turn_lo[i & 15]);
    const float f = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.f * f, &s, &c);
    return make_float2(c, s);
}

// Sixteen elements of a row: 8 at `at` and 8 half a row further.
struct RowHalves {
    uint4 lo, hi;
};
__device__ __forceinline__ void unpack8(const uint4 &v, float (&y)[8]) {
    y[0] = bf16_lo(v.x); y[1] = bf16_hi(v.x); y[2] = bf16_lo(v.y); y[3] = bf16_hi(v.y);
    y[4] = bf16_lo(v.z); y[5] = bf16_hi(v.z); y[6] = bf16_lo(v.w); y[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
    return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
}
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float inv) {
    uint32_t c[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint16_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * t] * inv, y[4 * t + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        const uint16_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * t + 2] * inv, y[4 * t + 3] * inv), __NV_SATFINITE, __NV_E4M3);
        c[t] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
    return make_uint2(c[0], c[1]);
}

// A warp takes a token (or a part of its rows where there are few tokens); LPR lanes make a row,
// a lane the elements i .. i + 7 of each half, so that both elements of every pair are its own,
// in either pairing, and its eight cosines and sines serve all rows of the token from registers.
// Bound by memory at best (the new rows are read once, a fused projection's slices in place; the
// codes and scales written once) and by instructions next: a form with one vector a lane, its
// partner by shuffles and the cosines in shared memory took 65 us for 8192 tokens of 64 + 2 * 8
// heads of 128 (floor 49).
template <int LPR>
__global__ void __launch_bounds__(kRowThreads) row_append_kernel(const __grid_constant__ RowAppendParams p) {
    constexpr int RPW = 32 / LPR;                // rows the warp handles at once
    // Of these in flight: two of the queries (8192 tokens of 64 + 2 * 8 heads of 128: 57.3 us, 58.5 with
    // one), one of the keys or values (two cost registers: 17.3 us for 8192 tokens of 8 + 2 * 8 heads of 64,
    // 14.3 with one, against 7.4 and 8.5 for 700 of the former).
    constexpr int UQ = 2;
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int n = (int)(item / p.parts), part = (int)(item - (long long)n * p.parts);
    if (n >= p.N) return;
    const int sub = lane / LPR, l = lane % LPR;
    const int n_rows = p.n_q + 2 * p.n_kv, half = p.d >> 1;
    const int r0 = part * p.rows_per_part, r1 = min(r0 + p.rows_per_part, n_rows);
    const bool lane_on = l * 8 < half;
    const int at = lane_on ? l * 8 : 0;
    const long long slot = __ldg(p.slots + n);

    auto load = [&](const __nv_bfloat16 *row) -> RowHalves {
        // (plain loads: the queries may be written in place)
        RowHalves x;
        x.lo = *reinterpret_cast<const uint4 *>(row + at);
        x.hi = *reinterpret_cast<const uint4 *>(row + half + at);
        return x;
    };
    // pairs of this lane: at + t (split halves); at / 2 + t and half / 2 + at / 2 + t (interleaved)
    float c[8], s[8];
    if (p.rotate && r0 < p.n_q + p.n_kv) {
        const int pos = __ldg(p.positions + n);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int i = p.interleaved ? (at >> 1) + (t & 3) + (t >= 4 ? half >> 1 : 0) : at + t;
            const float2 cs = rope_turn(p, pos, i);
            c[t] = cs.x;
            s[t] = cs.y;
        }
    }
    auto turn = [&](float (&a)[8], float (&b)[8]) {
        if (p.interleaved) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float x = a[2 * t], y = a[2 * t + 1], z = b[2 * t], w = b[2 * t + 1];
                a[2 * t] = fmaf(x, c[t], -y * s[t]);
                a[2 * t + 1] = fmaf(x, s[t], y * c[t]);
                b[2 * t] = fmaf(z, c[4 + t], -w * s[4 + t]);
                b[2 * t + 1] = fmaf(z, s[4 + t], w * c[4 + t]);
            }
        } else {
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float x = a[t], y = b[t];
                a[t] = fmaf(x, c[t], -y * s[t]);
                b[t] = fmaf(x, s[t], y * c[t]);
            }
        }
    };

    // ---- queries
    const int q1 = min(r1, p.n_q);
    if (r0 < q1) {
        const __nv_bfloat16 *src = p.q + (long long)n * p.q_stride;
        __nv_bfloat16 *dst = p.q_out + (long long)n * p.q_out_stride;
        for (int base = r0; base < q1; base += RPW * UQ) {
            RowHalves x[UQ];
#pragma unroll
            for (int u = 0; u < UQ; ++u) {
                const int r = base + u * RPW + sub;
                if (r < q1) x[u] = load(src + r * p.d);
            }
#pragma unroll
            for (int u = 0; u < UQ; ++u) {
                const int r = base + u * RPW + sub;
                if (r >= q1 || !lane_on) continue;
                if (p.rotate) {
                    float a[8], b[8];
                    unpack8(x[u].lo, a);
                    unpack8(x[u].hi, b);
                    turn(a, b);
                    x[u].lo = pack8(a);
                    x[u].hi = pack8(b);
                }
                *reinterpret_cast<uint4 *>(dst + r * p.d + at) = x[u].lo;
                *reinterpret_cast<uint4 *>(dst + r * p.d + half + at) = x[u].hi;
            }
        }
    }
    // ---- keys, then values
    if (slot < 0 || slot >= p.n_slots) return;
    const int page = (int)(slot / p.page_size), prow = (int)(slot - (long long)page * p.page_size);
    const long long row0 = (long long)page * p.n_kv * p.page_size + prow;
#pragma unroll 1
    for (int kv = 0; kv < 2; ++kv) {
        const int first = p.n_q + kv * p.n_kv;
        const int j0 = max(r0 - first, 0), j1 = min(r1 - first, p.n_kv);
        if (j0 >= j1) continue;
        const __nv_bfloat16 *src = kv ? p.v_new + (long long)n * p.v_stride : p.k_new + (long long)n * p.k_stride;
        uint8_t *codes = kv ? p.v_pages : p.k_pages;
        float *scales = kv ? p.v_scales : p.k_scales;
        for (int base = j0; base < j1; base += RPW) {
            const int j = base + sub;
            RowHalves x;
            x.lo = x.hi = make_uint4(0u, 0u, 0u, 0u);
            if (j < j1 && lane_on) x = load(src + j * p.d);
            float a[8], b[8];
            unpack8(x.lo, a);
            unpack8(x.hi, b);
            if (p.rotate && kv == 0 && lane_on) turn(a, b);
            float m = 0.f;
#pragma unroll
            for (int t = 0; t < 8; ++t) m = fmaxf(m, fmaxf(fabsf(a[t]), fabsf(b[t])));     // (passes over NaN)
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (j >= j1 || !lane_on) continue;
            m = fminf(fmaxf(m, kRowAmaxMin), kRowAmaxMax);
            const float inv = __fdiv_rn(448.f, m);
            const long long row = row0 + (long long)j * p.page_size;
            *reinterpret_cast<uint2 *>(codes + row * p.d + at) = codes8(a, inv);
            *reinterpret_cast<uint2 *>(codes + row * p.d + half + at) = codes8(b, inv);
            if (l == 0) scales[row] = __fdiv_rn(m, 448.f);
        }
    }
}

// ------------------------------------------------------------------------------- the read back
struct RowGatherParams {
    const uint8_t *k_pages, *v_pages;    // [num_pages, n_kv, page_size, d] codes
    const float *k_scales, *v_scales;    // [num_pages, n_kv, page_size]
    const long long *slots;              // [N]; outside the pool: a row of zeros
    __nv_bfloat16 *k_out, *v_out;        // [n_kv, N, d], heads k_head / v_head elements apart
    long long k_head, v_head;
    int N, n_kv, d, page_size;
    long long n_slots;
};

// Sixteen codes a lane (one 16-byte load, two 16-byte stores); LPR lanes make a row.  A CTA
// takes consecutive tokens of one head, whose rows lie next to each other within a page.
// Bound by memory (1 byte read and 2 written per element).  A lane has one row of keys and one of
// values in flight (with two a prompt of 32768 tokens took 41.7 us, with four 46.2; 39.7 so).
template <int LPR>
__global__ void __launch_bounds__(256) row_gather_kernel(const RowGatherParams p) {
    const int sub = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int j = blockIdx.y;
    const long long n = (long long)blockIdx.x * (256 / LPR) + sub;
    if (l * 16 >= p.d || n >= p.N) return;
    uint4 code[2];
    float sc[2] = {0.f, 0.f};
    code[0] = code[1] = make_uint4(0u, 0u, 0u, 0u);
    const long long slot = __ldg(p.slots + n);
    if (slot >= 0 && slot < p.n_slots) {
        const long long page = slot / p.page_size;
        const long long row = (page * p.n_kv + j) * p.page_size + (slot - page * p.page_size);
        code[0] = __ldcs(reinterpret_cast<const uint4 *>(p.k_pages + row * p.d + l * 16));
        code[1] = __ldcs(reinterpret_cast<const uint4 *>(p.v_pages + row * p.d + l * 16));
        sc[0] = __ldg(p.k_scales + row);
        sc[1] = __ldg(p.v_scales + row);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint32_t w[4] = {code[t].x, code[t].y, code[t].z, code[t].w};
        const float s = sc[t];
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // (codes are exact in f16, so the product with the scale is rounded once to bf16)
            const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((uint16_t)(w[e] & 0xffffu), __NV_E4M3)));
            const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((uint16_t)(w[e] >> 16), __NV_E4M3)));
            o[2 * e] = pack_bf16x2(a.x * s, a.y * s);
            o[2 * e + 1] = pack_bf16x2(b.x * s, b.y * s);
        }
        uint4 *dst = reinterpret_cast<uint4 *>((t ? p.v_out + j * p.v_head : p.k_out + j * p.k_head) + n * p.d + l * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

}  // namespace kvattn
