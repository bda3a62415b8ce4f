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
    double log2_base;              // rotation base, log2
    int rotate, interleaved;
    int rows_per_cta;              // rows (heads of q, then k, then v) of a token one CTA takes
};

constexpr int kRowThreads = 128;
constexpr int kRowMaxPairs = 128;  // head_dim <= 256

// cos and sin of position * base^(-2i/d) for pair i.  The angle is formed in turns in fp64
// (a position of 10^6 leaves it good to ~1e-10 of a turn) and only its fraction of a turn is
// taken to fp32, so no reduction of a large argument is left to the fp32 functions; their
// results are off by ~2e-7 at most, against 2^-9 of the bf16 rounding and 2^-4 of E4M3.
__device__ __forceinline__ float2 rope_turn(int pos, int i, int d, double log2_base) {
    const double turns = (double)pos * (exp2(-2.0 * (double)i / (double)d * log2_base) * 0.15915494309189533577);
    const float f = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.f * f, &s, &c);
    return make_float2(c, s);
}

// One CTA per token (or per part of a token's rows when there are few tokens); LPR lanes of
// eight elements make a row.  The rows' loads go out before the token's cos / sin table is
// formed, so the fp64 work hides behind them.
// Bound by memory: the new rows are read once (a fused projection's slices in place), the codes
// and scales written once.
template <int LPR>
__global__ void __launch_bounds__(kRowThreads) row_append_kernel(const RowAppendParams p) {
    __shared__ float2 s_turn[kRowMaxPairs];
    constexpr int RPC = kRowThreads / LPR;       // rows the CTA handles at once
    constexpr int U = 4;                         // of these per thread in flight
    const int n = blockIdx.x;
    const int sub = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int n_rows = p.n_q + 2 * p.n_kv;
    const int r0 = blockIdx.y * p.rows_per_cta;
    const int r1 = min(r0 + p.rows_per_cta, n_rows);
    const bool lane_on = l * 8 < p.d;
    const long long slot = __ldg(p.slots + n);
    const bool store = slot >= 0 && slot < p.n_slots;
    const int page = store ? (int)(slot / p.page_size) : 0;
    const int prow = store ? (int)(slot - (long long)page * p.page_size) : 0;

    auto source = [&](int r) -> const uint4 * {
        const __nv_bfloat16 *row;
        if (r < p.n_q) row = p.q + (long long)n * p.q_stride + (long long)r * p.d;
        else if (r < p.n_q + p.n_kv) row = p.k_new + (long long)n * p.k_stride + (long long)(r - p.n_q) * p.d;
        else row = p.v_new + (long long)n * p.v_stride + (long long)(r - p.n_q - p.n_kv) * p.d;
        return reinterpret_cast<const uint4 *>(row + l * 8);
    };
    bool have_table = !p.rotate;
    for (int base = r0; base < r1; base += RPC * U) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = base + u * RPC + sub;
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            if (r < r1 && lane_on && (r < p.n_q || store)) x[u] = *source(r);
        }
        if (!have_table) {       // (uniform over the CTA)
            const int pos = __ldg(p.positions + n);
            for (int i = threadIdx.x; i < p.d / 2; i += kRowThreads) s_turn[i] = rope_turn(pos, i, p.d, p.log2_base);
            __syncthreads();
            have_table = true;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = base + u * RPC + sub;
            const bool row_on = r < r1 && (r < p.n_q || store);
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            float y[8];
#pragma unroll
            for (int t = 0; t < 4; ++t) { y[2 * t] = bf16_lo(w[t]); y[2 * t + 1] = bf16_hi(w[t]); }
            // the other half's row elements (split halves): lanes d / 16 apart.  Every lane of
            // the warp takes part in the exchange, whatever its row.
            const int half = p.d / 16;
            uint32_t o[4];
            if (p.rotate && !p.interleaved) {
                const int src = l < half ? l + half : l - half;
#pragma unroll
                for (int t = 0; t < 4; ++t) o[t] = __shfl_sync(0xffffffffu, w[t], src & (LPR - 1), LPR);
            }
            if (p.rotate && r < p.n_q + p.n_kv && lane_on) {
                if (p.interleaved) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const float2 cs = s_turn[l * 4 + t];
                        const float a = y[2 * t], b = y[2 * t + 1];
                        y[2 * t] = fmaf(a, cs.x, -b * cs.y);
                        y[2 * t + 1] = fmaf(a, cs.y, b * cs.x);
                    }
                } else {
                    const bool low = l < half;
                    const int i0 = (low ? l : l - half) * 8;
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        const float2 cs = s_turn[i0 + t];
                        const float other = (t & 1) ? bf16_hi(o[t / 2]) : bf16_lo(o[t / 2]);
                        y[t] = low ? fmaf(y[t], cs.x, -other * cs.y) : fmaf(other, cs.y, y[t] * cs.x);
                    }
                }
            }
            float a = 0.f;
#pragma unroll
            for (int t = 0; t < 8; ++t) a = fmaxf(a, fabsf(y[t]));     // (fmaxf passes over NaN)
#pragma unroll
            for (int m = LPR / 2; m >= 1; m >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, m));
            if (!row_on || !lane_on) continue;
            if (r < p.n_q) {
                uint4 v;
                v.x = pack_bf16x2(y[0], y[1]);
                v.y = pack_bf16x2(y[2], y[3]);
                v.z = pack_bf16x2(y[4], y[5]);
                v.w = pack_bf16x2(y[6], y[7]);
                *reinterpret_cast<uint4 *>(p.q_out + (long long)n * p.q_out_stride + (long long)r * p.d + l * 8) = v;
                continue;
            }
            a = fminf(fmaxf(a, kRowAmaxMin), kRowAmaxMax);
            const float inv = __fdiv_rn(448.f, a);
            uint32_t c[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint16_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * t] * inv, y[4 * t + 1] * inv),
                                                             __NV_SATFINITE, __NV_E4M3);
                const uint16_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * t + 2] * inv, y[4 * t + 3] * inv),
                                                             __NV_SATFINITE, __NV_E4M3);
                c[t] = (uint32_t)lo | ((uint32_t)hi << 16);
            }
            const bool key = r < p.n_q + p.n_kv;
            const int j = r - p.n_q - (key ? 0 : p.n_kv);
            const long long row = ((long long)page * p.n_kv + j) * p.page_size + prow;
            *reinterpret_cast<uint2 *>((key ? p.k_pages : p.v_pages) + row * p.d + l * 8) = make_uint2(c[0], c[1]);
            if (l == 0) (key ? p.k_scales : p.v_scales)[row] = __fdiv_rn(a, 448.f);
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
// Bound by memory (1 byte read and 2 written per element).
constexpr int kGatherRows = 2;     // rows a lane has in flight
template <int LPR>
__global__ void __launch_bounds__(256) row_gather_kernel(const RowGatherParams p) {
    constexpr int RPC = 256 / LPR;
    constexpr int U = kGatherRows;
    const int sub = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int j = blockIdx.y;
    if (l * 16 >= p.d) return;
    long long row[U];
    uint4 code[2 * U];
    float sc[2 * U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long n = (long long)blockIdx.x * (RPC * U) + u * RPC + sub;
        row[u] = -1;
        if (n < p.N) {
            const long long slot = __ldg(p.slots + n);
            if (slot >= 0 && slot < p.n_slots) {
                const long long page = slot / p.page_size;
                row[u] = (page * p.n_kv + j) * p.page_size + (slot - page * p.page_size);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        code[2 * u] = code[2 * u + 1] = make_uint4(0u, 0u, 0u, 0u);
        sc[2 * u] = sc[2 * u + 1] = 0.f;
        if (row[u] >= 0) {
            code[2 * u] = __ldg(reinterpret_cast<const uint4 *>(p.k_pages + row[u] * p.d + l * 16));
            code[2 * u + 1] = __ldg(reinterpret_cast<const uint4 *>(p.v_pages + row[u] * p.d + l * 16));
            sc[2 * u] = __ldg(p.k_scales + row[u]);
            sc[2 * u + 1] = __ldg(p.v_scales + row[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long n = (long long)blockIdx.x * (RPC * U) + u * RPC + sub;
        if (n >= p.N) continue;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t w[4] = {code[2 * u + t].x, code[2 * u + t].y, code[2 * u + t].z, code[2 * u + t].w};
            const float s = sc[2 * u + t];
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
}

}  // namespace kvattn
