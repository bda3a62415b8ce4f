// rs_decode.cuh -- decode attention over a row-scaled E4M3 cache (rowscale.cuh).
//
// For query row r (a head of the group at one of the new tokens) and cached token t with codes
// kc_t, vc_t and scales ks_t, vs_t:
//     s_t = scale * ks_t * (q_r . kc_t),   out_r = sum_t softmax(s)_t * vs_t * vc_t
// The key scale multiplies a score, the value scale a weight, so the codes go into the products
// as they are: every E4M3 code is exact in f16, and so is a bf16 query after a power of two brings
// its largest element to [2^13, 2^14) (elements down to 2^-27 of it keep all their bits).  The
// weights fed to the value product are w_t = 2^(s_t - m) * vs_t in f16, m running over
// s_t + log2(vs_t) so that they stay at or below 2^8 and keep 11 bits; row sums take 2^(s_t - m).
//
// A decode step reads every cached byte once for a few query rows, so the kernel is bound by
// memory as long as an SM keeps up with ~23 bytes a cycle: 1400 cycles for a tile of 128 tokens.
// One CTA per SM streams its range of tiles (schedule.cuh) through a ring; the group's rows are
// the M rows of warp-level m16n8k16 f16 MMAs (MT m-tiles of 16), which need 560 cycles a tile for
// each m-tile (measured, 8.7 cycles an MMA and scheduler), the conversions E4M3 -> f16 270.  Streaming
// runs at 5.2 TB/s (16 equal sequences of 8192 tokens, 64 / 8 heads).  The same decode on tcgen05 with
// E4M3 operands (query and weights in two E4M3 parts, the tokens on the MMA rows, whose maxima cross
// the 128 token lanes) ran at 4.9; 42.4 us against 35.9 here for 16 sequences of 1024..8192 tokens, 20.4
// against 15.1 for 8 of up to 1000 with 5 new tokens, 22.5 against 24.3 for 4 of 32768 with 32 / 1
// heads.  The 8-bit mma.sync is no help: 20 cycles each here.
//
// Warps: a producer and 8 consumers.  A consumer works on 32 tokens at a time, all 128
// dimensions and one m-tile, with its own running maximum, sum and output in registers; blocks
// of 32 tokens go round the warps of an m-tile.  At a piece's end the warps' outputs are joined
// through shared memory and written as the unit's result or as a partial for the combine kernel.
#pragma once
#include "common.cuh"
#include "gqa_decode.cuh"
#include "schedule.cuh"
#include "tc05.cuh"
#include "window.cuh"

namespace kvattn {

// k_scale / v_scale of GqaParams are unused; out holds bf16.
struct RsParams : GqaParams {
    const float *k_rows, *v_rows;   // [pages, n_kv, page_size]
    int pages;
    int start_align;                // windowed ranges start at a tile boundary in a paged cache
};

namespace rs {

constexpr int TILE = 128, D = 128, BLK = 32;    // tokens a tile, dimensions, tokens a warp takes at once
constexpr int NCW = 8;                          // consumer warps
constexpr int NTHREADS = 128 + NCW * 32;        // the first warpgroup holds the producer
// registers of a thread after the split: a consumer holds its query rows and outputs
constexpr int REGS_LAUNCH = 168, REGS_PROD = 40, REGS_CONS = 232;
static_assert(128 * REGS_PROD + NCW * 32 * REGS_CONS <= NTHREADS * REGS_LAUNCH, "registers of the launch");
constexpr int KV_BYTES = TILE * D;
constexpr int STAGE = 2 * KV_BYTES;
constexpr int NST = 4;
constexpr int MPAD = D + 4;                     // (rows on different banks)
constexpr int MERGE_FLOATS = 16 * MPAD + 32;    // a warp's O[16][D], m[16], l[16]
constexpr int OFF_MERGE = NST * STAGE;
constexpr int OFF_WTS = OFF_MERGE + NCW * MERGE_FLOATS * 4;
constexpr int OFF_SCALES = OFF_WTS + 64 * (NCW + 1) * 4;    // [rows][slots] weights, [rows] lse
constexpr int OFF_BARS = OFF_SCALES + NCW * 3 * BLK * 4;    // a warp's block: ks, vs, log2(vs) of its 32 tokens
constexpr int OFF_PREFIX = OFF_BARS + 128;
// What a unit's start (its query, pages and scales) and end (the join of the warps) count for in
// the work split, in tiles (~4500 cycles and a worker's wait for its first tile; a tile is 1450 cycles
// with one m-tile, 3300 with two).  Without it a worker of many short sequences finishes last: 16 ragged
// sequences 43.5 us with 0, 38.7 with 3, 36.2 with 5; with two m-tiles 16.9, 16.0 and 17.6, 14.4 with 2.
__host__ __device__ constexpr int unit_cost(int MT) { return MT == 1 ? 5 : 2; }
constexpr float RESCALE = 8.f;
constexpr int smem_bytes(int B) { return 1024 + OFF_PREFIX + (B + 1) * 4; }

struct Bars {
    uint64_t full[NST], empty[NST], cons;
    int abort_flag;
};
static_assert(sizeof(Bars) <= 128, "barrier block overflows its slot");

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The four E4M3 codes of a word as f16 pairs (exact; the lower byte of each two in the lower half).
__device__ __forceinline__ void e4m3x4(uint32_t w, uint32_t &a, uint32_t &b) {
    asm("{\n\t.reg .b16 x, y;\n\t"
        "mov.b32 {x, y}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, x;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
}
// The NaN codes (0x7F or 0xFF) among four E4M3 codes: 0x80 in their bytes.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The piece at position p of the line (schedule.cuh), its tiles without the unit's cost; a piece
// that holds only that has none.
template <int COST>
__device__ __forceinline__ Piece piece_on(const int *s_prefix, int B, int U, long long p, long long p_end, long long w0,
                                          long long &next) {
    Piece pc = piece_at(s_prefix, B, U, p, p_end, w0);
    next = pc.ustart + pc.lt1;
    pc.n_tiles -= COST;
    pc.lt0 = min(pc.lt0, pc.n_tiles);
    pc.lt1 = min(pc.lt1, pc.n_tiles);
    pc.whole = pc.lt0 == 0 && pc.lt1 == pc.n_tiles;
    return pc;
}

}  // namespace rs

// NR: rows of an m-tile in use, 16 or (with one m-tile) 8, which halves a thread's rows.
// MULTI: several new tokens or a window, so that a tile may hold tokens which a row must not see.  Their NaN
// is kept out (below), for 16 ragged sequences with a window of 4096 at 31.3 us instead of 30.4, 8 of up to
// 1000 with 5 new tokens at 15.1 instead of 14.4; one new token without a window pays nothing.
template <int MT, int NR, bool MULTI>
__global__ void __launch_bounds__(rs::NTHREADS, 1)
rs_decode_kernel(const RsParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using namespace rs;
    constexpr int NTS = NCW / MT;                  // warps of an m-tile
    constexpr int BPT = TILE / BLK;                // blocks a tile
    constexpr int ROWS = 16 * MT;
    constexpr int NH = NR / 8;                     // rows a thread
    constexpr int COST = unit_cost(MT);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *merge = reinterpret_cast<float *>(smem + OFF_MERGE);
    float *wts = reinterpret_cast<float *>(smem + OFF_WTS);
    Bars *bars = reinterpret_cast<Bars *>(smem + OFF_BARS);
    volatile int *abort_flag = &bars->abort_flag;
    int *s_prefix = reinterpret_cast<int *>(smem + OFF_PREFIX);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int U = p.n_kv;

    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], MT == 1 ? NCW / 2 : NCW);   // the warps that have a block of the tile
        }
        mbar_init(&bars->cons, NCW);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0)
        build_tile_prefix_on(p.start_align, COST, p.seq_lens, p.B, p.T_max, TILE, s_prefix, lane, p.q_len, p.window);
    if (tid == 32) {
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    __syncthreads();

    const long long total = (long long)s_prefix[p.B] * U;
    const long long W = tiles_per_worker(total, p.workers, p.min_tiles);
    // The combine kernel may be scheduled now; it waits for this grid to finish.
    pdl_launch_dependents();
    long long p0 = (long long)blockIdx.x * W;
    long long p1 = p0 + W < total ? p0 + W : total;
    {   // equal units: consecutive parts of one unit per worker (schedule.cuh)
        const int n_cost = uniform_tile_count(s_prefix, p.B), n_uni = n_cost - COST;
        const long long units = (long long)p.B * U;
        int k = 0;
        const long long Wu = unit_part_tiles(n_uni, units, p.workers, p.min_tiles, &k);
        if (Wu > 0) {
            const long long u = blockIdx.x / k, i = blockIdx.x % k, ub = u * n_cost;
            p0 = p1 = total;
            if (u < units && i * Wu < n_uni) {
                p0 = ub + i * Wu;
                p1 = (i + 1) * Wu < n_uni ? p0 + Wu : ub + n_uni;
            }
        }
    }
    if (p0 >= total) return;

    if (warp < 4) {
        // ------------------------------------------------------------ producer
        regs_dec<REGS_PROD>();
        if (tid != 0) return;
        const uint64_t pol = l2_policy_evict_first();
        int k = 0;
        bool ok = true;
        for (long long pos = p0; pos < p1 && ok;) {
            const Piece pc = piece_on<COST>(s_prefix, p.B, U, pos, p1, p0, pos);
            const int len = clamp_len(__ldg(p.seq_lens + pc.b), p.T_max);
            const int start = active_start_on(p.start_align, len, p.q_len, p.window);
            for (int lt = pc.lt0; lt < pc.lt1; ++lt, ++k) {
                const int s = k % NST;
                if (!mbar_wait(&bars->empty[s], ((uint32_t)(k / NST) & 1u) ^ 1u, FLAG_EMPTY_WAIT, abort_flag)) { ok = false; break; }
                mbar_arrive_expect_tx(&bars->full[s], STAGE);
                const TileSrc src = tile_source(p.block_table, p.max_pages, p.page_size, pc.b, lt, TILE, len, start);
                // (a page outside the pool is read as zeros: a coordinate outside the map)
                const int z = src.page >= 0 && src.page < p.pages ? src.page * p.n_kv + pc.i : -1;
                uint8_t *st = smem + s * STAGE;
                // (the maps see a row of 128 codes as 64 two-byte elements)
                tma_load_3d(st, &kmap, &bars->full[s], 0, src.y, z, pol);
                tma_load_3d(st + KV_BYTES, &vmap, &bars->full[s], 0, src.y, z, pol);
            }
        }
        if (!ok)    // let the copies already issued land before the CTA can exit
            for (int kk = (k > NST ? k - NST : 0); kk < k; ++kk)
                mbar_wait_sleep(&bars->full[kk % NST], (uint32_t)(kk / NST) & 1u, FLAG_FULL_WAIT, nullptr);
        return;
    }

    // ---------------------------------------------------------------- consumers
    regs_inc<REGS_CONS>();
    const int cw = warp - 4, ctid = tid - 128;     // among the consumers
    const int mt = cw % MT, ts = cw / MT;
    const int gid = lane >> 2, c = lane & 3;
    float *my_merge = merge + cw * MERGE_FLOATS;
    float *s_ks = reinterpret_cast<float *>(smem + OFF_SCALES) + cw * 3 * BLK, *s_vs = s_ks + BLK, *s_lv = s_vs + BLK;
    uint32_t cons_uses = 0;
    auto consumer_sync = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->cons);
        return warp_all(mbar_wait(&bars->cons, (cons_uses++) & 1u, FLAG_FULL_WAIT, abort_flag));
    };
    const int R = p.g * p.q_len;                   // query rows of a unit, (position, head)

    // this thread's query rows: new token and head of the group
    bool row_on[NH];
    int row_qi[NH], row_hg[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
        const int row = mt * 16 + gid + 8 * h;
        row_on[h] = row < R;
        row_qi[h] = row_on[h] ? row / p.g : 0;
        row_hg[h] = row_on[h] ? row - row_qi[h] * p.g : 0;
    }

    int k = 0;
    long long pos = p0;
    Piece pc;
    auto next_piece = [&]() -> bool {
        while (pos < p1) {
            pc = piece_on<COST>(s_prefix, p.B, U, pos, p1, p0, pos);
            if (pc.lt0 < pc.lt1) return true;
        }
        return false;
    };
    for (bool more = next_piece(); more;) {
        const int len = clamp_len(__ldg(p.seq_lens + pc.b), p.T_max);
        const int start = active_start_on(p.start_align, len, p.q_len, p.window);
        const int j = pc.i;

        // ---- blocks of this warp: every NTS-th, from this piece's first tile on
        // (with one m-tile a warp has a block of every other tile: the CTA's tile count decides which)
        const int blk0 = MT == 1 ? (((ts >> 2) ^ (k & 1)) * BPT + (ts & 3)) : ts;
        const int n_blk = (pc.lt1 - pc.lt0) * BPT;
        // Scales are fetched a block ahead, and the page they lie in a block before that.  Where a
        // block lies: its first token's page (entry of the block table) and row in it.
        struct Place {
            int lp, row, page;
        };
        auto page_at = [&](Place &a) {
            a.page = p.block_table == nullptr ? pc.b
                     : a.lp < p.max_pages ? __ldg(p.block_table + (size_t)pc.b * p.max_pages + a.lp) : -1;
        };
        auto place_next = [&](Place a) -> Place {
            a.row += NTS * BLK;
            while (p.max_pages > 1 && a.row >= p.page_size) {    // (one page: a tile past its end is shifted back)
                a.row -= p.page_size;
                ++a.lp;
            }
            page_at(a);
            return a;
        };
        // scales of this lane's token of a block (1 past the sequence and outside the pool)
        auto load_scales = [&](int blk, const Place &a) -> float2 {
            const int tok0 = start + (pc.lt0 + blk / BPT) * TILE;
            const int back = max(tok0 + TILE - len, 0);          // (a unit's last tile is shifted back to end at len)
            const int in = (blk % BPT) * BLK + lane - back;      // token, from the tile's first
            if (blk >= n_blk || in < 0 || a.page < 0 || a.page >= p.pages) return make_float2(1.f, 1.f);
            const size_t at = ((size_t)a.page * p.n_kv + j) * p.page_size + (a.row + lane - back);
            return make_float2(__ldg(p.k_rows + at), __ldg(p.v_rows + at));
        };
        // (the page, then the query, then the scales, which wait for the page)
        Place here;
        {
            const int t = start + pc.lt0 * TILE + blk0 * BLK;
            here.lp = p.max_pages > 1 ? t / p.page_size : 0;
            here.row = t - here.lp * p.page_size;
            page_at(here);
        }
        // ---- the two query rows of this thread as A operands: word (kk, 0/2) of row gid holds
        //      dimensions 16 kk + 4 c .. + 3, the order in which ldmatrix hands out the key codes
        uint2 raw[NH][D / 16];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            const uint2 *q = reinterpret_cast<const uint2 *>(
                p.q + (((size_t)pc.b * p.q_len + row_qi[h]) * p.n_q + (size_t)j * p.g + row_hg[h]) * D);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) raw[h][kk] = row_on[h] ? __ldg(q + kk * 4 + c) : make_uint2(0u, 0u);
        }
        float2 next = load_scales(blk0, here);
        here = place_next(here);
        uint32_t qa[D / 16][4];
        float cs[2];                               // score scale of each row (log2 units)
        int lo[2], hi[2];                          // positions each row sees: [lo, hi)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h >= NH) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) qa[kk][1] = qa[kk][3] = 0u;
                break;
            }
            float amax = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                amax = fmaxf(amax, fmaxf(fmaxf(fabsf(bf16_lo(raw[h][kk].x)), fabsf(bf16_hi(raw[h][kk].x))),
                                         fmaxf(fabsf(bf16_lo(raw[h][kk].y)), fabsf(bf16_hi(raw[h][kk].y)))));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            int e = 0;
            if (amax > 0.f && amax <= 3.4e38f) {
                int x;
                frexpf(amax, &x);                  // amax in [2^(x-1), 2^x)
                e = min(max(14 - x, -126), 126);
            }
            const float up = __int_as_float((127 + e) << 23);
            cs[h] = p.scale_log2 * __int_as_float((127 - e) << 23);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qa[kk][h] = pack_f16x2(bf16_lo(raw[h][kk].x) * up, bf16_hi(raw[h][kk].x) * up);
                qa[kk][2 + h] = pack_f16x2(bf16_lo(raw[h][kk].y) * up, bf16_hi(raw[h][kk].y) * up);
            }
            hi[h] = len - p.q_len + row_qi[h] + 1;
            lo[h] = p.window > 0 ? window_start(hi[h], p.window) : 0;
        }
        // no mask for tiles of positions that every row sees
        const int free_lo = p.window > 0 ? len - p.window : 0, free_hi = len - p.q_len + 1;

        float o[D / 8][4];
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        bool aborted = false;

        int held = -1;                             // tile of the piece this warp holds
        for (int blk = blk0; blk < n_blk; blk += NTS) {
            __syncwarp();
            s_ks[lane] = next.x;
            s_vs[lane] = next.y;
            // (the maximum only picks a common factor: a zero scale must not make it -inf)
            s_lv[lane] = __log2f(fmaxf(next.y, 8.67361738e-19f));
            __syncwarp();
            next = load_scales(blk + NTS, here);
            here = place_next(here);
            const int it = blk / BPT, s = (k + it) % NST;
            if (it != held) {
                if (!warp_all(mbar_wait(&bars->full[s], (uint32_t)((k + it) / NST) & 1u, FLAG_FULL_WAIT, abort_flag))) {
                    aborted = true;
                    break;
                }
                held = it;
            }
            const int tok0 = start + (pc.lt0 + it) * TILE, y = min(tok0, len - TILE);
            const int r0 = (blk % BPT) * BLK;      // the block's first row of the tile
            // ldmatrix rows of this lane: a row's 16-byte chunk ch lies at (ch ^ (row & 7)), and blocks
            // start at multiples of 8 rows.  Keys: eight tokens x four chunks; values: sixteen x two.
            const uint32_t base = smem_u32(smem + s * STAGE) + r0 * 128;
            const uint32_t kb = base + (lane & 7) * 128 + (((lane >> 3) ^ (lane & 7)) << 4);
            const uint32_t vb = base + KV_BYTES + (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);

            // ---- S = Q K^T: 16 rows x 32 tokens
            float sc[4][4];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    uint32_t w[4];
                    ldmatrix_x4((kb ^ (half * 64)) + nt * 1024, w[0], w[1], w[2], w[3]);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t b0, b1;
                        e4m3x4(w[x], b0, b1);
                        mma_f16(sc[nt], qa[half * 4 + x], b0, b1);
                    }
                }
            }
            // ---- scales, mask, running maximum of s + log2(vs)
            const bool masked = y < tok0 || tok0 + TILE > free_hi || tok0 < free_lo;
            uint32_t vis = 0xFFFFu;                // seen: bit 4 nt + e (element e of n-tile nt)
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const float2 ks = *reinterpret_cast<const float2 *>(s_ks + nt * 8 + 2 * c);
                const float2 lv = *reinterpret_cast<const float2 *>(s_lv + nt * 8 + 2 * c);
#pragma unroll
                for (int e = 0; e < 2 * NH; ++e) {
                    const int h = e >> 1;
                    float x = sc[nt][e] * (cs[h] * (e & 1 ? ks.y : ks.x));
                    if (masked) {
                        const int at = y + r0 + nt * 8 + 2 * c + (e & 1);
                        if (!(at >= tok0 && at >= lo[h] && at < hi[h])) {
                            x = -INFINITY;
                            if (MULTI) vis &= ~(1u << (4 * nt + e));
                        }
                    }
                    sc[nt][e] = x;
                    mx[h] = fmaxf(mx[h], x + (e & 1 ? lv.y : lv.x));
                }
            }
            bool move = false;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                move |= mx[h] > m[h] + RESCALE || (m[h] == -INFINITY && mx[h] > m[h]);
            }
            if (__any_sync(0xffffffffu, move)) {
                float a[2] = {1.f, 1.f};
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float mn = fmaxf(m[h], mx[h]);
                    a[h] = m[h] == -INFINITY ? 0.f : fast_exp2(m[h] - mn);
                    m[h] = mn;
                    l[h] *= a[h];
                }
#pragma unroll
                for (int nt = 0; nt < D / 8; ++nt) {
                    o[nt][0] *= a[0]; o[nt][1] *= a[0];
                    if (NH > 1) { o[nt][2] *= a[1]; o[nt][3] *= a[1]; }
                }
            }
            // ---- weights: f16 A operands of two steps of 16 tokens
            const float off[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
            uint32_t pa[2][4] = {};
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const float2 vs = *reinterpret_cast<const float2 *>(s_vs + nt * 8 + 2 * c);
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float a = fast_exp2(sc[nt][2 * h] - off[h]), b = fast_exp2(sc[nt][2 * h + 1] - off[h]);
                    l[h] += a + b;
                    pa[nt >> 1][2 * (nt & 1) + h] = pack_f16x2(a * vs.x, b * vs.y);
                }
            }
            // ---- a token that a row must not see takes no part in it, whatever its scale and codes are: a
            //      weight of zero would still make NaN of them.  So the weights are cleared, and where the
            //      block has NaN codes the product is taken of a copy without them and the elements they belong
            //      to are found one by one.  (Without MULTI only a unit's last tile has such tokens, and the row
            //      sees them in the tile before.)
            uint32_t vp = vb;
            bool nan_codes = false;
            if (MULTI && masked) {
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        const uint32_t b = vis >> (4 * nt + 2 * h);
                        pa[nt >> 1][2 * (nt & 1) + h] &= (b & 1 ? 0x0000FFFFu : 0u) | (b & 2 ? 0xFFFF0000u : 0u);
                    }
                const uint4 *src = reinterpret_cast<const uint4 *>(smem + s * STAGE + KV_BYTES + r0 * 128);
                uint32_t any = 0;
#pragma unroll
                for (int i = lane; i < BLK * 8; i += 32) {
                    const uint4 w = src[i];
                    any |= nan_bytes(w.x) | nan_bytes(w.y) | nan_bytes(w.z) | nan_bytes(w.w);
                }
                nan_codes = __any_sync(0xffffffffu, any != 0);
                if (nan_codes) {
                    // (the warp's part of the join is free until the piece's end)
                    uint4 *copy = reinterpret_cast<uint4 *>(my_merge);
                    auto clean = [](uint32_t w) { return w & ~((nan_bytes(w) >> 7) * 0xFFu); };
#pragma unroll 1
                    for (int i = lane; i < BLK * 8; i += 32) {
                        const uint4 w = src[i];
                        copy[i] = make_uint4(clean(w.x), clean(w.y), clean(w.z), clean(w.w));
                    }
                    __syncwarp();
                    vp = smem_u32(my_merge) + (vb - (base + KV_BYTES));
                }
            }
            // ---- O += P V: the transposed load hands out pairs of dimensions (2p, 2p + 1) of two
            //      tokens; the even and the odd dimensions of a 16-byte chunk make an n-tile each
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
                for (int ch = 0; ch < D / 16; ch += 2) {
                    uint32_t w[4];
                    ldmatrix_x4_trans((vp ^ (ch * 16)) + st * 2048, w[0], w[1], w[2], w[3]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t b0, b1;
                        e4m3x4(__byte_perm(w[2 * x], w[2 * x + 1], 0x6420), b0, b1);
                        mma_f16(o[2 * (ch + x)], pa[st], b0, b1);
                        e4m3x4(__byte_perm(w[2 * x], w[2 * x + 1], 0x7531), b0, b1);
                        mma_f16(o[2 * (ch + x) + 1], pa[st], b0, b1);
                    }
                }
            if (MULTI && nan_codes) {
                // bit 4 ch + i of a row: a token that it sees has NaN at dimension 16 ch + 4 c + i
                uint32_t bad[2] = {0u, 0u};
#pragma unroll 1
                for (int t = 0; t < BLK; ++t) {
                    // (token 8 nt + 2 c' + i lies with lane c' of the row's four)
                    const uint32_t of = __shfl_sync(0xffffffffu, vis, (lane & 28) | ((t >> 1) & 3));
                    const uint8_t *row = smem + s * STAGE + KV_BYTES + (r0 + t) * 128 + 4 * c;
                    uint32_t found = 0u;
#pragma unroll 1
                    for (int ch = 0; ch < D / 16; ++ch) {
                        const uint32_t n = nan_bytes(*reinterpret_cast<const uint32_t *>(row + ((ch ^ (t & 7)) << 4)));
                        found |= ((n >> 7 & 1u) | (n >> 14 & 2u) | (n >> 21 & 4u) | (n >> 28 & 8u)) << (4 * ch);
                    }
#pragma unroll
                    for (int h = 0; h < NH; ++h)
                        if (of >> (4 * (t >> 3) + 2 * h + (t & 1)) & 1u) bad[h] |= found;
                }
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int ch = 0; ch < D / 16; ++ch)
#pragma unroll
                        for (int i = 0; i < 4; ++i)     // (the even dimensions' n-tile, then the odd ones')
                            if (bad[h] >> (4 * ch + i) & 1u) o[2 * ch + (i & 1)][2 * h + (i >> 1)] = NAN;
                __syncwarp();                           // (the copy is read)
            }
            if (blk + NTS >= n_blk || (blk + NTS) / BPT != it) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->empty[s]);
            }
        }
        if (aborted) return;
        k += pc.lt1 - pc.lt0;

        // ---- join the warps of each m-tile and write the piece's result; the next piece's query and
        //      page entry are fetched into L2 meanwhile
        const Piece done = pc;
        more = next_piece();
        if (more) {
            for (int r = ctid; r < 2 * R; r += NCW * 32)
                prefetch_l2(p.q + (((size_t)pc.b * p.q_len + (r >> 1) / p.g) * p.n_q + (size_t)pc.i * p.g + (r >> 1) % p.g) * D +
                            (r & 1) * 64);
            if (ctid == 0 && p.block_table != nullptr) prefetch_l2(p.block_table + (size_t)pc.b * p.max_pages);
        }
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
#pragma unroll
            for (int ch = 0; ch < D / 16; ++ch)    // dimensions 16 ch + 4 c .. + 3
                *reinterpret_cast<float4 *>(my_merge + (gid + 8 * h) * MPAD + 16 * ch + 4 * c) =
                    make_float4(o[2 * ch][2 * h], o[2 * ch + 1][2 * h], o[2 * ch][2 * h + 1], o[2 * ch + 1][2 * h + 1]);
            if (c == 0) {
                my_merge[16 * MPAD + gid + 8 * h] = m[h];
                my_merge[16 * MPAD + 16 + gid + 8 * h] = l[h];
            }
        }
        if (!consumer_sync()) return;
        if (ctid < ROWS) {
            const int rmt = ctid >> 4, rrow = ctid & 15;
            float M = -INFINITY, L = 0.f, w[NTS];
#pragma unroll
            for (int t = 0; t < NTS; ++t) M = fmaxf(M, merge[(t * MT + rmt) * MERGE_FLOATS + 16 * MPAD + rrow]);
            const float Mu = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int t = 0; t < NTS; ++t) {
                const float *mb = merge + (t * MT + rmt) * MERGE_FLOATS + 16 * MPAD;
                w[t] = fast_exp2(mb[rrow] - Mu);
                L += mb[16 + rrow] * w[t];
            }
            // (a NaN sum stays NaN)
            const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
            for (int t = 0; t < NTS; ++t) wts[ctid * NTS + t] = w[t] * inv;
            wts[ROWS * NTS + ctid] = L == 0.f ? -INFINITY : (Mu + __log2f(L)) * 0.69314718055994531f;
        }
        if (!consumer_sync()) return;
        const size_t part = ((size_t)blockIdx.x * 2 + done.slot) * ROWS;
        for (int i = ctid; i < ROWS * (D / 4); i += NCW * 32) {
            const int r = i / (D / 4), col = (i % (D / 4)) * 4;
            if (r >= R) break;
            const int rmt = r >> 4, rrow = r & 15;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int t = 0; t < NTS; ++t) {
                const float w = wts[r * NTS + t];
                const float4 x = *reinterpret_cast<const float4 *>(merge + (t * MT + rmt) * MERGE_FLOATS + rrow * MPAD + col);
                // (a warp that saw nothing of this row has zeros; a NaN stays under a weight that ran out of range)
                v.x += w * x.x; v.y += w * x.y; v.z += w * x.z; v.w += w * x.w;
            }
            if (done.whole) {
                const int qi = r / p.g;
                const size_t gh = ((size_t)done.b * p.q_len + qi) * p.n_q + (size_t)j * p.g + (r - qi * p.g);
                *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(p.out) + gh * D + col) =
                    make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                if (col == 0) p.lse[gh] = wts[ROWS * NTS + r];
            } else {
                *reinterpret_cast<float4 *>(p.ws_o + (part + r) * D + col) = v;
                if (col == 0) p.ws_lse[part + r] = wts[ROWS * NTS + r];
            }
        }
        if (!consumer_sync()) return;
    }
}

}  // namespace kvattn
