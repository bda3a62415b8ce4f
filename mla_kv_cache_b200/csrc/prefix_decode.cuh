// prefix_decode.cuh -- decode attention for a batch whose sequences share a prefix, on the
// sm_100a tensor cores.
//
// Every new token of the batch attends to the same P prefix tokens and then to its own
// sequence's cached suffix.  With s the scaled scores,
//     out = softmax([s_prefix, s_suffix]) [V_prefix; V_suffix]
// is the log-sum-exp merge of attention over the prefix and over the suffix, and over any
// parts of the two.  A decode per sequence would read the prefix once per sequence; here the
// prefix is read once for a block of query rows taken from all sequences:
//     rows of KV head j = the g = n_q / n_kv heads of the group at every new token of every
//     sequence (B * L * g rows),  S = Q K^T,  O += P V
// is then a matrix product with 128-row tiles, bound by the tensor cores (and the exponentials)
// instead of by memory.  The suffixes, read once each, run through the same pipeline with
// one sequence's L * g rows in the tile.
//
// Work.  A unit is (KV head, pair of 128-row tiles) over the prefix, or (sequence, KV head)
// over a suffix; each unit is a run of 128-token K/V tiles.  All units are laid end to end --
// a prefix tile that serves two row tiles counts twice -- and worker w (one CTA per SM) takes
// an equal contiguous range of that line, computed on the device from prefix_len and seq_lens
// (so a captured call may be replayed with other lengths).  Prefix and suffix work thus run side by
// side: some SMs keep the tensor cores busy while others stream suffixes from memory.  Every
// piece (a worker's part of a unit) leaves a normalised partial and its log-sum-exp in the
// caller's workspace; prefix_merge_kernel joins a row's partials.
//
// Pipeline of a CTA (384 threads):
//   warp 0       producer: TMA loads (128-byte swizzle, no multicast) of Q tiles and of K and
//                V tiles into a ring.
//   warp 1       one thread issues every tcgen05.mma: S_x = Q K^T (A, B from shared memory) and
//                O_x += P_x V (P_x read from tensor memory, V tile MN-major).
//   warps 4..11  two softmax groups x = 0, 1 of 128 threads, one thread per row: a row's 128
//                scores are one TMEM lane, so its maximum and sum need no exchange.  P_x
//                (bf16) overwrites the first half of S_x.
// Steps alternate between the groups, so that one group's exponentials run while the tensor
// cores work for the other: in a two-row-tile unit the groups hold the two row tiles and
// each K/V tile makes two steps; in a one-row-tile unit both groups hold the same rows and take
// alternate K/V tiles, each with its own (max, sum, O), which the merge joins.
// The running maximum moves lazily: only when a row's tile maximum exceeds it by 2^8 are that
// row's O and sum rescaled.
// Weights enter the value product rounded to bf16 (half a step, 2^-9 relative, each independent
// of the others; the output is rounded to bf16 itself); sums, maxima and O are fp32.
#pragma once
#include "common.cuh"
#include "schedule.cuh"
#include "tc05.cuh"

namespace kvattn {

struct PrefixParams {
    const int32_t *prefix_len;     // [1]
    const int32_t *seq_lens;       // [B]
    const int32_t *prefix_table;   // [prefix_pages_max] or null: one page
    const int32_t *block_table;    // [B, max_pages] or null: one page a sequence
    __nv_bfloat16 *out;            // [B, L, n_q, D]
    float *lse;                    // [B, L, n_q]
    long long *meta;               // [0] tiles of the prefix, [1] W; then int suffix tile prefix [B + 1]
    float *lse_p, *o_p;            // prefix partials [units_p + workers][2][128] (x D)
    float *lse_s, *o_s;            // suffix partials [B * n_kv + workers][2][L * g] (x D)
    int B, L, n_q, n_kv, g;
    int P_max, T_max;              // capacities (lengths are clamped to them)
    int prefix_page, page_size;    // rows per page of the prefix's and the suffixes' cache
    int max_pages;                 // block_table columns
    int tok_tile;                  // new tokens in a row tile: floor(128 / g)
    int row_tiles, pairs;          // ceil(B L / tok_tile), ceil(row_tiles / 2)
    int workers;
    int prefix_in_ws;              // the suffix tile prefix was written to the workspace before
    float scale_log2;              // scale * log2(e)
};

namespace pfx {

constexpr int TILE = 128;
constexpr int ROWS = 128;
constexpr int NTHREADS = 384;
// registers of a thread after the split between the first warpgroup (producer, issuer) and the
// softmax warpgroups: a row's 128 scores and its packed weights stay in registers
constexpr int REGS_CTRL = 80, REGS_SOFT = 208;
static_assert(128 * REGS_CTRL + 256 * REGS_SOFT <= NTHREADS * 168, "registers of the launch");
constexpr int CHUNK = 128 * 128;          // [128 rows x 128 bytes]
constexpr int NS_MAX = 10;
constexpr int MIN_TILES = 2;              // a worker takes at least two tiles
constexpr float RESCALE = 8.f;

template <int D>
struct Cfg {
    static constexpr int NCH = D / 64;                  // 64-wide chunks of a row
    static constexpr int KV_BYTES = NCH * CHUNK;        // a K or V tile
    static constexpr int Q_BYTES = NCH * CHUNK;         // a Q tile
    static constexpr int NS = (160 * 1024) / KV_BYTES;  // ring slots (K and V tiles alternate)
    static constexpr int OFF_Q = NS * KV_BYTES;
    static constexpr int OFF_BARS = OFF_Q + 2 * Q_BYTES;
    static constexpr int OFF_PREFIX = OFF_BARS + 512;
    // the suffix tile prefix lies in shared memory up to this batch, in the workspace beyond
    static constexpr int B_SMEM = 320;
    static constexpr int SMEM = 1024 + OFF_PREFIX + (B_SMEM + 1) * 4;
    static_assert(SMEM <= 232448, "shared memory of an SM");
    static_assert(NS <= NS_MAX, "ring barriers");
};

// tensor memory columns of group x: scores (and weights) at 128 x, output at 256 + 128 x
constexpr uint32_t TM_S = 0, TM_O = 256, TM_X = 128;

struct Bars {
    uint64_t full[NS_MAX], empty[NS_MAX];
    uint64_t qfull[2], qempty[2];
    uint64_t sready[2];      // scores of group x's next step are in TMEM (and its last value product is done)
    uint64_t pready[2];      // group x has written its weights (and rescaled O_x)
    uint64_t odone[2];       // group x's last value product of a piece is done
    uint64_t ofree[2];       // group x has read O_x
    uint32_t tmem;
    int abort_flag;
};
static_assert(sizeof(Bars) <= 512, "barrier block overflows its slot");

// The line of work, the same on every CTA and in the merge kernel.
struct Line {
    int n_p;                 // prefix tiles
    int wp;                  // line positions per prefix tile: 2 when row tiles pair up, else 1
    long long units_p;
    long long p_total;       // positions of the prefix units
    long long total, W;
};
__device__ __forceinline__ Line make_line(const PrefixParams &p, int suffix_tiles) {
    Line l;
    l.n_p = tiles_of(clamp_len(__ldg(p.prefix_len), p.P_max), TILE);
    l.wp = p.row_tiles > 1 ? 2 : 1;
    l.units_p = (long long)p.n_kv * p.pairs;
    l.p_total = l.units_p * l.n_p * l.wp;
    l.total = l.p_total + (long long)suffix_tiles * p.n_kv;
    l.W = (l.total + p.workers - 1) / p.workers;
    if (l.W < MIN_TILES) l.W = MIN_TILES;
    l.W = (l.W + 1) & ~1ll;              // (no boundary inside a prefix tile)
    return l;
}

struct Piece {
    bool prefix;
    bool two;            // two row tiles: each K/V tile makes two steps
    int j;               // KV head
    int b;               // sequence (suffix)
    int pair;            // row tile pair (prefix)
    int len;             // tokens of the unit
    int lt0, lt1;        // its tiles
    int steps;
    long long slot;      // partial
};

// The piece of worker w that starts at line position pos; pos moves to its end.
__device__ __forceinline__ Piece next_piece(const PrefixParams &p, const Line &l, const int *s_prefix, long long &pos,
                                            long long end, int w) {
    Piece c;
    if (pos < l.p_total) {
        const long long ul = (long long)l.n_p * l.wp;
        const long long u = pos / ul;
        const long long u0 = u * ul;
        const long long stop = end < u0 + ul ? end : u0 + ul;
        c.prefix = true;
        c.j = (int)(u / p.pairs);
        c.pair = (int)(u % p.pairs);
        c.two = 2 * c.pair + 1 < p.row_tiles;
        c.b = 0;
        c.len = clamp_len(__ldg(p.prefix_len), p.P_max);
        c.lt0 = (int)((pos - u0) / l.wp);
        c.lt1 = (int)((stop - u0) / l.wp);
        c.slot = u + w;
        pos = stop;
    } else {
        const long long sp = pos - l.p_total;
        c.prefix = false;
        c.two = false;
        c.b = find_seq(s_prefix, p.B, p.n_kv, sp);
        const int nt = s_prefix[c.b + 1] - s_prefix[c.b];
        const long long base = (long long)s_prefix[c.b] * p.n_kv;
        c.j = (int)((sp - base) / nt);
        c.pair = 0;
        const long long u0 = l.p_total + base + (long long)c.j * nt;
        const long long stop = end < u0 + nt ? end : u0 + nt;
        c.len = clamp_len(__ldg(p.seq_lens + c.b), p.T_max);
        c.lt0 = (int)(pos - u0);
        c.lt1 = (int)(stop - u0);
        c.slot = (long long)c.b * p.n_kv + c.j + w;
        pos = stop;
    }
    c.steps = (c.lt1 - c.lt0) * (c.two ? 2 : 1);
    return c;
}

struct Ctx {
    uint8_t *smem;
    Bars *bars;
    volatile int *abort_flag;
    const int *s_prefix;
    Line line;
    long long p0, p1;
    int w;
};

// ------------------------------------------------------------------ producer (warp 0, lane 0)
template <int D>
__device__ __forceinline__ void producer(const PrefixParams &p, const CUtensorMap *kp, const CUtensorMap *vp,
                                         const CUtensorMap *ks, const CUtensorMap *vs, const CUtensorMap *qm,
                                         const Ctx &c) {
    using C = Cfg<D>;
    Bars *bars = c.bars;
    const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_normal();
    uint32_t quse[2] = {0, 0};
    int qs = 0;
    uint32_t n = 0;                 // tiles (K and V) issued
    bool ok = true;
    for (long long pos = c.p0; pos < c.p1 && ok;) {
        const Piece pc = next_piece(p, c.line, c.s_prefix, pos, c.p1, c.w);
        const int nq = pc.two ? 2 : 1;
        for (int r = 0; r < nq && ok; ++r) {
            const int s = (qs + r) & 1;
            if (quse[s] > 0 && !mbar_wait(&bars->qempty[s], (quse[s] - 1) & 1u, FLAG_EMPTY_WAIT, c.abort_flag)) {
                ok = false;
                break;
            }
            const int tok = pc.prefix ? (2 * pc.pair + r) * p.tok_tile : pc.b * p.L;
            mbar_arrive_expect_tx(&bars->qfull[s], (uint32_t)(C::NCH * p.tok_tile * p.g * 128));
#pragma unroll
            for (int ch = 0; ch < C::NCH; ++ch)
                tma_load_4d(c.smem + C::OFF_Q + s * C::Q_BYTES + ch * CHUNK, qm, &bars->qfull[s], 64 * ch, 0, pc.j, tok,
                            keep);
            ++quse[s];
        }
        if (!pc.two) qs ^= 1;
        // (the prefix is read again by the CTAs that serve its other row tiles)
        const CUtensorMap *km = pc.prefix ? kp : ks, *vm = pc.prefix ? vp : vs;
        const uint64_t pol = pc.prefix ? keep : once;
        for (int lt = pc.lt0; lt < pc.lt1 && ok; ++lt) {
            const TileSrc src = pc.prefix ? tile_source(p.prefix_table, 0, p.prefix_page, 0, lt, TILE, pc.len)
                                          : tile_source(p.block_table, p.max_pages, p.page_size, pc.b, lt, TILE, pc.len);
            const int z = src.page * p.n_kv + pc.j;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++n) {
                const uint32_t s = n % C::NS;
                if (!mbar_wait(&bars->empty[s], ((n / C::NS) & 1u) ^ 1u, FLAG_EMPTY_WAIT, c.abort_flag)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&bars->full[s], C::KV_BYTES);
#pragma unroll
                for (int ch = 0; ch < C::NCH; ++ch)
                    tma_load_3d(c.smem + s * C::KV_BYTES + ch * CHUNK, kv ? vm : km, &bars->full[s], 64 * ch, src.y, z,
                                pol);
            }
        }
    }
    if (!ok) {
        // Let every copy already issued land before the CTA can exit.
        for (uint32_t m = n > C::NS ? n - C::NS : 0; m < n; ++m)
            mbar_wait_sleep(&bars->full[m % C::NS], (m / C::NS) & 1u, FLAG_FULL_WAIT, nullptr);
        for (int s = 0; s < 2; ++s)
            if (quse[s] > 0) mbar_wait_sleep(&bars->qfull[s], (quse[s] - 1) & 1u, FLAG_FULL_WAIT, nullptr);
    }
}

// ------------------------------------------------------------------ MMA issuer (warp 1, lane 0)
// A walk over the CTA's steps.
struct Walk {
    Piece pc;
    long long pos;
    int i;               // step within the piece
    uint32_t tile;       // K/V tiles of the pieces before
    int qs;              // Q slot of the piece's first row tile
    uint32_t quse[2];    // pieces' uses of a Q slot, this one included
    bool done;
};
__device__ __forceinline__ void walk_piece(Walk &k, const PrefixParams &p, const Ctx &c) {
    if (k.pos >= c.p1) {
        k.done = true;
        return;
    }
    k.pc = next_piece(p, c.line, c.s_prefix, k.pos, c.p1, c.w);
    k.i = 0;
    ++k.quse[k.qs];
    if (k.pc.two) ++k.quse[k.qs ^ 1];
}
__device__ __forceinline__ Walk walk_start(const PrefixParams &p, const Ctx &c) {
    Walk k;
    k.pos = c.p0;
    k.tile = 0;
    k.qs = 0;
    k.quse[0] = k.quse[1] = 0;
    k.done = false;
    walk_piece(k, p, c);
    return k;
}
__device__ __forceinline__ void walk_step(Walk &k, const PrefixParams &p, const Ctx &c) {
    if (++k.i < k.pc.steps) return;
    k.tile += k.pc.lt1 - k.pc.lt0;
    if (!k.pc.two) k.qs ^= 1;
    walk_piece(k, p, c);
}

template <int D>
__device__ __forceinline__ void mma_issuer(const PrefixParams &p, const Ctx &c) {
    using C = Cfg<D>;
    Bars *bars = c.bars;
    const uint32_t tmem = bars->tmem;
    const uint32_t smem = smem_u32(c.smem);
    constexpr uint32_t idesc_qk = idesc_f16_major(128, TILE, 1, 1, 0, 0);
    constexpr uint32_t idesc_pv = idesc_f16_major(128, D, 1, 1, 0, 1);
    uint32_t kseen = 0, vseen = 0;      // K / V tiles waited for

    auto scores = [&](Walk &k, int x) -> bool {
        const uint32_t t = k.tile + (uint32_t)(k.pc.two ? k.i >> 1 : k.i);
        const uint32_t nk = 2 * t;
        const int r = k.pc.two ? k.i & 1 : 0;
        const int s = (k.qs + r) & 1;
        if (!mbar_wait(&bars->qfull[s], (k.quse[s] - 1) & 1u, FLAG_FULL_WAIT, c.abort_flag)) return false;
        if (kseen == t) {
            if (!mbar_wait(&bars->full[nk % C::NS], (nk / C::NS) & 1u, FLAG_FULL_WAIT, c.abort_flag)) return false;
            ++kseen;
        }
        tc_fence_after();
        const uint32_t q = smem + C::OFF_Q + s * C::Q_BYTES, kt = smem + (nk % C::NS) * C::KV_BYTES;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * CHUNK + (kk & 3) * 32;
            umma_ss(tmem + TM_S + TM_X * x, smem_desc_sw128(q + off, 16, 1024), smem_desc_sw128(kt + off, 16, 1024),
                    idesc_qk, kk ? 1u : 0u);
        }
        umma_commit(&bars->sready[x]);
        if (!k.pc.two || (k.i & 1)) umma_commit(&bars->empty[nk % C::NS]);
        if (k.pc.two ? k.i >= k.pc.steps - 2 : k.i == k.pc.steps - 1) umma_commit(&bars->qempty[s]);
        return true;
    };

    Walk qk = walk_start(p, c), pv = qk;
    uint32_t steps_x[2] = {0, 0};     // value products issued per group
    uint32_t pieces_x[2] = {0, 0};    // pieces group x has taken part in
    int xq = 0, xp = 0;
    for (int i = 0; i < 2 && !qk.done; ++i, xq ^= 1) {
        if (!scores(qk, xq)) return;
        walk_step(qk, p, c);
    }
    while (!pv.done) {
        const int x = xp;
        const uint32_t t = pv.tile + (uint32_t)(pv.pc.two ? pv.i >> 1 : pv.i);
        const uint32_t nv = 2 * t + 1;
        const bool first = pv.i < 2, last = pv.i >= pv.pc.steps - 2;
        if (!mbar_wait(&bars->pready[x], steps_x[x] & 1u, FLAG_FULL_WAIT, c.abort_flag)) return;
        if (vseen == t) {
            if (!mbar_wait(&bars->full[nv % C::NS], (nv / C::NS) & 1u, FLAG_FULL_WAIT, c.abort_flag)) return;
            ++vseen;
        }
        if (first && pieces_x[x] > 0 &&
            !mbar_wait(&bars->ofree[x], (pieces_x[x] - 1) & 1u, FLAG_FULL_WAIT, c.abort_flag))
            return;
        tc_fence_after();
        const uint32_t vt = smem + (nv % C::NS) * C::KV_BYTES;
#pragma unroll
        for (int kk = 0; kk < TILE / 16; ++kk)
            umma_ts(tmem + TM_O + TM_X * x, tmem + TM_S + TM_X * x + kk * 8,
                    smem_desc_sw128(vt + kk * 2048, CHUNK, 1024), idesc_pv, (!first || kk) ? 1u : 0u);
        if (!pv.pc.two || (pv.i & 1)) umma_commit(&bars->empty[nv % C::NS]);
        if (last) {
            umma_commit(&bars->odone[x]);
            ++pieces_x[x];
        }
        ++steps_x[x];
        xp ^= 1;
        walk_step(pv, p, c);
        if (!qk.done) {
            if (!scores(qk, xq)) return;
            xq ^= 1;
            walk_step(qk, p, c);
        }
    }
}

// ------------------------------------------------------------------ softmax (warps 4..11)
template <int D>
__device__ __forceinline__ void softmax_group(const PrefixParams &p, const Ctx &c, int warp, int lane) {
    Bars *bars = c.bars;
    const uint32_t tmem = bars->tmem;
    const int x = (warp - 4) >> 2;
    const int quad = warp & 3;
    const int r = 32 * quad + lane;                   // row of the tile
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const uint32_t ts = tmem + lanes + TM_S + TM_X * x, to = tmem + lanes + TM_O + TM_X * x;
    const bool negate = p.scale_log2 < 0.f;           // (the maximum is taken of the unscaled scores)
    const float cs = fmaxf(fabsf(p.scale_log2), 1e-30f);   // (a zero scale: masked scores stay -inf)
    uint32_t n_x = 0, pieces = 0;                     // steps and pieces of this group
    uint32_t i0 = 0;                                  // steps of the pieces before
    for (long long pos = c.p0; pos < c.p1;) {
        const Piece pc = next_piece(p, c.line, c.s_prefix, pos, c.p1, c.w);
        const int first = (int)((i0 & 1u) ^ (uint32_t)x);      // this group's first step of the piece
        i0 += (uint32_t)pc.steps;
        const int part = first;                       // row tile (two) or share of the K/V tiles
        // rows of the tile that are real
        int rows = p.L * p.g;
        if (pc.prefix) {
            const int tok0 = (2 * pc.pair + (pc.two ? part : 0)) * p.tok_tile;
            rows = min(p.tok_tile, p.B * p.L - tok0) * p.g;
        }
        const bool warp_on = 32 * quad < rows;
        // positions this row sees: all of the prefix; a suffix up to its own token
        const int limit = pc.prefix ? pc.len : pc.len - p.L + 1 + min(r / p.g, p.L - 1);
        float m = -INFINITY, l = 0.f;                 // (log2 units; m in scaled scores)
        for (int i = first; i < pc.steps; i += 2, ++n_x) {
            const int lt = pc.lt0 + (pc.two ? i >> 1 : i);
            if (!warp_all(mbar_wait(&bars->sready[x], n_x & 1u, FLAG_MMA_WAIT, c.abort_flag))) return;
            if (warp_on) {
                tc_fence_after();
                float s[TILE];
#pragma unroll
                for (int h = 0; h < 4; ++h) tmem_ld32(ts + 32 * h, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * h));
                tmem_wait_ld();
                if (negate) {
#pragma unroll
                    for (int e = 0; e < TILE; ++e) s[e] = -s[e];
                }
                // the tile's first position (a unit's last tile ends at its length: its first
                // columns repeat earlier positions, or lie before the cache)
                const int tok0 = lt * TILE;
                const int y = min(tok0, pc.len - TILE);
                const bool masked = y < tok0 || (!pc.prefix && tok0 + TILE > pc.len - p.L + 1);
                if (masked) {
                    const int lo = tok0 - y, hi = limit - y;
#pragma unroll
                    for (int e = 0; e < TILE; ++e) s[e] = (e >= lo && e < hi) ? s[e] : -INFINITY;
                }
                float t0 = s[0], t1 = s[1], t2 = s[2], t3 = s[3];
#pragma unroll
                for (int e = 4; e < TILE; e += 4) {
                    t0 = fmaxf(t0, s[e]);
                    t1 = fmaxf(t1, s[e + 1]);
                    t2 = fmaxf(t2, s[e + 2]);
                    t3 = fmaxf(t3, s[e + 3]);
                }
                const float tm = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * cs;
                const bool move = tm > m + RESCALE || (m == -INFINITY && tm > m);
                const float m_new = move ? tm : m;
                if (__any_sync(0xffffffffu, move && m != -INFINITY)) {
                    // O_x up to the last step is complete (its product precedes these scores)
                    const float a = m == -INFINITY ? 1.f : fast_exp2(m - m_new);
                    l *= a;
#pragma unroll 1
                    for (int h = 0; h < D; h += 32) {
                        uint32_t o[32];
                        tmem_ld32(to + h, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                        tmem_st32(to + h, o);
                    }
                    tmem_wait_st();
                }
                m = m_new;
                const float off = m == -INFINITY ? 0.f : -m;
                float l0 = 0.f, l1 = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float a = fast_exp2(fmaf(s[64 * h + 2 * e], cs, off));
                        const float b = fast_exp2(fmaf(s[64 * h + 2 * e + 1], cs, off));
                        l0 += a;
                        l1 += b;
                        w[e] = pack_bf16x2(a, b);
                    }
                    tmem_st32(ts + 32 * h, w);
                }
                l += l0 + l1;
                tmem_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->pready[x]);
        }
        // ---- the piece's partial: O / l and log2 of the sum
        if (first < pc.steps) {
            if (!warp_all(mbar_wait(&bars->odone[x], pieces & 1u, FLAG_MMA_WAIT, c.abort_flag))) return;
            ++pieces;
            tc_fence_after();
        }
        if (warp_on) {
            const bool on = r < rows;
            // (a NaN sum stays NaN)
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float lse2 = l == 0.f ? -INFINITY : m + __log2f(l);
            const int nr = pc.prefix ? ROWS : p.L * p.g;
            const size_t at = ((size_t)pc.slot * 2 + part) * nr + r;
            if (on) (pc.prefix ? p.lse_p : p.lse_s)[at] = lse2;
            if (first < pc.steps) {
                float *dst = (pc.prefix ? p.o_p : p.o_s) + at * D;
#pragma unroll 1
                for (int h = 0; h < D; h += 32) {
                    uint32_t o[32];
                    tmem_ld32(to + h, o);
                    tmem_wait_ld();
                    if (on) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(dst + h + e) =
                                make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                                            __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                    }
                }
                tc_fence_before();
            }
        }
        if (first < pc.steps) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->ofree[x]);
        }
    }
}

}  // namespace pfx

template <int D>
__global__ void __launch_bounds__(pfx::NTHREADS, 1)
prefix_decode_kernel(const PrefixParams p, const __grid_constant__ CUtensorMap kp, const __grid_constant__ CUtensorMap vp,
                     const __grid_constant__ CUtensorMap ks, const __grid_constant__ CUtensorMap vs,
                     const __grid_constant__ CUtensorMap qm) {
    using namespace pfx;
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars *bars = reinterpret_cast<Bars *>(smem + C::OFF_BARS);
    int *pub = reinterpret_cast<int *>(p.meta + 2);
    int *s_prefix = p.prefix_in_ws ? pub : reinterpret_cast<int *>(smem + C::OFF_PREFIX);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->qfull[i], 1);
            mbar_init(&bars->qempty[i], 1);
            mbar_init(&bars->sready[i], 1);
            mbar_init(&bars->pready[i], 4);
            mbar_init(&bars->odone[i], 1);
            mbar_init(&bars->ofree[i], 4);
        }
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&bars->tmem), 512);
        tmem_relinquish();
    }
    if (warp == 2 && !p.prefix_in_ws) build_tile_prefix(p.seq_lens, p.B, p.T_max, TILE, s_prefix, lane);
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&kp);
        prefetch_tensormap(&vp);
        prefetch_tensormap(&ks);
        prefetch_tensormap(&vs);
        prefetch_tensormap(&qm);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    Ctx c;
    c.smem = smem;
    c.bars = bars;
    c.abort_flag = &bars->abort_flag;
    c.s_prefix = s_prefix;
    c.line = make_line(p, s_prefix[p.B]);
    c.w = blockIdx.x;
    c.p0 = (long long)blockIdx.x * c.line.W;
    c.p1 = c.p0 + c.line.W < c.line.total ? c.p0 + c.line.W : c.line.total;
    if (blockIdx.x == 0) {
        if (tid == 0) {
            p.meta[0] = c.line.n_p;
            p.meta[1] = c.line.W;
        }
        if (!p.prefix_in_ws)
            for (int i = tid; i <= p.B; i += NTHREADS) pub[i] = s_prefix[i];
    }
    // The merge kernel may be scheduled now; it waits for this grid to finish.
    pdl_launch_dependents();

    if (warp < 4) {
        regs_dec<REGS_CTRL>();
        if (c.p0 < c.p1) {
            if (warp == 0 && lane == 0) producer<D>(p, &kp, &vp, &ks, &vs, &qm, c);
            if (warp == 1 && lane == 0) mma_issuer<D>(p, c);
        }
    } else {
        regs_inc<REGS_SOFT>();
        if (c.p0 < c.p1) softmax_group<D>(p, c, warp, lane);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(bars->tmem, 512);
    }
}

// The suffix tile prefix of a batch too large for the decode kernel's shared memory.
__global__ void __launch_bounds__(32) prefix_tiles_kernel(const PrefixParams p) {
    build_tile_prefix(p.seq_lens, p.B, p.T_max, pfx::TILE, reinterpret_cast<int *>(p.meta + 2), threadIdx.x);
}

// Joins a row's partials: one warp per (new token, query head), its lanes across the head
// dimension.  The partials lie in L2 (they were just written); the loads of eight are in flight.
template <int D>
__global__ void __launch_bounds__(128) prefix_merge_kernel(const PrefixParams p) {
    using namespace pfx;
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);     // ((b * L + qi) * n_q + h)
    if (row >= (long long)p.B * p.L * p.n_q) return;
    const int h = (int)(row % p.n_q), tok = (int)(row / p.n_q);
    const int j = h / p.g, hg = h % p.g, b = tok / p.L, qi = tok % p.L;
    const int rt = tok / p.tok_tile, pr = (tok % p.tok_tile) * p.g + hg;      // row tile, row in it
    const long long u = (long long)j * p.pairs + rt / 2;
    const bool two = (rt | 1) < p.row_tiles;

    pdl_wait_primary();
    const int n_p = (int)p.meta[0];
    const long long W = p.meta[1];
    const int *pre = reinterpret_cast<const int *>(p.meta + 2);
    const int wp = p.row_tiles > 1 ? 2 : 1;
    const long long p_total = (long long)p.n_kv * p.pairs * n_p * wp;
    // prefix partials: workers [w0, w1], one part each (two row tiles) or two
    const long long ua = u * n_p * wp, ub = ua + (long long)n_p * wp;
    const int w0 = n_p > 0 ? (int)(ua / W) : 0, w1 = n_p > 0 ? (int)((ub - 1) / W) : -1;
    const int np = (w1 - w0 + 1) * (two ? 1 : 2);
    // suffix partials: workers [v0, v1], two parts each
    const int nt = pre[b + 1] - pre[b];
    const long long sa = p_total + (long long)pre[b] * p.n_kv + (long long)j * nt;
    const int v0 = nt > 0 ? (int)(sa / W) : 0, v1 = nt > 0 ? (int)((sa + nt - 1) / W) : -1;
    const int ns = (v1 - v0 + 1) * 2;
    const int rs = p.L * p.g, sr = qi * p.g + hg;

    float m = -INFINITY, sum = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    constexpr int U = 8;
    for (int k0 = 0; k0 < np + ns; k0 += U) {
        float ls[U], o[U][V];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = k0 + k;
            ls[k] = -INFINITY;
            const float *src = nullptr;
            if (i < np) {
                const int w = two ? i : i >> 1, part = two ? rt & 1 : i & 1;
                const size_t at = ((size_t)(u + w0 + w) * 2 + part) * ROWS + pr;
                ls[k] = p.lse_p[at];
                src = p.o_p + at * D;
            } else if (i < np + ns) {
                const int w = (i - np) >> 1, part = (i - np) & 1;
                const size_t at = ((size_t)((long long)b * p.n_kv + j + v0 + w) * 2 + part) * rs + sr;
                ls[k] = p.lse_s[at];
                src = p.o_s + at * D;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) o[k][v] = 0.f;
            if (src != nullptr) {
                if constexpr (V == 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(src + lane * 4);
                    o[k][0] = f.x; o[k][1] = f.y; o[k][2] = f.z; o[k][3] = f.w;
                } else {
                    const float2 f = *reinterpret_cast<const float2 *>(src + lane * 2);
                    o[k][0] = f.x; o[k][1] = f.y;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (ls[k] == -INFINITY) continue;      // nothing seen there (its values are not read)
            const float mn = fmaxf(m, ls[k]);
            const float a = fast_exp2(m - mn), w = fast_exp2(ls[k] - mn);
            sum = sum * a + w;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = acc[v] * a + w * o[k][v];
            m = mn;
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint32_t packed[V / 2];
#pragma unroll
    for (int v = 0; v < V; v += 2) packed[v / 2] = pack_bf16x2(acc[v] * inv, acc[v + 1] * inv);
    __nv_bfloat16 *dst = p.out + row * D + lane * V;
    if constexpr (V == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(packed[0], packed[1]);
    else
        *reinterpret_cast<uint32_t *>(dst) = packed[0];
    if (lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : (m + __log2f(sum)) * 0.69314718055994531f;
}

}  // namespace kvattn
