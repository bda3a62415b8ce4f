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
// over a suffix; each unit is a run of 128-token K/V tiles.  All units are laid end to end on a
// line whose positions stand for time -- WP2 a prefix tile that serves two row tiles, WP1 one that
// serves one, WS a suffix tile, and for a unit's start and end UP2, UP1 or US tiles more -- and
// worker w (one CTA per SM) takes an equal contiguous range of it, computed on the device from
// prefix_len and seq_lens (so a captured call may be replayed with other lengths).  Prefix and
// suffix work thus run side by side: some SMs keep the tensor cores busy while others stream
// suffixes from memory.  The weights are measured: with 4, 2, 4 and one tile a unit (8, 4, 8 and 1
// in these positions) 64 sequences behind 32768 tokens took 151 us and 16 of up to 4096 tokens
// 108 us; with 8, 6, 6 and one, one and three tiles they took 141 and 83 us.  A prefix unit of two row
// tiles that counts for one tile more leaves its workers behind where it is short (128 sequences of
// up to 64 behind 1000 tokens 89 us, 62 with four; of up to 300 behind 300 99 and 78 us); one of a
// single row tile does not (8 sequences behind 2000 tokens 18.7 us, 20.2 with four).  They are the
// same for both head sizes.  Every piece (a worker's part of a unit)
// leaves a normalised partial and its log-sum-exp in the caller's workspace; prefix_merge_kernel
// joins a row's partials.
//
// Pipeline of a CTA (384 threads):
//   warp 0       producer: TMA loads (128-byte swizzle, no multicast) of Q tiles, and of K and
//                V tiles into a ring each.
//   warp 1       one thread issues the tcgen05.mma of the scores, S = Q K^T (A, B from shared memory).
//   warp 2       one thread issues those of the outputs, O_x += P_x V (P_x read from tensor memory,
//                V tile MN-major).
//   warps 4..11  two softmax groups x = 0, 1 of 128 threads, one thread per row: a row's 128
//                scores are one TMEM lane, so its maximum and sum need no exchange.
// Steps alternate between the groups, so that one group's exponentials run while the tensor
// cores work for the other: in a two-row-tile unit the groups hold the two row tiles and
// each K/V tile makes two steps; in a one-row-tile unit both groups hold the same rows and take
// alternate K/V tiles, each with its own (max, sum, O), which the merge joins.
//
// Tensor memory holds O_0, O_1 (D columns each), P_0, P_1 (64 each, bf16) and, in what is left, one
// score buffer that the groups use in turn (D = 128) or two (D = 64).  A score buffer is free as soon
// as its scores are in registers, so the next step's scores are computed under this step's
// exponentials, which then follow one another without a wait.  Two more things keep them so.
// The weights are taken against the running maximum of the steps before, so no exponential waits
// for this step's; the maximum moves afterwards, when a row's scores have exceeded it by more
// than 2^8 (its O and sum are then rescaled before the next step's product), and at once only on
// a piece's first step and where they exceed it by 2^LIMIT.  And the weights are handed over in two
// halves of 64 tokens, the first half's product running under the second half's exponentials.
// Measured on 64 sequences of 64 heads behind 32768 tokens, cycles a pair of steps (the products
// alone: 2048, the exponentials alone: 2048):
//   weights over their scores, one issuer       6200  eight MMAs take ~600 to issue, a commit ~180
//   ... an issuer a group, issuing freely       5500  the groups' products interleave, both end late,
//                                                     and the groups fall into step
//   ... in turns                                4700
//   ... steps in halves, a score buffer each    4300  the score products of N = 64 are bound by shared
//                                                     memory, which also takes the TMA writes
//   ... two threads a row                       4900  a swap of maxima, and registers that do not reach
//   weights apart, an issuer a product          4000  (this kernel)
// What bounds it now is the softmax warps: two a scheduler, each 1300-1500 cycles for 64 columns
// when both run (the exponential unit's share is 1024), and 250-400 at each of four hand-overs.
// Asking for the barriers' phases ahead of their use changed nothing.  A suffix is bound by
// memory where it is long (4.5 TB/s at 8 sequences of up to 8000 tokens behind 32768) and by the
// start and end of a piece, some 5000 cycles, where it is short.
// Weights enter the value product rounded to bf16 (at most half a step, 2^-8 relative, each independent
// of the others; the output is rounded to bf16 itself); sums, maxima and O are fp32.  A bf16 remainder
// beside them, as the decode kernels of one sequence have it, finds no room: tensor memory is full.  The
// error of an output, relative to its size, is 0.0019 to 0.0024 where its own rounding alone gives 0.0017.
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
    uint32_t *meta;                // [0] tiles of the prefix; from [2] on the suffix table [B + 1]
    float *lse_p, *o_p;            // prefix partials [units_p + workers][2][128], [..][2][D][128]
    float *lse_s, *o_s;            // suffix partials [B * n_kv + workers][2][L * g], [..][2][L * g][D]
    int B, L, n_q, n_kv, g;
    int P_max, T_max;              // capacities (lengths are clamped to them)
    int prefix_page, page_size;    // rows per page of the prefix's and the suffixes' cache
    int prefix_pages, pages;       // pages of the two (one pool when paged)
    int max_pages;                 // block_table columns
    int tok_tile;                  // new tokens in a row tile: floor(128 / g)
    int row_tiles, pairs;          // ceil(B L / tok_tile), ceil(row_tiles / 2)
    int workers;
    int table_in_ws;               // the suffix table was written to the workspace before
    float scale_log2;              // scale * log2(e)
};

namespace pfx {

constexpr int TILE = 128;
constexpr int ROWS = 128;
constexpr int NTHREADS = 384;
// registers of a thread after the split between the first warpgroup (producer, issuers) and the
// softmax warpgroups: a row's 128 scores and its packed weights stay in registers (64 sequences behind
// 32768 tokens: 131 us with 56 and 224, 139 with 72 and 216, 132 with 40 and 232)
constexpr int REGS_LAUNCH = 168, REGS_CTRL = 56, REGS_SOFT = 224;
static_assert(128 * REGS_CTRL + 256 * REGS_SOFT <= NTHREADS * REGS_LAUNCH, "registers of the launch");
constexpr int CHUNK = 128 * 128;          // [128 rows x 128 bytes]
constexpr int NS_MAX = 10;
// How far (log2 units) scores may exceed the maximum the weights are taken against: RESCALE from the
// next step on, LIMIT within a step.  Sums then stay below (2^8 T + 2^16 TILE) of the largest value over T
// tokens, so values of up to 2^80 keep them in range (with a LIMIT of 64 values above 2^60 left it).
constexpr float RESCALE = 8.f, LIMIT = 16.f;
// Line positions (see above), and the least a worker takes.
constexpr uint32_t WP2 = 8, WP1 = 6, WS = 6, UP2 = 4, UP1 = 1, US = 3, W_MIN = 8;
constexpr long long LINE_LIMIT = 1ll << 30;

// Two fp32 values in one 64-bit register pair: one instruction works on both.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

template <int D>
struct Cfg {
    static constexpr int NCH = D / 64;                  // 64-wide chunks of a row
    static constexpr int KV_BYTES = NCH * CHUNK;        // a K or V tile
    static constexpr int Q_BYTES = NCH * CHUNK;         // a Q tile
    // Slots: a ring of K tiles and one of V tiles.  (In one ring with an odd number of slots the
    // score issuer, which waits for K tiles alone, could be a use of the slot behind and take its
    // barrier's parity for the next one's.)
    static constexpr uint32_t NS = (160 * 1024) / KV_BYTES, NK = NS / 2, NV = NS - NK;
    static constexpr int OFF_Q = NS * KV_BYTES;
    static constexpr int OFF_BARS = OFF_Q + 2 * Q_BYTES;
    static constexpr int OFF_TABLE = OFF_BARS + 384;
    // the suffix table lies in shared memory up to this batch, in the workspace beyond
    static constexpr int B_SMEM = 640;
    static constexpr int SMEM = OFF_TABLE + (B_SMEM + 1) * 4;
    static_assert(NS <= NS_MAX, "ring barriers");
    static_assert(SMEM <= 232448, "shared memory of an SM");
};

// Operand descriptors (tc05.cuh, 128-byte swizzle, 8-row groups 1024 bytes apart) and MMAs from
// their low words: an operand's steps differ there alone, by the step's offset in 16-byte units.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16); }
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "n"(DESC_HI), "r"(idesc), "n"(ACC ? 1 : 0)
        : "memory");
}
template <bool ACC>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "n"(DESC_HI), "r"(idesc), "n"(ACC ? 1 : 0)
        : "memory");
}

// Tensor memory columns: NSB score buffers of 128, the groups' weights (bf16 pairs, 64 columns
// each), the groups' outputs (D columns each); all 512 for either head size.
template <int D>
struct Tm {
    static constexpr uint32_t NSB = D == 64 ? 2 : 1;
    static constexpr uint32_t S = 0, P = 128 * NSB, O = 512 - 2 * D;
    static_assert(P + 2 * 64 == O, "columns");
};

struct Bars {
    uint64_t full[NS_MAX], empty[NS_MAX];
    uint64_t qfull[2], qempty[2];
    uint64_t sready[2];      // group x's next scores are in tensor memory
    uint64_t sfree[2];       // [buffer] the scores have been read
    uint64_t pready[2][2];   // [group][half] the weights are written (and O_x rescaled)
    uint64_t pdone[2];       // group x's value product is done
    uint64_t ofree[2];       // group x has read O_x
    uint64_t drain[2];       // an issuer's products after a wait that gave up
    uint32_t tmem;
    int prefix_len;
    int abort_flag;
};
static_assert(sizeof(Bars) <= 384, "barrier block overflows its slot");

// ------------------------------------------------------------------ the line of work
// The suffix table: word b holds, in its upper 25 bits, the sum over the sequences before b of
// their line units c = tiles + US (0 without tokens), and in its lower 7 the last tile's tokens
// less one: a sequence's tiles and length without another load.
__device__ __forceinline__ uint32_t table_units(uint32_t w) { return w >> 7; }

// Fills tab[0..B] by one warp.
__device__ __forceinline__ void build_table(const int32_t *seq_lens, int B, int T_max, uint32_t *tab, int lane) {
    uint32_t running = 0;
    constexpr int U = 4;
    for (int base = 0; base < B; base += 32 * U) {
        int len[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + 32 * u + lane;
            len[u] = i < B ? clamp_len(__ldg(seq_lens + i), T_max) : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (base + 32 * u >= B) break;
            const int i = base + 32 * u + lane;
            const uint32_t nt = (uint32_t)tiles_of(len[u], TILE);
            const uint32_t c = nt ? nt + US : 0;
            uint32_t s = c;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, s, off);
                if (lane >= off) s += y;
            }
            if (i < B) tab[i] = ((running + s - c) << 7) | (nt ? (uint32_t)(len[u] - 1) & 127u : 0u);
            running += __shfl_sync(0xffffffffu, s, 31);
        }
    }
    if (lane == 0) tab[B] = running << 7;
}

// The same on every CTA and in the merge kernel.
struct Line {
    uint32_t n_p;            // prefix tiles
    uint32_t wp;             // positions of a prefix tile
    uint32_t unit_p;         // positions of a prefix unit
    uint32_t p_total;        // of all of them
    uint32_t total, W;
};
__device__ __forceinline__ Line make_line(const PrefixParams &p, uint32_t n_p, uint32_t suffix_units) {
    Line l;
    l.n_p = n_p;
    l.wp = p.row_tiles > 1 ? WP2 : WP1;
    l.unit_p = n_p ? (n_p + (p.row_tiles > 1 ? UP2 : UP1)) * l.wp : 0;
    l.p_total = (uint32_t)(p.n_kv * p.pairs) * l.unit_p;
    l.total = l.p_total + suffix_units * (uint32_t)p.n_kv * WS;
    l.W = (l.total + p.workers - 1) / p.workers;
    if (l.W < W_MIN) l.W = W_MIN;
    return l;
}
// Tiles of a unit (nt tiles of WT positions from u0 on) that start in worker w's range.
template <uint32_t WT>
__device__ __forceinline__ void piece_tiles_of(const Line &l, uint32_t u0, uint32_t nt, uint32_t w, uint32_t &lt0, uint32_t &lt1) {
    const uint32_t a = w * l.W, b = a + l.W;
    lt0 = a <= u0 ? 0u : min(nt, (a - u0 + WT - 1) / WT);
    lt1 = b <= u0 ? 0u : min(nt, (b - u0 + WT - 1) / WT);
}
__device__ __forceinline__ void prefix_piece(const Line &l, uint32_t u0, uint32_t w, uint32_t &lt0, uint32_t &lt1) {
    if (l.wp == WP2) piece_tiles_of<WP2>(l, u0, l.n_p, w, lt0, lt1);
    else piece_tiles_of<WP1>(l, u0, l.n_p, w, lt0, lt1);
}
__device__ __forceinline__ void suffix_piece(const Line &l, uint32_t u0, uint32_t nt, uint32_t w, uint32_t &lt0, uint32_t &lt1) {
    piece_tiles_of<WS>(l, u0, nt, w, lt0, lt1);
}

// In a suffix the two groups hold the same few rows: group 1 holds them `shift` lanes further up,
// so that the groups' warps that work lie on different schedulers.  Its Q operand starts that
// many rows before the tile (in shared memory of the CTA; those lanes are not read).
__device__ __forceinline__ int suffix_shift(int rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : 0; }

struct Piece {
    bool prefix;
    bool two;            // two row tiles: each K/V tile makes two steps
    int j;               // KV head
    int b;               // sequence (suffix)
    int pair;            // row tile pair (prefix)
    int len;             // tokens of the unit
    int lt0, lt1;        // its tiles
    int steps;
    uint32_t slot;       // partial
};

// A walk over worker w's pieces, with what the roles keep of the pieces before.
struct Walk {
    Piece pc;
    uint32_t pos, end;       // line positions still to take
    uint32_t u0, u1;         // the present unit's
    uint32_t steps, tiles;   // of the pieces before (the steps' parity is the group that takes the first)
    int qs;                  // Q slot of the piece's first row tile
    uint32_t quse0, quse1;   // uses of each Q slot, this piece's included
};
__device__ __forceinline__ Walk walk_start(const Line &l, int w) {
    Walk k;
    k.pos = (uint32_t)w * l.W;
    k.end = k.pos + l.W < l.total ? k.pos + l.W : l.total;
    k.u0 = k.u1 = 0;
    k.steps = k.tiles = 0;
    k.qs = 0;
    k.quse0 = k.quse1 = 0;
    k.pc.steps = 0;
    k.pc.lt0 = k.pc.lt1 = 0;
    k.pc.two = true;
    k.pc.prefix = true;
    k.pc.b = k.pc.j = k.pc.pair = 0;
    return k;
}
// Moves to the next piece with tiles; false after the last.
__device__ __forceinline__ bool walk_next(Walk &k, const PrefixParams &p, const Line &l, const uint32_t *tab,
                                          int prefix_len, int w) {
    Piece &c = k.pc;
    k.steps += (uint32_t)c.steps;
    k.tiles += (uint32_t)(c.lt1 - c.lt0);
    if (!c.two) k.qs ^= 1;
    c.two = true;            // (skipped pieces take no slot)
    while (k.pos < k.end) {
        uint32_t a, b;
        if (k.pos < l.p_total) {
            const uint32_t ul = l.unit_p, u = k.pos / ul;
            c.prefix = true;
            c.j = (int)(u / (uint32_t)p.pairs);
            c.pair = (int)u - c.j * p.pairs;
            c.len = prefix_len;
            c.slot = u + (uint32_t)w;
            k.u0 = u * ul;
            k.u1 = k.u0 + ul;
            prefix_piece(l, k.u0, (uint32_t)w, a, b);
        } else {
            if (!c.prefix && c.j + 1 < p.n_kv && k.pos == k.u1) {
                // the same sequence's next head
                ++c.j;
                const uint32_t ul = k.u1 - k.u0;
                k.u0 = k.u1;
                k.u1 += ul;
            } else {
                // the sequence at this position (the last one whose first unit is not past it)
                const uint32_t at = (k.pos - l.p_total) / ((uint32_t)p.n_kv * WS);
                int lo = 0, hi = p.B - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (table_units(tab[mid]) <= at) lo = mid; else hi = mid - 1;
                }
                c.b = lo;
                const uint32_t w0 = tab[lo];
                const uint32_t cu = table_units(tab[lo + 1]) - table_units(w0);
                c.len = (int)((cu - US - 1) * TILE + (w0 & 127u) + 1);
                c.j = (int)((k.pos - l.p_total - table_units(w0) * (uint32_t)p.n_kv * WS) / (cu * WS));
                c.prefix = false;
                k.u0 = l.p_total + (table_units(w0) * (uint32_t)p.n_kv + (uint32_t)c.j * cu) * WS;
                k.u1 = k.u0 + cu * WS;
            }
            c.slot = (uint32_t)(c.b * p.n_kv + c.j + w);
            suffix_piece(l, k.u0, (uint32_t)tiles_of(c.len, TILE), (uint32_t)w, a, b);
        }
        k.pos = k.u1 < k.end ? k.u1 : k.end;
        if (a < b) {
            c.lt0 = (int)a;
            c.lt1 = (int)b;
            c.two = c.prefix && 2 * c.pair + 1 < p.row_tiles;
            c.steps = (c.lt1 - c.lt0) * (c.two ? 2 : 1);
            if (c.two || k.qs == 0) ++k.quse0;
            if (c.two || k.qs == 1) ++k.quse1;
            return true;
        }
    }
    c.steps = 0;
    c.lt0 = c.lt1 = 0;
    return false;
}

struct Ctx {
    uint8_t *smem;
    Bars *bars;
    volatile int *abort_flag;
    const uint32_t *tab;
    Line line;
    int prefix_len;
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
    uint32_t n[2] = {0, 0};         // K and V tiles issued
    bool ok = true;
    Walk k = walk_start(c.line, c.w);
    while (ok && walk_next(k, p, c.line, c.tab, c.prefix_len, c.w)) {
        const Piece &pc = k.pc;
        const int nq = pc.two ? 2 : 1;
        for (int r = 0; r < nq && ok; ++r) {
            const int s = (k.qs + r) & 1;
            const uint32_t use = s ? k.quse1 : k.quse0;
            if (use > 1 && !mbar_wait(&bars->qempty[s], use & 1u, FLAG_EMPTY_WAIT, c.abort_flag)) {
                ok = false;
                break;
            }
            const int tok = pc.prefix ? (2 * pc.pair + r) * p.tok_tile : pc.b * p.L;
            mbar_arrive_expect_tx(&bars->qfull[s], (uint32_t)(C::NCH * p.tok_tile * p.g * 128));
#pragma unroll
            for (int ch = 0; ch < C::NCH; ++ch)
                tma_load_4d(c.smem + C::OFF_Q + s * C::Q_BYTES + ch * CHUNK, qm, &bars->qfull[s], 64 * ch, 0, pc.j, tok,
                            keep);
        }
        // (the prefix is read again by the CTAs that serve its other row tiles)
        const CUtensorMap *km = pc.prefix ? kp : ks, *vm = pc.prefix ? vp : vs;
        const uint64_t pol = pc.prefix ? keep : once;
        for (int lt = pc.lt0; lt < pc.lt1 && ok; ++lt) {
            const TileSrc src = pc.prefix ? tile_source(p.prefix_table, 0, p.prefix_page, 0, lt, TILE, pc.len)
                                          : tile_source(p.block_table, p.max_pages, p.page_size, pc.b, lt, TILE, pc.len);
            // (a page outside the pool is read as zeros: a coordinate outside the map)
            const bool inside = src.page >= 0 && src.page < (pc.prefix ? p.prefix_pages : p.pages);
            const int z = inside ? src.page * p.n_kv + pc.j : -1;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const uint32_t ring = kv ? C::NV : C::NK, s = (kv ? C::NK : 0) + n[kv] % ring;
                if (!ok || !mbar_wait(&bars->empty[s], ((n[kv] / ring) & 1u) ^ 1u, FLAG_EMPTY_WAIT, c.abort_flag)) {
                    ok = false;
                    break;
                }
                ++n[kv];
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
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint32_t ring = kv ? C::NV : C::NK, base = kv ? C::NK : 0;
            for (uint32_t m = n[kv] > ring ? n[kv] - ring : 0; m < n[kv]; ++m)
                mbar_wait_sleep(&bars->full[base + m % ring], (m / ring) & 1u, FLAG_FULL_WAIT, nullptr);
        }
        if (k.quse0 > 0) mbar_wait_sleep(&bars->qfull[0], (k.quse0 - 1) & 1u, FLAG_FULL_WAIT, nullptr);
        if (k.quse1 > 0) mbar_wait_sleep(&bars->qfull[1], (k.quse1 - 1) & 1u, FLAG_FULL_WAIT, nullptr);
    }
}

// ------------------------------------------------------------------ MMA issuers (warps 1 and 2, lane 0)
// Step n of the CTA belongs to group n & 1.  The tiles are given back by the commits behind their
// last products.
// S = Q K^T of every step, into the score buffers in turn.
template <int D>
__device__ __forceinline__ bool score_issuer(const PrefixParams &p, const Ctx &c) {
    using C = Cfg<D>;
    constexpr uint32_t NSB = Tm<D>::NSB;
    Bars *bars = c.bars;
    const uint32_t smem = smem_u32(c.smem);
    constexpr uint32_t idesc = idesc_f16_major(128, TILE, 1, 1, 0, 0);
    const int qoff_suffix = suffix_shift(p.L * p.g) * 128;
    uint32_t n = 0;
    Walk k = walk_start(c.line, c.w);
    while (walk_next(k, p, c.line, c.tab, c.prefix_len, c.w)) {
        const Piece &pc = k.pc;
        for (int i = 0; i < pc.steps; ++i, ++n) {
            const uint32_t x = n & 1u, buf = n % NSB;
            const int qslot = pc.two ? (k.qs + i) & 1 : k.qs;
            const uint32_t t = k.tiles + (uint32_t)(pc.two ? i >> 1 : i), slot = t % C::NK;
            if (i < (pc.two ? 2 : 1) &&
                !mbar_wait(&bars->qfull[qslot], ((qslot ? k.quse1 : k.quse0) - 1) & 1u, FLAG_FULL_WAIT, c.abort_flag))
                return false;
            if (!mbar_wait(&bars->full[slot], (t / C::NK) & 1u, FLAG_FULL_WAIT, c.abort_flag)) return false;
            if (n >= NSB && !mbar_wait(&bars->sfree[buf], (n / NSB - 1) & 1u, FLAG_MMA_WAIT, c.abort_flag)) return false;
            tc_fence_after();
            const uint32_t ts = bars->tmem + Tm<D>::S + 128 * buf;
            const uint32_t q = desc_lo(smem + C::OFF_Q + qslot * C::Q_BYTES - (!pc.prefix && x == 1 ? qoff_suffix : 0), 16);
            const uint32_t kt = desc_lo(smem + slot * C::KV_BYTES, 16);
            mma_ss<false>(ts, q, kt, idesc);
#pragma unroll
            for (int kk = 1; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * CHUNK + (kk & 3) * 32) >> 4;
                mma_ss<true>(ts, q + off, kt + off, idesc);
            }
            umma_commit(&bars->sready[x]);
            if (!pc.two || (i & 1)) umma_commit(&bars->empty[slot]);
            if (i + (pc.two ? 2 : 1) >= pc.steps) umma_commit(&bars->qempty[qslot]);
        }
    }
    return true;
}
// O_x += P_x V of every step, each in two halves of 64 tokens as the weights come.
template <int D>
__device__ __forceinline__ bool value_issuer(const PrefixParams &p, const Ctx &c) {
    using C = Cfg<D>;
    Bars *bars = c.bars;
    const uint32_t smem = smem_u32(c.smem);
    constexpr uint32_t idesc = idesc_f16_major(128, D, 1, 1, 0, 1);
    uint32_t n = 0, pieces[2] = {0, 0};
    Walk k = walk_start(c.line, c.w);
    while (walk_next(k, p, c.line, c.tab, c.prefix_len, c.w)) {
        const Piece &pc = k.pc;
        for (int i = 0; i < pc.steps; ++i, ++n) {
            const uint32_t x = n & 1u, par = (n >> 1) & 1u;
            const uint32_t t = k.tiles + (uint32_t)(pc.two ? i >> 1 : i), slot = C::NK + t % C::NV;
            if (!mbar_wait(&bars->full[slot], (t / C::NV) & 1u, FLAG_FULL_WAIT, c.abort_flag)) return false;
            if (i < 2) {
                const uint32_t before = x ? pieces[1]++ : pieces[0]++;
                if (before > 0 && !mbar_wait(&bars->ofree[x], (before - 1) & 1u, FLAG_MMA_WAIT, c.abort_flag)) return false;
            }
            const uint32_t tp = bars->tmem + Tm<D>::P + 64 * x, to = bars->tmem + Tm<D>::O + D * x;
            const uint32_t vt = desc_lo(smem + slot * C::KV_BYTES, CHUNK);
            if (!mbar_wait(&bars->pready[x][0], par, FLAG_MMA_WAIT, c.abort_flag)) return false;
            tc_fence_after();
            if (i < 2) mma_ts<false>(to, tp, vt, idesc);
            else mma_ts<true>(to, tp, vt, idesc);
#pragma unroll
            for (int kk = 1; kk < TILE / 32; ++kk) mma_ts<true>(to, tp + kk * 8, vt + kk * (2048 >> 4), idesc);
            if (!mbar_wait(&bars->pready[x][1], par, FLAG_MMA_WAIT, c.abort_flag)) return false;
            tc_fence_after();
#pragma unroll
            for (int kk = TILE / 32; kk < TILE / 16; ++kk) mma_ts<true>(to, tp + kk * 8, vt + kk * (2048 >> 4), idesc);
            if (!pc.two || (i & 1)) umma_commit(&bars->empty[slot]);
            umma_commit(&bars->pdone[x]);
        }
    }
    return true;
}

// ------------------------------------------------------------------ softmax (warps 4..11)
// 64 weights 2^(cs s - m) as bf16 pairs, and their sum.
__device__ __forceinline__ float weights64(const float *s, float cs, float m, uint32_t (&w)[32]) {
    const float off = m == -INFINITY ? 0.f : -m;
    const uint64_t cs2 = pack2(cs, cs), off2 = pack2(off, off);
    uint64_t l2[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        const uint64_t z = fma2(pack2(s[2 * e], s[2 * e + 1]), cs2, off2);
        float a, b;
        unpack2(z, a, b);
        a = fast_exp2(a);
        b = fast_exp2(b);
        l2[e & 1] = add2(l2[e & 1], pack2(a, b));
        w[e] = pack_bf16x2(a, b);
    }
    float la, lb;
    unpack2(add2(l2[0], l2[1]), la, lb);
    return la + lb;
}
__device__ __forceinline__ float max128(const float *s) {
    float t0 = s[0], t1 = s[1], t2 = s[2], t3 = s[3];
#pragma unroll
    for (int e = 4; e + 8 <= TILE; e += 8) {
        t0 = max3(t0, s[e], s[e + 1]);
        t1 = max3(t1, s[e + 2], s[e + 3]);
        t2 = max3(t2, s[e + 4], s[e + 5]);
        t3 = max3(t3, s[e + 6], s[e + 7]);
    }
    t0 = max3(t0, s[TILE - 4], s[TILE - 3]);
    t1 = max3(t1, s[TILE - 2], s[TILE - 1]);
    return fmaxf(fmaxf(t0, t1), fmaxf(t2, t3));
}
// O *= a (the columns of this thread's row).
template <int D>
__device__ __forceinline__ void rescale(uint32_t to, float a) {
#pragma unroll 1
    for (int d = 0; d < D; d += 16) {
        uint32_t o[16];
        tmem_ld16(to + d, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
        tmem_st16(to + d, o);
    }
    tmem_wait_st();
}

template <int D>
__device__ __forceinline__ void softmax_group(const PrefixParams &p, const Ctx &c, int warp, int lane) {
    using C = Cfg<D>;
    Bars *bars = c.bars;
    const uint32_t tmem = bars->tmem;
    const int x = (warp - 4) >> 2;
    const int quad = warp & 3;
    const int lrow = 32 * quad + lane;                // TMEM lane
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    constexpr uint32_t NSB = Tm<D>::NSB;
    const uint32_t tp = tmem + lanes + Tm<D>::P + 64 * x, to = tmem + lanes + Tm<D>::O + D * x;
    const bool negate = p.scale_log2 < 0.f;           // (the maximum is taken of the unscaled scores)
    const float cs = fmaxf(fabsf(p.scale_log2), 1e-30f);   // (a zero scale: masked scores stay -inf)
    uint32_t n_x = 0;                                 // steps of this group
    Walk k = walk_start(c.line, c.w);
    const Piece &pc = k.pc;
    while (walk_next(k, p, c.line, c.tab, c.prefix_len, c.w)) {
        const int first = (int)((k.steps & 1u) ^ (uint32_t)x);      // this group's first step of the piece
        const int part = first;                       // row tile (two) or share of the K/V tiles
        // rows of the tile that are real
        int rows = p.L * p.g;
        if (pc.prefix) {
            const int tok0 = (2 * pc.pair + (pc.two ? part : 0)) * p.tok_tile;
            rows = min(p.tok_tile, p.B * p.L - tok0) * p.g;
        }
        // row of the tile (suffixes: group 1's lie further up)
        const int r = lrow - (!pc.prefix && x == 1 ? suffix_shift(rows) : 0);
        const int q_on = r - lane;                    // the warp's first row
        const bool warp_on = q_on >= 0 && q_on < rows;
        // (lanes past the rows hold scores of what else lies in the Q tile, NaN among it, and have no say in the
        // rescaling: with it groups of 12 heads took 141 us where they take 129, of 7 37.9 and 35.4)
        const bool on = r < rows;
        // the suffixes come last and all have as many rows: warps without any are done, and the
        // first answers for them
        if (!pc.prefix && !warp_on) return;
        const uint32_t arrivals = pc.prefix || q_on > 0 ? 1u : 4u - (uint32_t)((rows - 1) / 32);
        // positions this row sees: all of the prefix; a suffix up to its own token
        const int limit = pc.prefix ? pc.len : pc.len - p.L + 1 + min(r / p.g, p.L - 1);
        float m = -INFINITY, l = 0.f;                 // (log2 units; m in scaled scores)
        float m_next = -INFINITY;                     // the maximum from the next step on
        for (int i = first; i < pc.steps; i += 2, ++n_x) {
            const int it = pc.two ? i >> 1 : i;
            if (!warp_all(mbar_wait(&bars->sready[x], n_x & 1u, FLAG_MMA_WAIT, c.abort_flag))) return;
            const uint32_t buf = (2 * n_x + (uint32_t)x) % NSB, ts = tmem + lanes + Tm<D>::S + 128 * buf;
            // the step before must be through its value product before its weights are overwritten
            // or O_x is rescaled
            bool settled = i == first;
            auto settle = [&]() -> bool {
                if (settled) return true;
                settled = true;
                if (!warp_all(mbar_wait(&bars->pdone[x], (n_x - 1) & 1u, FLAG_MMA_WAIT, c.abort_flag))) return false;
                tc_fence_after();
                return true;
            };
            float s[TILE];
            uint32_t w[32];
            if (warp_on) {
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 4; ++h) tmem_ld32(ts + 32 * h, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * h));
                tmem_wait_ld();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_n(&bars->sfree[buf], arrivals);
            if (warp_on) {
                if (__any_sync(0xffffffffu, on && m_next != m)) {
                    if (!settle()) return;
                    const float a = m == -INFINITY ? 1.f : fast_exp2(m - m_next);
                    l *= a;
                    rescale<D>(to, a);
                    m = m_next;
                }
                if (negate) {
#pragma unroll
                    for (int e = 0; e < TILE; ++e) s[e] = -s[e];
                }
                // the tile's first position (a unit's last tile ends at its length: its first
                // columns repeat earlier positions, or lie before the cache)
                const int tok0 = (pc.lt0 + it) * TILE;
                const int y = min(tok0, pc.len - TILE);
                if (y < tok0 || (!pc.prefix && tok0 + TILE > pc.len - p.L + 1)) {
                    const int lo = tok0 - y, hi = limit - y;
#pragma unroll
                    for (int e = 0; e < TILE; ++e) s[e] = (e >= lo && e < hi) ? s[e] : -INFINITY;
                }
                if (i == first) m = m_next = max128(s) * cs;
                float lsum = weights64(s, cs, m, w);
                const float tm = max128(s) * cs;
                if (__any_sync(0xffffffffu, on && tm > m + LIMIT)) {
                    const float m_new = fmaxf(m, tm);
                    if (i != first) {
                        if (!settle()) return;
                        const float a = m == -INFINITY ? 1.f : fast_exp2(m - m_new);
                        l *= a;
                        rescale<D>(to, a);
                    }
                    m = m_new;
                    lsum = weights64(s, cs, m, w);
                }
                m_next = tm > m + RESCALE ? tm : m;
                l += lsum;
                if (!settle()) return;
                tmem_st32(tp, w);
                tmem_wait_st();
                tc_fence_before();
            } else if (!settle()) {
                return;      // (or its arrivals would count for the step before)
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_n(&bars->pready[x][0], arrivals);
            if (warp_on) {
                l += weights64(s + 64, cs, m, w);
                tmem_st32(tp + 32, w);
                tmem_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_n(&bars->pready[x][1], arrivals);
        }
        // ---- the piece's partial: O / l and log2 of the sum
        const bool took = first < pc.steps;
        if (took) {
            if (!warp_all(mbar_wait(&bars->pdone[x], (n_x - 1) & 1u, FLAG_MMA_WAIT, c.abort_flag))) return;
            tc_fence_after();
        }
        if (warp_on) {
            // (a NaN sum stays NaN)
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float lse2 = l == 0.f ? -INFINITY : m + __log2f(l);
            const size_t at = (size_t)pc.slot * 2 + part;
            const uint32_t rs = (uint32_t)(p.L * p.g);
            if (on) {
                if (pc.prefix) p.lse_p[at * ROWS + r] = lse2;
                else p.lse_s[at * rs + r] = lse2;
            }
            if (took) {
                // prefix rows next to each other, so that a warp stores whole lines; a suffix's few
                // rows each by itself
                float *dst = pc.prefix ? p.o_p + at * D * ROWS + r : p.o_s + (at * rs + r) * D;
#pragma unroll
                for (int d0 = 0; d0 < D; d0 += 64) {
                    uint32_t o[64];
                    tmem_ld32(to + d0, *reinterpret_cast<uint32_t(*)[32]>(o));
                    tmem_ld32(to + d0 + 32, *reinterpret_cast<uint32_t(*)[32]>(o + 32));
                    tmem_wait_ld();
                    if (d0 + 64 == D) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_n(&bars->ofree[x], arrivals);
                    }
                    if (on && pc.prefix) {
#pragma unroll
                        for (int d = 0; d < 64; ++d) dst[(d0 + d) * ROWS] = __uint_as_float(o[d]) * inv;
                    } else if (on) {
#pragma unroll
                        for (int d = 0; d < 64; d += 4)
                            *reinterpret_cast<float4 *>(dst + d0 + d) =
                                make_float4(__uint_as_float(o[d]) * inv, __uint_as_float(o[d + 1]) * inv,
                                            __uint_as_float(o[d + 2]) * inv, __uint_as_float(o[d + 3]) * inv);
                    }
                }
            }
        } else if (took) {
            if (lane == 0) mbar_arrive_n(&bars->ofree[x], arrivals);
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
    extern __shared__ __align__(1024) uint8_t prefix_smem[];
    uint8_t *smem = prefix_smem;
    Bars *bars = reinterpret_cast<Bars *>(smem + C::OFF_BARS);
    uint32_t *pub = p.meta + 2;
    uint32_t *tab = p.table_in_ws ? pub : reinterpret_cast<uint32_t *>(smem + C::OFF_TABLE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (uint32_t s = 0; s < C::NS; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->qfull[i], 1);
            mbar_init(&bars->qempty[i], 1);
            mbar_init(&bars->sready[i], 1);
            mbar_init(&bars->pready[i][0], 4);
            mbar_init(&bars->pready[i][1], 4);
            mbar_init(&bars->sfree[i], 4);
            mbar_init(&bars->pdone[i], 1);
            mbar_init(&bars->ofree[i], 4);
            mbar_init(&bars->drain[i], 1);
        }
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (tid == 32 * 2) bars->prefix_len = clamp_len(__ldg(p.prefix_len), p.P_max);
    if (warp == 1) {
        tmem_alloc(smem_u32(&bars->tmem), 512);
        tmem_relinquish();
    }
    if (warp == 3 && !p.table_in_ws) build_table(p.seq_lens, p.B, p.T_max, tab, lane);
    if (warp == 0 && lane == 1) {
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
    c.tab = tab;
    c.prefix_len = bars->prefix_len;
    c.line = make_line(p, (uint32_t)tiles_of(c.prefix_len, TILE), table_units(tab[p.B]));
    c.w = blockIdx.x;
    if (blockIdx.x == 0 && warp == 3) {
        if (lane == 0) p.meta[0] = c.line.n_p;
        if (!p.table_in_ws)
            for (int i = lane; i <= p.B; i += 32) pub[i] = tab[i];
    }
    // The merge kernel may be scheduled now; it waits for this grid to finish.
    pdl_launch_dependents();

    if (warp < 4) {
        regs_dec<REGS_CTRL>();
        if (warp == 0 && lane == 0) producer<D>(p, &kp, &vp, &ks, &vs, &qm, c);
        // (an issuer that gave up lets its products in flight end before the CTA can)
        if ((warp == 1 || warp == 2) && lane == 0 && !(warp == 1 ? score_issuer<D>(p, c) : value_issuer<D>(p, c))) {
            umma_commit(&bars->drain[warp - 1]);
            mbar_wait_sleep(&bars->drain[warp - 1], 0, FLAG_MMA_WAIT, nullptr);
        }
    } else {
        regs_inc<REGS_SOFT>();
        softmax_group<D>(p, c, warp, lane);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(bars->tmem, 512);
    }
}

// The suffix table of a batch too large for the decode kernel's shared memory.
__global__ void __launch_bounds__(32) prefix_table_kernel(const PrefixParams p) {
    pfx::build_table(p.seq_lens, p.B, p.T_max, p.meta + 2, threadIdx.x);
}

// Joins the rows' partials.  A CTA takes 32 rows of a row tile, a lane each (the partials lie
// row by row), and 32 dimensions, four a warp.  Its time is the round trips that follow one another
// (the table, the partials, the stores), not its bytes: the partials' addresses follow from the
// table alone, so the log-sum-exps and the values of up to MC_P prefix and MC_S suffix partials are
// loaded together, without branches (places that hold no partial are read and dropped).  8 sequences
// behind 2000 tokens: 23.4 us a call with loads that wait for the log-sum-exps, 19.3 us so.
// The result goes through shared memory to be written in whole rows.
constexpr int kMergeWarps = 8;
namespace pfx {
constexpr int MC_P = 8, MC_S = 4, MV = 32 / kMergeWarps;
// The weighted sum of a row's partials, and a chunk of N more.
struct Joined {
    float m, sum, acc[MV];
};
template <int N>
__device__ __forceinline__ void join(Joined &r, const float (&x)[N], const float (&f)[N][MV]) {
    float m = r.m;
#pragma unroll
    for (int k = 0; k < N; ++k) m = x[k] > m || x[k] != x[k] ? x[k] : m;      // (NaN stays)
    const float off = m == -INFINITY ? 0.f : m;
    const float scale = fast_exp2(r.m - off);
    r.m = m;
    r.sum *= scale;
#pragma unroll
    for (int v = 0; v < MV; ++v) r.acc[v] *= scale;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float w = fast_exp2(x[k] - off);
        r.sum += w;
#pragma unroll
        for (int v = 0; v < MV; ++v) r.acc[v] = x[k] == -INFINITY ? r.acc[v] : fmaf(w, f[k][v], r.acc[v]);
    }
}
}  // namespace pfx
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) prefix_merge_kernel(const PrefixParams p) {
    using namespace pfx;
    __shared__ float s_out[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // block -> (KV head, row tile, quarter)
    const int quarter = blockIdx.x & 3, rt = (blockIdx.x >> 2) % p.row_tiles, j = (blockIdx.x >> 2) / p.row_tiles;
    const int pr = 32 * quarter + lane;
    const int tok = rt * p.tok_tile + pr / p.g, hg = pr % p.g;
    const bool on = pr < p.tok_tile * p.g && tok < p.B * p.L;
    if (__syncthreads_or(on) == 0) return;
    const int b = on ? tok / p.L : 0, qi = on ? tok % p.L : 0;
    const uint32_t u = (uint32_t)(j * p.pairs + rt / 2);
    const bool two = (rt | 1) < p.row_tiles;
    const uint32_t rs = (uint32_t)(p.L * p.g), sr = (uint32_t)(qi * p.g + hg);
    const int d0 = 32 * blockIdx.y + warp * MV;

    pdl_wait_primary();
    const uint32_t *tab = p.meta + 2;
    const uint32_t tb = table_units(tab[b]), cu = on ? table_units(tab[b + 1]) - tb : 0;
    const Line l = make_line(p, p.meta[0], table_units(tab[p.B]));
    // prefix partials: workers w0 .. w1, one part each (two row tiles) or two
    const uint32_t ua = u * l.unit_p;
    const int w0 = (int)(ua / l.W), w1 = l.n_p > 0 ? (int)((ua + l.unit_p - 1) / l.W) : w0 - 1;
    const int sh = two ? 0 : 1, part0 = two ? rt & 1 : 0;
    const int np = (w1 - w0 + 1) << sh;
    // suffix partials: workers v0 .. v1, two parts each
    const uint32_t sa = l.p_total + (tb * (uint32_t)p.n_kv + (uint32_t)j * cu) * WS;
    const int v0 = (int)(sa / l.W), v1 = cu > 0 ? (int)((sa + cu * WS - 1) / l.W) : v0 - 1;
    const int ns = 2 * (v1 - v0 + 1), ns_max = __reduce_max_sync(0xffffffffu, ns);
    const uint32_t at_p = (u + (uint32_t)w0) * 2 + (uint32_t)part0;      // prefix partial i: at_p + (two ? 2 i : i)
    const uint32_t at_s = (uint32_t)(b * p.n_kv + j + v0) * 2;           // suffix partial i: at_s + i

    auto load_p = [&](int i0, float (&x)[MC_P], float (&f)[MC_P][MV]) {
#pragma unroll
        for (int k = 0; k < MC_P; ++k) {
            const int i = max(min(i0 + k, np - 1), 0);
            const size_t at = at_p + (two ? 2 * i : i);
            x[k] = p.lse_p[at * ROWS + pr];
            const float *o = p.o_p + (at * D + d0) * ROWS + pr;
#pragma unroll
            for (int v = 0; v < MV; ++v) f[k][v] = o[v * ROWS];
        }
#pragma unroll
        for (int k = 0; k < MC_P; ++k) {
            uint32_t a, z;
            prefix_piece(l, ua, (uint32_t)(w0 + ((i0 + k) >> sh)), a, z);
            if (!on || i0 + k >= np || a >= z) x[k] = -INFINITY;     // no such partial
        }
    };
    auto load_s = [&](int i0, float (&x)[MC_S], float (&f)[MC_S][MV]) {
#pragma unroll
        for (int k = 0; k < MC_S; ++k) {
            const int i = max(min(i0 + k, ns - 1), 0);
            const size_t at = (size_t)(at_s + i) * rs + sr;
            x[k] = p.lse_s[at];
            const float4 o = *reinterpret_cast<const float4 *>(p.o_s + at * D + d0);
            f[k][0] = o.x; f[k][1] = o.y; f[k][2] = o.z; f[k][3] = o.w;
        }
#pragma unroll
        for (int k = 0; k < MC_S; ++k) {
            uint32_t a, z;
            suffix_piece(l, sa, cu - US, (uint32_t)(v0 + ((i0 + k) >> 1)), a, z);
            if (i0 + k >= ns || a >= z) x[k] = -INFINITY;
        }
    };
    static_assert(MV == 4, "a float4 a partial");
    Joined r = {-INFINITY, 0.f, {}};
    {
        float xp[MC_P], fp[MC_P][MV], xs[MC_S], fs[MC_S][MV];
        load_p(0, xp, fp);
        load_s(0, xs, fs);
        join(r, xp, fp);
        join(r, xs, fs);
    }
    for (int i = MC_P; i < np; i += MC_P) {
        float x[MC_P], f[MC_P][MV];
        load_p(i, x, f);
        join(r, x, f);
    }
    for (int i = MC_S; i < ns_max; i += MC_S) {
        float x[MC_S], f[MC_S][MV];
        load_s(i, x, f);
        join(r, x, f);
    }
    const float inv = r.sum == 0.f ? 0.f : 1.f / r.sum;
#pragma unroll
    for (int v = 0; v < MV; ++v) s_out[lane][warp * MV + v] = r.acc[v] * inv;
    if (blockIdx.y == 0 && warp == 0 && on)
        p.lse[(size_t)tok * p.n_q + j * p.g + hg] = r.sum == 0.f ? -INFINITY : (r.m + __log2f(r.sum)) * 0.69314718055994531f;
    __syncthreads();
    // four bf16 a thread, eight threads a row
    const int rr = threadIdx.x >> 3, c4 = (threadIdx.x & 7) * 4;
    const int q = 32 * quarter + rr, t = rt * p.tok_tile + q / p.g;
    if (q < p.tok_tile * p.g && t < p.B * p.L) {
        const float *s = &s_out[rr][c4];
        *reinterpret_cast<uint2 *>(p.out + ((size_t)t * p.n_q + j * p.g + q % p.g) * D + 32 * blockIdx.y + c4) =
            make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
    }
}

}  // namespace kvattn
