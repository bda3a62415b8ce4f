// serving_api.cuh -- entry points of the serving operators around the decode kernels: the
// row-scaled E4M3 cache, decode over a shared prefix, verification of drafted tokens.
// Included by kvattn_api.cu (it uses that file's checks, device state and map encoding).

namespace {

int check_pool(long long num_pages, int n_kv, long long page_size) {
    if (num_pages <= 0 || n_kv <= 0 || page_size <= 0) return KVATTN_ERR_INVALID_ARG;
    if (num_pages * page_size >= (1ll << 31) || num_pages * page_size * n_kv >= (1ll << 31)) return KVATTN_ERR_UNSUPPORTED;
    return KVATTN_OK;
}

// Bytes from the first element of N tokens of `row` elements, `stride` apart, to the last one.
size_t span(long long N, long long stride, long long row, int size) {
    return (size_t)((N - 1) * stride + row) * size;
}

// Whether N rows of `na` 2-byte elements, `sa` apart, share memory with N rows of `nb`, `sb` apart.  Rows of
// one stride may lie between each other, as the slices of a fused projection do.
bool rows_overlap(const void *a, long long sa, long long na, const void *b, long long sb, long long nb, long long N) {
    if (!overlaps(a, span(N, sa, na, 2), b, span(N, sb, nb, 2))) return false;
    if (sa != sb) return true;
    // b's row from the start of the row of a at or before it
    const long long diff = (long long)(reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a)) / 2;
    const long long at = (diff % sa + sa) % sa;
    return at < na || at + nb > sa;
}

template <int D>
int launch_prefix(PrefixParams &p, const CUtensorMap *maps, DeviceState *dev, cudaStream_t s) {
    using C = pfx::Cfg<D>;
    auto kern = prefix_decode_kernel<D>;
    cudaError_t e = set_smem_limit(reinterpret_cast<const void *>(kern), dev, C::SMEM);
    if (e != cudaSuccess) return fail_cuda(e, "cudaFuncSetAttribute(prefix decode)");
    p.table_in_ws = p.B > C::B_SMEM;
    if (p.table_in_ws) {
        prefix_table_kernel<<<1, 32, 0, s>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return fail_cuda(e, "prefix table launch");
        ++t_launches;
    }
    kern<<<p.workers, pfx::NTHREADS, C::SMEM, s>>>(p, maps[0], maps[1], maps[2], maps[3], maps[4]);
    e = cudaGetLastError();
    if (e != cudaSuccess) return fail_cuda(e, "prefix decode launch");
    ++t_launches;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(4 * p.row_tiles * p.n_kv), D / 32, 1);
    cfg.blockDim = dim3(32 * kMergeWarps, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, prefix_merge_kernel<D>, p);
    if (e != cudaSuccess) return fail_cuda(e, "prefix merge launch");
    ++t_launches;
    return KVATTN_OK;
}

// The plan of a prefix decode: row tiles, workers and the workspace's layout.
struct PrefixPlan {
    int tok_tile, row_tiles, pairs, workers;
    size_t meta, lse_p, lse_s, o_p, o_s, bytes;   // byte offsets, total
    long long line;                               // positions of the full capacity
};
PrefixPlan prefix_plan(const DeviceState *dev, int B, int L, int n_q, int n_kv, int D, int P_max, int T_max) {
    PrefixPlan w;
    const int g = n_q / n_kv;
    w.tok_tile = pfx::ROWS / g;
    w.row_tiles = (int)(((long long)B * L + w.tok_tile - 1) / w.tok_tile);
    w.pairs = (w.row_tiles + 1) / 2;
    const long long tiles_p = (P_max + pfx::TILE - 1) / pfx::TILE, tiles_s = (T_max + pfx::TILE - 1) / pfx::TILE;
    const long long units_p = (long long)n_kv * w.pairs, units_s = (long long)B * n_kv;
    w.line = (w.row_tiles > 1 ? units_p * (tiles_p + pfx::UP2) * pfx::WP2 : units_p * (tiles_p + pfx::UP1) * pfx::WP1) + units_s * (tiles_s + pfx::US) * pfx::WS;
    long long workers = g_force_workers > 0 ? g_force_workers : dev->sms;
    const long long most = (w.line + pfx::W_MIN - 1) / pfx::W_MIN;
    if (workers > most) workers = most;
    if (workers < 1) workers = 1;
    w.workers = (int)workers;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t rows_p = (size_t)(units_p + workers) * 2 * pfx::ROWS, rows_s = (size_t)(units_s + workers) * 2 * L * g;
    w.meta = 0;
    w.lse_p = up(8 + (size_t)(B + 1) * 4);
    w.lse_s = w.lse_p + up(rows_p * 4);
    w.o_p = w.lse_s + up(rows_s * 4);
    w.o_s = w.o_p + up(rows_p * D * 4);
    w.bytes = w.o_s + up(rows_s * D * 4);
    return w;
}

int check_prefix_sizes(int max_prefix_len, int max_seq_len, int batch, int q_len, int n_q_heads, int n_kv_heads,
                       int head_dim) {
    if (batch <= 0 || q_len <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 || max_prefix_len <= 0 || max_seq_len <= 0)
        return KVATTN_ERR_INVALID_ARG;
    if (n_q_heads % n_kv_heads != 0) return KVATTN_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return KVATTN_ERR_UNSUPPORTED;
    if ((long long)(n_q_heads / n_kv_heads) * q_len > pfx::ROWS) return KVATTN_ERR_UNSUPPORTED;
    if ((long long)batch * q_len > kMaxBatch) return KVATTN_ERR_UNSUPPORTED;
    if ((long long)batch * n_kv_heads * max_seq_len >= (1ll << 31) || (long long)n_kv_heads * max_prefix_len >= (1ll << 31))
        return KVATTN_ERR_UNSUPPORTED;
    return KVATTN_OK;
}

// Both forms: a contiguous cache is one page (the prefix) or one page a sequence (the suffixes).
int prefix_entry(const uint16_t *q, const uint16_t *kp, const uint16_t *vp, const int32_t *prefix_table,
                 const int32_t *prefix_len, long long prefix_pages, int prefix_page, int max_prefix_len, const uint16_t *ks,
                 const uint16_t *vs, const int32_t *block_table, const int32_t *seq_lens, long long pages, int page_size,
                 int max_pages, int max_seq_len, int batch, int q_len, int n_q, int n_kv, int d, float scale, uint16_t *out,
                 float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    if (!aligned16(q) || !aligned16(kp) || !aligned16(vp) || !aligned16(ks) || !aligned16(vs) || !aligned16(prefix_len) ||
        !aligned16(seq_lens) || !aligned16(prefix_table) || !aligned16(block_table) || !aligned16(out) || !aligned16(lse) ||
        !aligned16(workspace))
        return KVATTN_ERR_MISALIGNED;
    const size_t rows = (size_t)batch * q_len * n_q;
    const size_t pb = (size_t)prefix_pages * n_kv * prefix_page * d * 2, sb = (size_t)pages * n_kv * page_size * d * 2;
    const void *outs[3] = {out, lse, workspace};
    const size_t on[3] = {rows * d * 2, rows * 4, workspace_bytes};
    const void *ins[9] = {q, kp, vp, ks, vs, prefix_len, seq_lens, prefix_table, block_table};
    const size_t in[9] = {rows * d * 2, pb, pb, sb, sb, 4, (size_t)batch * 4,
                          prefix_table ? (size_t)(max_prefix_len / prefix_page) * 4 : 0,
                          block_table ? (size_t)batch * max_pages * 4 : 0};
    for (int i = 0; i < 3; ++i) {
        for (int k = 0; k < 9; ++k)
            if (ins[k] && overlaps(outs[i], on[i], ins[k], in[k])) return KVATTN_ERR_INVALID_ARG;
        for (int k = i + 1; k < 3; ++k)
            if (overlaps(outs[i], on[i], outs[k], on[k])) return KVATTN_ERR_INVALID_ARG;
    }
    DeviceState *dev = nullptr;
    int st = device_state(&dev);
    if (st != KVATTN_OK) return st;
    const PrefixPlan w = prefix_plan(dev, batch, q_len, n_q, n_kv, d, max_prefix_len, max_seq_len);
    if (w.line >= pfx::LINE_LIMIT) {
        snprintf(t_detail, sizeof(t_detail), "prefix and caches hold more tiles than the work split counts");
        return KVATTN_ERR_UNSUPPORTED;
    }
    if (workspace_bytes < w.bytes) {
        snprintf(t_detail, sizeof(t_detail), "workspace of %zu B, %zu needed", workspace_bytes, w.bytes);
        return KVATTN_ERR_INVALID_ARG;
    }
    if (4ll * w.row_tiles * n_kv >= (1ll << 31)) return KVATTN_ERR_UNSUPPORTED;
    const int g = n_q / n_kv;
    CUtensorMap maps[5];
    const void *base[4] = {kp, vp, ks, vs};
    for (int i = 0; i < 4; ++i) {
        st = encode_map_3d(&maps[i], base[i], d, i < 2 ? prefix_page : page_size,
                           (uint64_t)(i < 2 ? prefix_pages : pages) * n_kv, 64, pfx::TILE, CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != KVATTN_OK) return st;
    }
    // a row tile: the g heads of a KV head at tok_tile new tokens
    st = make_map_4d(&maps[4], q, d, g, n_kv, (uint64_t)batch * q_len, 64, g, 1, w.tok_tile, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != KVATTN_OK) return st;

    PrefixParams p = {};
    p.prefix_len = prefix_len;
    p.seq_lens = seq_lens;
    p.prefix_table = prefix_table;
    p.block_table = block_table;
    p.out = reinterpret_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    char *ws = static_cast<char *>(workspace);
    p.meta = reinterpret_cast<uint32_t *>(ws + w.meta);
    p.lse_p = reinterpret_cast<float *>(ws + w.lse_p);
    p.lse_s = reinterpret_cast<float *>(ws + w.lse_s);
    p.o_p = reinterpret_cast<float *>(ws + w.o_p);
    p.o_s = reinterpret_cast<float *>(ws + w.o_s);
    p.B = batch;
    p.L = q_len;
    p.n_q = n_q;
    p.n_kv = n_kv;
    p.g = g;
    p.P_max = max_prefix_len;
    p.T_max = max_seq_len;
    p.prefix_page = prefix_page;
    p.page_size = page_size;
    p.prefix_pages = (int)prefix_pages;
    p.pages = (int)pages;
    p.max_pages = max_pages;
    p.tok_tile = w.tok_tile;
    p.row_tiles = w.row_tiles;
    p.pairs = w.pairs;
    p.workers = w.workers;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return d == 128 ? launch_prefix<128>(p, maps, dev, s) : launch_prefix<64>(p, maps, dev, s);
}

}  // namespace

extern "C" {

int kvattn_rope_append_rowscale(const uint16_t *q, const uint16_t *k_new, const uint16_t *v_new,
                                const int32_t *positions, const int64_t *slots, uint16_t *q_out, uint8_t *k_pages,
                                uint8_t *v_pages, float *k_scales, float *v_scales, int n_tokens, int n_q_heads,
                                int n_kv_heads, int head_dim, int64_t q_stride, int64_t q_out_stride, int64_t k_stride,
                                int64_t v_stride, int num_pages, int page_size, float rope_base, int interleaved,
                                void *stream) {
    if (!k_new || !v_new || !slots || !k_pages || !v_pages || !k_scales || !v_scales) return KVATTN_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_out == nullptr)) return KVATTN_ERR_INVALID_ARG;
    if (n_tokens < 0 || n_kv_heads <= 0 || (q ? n_q_heads <= 0 : n_q_heads != 0)) return KVATTN_ERR_INVALID_ARG;
    if (!std::isfinite(rope_base) || rope_base < 0.f) return KVATTN_ERR_INVALID_ARG;
    if (rope_base > 0.f && !positions) return KVATTN_ERR_INVALID_ARG;
    if (head_dim <= 0 || head_dim % 16 || head_dim > 256) return KVATTN_ERR_UNSUPPORTED;
    int st = check_pool(num_pages, n_kv_heads, page_size);
    if (st != KVATTN_OK) return st;
    const long long q_row = (long long)n_q_heads * head_dim, kv_row = (long long)n_kv_heads * head_dim;
    if (k_stride < kv_row || v_stride < kv_row || (q && (q_stride < q_row || q_out_stride < q_row)))
        return KVATTN_ERR_INVALID_ARG;
    if (k_stride > (1ll << 31) || v_stride > (1ll << 31) || (q && (q_stride > (1ll << 31) || q_out_stride > (1ll << 31))))
        return KVATTN_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) ||
        !aligned16(v_pages) || !aligned16(slots) || !aligned16(positions) || !aligned16(k_scales) || !aligned16(v_scales) ||
        k_stride % 8 || v_stride % 8 || (q && (q_stride % 8 || q_out_stride % 8)))
        return KVATTN_ERR_MISALIGNED;
    if (n_tokens == 0) return KVATTN_OK;
    const size_t pool = (size_t)num_pages * n_kv_heads * page_size;
    const void *ins[5] = {q, k_new, v_new, positions, slots};
    const size_t in[5] = {q ? span(n_tokens, q_stride, q_row, 2) : 0, span(n_tokens, k_stride, kv_row, 2),
                          span(n_tokens, v_stride, kv_row, 2), (size_t)n_tokens * 4, (size_t)n_tokens * 8};
    const void *outs[5] = {k_pages, v_pages, k_scales, v_scales, q_out};
    const size_t on[5] = {pool * head_dim, pool * head_dim, pool * 4, pool * 4,
                          q ? span(n_tokens, q_out_stride, q_row, 2) : 0};
    // the rotated queries may be written in place, and next to the keys and values of a fused projection
    const long long stride[3] = {q_stride, k_stride, v_stride}, row[3] = {q_row, kv_row, kv_row};
    const bool in_place = q && q_out == q && q_out_stride == q_stride;
    for (int i = 0; i < 5; ++i) {
        if (!outs[i]) continue;
        for (int k = 0; k < 5; ++k) {
            if (!ins[k] || (i == 4 && k == 0 && in_place)) continue;
            if (i == 4 && k < 3 ? rows_overlap(q_out, q_out_stride, q_row, ins[k], stride[k], row[k], n_tokens)
                                : overlaps(outs[i], on[i], ins[k], in[k]))
                return KVATTN_ERR_INVALID_ARG;
        }
        for (int k = i + 1; k < 5; ++k)
            if (outs[k] && overlaps(outs[i], on[i], outs[k], on[k])) return KVATTN_ERR_INVALID_ARG;
    }
    DeviceState *dev = nullptr;
    st = device_state(&dev);
    if (st != KVATTN_OK) return st;
    RowAppendParams p = {};
    p.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    p.q_out = reinterpret_cast<__nv_bfloat16 *>(q_out);
    p.k_new = reinterpret_cast<const __nv_bfloat16 *>(k_new);
    p.v_new = reinterpret_cast<const __nv_bfloat16 *>(v_new);
    p.positions = positions;
    p.slots = reinterpret_cast<const long long *>(slots);
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.q_stride = q_stride;
    p.q_out_stride = q_out_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.N = n_tokens;
    p.n_q = n_q_heads;
    p.n_kv = n_kv_heads;
    p.d = head_dim;
    p.page_size = page_size;
    p.n_slots = (long long)num_pages * page_size;
    p.rotate = rope_base > 0.f;
    const double log2_base = p.rotate ? std::log2((double)rope_base) : 0.0;
    for (int i = 0; i < 16; ++i) p.turn_lo[i] = std::exp2(-2.0 * i / head_dim * log2_base) * 0.15915494309189533577;
    for (int i = 0; i < 8; ++i) p.turn_hi[i] = std::exp2(-2.0 * 16 * i / head_dim * log2_base);
    p.interleaved = interleaved ? 1 : 0;
    // few tokens: a token's rows are shared out over several warps, as many as keep every SM busy
    const int lpr = head_dim <= 64 ? 4 : head_dim <= 128 ? 8 : 16;
    const int at_once = 32 / lpr, rows = n_q_heads + 2 * n_kv_heads;
    int parts = (int)((16ll * dev->sms + n_tokens - 1) / n_tokens);
    if (parts > (rows + at_once - 1) / at_once) parts = (rows + at_once - 1) / at_once;
    p.rows_per_part = (rows + parts - 1) / parts;
    p.parts = (rows + p.rows_per_part - 1) / p.rows_per_part;
    const long long items = (long long)n_tokens * p.parts;
    const unsigned grid = (unsigned)((items + kRowThreads / 32 - 1) / (kRowThreads / 32));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (lpr == 4)
        row_append_kernel<4><<<grid, kRowThreads, 0, s>>>(p);
    else if (lpr == 8)
        row_append_kernel<8><<<grid, kRowThreads, 0, s>>>(p);
    else
        row_append_kernel<16><<<grid, kRowThreads, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail_cuda(e, "row append launch");
    ++t_launches;
    return KVATTN_OK;
}

int kvattn_gather_rowscale(const uint8_t *k_pages, const uint8_t *v_pages, const float *k_scales, const float *v_scales,
                           const int64_t *slots, uint16_t *k_out, uint16_t *v_out, int n_tokens, int n_kv_heads,
                           int head_dim, int64_t k_head_stride, int64_t v_head_stride, int num_pages, int page_size,
                           void *stream) {
    if (!k_pages || !v_pages || !k_scales || !v_scales || !slots || !k_out || !v_out) return KVATTN_ERR_INVALID_ARG;
    if (n_tokens < 0 || n_kv_heads <= 0) return KVATTN_ERR_INVALID_ARG;
    if (head_dim <= 0 || head_dim % 16 || head_dim > 256 || n_kv_heads > 65535) return KVATTN_ERR_UNSUPPORTED;
    int st = check_pool(num_pages, n_kv_heads, page_size);
    if (st != KVATTN_OK) return st;
    const long long row = (long long)n_tokens * head_dim;
    if (n_kv_heads > 1 && (k_head_stride < row || v_head_stride < row)) return KVATTN_ERR_INVALID_ARG;
    if (k_head_stride > (1ll << 40) || v_head_stride > (1ll << 40)) return KVATTN_ERR_UNSUPPORTED;
    if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_scales) || !aligned16(v_scales) || !aligned16(slots) ||
        !aligned16(k_out) || !aligned16(v_out) || (n_kv_heads > 1 && (k_head_stride % 8 || v_head_stride % 8)))
        return KVATTN_ERR_MISALIGNED;
    if (n_tokens == 0) return KVATTN_OK;
    const size_t pool = (size_t)num_pages * n_kv_heads * page_size;
    const void *ins[5] = {k_pages, v_pages, k_scales, v_scales, slots};
    const size_t in[5] = {pool * head_dim, pool * head_dim, pool * 4, pool * 4, (size_t)n_tokens * 8};
    const size_t kn = span(n_kv_heads, k_head_stride, row, 2), vn = span(n_kv_heads, v_head_stride, row, 2);
    for (int k = 0; k < 5; ++k)
        if (overlaps(k_out, kn, ins[k], in[k]) || overlaps(v_out, vn, ins[k], in[k])) return KVATTN_ERR_INVALID_ARG;
    // (the heads of the two may alternate in one buffer)
    if (n_kv_heads > 1 ? rows_overlap(k_out, k_head_stride, row, v_out, v_head_stride, row, n_kv_heads)
                       : overlaps(k_out, kn, v_out, vn))
        return KVATTN_ERR_INVALID_ARG;
    DeviceState *dev = nullptr;
    st = device_state(&dev);
    if (st != KVATTN_OK) return st;
    RowGatherParams p = {};
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.slots = reinterpret_cast<const long long *>(slots);
    p.k_out = reinterpret_cast<__nv_bfloat16 *>(k_out);
    p.v_out = reinterpret_cast<__nv_bfloat16 *>(v_out);
    p.k_head = k_head_stride;
    p.v_head = v_head_stride;
    p.N = n_tokens;
    p.n_kv = n_kv_heads;
    p.d = head_dim;
    p.page_size = page_size;
    p.n_slots = (long long)num_pages * page_size;
    const int lpr = head_dim <= 64 ? 4 : head_dim <= 128 ? 8 : 16;
    const int per = 256 / lpr;
    const dim3 grid((unsigned)((n_tokens + per - 1) / per), (unsigned)n_kv_heads, 1);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (lpr == 4)
        row_gather_kernel<4><<<grid, 256, 0, s>>>(p);
    else if (lpr == 8)
        row_gather_kernel<8><<<grid, 256, 0, s>>>(p);
    else
        row_gather_kernel<16><<<grid, 256, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail_cuda(e, "row gather launch");
    ++t_launches;
    return KVATTN_OK;
}

int kvattn_gqa_decode_rowscale(const uint16_t *q, const uint8_t *k_pages, const uint8_t *v_pages, const float *k_scales,
                               const float *v_scales, const int32_t *block_table, const int32_t *seq_lens, int num_pages,
                               int page_size, int max_pages_per_seq, int batch, int q_len, int n_q_heads, int n_kv_heads,
                               int head_dim, float scale, int window, uint16_t *out, float *lse, void *stream) {
    if (!q || !k_pages || !v_pages || !k_scales || !v_scales || !seq_lens || !out || !lse) return KVATTN_ERR_INVALID_ARG;
    if (batch <= 0 || q_len <= 0 || n_q_heads <= 0 || max_pages_per_seq <= 0 || window < 0) return KVATTN_ERR_INVALID_ARG;
    int st = check_pool(num_pages, n_kv_heads, page_size);
    if (st != KVATTN_OK) return st;
    if (n_q_heads % n_kv_heads != 0) return KVATTN_ERR_INVALID_ARG;
    if (!block_table && (num_pages != batch || max_pages_per_seq != 1)) return KVATTN_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return KVATTN_ERR_INVALID_ARG;
    if (head_dim != 128 || n_q_heads / n_kv_heads > 64 || (block_table && page_size % rs::TILE != 0))
        return KVATTN_ERR_UNSUPPORTED;
    if ((long long)batch * q_len > kMaxBatch || (long long)max_pages_per_seq * page_size >= (1ll << 31))
        return KVATTN_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_scales) || !aligned16(v_scales) ||
        !aligned16(block_table) || !aligned16(seq_lens) || !aligned16(out) || !aligned16(lse))
        return KVATTN_ERR_MISALIGNED;
    const size_t rows = (size_t)batch * q_len * n_q_heads, pool = (size_t)num_pages * n_kv_heads * page_size;
    const void *ins[7] = {q, k_pages, v_pages, k_scales, v_scales, seq_lens, block_table};
    const size_t in[7] = {rows * head_dim * 2, pool * head_dim, pool * head_dim, pool * 4, pool * 4, (size_t)batch * 4,
                          (size_t)batch * max_pages_per_seq * 4};
    for (int k = 0; k < 7; ++k)
        if (ins[k] && (overlaps(out, rows * head_dim * 2, ins[k], in[k]) || overlaps(lse, rows * 4, ins[k], in[k])))
            return KVATTN_ERR_INVALID_ARG;
    if (overlaps(out, rows * head_dim * 2, lse, rows * 4)) return KVATTN_ERR_INVALID_ARG;
    GqaCache cache{k_pages, v_pages, block_table, max_pages_per_seq * page_size, page_size, max_pages_per_seq, num_pages};
    return rs_decode_impl(q, cache, k_scales, v_scales, seq_lens, batch, n_q_heads, n_kv_heads, scale, out, lse,
                          static_cast<cudaStream_t>(stream), q_len, window);
}

int kvattn_gqa_decode_prefix_workspace(int max_prefix_len, int max_seq_len, int batch, int q_len, int n_q_heads,
                                       int n_kv_heads, int head_dim, size_t *bytes) {
    if (!bytes) return KVATTN_ERR_INVALID_ARG;
    int st = check_prefix_sizes(max_prefix_len, max_seq_len, batch, q_len, n_q_heads, n_kv_heads, head_dim);
    if (st != KVATTN_OK) return st;
    DeviceState *dev = nullptr;
    st = device_state(&dev);
    if (st != KVATTN_OK) return st;
    *bytes = prefix_plan(dev, batch, q_len, n_q_heads, n_kv_heads, head_dim, max_prefix_len, max_seq_len).bytes;
    return KVATTN_OK;
}

int kvattn_gqa_decode_prefix(const uint16_t *q, const uint16_t *k_prefix, const uint16_t *v_prefix,
                             const int32_t *prefix_len, int max_prefix_len, const uint16_t *k_cache,
                             const uint16_t *v_cache, const int32_t *seq_lens, int max_seq_len, int batch, int q_len,
                             int n_q_heads, int n_kv_heads, int head_dim, float scale, uint16_t *out, float *lse,
                             void *workspace, size_t workspace_bytes, void *stream) {
    if (!q || !k_prefix || !v_prefix || !prefix_len || !k_cache || !v_cache || !seq_lens || !out || !lse || !workspace)
        return KVATTN_ERR_INVALID_ARG;
    int st = check_prefix_sizes(max_prefix_len, max_seq_len, batch, q_len, n_q_heads, n_kv_heads, head_dim);
    if (st != KVATTN_OK) return st;
    if (!std::isfinite(scale)) return KVATTN_ERR_INVALID_ARG;
    return prefix_entry(q, k_prefix, v_prefix, nullptr, prefix_len, 1, max_prefix_len, max_prefix_len, k_cache, v_cache,
                        nullptr, seq_lens, batch, max_seq_len, 1, max_seq_len, batch, q_len, n_q_heads, n_kv_heads,
                        head_dim, scale, out, lse, workspace, workspace_bytes, stream);
}

int kvattn_gqa_decode_prefix_paged(const uint16_t *q, const uint16_t *k_pages, const uint16_t *v_pages,
                                   const int32_t *prefix_table, const int32_t *prefix_len, int max_prefix_pages,
                                   const int32_t *block_table, const int32_t *seq_lens, int num_pages, int page_size,
                                   int max_pages_per_seq, int batch, int q_len, int n_q_heads, int n_kv_heads,
                                   int head_dim, float scale, uint16_t *out, float *lse, void *workspace,
                                   size_t workspace_bytes, void *stream) {
    if (!q || !k_pages || !v_pages || !prefix_table || !prefix_len || !block_table || !seq_lens || !out || !lse || !workspace)
        return KVATTN_ERR_INVALID_ARG;
    if (max_prefix_pages <= 0 || max_pages_per_seq <= 0) return KVATTN_ERR_INVALID_ARG;
    int st = check_pool(num_pages, n_kv_heads, page_size);
    if (st != KVATTN_OK) return st;
    if (page_size % pfx::TILE != 0) return KVATTN_ERR_UNSUPPORTED;
    const long long P = (long long)max_prefix_pages * page_size, T = (long long)max_pages_per_seq * page_size;
    if (P >= (1ll << 31) || T >= (1ll << 31)) return KVATTN_ERR_UNSUPPORTED;
    st = check_prefix_sizes((int)P, (int)T, batch, q_len, n_q_heads, n_kv_heads, head_dim);
    if (st != KVATTN_OK) return st;
    if (!std::isfinite(scale)) return KVATTN_ERR_INVALID_ARG;
    return prefix_entry(q, k_pages, v_pages, prefix_table, prefix_len, num_pages, page_size, (int)P, k_pages, v_pages,
                        block_table, seq_lens, num_pages, page_size, max_pages_per_seq, (int)T, batch, q_len, n_q_heads,
                        n_kv_heads, head_dim, scale, out, lse, workspace, workspace_bytes, stream);
}

int kvattn_verify_drafts(const void *target_probs, const void *draft_probs, const int32_t *draft_tokens,
                         const int32_t *draft_lens, const float *u_accept, const float *u_sample, int32_t *accepted,
                         int32_t *tokens, int batch, int n_drafts, int vocab, int bf16, int64_t target_batch_stride,
                         int64_t target_pos_stride, int64_t draft_batch_stride, int64_t draft_pos_stride, void *stream) {
    if (!target_probs || !u_sample || !accepted || !tokens) return KVATTN_ERR_INVALID_ARG;
    if (batch <= 0 || n_drafts < 0 || vocab <= 0) return KVATTN_ERR_INVALID_ARG;
    if (n_drafts > 0 && (!draft_tokens || !u_accept)) return KVATTN_ERR_INVALID_ARG;
    if (batch > kMaxBatch || n_drafts > 1024 || vocab > (1 << 28)) return KVATTN_ERR_UNSUPPORTED;
    const bool dq = draft_probs != nullptr && n_drafts > 0;
    const long long strides[4] = {target_batch_stride, target_pos_stride, dq ? draft_batch_stride : 0, dq ? draft_pos_stride : 0};
    for (int i = 0; i < 4; ++i) {
        if (strides[i] < 0) return KVATTN_ERR_INVALID_ARG;
        if (strides[i] > (1ll << 40)) return KVATTN_ERR_UNSUPPORTED;
    }
    const int size = bf16 ? 2 : 4;
    const uintptr_t align = (uintptr_t)(size - 1);
    if ((reinterpret_cast<uintptr_t>(target_probs) & align) || (reinterpret_cast<uintptr_t>(draft_probs) & align) ||
        !aligned16(draft_tokens) || !aligned16(draft_lens) || !aligned16(u_accept) || !aligned16(u_sample) ||
        !aligned16(accepted) || !aligned16(tokens))
        return KVATTN_ERR_MISALIGNED;
    const size_t L = (size_t)n_drafts;
    const size_t tn = ((size_t)(batch - 1) * strides[0] + L * strides[1] + vocab) * size;
    const size_t dn = dq ? ((size_t)(batch - 1) * strides[2] + (L - 1) * strides[3] + vocab) * size : 0;
    const void *ins[6] = {target_probs, dq ? draft_probs : nullptr, draft_tokens, draft_lens, u_accept, u_sample};
    const size_t in[6] = {tn, dn, batch * L * 4, (size_t)batch * 4, batch * L * 4, (size_t)batch * 4};
    const size_t an = (size_t)batch * 4, kn = (size_t)batch * (L + 1) * 4;
    for (int i = 0; i < 6; ++i)
        if (ins[i] && (overlaps(accepted, an, ins[i], in[i]) || overlaps(tokens, kn, ins[i], in[i])))
            return KVATTN_ERR_INVALID_ARG;
    if (overlaps(accepted, an, tokens, kn)) return KVATTN_ERR_INVALID_ARG;
    DeviceState *dev = nullptr;
    int st = device_state(&dev);
    if (st != KVATTN_OK) return st;
    VerifyParams p = {};
    p.p = target_probs;
    p.q = dq ? draft_probs : nullptr;
    p.drafts = draft_tokens;
    p.lens = draft_lens;
    p.u_accept = u_accept;
    p.u_sample = u_sample;
    p.accepted = accepted;
    p.tokens = tokens;
    p.p_b = strides[0];
    p.p_l = strides[1];
    p.q_b = strides[2];
    p.q_l = strides[3];
    p.B = batch;
    p.L = n_drafts;
    p.V = vocab;
    const int per16 = 16 / size;
    p.vec = aligned16(target_probs) && aligned16(p.q) && strides[0] % per16 == 0 && strides[1] % per16 == 0 &&
            strides[2] % per16 == 0 && strides[3] % per16 == 0;
    // CTAs a sequence: as many as still run at once, each with at least a vector a thread (64
    // sequences of 128000: 14.7 us with 8, 17.2 with 2, and 29 with CTAs of twice the size that do
    // not all fit)
    int C = 1;
    while (C < kVerifyMaxCluster && 2ll * C * batch <= (long long)kVerifyPerSm * dev->sms && (long long)C * kVerifyThreads * per16 < vocab) C *= 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(batch * C), 1, 1);
    cfg.blockDim = dim3(kVerifyThreads, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = bf16 ? cudaLaunchKernelEx(&cfg, verify_kernel<__nv_bfloat16>, p)
                         : cudaLaunchKernelEx(&cfg, verify_kernel<float>, p);
    if (e != cudaSuccess) return fail_cuda(e, "verify launch");
    ++t_launches;
    return KVATTN_OK;
}

}  // extern "C"
