"""GPU tests of the row-scaled E4M3 cache: the write (with its rotation), the read back and the decode
over it, against plain 64-bit forms (B200)."""
import math

import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from tests import plain64

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(autouse=True)
def _knobs():
    kb.kvattn_debug_set_workers(0, 0)
    kb.kvattn_clear_device_flags()
    yield
    kb.kvattn_debug_set_workers(0, 0)
    assert kb.kvattn_read_device_flags() == 0


def pool(P, n_kv, S, d, fill=0x7F):
    """Codes (all NaN codes unless told otherwise) and scales of a page pool."""
    codes = torch.full((P, n_kv, S, d), fill, dtype=torch.uint8, device="cuda")
    return codes, torch.full((P, n_kv, S), float("nan"), device="cuda")


def rows_of(pages, scales, slots):
    """Rows [N, n_kv, d] and scales [N, n_kv] at slots, on the CPU."""
    S = pages.shape[2]
    page, row = slots // S, slots % S
    codes = pages.cpu().view(torch.float8_e4m3fn).float()
    return codes[page, :, row], scales.cpu()[page, :, row]


def check_written(pages, scales, slots, y, norm):
    """Codes and scales at `slots` against the exact rows y [N, n_kv, d] (64 bits); norm bounds the
    rotated pair, whose fp32 turn is off by at most 2^-21 of it."""
    code, scale = rows_of(pages, scales, slots)
    a = y.abs().amax(-1).clamp(min=2.0 ** -55)
    slack = 2.0 ** -21 * norm.amax(-1) / a
    plain64.assert_within(scale, a / 448, (2.0 ** -22 + slack) * a / 448, "scale")
    t = y * (448 / a)[..., None]
    half = (plain64.HALF_E4M3 * t.abs()).clamp(min=2.0 ** -10)
    plain64.assert_within(code, t, half + 448 * (2 * slack + 2.0 ** -22)[..., None], "code")


WRITE = [
    # N, n_q, n_kv, d, page, interleaved, base
    (1, 8, 2, 128, 128, False, 10000.0),
    (64, 64, 8, 128, 128, False, 10000.0),
    (37, 4, 1, 64, 16, True, 10000.0),
    (129, 6, 3, 96, 64, False, 500000.0),
    (50, 2, 2, 256, 7, True, 10000.0),
    (1000, 5, 1, 16, 128, False, 10000.0),
    (33, 32, 32, 80, 1, False, 10000.0),
    (300, 8, 8, 128, 256, False, 0.0),
]


@pytest.mark.parametrize("N,n_q,n_kv,d,S,inter,base", WRITE, ids=[f"n{c[0]}_d{c[3]}_s{c[4]}_{i}" for i, c in enumerate(WRITE)])
def test_write(N, n_q, n_kv, d, S, inter, base):
    g = torch.Generator().manual_seed(N + d)
    fused = torch.randn((N, n_q + 2 * n_kv, d), generator=g)
    fused[:, n_q:] *= torch.exp(3 * torch.randn((N, 2 * n_kv, 1), generator=g))      # rows of very different sizes
    fused = fused.to(torch.bfloat16)
    positions = torch.randint(0, 200000, (N,), generator=g).to(torch.int32)
    P = (N + S - 1) // S + 2
    slots = torch.randperm(P * S, generator=g)[:N]
    skip = torch.rand((N,), generator=g) < 0.2
    slots[skip] = torch.tensor([-1, P * S, -(1 << 40), 1 << 40])[torch.arange(int(skip.sum())) % 4]
    dev = fused.cuda()
    q, k, v = dev[:, :n_q], dev[:, n_q:n_q + n_kv], dev[:, n_q + n_kv:]              # slices of the projection
    kp, ks = pool(P, n_kv, S, d)
    vp, vs = pool(P, n_kv, S, d)
    q_out = torch.full((N, n_q, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = kb.kvattn_rope_append_rowscale(q, k, v, positions.cuda() if base else None, slots.cuda(), kp, vp, ks, vs,
                                         rope_base=base, interleaved=inter, q_out=q_out)
    torch.cuda.synchronize()
    assert got is q_out and torch.equal(dev.cpu(), fused), "inputs were changed"
    turn = (lambda x: plain64.rotate(x, positions, base, inter)) if base else (lambda x: x.double())
    ref = turn(fused[:, :n_q])
    size = fused[:, :n_q].double().abs().amax(-1, keepdim=True)
    plain64.assert_within(q_out, ref, plain64.HALF_BF16 * ref.abs() + 2.0 ** -20 * size, "q")
    keep = ~skip
    kk, vv = fused[:, n_q:n_q + n_kv], fused[:, n_q + n_kv:]
    check_written(kp, ks, slots[keep], turn(kk)[keep], kk.double().abs()[keep] * 2)
    check_written(vp, vs, slots[keep], vv.double()[keep], torch.zeros((int(keep.sum()), n_kv, d), dtype=torch.float64))
    # rows that no token was written to are as they were
    left = torch.ones((P * S,), dtype=torch.bool)
    left[slots[keep]] = False
    for codes, scales in ((kp, ks), (vp, vs)):
        flat = codes.cpu().transpose(1, 2).reshape(P * S, -1)
        assert bool((flat[left] == 0x7F).all())
        assert bool(torch.isnan(scales.cpu().transpose(1, 2).reshape(P * S, -1)[left]).all())


def test_write_in_place_and_without_query():
    N, n_q, n_kv, d, S, P = 20, 4, 2, 128, 16, 3
    g = torch.Generator().manual_seed(3)
    fused = torch.randn((N, n_q + 2 * n_kv, d), generator=g).to(torch.bfloat16)
    positions, slots = torch.arange(N).to(torch.int32), torch.arange(N)
    pools = []
    for with_q in (True, False):
        dev = fused.cuda()
        kp, ks = pool(P, n_kv, S, d)
        vp, vs = pool(P, n_kv, S, d)
        q = dev[:, :n_q] if with_q else None
        out = kb.kvattn_rope_append_rowscale(q, dev[:, n_q:n_q + n_kv], dev[:, n_q + n_kv:], positions.cuda(), slots.cuda(),
                                             kp, vp, ks, vs)
        torch.cuda.synchronize()
        if with_q:
            assert out.data_ptr() == dev.data_ptr()
            ref = plain64.rotate(fused[:, :n_q], positions, 10000.0, False)
            plain64.assert_within(dev[:, :n_q].cpu(), ref, plain64.HALF_BF16 * ref.abs() + 2.0 ** -18, "q in place")
        else:
            assert out is None and torch.equal(dev.cpu()[:, :n_q], fused[:, :n_q])
        assert torch.equal(dev.cpu()[:, n_q:], fused[:, n_q:])
        pools.append((kp.cpu(), ks.cpu(), vp.cpu(), vs.cpu()))
    for a, b in zip(*pools):
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


def test_write_odd_values():
    """Zero rows, tiny rows, infinities and NaN: a zero or tiny row keeps a usable scale, an infinity saturates at
    the largest float, a NaN becomes the NaN code and leaves its row alone."""
    d, S = 64, 8
    x = torch.ones((6, 1, d)).to(torch.bfloat16)
    x[0] = 0
    x[1] = 2.0 ** -80
    x[2, 0, 5] = float("inf")
    x[3, 0, 7] = float("nan")
    x[4] = 2.0 ** 100
    x[5] = float("nan")
    kp, ks = pool(1, 1, S, d)
    vp, vs = pool(1, 1, S, d)
    slots = torch.arange(6, device="cuda")
    kb.kvattn_rope_append_rowscale(None, x.cuda(), x.cuda(), None, slots, kp, vp, ks, vs, rope_base=0.0)
    k, v = kb.kvattn_gather_rowscale(kp, vp, ks, vs, slots)
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(k, nan=7.0), torch.nan_to_num(v, nan=7.0))
    k = k.cpu()[0].float()
    scale = ks.cpu()[0, 0]
    assert bool((k[0] == 0).all()) and bool((k[1] == 0).all())
    assert scale[0] == scale[1] == torch.tensor(2.0 ** -55) / 448
    assert bool((k[2][torch.arange(d) != 5] == 0).all()) and k[2, 5] > 3.3e38
    assert bool(torch.isnan(k[3, 7])) and bool((k[3][torch.arange(d) != 7] == 1).all())
    assert bool((k[4] == 2.0 ** 100).all()) and bool(torch.isnan(k[5]).all())


@pytest.mark.parametrize("N,n_kv,d,S", [(1, 1, 16, 1), (77, 3, 96, 16), (513, 8, 128, 128), (130, 2, 256, 64), (1000, 1, 64, 7)])
def test_read_back(N, n_kv, d, S):
    """Equal to the product of code and scale, rounded once, to the bit; slots outside the pool read as zeros."""
    g = torch.Generator().manual_seed(N)
    P = (N + S - 1) // S + 1
    codes = torch.randint(0, 256, (2, P, n_kv, S, d), generator=g).to(torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x30
    scales = torch.exp(5 * torch.randn((2, P, n_kv, S), generator=g))
    slots = torch.randint(0, P * S, (N,), generator=g)          # the same row may be read twice
    slots[::5] = torch.tensor([-1, P * S, -(1 << 50)])[torch.arange(len(slots[::5])) % 3]
    dev = [c.cuda() for c in codes], [s.cuda() for s in scales]
    big = torch.full((n_kv, N + 9, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    k, v = kb.kvattn_gather_rowscale(dev[0][0], dev[0][1].view(torch.float8_e4m3fn), dev[1][0], dev[1][1], slots.cuda(),
                                     k_out=big[:, 4:4 + N])
    torch.cuda.synchronize()
    inside = (slots >= 0) & (slots < P * S)
    at = slots.clamp(0, P * S - 1)
    for out, c, s in ((k, codes[0], scales[0]), (v, codes[1], scales[1])):
        ref = c.view(torch.float8_e4m3fn).float()[at // S, :, at % S] * s[at // S, :, at % S][..., None]
        ref = torch.where(inside[:, None, None], ref, torch.zeros(())).to(torch.bfloat16).transpose(0, 1)
        assert torch.equal(out.cpu(), ref)
    assert bool(torch.isnan(big[:, :4]).all()) and bool(torch.isnan(big[:, 4 + N:]).all())


def row_cache(shape, g):
    """Random rows of very different sizes as codes and scales (CPU)."""
    x = torch.randn(shape, generator=g) * torch.exp(torch.randn(shape[:-1], generator=g))[..., None]
    amax = x.abs().amax(-1)
    return (x * (448 / amax)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn), amax / 448


def paginate(codes, scales, lens, S, g):
    """The rows of [B, n_kv, T, ...] caches in shuffled pages; unused rows hold NaN codes and scales."""
    B, n_kv, T, d = codes[0].shape
    used = [(n + S - 1) // S for n in lens]
    M, P = max(max(used), 1) + 1, sum(used) + 2
    perm = torch.randperm(P, generator=g).tolist()
    table = torch.full((B, M), -7, dtype=torch.int32)
    out = [torch.full((P, n_kv, S, d), 0x7F, dtype=torch.uint8) for _ in codes]
    rows = [torch.full((P, n_kv, S), float("nan")) for _ in codes]
    for b, n in enumerate(lens):
        for i in range(used[b]):
            page = perm.pop()
            table[b, i] = page
            m = min(S, n - i * S)
            for x in range(2):
                out[x][page, :, :m] = codes[x].view(torch.uint8)[b, :, i * S:i * S + m]
                rows[x][page, :, :m] = scales[x][b, :, i * S:i * S + m]
    return out, rows, table


def run_decode(B, L, n_q, n_kv, lens, S, seed, window=0, scale=1 / math.sqrt(128.0), forced=None):
    g = torch.Generator().manual_seed(seed)
    T = max(max(lens), 1) + 3
    kc, ks = row_cache((B, n_kv, T, 128), g)
    vc, vs = row_cache((B, n_kv, T, 128), g)
    q = torch.randn((B, L, n_q, 128), generator=g).to(torch.bfloat16)
    if S:
        (kp, vp), (kr, vr), table = paginate((kc, vc), (ks, vs), lens, S, g)
    else:
        kp, vp, kr, vr, table = kc.view(torch.uint8).clone(), vc.view(torch.uint8).clone(), ks.clone(), vs.clone(), None
        for b, n in enumerate(lens):
            kp[b, :, n:], vp[b, :, n:] = 0x7F, 0x7F
            kr[b, :, n:], vr[b, :, n:] = float("nan"), float("nan")
    out = torch.full((B, L, n_q, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, L, n_q), float("nan"), device="cuda")
    if forced:
        kb.kvattn_debug_set_workers(*forced)
    kb.kvattn_gqa_decode_rowscale(q.cuda(), kp.cuda(), vp.cuda(), kr.cuda(), vr.cuda(),
                                  torch.tensor(lens, dtype=torch.int32, device="cuda"), scale,
                                  block_table=None if table is None else table.cuda(), window=window, out=out, lse=lse)
    torch.cuda.synchronize()
    group = n_q // n_kv
    worst = 0.0
    for b, n in enumerate(lens):
        see = plain64.visible(n, L, n, window).repeat_interleave(group, 0)
        for j in range(n_kv):
            k = kc[b, j, :n].double() * ks[b, j, :n, None].double()
            v = vc[b, j, :n].double() * vs[b, j, :n, None].double()
            rows = q[b, :, j * group:(j + 1) * group].reshape(L * group, 128)
            ref, rl, p = plain64.attention(rows, k, v, see, scale)
            slack = plain64.score_slack(rows, k, scale, "e4m3")
            o = out[b, :, j * group:(j + 1) * group].reshape(L * group, 128)
            l = lse[b, :, j * group:(j + 1) * group].reshape(L * group)
            worst = max(worst, plain64.assert_within(o, ref, plain64.out_bound(ref, p, v, slack, "e4m3"), f"out {b} {j}"))
            plain64.assert_within(l, rl, slack + 2.0 ** -21 * rl.abs() + 2e-6, f"lse {b} {j}")
    return worst


DECODE = [
    # n_q, n_kv, L, page, lens
    (8, 8, 1, 128, [0, 1, 127, 128, 129, 300]),
    (64, 8, 1, 128, [1000, 0, 1, 511, 512]),
    (32, 2, 1, 256, [700, 257, 3]),
    (32, 1, 1, 0, [1500, 200]),
    (64, 1, 1, 0, [640, 77]),
    (20, 4, 1, 128, [400, 129]),
    (32, 8, 5, 128, [1, 4, 5, 6, 300]),
    (16, 4, 4, 0, [0, 3, 200]),
    (64, 2, 3, 128, [130, 2, 500]),
]


@pytest.mark.parametrize("n_q,n_kv,L,S,lens", DECODE, ids=[f"g{c[0] // c[1]}_L{c[2]}_s{c[3]}" for c in DECODE])
def test_decode(n_q, n_kv, L, S, lens):
    run_decode(len(lens), L, n_q, n_kv, lens, S, seed=n_q + L)


@pytest.mark.parametrize("window,L", [(1, 1), (100, 1), (130, 5), (5000, 2)])
def test_decode_window(window, L):
    run_decode(4, L, 32, 8, [700, 1, 129, 260], 128, seed=window, window=window)


@pytest.mark.parametrize("forced", [(5, 1), (97, 1)])
def test_decode_forced_splits(forced):
    run_decode(3, 1, 32, 8, [900, 1, 400], 128, seed=9, forced=forced)


@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_decode_score_scales(scale):
    run_decode(2, 1, 16, 2, [300, 40], 128, seed=11, scale=scale)


def test_decode_zero_rows_next_to_large_ones():
    """A row of zeros (its scale is the smallest there is) among ordinary rows keeps its share of the sum."""
    B, n_q, n_kv, T = 1, 8, 1, 200
    g = torch.Generator().manual_seed(4)
    x = torch.randn((T, n_kv, 128), generator=g).to(torch.bfloat16)
    x[::3] = 0
    kp, ks = pool(B, n_kv, 256, 128)
    vp, vs = pool(B, n_kv, 256, 128)
    kb.kvattn_rope_append_rowscale(None, x.cuda(), x.cuda(), None, torch.arange(T, device="cuda"), kp, vp, ks, vs, rope_base=0.0)
    q = torch.randn((B, n_q, 128), generator=g).to(torch.bfloat16)
    out, lse = kb.kvattn_gqa_decode_rowscale(q.cuda(), kp, vp, ks, vs, torch.tensor([T], dtype=torch.int32, device="cuda"), 0.1)
    torch.cuda.synchronize()
    k = kp.cpu().view(torch.float8_e4m3fn)[0, 0, :T].double() * ks.cpu()[0, 0, :T, None].double()
    ref, rl, p = plain64.attention(q[0], k, k, torch.ones((n_q, T), dtype=torch.bool), 0.1)
    slack = plain64.score_slack(q[0], k, 0.1, "e4m3")
    plain64.assert_within(out[0], ref, plain64.out_bound(ref, p, k, slack, "e4m3"), "out")
    plain64.assert_within(lse[0], rl, slack + 2.0 ** -21 * rl.abs() + 2e-6, "lse")
