"""GPU tests of the serving operators over buffers whose offsets pass 32 bits (B200)."""
import math

import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from tests import plain64
from tests import rowscale64 as r64

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(autouse=True)
def _flags():
    kb.kvattn_clear_device_flags()
    yield
    torch.cuda.empty_cache()
    assert kb.kvattn_read_device_flags() == 0


def normal(*s, seed=1):
    return torch.randn(s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


def test_row_scaled_pool():
    """A pool of 4.6 GB of codes: the rows of its last pages are written, read back and attended to."""
    n_kv, S, d, P = 8, 128, 128, 35000                     # 2^31 bytes end in page 16384, 2^32 in page 32768
    N, n_q = 700, 32
    pools = [torch.full((P, n_kv, S, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    rows = [torch.full((P, n_kv, S), float("nan"), device="cuda") for _ in range(2)]
    x = normal(N, 2 * n_kv, d)
    pages = torch.tensor([P - 1, 16383, 16384, 32768, 32767, 0])
    t = torch.arange(N)
    slots = (pages[t // S] * S + t % S).cuda()
    kb.kvattn_rope_append_rowscale(None, x[:, :n_kv], x[:, n_kv:], None, slots, *pools, *rows, rope_base=0.0)
    k, v = kb.kvattn_gather_rowscale(*pools, *rows, slots)
    q = normal(1, n_q, d, seed=2)
    lens = torch.tensor([N], dtype=torch.int32, device="cuda")
    out, lse = kb.kvattn_gqa_decode_rowscale(q, *pools, *rows, lens, 0.09, block_table=pages.to(torch.int32)[None].cuda())
    torch.cuda.synchronize()
    for got, new in ((k, x[:, :n_kv]), (v, x[:, n_kv:])):
        ref = new.transpose(0, 1).double()
        err = (got.double() - ref).abs()
        # (a code's half step, 2^-10 of a 448th of the largest where codes are smallest, and bf16's)
        assert bool((err <= (2.0 ** -4 + 2.0 ** -8) * ref.abs() + 2.0 ** -10 / 448 * ref.abs().amax(-1, keepdim=True) * 1.01).all())
    at = slots.cpu()
    for j in (0, n_kv - 1):
        code = [p[pages.cuda(), j].cpu().view(torch.float8_e4m3fn).double().view(-1, d)[:N] for p in pools]
        sc = [r[pages.cuda(), j].cpu().double().view(-1)[:N] for r in rows]
        kk, vv = (c * s[:, None] for c, s in zip(code, sc))
        see = torch.ones((4, N), dtype=torch.bool)
        ref, rl, p = r64.attention(q[0, 4 * j:4 * j + 4].cpu(), kk, vv, see, 0.09)
        bo, bl = r64.bounds(q[0, 4 * j:4 * j + 4].cpu(), kk, code[1], sc[1], see, ref, p, 0.09)
        r64.assert_within(out[0, 4 * j:4 * j + 4], ref, bo, f"out {j}")
        r64.assert_within(lse[0, 4 * j:4 * j + 4], rl, bl + 2.0 ** -21 * rl.abs(), f"lse {j}")
    assert int(at.max()) * n_kv * d > 2 ** 32
    free = torch.ones((P,), dtype=torch.bool, device="cuda")
    free[pages.cuda()] = False
    for i in range(0, P, 5000):                            # every other page is as it was
        assert bool((pools[0][i:i + 5000][free[i:i + 5000]] == 0x7F).all())


def check_rows(q, k, v, out, lse, scale, what):
    """[r, d] rows against [T, d] keys and values on the GPU, in 64 bits."""
    see = torch.ones((q.shape[0], k.shape[0]), dtype=torch.bool)
    ref, rl, p = plain64.attention(q.cpu(), k.cpu(), v.cpu(), see, scale)
    slack = plain64.score_slack(q.cpu(), k.cpu(), scale, "bf16")
    plain64.assert_within(out, ref, plain64.out_bound(ref, p, v.cpu(), slack, "bf16"), f"out {what}")
    plain64.assert_within(lse, rl, slack + 2.0 ** -21 * rl.abs() + 2e-6, f"lse {what}")


def test_prefix_and_caches():
    """A prefix buffer of 2.3e9 elements (the last KV head begins past 2^31) and caches of 2.2e9, little of either
    in use."""
    n_kv, d, P_max, B, T, n_q = 8, 128, 2250000, 40, 54000, 16
    kp = torch.empty((n_kv, P_max, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    kc = torch.empty((B, n_kv, T, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    for t in (kp, vp, kc, vc):
        assert t.numel() > 2 ** 31
        t.fill_(float("nan"))
    P, lens = 3000, [i * 13 % 400 for i in range(B - 1)] + [20000]
    for i, t in enumerate((kp, vp)):
        t[:, :P] = normal(n_kv, P, d, seed=i)
    for b, n in enumerate(lens):
        kc[b, :, :n], vc[b, :, :n] = normal(n_kv, n, d, seed=10 + b), normal(n_kv, n, d, seed=100 + b)
    q = normal(B, 1, n_q, d, seed=3)
    plen, dlens = torch.tensor([P], dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    scale = 1 / math.sqrt(d)
    out, lse = kb.kvattn_gqa_decode_prefix(q, kp, vp, plen, kc, vc, dlens, scale)
    torch.cuda.synchronize()
    for b in (0, 1, 20, B - 1):
        for j in (0, 7):
            k, v = torch.cat((kp[j, :P], kc[b, j, :lens[b]])), torch.cat((vp[j, :P], vc[b, j, :lens[b]]))
            check_rows(q[b, 0, 2 * j:2 * j + 2], k, v, out[b, 0, 2 * j:2 * j + 2], lse[b, 0, 2 * j:2 * j + 2], scale, f"{b} {j}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_verification(dtype):
    """4096 sequences over 2.2e9 entries; a few are checked, the last among them."""
    B, L, V = 4096, 3, 135001
    p = torch.empty((B, L + 1, V), dtype=dtype, device="cuda").uniform_()
    q = torch.empty((B, L, V), dtype=dtype, device="cuda").uniform_()
    g = torch.Generator().manual_seed(1)
    drafts = torch.randint(0, V, (B, L), generator=g).to(torch.int32)
    ua, us = torch.rand((B, L), generator=g), torch.rand((B,), generator=g)
    assert p.numel() > 2 ** 31
    acc, tok = kb.kvattn_verify_drafts(p, q, drafts.cuda(), ua.cuda(), us.cuda())
    torch.cuda.synchronize()
    some = torch.tensor([0, 1, 2048, 3976, 3977, 4000, 4094, 4095])
    ra, rt = plain64.verify(p[some.cuda()].cpu(), q[some.cuda()].cpu(), drafts[some], None, ua[some], us[some])
    assert torch.equal(acc.cpu()[some], ra) and torch.equal(tok.cpu()[some], rt)
    assert bool((tok.cpu()[torch.arange(B), acc.cpu().long()] >= 0).all())
