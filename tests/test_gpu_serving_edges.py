"""GPU tests of the serving operators at the edges of what their documentation allows (B200)."""
import math

import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from tests import plain64
from tests.test_gpu_prefix import check, inputs, paged, run
from tests.test_gpu_rowscale import paginate, row_cache, run_decode

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(autouse=True)
def _flags():
    kb.kvattn_debug_set_workers(0, 0)
    kb.kvattn_clear_device_flags()
    yield
    assert kb.kvattn_read_device_flags() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P,lens", [(1, [1]), (1, [0]), (127, [1, 1]), (129, [2, 129])])
def test_prefix_smallest_capacities(d, P, lens):
    """Caches of no more rows than their lengths, down to one."""
    x = inputs(len(lens), 1, 4, 2, d, P, lens, seed=P, extra=0)
    check(x, *run(x, 0.2), 0.2)


@pytest.mark.parametrize("d", [64, 128])
def test_prefix_scores_that_jump(d):
    """Scores that grow by hundreds from one tile to the next (log2 units): the maximum moves within a step."""
    x = inputs(36, 1, 16, 2, d, 900, [150] * 36, seed=3, key_scale=0.02)
    x["kp"][:, 300:] *= 2000
    x["ks"][:, :, 130:] *= 40000
    scale = 1 / math.sqrt(d)
    check(x, *run(x, scale), scale)


def test_prefix_calls_agree():
    """Suffixes and a prefix that stream from memory, called again and again: every call gives the same bits."""
    g = torch.Generator(device="cuda").manual_seed(5)
    B, n_q, n_kv, d, P, T = 8, 32, 8, 128, 20000, 8192
    normal = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, kp, vp, ks, vs = normal(B, 1, n_q, d), normal(n_kv, P, d), normal(n_kv, P, d), normal(B, n_kv, T, d), normal(B, n_kv, T, d)
    lens = torch.tensor([8000, 7777, 1, 5000, 8192, 6001, 130, 4095], dtype=torch.int32, device="cuda")
    plen = torch.tensor([P], dtype=torch.int32, device="cuda")
    call = lambda: kb.kvattn_gqa_decode_prefix(q, kp, vp, plen, ks, vs, lens, 0.09)  # noqa: E731
    out, lse = call()
    for _ in range(60):
        o, l = call()
        assert torch.equal(o, out) and torch.equal(l, lse)
    for b in (0, 2):
        n = int(lens[b])
        k, v = torch.cat((kp[1], ks[b, 1, :n])).cpu(), torch.cat((vp[1], vs[b, 1, :n])).cpu()
        ref, rl, p = plain64.attention(q[b, 0, 4:8].cpu(), k, v, torch.ones((4, P + n), dtype=torch.bool), 0.09)
        slack = plain64.score_slack(q[b, 0, 4:8].cpu(), k, 0.09, "bf16")
        plain64.assert_within(out[b, 0, 4:8], ref, plain64.out_bound(ref, p, v, slack, "bf16"), f"out {b}")
        plain64.assert_within(lse[b, 0, 4:8], rl, slack + 2.0 ** -21 * rl.abs() + 2e-6, f"lse {b}")


BAD = [-1, 1 << 20, 1 << 29, -(1 << 31), (1 << 31) - 1]     # (1 << 29 times 8 heads is 0 in 32 bits)


@pytest.mark.parametrize("bad", BAD)
def test_prefix_pages_outside_the_pool(bad):
    """They read as zeros: a score of 0 and no value."""
    x = inputs(3, 1, 16, 8, 128, 400, [200, 300, 90], seed=14)
    kp, vp, ptab, tab = paged(x, 128, torch.Generator().manual_seed(2))
    ptab[1], tab[1, 1] = bad, bad
    for t in ("kp", "vp"):
        x[t][:, 128:256] = 0
    for t in ("ks", "vs"):
        x[t][1, :, 128:256] = 0
    lens, plen = torch.tensor(x["lens"], dtype=torch.int32, device="cuda"), torch.tensor([400], dtype=torch.int32, device="cuda")
    out, lse = kb.kvattn_gqa_decode_prefix_paged(x["q"].cuda(), kp.cuda(), vp.cuda(), ptab.cuda(), plen, tab.cuda(), lens, 0.1)
    torch.cuda.synchronize()
    check(x, out, lse, 0.1)


@pytest.mark.parametrize("bad", BAD)
def test_rowscale_pages_outside_the_pool(bad):
    g = torch.Generator().manual_seed(6)
    lens, n_kv = [300, 140], 8
    kc, ks = row_cache((2, n_kv, 300, 128), g)
    vc, vs = row_cache((2, n_kv, 300, 128), g)
    (kp, vp), (kr, vr), table = paginate((kc, vc), (ks, vs), lens, 128, g)
    table[0, 1] = bad
    q = torch.randn((2, 1, 16, 128), generator=g).to(torch.bfloat16)
    out, lse = kb.kvattn_gqa_decode_rowscale(q.cuda(), kp.cuda(), vp.cuda(), kr.cuda(), vr.cuda(),
                                             torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.1, block_table=table.cuda())
    torch.cuda.synchronize()
    for j in range(n_kv):
        k = kc[0, j].double() * ks[0, j, :, None].double()
        v = vc[0, j].double() * vs[0, j, :, None].double()
        k[128:256], v[128:256] = 0, 0
        rows = q[0, 0, 2 * j:2 * j + 2]
        ref, rl, p = plain64.attention(rows, k, v, torch.ones((2, 300), dtype=torch.bool), 0.1)
        slack = plain64.score_slack(rows, k, 0.1, "e4m3")
        plain64.assert_within(out[0, 0, 2 * j:2 * j + 2], ref, plain64.out_bound(ref, p, v, slack, "e4m3"), f"out {j}")
        plain64.assert_within(lse[0, 0, 2 * j:2 * j + 2], rl, slack + 2.0 ** -21 * rl.abs() + 2e-6, f"lse {j}")


@pytest.mark.parametrize("S", [0, 128])
@pytest.mark.parametrize("n_q,n_kv,L,window", [(64, 2, 3, 100), (16, 4, 4, 77), (8, 8, 1, 130), (48, 1, 1, 1)])
def test_rowscale_windows(n_q, n_kv, L, window, S):
    """Windows over both kinds of cache; the first case runs as a virtual batch."""
    run_decode(4, L, n_q, n_kv, [400, 2, 129, 0], S, seed=window, window=window)


def test_rowscale_largest_batch_of_short_sequences():
    run_decode(300, 1, 4, 2, [i % 5 for i in range(300)], 0, seed=8)


def test_launches_are_counted():
    def count(call):
        before = kb.kvattn_kernel_launches()
        call()
        torch.cuda.synchronize()
        return kb.kvattn_kernel_launches() - before

    x = inputs(3, 1, 8, 2, 128, 200, [5, 0, 60], seed=10)
    assert count(lambda: run(x, 0.1)) == 2
    B = 641
    x = inputs(B, 1, 2, 1, 64, 30, [i % 3 for i in range(B)], seed=11)
    assert count(lambda: run(x, 0.1)) == 3
    p = torch.rand((2, 1, 50), device="cuda")
    u = torch.rand((2,), device="cuda")
    assert count(lambda: kb.kvattn_verify_drafts(p, None, None, None, u)) == 1
