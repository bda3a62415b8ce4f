"""GPU tests of decode over a shared prefix against a plain 64-bit form (B200).  Cache rows past every
length hold NaN, so a read of one into a result shows."""
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


def inputs(B, L, n_q, n_kv, d, P, lens, seed, extra=5, key_scale=2.0):
    g = torch.Generator().manual_seed(seed)
    T = max(max(lens), 1) + extra
    normal = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    x = {"q": normal(B, L, n_q, d), "kp": normal(n_kv, P + extra, d) * key_scale, "vp": normal(n_kv, P + extra, d),
         "ks": normal(B, n_kv, T, d) * key_scale, "vs": normal(B, n_kv, T, d), "lens": lens, "P": P}
    for t in ("kp", "vp"):
        x[t][:, P:] = float("nan")
    for b, n in enumerate(lens):
        x["ks"][b, :, n:] = float("nan")
        x["vs"][b, :, n:] = float("nan")
    return x


def check(x, out, lse, scale):
    B, L, n_q, d = x["q"].shape
    n_kv = x["kp"].shape[0]
    g, P = n_q // n_kv, x["P"]
    for b, n in enumerate(x["lens"]):
        see = torch.cat((torch.ones((L, P), dtype=torch.bool), plain64.visible(n, L, n)), 1).repeat_interleave(g, 0)
        for j in range(n_kv):
            k = torch.cat((x["kp"][j, :P], x["ks"][b, j, :n])).double()
            v = torch.cat((x["vp"][j, :P], x["vs"][b, j, :n])).double()
            rows = x["q"][b, :, j * g:(j + 1) * g].reshape(L * g, d)
            ref, rl, p = plain64.attention(rows, k, v, see, scale)
            slack = plain64.score_slack(rows, k, scale, "bf16")
            o = out[b, :, j * g:(j + 1) * g].reshape(L * g, d)
            l = lse[b, :, j * g:(j + 1) * g].reshape(L * g)
            plain64.assert_within(o, ref, plain64.out_bound(ref, p, v, slack, "bf16"), f"out {b} {j}")
            plain64.assert_within(l, rl, slack + 2.0 ** -21 * rl.abs() + 2e-6, f"lse {b} {j}")


def run(x, scale, **kw):
    dev = {k: v.cuda() for k, v in x.items() if torch.is_tensor(v)}
    lens = torch.tensor(x["lens"], dtype=torch.int32, device="cuda")
    plen = torch.tensor([x["P"]], dtype=torch.int32, device="cuda")
    out = torch.full(x["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(x["q"].shape[:-1], float("nan"), device="cuda")
    kb.kvattn_gqa_decode_prefix(dev["q"], dev["kp"], dev["vp"], plen, dev["ks"], dev["vs"], lens, scale, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


CASES = [
    # B, L, n_q, n_kv, d, P, lens
    (1, 1, 8, 8, 128, 1, [1]),
    (3, 1, 8, 2, 128, 300, [0, 1, 130]),
    (2, 1, 8, 2, 64, 128, [128, 129]),
    (5, 1, 32, 8, 128, 1000, [1, 127, 128, 300, 0]),
    (40, 1, 16, 2, 128, 777, list(range(0, 80, 2))),          # 320 rows a KV head: row tiles 2 + 1
    (70, 1, 4, 1, 64, 515, [i % 9 for i in range(70)]),       # 280 rows
    (64, 1, 32, 4, 128, 2000, [i * 7 % 200 for i in range(64)]),
    (9, 5, 12, 4, 128, 400, [0, 1, 4, 5, 6, 127, 128, 130, 260]),   # drafts; groups of 3
    (7, 2, 64, 1, 128, 260, [1, 2, 3, 129, 0, 64, 200]),      # 64 heads on one KV head, 2 tokens: 128 rows a sequence
    (4, 4, 28, 4, 64, 129, [4, 3, 200, 128]),                 # groups of 7
    (3, 1, 100, 1, 64, 400, [10, 0, 300]),                    # 100 heads on one KV head
    (2, 1, 128, 1, 128, 130, [5, 140]),
]


@pytest.mark.parametrize("case", CASES, ids=[f"B{c[0]}_L{c[1]}_g{c[2] // c[3]}_d{c[4]}_P{c[5]}" for c in CASES])
def test_prefix(case):
    B, L, n_q, n_kv, d, P, lens = case
    x = inputs(B, L, n_q, n_kv, d, P, lens, seed=P)
    scale = 1 / math.sqrt(d)
    check(x, *run(x, scale), scale)


@pytest.mark.parametrize("P,lens", [(0, [3, 0, 200]), (0, [0, 0, 0]), (64, [0, 0, 0])])
def test_empty_parts(P, lens):
    """No prefix, no own tokens, neither: a row with nothing to attend to gives 0 and -inf."""
    x = inputs(3, 1, 8, 2, 128, P, lens, seed=5)
    out, lse = run(x, 0.1)
    check(x, out, lse, 0.1)


@pytest.mark.parametrize("forced", [(1, 1), (5, 1), (61, 1), (400, 1)])
def test_forced_splits(forced):
    kb.kvattn_debug_set_workers(*forced)
    x = inputs(40, 1, 16, 2, 128, 1500, [i * 5 for i in range(40)], seed=6)
    scale = 1 / math.sqrt(128.0)
    check(x, *run(x, scale), scale)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_score_scales(scale):
    x = inputs(17, 1, 16, 2, 128, 500, [i * 11 for i in range(17)], seed=7, key_scale=1.0)
    check(x, *run(x, scale), scale)


def test_growing_scores():
    """Keys that grow along the prefix move every row's maximum again and again (the rescaling path)."""
    x = inputs(40, 1, 16, 2, 128, 1400, [100] * 40, seed=8)
    x["kp"] *= torch.linspace(0.1, 12, x["kp"].shape[1]).to(torch.bfloat16)[None, :, None]
    scale = 1 / math.sqrt(128.0)
    check(x, *run(x, scale), scale)


def test_large_batch():
    """More sequences than the kernel keeps lengths of in shared memory."""
    B = 700
    x = inputs(B, 1, 4, 2, 64, 200, [i % 7 for i in range(B)], seed=9)
    check(x, *run(x, 0.125), 0.125)


def test_three_dim_query_and_own_workspace():
    x = inputs(3, 1, 8, 2, 128, 200, [5, 0, 60], seed=10)
    dev = {k: v.cuda() for k, v in x.items() if torch.is_tensor(v)}
    lens, plen = torch.tensor(x["lens"], dtype=torch.int32, device="cuda"), torch.tensor([200], dtype=torch.int32, device="cuda")
    need = kb.kvattn_gqa_decode_prefix_workspace(x["kp"].shape[1], x["ks"].shape[2], 3, 1, 8, 2, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")          # NaN wherever it is read unwritten
    out, lse = kb.kvattn_gqa_decode_prefix(dev["q"][:, 0].contiguous(), dev["kp"], dev["vp"], plen, dev["ks"], dev["vs"],
                                           lens, 0.1, workspace=ws)
    torch.cuda.synchronize()
    check(x, out[:, None], lse[:, None], 0.1)
    with pytest.raises(kb.KvattnError):
        kb.kvattn_gqa_decode_prefix(dev["q"], dev["kp"], dev["vp"], plen, dev["ks"], dev["vs"], lens, 0.1, workspace=ws[:-1])


def paged(x, S, g):
    """Prefix and own rows in one pool of shuffled pages, the rest of which holds NaN."""
    n_kv, d = x["kp"].shape[0], x["kp"].shape[2]
    B, P = len(x["lens"]), x["P"]
    np_ = (P + S - 1) // S
    used = [(n + S - 1) // S for n in x["lens"]]
    N = np_ + sum(used) + 2
    perm = torch.randperm(N, generator=g).tolist()
    kp = torch.full((N, n_kv, S, d), float("nan"), dtype=torch.bfloat16)
    vp = kp.clone()
    ptab = torch.full((np_ + 1,), 1 << 20, dtype=torch.int32)
    tab = torch.full((B, max(max(used), 1) + 1), -3, dtype=torch.int32)

    def put(k, v, n, i):
        page = perm.pop()
        m = min(S, n - i * S)
        kp[page, :, :m], vp[page, :, :m] = k[:, i * S:i * S + m], v[:, i * S:i * S + m]
        return page

    for i in range(np_):
        ptab[i] = put(x["kp"], x["vp"], P, i)
    for b in range(B):
        for i in range(used[b]):
            tab[b, i] = put(x["ks"][b], x["vs"][b], x["lens"][b], i)
    return kp, vp, ptab, tab


@pytest.mark.parametrize("S,d", [(128, 128), (256, 64)])
def test_paged_equals_contiguous(S, d):
    x = inputs(20, 2, 16, 4, d, 700, [(i * 37) % 300 for i in range(20)], seed=12)
    kp, vp, ptab, tab = paged(x, S, torch.Generator().manual_seed(1))
    lens, plen = torch.tensor(x["lens"], dtype=torch.int32, device="cuda"), torch.tensor([700], dtype=torch.int32, device="cuda")
    out, lse = kb.kvattn_gqa_decode_prefix_paged(x["q"].cuda(), kp.cuda(), vp.cuda(), ptab.cuda(), plen, tab.cuda(), lens, 0.1)
    torch.cuda.synchronize()
    check(x, out, lse, 0.1)


def test_lengths_out_of_range_are_clamped():
    x = inputs(2, 1, 8, 2, 128, 300, [40, 50], seed=13, extra=0)
    lens = torch.tensor([1 << 30, -4], dtype=torch.int32, device="cuda")
    plen = torch.tensor([1 << 30], dtype=torch.int32, device="cuda")
    dev = {k: torch.nan_to_num(v).cuda() for k, v in x.items() if torch.is_tensor(v)}
    out, lse = kb.kvattn_gqa_decode_prefix(dev["q"], dev["kp"], dev["vp"], plen, dev["ks"], dev["vs"], lens, 0.1)
    torch.cuda.synchronize()
    x = {**x, "ks": torch.nan_to_num(x["ks"]), "vs": torch.nan_to_num(x["vs"]), "lens": [50, 0]}
    check(x, out, lse, 0.1)


def test_two_streams_at_once():
    """Calls on two streams share nothing: each has its own workspace."""
    xs = [inputs(40, 1, 16, 2, 128, 1500, [50 + i for i in range(40)], seed=s) for s in (20, 21)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    dev = [{k: v.cuda() for k, v in x.items() if torch.is_tensor(v)} for x in xs]
    lens = [torch.tensor(x["lens"], dtype=torch.int32, device="cuda") for x in xs]
    plen = torch.tensor([1500], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(6):
        for i in range(2):
            got[i] = kb.kvattn_gqa_decode_prefix(dev[i]["q"], dev[i]["kp"], dev[i]["vp"], plen, dev[i]["ks"], dev[i]["vs"],
                                                 lens[i], 0.1, stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        check(xs[i], *got[i], 0.1)
