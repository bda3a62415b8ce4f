"""GPU tests of the row-scaled decode at the error bound of its f16 products, tests/rowscale64.py (B200)."""
import math

import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from tests import plain64
from tests import rowscale64 as r64
from tests.test_gpu_rowscale import DECODE, paginate, row_cache

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


def caches(B, n_kv, T, seed):
    """[k codes, k scales, v codes, v scales] of [B, n_kv, T, 128] rows, codes as floats (CPU)."""
    g = torch.Generator().manual_seed(seed)
    (kc, ks), (vc, vs) = row_cache((B, n_kv, T, 128), g), row_cache((B, n_kv, T, 128), g)
    return [kc.float(), ks, vc.float(), vs]


def run(q, x, lens, scale, window=0, S=0, forced=None):
    """Decodes q [B, L, n_q, 128] over caches x (rows past the lengths hold NaN), in pages of S rows or contiguous,
    and compares with the definition.  Returns (out, lse) on the CPU."""
    B, L, n_q, _ = q.shape
    kc, ks, vc, vs = x
    n_kv = kc.shape[1]
    code = lambda c: c.to(torch.float8_e4m3fn)  # noqa: E731
    if S:
        (kp, vp), (kr, vr), table = paginate((code(kc), code(vc)), (ks, vs), lens, S, torch.Generator().manual_seed(1))
        table = table.cuda()
    else:
        kp, vp, kr, vr, table = code(kc).view(torch.uint8), code(vc).view(torch.uint8), ks.clone(), vs.clone(), None
        for b, n in enumerate(lens):
            kp[b, :, n:], vp[b, :, n:] = 0x7F, 0x7F
            kr[b, :, n:], vr[b, :, n:] = float("nan"), float("nan")
    if forced:
        kb.kvattn_debug_set_workers(*forced)
    out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:-1], -7.0, device="cuda")
    kb.kvattn_gqa_decode_rowscale(q.cuda(), kp.cuda(), vp.cuda(), kr.cuda(), vr.cuda(),
                                  torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, block_table=table, window=window,
                                  out=out, lse=lse)
    torch.cuda.synchronize()
    out, lse = out.cpu(), lse.cpu()
    g = n_q // n_kv
    for b, n in enumerate(lens):
        see = plain64.visible(n, L, n, window).repeat_interleave(g, 0)
        for j in range(n_kv):
            k = kc[b, j, :n].double() * ks[b, j, :n, None].double()
            v = vc[b, j, :n].double() * vs[b, j, :n, None].double()
            rows = q[b, :, j * g:(j + 1) * g].reshape(L * g, 128)
            ref, rl, p = r64.attention(rows, k, v, see, scale)
            bo, bl = r64.bounds(rows, k, vc[b, j, :n], vs[b, j, :n], see, torch.nan_to_num(ref), p, scale)
            r64.assert_within(out[b, :, j * g:(j + 1) * g].reshape(L * g, 128), ref, bo, f"out {b} {j}")
            r64.assert_within(lse[b, :, j * g:(j + 1) * g].reshape(L * g), rl, bl + 2.0 ** -21 * torch.nan_to_num(rl, neginf=0.0).abs(),
                              f"lse {b} {j}")
    return out, lse


def queries(B, L, n_q, seed):
    return torch.randn((B, L, n_q, 128), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("n_q,n_kv,L,S,lens", DECODE, ids=[f"g{c[0] // c[1]}_L{c[2]}_s{c[3]}" for c in DECODE])
def test_random_rows(n_q, n_kv, L, S, lens):
    run(queries(len(lens), L, n_q, 1), caches(len(lens), n_kv, max(lens) + 3, 2), lens, 1 / math.sqrt(128.0), S=S)


@pytest.mark.parametrize("forced", [None, (3, 1)])
@pytest.mark.parametrize("n", [1, 40, 300])
@pytest.mark.parametrize("L", [1, 2, 4])
def test_values_that_cancel(n, L, forced):
    """Weights or value scales of fewer bits than f16's show here (tests/test_rowscale_bounds.py)."""
    q, kc, ks, vc, vs = r64.cancelling(n)
    T = len(vs)
    x = [kc[None, None], ks[None, None], vc[None, None], vs[None, None]]
    run(q[:1].expand(1, L, 8, 128).contiguous(), x, [T], 0.1, forced=forced)
