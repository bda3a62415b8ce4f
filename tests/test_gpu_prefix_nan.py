"""GPU tests of NaN within what a shared-prefix decode attends to: it reaches the rows and elements that it belongs to,
and no others, however the prefix and the suffixes are cut (B200)."""
import math

import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from tests import plain64
from tests import rowscale64 as r64
from tests.test_gpu_prefix import inputs, run

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(autouse=True)
def _flags():
    kb.kvattn_clear_device_flags()
    yield
    kb.kvattn_debug_set_workers(0, 0)
    assert kb.kvattn_read_device_flags() == 0


def check(x, out, lse, scale):
    B, L, n_q, d = x["q"].shape
    n_kv, P = x["kp"].shape[0], x["P"]
    g = n_q // n_kv
    for b, n in enumerate(x["lens"]):
        see = torch.cat((torch.ones((L, P), dtype=torch.bool), plain64.visible(n, L, n)), 1).repeat_interleave(g, 0)
        for j in range(n_kv):
            k, v = torch.cat((x["kp"][j, :P], x["ks"][b, j, :n])), torch.cat((x["vp"][j, :P], x["vs"][b, j, :n]))
            rows = x["q"][b, :, j * g:(j + 1) * g].reshape(L * g, d)
            ref, rl, p = r64.attention(rows, k, v, see, scale)
            num = torch.nan_to_num
            slack = plain64.score_slack(num(rows), num(k), scale, "bf16")
            r64.assert_within(out[b, :, j * g:(j + 1) * g].reshape(L * g, d), ref,
                              plain64.out_bound(num(ref), num(p), num(v), slack, "bf16"), f"out {b} {j}")
            r64.assert_within(lse[b, :, j * g:(j + 1) * g].reshape(L * g), rl, slack + 2.0 ** -21 * num(rl, neginf=0.0).abs() + 2e-6,
                              f"lse {b} {j}")


@pytest.mark.parametrize("forced", [None, (1, 1), (7, 1)])
@pytest.mark.parametrize("what", ["query", "prefix key", "own key", "prefix value", "own value"])
@pytest.mark.parametrize("B,n_q,n_kv,d", [(24, 24, 2, 128), (30, 16, 2, 64)])
def test_nan(B, n_q, n_kv, d, what, forced):
    x = inputs(B, 1, n_q, n_kv, d, 700, [(i * 53) % 300 + 1 for i in range(B)], seed=4)
    if what == "query":
        x["q"][3, 0, 5, 7] = float("nan")
        x["q"][4, 0, n_q - 1] = float("nan")
    elif what == "prefix key":
        x["kp"][1, 600, 9] = float("nan")
    elif what == "own key":
        x["ks"][6, 0, 0, 9] = float("nan")
        x["ks"][7, 1, x["lens"][7] - 1] = float("nan")
    elif what == "prefix value":
        x["vp"][0, 699, 11] = float("nan")
    else:
        x["vs"][6, 0, 0, 9] = float("nan")
        x["vs"][7, 1, x["lens"][7] - 1, 10:20] = float("nan")
    if forced:
        kb.kvattn_debug_set_workers(*forced)
    scale = 1 / math.sqrt(d)
    check(x, *run(x, scale), scale)
