"""GPU tests of the row-scaled decode over the range of scales its documentation gives (B200)."""
import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from tests.test_gpu_rowscale_bounds import caches, queries, run

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


RANGE = 40


@pytest.mark.parametrize("k_exp,v_exp", [(RANGE, RANGE), (-RANGE, -RANGE), (RANGE, -RANGE), (-RANGE, RANGE)])
@pytest.mark.parametrize("L,n_q", [(1, 8), (3, 16), (1, 32)])
def test_all_rows_large_or_small(L, n_q, k_exp, v_exp):
    """Scales at either end (the query at the other end of the keys')."""
    lens = [300, 129, 1]
    x = caches(3, 1, 303, 1)
    x[1] *= 2.0 ** k_exp
    x[3] *= 2.0 ** v_exp
    q = (queries(3, L, n_q, 2).double() * 2.0 ** -k_exp).to(torch.bfloat16)
    run(q, x, lens, 0.09, S=128)


@pytest.mark.parametrize("forced", [None, (1, 1)])
@pytest.mark.parametrize("order", ["up", "down", "blocks", "one"])
@pytest.mark.parametrize("gap", [-12.0, -5.0, 0.0, 5.0])
def test_value_scales_from_end_to_end(gap, order, forced):
    """Value scales of 2^RANGE beside 2^-RANGE, the scores of the latter `gap` nats above: both keep their share of
    the weights' sum."""
    T = 640
    t = torch.arange(T)
    small = {"up": t < 300, "down": t >= 300, "blocks": t // 32 % 2 == 0, "one": t != 77}[order]
    x = caches(1, 1, T, 3)
    x[0], x[1] = torch.zeros_like(x[0]), torch.ones_like(x[1])
    x[0][..., 5] = torch.where(small, 1.0, 0.0)              # the score's two values
    x[2] = x[2].clamp(-16, 16)
    x[3] = torch.where(small, 2.0 ** -RANGE, 2.0 ** RANGE)[None, None].float()
    q = queries(1, 1, 8, 4) * 0
    q[..., 5] = gap * 8
    run(q, x, [T], 1 / 8, forced=forced)
