"""GPU tests of the log-sum-exp of rows with a NaN score: NaN wherever the unit is cut, as where it is not (B200)."""
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


@pytest.mark.parametrize("forced", [None, (1, 1), (7, 1), (40, 1)])
@pytest.mark.parametrize("what", ["query", "key scale", "key code"])
def test_rowscale(what, forced):
    lens = [1500, 300]
    q, x = queries(2, 1, 16, 1), caches(2, 2, 1503, 2)
    if what == "query":
        q[0, 0, 3, 17] = float("nan")
    elif what == "key scale":
        x[1][0, 1, 700] = float("nan")
    else:
        x[0][0, 1, 1, 3] = float("nan")
    out, lse = run(q, x, lens, 0.09, S=128, forced=forced)
    assert int(torch.isnan(lse).sum()) == (1 if what == "query" else 8)
    assert bool((torch.isnan(lse)[..., None] == torch.isnan(out.float())).all())
