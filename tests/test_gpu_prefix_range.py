"""GPU tests of the shared-prefix decode over the range of values its documentation gives (B200)."""
import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from tests.test_gpu_prefix import check, inputs, run

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(autouse=True)
def _flags():
    kb.kvattn_clear_device_flags()
    yield
    kb.kvattn_debug_set_workers(0, 0)
    assert kb.kvattn_read_device_flags() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nats", [4.0, 7.0, 12.0, 18.0, 21.0, 34.0, 43.0, 60.0])
@pytest.mark.parametrize("exponent", [-80, 80])
@pytest.mark.parametrize("B", [20, 40])
def test_large_values_behind_growing_scores(d, nats, exponent, B):
    """Values of 2^80 in size, and scores that rise by up to 60 nats (2^86) from one tile to the next: the weights
    before the maximum moves must not carry the sums out of range.  (One row tile: every other tile is a group's
    own; two: every tile is both groups'.)"""
    x = inputs(B, 1, 8, 2, d, 600, [260] * B, seed=int(nats), key_scale=0.05)
    unit = torch.zeros(d)
    unit[3] = 1.0
    x["q"][..., 3] = 8.0
    for t, n in (("kp", 600), ("ks", 260)):
        step = (torch.arange(n) // 128).float()             # tiles since the first
        x[t][..., :n, :] += (step * nats / 8.0)[:, None] * unit
        x[t] = x[t].to(torch.bfloat16)
    for t in ("vp", "vs"):
        x[t] = (x[t].double() * 2.0 ** exponent).to(torch.bfloat16)
    kb.kvattn_debug_set_workers(3, 1)                       # several tiles a worker
    check(x, *run(x, 1.0), 1.0)
