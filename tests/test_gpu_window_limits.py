"""GPU tests of windows up to the largest there is, over batches with sequences shorter than their new tokens: a
window no shorter than the cache is no window (B200)."""
import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from tests.test_gpu_rowscale import run_decode

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

MAX = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def _knobs():
    kb.kvattn_debug_set_workers(0, 0)
    kb.kvattn_clear_device_flags()
    yield
    kb.kvattn_debug_set_workers(0, 0)
    assert kb.kvattn_read_device_flags() == 0


@pytest.mark.parametrize("S", [0, 128])
@pytest.mark.parametrize("window", [MAX, MAX - 3, 5000])
@pytest.mark.parametrize("L,forced", [(1, None), (3, None), (5, (7, 1))])
def test_rowscale(S, window, L, forced):
    run_decode(4, L, 32, 8, [0, 1, 300, 4], S, seed=L, window=window, forced=forced)


@pytest.mark.parametrize("L", [1, 3, 5])
def test_multi_and_e4m3(L):
    """The older windowed calls share the work split: the same result as without a window."""
    g = torch.Generator().manual_seed(L)
    lens = torch.tensor([0, 1, 300, 4, 129], dtype=torch.int32, device="cuda")
    q = torch.randn((5, L, 32, 128), generator=g).to(torch.bfloat16).cuda()
    k, v = (torch.randn((5, 8, 320, 128), generator=g).cuda() for _ in range(2))
    for k, v, call in ((k.to(torch.bfloat16), v.to(torch.bfloat16), kb.kvattn_gqa_decode_multi),
                       (k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), None)):
        got = []
        for window in (5000, MAX):
            if call:
                got.append(call(q, k, v, lens, 0.1, window=window))
            else:
                got.append(kb.kvattn_gqa_decode_fp8(q, k, v, lens, 0.1, 1.0, 1.0, window=window))
        torch.cuda.synchronize()
        for a, b in zip(*got):
            assert torch.equal(a, b) and not bool(torch.isnan(a).any())
