"""GPU tests of the decodes at the limits that their documentation gives: the largest batches, the most new tokens, the
widest groups (B200)."""
import math

import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from tests.test_gpu_prefix import check, inputs
from tests.test_gpu_prefix import run as run_prefix
from tests.test_gpu_rowscale_bounds import caches, queries, run

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(autouse=True)
def _flags():
    kb.kvattn_clear_device_flags()
    yield
    assert kb.kvattn_read_device_flags() == 0


@pytest.mark.parametrize("B,L,n_q,lens", [
    (4096, 1, 2, [i * 7 % 150 for i in range(4096)]),      # the largest batch
    (64, 64, 1, [i * 5 for i in range(64)]),               # 64 rows a unit
    (32, 128, 1, [i * 9 for i in range(32)]),              # more than a unit's rows: one new token a sequence each
    (1, 4096, 1, [4100]),                                  # a prompt of the most new tokens
    (1, 4096, 1, [700]),                                   # ... most of which see nothing
], ids=["B4096", "L64", "L128", "L4096", "L4096 short"])
@pytest.mark.parametrize("window", [0, 40])
def test_rowscale(B, L, n_q, lens, window):
    run(queries(B, L, n_q, 1), caches(B, 1, max(lens) + 1, 2), lens, 0.09, window=window)


@pytest.mark.parametrize("B,L,n_q,n_kv,d,P,lens", [
    (4096, 1, 2, 1, 64, 300, [i * 7 % 40 for i in range(4096)]),
    (32, 128, 1, 1, 128, 200, [i * 9 for i in range(32)]),
    (2048, 2, 64, 1, 64, 140, [i % 4 for i in range(2048)]),
    (1, 1, 1, 1, 128, 40000, [30000]),
], ids=["B4096", "L128", "rows128", "one row"])
def test_prefix(B, L, n_q, n_kv, d, P, lens):
    x = inputs(B, L, n_q, n_kv, d, P, lens, seed=B)
    scale = 1 / math.sqrt(d)
    check(x, *run_prefix(x, scale), scale)
