"""GPU tests of the serving operators' binding: numbers of other types than Python's, windows past 32 bits, arguments
that are no tensors (B200)."""
import numpy as np
import pytest
import torch

from mla_kv_cache_b200 import binding as kb

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def test_numpy_numbers_and_long_windows():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((40, 4, 128), generator=g).to(torch.bfloat16).cuda()
    pos, slots = torch.arange(40, dtype=torch.int32, device="cuda"), torch.arange(40, device="cuda")
    pools = []
    for base in (np.float32(10000.0), 10000.0):
        pool = (torch.zeros((1, 1, 128, 128), dtype=torch.uint8, device="cuda"), torch.zeros((1, 1, 128, 128), dtype=torch.uint8, device="cuda"),
                torch.zeros((1, 1, 128), device="cuda"), torch.zeros((1, 1, 128), device="cuda"))
        kb.kvattn_rope_append_rowscale(None, x[:, :1], x[:, 1:2], pos, slots, *pool, rope_base=base)
        pools.append(pool)
    assert all(torch.equal(a, b) for a, b in zip(*pools))
    lens, table = torch.tensor([40], dtype=torch.int32, device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    got = [kb.kvattn_gqa_decode_rowscale(x[:1], *pools[0], lens, scale, block_table=table, window=w)
           for scale, w in ((0.125, 1000), (np.float32(0.125), np.int64(1000)), (np.float64(0.125), 2 ** 32 + 5), (0.125, 2 ** 31))]
    k, v = kb.kvattn_gather_rowscale(*pools[0], slots)
    own = torch.zeros((1, 1, 8, 128), dtype=torch.bfloat16, device="cuda")
    none = torch.zeros((1,), dtype=torch.int32, device="cuda")
    prefix = [kb.kvattn_gqa_decode_prefix(x[:1], k, v, lens, own, own, none, s) for s in (0.125, np.float32(0.125))]
    torch.cuda.synchronize()
    for a in got[1:]:
        assert torch.equal(a[0], got[0][0]) and torch.equal(a[1], got[0][1])
    assert torch.equal(prefix[0][0], prefix[1][0])
    with pytest.raises(TypeError):
        kb.kvattn_gqa_decode_rowscale(x[:1], *pools[0], [40], 0.125, block_table=table)
    with pytest.raises(TypeError):
        kb.kvattn_gqa_decode_prefix(x[:1], k, v, 40, own, own, none, 0.125)
