"""GPU tests of strided operands that lie between one another: rotated queries next to the keys and values of a fused
projection, rows read back into alternating heads of one buffer (B200)."""
import pytest
import torch

from mla_kv_cache_b200 import binding as kb

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

N, NQ, NKV, D, S, P = 50, 6, 2, 128, 16, 4


def pools():
    z = lambda *s, **k: torch.zeros((P, NKV, S, *s), device="cuda", **k)  # noqa: E731
    return z(D, dtype=torch.uint8), z(D, dtype=torch.uint8), z(), z()


def test_rotated_queries_into_the_projection():
    """In place, and into a part of the rows that nothing else uses: as into a buffer of their own."""
    g = torch.Generator().manual_seed(1)
    heads = 2 * NQ + 2 * NKV
    x = torch.randn((N, heads, D), generator=g).to(torch.bfloat16)
    pos, slots = torch.arange(N, dtype=torch.int32, device="cuda"), torch.arange(N, device="cuda")
    got = []
    for where in ("own", "in place", "beside"):
        dev = x.cuda()
        q, k, v, rest = dev.split((NQ, NKV, NKV, NQ), 1)
        out = {"own": torch.empty((N, NQ, D), dtype=torch.bfloat16, device="cuda"), "in place": q, "beside": rest}[where]
        pool = pools()
        kb.kvattn_rope_append_rowscale(q, k, v, pos, slots, *pool, q_out=out)
        torch.cuda.synchronize()
        assert torch.equal(dev[:, NQ:NQ + 2 * NKV].cpu(), x[:, NQ:NQ + 2 * NKV])
        assert where == "in place" or torch.equal(q.cpu(), x[:, :NQ])
        assert where == "beside" or torch.equal(rest.cpu(), x[:, NQ + 2 * NKV:])
        got.append([out.cpu(), *(t.cpu() for t in pool)])
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    with pytest.raises(kb.KvattnError):          # one head too far: the last query head is the first key head
        dev = x.cuda()
        kb.kvattn_rope_append_rowscale(dev[:, :NQ], dev[:, NQ - 1:NQ - 1 + NKV], dev[:, NQ + NKV:NQ + 2 * NKV], pos, slots, *pools())


@pytest.mark.parametrize("n_kv", [1, 2, 5])
def test_read_back_into_alternating_heads(n_kv):
    g = torch.Generator().manual_seed(n_kv)
    codes = torch.randint(0, 0x70, (2, P, n_kv, S, D), generator=g).to(torch.uint8).cuda()
    scales = torch.rand((2, P, n_kv, S), generator=g).cuda()
    slots = torch.randperm(P * S, generator=g)[:N].cuda()
    k, v = kb.kvattn_gather_rowscale(codes[0], codes[1], scales[0], scales[1], slots)
    both = torch.full((n_kv, 2, N, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    kb.kvattn_gather_rowscale(codes[0], codes[1], scales[0], scales[1], slots, k_out=both[:, 0], v_out=both[:, 1])
    torch.cuda.synchronize()
    assert torch.equal(both[:, 0], k) and torch.equal(both[:, 1], v)
