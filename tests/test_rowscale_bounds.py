"""The row-scaled decode's error bound (tests/rowscale64.py) on the CPU: the kernel's own arithmetic lies within it,
coarser weights or value scales do not."""
import pytest
import torch

from tests import rowscale64 as r64


def worst(data, **kw):
    q, kcode, ks, vcode, vs = data
    k, v = kcode.double() * ks.double()[:, None], vcode.double() * vs.double()[:, None]
    see = torch.ones((q.shape[0], k.shape[0]), dtype=torch.bool)
    ref, _, p = r64.attention(q, k, v, see, 0.1)
    got = r64.emulate(q, kcode, ks, vcode, vs, 0.1, **kw).double()
    return float(((got - ref).abs() / r64.bounds(q, k, vcode, vs, see, ref, p, 0.1)[0]).max())


def random_rows(T, seed):
    g = torch.Generator().manual_seed(seed)
    code = lambda: torch.randn((T, 128), generator=g).mul(100).clamp(-448, 448).to(torch.float8_e4m3fn).float()  # noqa: E731
    scale = lambda: torch.exp(torch.randn((T,), generator=g)) / 448  # noqa: E731
    return torch.randn((8, 128), generator=g).to(torch.bfloat16), code(), scale(), code(), scale()


@pytest.mark.parametrize("T", [2, 40, 900])
def test_f16_weights_lie_within(T):
    assert worst(random_rows(T, T)) <= 1.0
    assert worst(r64.cancelling(T)) <= 0.5


@pytest.mark.parametrize("kw", [dict(weight_type=torch.bfloat16), dict(vs_type=torch.bfloat16)], ids=["weights", "value scales"])
@pytest.mark.parametrize("n", [1, 16, 150])
def test_bf16_does_not(n, kw):
    assert worst(r64.cancelling(n), **kw) > 2.0
