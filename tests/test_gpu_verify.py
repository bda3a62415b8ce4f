"""GPU tests of draft verification: every accepted count and token equal to the plain 64-bit form (B200)."""
import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from tests import plain64

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def inputs(B, L, V, dtype, seed, point=False, near=0.5):
    g = torch.Generator().manual_seed(seed)
    logits = 2.5 * torch.randn((B, L + 1, V), generator=g)
    draft = logits[:, :L] + near * torch.randn((B, L, V), generator=g)
    q = torch.softmax(draft, -1)
    x = {"p": torch.softmax(logits, -1).to(dtype), "q": None if point else q.to(dtype)}
    x["tokens"] = (draft.argmax(-1) if point or not L else torch.multinomial(q.view(B * L, V), 1, generator=g).view(B, L)).to(torch.int32)
    x["lens"] = torch.randint(0, L + 1, (B,), generator=g).to(torch.int32)
    x["lens"][: (B + 1) // 2] = L
    x["ua"], x["us"] = torch.rand((B, L), generator=g), torch.rand((B,), generator=g)
    return x


def check(x, p=None, q=None, **kw):
    dev = {k: (v.cuda() if v is not None else None) for k, v in x.items()}
    p = dev["p"] if p is None else p
    q = dev["q"] if q is None else q
    acc, tok = kb.kvattn_verify_drafts(p, q, dev["tokens"], dev["ua"], dev["us"], draft_lens=dev["lens"], **kw)
    torch.cuda.synchronize()
    ra, rt = plain64.verify(x["p"], x["q"], x["tokens"], x["lens"], x["ua"], x["us"])
    assert torch.equal(acc.cpu(), ra) and torch.equal(tok.cpu(), rt)
    return ra, rt


CASES = [(1, 1, 1), (1, 8, 32000), (3, 4, 7), (64, 4, 1001), (5, 3, 50021), (2, 2, 131072), (200, 1, 257), (1, 40, 300), (16, 5, 4096)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("point", [False, True], ids=["probs", "point"])
@pytest.mark.parametrize("B,L,V", CASES)
def test_verify(B, L, V, dtype, point):
    x = inputs(B, L, V, dtype, seed=B + L + V, point=point)
    ra, _ = check(x)
    if B >= 64 and not point:
        assert 0 < int((ra < x["lens"]).sum()) < B, "the case should both accept and refuse"


def test_all_lengths_given_by_default():
    x = inputs(6, 3, 500, torch.float32, seed=1)
    x["lens"] = None
    check(x)


def test_no_drafts():
    """A plain draw from the target."""
    x = inputs(9, 0, 3000, torch.float32, seed=2)
    check(x)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_padded_vocabulary(dtype):
    """Rows out of wider buffers (vectors or single elements, as their alignment allows)."""
    for pad in (8, 3):
        x = inputs(4, 3, 1000, dtype, seed=3)
        p = torch.full((4, 4, 1000 + pad), 9.0, dtype=dtype, device="cuda")
        q = torch.full((4, 3, 1000 + pad), 9.0, dtype=dtype, device="cuda")
        p[..., :1000], q[..., :1000] = x["p"].cuda(), x["q"].cuda()
        check(x, p=p[..., :1000], q=q[..., :1000])


def test_edges():
    """Equal tables (all accepted), a draft that covers the target (drawn from the target), disjoint ones, u of 0 and
    next to 1, a token outside the vocabulary, rows with a single entry, NaN and negative entries, an empty row."""
    V = 300
    p = torch.rand((9, 3, V)) + 0.01
    q = p[:, :2].clone()
    tokens = torch.randint(0, V, (9, 2)).to(torch.int32)
    q[1] = 2 * p[1, :2]                       # refused by u; nothing is left after the subtraction
    p[2, :, : V // 2], q[2, :, V // 2:] = 0, 0
    tokens[2] = 3                             # target probability zero: refused whatever u
    tokens[3, 0] = V
    tokens[4, 1] = -1
    p[5] = 0
    p[5, :, 17] = 0.25
    p[6, 0, ::2] = float("nan")
    p[6, 0, 1] = -3.0
    tokens[6, 0] = 2                          # NaN there: refused
    p[7] = 0
    x = {"p": p, "q": q, "tokens": tokens, "lens": None,
         "ua": torch.full((9, 2), 0.9), "us": torch.tensor([0.0, 0.5, 1 - 2.0 ** -24, 0.0, 0.3, 0.99, 0.5, 0.5, 1.0])}
    x["ua"][2] = 0.0
    ra, rt = check(x)
    assert ra[0] == 2 and ra[1] == 0 and ra[2] == 0 and ra[3] == 0 and ra[4] <= 1 and rt[7, 0] == -1


def test_lengths_are_clamped():
    x = inputs(3, 4, 64, torch.float32, seed=5)
    x["lens"] = torch.tensor([-5, 99, 2], dtype=torch.int32)
    check(x)


def test_accepts_as_often_as_it_should():
    """Over uniform u, tokens come out with the target's distribution: a tiny vocabulary, every u on a grid, against the
    exact probability of each first token."""
    V, n = 3, 64
    p, q = torch.tensor([0.5, 0.2, 0.3]), torch.tensor([0.2, 0.6, 0.2])
    grid = (torch.arange(n).float() + 0.5) / n
    ua, us = grid.repeat_interleave(n), grid.repeat(n)
    count = torch.zeros(V, dtype=torch.float64)
    for x in range(V):
        B = n * n
        acc, tok = kb.kvattn_verify_drafts(p.expand(B, 2, V).contiguous().cuda(), q.expand(B, 1, V).contiguous().cuda(),
                                           torch.full((B, 1), x, dtype=torch.int32, device="cuda"), ua[:, None].cuda(), us.cuda())
        first = tok[:, 0].cpu().long()
        count += float(q[x]) * torch.bincount(first, minlength=V).double() / B
    # a grid of 64 points is off by at most one point per border
    assert bool(((count - p.double()).abs() <= 2 / 64).all())
