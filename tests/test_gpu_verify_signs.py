"""GPU tests of draft verification with entries below zero: they are never accepted or drawn (B200)."""
import pytest
import torch

from mla_kv_cache_b200 import binding as kb

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("V", [37, 4096])
def test_entries_below_zero(V, dtype):
    """A draft entry below zero counts as zero: a target entry of zero or less is neither accepted nor drawn next to it."""
    B = 64
    p = torch.zeros((B, 2, V))
    q = torch.full((B, 1, V), -0.5)          # below zero everywhere
    p[:, 0, 1::3] = -0.25
    at = torch.arange(B) % V
    p[torch.arange(B), 0, at] = 0.125        # the only entry above zero
    drafts = ((at + 1) % V).to(torch.int32)[:, None]
    even = torch.arange(0, B, 2)
    q[even, 0, drafts[even, 0].long()] = 1.0              # (the odd ones draft an entry below zero: refused as well)
    u = (torch.arange(B).float() + 0.5) / B
    acc, tok = kb.kvattn_verify_drafts(p.to(dtype).cuda(), q.to(dtype).cuda(), drafts.cuda(), torch.full((B, 1), 0.9, device="cuda"),
                                       u.cuda())
    torch.cuda.synchronize()
    assert not bool(acc.any()) and torch.equal(tok[:, 0].cpu(), at.to(torch.int32))
    p[:, 0] = torch.where(p[:, 0] > 0, -0.125, p[:, 0])   # nothing above zero: nothing to draw
    acc, tok = kb.kvattn_verify_drafts(p.to(dtype).cuda(), q.to(dtype).cuda(), drafts.cuda(), torch.full((B, 1), 0.9, device="cuda"),
                                       u.cuda())
    torch.cuda.synchronize()
    assert not bool(acc.any()) and bool((tok[:, 0] == -1).all())
