"""GPU tests of the row-scaled decode over rows that a query must not see: NaN and infinities in them leave its result
alone, and reach the queries that do see them (B200)."""
import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from tests.test_gpu_rowscale import paginate
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


def before_the_window(x, lens, L, window):
    """NaN codes and scales in every row before the first that any query sees, infinite scales in the last two."""
    for b, n in enumerate(lens):
        first = max(0, n - L + 1 - window)
        for i in range(4):
            x[i][b, :, :first] = float("nan")
        for i in (1, 3):
            x[i][b, :, max(0, first - 2):first] = float("inf")
    return x


WINDOWS = [(8, 8, 1, 1), (64, 2, 1, 100), (32, 8, 1, 130), (32, 8, 5, 77), (16, 4, 3, 200), (64, 1, 2, 129)]


@pytest.mark.parametrize("forced", [None, (5, 1)])
@pytest.mark.parametrize("S", [0, 128])
@pytest.mark.parametrize("n_q,n_kv,L,window", WINDOWS)
def test_nan_before_the_window(n_q, n_kv, L, window, S, forced):
    lens = [400, 2, 129, 257, 640]
    x = before_the_window(caches(5, n_kv, 643, 3), lens, L, window)
    out, lse = run(queries(5, L, n_q, 4), x, lens, 0.09, window=window, S=S, forced=forced)
    assert not bool(torch.isnan(out.float()).any()) and not bool(torch.isnan(lse).any())


DRAFTS = [(8, 8, 2), (32, 8, 5), (16, 4, 4), (64, 2, 2), (64, 8, 8), (64, 1, 3)]


@pytest.mark.parametrize("S,window", [(0, 0), (128, 0), (128, 60), (0, 3)])
@pytest.mark.parametrize("what", ["code", "value scale", "key", "inf"])
@pytest.mark.parametrize("n_q,n_kv,L", DRAFTS)
def test_nan_in_the_newest_token(n_q, n_kv, L, what, S, window):
    """The newest token's row: its own query meets it, the older ones do not."""
    lens = [300, 128, 129, 1 + L, 1]
    x = caches(5, n_kv, 303, 5)
    for b, n in enumerate(lens):
        if what == "code":
            x[2][b, :, n - 1, 5] = float("nan")
            x[2][b, :, n - 1, 70::7] = float("nan")
        else:
            x[1 if what == "key" else 3][b, :, n - 1] = float("nan" if what != "inf" else "inf")
    if what == "inf":       # (the newest row's own result is not told here)
        out, lse = call_only(queries(5, L, n_q, 6), x, lens, window, S)
        assert not bool(torch.isnan(out[:, :-1].float()).any()) and not bool(torch.isinf(out[:, :-1].float()).any())
    else:
        run(queries(5, L, n_q, 6), x, lens, 0.09, window=window, S=S)


def call_only(q, x, lens, window, S):
    kc, ks, vc, vs = x
    code = lambda c: c.to(torch.float8_e4m3fn)  # noqa: E731
    if S:
        (kp, vp), (kr, vr), table = paginate((code(kc), code(vc)), (ks, vs), lens, S, torch.Generator().manual_seed(1))
        table = table.cuda()
    else:
        kp, vp, kr, vr, table = code(kc).view(torch.uint8), code(vc).view(torch.uint8), ks, vs, None
    out, lse = kb.kvattn_gqa_decode_rowscale(q.cuda(), kp.cuda(), vp.cuda(), kr.cuda(), vr.cuda(),
                                             torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.09, block_table=table,
                                             window=window)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def test_nan_in_a_row_that_is_seen():
    """It reaches the elements it belongs to, for the queries that see it, and no others."""
    lens = [300, 500]
    x = caches(2, 2, 503, 7)
    x[2][0, :, 297, 9] = float("nan")        # seen by the last three of five queries
    x[2][1, :, 20, 11] = float("nan")        # by all, far from the masked tiles
    out, _ = run(queries(2, 5, 16, 8), x, lens, 0.09, S=128)
    assert bool(torch.isnan(out[0, 2:, :, 9].float()).all()) and not bool(torch.isnan(out[0, :2].float()).any())
    assert bool(torch.isnan(out[1, :, :, 11].float()).all())
