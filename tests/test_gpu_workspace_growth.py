"""GPU tests of captured decodes replayed after the library's workspace has grown behind them: the memory they were
captured with is still theirs (B200)."""
import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from tests import plain64
from tests import rowscale64 as r64
from tests.test_gpu_rowscale_bounds import caches, queries

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(autouse=True)
def _flags():
    torch.cuda.synchronize()
    kb.kvattn_release_workspace()
    kb.kvattn_clear_device_flags()
    yield
    torch.cuda.synchronize()
    kb.kvattn_release_workspace()
    assert kb.kvattn_read_device_flags() == 0


class Call:
    def __init__(self, B, L, n_q, lens, seed, columns=0):
        """columns: pages of 128, one a sequence, under a block table of so many columns."""
        self.lens, self.x, self.q = lens, caches(B, 1, 128 if columns else max(lens) + 1, seed), queries(B, L, n_q, seed)
        self.table = None
        if columns:
            self.table = torch.full((B, columns), -1, dtype=torch.int32, device="cuda")
            self.table[:, 0] = torch.arange(B)
        code = lambda c: c.to(torch.float8_e4m3fn).cuda()  # noqa: E731
        kc, ks, vc, vs = self.x
        self.args = (self.q.cuda(), code(kc), code(vc), ks.cuda(), vs.cuda())
        self.n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.out = torch.zeros(self.q.shape, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros(self.q.shape[:-1], device="cuda")

    def __call__(self):
        kb.kvattn_gqa_decode_rowscale(*self.args, self.n, 0.09, block_table=self.table, out=self.out, lse=self.lse)

    def check(self):
        L, n_q = self.q.shape[1:3]
        kc, ks, vc, vs = self.x
        for b, n in enumerate(self.lens):
            k, v = kc[b, 0, :n].double() * ks[b, 0, :n, None], vc[b, 0, :n].double() * vs[b, 0, :n, None]
            see = plain64.visible(n, L, n).repeat_interleave(n_q, 0)
            rows = self.q[b].reshape(L * n_q, 128)
            ref, rl, p = r64.attention(rows, k, v, see, 0.09)
            bo, bl = r64.bounds(rows, k, vc[b, 0, :n], vs[b, 0, :n], see, ref, p, 0.09)
            r64.assert_within(self.out[b].reshape(L * n_q, 128), ref, bo, f"out {b}")
            r64.assert_within(self.lse[b].reshape(L * n_q), rl, bl + 2.0 ** -21 * torch.nan_to_num(rl, neginf=0.0).abs(), f"lse {b}")


def test_replays_after_growth():
    stream = torch.cuda.Stream()
    # (a virtual batch needs the second buffer too)
    small = [Call(1, 1, 4, [900], 1), Call(1, 3, 32, [500], 2)]
    graphs = []
    for c in small:
        with torch.cuda.stream(stream):
            c()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            c()
        graphs.append(g)
    large = [Call(2, 1, 64, [40000, 30000], 3), Call(24, 40, 4, [300 + 7 * i for i in range(24)], 4), Call(64, 10, 20, [60 + i for i in range(64)], 5, columns=1000)]
    for c in large:
        c()
        junk = torch.full((1 << 22,), float("nan"), device="cuda")       # what a freed buffer would be given to
        for s, g in zip(small, graphs):
            s.out.fill_(float("nan"))
            s.lse.fill_(float("nan"))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            s.check()
        c.check()
        assert bool(torch.isnan(junk).all())
    del graphs
