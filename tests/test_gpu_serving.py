"""The serving operators together, as a server runs them: a shared prompt and each sequence's own tokens written into
row-scaled pages, the prompt read back once and shared by the batch's decode, the same attention over the pages
themselves, the drafted tokens verified; eagerly, and captured in a graph and replayed with other lengths (B200)."""
import math

import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from tests import plain64

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

B, L, NQ, NKV, D, S, PROMPT, OWN, V = 6, 3, 16, 4, 128, 128, 500, 200, 700
SCALE = 1 / math.sqrt(D)


@pytest.fixture(autouse=True)
def _flags():
    kb.kvattn_clear_device_flags()
    yield
    assert kb.kvattn_read_device_flags() == 0


class Server:
    """Pages 0.. hold the prompt, then two pages a sequence its own tokens (after the prompt's last page)."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        self.prompt_pages = (PROMPT + S - 1) // S
        pages = self.prompt_pages + 2 * B
        self.k = torch.full((pages, NKV, S, D), 0x7F, dtype=torch.uint8, device="cuda")
        self.v = self.k.clone()
        self.ks = torch.full((pages, NKV, S), float("nan"), device="cuda")
        self.vs = self.ks.clone()
        self.prompt = normal(PROMPT, NQ + 2 * NKV, D)
        self.own = normal(B, OWN, NQ + 2 * NKV, D)
        self.head = torch.randn((NQ * D, V), generator=g).cuda() * 0.05
        self.drafts = torch.randint(0, V, (B, L - 1), generator=g).to(torch.int32).cuda()
        self.ua, self.us = torch.rand((B, L - 1), generator=g).cuda(), torch.rand((B,), generator=g).cuda()
        self.prompt_slots = torch.arange(PROMPT, device="cuda")
        self.own_slots = (self.prompt_pages * S + torch.arange(B, device="cuda")[:, None] * 2 * S +
                          torch.arange(OWN, device="cuda")[None])
        self.table = (self.prompt_pages + 2 * torch.arange(B)[:, None] + torch.arange(2)[None]).to(torch.int32).cuda()
        self.lens = torch.zeros((B,), dtype=torch.int32, device="cuda")
        self.plen = torch.tensor([PROMPT], dtype=torch.int32, device="cuda")
        self.kp = torch.zeros((NKV, PROMPT, D), dtype=torch.bfloat16, device="cuda")
        self.vp = torch.zeros_like(self.kp)
        self.kc = torch.zeros((B, NKV, OWN, D), dtype=torch.bfloat16, device="cuda")
        self.vc = torch.zeros_like(self.kc)

    def write(self, x, positions, slots):
        q = torch.empty((x.shape[0], NQ, D), dtype=torch.bfloat16, device="cuda")
        return kb.kvattn_rope_append_rowscale(x[:, :NQ], x[:, NQ:NQ + NKV], x[:, NQ + NKV:], positions, slots, self.k, self.v,
                                              self.ks, self.vs, q_out=q)

    def prefill(self):
        self.write(self.prompt, torch.arange(PROMPT, dtype=torch.int32, device="cuda"), self.prompt_slots)
        self.q_own = self.write(self.own.view(B * OWN, -1, D), torch.arange(PROMPT, PROMPT + OWN, device="cuda").repeat(B).to(torch.int32),
                                self.own_slots.reshape(-1)).view(B, OWN, NQ, D)

    def step(self):
        """One scoring of L new tokens a sequence behind the prompt; every tensor stays on the device."""
        at = (self.lens[:, None] - L + torch.arange(L, device="cuda")[None]).clamp(min=0)
        q = self.q_own.gather(1, at.long()[..., None, None].expand(B, L, NQ, D))
        kb.kvattn_gather_rowscale(self.k, self.v, self.ks, self.vs, self.prompt_slots, k_out=self.kp, v_out=self.vp)
        k, v = kb.kvattn_gather_rowscale(self.k, self.v, self.ks, self.vs, self.own_slots.reshape(-1))
        self.kc.copy_(k.view(NKV, B, OWN, D).transpose(0, 1))
        self.vc.copy_(v.view(NKV, B, OWN, D).transpose(0, 1))
        out, lse = kb.kvattn_gqa_decode_prefix(q, self.kp, self.vp, self.plen, self.kc, self.vc, self.lens, SCALE)
        own, own_lse = kb.kvattn_gqa_decode_rowscale(q, self.k, self.v, self.ks, self.vs, self.lens, SCALE, block_table=self.table)
        probs = torch.softmax(out.float().view(B, L, NQ * D) @ self.head, -1)
        acc, tok = kb.kvattn_verify_drafts(probs, None, self.drafts, self.ua, self.us)
        return {"q": q, "out": out, "lse": lse, "own": own, "own_lse": own_lse, "probs": probs, "acc": acc, "tok": tok}

    def check(self, r, lens):
        r = {k: v.cpu() for k, v in r.items()}
        rows = lambda c, s, slots: (c.cpu().view(torch.float8_e4m3fn).double() * s.cpu().double()[..., None])[  # noqa: E731
            slots // S, :, slots % S]
        kp, vp = rows(self.k, self.ks, self.prompt_slots.cpu()), rows(self.v, self.vs, self.prompt_slots.cpu())
        # the prompt's keys are the rotated ones, to E4M3
        ref = plain64.rotate(self.prompt.cpu()[:, NQ:NQ + NKV], torch.arange(PROMPT), 10000.0, False)
        assert bool(((kp - ref).abs() <= plain64.HALF_E4M3 * ref.abs() + 2.0 ** -10 / 448 * 1.01 * ref.abs().amax(-1, keepdim=True) + 1e-5).all())
        g = NQ // NKV
        for b, n in enumerate(lens):
            ko, vo = rows(self.k, self.ks, self.own_slots[b, :n].cpu()), rows(self.v, self.vs, self.own_slots[b, :n].cpu())
            see = plain64.visible(n, L, n).repeat_interleave(g, 0)
            for j in range(NKV):
                q = r["q"][b, :, j * g:(j + 1) * g].reshape(L * g, D)
                flat = lambda x: x[b, :, j * g:(j + 1) * g].reshape(L * g, *x.shape[3:])  # noqa: E731
                # over the pages: the exact codes and scales
                o, l, p = plain64.attention(q, ko[:, j], vo[:, j], see, SCALE)
                slack = plain64.score_slack(q, ko[:, j], SCALE, "e4m3")
                plain64.assert_within(flat(r["own"]), o, plain64.out_bound(o, p, vo[:, j], slack, "e4m3"), f"own {b} {j}")
                plain64.assert_within(flat(r["own_lse"]), l, slack + 2.0 ** -21 * l.abs() + 2e-6, f"own lse {b} {j}")
                # behind the prompt: the rows read back to bf16
                k = torch.cat((kp[:, j], ko[:, j])).float().to(torch.bfloat16)
                v = torch.cat((vp[:, j], vo[:, j])).float().to(torch.bfloat16)
                o, l, p = plain64.attention(q, k, v, torch.cat((torch.ones((L * g, PROMPT), dtype=torch.bool), see), 1), SCALE)
                slack = plain64.score_slack(q, k, SCALE, "bf16")
                plain64.assert_within(flat(r["out"]), o, plain64.out_bound(o, p, v, slack, "bf16"), f"out {b} {j}")
                plain64.assert_within(flat(r["lse"]), l, slack + 2.0 ** -21 * l.abs() + 2e-6, f"lse {b} {j}")
        acc, tok = plain64.verify(r["probs"], None, self.drafts.cpu(), None, self.ua.cpu(), self.us.cpu())
        assert torch.equal(r["acc"], acc) and torch.equal(r["tok"], tok)


def test_a_step_of_a_server():
    s = Server(1)
    s.prefill()
    lens = [3, 200, 129, 128, 64, 131]
    s.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    r = s.step()
    torch.cuda.synchronize()
    s.check(r, lens)


def test_captured_and_replayed():
    """One capture, replayed with other lengths, while a second capture of the same step lives and replays in between."""
    s = [Server(2), Server(3)]
    graphs, outs = [], []
    stream = torch.cuda.Stream()
    for x in s:
        x.prefill()
        x.lens.fill_(OWN)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            x.step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs.append(x.step())
        graphs.append(graph)
    for lens in ([200, 3, 130, 128, 129, 64], [5, 4, 200, 199, 127, 100]):
        for i in range(2):
            for t in ("out", "lse", "own", "own_lse"):
                outs[i][t].fill_(float("nan"))
            s[i].lens.copy_(torch.tensor(lens, dtype=torch.int32))
        for i in (0, 1):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            s[i].check(outs[i], lens)
    del graphs


def test_other_stream_and_device_context():
    """Work given a stream runs there, in order with it, and leaves the current stream as it was."""
    s = Server(4)
    stream = torch.cuda.Stream()
    slots = s.prompt_slots
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)
    before = torch.cuda.current_stream()
    pos = torch.arange(PROMPT, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)
    kb.kvattn_rope_append_rowscale(None, s.prompt[:, NQ:NQ + NKV], s.prompt[:, NQ + NKV:], pos, slots, s.k, s.v, s.ks, s.vs,
                                   stream=stream)
    k, v = kb.kvattn_gather_rowscale(s.k, s.v, s.ks, s.vs, slots, stream=stream)
    assert torch.cuda.current_stream() == before
    stream.synchronize()
    ref = plain64.rotate(s.prompt.cpu()[:, NQ:NQ + NKV], torch.arange(PROMPT), 10000.0, False).transpose(0, 1)
    assert bool(((k.cpu().double() - ref).abs() <= 2.0 ** -3.9 * ref.abs() + 0.02).all())
    assert not bool(torch.isnan(v).any())
