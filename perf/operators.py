"""What is measured of the serving operators around the decode kernels: a row-scaled E4M3 cache
(written, read back, attended to), decode attention over a prefix the whole batch shares, and the
verification of drafted tokens.

Each case is one call a serving loop makes.  ``run`` computes it in plain torch operations, or, where
``own`` is set, by the library's entry point; ``exact`` gives the same from the definition in 64 bits.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
ROW_AMAX_MIN = 2.0 ** -55     # the smallest row maximum a scale is formed from

# ------------------------------------------------------------------------------- the cases


def listed():
    return [
        # one new token for each of 64 sequences: the per-step cache write of a 70B-shaped layer
        {"name": "write_step", "op": "write", "tokens": 64, "n_q": 64, "n_kv": 8, "d": 128, "page": 128,
         "pages": 256, "interleaved": False, "rotate": True},
        # a long prompt's keys and values on their way into the pages, sliced out of a fused
        # projection; some tokens are padding and are not written
        {"name": "write_prompt", "op": "write", "tokens": 8192, "n_q": 64, "n_kv": 8, "d": 128, "page": 128,
         "pages": 80, "interleaved": True, "rotate": True},
        # a short odd chunk of a prompt read back
        {"name": "read_chunk", "op": "read", "tokens": 1001, "n_kv": 8, "d": 128, "page": 128, "pages": 32},
        # a shared prompt read back whole, to be attended to by a batch
        {"name": "read_prompt", "op": "read", "tokens": 32768, "n_kv": 8, "d": 128, "page": 256, "pages": 160},
        # decode of a ragged batch over the row-scaled pages: 64 query heads on 8 KV heads
        {"name": "decode_ragged", "op": "decode", "batch": 16, "q_len": 1, "n_q": 64, "n_kv": 8, "page": 128,
         "lo": 1024, "hi": 8192, "window": 0},
        # long-context MQA
        {"name": "decode_mqa", "op": "decode", "batch": 4, "q_len": 1, "n_q": 32, "n_kv": 1, "page": 0,
         "lo": 32768, "hi": 32768, "window": 0},
        # four drafted tokens and the last accepted one, scored in one pass over short contexts
        {"name": "decode_drafts", "op": "decode", "batch": 8, "q_len": 5, "n_q": 32, "n_kv": 8, "page": 128,
         "lo": 1, "hi": 1000, "window": 0},
        # a small batch behind one short system prompt: where latency counts
        {"name": "prefix_small", "op": "prefix", "batch": 8, "q_len": 1, "n_q": 32, "n_kv": 8, "d": 128,
         "prefix": 2000, "cap": 256, "lo": 1, "hi": 200},
        # a full batch behind a long document
        {"name": "prefix_long", "op": "prefix", "batch": 64, "q_len": 1, "n_q": 64, "n_kv": 8, "d": 128,
         "prefix": 32768, "cap": 1024, "lo": 16, "hi": 1000},
        # drafted tokens behind a shared prompt, narrow heads
        {"name": "prefix_drafts", "op": "prefix", "batch": 32, "q_len": 4, "n_q": 32, "n_kv": 4, "d": 64,
         "prefix": 8191, "cap": 512, "lo": 4, "hi": 500},
        # one user's eight drafted tokens over a 32k vocabulary
        {"name": "verify_one", "op": "verify", "batch": 1, "drafts": 8, "vocab": 32000, "type": "float32",
         "point": False},
        # a full batch over a vocabulary of 128k
        {"name": "verify_batch", "op": "verify", "batch": 64, "drafts": 4, "vocab": 128000, "type": "float32",
         "point": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "decode", "prefix", "verify"))
    if op == "write":
        n, n_kv, d = _log(rng, 1, 8192), rng.choice((1, 2, 4, 8, 32)), rng.choice((64, 96, 128, 256))
        n_q = n_kv * rng.choice((1, 4, 8))
        while n * (n_q + 2 * n_kv) * d > 8192 * 80 * 128:
            n = n // 2 + 1
        page = rng.choice((16, 64, 128, 256))
        return {"op": op, "tokens": n, "n_q": n_q, "n_kv": n_kv, "d": d, "page": page,
                "pages": (n + page - 1) // page + rng.randint(1, 8), "interleaved": rng.random() < 0.5,
                "rotate": rng.random() < 0.8}
    if op == "read":
        n, n_kv, d = _log(rng, 1, 32768), rng.choice((1, 2, 4, 8, 32)), rng.choice((64, 96, 128, 256))
        while n * n_kv * d > 32768 * 8 * 128:
            n = n // 2 + 1
        page = rng.choice((16, 64, 128, 256))
        return {"op": op, "tokens": n, "n_kv": n_kv, "d": d, "page": page,
                "pages": (n + page - 1) // page + rng.randint(1, 8)}
    if op == "decode":
        n_kv, g, q_len = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 5, 8, 16, 32)), rng.choice((1, 1, 1, 2, 5))
        hi = _log(rng, 1, 32768)
        batch = _log(rng, 1, 64)
        while batch * hi * n_kv > 16 * 8192 * 8 or (batch * q_len * n_kv * g * hi) > 64 * 16 * 8192:
            batch, hi = max(1, batch - batch // 3 - (batch > 1)), max(1, hi - hi // 4)
        return {"op": op, "batch": batch, "q_len": q_len, "n_q": n_kv * g, "n_kv": n_kv,
                "page": rng.choice((0, 128, 256)), "lo": rng.randint(0, hi), "hi": hi,
                "window": rng.choice((0, 0, 0, _log(rng, 1, 4096)))}
    if op == "prefix":
        n_kv, g, q_len = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 8, 16)), rng.choice((1, 1, 1, 2, 5))
        d, batch = rng.choice((64, 128)), _log(rng, 1, 128)
        prefix, cap = _log(rng, 1, 32768), _log(rng, 1, 2048)
        while batch * q_len * n_kv * g * (prefix + cap) * d > 64 * 64 * 32768 * 128 or \
                batch * n_kv * cap * d > 64 * 8 * 1024 * 128:
            batch, prefix, cap = max(1, batch - batch // 3), max(1, prefix - prefix // 4), max(1, cap - cap // 4)
        return {"op": op, "batch": batch, "q_len": q_len, "n_q": n_kv * g, "n_kv": n_kv, "d": d,
                "prefix": prefix, "cap": cap, "lo": rng.randint(0, cap), "hi": cap}
    batch, drafts, vocab = _log(rng, 1, 64), rng.randint(1, 8), _log(rng, 1000, 160000)
    while batch * (drafts + 1) * vocab > 64 * 5 * 128000:
        batch = max(1, batch - batch // 3 - (batch > 1))
    return {"op": "verify", "batch": batch, "drafts": drafts, "vocab": vocab,
            "type": rng.choice(("float32", "float32", "bfloat16")), "point": rng.random() < 0.25}


def _lens(case, n):
    """The batch's lengths: the case's own, so that its work is known."""
    r = random.Random("%s %s %s %s" % (case["batch"], case["lo"], case["hi"], case["n_q"]))
    return [r.randint(case["lo"], case["hi"]) for _ in range(n)]


def _seen(length, q_len, window):
    """Pairs of (new token, cached token) that a sequence attends to."""
    hi = [max(0, length - q_len + 1 + i) for i in range(q_len)]
    return sum(min(h, window) if window else h for h in hi)


def work(case):
    op = case["op"]
    if op == "write":
        n, n_q, n_kv, d = case["tokens"], case["n_q"], case["n_kv"], case["d"]
        return {"bytes": n * (4 * n_q * d + 2 * n_kv * (2 * d + d + 4) + 12),
                "flops": n * (3 * (n_q + n_kv) * d + 4 * n_kv * d)}
    if op == "read":
        n, n_kv, d = case["tokens"], case["n_kv"], case["d"]
        return {"bytes": n * (2 * n_kv * (3 * d + 4) + 8), "flops": 2 * n * n_kv * d}
    if op == "decode":
        lens, L, n_q, n_kv, w = _lens(case, case["batch"]), case["q_len"], case["n_q"], case["n_kv"], case["window"]
        rows = sum(min(x, w + L - 1) if w else x for x in lens)
        return {"bytes": rows * n_kv * 2 * 132 + len(lens) * L * n_q * (4 * 128 + 4),
                "flops": 4 * 128 * n_q * sum(_seen(x, L, w) for x in lens)}
    if op == "prefix":
        lens, L, n_q, n_kv, d = _lens(case, case["batch"]), case["q_len"], case["n_q"], case["n_kv"], case["d"]
        return {"bytes": (case["prefix"] + sum(lens)) * n_kv * 4 * d + len(lens) * L * n_q * (4 * d + 4),
                "flops": 4 * d * n_q * (len(lens) * L * case["prefix"] + sum(_seen(x, L, 0) for x in lens))}
    # the rows that are drawn from: one of each table a sequence (a point draft has none)
    size = 2 if case["type"] == "bfloat16" else 4
    rows = case["batch"] * case["vocab"]
    return {"bytes": rows * size * (1 if case["point"] else 2) + case["batch"] * case["drafts"] * (12 + 2 * size),
            "flops": rows * (1 if case["point"] else 3)}


# ------------------------------------------------------------------------------- the inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _row_scaled(shape, g):
    """Codes and scales of a cache whose rows differ in size, as rows of real keys do: one row in
    forty is an outlier of ten times the size."""
    rows = shape[:-1]
    x = torch.randn(shape, generator=g, device="cuda")
    big = 1.0 + 9.0 * (torch.rand(rows, generator=g, device="cuda") < 0.025)
    size = big * torch.exp(0.3 * torch.randn(rows, generator=g, device="cuda"))
    x *= size[..., None]
    amax = x.abs().amax(-1)
    codes = (x * (E4M3_MAX / amax)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, amax / E4M3_MAX


def _slots(n, total, g):
    return torch.randperm(total, generator=g, device="cuda")[:n].to(torch.int64)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "write":
        n, n_q, n_kv, d, S, P = (case[k] for k in ("tokens", "n_q", "n_kv", "d", "page", "pages"))
        qkv = _normal((n, n_q + 2 * n_kv, d), g)
        s["q"], s["k"], s["v"] = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
        s["k"].mul_(1.0 + 9.0 * (torch.rand((n, n_kv, 1), generator=g, device="cuda") < 0.025).to(torch.bfloat16))
        s["positions"] = torch.randint(0, 131072, (n,), generator=g, device="cuda").to(torch.int32)
        slots = _slots(n, S * P, g)
        slots[torch.rand((n,), generator=g, device="cuda") < 0.03] = -1      # padding: not written
        s["slots"] = slots
        s["k_pages"], s["k_scales"] = _row_scaled((P, n_kv, S, d), g)
        s["v_pages"], s["v_scales"] = _row_scaled((P, n_kv, S, d), g)
        s["q_out"] = torch.zeros((n, n_q, d), dtype=torch.bfloat16, device="cuda")
    elif op == "read":
        n, n_kv, d, S, P = (case[k] for k in ("tokens", "n_kv", "d", "page", "pages"))
        s["k_pages"], s["k_scales"] = _row_scaled((P, n_kv, S, d), g)
        s["v_pages"], s["v_scales"] = _row_scaled((P, n_kv, S, d), g)
        pages = torch.randperm(P, generator=g, device="cuda")
        at = torch.arange(n, device="cuda")
        s["slots"] = pages[at // S] * S + at % S        # consecutive tokens of shuffled pages
        s["k_out"] = torch.zeros((n_kv, n, d), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros((n_kv, n, d), dtype=torch.bfloat16, device="cuda")
    elif op == "decode":
        B, L, n_q, n_kv, S = (case[k] for k in ("batch", "q_len", "n_q", "n_kv", "page"))
        lens = _lens(case, B)
        s["q"] = _normal((B, L, n_q, 128), g)
        if S:
            M = (max(lens) + S - 1) // S + 1
            used = [(x + S - 1) // S for x in lens]
            P = sum(used) + 2
            perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
            table = torch.zeros((B, M), dtype=torch.int32, device="cuda")
            at = 0
            for b, u in enumerate(used):
                table[b, :u] = perm[at:at + u]
                at += u
            s["table"] = table
            shape = (P, n_kv, S, 128)
        else:
            s["table"] = None
            shape = (B, n_kv, case["hi"] + 5, 128)
        s["k_pages"], s["k_scales"] = _row_scaled(shape, g)
        s["v_pages"], s["v_scales"] = _row_scaled(shape, g)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["scale"] = 1.0 / math.sqrt(128.0)
        s["out"] = torch.zeros((B, L, n_q, 128), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros((B, L, n_q), dtype=torch.float32, device="cuda")
    elif op == "prefix":
        B, L, n_q, n_kv, d, P, T = (case[k] for k in ("batch", "q_len", "n_q", "n_kv", "d", "prefix", "cap"))
        s["q"] = _normal((B, L, n_q, d), g)
        # keys of twice the size sharpen the softmax, as the sharp-keys decode workload does
        s["k_prefix"], s["v_prefix"] = _normal((n_kv, P + 7, d), g, 2.0), _normal((n_kv, P + 7, d), g)
        s["k_cache"], s["v_cache"] = _normal((B, n_kv, T, d), g, 2.0), _normal((B, n_kv, T, d), g)
        s["prefix_len"] = torch.tensor([P], dtype=torch.int32, device="cuda")
        s["lens"] = torch.tensor(_lens(case, B), dtype=torch.int32, device="cuda")
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.zeros((B, L, n_q, d), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros((B, L, n_q), dtype=torch.float32, device="cuda")
    else:
        B, L, V = case["batch"], case["drafts"], case["vocab"]
        dtype = getattr(torch, case["type"])
        # a peaked target, and a draft model near it; the drafts are drawn from the draft model
        logits = 2.5 * torch.randn((B, L + 1, V), generator=g, device="cuda")
        near = logits[:, :L] + 0.5 * torch.randn((B, L, V), generator=g, device="cuda")
        s["p"] = torch.softmax(logits, -1).to(dtype)
        q = torch.softmax(near, -1)
        s["q"] = None if case["point"] else q.to(dtype)
        if case["point"]:
            s["tokens"] = near.argmax(-1).to(torch.int32)
        else:
            s["tokens"] = torch.multinomial(q.view(B * L, V), 1, generator=g).view(B, L).to(torch.int32)
        s["lens"] = torch.randint(0, L + 1, (B,), generator=g, device="cuda").to(torch.int32)
        s["lens"][: (B + 1) // 2] = L
        s["u_accept"] = torch.rand((B, L), generator=g, device="cuda")
        s["u_sample"] = torch.rand((B,), generator=g, device="cuda")
        s["accepted"] = torch.zeros((B,), dtype=torch.int32, device="cuda")
        s["out"] = torch.zeros((B, L + 1), dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------- plain forms

ROPE_BASE = 10000.0


def _rotate(x, positions, interleaved):
    """x [N, heads, d] in 32 bits, turned by its position; the angle in 64."""
    d = x.shape[-1]
    i = torch.arange(d // 2, device=x.device, dtype=torch.float64)
    theta = positions.double()[:, None] * ROPE_BASE ** (-2.0 * i / d)
    c, s = theta.cos().float()[:, None], theta.sin().float()[:, None]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    a, b = x[..., : d // 2], x[..., d // 2:]
    return torch.cat((a * c - b * s, a * s + b * c), -1)


def _plain_write(s):
    case = s["case"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if case["rotate"]:
        q = _rotate(q, s["positions"], case["interleaved"])
        k = _rotate(k, s["positions"], case["interleaved"])
    s["q_out"].copy_(q.to(torch.bfloat16))
    keep = s["slots"] >= 0
    page, row = s["slots"][keep] // case["page"], s["slots"][keep] % case["page"]

    def store(x, pages, scales):
        amax = x.abs().amax(-1).clamp(min=ROW_AMAX_MIN)
        codes = (x * (E4M3_MAX / amax)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        pages.view(torch.uint8)[page, :, row] = codes.view(torch.uint8)[keep]
        scales[page, :, row] = (amax / E4M3_MAX)[keep]

    store(k, s["k_pages"], s["k_scales"])
    store(v, s["v_pages"], s["v_scales"])
    return {"q": s["q_out"], "k": s["k_pages"], "ks": s["k_scales"], "v": s["v_pages"], "vs": s["v_scales"]}


def _plain_read(s):
    S = s["case"]["page"]
    page, row = s["slots"] // S, s["slots"] % S

    def load(pages, scales):
        x = pages.view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn).float() * scales[page, :, row][..., None]
        return x.to(torch.bfloat16).transpose(0, 1).contiguous()

    return {"k": load(s["k_pages"], s["k_scales"]), "v": load(s["v_pages"], s["v_scales"])}


def _dequantised(s, pages, scales):
    """[B, n_kv, T, 128] in 32 bits, out of the pages of each sequence."""
    x = pages.float() * scales[..., None]
    if s["table"] is None:
        return x
    x = x[s["table"].long()]                       # [B, M, n_kv, S, 128]
    return x.transpose(1, 2).flatten(2, 3)


def _softmax_values(sc, v):
    """Softmax over the last axis times v, and the log-sum-exp; a row that sees nothing gives 0 and -inf."""
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(sc - m)
    total = e.sum(-1, keepdim=True)
    return e @ v / total.clamp(min=1e-37), (m + torch.log(total))[..., 0]


def _visible(lens, L, T, window, device):
    """[B, L, T]: which cached rows new token i of a sequence attends to."""
    t = torch.arange(T, device=device)[None, None]
    last = (lens[:, None] - L + torch.arange(L, device=device)[None])[..., None]
    see = t <= last
    return see & (t > last - window) if window else see


def _grouped(q, n_kv):
    """[B, L, n_q, d] -> [B, n_kv, L * g, d]"""
    B, L, n_q, d = q.shape
    return q.view(B, L, n_kv, n_q // n_kv, d).permute(0, 2, 1, 3, 4).reshape(B, n_kv, -1, d)


def _ungrouped(x, B, L, n_q):
    """[B, n_kv, L * g, ...] -> [B, L, n_q, ...]"""
    n_kv = x.shape[1]
    x = x.view(B, n_kv, L, n_q // n_kv, *x.shape[3:]).transpose(1, 2)
    return x.reshape(B, L, n_q, *x.shape[4:])


def _plain_decode(s):
    case = s["case"]
    B, L, n_q, n_kv = (case[k] for k in ("batch", "q_len", "n_q", "n_kv"))
    k, v = _dequantised(s, s["k_pages"], s["k_scales"]), _dequantised(s, s["v_pages"], s["v_scales"])
    sc = _grouped(s["q"].float(), n_kv) @ k.transpose(2, 3) * s["scale"]
    see = _visible(s["lens"].long(), L, k.shape[2], case["window"], k.device)
    see = see.repeat_interleave(n_q // n_kv, 1)[:, None]
    out, lse = _softmax_values(sc.masked_fill(~see, -math.inf), v)
    return {"out": _ungrouped(out, B, L, n_q).to(torch.bfloat16), "lse": _ungrouped(lse, B, L, n_q)}


def _plain_prefix(s):
    case = s["case"]
    B, L, n_q, n_kv, d = (case[k] for k in ("batch", "q_len", "n_q", "n_kv", "d"))
    q = _grouped(s["q"].float(), n_kv)                                          # [B, n_kv, r, d]
    r = q.shape[2]
    flat = q.transpose(0, 1).reshape(n_kv, B * r, d)                            # every row of a KV head
    sp = flat @ s["k_prefix"].float().transpose(1, 2) * s["scale"]              # against the one prefix
    sp = sp.masked_fill(torch.arange(sp.shape[2], device=q.device) >= s["prefix_len"], -math.inf)
    ss = q @ s["k_cache"].float().transpose(2, 3) * s["scale"]
    see = _visible(s["lens"].long(), L, ss.shape[3], 0, q.device).repeat_interleave(n_q // n_kv, 1)[:, None]
    ss = ss.masked_fill(~see, -math.inf)
    m = torch.maximum(sp.amax(-1).view(n_kv, B, r).transpose(0, 1), ss.amax(-1))
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    ep = torch.exp(sp - m0.transpose(0, 1).reshape(n_kv, B * r, 1))
    es = torch.exp(ss - m0[..., None])
    total = ep.sum(-1).view(n_kv, B, r).transpose(0, 1) + es.sum(-1)
    acc = (ep @ s["v_prefix"].float()).view(n_kv, B, r, d).transpose(0, 1) + es @ s["v_cache"].float()
    out = acc / total.clamp(min=1e-37)[..., None]
    lse = m0 + torch.log(total)
    return {"out": _ungrouped(out, B, L, n_q).to(torch.bfloat16), "lse": _ungrouped(lse, B, L, n_q)}


def _plain_verify(s):
    B, L, V = (s["case"][k] for k in ("batch", "drafts", "vocab"))
    p, tok = s["p"], s["tokens"].long()
    pt = p[:, :L].gather(2, tok[..., None])[..., 0].double()
    qt = torch.ones_like(pt) if s["q"] is None else s["q"].gather(2, tok[..., None])[..., 0].double()
    at = torch.arange(L, device=p.device)
    ok = (s["u_accept"].double() * qt < pt) & (at[None] < s["lens"][:, None])
    n = ok.long().cumprod(1).sum(1)                                              # accepted before the first refusal
    batch = torch.arange(B, device=p.device)
    row = p[batch, n].double()
    refused = (n < s["lens"])[:, None]
    i = n.clamp(max=L - 1)
    if s["q"] is None:
        drafted = torch.zeros_like(row).scatter_(1, tok[batch, i][:, None], 1.0)
    else:
        drafted = s["q"][batch, i].double()
    rest = torch.where(refused, (row - drafted).clamp(min=0), row)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, row)                # the draft covers the target: draw from it
    c = rest.cumsum(1)
    drawn = (c > s["u_sample"].double()[:, None] * c[:, -1:]).int().argmax(1)
    slots = torch.arange(L + 1, device=p.device)[None]
    kept = torch.cat((tok, tok[:, :1]), 1)
    out = torch.where(slots < n[:, None], kept, torch.where(slots == n[:, None], drawn[:, None], -1))
    return {"accepted": n.to(torch.int32), "tokens": out.to(torch.int32)}


_PLAIN = {"write": _plain_write, "read": _plain_read, "decode": _plain_decode, "prefix": _plain_prefix,
          "verify": _plain_verify}


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return _PLAIN[op](s)
    from mla_kv_cache_b200 import binding as kb
    if op == "write":
        kb.kvattn_rope_append_rowscale(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_pages"], s["v_pages"],
                                       s["k_scales"], s["v_scales"], rope_base=ROPE_BASE if case["rotate"] else 0.0,
                                       interleaved=case["interleaved"], q_out=s["q_out"])
        return {"q": s["q_out"], "k": s["k_pages"], "ks": s["k_scales"], "v": s["v_pages"], "vs": s["v_scales"]}
    if op == "read":
        k, v = kb.kvattn_gather_rowscale(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["slots"],
                                         k_out=s["k_out"], v_out=s["v_out"])
        return {"k": k, "v": v}
    if op == "decode":
        out, lse = kb.kvattn_gqa_decode_rowscale(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"],
                                                 s["lens"], s["scale"], block_table=s["table"], window=case["window"],
                                                 out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    if op == "prefix":
        out, lse = kb.kvattn_gqa_decode_prefix(s["q"], s["k_prefix"], s["v_prefix"], s["prefix_len"], s["k_cache"],
                                               s["v_cache"], s["lens"], s["scale"], out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    accepted, tokens = kb.kvattn_verify_drafts(s["p"], s["q"], s["tokens"], s["u_accept"], s["u_sample"],
                                               draft_lens=s["lens"], accepted=s["accepted"], tokens=s["out"])
    return {"accepted": accepted, "tokens": tokens}


# ------------------------------------------------------------------------------- in 64 bits


def _exact_attention(q, keys, values, see, scale):
    """q [r, d], keys and values [T, d], see [r, T]: out and log-sum-exp in 64 bits."""
    sc = (q @ keys.T) * scale
    sc[~see] = -math.inf
    lse = torch.logsumexp(sc, 1)
    w = torch.exp(sc - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None])
    return w @ values, lse


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "write":
        def turned(x):
            x = x.double()
            if not case["rotate"]:
                return x
            d = x.shape[-1]
            half = torch.arange(d // 2, device=x.device, dtype=torch.float64)
            angle = torch.outer(s["positions"].double(), torch.exp(-2.0 * half / d * math.log(ROPE_BASE)))
            z = torch.polar(torch.ones_like(angle), angle)[:, None]
            if case["interleaved"]:
                y = torch.view_as_complex(x.reshape(*x.shape[:-1], d // 2, 2).contiguous()) * z
                return torch.view_as_real(y).reshape(x.shape)
            y = torch.complex(x[..., : d // 2], x[..., d // 2:]) * z
            return torch.cat((y.real, y.imag), -1)

        k_out, v_out = s["k_pages"].double(), s["v_pages"].double()
        ks, vs = s["k_scales"].double(), s["v_scales"].double()
        written = (s["slots"] >= 0).nonzero()[:, 0]
        where = s["slots"][written]
        for x, codes, scales in ((turned(s["k"]), k_out, ks), (s["v"].double(), v_out, vs)):
            top = x.abs().max(-1).values.clamp(min=ROW_AMAX_MIN)
            codes[where // case["page"], :, where % case["page"]] = (x / top[..., None] * E4M3_MAX)[written]
            scales[where // case["page"], :, where % case["page"]] = (top / E4M3_MAX)[written]
        return {"q": turned(s["q"]), "k": k_out, "ks": ks, "v": v_out, "vs": vs}
    if op == "read":
        flat = lambda x: x.double().transpose(1, 2).flatten(0, 1)[s["slots"]]  # noqa: E731
        k = flat(s["k_pages"]) * flat(s["k_scales"][..., None])
        v = flat(s["v_pages"]) * flat(s["v_scales"][..., None])
        return {"k": k.transpose(0, 1), "v": v.transpose(0, 1)}
    if op in ("decode", "prefix"):
        B, L, n_q, n_kv = (case[k] for k in ("batch", "q_len", "n_q", "n_kv"))
        g, window = n_q // n_kv, case.get("window", 0)
        d = 128 if op == "decode" else case["d"]
        out = torch.zeros((B, L, n_q, d), dtype=torch.float64, device="cuda")
        lse = torch.full((B, L, n_q), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lens(case, B)):
            last = torch.arange(n - L, n, device="cuda")[:, None]
            t = torch.arange(n, device="cuda")[None]
            see = (t <= last) & (t > last - (window or n + L + 1))
            for j in range(n_kv):
                if op == "decode":
                    if s["table"] is None:
                        k, v = (s[x + "_pages"][b, j, :n].double() * s[x + "_scales"][b, j, :n, None].double()
                                for x in "kv")
                    else:
                        page = s["table"][b].long()
                        k, v = ((s[x + "_pages"][page, j].double() * s[x + "_scales"][page, j, :, None].double())
                                .flatten(0, 1)[:n] for x in "kv")
                    mask = see
                else:
                    P = case["prefix"]
                    k = torch.cat((s["k_prefix"][j, :P], s["k_cache"][b, j, :n])).double()
                    v = torch.cat((s["v_prefix"][j, :P], s["v_cache"][b, j, :n])).double()
                    mask = torch.cat((torch.ones((L, P), dtype=torch.bool, device="cuda"), see), 1)
                q = s["q"][b, :, j * g:(j + 1) * g].double().flatten(0, 1)
                if k.shape[0]:
                    o, l = _exact_attention(q, k, v, mask.repeat_interleave(g, 0), s["scale"])
                    out[b, :, j * g:(j + 1) * g], lse[b, :, j * g:(j + 1) * g] = o.view(L, g, d), l.view(L, g)
        return {"out": out, "lse": lse}
    n_out, tok_out = [], []
    p, q = s["p"].double(), None if s["q"] is None else s["q"].double()
    drafts, u, r, lens = s["tokens"].tolist(), s["u_accept"].tolist(), s["u_sample"].tolist(), s["lens"].tolist()
    for b in range(case["batch"]):
        got = []
        while len(got) < lens[b]:
            i, x = len(got), drafts[b][len(got)]
            if not u[b][i] * (1.0 if q is None else float(q[b, i, x])) < float(p[b, i, x]):
                break
            got.append(x)
        n, left = len(got), p[b, len(got)].clone()
        if n < lens[b]:
            if q is None:
                left[drafts[b][n]] -= 1.0
            else:
                left -= q[b, n]
            left = left.clamp(min=0)
            left = left if float(left.sum()) > 0 else p[b, n]
        c = torch.cumsum(left, 0)
        got.append(int(torch.searchsorted(c, (c[-1] * r[b])[None], right=True)[0]))
        n_out.append(n)
        tok_out.append(got + [-1] * (case["drafts"] - n))
    return {"accepted": torch.tensor(n_out, dtype=torch.int32), "tokens": torch.tensor(tok_out, dtype=torch.int32)}
