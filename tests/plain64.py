"""Plain 64-bit forms of the serving operators (CPU tensors), with the error bounds of the kernels'
formats, which the GPU tests compare against.

Half a step of rounding, relative to the value: bf16 2^-8, E4M3 2^-4 (2^-10 absolute below its
smallest normal, 2^-6)."""
import math

import torch

HALF_BF16, HALF_E4M3 = 2.0 ** -8, 2.0 ** -4


def rotate(x, positions, base, interleaved):
    """x [N, heads, d]: every pair turned by positions[n] * base^(-2i/d)."""
    x = x.double()
    d = x.shape[-1]
    i = torch.arange(d // 2, dtype=torch.float64)
    theta = positions.double()[:, None] * base ** (-2.0 * i / d)
    c, s = theta.cos()[:, None], theta.sin()[:, None]
    y = torch.empty_like(x)
    even, odd = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, None))
    y[..., even] = x[..., even] * c - x[..., odd] * s
    y[..., odd] = x[..., even] * s + x[..., odd] * c
    return y


def visible(length, L, T, window=0):
    """[L, T]: the cached positions each of a sequence's L newest tokens attends to."""
    last = torch.arange(length - L, length)[:, None]
    t = torch.arange(T)[None]
    see = t <= last
    return see & (t > last - window) if window else see


def attention(q, k, v, see, scale):
    """q [r, d], k / v [T, d], see [r, T] -> (out, lse, weights); a row that sees nothing: 0, -inf."""
    s = (q.double() @ k.double().T) * scale
    s = s.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, 1) if s.shape[1] else torch.full((s.shape[0],), -math.inf, dtype=torch.float64)
    p = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None])
    return p @ v.double(), lse, p


def score_slack(q, k, scale, fmt):
    """Bound of a score's error: an fp32 product of d terms (2^-24 each of the running sum, taken as
    d / 2 roundings), and for an E4M3 cache the query's two parts, off by at most 2^-18 of the
    largest query element (the remainder's smallest step, 2^-10, over a maximum of at least 128)."""
    q, k = q.double().abs(), k.double().abs()
    d = q.shape[1]
    slack = (q @ k.T) * (d / 2 * 2.0 ** -24)
    if fmt == "e4m3":
        slack = slack + 2.0 ** -17 * q.max() * k.sum(1)[None]
    return slack.amax(1) * abs(scale) + 1e-6 if k.shape[0] else torch.full((q.shape[0],), 1e-6, dtype=torch.float64)


def out_bound(ref, p, v, slack, fmt):
    """Elementwise bound of a bf16 output: its own rounding, the weights' rounding, the scores' error.
    bf16 weights: half a step each.  E4M3 weights in two parts: the remainder's half step of a
    remainder of at most a half step (2^-8), or, where the parts run out of range, the smallest
    half step 2^-10 of weights that reach at least 2^4 of 2^6 (the lazy maximum moves after a
    factor of 4): 2^-14 of the largest weighted row, never more than the weight itself.  (Weights
    in f16, half a step 2^-12 and 2^-25 absolute of weights that reach at least 2^0, lie within.)"""
    p = p.double()
    v = v.double().abs()
    w = p @ v
    bound = HALF_BF16 * ref.abs() + (HALF_BF16 + 2 * slack[:, None] + 1e-5) * w
    if fmt == "e4m3" and v.shape[0]:
        size = v.amax(1)                               # the value scale's share of a weight
        weight = p * size[None]
        floor = torch.minimum(weight, 2.0 ** -14 * weight.amax(1, keepdim=True))
        bound = bound + floor.sum(1)[:, None]
    return bound + 1e-30


def assert_within(got, ref, bound, what):
    got, ref = got.double().cpu(), ref.double()
    bad_inf = ~(torch.isfinite(ref)) & (got != ref)
    assert not bool(bad_inf.any()), f"{what}: infinities differ"
    fin = torch.isfinite(ref)
    assert bool(torch.isfinite(got[fin]).all()), f"{what}: not finite"
    err = (got - ref).abs()[fin]
    b = (bound.expand_as(ref) if torch.is_tensor(bound) else torch.full_like(ref, bound))[fin]
    worst = float((err / b).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound (largest error {float(err.max()):.3e})"
    return worst


def verify(p, q, drafts, lens, u_accept, u_sample):
    """One sequence after the other, as the definition reads; p [B, L + 1, V], q [B, L, V] or None."""
    p = p.double()
    q = None if q is None else q.double()
    B, L1, V = p.shape
    accepted, tokens = [], []
    for b in range(B):
        m = L1 - 1 if lens is None else max(0, min(L1 - 1, int(lens[b])))
        n = 0
        while n < m:
            x = int(drafts[b, n])
            if not 0 <= x < V:
                break
            qx = 1.0 if q is None else float(q[b, n, x])
            if not float(u_accept[b, n]) * qx < float(p[b, n, x]):
                break
            n += 1
        row = torch.nan_to_num(p[b, n], nan=-1.0).clamp(min=0)
        r = p[b, n].clone()
        if n < m:
            if q is not None:
                r -= q[b, n]
            elif 0 <= int(drafts[b, n]) < V:
                r[int(drafts[b, n])] -= 1.0
        r = torch.nan_to_num(r, nan=-1.0).clamp(min=0)
        if not float(r.sum()) > 0:
            r = row
        if float(r.sum()) > 0:
            c = r.cumsum(0)
            hit = ((c > float(u_sample[b]) * c[-1]) & (r > 0)).nonzero()
            new = int(hit[0]) if len(hit) else int((r > 0).nonzero()[-1])
        else:
            new = -1
        accepted.append(n)
        tokens.append([int(t) for t in drafts[b, :n]] + [new] + [-1] * (L1 - 1 - n))
    return torch.tensor(accepted, dtype=torch.int32), torch.tensor(tokens, dtype=torch.int32)
