"""Plain 64-bit attention over row-scaled rows, with the error bounds of the f16 decode kernel.

The kernel's formats: E4M3 codes and the query (times a power of two) exact in f16 but for query elements below 2^-27
of the row's largest, which keep an absolute 2^-38 of it; scores, maxima, sums and outputs in fp32; a weight times its
token's value scale in f16 (half a step 2^-11 relative, or 2^-25 absolute where weights reach at least 2^0); the
output rounded once to bf16 (2^-8)."""
import math

import torch

HALF_BF16, HALF_F16, FLOOR_F16 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -25


def attention(q, k, v, see, scale):
    """q [r, d], k / v [T, d], see [r, T] -> (out, lse, weights), sums over the visible rows alone: a NaN in a row
    that is not seen stays out."""
    q, k, v = q.double(), k.double(), v.double()
    s = ((q @ k.T) * scale).masked_fill(~see, -math.inf)
    r, T = s.shape
    lse = torch.logsumexp(s, 1) if T else torch.full((r,), -math.inf, dtype=torch.float64)
    p = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None]).masked_fill(~see, 0)
    out = torch.stack([p[i][see[i]] @ v[see[i]] for i in range(r)]) if r else q
    return out, lse, p


def bounds(q, k, code, vs, see, ref, p, scale):
    """(elementwise bound of the bf16 output, bound of the lse) for value rows code [T, d] * vs [T]."""
    q, k, code, vs = (torch.nan_to_num(x.double(), nan=0.0, posinf=0.0).abs() for x in (q, k, code, vs))
    p = torch.nan_to_num(p)
    T, d = k.shape
    if not T:
        return HALF_BF16 * ref.abs() + 1e-30, torch.full((q.shape[0],), 2e-6, dtype=torch.float64)
    size = (q @ k.T).masked_fill(~see, 0)                       # sum of the score's terms
    # an fp32 product of d terms (d / 2 roundings of the running sum), the query's smallest elements, and
    # the roundings of the score's factors, of its difference to the maximum and of the exponential
    score = (size * (d / 2 * 2.0 ** -24) + 2.0 ** -38 * q.amax(1, keepdim=True) * k.sum(1)[None]) * abs(scale)
    score = score.masked_fill(~see, 0).amax(1) + 2.0 ** -21 * (size.amax(1) * abs(scale) + 1)
    sums = 2.0 ** -23 * (T / 16 + 48)                           # additions of T terms by 16 threads or steps, and the merge
    w = p * vs[None]
    floor = torch.minimum(w, FLOOR_F16 * w.amax(1, keepdim=True)) @ code
    out = HALF_BF16 * ref.abs() + (1 + HALF_BF16) * ((HALF_F16 + 2 * score + 2 * sums)[:, None] * (w @ code) + floor)
    return out + 1e-30, score + sums + 2e-6


def assert_within(got, ref, bound, what):
    """NaN where the reference has NaN, the same infinities, everything else within the bound."""
    got, ref = got.double().cpu(), ref.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN differs"
    fin = torch.isfinite(ref)
    inf = ~fin & ~torch.isnan(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    assert bool(torch.isfinite(got[fin]).all()), f"{what}: not finite"
    err, b = (got - ref).abs()[fin], bound.expand_as(ref)[fin]
    worst = float((err / b).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"
    return worst


def emulate(q, kcode, ks, vcode, vs, scale, weight_type=torch.float16, vs_type=torch.float32):
    """The kernel's arithmetic over one unit, every token visible: weights * value scales rounded to weight_type,
    value scales held in vs_type; everything else in 64 bits."""
    s = (q.double() @ kcode.double().T) * ks.double()[None] * scale
    vs = vs.to(vs_type).double()
    m = (s + vs.log()[None]).amax(1, keepdim=True)
    a = torch.exp(s - m)
    w = (a * vs[None]).float().to(weight_type).double()
    return ((w @ vcode.double()) / a.sum(1, keepdim=True)).to(torch.bfloat16)


def cancelling(n):
    """Rows whose values nearly cancel, so that a weight's own rounding shows: a query of zeros (equal weights), codes
    +c under a scale of 1 + 2^-8 and -c under 1, and a row of zeros whose larger scale keeps those weights off a power
    of two.  (q, k codes, k scales, v codes, v scales) of 2 n + 1 tokens."""
    g = torch.Generator().manual_seed(n)
    c = torch.randint(1, 15, (n, 128), generator=g).float()
    vcode = torch.cat((torch.stack((c, -c), 1).reshape(2 * n, 128), torch.zeros((1, 128))))
    vs = torch.cat((torch.tensor([1 + 2.0 ** -8, 1.0]).repeat(n), torch.tensor([1.5])))
    kcode = torch.randint(-7, 8, (2 * n + 1, 128), generator=g).float()
    return torch.zeros((8, 128), dtype=torch.bfloat16), kcode, torch.rand((2 * n + 1,), generator=g) + 0.5, vcode, vs
