"""The serving operators' entry points on the CPU: bad arguments are refused on the host before any
device work, by the C functions (fake, never-dereferenced addresses) and by the binding."""
import ctypes

import pytest
import torch

from mla_kv_cache_b200 import binding as kb
from mla_kv_cache_b200 import build as kbuild

INVALID, UNSUPPORTED, MISALIGNED = kb.KVATTN_ERR_INVALID_ARG, kb.KVATTN_ERR_UNSUPPORTED, kb.KVATTN_ERR_MISALIGNED
A = 1 << 40      # fake 16-byte aligned addresses, far apart


@pytest.fixture(scope="module")
def lib():
    kbuild.build(quiet=True)
    return kb.lib()


def call(lib, name, defaults, kw):
    unknown = set(kw) - set(defaults)
    assert not unknown, unknown
    return getattr(lib, name)(*{**defaults, **kw}.values())


APPEND = dict(q=A, k=2 * A, v=3 * A, pos=4 * A, slots=5 * A, q_out=6 * A, kp=7 * A, vp=8 * A, ks=9 * A, vs=10 * A, N=16,
              n_q=8, n_kv=2, d=128, qs=1024, qos=1024, kst=256, vst=256, P=4, S=128, base=10000.0, inter=0, stream=None)


@pytest.mark.parametrize("kw,expected", [
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(slots=0), INVALID), (dict(kp=0), INVALID), (dict(vs=0), INVALID),
    (dict(q=0), INVALID), (dict(q_out=0), INVALID), (dict(q=0, q_out=0), INVALID),      # n_q without a query
    (dict(pos=0), INVALID), (dict(N=-1), INVALID), (dict(n_kv=0), INVALID), (dict(n_q=0), INVALID),
    (dict(P=0), INVALID), (dict(S=0), INVALID), (dict(base=-1.0), INVALID), (dict(base=float("nan")), INVALID),
    (dict(kst=255), INVALID), (dict(vst=128), INVALID), (dict(qs=1000), INVALID), (dict(qos=0), INVALID),
    (dict(d=120), UNSUPPORTED), (dict(d=272, kst=1024, vst=1024, qs=4096, qos=4096), UNSUPPORTED), (dict(d=0), UNSUPPORTED),
    (dict(P=1 << 20, S=1 << 11), UNSUPPORTED), (dict(kst=1 << 33), UNSUPPORTED),
    (dict(k=2 * A + 8), MISALIGNED), (dict(slots=5 * A + 8), MISALIGNED), (dict(kst=257), MISALIGNED),
    (dict(qs=1028), MISALIGNED), (dict(ks=9 * A + 4), MISALIGNED),
    (dict(q_out=2 * A), INVALID), (dict(kp=3 * A), INVALID), (dict(ks=7 * A), INVALID), (dict(vp=7 * A), INVALID),
    (dict(q_out=A, qos=2048), INVALID),                  # the query's own buffer at another stride
])
def test_append_refuses(lib, kw, expected):
    assert call(lib, "kvattn_rope_append_rowscale", APPEND, kw) == expected


def test_append_of_nothing(lib):
    assert call(lib, "kvattn_rope_append_rowscale", APPEND, dict(N=0)) == kb.KVATTN_OK


GATHER = dict(kp=A, vp=2 * A, ks=3 * A, vs=4 * A, slots=5 * A, ko=6 * A, vo=7 * A, N=100, n_kv=2, d=128, kh=12800,
              vh=12800, P=4, S=128, stream=None)


@pytest.mark.parametrize("kw,expected", [
    (dict(kp=0), INVALID), (dict(vs=0), INVALID), (dict(slots=0), INVALID), (dict(vo=0), INVALID), (dict(N=-2), INVALID),
    (dict(n_kv=0), INVALID), (dict(P=0), INVALID), (dict(kh=12799), INVALID), (dict(vh=0), INVALID),
    (dict(d=24), UNSUPPORTED), (dict(d=512, kh=1 << 20, vh=1 << 20), UNSUPPORTED), (dict(P=1 << 30), UNSUPPORTED),
    (dict(kp=A + 1), MISALIGNED), (dict(ko=6 * A + 8), MISALIGNED), (dict(kh=12804), MISALIGNED),
    (dict(ko=A), INVALID), (dict(vo=6 * A + 16), INVALID),
])
def test_gather_refuses(lib, kw, expected):
    assert call(lib, "kvattn_gather_rowscale", GATHER, kw) == expected


DECODE = dict(q=A, kp=2 * A, vp=3 * A, ks=4 * A, vs=5 * A, table=6 * A, lens=7 * A, P=8, S=128, M=4, B=2, L=1, n_q=16, n_kv=2,
              d=128, scale=0.1, window=0, out=8 * A, lse=9 * A, stream=None)


@pytest.mark.parametrize("kw,expected", [
    (dict(q=0), INVALID), (dict(ks=0), INVALID), (dict(lens=0), INVALID), (dict(out=0), INVALID), (dict(B=0), INVALID),
    (dict(L=0), INVALID), (dict(n_q=15), INVALID), (dict(n_kv=0), INVALID), (dict(M=0), INVALID), (dict(window=-1), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(table=0), INVALID), (dict(table=0, P=2, M=2), INVALID),
    (dict(d=64), UNSUPPORTED), (dict(n_q=130), UNSUPPORTED), (dict(S=64), UNSUPPORTED), (dict(S=192), UNSUPPORTED),
    (dict(B=4096, L=2), UNSUPPORTED), (dict(M=1 << 25), UNSUPPORTED), (dict(P=1 << 24), UNSUPPORTED),
    (dict(q=A + 2), MISALIGNED), (dict(vs=5 * A + 4), MISALIGNED), (dict(out=8 * A + 8), MISALIGNED),
    (dict(out=2 * A), INVALID), (dict(lse=4 * A), INVALID), (dict(lse=8 * A), INVALID),
])
def test_decode_refuses(lib, kw, expected):
    assert call(lib, "kvattn_gqa_decode_rowscale", DECODE, kw) == expected


PREFIX = dict(q=A, kp=2 * A, vp=3 * A, plen=4 * A, P=1000, kc=5 * A, vc=6 * A, lens=7 * A, T=200, B=4, L=1, n_q=16, n_kv=2,
              d=128, scale=0.1, out=8 * A, lse=9 * A, ws=10 * A, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,expected", [
    (dict(q=0), INVALID), (dict(kp=0), INVALID), (dict(plen=0), INVALID), (dict(lens=0), INVALID), (dict(lse=0), INVALID),
    (dict(ws=0), INVALID), (dict(P=0), INVALID), (dict(T=0), INVALID), (dict(B=0), INVALID), (dict(L=0), INVALID),
    (dict(n_q=17), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(n_q=258), UNSUPPORTED), (dict(n_q=64, L=5), UNSUPPORTED), (dict(B=4096, L=2), UNSUPPORTED),
    (dict(T=1 << 30), UNSUPPORTED), (dict(P=1 << 30), UNSUPPORTED),
    (dict(q=A + 8), MISALIGNED), (dict(plen=4 * A + 4), MISALIGNED), (dict(ws=10 * A + 8), MISALIGNED),
    (dict(out=A), INVALID), (dict(lse=8 * A), INVALID), (dict(ws=5 * A), INVALID), (dict(ws=8 * A), INVALID),
])
def test_prefix_refuses(lib, kw, expected):
    assert call(lib, "kvattn_gqa_decode_prefix", PREFIX, kw) == expected


PAGED = dict(q=A, kp=2 * A, vp=3 * A, ptab=4 * A, plen=5 * A, PM=8, tab=6 * A, lens=7 * A, N=64, S=128, M=4, B=4, L=1, n_q=16,
             n_kv=2, d=128, scale=0.1, out=8 * A, lse=9 * A, ws=10 * A, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,expected", [
    (dict(ptab=0), INVALID), (dict(tab=0), INVALID), (dict(PM=0), INVALID), (dict(M=0), INVALID), (dict(N=0), INVALID),
    (dict(S=64), UNSUPPORTED), (dict(S=100), UNSUPPORTED), (dict(PM=1 << 25), UNSUPPORTED), (dict(N=1 << 24), UNSUPPORTED),
    (dict(ptab=4 * A + 4), MISALIGNED), (dict(out=2 * A + (1 << 12)), INVALID),
])
def test_prefix_paged_refuses(lib, kw, expected):
    assert call(lib, "kvattn_gqa_decode_prefix_paged", PAGED, kw) == expected


def test_workspace_refuses(lib):
    n = ctypes.c_size_t(0)
    good = [1000, 200, 4, 1, 16, 2, 128]
    assert lib.kvattn_gqa_decode_prefix_workspace(*good, None) == INVALID
    for i, bad, expected in [(0, 0, INVALID), (2, 0, INVALID), (4, 15, INVALID), (6, 32, UNSUPPORTED), (3, 100, UNSUPPORTED)]:
        a = list(good)
        a[i] = bad
        assert lib.kvattn_gqa_decode_prefix_workspace(*a, ctypes.byref(n)) == expected


VERIFY = dict(p=A, q=2 * A, drafts=3 * A, lens=4 * A, ua=5 * A, us=6 * A, acc=7 * A, tok=8 * A, B=4, L=3, V=1000, bf16=0, pb=4000,
              pl=1000, qb=3000, ql=1000, stream=None)


@pytest.mark.parametrize("kw,expected", [
    (dict(p=0), INVALID), (dict(us=0), INVALID), (dict(acc=0), INVALID), (dict(tok=0), INVALID), (dict(drafts=0), INVALID),
    (dict(ua=0), INVALID), (dict(B=0), INVALID), (dict(L=-1), INVALID), (dict(V=0), INVALID), (dict(pb=-4), INVALID),
    (dict(ql=-1), INVALID), (dict(B=5000), UNSUPPORTED), (dict(L=1025), UNSUPPORTED), (dict(V=(1 << 28) + 1), UNSUPPORTED),
    (dict(pb=1 << 41), UNSUPPORTED), (dict(p=A + 2), MISALIGNED), (dict(drafts=3 * A + 4), MISALIGNED),
    (dict(acc=7 * A + 4), MISALIGNED), (dict(acc=A), INVALID), (dict(tok=3 * A), INVALID), (dict(tok=7 * A), INVALID),
])
def test_verify_refuses(lib, kw, expected):
    assert call(lib, "kvattn_verify_drafts", VERIFY, kw) == expected


def test_binding_refuses_cpu_tensors():
    b = dict(dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kb.kvattn_rope_append_rowscale(None, torch.zeros(2, 1, 64, **b), torch.zeros(2, 1, 64, **b), None,
                                       torch.zeros(2, dtype=torch.int64), torch.zeros(1, 1, 4, 64, dtype=torch.uint8),
                                       torch.zeros(1, 1, 4, 64, dtype=torch.uint8), torch.zeros(1, 1, 4), torch.zeros(1, 1, 4),
                                       rope_base=0.0)
    with pytest.raises(ValueError):
        kb.kvattn_verify_drafts(torch.zeros(1, 2, 8), None, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1),
                                torch.zeros(1))
    with pytest.raises(ValueError):
        kb.kvattn_verify_drafts(torch.zeros(1, 2, 8, dtype=torch.float16), None, torch.zeros(1, 1, dtype=torch.int32),
                                torch.zeros(1, 1), torch.zeros(1))
    with pytest.raises(ValueError):
        kb.kvattn_gqa_decode_prefix(torch.zeros(1, 4, 64, **b), torch.zeros(2, 8, 64, **b), torch.zeros(2, 8, 64, **b),
                                    torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, 8, 64, **b),
                                    torch.zeros(1, 2, 8, 64, **b), torch.zeros(1, dtype=torch.int32), 0.1)
