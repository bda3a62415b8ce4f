"""Overlaps of strided operands on the CPU: queries rotated in place whose rows run into their keys or values, and read
back rows that run into each other, are refused on the host (fake, never-dereferenced addresses)."""
import pytest

from tests.test_serving_abi import A, APPEND, GATHER, INVALID, call, lib  # noqa: F401

# a fused projection of 8 query heads, 2 of keys and 2 of values, 128 each: rows of 1536 elements
FUSED = dict(q=A, q_out=A, k=A + 2 * 1024, v=A + 2 * 1280, qs=1536, qos=1536, kst=1536, vst=1536)


@pytest.mark.parametrize("kw", [
    dict(k=A + 2 * (1024 - 8)),                          # a vector into the last query head
    dict(v=A + 2 * 512),                                 # inside the queries
    dict(v=A),                                           # the queries themselves
    dict(k=A + 2 * (1536 - 128)),                        # into the next token's queries
    dict(k=A - 2 * 128),                                 # from before the first token's into them
    dict(v=A + 2 * (1536 * 5 + 1000)),                   # the same, further on
    dict(kst=1544),                                      # another stride
    dict(q_out=A + 2 * 512, k=2 * A, v=3 * A),           # the output within the queries, not in place
    dict(q_out=A + 2 * 1024, k=A + 2 * 1280, v=3 * A),   # the output over the keys and beyond the row
], ids=range(9))
def test_queries_that_run_into_their_keys_or_values(lib, kw):  # noqa: F811
    assert call(lib, "kvattn_rope_append_rowscale", APPEND, {**FUSED, **kw}) == INVALID


@pytest.mark.parametrize("kw", [
    dict(vo=6 * A + 2 * 12800, kh=25600, vh=25616),      # alternating heads of other strides
    dict(vo=6 * A + 2 * 12792, kh=25600, vh=25600),      # a vector into the keys' row
    dict(vo=6 * A + 2 * 12808, kh=25600, vh=25600),      # a vector into the next head's keys
    dict(vo=6 * A, kh=25600, vh=25600),
], ids=range(4))
def test_read_back_rows_that_run_into_each_other(lib, kw):  # noqa: F811
    assert call(lib, "kvattn_gather_rowscale", GATHER, kw) == INVALID
