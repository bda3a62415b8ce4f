"""The binding's argument conversions of the serving operators on the CPU: what is no tensor is a TypeError, and
a window past 32 bits is the longest there is."""
import numpy as np
import pytest
import torch

from mla_kv_cache_b200 import binding as kb


@pytest.mark.parametrize("thing", [None, [1, 2], np.zeros((2,), dtype=np.int32), 7])
def test_no_tensor_is_a_type_error(thing):
    with pytest.raises(TypeError):
        kb._at(thing, "seq_lens", torch.int32, (2,), 0)
    with pytest.raises(TypeError):
        kb._codes_at(thing, "k_pages", (2,), 0)
    with pytest.raises(TypeError):
        kb._rows_at(thing, "k_new", torch.bfloat16, (2, 1, 8), 0)
    with pytest.raises(TypeError):
        kb.kvattn_gather_rowscale(thing, None, None, None, None)
    with pytest.raises(TypeError):
        kb.kvattn_gqa_decode_prefix(thing, None, None, None, None, None, None, 0.1)


@pytest.mark.parametrize("window,passed", [(0, 0), (5, 5), (-1, -1), (np.int64(7), 7), (2 ** 31 - 1, 2 ** 31 - 1),
                                           (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1), (1 << 62, 2 ** 31 - 1)])
def test_windows(window, passed):
    assert kb._window(window) == passed
