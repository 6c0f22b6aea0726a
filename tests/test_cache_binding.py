"""The cache's Python entries refuse what the C entries cannot be asked: a cache
of no heads or empty pages, flags that are no truth value, paths out of range.
No GPU needed."""

import numpy as np
import pytest
import torch

import dequant_gemm_int4_b200 as q4


def tensors(heads=2, page_size=16):
    packed = torch.zeros((3, 2, heads, page_size, 32), dtype=torch.uint8)
    scales = torch.zeros((3, 2, heads, page_size, 2), dtype=torch.float16)
    table, lens = torch.zeros((5, 2), dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    return torch.zeros((5, 4, 64), dtype=torch.bfloat16), packed, scales, table, lens


@pytest.mark.parametrize("kw", [dict(heads=0), dict(page_size=0)])
def test_a_cache_of_no_heads_or_empty_pages(kw):
    q, packed, scales, table, lens = tensors(**kw)
    slots = torch.zeros(5, dtype=torch.int64)
    k = q[:, :packed.shape[2]]
    for call in (lambda: q4.int4_cache_attention(q, packed, scales, table, lens, 32),
                 lambda: q4.cache_attention_workspace_size(q, packed, scales, table, 32),
                 lambda: q4.int4_cache_read(packed, scales, slots, 64, 32),
                 lambda: q4.int4_cache_write(k, k, packed, scales, slots, 32)):
        with pytest.raises(ValueError, match="heads and page_size"):
            call()


@pytest.mark.parametrize("name", ["causal", "return_lse"])
@pytest.mark.parametrize("value", [torch.tensor([True, False]), np.array([1, 0])])
def test_flags_that_are_no_truth_value(name, value):
    q, packed, scales, table, lens = tensors()
    with pytest.raises(TypeError, match=name):
        q4.int4_cache_attention(q, packed, scales, table, lens, 32, **{name: value})


@pytest.mark.parametrize("path", [1 << 32, -(1 << 40), (1 << 32) + q4.PATH_DECODE, 2.0, None])
def test_paths_out_of_range(path):
    q, packed, scales, table, lens = tensors()
    for call in (q4.int4_cache_attention, q4.cache_attention_workspace_size):
        args = (q, packed, scales, table) + ((lens,) if call is q4.int4_cache_attention else ())
        with pytest.raises((ValueError, TypeError), match="path must"):
            call(*args, 32, path=path)
