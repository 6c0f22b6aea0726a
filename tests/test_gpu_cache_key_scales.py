"""GPU tests of attention over the 4-bit cache with one group's key scale not finite."""

import math

import pytest
import torch

import dequant_gemm_int4_b200 as q4
from cache_checks import made_cache, made_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path", [q4.PATH_SIMT, q4.PATH_DECODE, q4.PATH_PREFILL])
@pytest.mark.parametrize("D, group", [(128, 32), (128, 128), (96, 32), (64, 64)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_key_scale_that_is_not_finite(bad, D, group, path):
    """The rows that see its token are NaN; the others do not change."""
    lens, counts = [70, 45], [4, 4]
    table, pages = made_table(lens, 16)
    packed, scales, _ = made_cache(pages, 16, 2, D, group, False)
    q = torch.randn((8, 8, D), generator=torch.Generator().manual_seed(3)).cuda().bfloat16()
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    call = lambda s: q4.int4_cache_attention(q, packed, s, table, lens_t, group, return_lse=True, path=path)  # noqa: E731
    clean = call(scales)
    dirty = scales.clone()
    dirty[table[0, 4].long(), 0, :, 4, -1] = bad  # token 68: seen by the last two queries of sequence 0
    out, lse = call(dirty)
    keep = [0, 1, 4, 5, 6, 7]
    if path != q4.PATH_PREFILL:
        assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])
    assert torch.isfinite(out[keep]).all() and torch.isfinite(lse[keep]).all()
    # 32 products or more of both signs with infinity: NaN, as with a NaN scale.
    assert torch.isnan(lse[2:4]).all() and torch.isnan(out[2:4]).all()
