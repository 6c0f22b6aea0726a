"""The checks of cache_checks.py: they agree with cache_util.py's arithmetic
and see what its bounds for each element do not.  No GPU needed."""

import pytest
import torch

from cache_checks import assert_attention_sharp, attention_64, made_cache, made_table, token_rows
from cache_util import attention_ref, random_cache, value_rows


def setup(n, D=64, group=64, H=4, ratio=8, affine=False, seed=0):
    table, pages = made_table([n], 64, seed=seed, device="cpu")
    packed, scales, zeros = made_cache(pages, 64, H, D, group, affine, seed=seed, device="cpu")
    q = torch.randn((1, H * ratio, D), generator=torch.Generator().manual_seed(seed))
    return q, packed, scales, zeros, table, group


@pytest.mark.parametrize("affine", [False, True])
def test_values_are_the_oracles(affine):
    packed, scales, zeros = random_cache(3, 4, 2, 10, 4, affine, device="cpu")
    page, offset = torch.tensor([2, 0, 1]), torch.tensor([3, 1, 0])
    for kv in (0, 1):
        got, size = token_rows(packed, scales, zeros, page, kv, offset, 10, 4)
        pick = lambda t: t[page, kv, :, offset].reshape(-1, t.shape[-1]).numpy()  # noqa: E731
        ref = value_rows(pick(packed), pick(scales), pick(zeros) if affine else None, 10, 4)
        assert torch.equal(got.reshape(-1, 10), torch.from_numpy(ref))
        assert (size >= got.abs()).all()


@pytest.mark.parametrize("causal, window", [(True, 0), (True, 7), (False, 0), (False, 30)])
def test_attention_is_the_other_reference(causal, window):
    table, pages = made_table([50, 3], 16, device="cpu")
    packed, scales, zeros = made_cache(pages, 16, 2, 24, 8, True, device="cpu")
    q = torch.randn((9, 4, 24), generator=torch.Generator().manual_seed(1))
    args = (q, packed, scales, zeros, table, [50, 3], [4, 5], 8)
    out, lse, _, _ = attention_64(*args, causal=causal, window=window)
    ref, ref_lse, _, _ = attention_ref(*args, causal=causal, window=window)
    assert torch.allclose(out, ref, atol=1e-12) and torch.allclose(lse, ref_lse, atol=1e-12)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D, group", [(64, 64), (128, 32)])
def test_the_sharp_check_sees_small_faults(D, group, dtype):
    q, packed, scales, zeros, table, group = setup(4097, D, group)
    q = q.to(dtype)
    want = attention_64(q, packed, scales, zeros, table, [4097], [1], group)
    out, lse = want[0], want[1].float()
    assert_attention_sharp((out.to(dtype), lse), want)
    for window, match in ((4096, "lse is"), (4033, "out is")):  # the first token missing, the first 64
        less = attention_64(q, packed, scales, zeros, table, [4097], [1], group, causal=False, window=window)
        with pytest.raises(AssertionError, match=match):
            assert_attention_sharp((less[0].to(dtype), less[1].float() if match == "lse is" else lse), want)
    with pytest.raises(AssertionError, match="out is"):
        assert_attention_sharp(((out * (1 + 2.0 ** -7)).to(dtype), lse), want)
    with pytest.raises(AssertionError):
        assert_attention_sharp((out.to(dtype), lse + 1e-4), want)
