"""GPU tests of attention over the 4-bit cache where the weights are spread over
many tokens: outputs are then far smaller than the values, and so has to be
what the sums are off by."""

import pytest
import torch

import dequant_gemm_int4_b200 as q4
from cache_checks import assert_attention_sharp, attention_64, made_cache, made_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path", [q4.PATH_DECODE, q4.PATH_PREFILL])
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D, group, queries", [(64, 64, 1), (64, 32, 2), (96, 96, 4), (96, 32, 1), (128, 128, 1),
                                               (128, 64, 2), (128, 32, 4), (256, 256, 1), (256, 64, 2)])
def test_weights_spread_over_many_tokens(D, group, queries, dtype, affine, path):
    if D == 256 and path == q4.PATH_PREFILL:
        pytest.skip("heads of 64 to 128")
    lens = [4096, 1500, 9000]
    table, pages = made_table(lens, 64)
    packed, scales, zeros = made_cache(pages, 64, 4, D, group, affine)
    q = (0.02 * torch.randn((3 * queries, 32, D), generator=torch.Generator().manual_seed(1))).cuda().to(dtype)
    got = q4.int4_cache_attention(q, packed, scales, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), group,
                                  zeros=zeros, return_lse=True, path=path)
    assert_attention_sharp(got, attention_64(q, packed, scales, zeros, table, lens, [queries] * 3, group))


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("n", [1, 2, 16, 64, 700, 4096])
@pytest.mark.parametrize("D, group", [(64, 32), (96, 96), (128, 128), (128, 32), (256, 256)])
def test_values_at_their_zero_point(D, group, n, affine):
    """Outputs whose every value is 0.  The kernel for many rows takes n - z
    first and gives 0; the one for few rows sums the codes and the zero points
    apart, in tensor core steps of 16 tokens.  A step aligns 17 terms at the
    largest and cuts them off 25 bits below; codes are fp16 subnormals and
    count there as 2^-14, z = 8 of them as 2^-21: 17 2^-25 2^7 < 2^-13 of the
    step's sum of w z, once for the codes and once for the zero points; cut off
    to the same side, so that half of it can remain on average of either.  2^-13
    of sum p s z is asked for."""
    table, pages = made_table([n], 64)
    packed, scales, zeros = made_cache(pages, 64, 4, D, group, affine, seed=n)
    packed[:, 1] = 0x88 if affine else 0
    if affine:
        zeros[:, 1] = 8
    q = torch.randn((1, 32, D), generator=torch.Generator().manual_seed(n)).cuda().half()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    call = lambda path: q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros, path=path)  # noqa: E731
    sizes = packed.clone()
    sizes[:, 1] = 0 if affine else 0x88  # values of -8 s: their outputs are the bound's sums
    eight = attention_64(q, sizes, scales, zeros, table, [n], [1], group)[0].abs()
    assert (call(q4.PATH_DECODE).double().abs() <= 2.0 ** -13 * eight).all()
    if D <= 128:
        assert (call(q4.PATH_PREFILL) == 0).all()
    assert (call(q4.PATH_SIMT) == 0).all()
