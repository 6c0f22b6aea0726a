"""GPU tests of the 4-bit cache at the ends of its 32-bit counts."""

import pytest
import torch

import dequant_gemm_int4_b200 as q4
from cache_checks import made_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 4, 2 ** 31 - 6])
def test_general_kernel_at_the_longest_sequence(n):
    """Positions up to 2^31 - 2, of which a window sees the last ones; the pages before are all one page."""
    S, D, window = 1 << 20, 8, 9
    packed, scales, zeros = made_cache(2, S, 1, D, 4, True)
    table = torch.zeros((1, 2048), dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    q = torch.randn((3, 2, D), generator=torch.Generator().manual_seed(0)).cuda()
    call = lambda t, length: q4.int4_cache_attention(  # noqa: E731
        q, packed, scales, t, torch.tensor([length], dtype=torch.int32, device="cuda"), 4, zeros=zeros,
        q_starts=torch.tensor([0, 3], dtype=torch.int32, device="cuda"), window=window, return_lse=True)
    got = call(table, n)
    # The last page alone holds all that the window sees, at the same offsets.
    want = call(table[:, -1:], n - 2047 * S)
    # Warps take tokens in turn from the first one seen on, in both calls alike.
    assert all(torch.equal(a, b) for a, b in zip(got, want))
