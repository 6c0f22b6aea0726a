"""GPU tests of the 4-bit cache at the ends of its 32-bit counts."""

import pytest
import torch

import dequant_gemm_int4_b200 as q4
from cache_checks import assert_attention_sharp, attention_64, made_cache

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


@pytest.mark.parametrize("affine", [False, True])
def test_more_heads_than_2_to_30(affine):
    """Rows of a token (keys and values of all heads) counted beyond 2^31."""
    H, D = 2 ** 30 + 5, 1
    cache = q4.Int4KVCache(1, 1, H, D, scheme="affine" if affine else "symmetric")
    x = torch.zeros((2, 1, H, D), dtype=torch.float16, device="cuda")
    at = torch.tensor([0, 1, 7, 2 ** 29, 2 ** 30 - 1, 2 ** 30, H - 2, H - 1], device="cuda")
    x[:, 0, at, 0] = torch.arange(1, 17, device="cuda").half().view(2, 8) * 0.07
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    cache.write(x[0], x[1], slots)
    got = cache.read(slots, torch.float16)
    small = q4.Int4KVCache(1, 1, 8, D, scheme="affine" if affine else "symmetric")
    small.write(x[0][:, at], x[1][:, at], slots)
    for i, (a, b) in enumerate(zip(got, small.read(slots, torch.float16))):
        assert torch.equal(a[:, at], b) and (b != 0).any() != affine
        assert a.count_nonzero() == b.count_nonzero()
        assert torch.equal(cache.packed[0, i, at, 0], small.packed[0, i, :, 0])
        assert torch.equal(cache.scales[0, i, at, 0], small.scales[0, i, :, 0])


def test_a_large_prompt_through_a_window():
    """131072 rows on 262144 tokens: many steps in the table, few in the window."""
    rows, n, D, H, S = 131072, 262144, 64, 2, 128
    packed, scales, zeros = made_cache(n // S, S, H, D, 64, False)
    table = torch.randperm(n // S, generator=torch.Generator().manual_seed(1)).int().cuda()[None]
    q = torch.randn((rows, 32, D), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").bfloat16()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = q4.int4_cache_attention(q, packed, scales, table, lens, 64, window=100, return_lse=True)
    for first in (0, 70000, rows - 50):  # 50 rows at a time, their last token the sequence's last
        part = slice(first, first + 50)
        length = n - rows + first + 50
        first_page = max(0, length - 200) // S  # what the window does not reach left out
        want = attention_64(q[part], packed, scales, zeros, table[:, first_page:], [length - first_page * S], [50], 64,
                            window=100)
        assert_attention_sharp((out[part], lse[part]), want)
    assert q4.device_status() == q4.OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D, group", [(128, 32), (64, 64), (80, 48), (33, 7)])
def test_write_codes_as_the_weight_quantizers_at_any_size(D, group, dtype):
    """The cache codes its rows in arithmetic of its own: the same bits as
    quantize_int4 and quantize_int4_affine from fp16's subnormal scales to its
    largest, for groups far from 0, constant groups and single large elements."""
    T, H = 2048, 4
    gen = torch.Generator(device="cuda").manual_seed(D)
    x = torch.randn((T, H, D), generator=gen, device="cuda")
    most = 14 if dtype == torch.float16 else 17
    x *= torch.exp2(torch.randint(-30, most, (T, H, 1), generator=gen, device="cuda").float())
    x[::5] += x[::5].abs().amax(-1, keepdim=True) * torch.exp2(torch.randint(-8, 2 if most == 14 else 9, (len(x[::5]), H, 1),
                                                                           generator=gen, device="cuda").float())
    x[1::7, :, ::3] = 0.5
    x[2::11, :, D // 2] *= 100.0
    x = x.clamp(-6e4, 6e4) if dtype == torch.float16 else x.clamp(-4e5, 4e5)
    x = x.to(dtype)
    for scheme, f in (("symmetric", q4.quantize_int4), ("affine", q4.quantize_int4_affine)):
        y = x if scheme == "symmetric" else x.clamp(-2e5, 2e5)
        cache = q4.Int4KVCache(T // 64, 64, H, D, group=group, scheme=scheme)
        cache.write(y, y.flip(0), torch.arange(T, device="cuda"))
        for i, z in enumerate((y, y.flip(0))):
            for got, ref in zip(cache.buffers(), f(z.reshape(-1, D).contiguous(), group)[:-1]):
                got = got[:, i].transpose(1, 2).reshape(T * H, -1)
                assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))


def test_read_refuses_outputs_that_overlap():
    """The keys' and the values' rows would be written over one another."""
    cache = q4.Int4KVCache(2, 16, 2, 64)
    slots = torch.arange(8, device="cuda")
    both = torch.empty((24, 2, 64), dtype=torch.bfloat16, device="cuda")
    args = (cache.packed, cache.scales, slots, 64, 64, torch.bfloat16)
    for k, v in ((both[:8], both[:8]), (both[:8], both[4:12]), (both[15:23], both[8:16])):
        with pytest.raises(ValueError, match="overlap"):
            q4.int4_cache_read(*args, out=(k, v))
    assert q4.int4_cache_read(*args, out=(both[:8], both[8:16]))[1].shape == (8, 2, 64)
    none = both[:0]
    q4.int4_cache_read(cache.packed, cache.scales, slots[:0], 64, 64, torch.bfloat16, out=(none, none))
