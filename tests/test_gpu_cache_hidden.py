"""GPU tests that places which no query sees have no effect on attention over
the 4-bit cache: large finite scales there, and whatever an earlier kernel
left in shared memory."""

import pytest
import torch

import dequant_gemm_int4_b200 as q4
from cache_checks import assert_attention_sharp, attention_64, made_cache, made_table

pytestmark = pytest.mark.gpu

PATHS = [q4.PATH_SIMT, q4.PATH_DECODE, q4.PATH_PREFILL]


def fill_shared_memory(path):
    """Leaves the largest value scales in the shared memory of every SM."""
    packed, scales, zeros = made_cache(64, 64, 8, 128, 32, True, seed=9)
    scales.fill_(65504.0)
    table = torch.arange(64, dtype=torch.int32, device="cuda").repeat(32, 1)
    q = torch.zeros((64, 64, 128), dtype=torch.bfloat16, device="cuda")
    lens = torch.full((32,), 4096, dtype=torch.int32, device="cuda")
    q4.int4_cache_attention(q, packed, scales, table, lens, 32, zeros=zeros, path=path)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
@pytest.mark.parametrize("D, group, queries", [(128, 128, 1), (64, 32, 1), (96, 32, 5), (128, 32, 9), (64, 64, 30)])
@pytest.mark.parametrize("window", [None, 20])
def test_hidden_scales_do_not_count(D, group, queries, page_size, path, window):
    """Past the sequences' ends, before a window, in pages of nobody: bit for
    bit the same with scales of 65504 there, beside visible ones near 1e-4."""
    lens = [70, 33, 150, 64, 290, 1]
    table, pages = made_table(lens, page_size)
    packed, scales, zeros = made_cache(pages, page_size, 2, D, group, D == 96)
    scales[:, 1] = (scales[:, 1].float() * 3e-4).half()
    table = torch.cat([table, torch.full((len(lens), 40), -1, dtype=torch.int32, device="cuda")], 1)
    q = torch.randn((queries * len(lens), 8, D), generator=torch.Generator().manual_seed(1)).cuda().half()
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def call():
        return q4.int4_cache_attention(q, packed, scales, table, lens_t, group, zeros=zeros, window=window,
                                       return_lse=True, path=path)
    clean = call()
    assert_attention_sharp(clean, attention_64(q, packed, scales, zeros, table, lens, [queries] * len(lens), group,
                                               window=window or 0))
    hidden = torch.ones((pages, page_size), dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        j = torch.arange(max(0, n - (window + queries - 1 if window else n)), n, device="cuda")
        hidden[table[b, j // page_size].long(), j % page_size] = False
    scales.masked_fill_(hidden[:, None, None, :, None], 65504.0)
    dirty = call()
    fill_shared_memory(path)
    again = call()
    for a, b, c in zip(clean, dirty, again):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("page_size", [16, 32, 64])
def test_pages_that_are_not_there_do_not_count(page_size, path):
    """Unknown pages between known ones, whose places in shared memory hold an earlier kernel's scales."""
    lens = [200, 290]
    table, pages = made_table(lens, page_size)
    packed, scales, zeros = made_cache(pages, page_size, 2, 128, 128, False)
    scales[:, 1] = (scales[:, 1].float() * 3e-4).half()
    table[0, 1], table[1, 2], table[1, 0] = -3, pages, 1 << 30
    q = torch.randn((4, 8, 128), generator=torch.Generator().manual_seed(1)).cuda().half()
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = []
    for _ in range(2):
        got.append(q4.int4_cache_attention(q, packed, scales, table, lens_t, 128, return_lse=True, path=path))
        fill_shared_memory(path)
    got.append(q4.int4_cache_attention(q, packed, scales, table, lens_t, 128, return_lse=True, path=path))
    assert all(torch.equal(x[i], got[0][i]) for x in got for i in (0, 1))
