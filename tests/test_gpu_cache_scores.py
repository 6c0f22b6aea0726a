"""GPU tests of attention over the 4-bit cache with scores far from 1."""

import math

import pytest
import torch

import dequant_gemm_int4_b200 as q4
from cache_checks import assert_attention_sharp, attention_64, made_cache, made_table, token_rows

pytestmark = pytest.mark.gpu

PATHS = [q4.PATH_SIMT, q4.PATH_DECODE, q4.PATH_PREFILL]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("D, group, dtype", [(128, 128, torch.bfloat16), (64, 32, torch.float16),
                                             (96, 96, torch.float16), (128, 32, torch.bfloat16)])
@pytest.mark.parametrize("magnitude", [1e5, 5e6, 3e7, 1e8, 3e9, 1e15, 1e30])
def test_large_scores(magnitude, D, group, dtype, path):
    """A row whose best score is ahead of the next by more than S can be off
    takes that token's value, and its score as lse, however large the score."""
    lens, counts = [700, 130, 33, 1], [40, 40, 30, 1]
    table, pages = made_table(lens, 32)
    packed, scales, zeros = made_cache(pages, 32, 2, D, group, D == 96)
    q = torch.randn((sum(counts), 16, D), generator=torch.Generator().manual_seed(2)).cuda().to(dtype)
    typical = 1.4 * math.sqrt(D)
    sm_scale = magnitude / typical
    starts = torch.tensor([0, *counts], device="cuda").cumsum(0).int()
    out, lse = q4.int4_cache_attention(q, packed, scales, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                       group, zeros=zeros, q_starts=starts, sm_scale=sm_scale, return_lse=True,
                                       path=path)
    sm_scale = torch.tensor(sm_scale, dtype=torch.float32).item()
    want, want_lse, _, _ = attention_64(q, packed, scales, zeros, table, lens, counts, group, sm_scale=sm_scale)
    gap, size = best_scores(q, packed, scales, zeros, table, lens, counts, group, sm_scale)
    held = torch.isfinite(want_lse)
    assert torch.equal(torch.isfinite(lse), held) and torch.isfinite(out).all()
    # S is off by at most D + 64 roundings of 2^-23 of its terms' sizes, which
    # their partial sums do not pass.
    off = (D + 64) * 2.0 ** -23 * size
    assert ((lse.double() - want_lse).abs() <= off + 2.0 ** -20 + 2.0 ** -21 * want_lse.abs())[held].all()
    # Sure of its token: the second stays behind by e^60 whatever S is off by.
    sure = held & (gap > 2 * off + 60)
    assert sure.float().mean() > (0.2 if magnitude < 1e6 else 0.8)
    # One rounding of the weight and one of the value to fp16, one of the
    # output; fp32 sums of terms below 30 s.
    tol = (torch.finfo(dtype).eps / 2 + 2.0 ** -10 + 2.0 ** -18) * want.abs() + 2.0 ** -18
    assert ((out.double() - want).abs() <= tol)[sure].all()


def best_scores(q, packed, scales, zeros, table, lens, counts, group, sm_scale):
    """How far the best visible score of each (row, head) is ahead of the
    second (infinitely, of one token alone), and the largest size of a token's terms."""
    H, S, D = packed.shape[2], packed.shape[3], q.shape[2]
    gap = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    size = torch.zeros_like(gap)
    row = 0
    for n, m, pages in zip(lens, counts, table):
        at, row = slice(row, row + m), row + m
        j = torch.arange(n, device="cuda")
        k, k_size = token_rows(packed, scales, zeros, pages[j // S].long(), 0, j % S, D, group)
        x, ratio = q[at].double(), q.shape[1] // H
        s = torch.einsum("thd,jhd->thj", x, k.repeat_interleave(ratio, 1)) * sm_scale
        pos = n - m + torch.arange(m, device="cuda")
        s = s.masked_fill((j[None] > pos[:, None])[:, None], -math.inf)
        best = s.topk(min(2, n), dim=-1).values
        gap[at] = best[..., 0] - best[..., 1] if n > 1 else math.inf
        size[at] = sm_scale * x.norm(dim=2) * k_size.norm(dim=2).amax(0).repeat_interleave(ratio)
    return gap.nan_to_num(0.0, math.inf, 0.0), size


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("code", [-3, 0, 5])
def test_infinite_query_makes_its_row_nan(code, bad, dtype, path):
    """Whatever the sign of its products: here every key's element is the same,
    so that all scores of the row are minus infinity, NaN or infinity alike.  A
    row that sees no token is 0 all the same, and the other rows stay right."""
    if dtype == torch.float32 and path != q4.PATH_SIMT:
        pytest.skip("fp32 queries take the general kernel")
    lens, counts = [300, 0, 2], [5, 2, 4]  # the last sequence's first two rows see nothing
    table, pages = made_table(lens, 16)
    packed, scales, _ = made_cache(pages, 16, 2, 64, 64, False)
    packed[:, 0, :, :, 8] = (packed[:, 0, :, :, 8] & 0x0F) | ((code & 15) << 4)  # element 17
    q = torch.randn((sum(counts), 4, 64), generator=torch.Generator().manual_seed(2)).cuda().to(dtype)
    starts = torch.tensor([0, *counts], device="cuda").cumsum(0).int()

    def call():
        return q4.int4_cache_attention(q, packed, scales, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                       64, q_starts=starts, return_lse=True, path=path)
    clean, clean_q = call(), q.clone()
    rows = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    rows[[1, 4, 5, 7, 8, 9, 10], [0, 3, 1, 2, 1, 0, 3]] = True
    q[:, :, 17].masked_fill_(rows, bad)
    out, lse = call()
    empty = torch.isinf(clean[1])
    assert empty.sum() == 4 * 4
    assert torch.isnan(out[rows & ~empty]).all() and torch.isnan(lse[rows & ~empty]).all()
    assert (out[empty] == 0).all() and torch.equal(lse[empty], clean[1][empty])
    if path == q4.PATH_PREFILL:  # 32 rows move their reference together, so that the others may round anew
        out, lse = torch.where(rows[..., None], clean[0], out), torch.where(rows, clean[1], lse)
        assert_attention_sharp((out, lse), attention_64(clean_q, packed, scales, None, table, lens, counts, 64))
    else:
        assert torch.equal(out[~rows], clean[0][~rows]) and torch.equal(lse[~rows], clean[1][~rows])
