"""GPU tests of attention over the 4-bit cache where a block has many tiles and
several items: stages filled again, sums rescaled on the way, shares that end
inside one item and begin in another.  Against 64-bit arithmetic by the sharp
checks of cache_checks.py."""

import pytest
import torch

import dequant_gemm_int4_b200 as q4
from cache_checks import assert_attention_sharp, attention_64, made_cache, made_table

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def run(H, ratio, D, group, S, lens, counts, dtype, path, *, affine=False, causal=True, window=None, seed=0,
        rising=False):
    table, pages = made_table(lens, S, seed=seed)
    packed, scales, zeros = made_cache(pages, S, H, D, group, affine, seed=seed)
    if rising:  # scores and value scales that grow along the sequences, the latter over 2^10
        place = torch.zeros((pages, S), device="cuda")
        for b, n in enumerate(lens):
            j = torch.arange(n, device="cuda")
            place[table[b, j // S].long(), j % S] = j / max(n, 1)
        place = place[:, None, :, None]
        scales[:, 0] = (scales[:, 0].float() * (0.2 + place)).half()
        scales[:, 1] = (scales[:, 1].float() * torch.exp2(10 * place - 8)).half()
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (0.6 * torch.randn((sum(counts), H * ratio, D), generator=gen, device="cuda")).to(DTYPES[dtype])
    starts = torch.tensor([0, *counts], device="cuda").cumsum(0).int()
    got = q4.int4_cache_attention(q, packed, scales, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                  group, zeros=zeros, q_starts=starts, causal=causal, window=window,
                                  return_lse=True, path=path)
    want = attention_64(q, packed, scales, zeros, table, lens, counts, group, causal=causal, window=window or 0)
    assert_attention_sharp(got, want)


MANY = dict(H=8, ratio=8, S=64, lens=[4000, 2500, 130], counts=[700, 300, 1])  # 6000 tiles for 148 blocks


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D, group", [(64, 64), (64, 32), (96, 96), (96, 32), (128, 128), (128, 64), (128, 32)])
def test_many_rows(D, group, dtype, affine):
    run(**MANY, D=D, group=group, dtype=dtype, affine=affine, path=q4.PATH_PREFILL, seed=D + group)


@pytest.mark.parametrize("causal, window", [(True, 1500), (True, 70), (False, None), (False, 900)])
@pytest.mark.parametrize("D, group, dtype", [(128, 128, "bf16"), (64, 32, "f16")])
def test_many_rows_masked(D, group, dtype, causal, window):
    run(**MANY, D=D, group=group, dtype=dtype, causal=causal, window=window, path=q4.PATH_PREFILL)


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("D, group, dtype", [(128, 128, "bf16"), (128, 32, "f16"), (96, 32, "bf16"), (64, 64, "f16")])
def test_many_rows_rising(D, group, dtype, affine):
    run(**MANY, D=D, group=group, dtype=dtype, affine=affine, rising=True, path=q4.PATH_PREFILL)


def test_many_rows_of_one_long_sequence():
    """One item in many blocks: 200 tiles of tokens to each."""
    run(1, 2, 128, 128, 32, [25600], [100], "bf16", q4.PATH_PREFILL)


# Up to 24 sequences: 5 steps a block and more, so that the ring of copies is filled again.
LENS = [16000, 9000, 130, 0, 2500, 12000, 1, 7777, 4096, 15000, 64, 11111] * 2


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("rows", [8, 16, 32])
@pytest.mark.parametrize("D, group", [(64, 64), (64, 32), (96, 96), (96, 32), (128, 128), (128, 64), (128, 32),
                                      (256, 256), (256, 64), (256, 32)])
def test_few_rows(D, group, rows, affine):
    """Tiles of 8, 16 and 32 rows (of 256 elements: 8 and 16)."""
    lens, counts = (LENS, [rows // 4] * 24) if rows < 32 else (LENS[:8], [8] * 8)
    run(8, 4, D, group, 64, lens, counts, "f16" if affine else "bf16", q4.PATH_DECODE, affine=affine, seed=rows)


@pytest.mark.parametrize("D, group, dtype, rows", [(128, 128, "bf16", 8), (128, 32, "f16", 16), (64, 64, "f16", 32),
                                                   (256, 128, "bf16", 8)])
@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("window", [None, 3000])
def test_few_rows_masked_and_rising(D, group, dtype, rows, window, rising):
    run(8, 4, D, group, 16, LENS[:12], [rows // 4] * 12, dtype, q4.PATH_DECODE, window=window, rising=rising,
        affine=rising)


def test_few_rows_of_one_long_sequence():
    run(4, 8, 128, 32, 128, [100003], [1], "bf16", q4.PATH_DECODE)
    run(4, 8, 128, 128, 128, [100003], [3], "f16", q4.PATH_DECODE, affine=True)


def test_general_kernel():
    run(4, 4, 80, 16, 24, [700, 333, 0], [5, 1, 2], "bf16", q4.PATH_SIMT, affine=True)
    run(2, 16, 512, 128, 64, [2000], [2], "f16", q4.PATH_SIMT)


def many_rows_setup(seed):
    lens, counts = [900, 1700], [150, 90]
    table, pages = made_table(lens, 64, seed=seed)
    packed, scales, zeros = made_cache(pages, 64, 4, 128, 128, True, seed=seed)
    q = torch.randn((240, 16, 128), generator=torch.Generator().manual_seed(seed)).cuda().bfloat16()
    starts = torch.tensor([0, 150, 240], dtype=torch.int32, device="cuda")
    return q, packed, scales, zeros, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), starts


def test_many_rows_on_streams_and_in_graphs():
    """Two streams at once, and captured calls replayed at once, with other lengths and in a chain."""
    def call(x, **kw):
        q, packed, scales, zeros, table, lens, starts = x
        return q4.int4_cache_attention(q, packed, scales, table, lens, 128, zeros=zeros, q_starts=starts,
                                       return_lse=True, path=q4.PATH_PREFILL, **kw)
    sets = [many_rows_setup(s) for s in (1, 2)]
    want = [call(x) for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (s, x) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(s):
                got[i].append(call(x))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for y in got[i] for a, b in zip(y, want[i]))
    graphs, outs = [], []
    for x in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(x))
        graphs.append(g)
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for y, w in zip(outs, want) for a, b in zip(y, w))
    sets[0][0].neg_()
    sets[0][5].copy_(torch.tensor([300, 1699], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], call(sets[0])))
    assert q4.device_status() == q4.OK


def test_many_rows_past_four_gigabytes():
    """Offsets beyond 32 bits: the last pages of a cache of 4.6 GB of codes."""
    H, D, S, P, n = 8, 128, 64, 70000, 200
    small = made_cache(4, S, H, D, 128, False)
    packed = torch.zeros((P, 2, H, S, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((P, 2, H, S, 1), dtype=torch.float16, device="cuda")
    at = [P - 1, 5, P - 2, P - 3]
    packed[at], scales[at] = small[0], small[1]
    q = torch.randn((100, 16, D), generator=torch.Generator().manual_seed(0)).cuda().bfloat16()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    call = lambda c, pages: q4.int4_cache_attention(  # noqa: E731
        q, c[0], c[1], torch.tensor([pages], dtype=torch.int32, device="cuda"), lens, 128, return_lse=True,
        path=q4.PATH_PREFILL)
    for a, b in zip(call((packed, scales), at), call(small, [0, 1, 2, 3])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("D, group, ratio", [(64, 64, 8), (128, 128, 3), (128, 32, 8), (96, 96, 1), (256, 256, 4),
                                             (256, 32, 8)])
@pytest.mark.parametrize("window", [None, 100])
def test_few_rows_kernel_on_many_row_tiles(D, group, ratio, window, affine):
    """Several row tiles a sequence, split items among them, rows that see nothing, a mixed batch."""
    run(2, ratio, D, group, 32, [3000, 40, 0, 700, 1500], [333, 60, 7, 1, 90], "f16" if affine else "bf16",
        q4.PATH_DECODE, affine=affine, window=window)
    run(2, ratio, D, group, 64, [900] + [500] * 40, [200] + [1] * 40, "bf16", q4.PATH_DECODE, affine=affine,
        window=window)


@pytest.mark.parametrize("D, counts", [(256, 1), (128, 1), (64, 4)])
def test_the_few_rows_kernel_is_linear_in_its_rows(D, counts):
    """Four times the rows, each of which sees 64 tokens, in less than eight times the time."""
    times = []
    for rows in (4096, 16384):
        table, pages = made_table([rows], 64)
        packed, scales, _ = made_cache(pages, 64, 4, D, D, False)
        q = torch.randn((rows, 32, D), device="cuda").bfloat16()
        starts = torch.tensor([0] * counts + [rows], dtype=torch.int32, device="cuda")
        table, lens = table.repeat(counts, 1), torch.full((counts,), rows, dtype=torch.int32, device="cuda")
        best = 1e30
        for _ in range(5):
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            begin.record()
            q4.int4_cache_attention(q, packed, scales, table, lens, D, q_starts=starts, window=64, path=q4.PATH_DECODE)
            end.record()
            torch.cuda.synchronize()
            best = min(best, begin.elapsed_time(end))
        times.append(best)
    assert times[1] < 8 * times[0], times
