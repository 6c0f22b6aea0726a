"""GPU tests of the 4-bit key/value cache: writing and reading bit for bit
against the CPU oracle, attention against 64-bit arithmetic within derived
bounds (tests/cache_util.py), masks, empty rows, unused pages, strides,
streams, graphs, and the three operators together between two Int4Linear
layers."""

import math

import numpy as np
import pytest
import torch

import dequant_gemm_int4_b200 as q4
from cache_util import (assert_attention_close, attention_ref, code_rows, page_table, random_cache,
                        value_rows)
from gpu_util import to_np

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def rows_f32(x):
    return to_np(x).astype(np.float32)


def make_kv(tokens, heads, D, dtype, seed, fused):
    """k and v [tokens, heads, D]; fused: slices of one projection's rows."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(tokens, 3 * heads, D)).astype(np.float32)
    x[:, ::4] *= 30.0
    if tokens > 2:
        x[1] = 0.0                    # zero groups
        x[2] = np.abs(x[2]) + 4.0     # one sign: zero points at the border
    x = torch.from_numpy(x).to("cuda").to(dtype)
    k, v = x[:, heads:2 * heads], x[:, 2 * heads:]
    return (k, v) if fused else (k.contiguous(), v.contiguous())


WRITE_CASES = [
    # dtype, tokens, heads, D, group, page_size, pages
    ("bf16", 1, 1, 64, 64, 16, 1),
    ("bf16", 16, 8, 128, 128, 64, 3),
    ("f16", 77, 3, 128, 32, 16, 7),
    ("f32", 33, 5, 64, 32, 7, 9),
    ("bf16", 300, 1, 96, 32, 64, 6),
    ("f16", 41, 2, 256, 256, 32, 2),
    ("f32", 19, 2, 256, 8, 32, 2),
    ("bf16", 23, 4, 80, 80, 16, 2),       # a group that is no power of two
    ("f16", 9, 2, 80, 32, 16, 1),         # a partial last group
    ("f32", 12, 3, 7, 3, 5, 3),           # odd sizes, groups that share a byte
    ("bf16", 8, 1, 1, 1, 16, 1),
    ("bf16", 6, 2, 33, 128, 16, 1),       # a group longer than the head
    ("f32", 5, 2, 511, 100, 16, 1),
    ("f16", 2000, 40, 512, 512, 128, 16),
]


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("case", WRITE_CASES, ids=lambda c: "-".join(map(str, c)))
def test_write_and_read_bit_exact(case, affine):
    name, T, H, D, group, S, P = case
    dtype = DTYPES[name]
    cache = q4.Int4KVCache(P, S, H, D, group=group, scheme="affine" if affine else "symmetric")
    G = -(-D // group)
    cache.packed.fill_(0xA5)
    cache.scales.fill_(3.0)
    if affine:
        cache.zeros.fill_(9)
    before = [x.clone() for x in cache.buffers()]
    k, v = make_kv(T, H, D, dtype, seed=T + D, fused=T % 2 == 1)
    slots = torch.from_numpy(np.random.default_rng(T).permutation(P * S)[:T].astype(np.int64)).cuda()
    if T >= 8:  # padding: tokens that are not written
        slots[3], slots[T - 1] = -1, P * S
    cache.write(k, v, slots)
    live = ((slots >= 0) & (slots < P * S)).cpu()
    page, offset = (slots[live.cuda()] // S).cpu(), (slots[live.cuda()] % S).cpu()
    want = [x.cpu() for x in before]
    for i, x in enumerate((k, v)):
        p, s, z = code_rows(rows_f32(x)[live.numpy()].reshape(-1, D), group, affine)
        n = int(live.sum())
        want[0][page, i, :, offset] = torch.from_numpy(p.reshape(n, H, -1))
        want[1][page, i, :, offset] = torch.from_numpy(s.reshape(n, H, G))
        if affine:
            want[2][page, i, :, offset] = torch.from_numpy(z.reshape(n, H, G))
    for got, ref, what in zip(cache.buffers(), want, ("packed", "scales", "zeros")):
        got = got.cpu()
        if what == "scales":
            got, ref = got.view(torch.int16), ref.view(torch.int16)
        assert torch.equal(got, ref), what  # slots that were not written included

    # Read back: repeated slots, slots outside, each output type.
    ask = torch.cat([slots, slots[:2], torch.tensor([-5, P * S + 7, 1 << 40], device="cuda")])
    inside = ((ask >= 0) & (ask < P * S)).cpu()
    at = ask.cpu()[inside]
    for out_dtype in DTYPES.values():
        got = cache.read(ask, out_dtype)
        for i, x in enumerate(got):
            assert x.dtype == out_dtype and x.shape == (ask.numel(), H, D)
            pick = lambda t: t[at // S, i, :, at % S].reshape(-1, t.shape[-1]).numpy()  # noqa: E731
            ref = value_rows(pick(want[0]), pick(want[1]), pick(want[2]) if affine else None, D, group)
            ref = torch.from_numpy(ref.astype(np.float32)).to(out_dtype).reshape(-1, H, D)
            assert torch.equal(x.cpu()[inside], ref)
            assert (x.cpu()[~inside] == 0).all()


def test_write_is_quantize_int4_of_the_row():
    """A cache row is what quantize_int4 and quantize_int4_affine give for it."""
    T, H, D, group = 50, 4, 128, 32
    k, v = make_kv(T, H, D, torch.bfloat16, 5, True)
    slots = torch.arange(T, device="cuda")
    for scheme, f in (("symmetric", q4.quantize_int4), ("affine", q4.quantize_int4_affine)):
        cache = q4.Int4KVCache(1, 64, H, D, group=group, scheme=scheme)
        cache.write(k, v, slots)
        for i, x in enumerate((k, v)):
            parts = f(x.reshape(-1, D).contiguous(), group)[:-1]
            for got, ref in zip(cache.buffers(), parts):
                assert torch.equal(got[0, i, :, :T].transpose(0, 1).reshape(T * H, -1), ref)


def test_write_extreme_values():
    """Scales that underflow, that are fp16 subnormals, that are infinite, and
    groups far from zero whose quotients are huge, as the oracle codes them."""
    D, group = 64, 32
    base = np.linspace(-1.0, 1.0, D, dtype=np.float32)
    rows = np.stack([base * m for m in (1e-12, 2e-7, 4e-7, 3e-6, 1e-3, 4e5, 3e6, 1e30)]
                    + [1000.0 + base * 1e-3, -3e30 + 0 * base, np.where(base > 0.9, 1.0, 0.0).astype(np.float32)])
    k = torch.from_numpy(rows.astype(np.float32)).cuda().unsqueeze(1)
    slots = torch.arange(len(rows), device="cuda")
    for affine in (False, True):
        if affine:
            k = k[[0, 1, 2, 3, 4, 8, 9, 10]]  # the affine scheme's ranges end at 15 * 65520
            slots = slots[:k.shape[0]]
        cache = q4.Int4KVCache(1, 16, 1, D, group=group, scheme="affine" if affine else "symmetric")
        cache.write(k, k, slots)
        with np.errstate(over="ignore", invalid="ignore"):
            p, s, z = code_rows(rows_f32(k)[:, 0], group, affine)
        n = len(p)
        assert np.array_equal(cache.packed[0, 0, 0, :n].cpu().numpy(), p)
        assert np.array_equal(cache.scales[0, 1, 0, :n].cpu().numpy().view(np.uint16), s.view(np.uint16))
        if affine:
            assert np.array_equal(cache.zeros[0, 0, 0, :n].cpu().numpy(), z)


def run_attention(H, ratio, D, group, S, lens, counts, dtype, *, affine=False, causal=True, window=None,
                  path=q4.PATH_AUTO, seed=0, sm_scale=None, q_scale=1.5, ragged=None):
    pages = sum(-(-n // S) for n in lens) + 2
    packed, scales, zeros = random_cache(pages, S, H, D, group, affine, seed=seed)
    table = page_table(lens, S, pages, seed=seed, extra=1)
    rng = np.random.default_rng(seed + 3)
    q = torch.from_numpy(q_scale * rng.normal(size=(sum(counts), H * ratio, D)).astype(np.float32)).cuda().to(dtype)
    ragged = len(set(counts)) > 1 if ragged is None else ragged
    starts = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda") if ragged else None
    got = q4.int4_cache_attention(q, packed, scales, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                  group, zeros=zeros, q_starts=starts, causal=causal, window=window,
                                  sm_scale=sm_scale, return_lse=True, path=path)
    want = attention_ref(q, packed, scales, zeros, table, lens, counts, group, causal=causal,
                         window=window or 0, sm_scale=sm_scale)
    assert_attention_close(got, want)


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("D, group, dtype, path", [
    (64, 32, "bf16", q4.PATH_DECODE), (64, 64, "f16", q4.PATH_DECODE),
    (96, 32, "f16", q4.PATH_DECODE), (96, 96, "bf16", q4.PATH_DECODE),
    (128, 32, "bf16", q4.PATH_DECODE), (128, 64, "f16", q4.PATH_DECODE), (128, 128, "bf16", q4.PATH_DECODE),
    (256, 32, "bf16", q4.PATH_DECODE), (256, 64, "f16", q4.PATH_DECODE), (256, 128, "bf16", q4.PATH_DECODE),
    (256, 256, "f16", q4.PATH_DECODE),
    (128, 128, "bf16", q4.PATH_SIMT), (64, 32, "f32", q4.PATH_AUTO), (80, 80, "bf16", q4.PATH_AUTO),
    (72, 16, "f16", q4.PATH_AUTO), (7, 3, "f32", q4.PATH_AUTO), (512, 128, "bf16", q4.PATH_AUTO),
    (1, 1, "bf16", q4.PATH_AUTO), (33, 64, "f16", q4.PATH_AUTO),
])
@pytest.mark.parametrize("ratio, counts", [
    (1, [1, 1, 1, 1, 1]),      # a row a sequence
    (5, [1, 1, 1, 1, 1]),      # fewer rows than a tile
    (4, [3, 1, 7, 2, 5]),      # tiles of 32 rows, unevenly filled
    (3, [4, 4, 4, 4, 4]),
])
def test_attention(D, group, dtype, path, affine, ratio, counts):
    run_attention(2, ratio, D, group, 16, [37, 1, 300, 129, 64], counts, DTYPES[dtype], affine=affine, path=path)


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("D, group, dtype", [(64, 64, "bf16"), (64, 32, "f16"), (96, 96, "f16"), (96, 32, "bf16"),
                                             (128, 128, "bf16"), (128, 128, "f16"), (128, 64, "f16"), (128, 32, "bf16")])
@pytest.mark.parametrize("H, ratio, lens, counts", [
    (1, 1, [128], [128]),                       # one tile of keys, one of rows
    (1, 1, [1], [1]),
    (2, 4, [500, 37, 300], [100, 37, 1]),
    (1, 8, [1500, 129], [200, 70]),             # several row tiles
    (3, 3, [1000], [333]),                      # a ratio that does not divide the tile
    (2, 1, [3000, 5], [600, 9]),                # a sequence of fewer tokens than queries
])
def test_attention_many_rows(D, group, dtype, affine, H, ratio, lens, counts):
    run_attention(H, ratio, D, group, 32, lens, counts, DTYPES[dtype], affine=affine, path=q4.PATH_PREFILL)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 65, 127, 128, 129, 255, 257, 1000, 4097])
def test_attention_lengths(n):
    run_attention(1, 8, 64, 64, 64, [n], [1], torch.bfloat16, seed=n)
    run_attention(3, 1, 128, 128, 32, [n, max(1, n - 1)], [1, 1], torch.float16, affine=True, seed=n)


@pytest.mark.parametrize("page_size", [1, 3, 8, 16, 24, 32, 64, 256, 1024])
def test_attention_page_sizes(page_size):
    """Powers of two from 16 on take the tensor-core kernels, others the general one."""
    run_attention(2, 4, 64, 32, page_size, [333, 40, 7], [1, 1, 1], torch.bfloat16, seed=page_size)


@pytest.mark.parametrize("path", [q4.PATH_SIMT, q4.PATH_DECODE, q4.PATH_PREFILL])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [None, 1, 2, 31, 100, 5000])
def test_attention_masks(path, causal, window):
    """Windows and causality, with queries before the first token (rows that see nothing)."""
    run_attention(2, 2, 64, 64, 16, [200, 5, 0, 64, 90], [9, 12, 3, 1, 40], torch.bfloat16, causal=causal,
                  window=window, path=path, seed=window or 0)


@pytest.mark.parametrize("ratio, count", [(1, 8), (1, 9), (2, 8), (1, 17), (16, 1), (16, 2), (32, 1), (40, 1),
                                          (7, 5), (1, 33), (2, 100)])
@pytest.mark.parametrize("D", [64, 256])
def test_attention_row_tiles(ratio, count, D):
    """Row counts around the tiles of 8, 16 and 32 rows, and several tiles."""
    run_attention(2, ratio, D, 64, 32, [150, 260], [count, count], torch.bfloat16, seed=count)


@pytest.mark.parametrize("batch", [127, 128, 129, 300])
def test_attention_many_sequences(batch):
    """More sequences than threads of a block look at together; every seventh empty."""
    rng = np.random.default_rng(batch)
    lens = [0 if b % 7 == 3 else int(rng.integers(1, 200)) for b in range(batch)]
    run_attention(1, 4, 64, 32, 16, lens, [1] * batch, torch.bfloat16, seed=batch)
    run_attention(1, 4, 64, 32, 16, lens, [1 + b % 3 for b in range(batch)], torch.bfloat16, seed=batch)


def test_attention_long_and_short_together():
    """One sequence many blocks long beside short ones: shares begin and end inside items."""
    run_attention(4, 8, 128, 128, 64, [30000, 1, 700, 0, 9000], [1] * 5, torch.bfloat16)
    run_attention(2, 4, 128, 32, 128, [20011], [6], torch.float16, affine=True)


@pytest.mark.parametrize("sm_scale", [0.0, 1.0, -0.2])
def test_attention_scale(sm_scale):
    run_attention(2, 4, 64, 64, 16, [100, 33], [2, 2], torch.bfloat16, sm_scale=sm_scale)


@pytest.mark.parametrize("magnitude", [1e-30, 1e-6, 300.0])
def test_attention_query_magnitudes(magnitude):
    """Queries far from 1, with sm_scale bringing the scores back."""
    dtype = torch.bfloat16 if magnitude != 300.0 else torch.float16
    run_attention(2, 4, 64, 64, 16, [100, 33], [2, 2], dtype, q_scale=magnitude, sm_scale=0.2 / magnitude)


def attention_setup(H=2, ratio=4, D=128, group=128, S=16, lens=(70, 33), seed=1, affine=True, extra=2):
    pages = sum(-(-n // S) for n in lens) + 3
    packed, scales, zeros = random_cache(pages, S, H, D, group, affine, seed=seed)
    table = page_table(lens, S, pages, seed=seed, extra=extra)
    rng = np.random.default_rng(seed)
    q = torch.from_numpy(rng.normal(size=(len(lens), H * ratio, D)).astype(np.float32)).cuda().bfloat16()
    return q, packed, scales, zeros, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), group


@pytest.mark.parametrize("path", [q4.PATH_SIMT, q4.PATH_DECODE, q4.PATH_PREFILL])
def test_attention_hidden_places_do_not_count(path):
    """NaN and infinite scales past the sequences' ends, in pages of nobody,
    and before a window change nothing, bit for bit."""
    q, packed, scales, zeros, table, lens, group = attention_setup()
    for window in (None, 20):
        def call():
            return q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros, window=window,
                                           return_lse=True, path=path)
        clean = call()
        keep = scales.clone()
        mask = torch.ones(scales.shape[0], scales.shape[3], dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens.tolist()):
            j = torch.arange(max(0, n - (window or n)), n, device="cuda")
            mask[table[b, j // 16].long(), j % 16] = False
        bad = mask[:, None, None, :, None].expand_as(scales)
        scales.masked_fill_(bad, math.nan)
        dirty = call()
        scales.masked_fill_(bad, math.inf)
        dirty2 = call()
        scales.copy_(keep)
        for a, b, c in zip(clean, dirty, dirty2):
            assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("path", [q4.PATH_SIMT, q4.PATH_DECODE, q4.PATH_PREFILL])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attention_tokens_hidden_from_some_rows(path, bad):
    """A value scale that is not finite reaches only the rows that see its
    token, a key scale likewise; the other rows of the tile stay right."""
    q, packed, scales, zeros, table, lens, group = attention_setup(lens=(70, 45), ratio=2)
    q = torch.randn((8, 4, 128), generator=torch.Generator().manual_seed(3)).cuda().bfloat16()
    want = attention_ref(q, packed, scales, zeros, table, [70, 45], [4, 4], group)
    for kv in (0, 1):
        dirty = scales.clone()
        dirty[table[0, 68 // 16].long(), kv, :, 68 % 16] = bad  # seen by the last two queries of sequence 0
        out, lse = q4.int4_cache_attention(q, packed, dirty, table, lens, group, zeros=zeros, return_lse=True, path=path)
        assert not torch.isfinite(out[2:4]).any()
        assert torch.isfinite(lse[2:4]).all() if kv else torch.isnan(lse[2:4]).all()
        keep = [0, 1, 4, 5, 6, 7]
        assert_attention_close((out[keep], lse[keep]), tuple(x[keep] for x in want))


@pytest.mark.parametrize("path", [q4.PATH_SIMT, q4.PATH_DECODE, q4.PATH_PREFILL])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("D, group", [(128, 32), (128, 64), (96, 32), (64, 32)])
def test_attention_one_bad_group(D, group, bad, path):
    """One group's scale that is not finite: its token's readers and no other row."""
    q, packed, scales, zeros, table, lens, group = attention_setup(D=D, group=group, lens=(70, 45), ratio=2, affine=False)
    q = torch.randn((8, 4, D), generator=torch.Generator().manual_seed(3)).cuda().bfloat16()
    for kv in (0, 1):
        dirty = scales.clone()
        dirty[table[0, 68 // 16].long(), kv, :, 68 % 16, -1] = bad  # seen by the last two queries of sequence 0
        packed[table[0, 68 // 16].long(), kv, :, 68 % 16, -1] = 0x21  # values that are not 0
        out, lse = q4.int4_cache_attention(q, packed, dirty, table, lens, group, zeros=zeros, return_lse=True, path=path)
        if kv:
            assert not torch.isfinite(out[2:4, :, -2:]).any() and torch.isfinite(lse[2:4]).all()
        else:
            assert not torch.isfinite(lse[2:4]).any() or bad == math.inf
        want = attention_ref(q, packed, scales, zeros, table, [70, 45], [4, 4], group)
        keep = [0, 1, 4, 5, 6, 7]
        assert_attention_close((out[keep], lse[keep]), tuple(x[keep] for x in want))


@pytest.mark.parametrize("path", [q4.PATH_SIMT, q4.PATH_DECODE, q4.PATH_PREFILL])
def test_attention_unknown_pages_hold_no_tokens(path):
    q, packed, scales, zeros, table, lens, group = attention_setup(lens=(200, 33, 64))
    table[0, 2], table[0, 5], table[2, :] = -7, packed.shape[0], 1 << 30
    got = q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros, return_lse=True, path=path)
    assert_attention_close(got, attention_ref(q, packed, scales, zeros, table, lens.tolist(), [1, 1, 1], group))
    assert (got[0][2] == 0).all() and torch.isinf(got[1][2]).all()


@pytest.mark.parametrize("path", [q4.PATH_SIMT, q4.PATH_DECODE, q4.PATH_PREFILL])
def test_attention_lengths_outside_the_table(path):
    """A negative length counts as 0, one past the table as what the table holds."""
    q, packed, scales, zeros, table, lens, group = attention_setup(extra=0, lens=(80, 33))
    got = q4.int4_cache_attention(q, packed, scales, table, torch.tensor([500, -3], dtype=torch.int32, device="cuda"),
                                  group, zeros=zeros, return_lse=True, path=path)
    assert_attention_close(got, attention_ref(q, packed, scales, zeros, table, [80, 0], [1, 1], group))


@pytest.mark.parametrize("path", [q4.PATH_SIMT, q4.PATH_DECODE, q4.PATH_PREFILL])
def test_attention_rows_of_no_sequence_stay(path):
    q, packed, scales, zeros, table, lens, group = attention_setup()
    q = q.repeat(4, 1, 1)
    out, lse = torch.full_like(q, 42.0), torch.full(q.shape[:2], 43.0, device="cuda")
    starts = torch.tensor([2, 3, 5], dtype=torch.int32, device="cuda")
    q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros, q_starts=starts, out=out, lse=lse,
                            path=path)
    assert (out[:2] == 42).all() and (out[5:] == 42).all() and (lse[:2] == 43).all() and (lse[5:] == 43).all()
    want = attention_ref(q, packed, scales, zeros, table, lens.tolist(), [1, 2], group, starts=[2, 3])
    assert_attention_close((out, lse), want)


def test_attention_strided_and_unaligned_queries():
    """Queries inside a fused projection's rows, and rows that start at odd elements."""
    q, packed, scales, zeros, table, lens, group = attention_setup()
    want = q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros)
    fused = torch.zeros(2, 20, 128, dtype=torch.bfloat16, device="cuda")
    fused[:, 5:13] = q
    wide = torch.zeros(2, 8, 131, dtype=torch.bfloat16, device="cuda")
    wide[:, :, 3:] = q
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    rows = torch.full((2, table.shape[1] + 5), 1 << 20, dtype=torch.int32, device="cuda")
    rows[:, 2:2 + table.shape[1]] = table
    for x in (fused[:, 5:13], wide[:, :, 3:], turned):
        assert torch.equal(q4.int4_cache_attention(x, packed, scales, rows[:, 2:2 + table.shape[1]], lens, group,
                                                   zeros=zeros), want)


@pytest.mark.parametrize("path", [q4.PATH_SIMT, q4.PATH_DECODE, q4.PATH_PREFILL])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attention_nan_in_a_query_stays_in_its_rows(path, bad):
    q, packed, scales, zeros, table, lens, group = attention_setup()
    clean = q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros, return_lse=True, path=path)
    q = q.clone()
    q[1, 3, 17] = bad
    got = q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros, return_lse=True, path=path)
    assert torch.isnan(got[0][1, 3]).all() and torch.isnan(got[1][1, 3])
    keep = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    keep[1, 3] = False
    assert torch.equal(got[0][keep], clean[0][keep]) and torch.equal(got[1][keep], clean[1][keep])


def test_attention_many_rows_strided_and_unaligned():
    """The kernel for many rows on queries inside wider rows, aligned and not."""
    q, packed, scales, zeros, table, lens, group = attention_setup(lens=(300, 200))
    q = torch.randn((150, 8, 128), generator=torch.Generator().manual_seed(1)).cuda().bfloat16()
    starts = torch.tensor([0, 100, 150], dtype=torch.int32, device="cuda")
    call = lambda x: q4.int4_cache_attention(x, packed, scales, table, lens, group, zeros=zeros, q_starts=starts,  # noqa: E731
                                             return_lse=True, path=q4.PATH_PREFILL)
    want = call(q)
    assert_attention_close(want, attention_ref(q, packed, scales, zeros, table, [300, 200], [100, 50], group))
    fused = torch.zeros(150, 20, 128, dtype=torch.bfloat16, device="cuda")
    fused[:, 5:13] = q
    wide = torch.zeros(150, 8, 131, dtype=torch.bfloat16, device="cuda")
    wide[:, :, 3:] = q
    for x in (fused[:, 5:13], wide[:, :, 3:]):
        assert all(torch.equal(a, b) for a, b in zip(call(x), want))
    # An output that is not 16-byte aligned: refused when forced, else another kernel's.
    odd = torch.empty(150 * 8 * 128 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(150, 8, 128)
    with pytest.raises(q4.Int4Error, match="cannot run"):
        q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros, q_starts=starts, out=odd,
                                path=q4.PATH_PREFILL)
    q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros, q_starts=starts, out=odd)
    assert_attention_close((odd, want[1]), attention_ref(q, packed, scales, zeros, table, [300, 200], [100, 50], group))


@pytest.mark.parametrize("path", [q4.PATH_SIMT, q4.PATH_DECODE, q4.PATH_PREFILL])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_largest_window(path, causal):
    """A window past every token, with queries before the first one."""
    run_attention(1, 2, 64, 64, 16, [40, 3], [60, 9], torch.bfloat16, causal=causal, window=2 ** 31 + 5, path=path)


@pytest.mark.parametrize("pages", [1, 2, 4, 8, 16, 33, 64])
@pytest.mark.parametrize("batch, H", [(1, 1), (3, 8), (80, 8)])
def test_attention_table_sizes(pages, batch, H):
    """Tables with room for one step to many: joined in clusters of 1 to 8 blocks, or in shares; lengths from 0 to all of it."""
    D, S = 64, 128
    P = 40
    packed, scales, zeros = random_cache(P, S, H, D, 64, False, seed=pages)
    rng = np.random.default_rng(pages + batch)
    table = torch.from_numpy(rng.integers(0, P, (batch, pages)).astype(np.int32)).cuda()  # pages may be shared
    lens = [int(n) for n in rng.integers(0, pages * S + 1, batch)]
    lens[0] = pages * S
    if batch > 1:
        lens[1] = 0
    q = torch.from_numpy(rng.normal(size=(2 * batch, 3 * H, D)).astype(np.float32)).cuda().bfloat16()
    got = q4.int4_cache_attention(q, packed, scales, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), 64,
                                  zeros=zeros, return_lse=True, path=q4.PATH_DECODE)
    assert_attention_close(got, attention_ref(q, packed, scales, zeros, table, lens, [2] * batch, 64))


def test_attention_value_scales_of_all_sizes():
    """Value scales from fp16 subnormals to its largest, growing and shrinking along the sequence."""
    for affine, group in ((False, 128), (True, 128), (False, 32), (True, 64)):
        q, packed, scales, zeros, table, lens, group = attention_setup(H=1, ratio=8, lens=(600, 300), affine=affine, group=group)
        factor = torch.from_numpy(np.exp2(np.random.default_rng(2).integers(-13, 14, scales[:, 1].shape)).astype(np.float32)).cuda()
        scales[:, 1] = (scales[:, 1].float() * factor).half()
        for sm_scale in (0.02, 0.3):
            want = attention_ref(q, packed, scales, zeros, table, [600, 300], [1, 1], group, sm_scale=sm_scale)
            for path in (q4.PATH_DECODE, q4.PATH_PREFILL):
                got = q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros, return_lse=True,
                                              sm_scale=sm_scale, path=path)
                assert_attention_close(got, want)


def test_attention_is_deterministic_and_keeps_nothing():
    q, packed, scales, zeros, table, lens, group = attention_setup(lens=(5000, 3000, 17), S=64, H=4)
    a = q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros, return_lse=True)
    need = q4.cache_attention_workspace_size(q, packed, scales, table, group, zeros=zeros)
    workspace = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # of any content: NaN
    for _ in range(3):
        b = q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros, return_lse=True,
                                    workspace=workspace)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(q4.Int4Error, match="workspace"):
        q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros, workspace=workspace[:-256])
    # Without lse the same output.
    assert torch.equal(q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros), a[0])


def test_attention_on_streams_and_in_graphs():
    """Two streams at once, and captured calls replayed with other lengths and queries."""
    sets = [attention_setup(lens=(3000, 900), seed=s, S=64) for s in (1, 2)]
    want = [q4.int4_cache_attention(*x[:3], *x[4:], zeros=x[3]) for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (s, x) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(s):
                got[i].append(q4.int4_cache_attention(*x[:3], *x[4:], zeros=x[3]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(y, want[i]) for y in got[i])

    graphs, outs = [], []
    for x in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(q4.int4_cache_attention(*x[:3], *x[4:], zeros=x[3]))
        graphs.append(g)
    for s, g in zip(streams, graphs):  # both at once: each has its own workspace
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    q, packed, scales, zeros, table, lens, group = sets[0]
    q.neg_()
    lens.copy_(torch.tensor([17, 800], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], q4.int4_cache_attention(q, packed, scales, table, lens, group, zeros=zeros))


def test_cache_past_four_gigabytes():
    """Offsets beyond 32 bits: the last pages of a cache of 4.6 GB of codes."""
    H, D, S, P = 8, 128, 64, 70000
    cache = q4.Int4KVCache(P, S, H, D)
    n = 200
    table = torch.tensor([[P - 1, 5, P - 2, P - 3]], dtype=torch.int32, device="cuda")
    j = torch.arange(n, device="cuda")
    slots = table[0, j // S].long() * S + j % S
    k, v = make_kv(n, H, D, torch.bfloat16, 3, True)
    cache.write(k, v, slots)
    got = cache.read(slots)
    small = q4.Int4KVCache(4, S, H, D)
    small.write(k, v, j)
    for a, b in zip(got, small.read(j)):
        assert torch.equal(a, b)
    q = torch.randn(1, 16, D, device="cuda").bfloat16()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    order = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    for path in (q4.PATH_SIMT, q4.PATH_DECODE):
        assert torch.equal(cache.attend(q, table, lens, path=path), small.attend(q, order, lens, path=path))


def test_empty_calls():
    cache = q4.Int4KVCache(2, 16, 2, 64)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    cache.write(none, none, slots)
    assert cache.read(slots)[0].shape == (0, 2, 64)
    table = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    lens = torch.empty(0, dtype=torch.int32, device="cuda")
    assert cache.attend(none, table, lens).shape == (0, 2, 64)
    # A table of no pages: every row sees nothing.
    q = torch.ones((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = cache.attend(q, torch.empty((3, 0), dtype=torch.int32, device="cuda"),
                            torch.ones(3, dtype=torch.int32, device="cuda"), return_lse=True)
    assert (out == 0).all() and torch.isinf(lse).all()
    # A cache of no pages holds nothing.
    cache = q4.Int4KVCache(0, 16, 2, 64)
    cache.write(q[:, :2], q[:, :2], torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert (cache.read(torch.zeros(3, dtype=torch.int64, device="cuda"))[1] == 0).all()
    assert (cache.attend(q, torch.zeros((3, 1), dtype=torch.int32, device="cuda"),
                         torch.ones(3, dtype=torch.int32, device="cuda")) == 0).all()


@pytest.mark.parametrize("scheme", ["symmetric", "affine"])
def test_decoding_with_int4_layers(scheme):
    """A prompt in two chunks and then single tokens of two sequences through
    a fused projection, the cache and an output projection, all in 4 bits:
    each step's attention against 64-bit arithmetic on the same cache, whose
    content is read back and equals the projections' coded rows."""
    H, ratio, D, S, hidden, group = 2, 4, 64, 16, 256, 32
    torch.manual_seed(0)
    qkv = q4.Int4Linear.from_linear(torch.nn.Linear(hidden, (H * ratio + 2 * H) * D, bias=False).cuda(), group=32)
    proj = q4.Int4Linear.from_linear(torch.nn.Linear(H * ratio * D, hidden).cuda(), group=32)
    cache = q4.Int4KVCache(12, S, H, D, group=group, scheme=scheme)
    table = torch.tensor([[7, 2, 9, 0, 4], [1, 3, 11, 5, 10]], dtype=torch.int32, device="cuda")
    lens = [0, 0]
    written = [[], []]
    for step, counts in enumerate([[20, 33], [15, 1], [1, 1], [1, 1], [1, 1]]):
        x = torch.randn(sum(counts), hidden, device="cuda").bfloat16()
        y = qkv(x).view(sum(counts), -1, D)
        q, k, v = y[:, :H * ratio], y[:, H * ratio:H * ratio + H], y[:, H * ratio + H:]
        lens_new = [n + m for n, m in zip(lens, counts)]
        slots = torch.cat([table[b, torch.arange(n, n + m, device="cuda") // S].long() * S
                           + torch.arange(n, n + m, device="cuda") % S for b, (n, m) in enumerate(zip(lens, counts))])
        cache.write(k, v, slots)
        for b, at in enumerate((slice(0, counts[0]), slice(counts[0], None))):
            written[b].append((k[at], v[at]))
        starts = torch.tensor([0, counts[0], sum(counts)], dtype=torch.int32, device="cuda")
        lens_t = torch.tensor(lens_new, dtype=torch.int32, device="cuda")
        got = cache.attend(q, table, lens_t, q_starts=starts, return_lse=True)
        want = attention_ref(q, cache.packed, cache.scales, cache.zeros, table, lens_new, counts, group)
        assert_attention_close(got, want)
        assert torch.isfinite(proj(got[0].reshape(sum(counts), -1))).all()
        lens = lens_new
    for b in (0, 1):
        j = torch.arange(lens[b], device="cuda")
        back = cache.read(table[b, j // S].long() * S + j % S, torch.float32)
        for i in (0, 1):
            x = torch.cat([w[i] for w in written[b]])
            p, s, z = code_rows(rows_f32(x).reshape(-1, D), group, scheme == "affine")
            ref = value_rows(p, s, z, D, group).astype(np.float32)
            assert np.array_equal(back[i].cpu().numpy().reshape(-1, D), ref)
