"""Host-side tests of the 4-bit key/value cache: the C entries refuse bad
arguments before launching anything, the binding refuses bad tensors, and the
tests' own reference agrees with a case worked by hand.  No GPU needed."""

import ctypes
import math

import numpy as np
import pytest
import torch

import dequant_gemm_int4_b200 as q4
from cache_util import attention_ref, code_rows, random_cache, value_rows
from dequant_gemm_int4_b200 import build as q4build


class _Cache(ctypes.Structure):
    """int4_cache of include/int4.h."""

    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("group", ctypes.c_int32)]


FAKE = 256  # an address that is never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    q4build.build()
    return q4.lib()


def cache(**kw):
    a = dict(packed=FAKE, scales=FAKE, zeros=None, pages=4, page_size=16, heads=2, head_dim=64, group=32)
    a.update(kw)
    return ctypes.byref(_Cache(*(a[n] for n, _ in _Cache._fields_)))


def test_cache_write_and_read_reject_bad_arguments(L):
    def write(c=None, k=FAKE, v=FAKE, t=1, n=3, slots=FAKE):
        return L.int4_cache_write(c or cache(), k, 128, 64, v, 128, 64, t, n, slots, None)

    def read(c=None, k=FAKE, v=FAKE, t=1, n=3, slots=FAKE):
        return L.int4_cache_read(c or cache(), slots, n, k, v, t, None)

    for f in (write, read):
        assert f(t=7) == q4.ERR_DTYPE
        for bad in (dict(page_size=0), dict(heads=0), dict(head_dim=0), dict(head_dim=513), dict(group=0),
                    dict(pages=-1), dict(packed=None), dict(scales=None), dict(pages=1 << 60)):
            assert f(cache(**bad)) == q4.ERR_ARG, bad
        assert f(cache(scales=257)) == q4.ERR_ALIGN
        assert f(n=-1) == q4.ERR_ARG
        assert f(k=None) == q4.ERR_ARG
        assert f(v=None) == q4.ERR_ARG
        assert f(slots=None) == q4.ERR_ARG
        assert f(k=257) == q4.ERR_ALIGN
        assert f(slots=260) == q4.ERR_ALIGN
        assert f(n=1 << 60) == q4.ERR_ARG
        assert f(n=0) == q4.OK
    assert L.int4_cache_write(None, FAKE, 1, 1, FAKE, 1, 1, 1, 1, FAKE, None) == q4.ERR_ARG
    assert b"int4_cache_write" in L.int4_last_error()
    assert write(cache(pages=0, packed=None, scales=None)) == q4.OK  # no slot to write


def test_cache_attention_rejects_bad_arguments(L):
    def call(c=None, q=FAKE, t=1, rows=6, hq=4, table=FAKE, pages=8, lens=FAKE, starts=None, batch=3,
             window=0, scale=0.125, out=FAKE, lse=None, path=q4.PATH_SIMT, ws=None, n=0):
        return L.int4_cache_attention(c or cache(), q, 256, 64, t, rows, hq, table, 8, pages, lens, starts,
                                      batch, 1, window, scale, out, lse, path, ws, n, None)

    assert call(t=4) == q4.ERR_DTYPE
    for bad in (dict(rows=-1), dict(hq=3), dict(hq=0), dict(batch=-1), dict(pages=-1), dict(window=-1),
                dict(scale=math.nan), dict(scale=math.inf), dict(rows=7), dict(q=None), dict(table=None),
                dict(lens=None), dict(out=None), dict(path=9), dict(path=-1), dict(n=64),
                dict(rows=1 << 40), dict(c=cache(head_dim=0))):
        assert call(**bad) == q4.ERR_ARG, bad
    for bad in (dict(q=257), dict(out=257), dict(table=258), dict(lens=258), dict(starts=258), dict(lse=258),
                dict(ws=272, n=64)):
        assert call(**bad) == q4.ERR_ALIGN, bad
    assert call(rows=0) == q4.OK
    assert call(batch=0) == q4.OK
    # The tensor-core kernels refuse what they cannot run ...
    for bad in (dict(t=0), dict(c=cache(head_dim=80, group=80)), dict(c=cache(group=16)),
                dict(c=cache(page_size=24)), dict(c=cache(page_size=8)), dict(c=cache(packed=264)),
                dict(out=260), dict(pages=1 << 27)):
        assert call(path=q4.PATH_DECODE, **bad) == q4.ERR_UNSUPPORTED, bad
        assert b"int4_cache_attention" in L.int4_last_error()
    # ... and ask for their workspace.
    assert call(path=q4.PATH_DECODE) == q4.ERR_ARG
    assert b"workspace" in L.int4_last_error()


def test_cache_attention_workspace_size(L):
    size = ctypes.c_size_t(1)

    def ask(c=None, t=1, rows=6, hq=4, batch=3, pages=8, path=q4.PATH_AUTO):
        return L.int4_cache_attention_workspace_size(c or cache(), t, rows, hq, batch, pages, path,
                                                     ctypes.byref(size))

    assert ask() == q4.OK and size.value > 0 and size.value % 256 == 0
    small = size.value
    assert ask(rows=60) == q4.OK and size.value > small  # larger row tiles
    for kw in (dict(t=0), dict(path=q4.PATH_SIMT), dict(rows=0), dict(batch=0), dict(c=cache(head_dim=72, group=72))):
        assert ask(**kw) == q4.OK and size.value == 0, kw
    assert ask(hq=3) == q4.ERR_ARG
    assert ask(t=5) == q4.ERR_DTYPE
    assert ask(t=0, path=q4.PATH_DECODE) == q4.ERR_UNSUPPORTED
    assert L.int4_cache_attention_workspace_size(cache(), 1, 6, 4, 3, 8, 0, None) == q4.ERR_ARG


def test_cache_binding_refuses_bad_tensors():
    packed = torch.zeros((3, 2, 2, 16, 32), dtype=torch.uint8)
    scales = torch.zeros((3, 2, 2, 16, 2), dtype=torch.float16)
    k = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    slots = torch.zeros(5, dtype=torch.int64)
    # Shapes and types first; then, all being right, the missing GPU.
    with pytest.raises(TypeError, match="CUDA"):
        q4.int4_cache_write(k, k, packed, scales, slots, 32)
    with pytest.raises(ValueError, match="packed"):
        q4.int4_cache_write(k, k, packed[..., :31], scales, slots, 32)
    with pytest.raises(ValueError, match="packed"):
        q4.int4_cache_write(k, k, packed[:, 0], scales, slots, 32)
    with pytest.raises(ValueError, match="scales"):
        q4.int4_cache_write(k, k, packed, scales, slots, 64)
    with pytest.raises(ValueError, match="scales"):
        q4.int4_cache_write(k, k, packed, scales.float(), slots, 32)
    with pytest.raises(ValueError, match="zeros"):
        q4.int4_cache_write(k, k, packed, scales, slots, 32, zeros=scales)
    with pytest.raises(ValueError, match="group"):
        q4.int4_cache_read(packed, scales, slots, 64, 0)
    with pytest.raises(TypeError, match="packed"):
        q4.int4_cache_read(None, scales, slots, 64, 32)
    with pytest.raises(ValueError, match=r"q must be \[rows"):
        q4.int4_cache_attention(k[0], packed, scales, slots, slots, 32)
    with pytest.raises(TypeError, match="CUDA"):
        q4.int4_cache_attention(k, packed, scales, slots, slots, 32)
    for bad in (dict(scheme="fp4"), dict(pages=-1), dict(page_size=0), dict(head_dim=513), dict(group=0)):
        a = dict(dict(pages=2, page_size=16, heads=2, head_dim=64, group=32, scheme="affine"), **bad)
        with pytest.raises(ValueError):
            q4.Int4KVCache(a["pages"], a["page_size"], a["heads"], a["head_dim"], group=a["group"],
                           scheme=a["scheme"], device="cpu")


def test_cache_module_buffers():
    c = q4.Int4KVCache(3, 16, 2, 80, group=32, scheme="affine", device="cpu")
    assert c.packed.shape == (3, 2, 2, 16, 40) and c.scales.shape == (3, 2, 2, 16, 3)
    assert set(c.state_dict()) == {"packed", "scales", "zeros"}
    c = q4.Int4KVCache(3, 16, 2, 64, device="cpu")  # the default group of 128, cut to the head
    assert c.group == 64 and set(c.state_dict()) == {"packed", "scales"}
    assert "head_dim=64" in repr(c)


def test_reference_attention_by_hand():
    """Two tokens, one head of 2: S = (q.k1, q.k2) / sqrt(2) = (0, ln 3)."""
    k = np.array([[0.0, 0.0], [1.0, 7.0]], dtype=np.float32)
    v = np.array([[7.0, 1.0], [-7.0, 2.0]], dtype=np.float32)
    rows = np.stack([k, v])  # scale 1 (absmax 7): coded exactly
    packed, scales, _ = code_rows(rows.reshape(-1, 2), 2, False)
    assert np.array_equal(value_rows(packed, scales, None, 2, 2)[1:], rows.reshape(-1, 2)[1:])
    packed = torch.from_numpy(packed.reshape(1, 2, 1, 2, 1))
    scales = torch.from_numpy(scales.reshape(1, 2, 1, 2, 1))
    s = math.log(3.0) * math.sqrt(2.0)
    q = torch.tensor([[[s - 7 * 0.25, 0.25]]], dtype=torch.float32)
    table = torch.zeros((1, 1), dtype=torch.int32)
    out, lse, tol, _ = attention_ref(q, packed, scales, None, table, [2], [1], 2)
    assert torch.allclose(out, torch.tensor([[[0.25 * 7 - 0.75 * 7, 0.25 + 0.75 * 2]]], dtype=torch.float64), atol=1e-6)
    assert abs(lse.item() - math.log(4.0)) < 1e-6 and (tol > 0).all()
    # One query more than tokens: the first sees nothing.
    out, lse, _, _ = attention_ref(q.repeat(3, 1, 1), packed, scales, None, table, [2], [3], 2)
    assert lse[0].item() == -math.inf and (out[0] == 0).all() and lse[1].item() == 0.0
    # A window of one token sees the last only.
    out, _, _, _ = attention_ref(q, packed, scales, None, table, [2], [1], 2, window=1)
    assert torch.equal(out[0, 0], torch.tensor([-7.0, 2.0], dtype=torch.float64))


def test_random_cache_is_the_oracles():
    packed, scales, zeros = random_cache(2, 4, 3, 10, 4, True, device="cpu")
    assert packed.shape == (2, 2, 3, 4, 5) and scales.shape == (2, 2, 3, 4, 3) and zeros.shape == scales.shape
