"""The 4-bit key/value cache: writing it, reading it back, attending over it.

Binding of the ``int4_cache_*`` entries of ``include/int4.h``, with the
cache's layout and every operator's definition.  A cache is the tensors

* ``packed`` uint8 [P, 2, H, S, ceil(D / 2)] (P pages of S tokens, keys at
  index 0 and values at index 1, H heads of D elements),
* ``scales`` float16 [P, 2, H, S, ceil(D / group)],
* ``zeros`` uint8, shaped as ``scales``, in the affine scheme only,

whose rows are coded bit for bit as ``quantize_int4`` (or
``quantize_int4_affine``) codes a row of D weights.  ``Int4KVCache`` holds
them as a module's buffers.  All arithmetic runs in the library's CUDA
kernels; nothing here waits for the GPU.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import (_DTYPE_CODE, PATH_AUTO, _check, _need_cuda, _nullctx, _raw_stream, lib)

__all__ = ["int4_cache_write", "int4_cache_read", "int4_cache_attention",
           "cache_attention_workspace_size", "Int4KVCache"]


class _Cache(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("group", ctypes.c_int32)]


def _cache_of(packed, scales, zeros, head_dim: int, group: int) -> _Cache:
    """The C view of a cache's tensors, which are checked."""
    for name, x in (("packed", packed), ("scales", scales)) if zeros is None else (
            ("packed", packed), ("scales", scales), ("zeros", zeros)):
        if not isinstance(x, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if group < 1 or head_dim < 1:
        raise ValueError("group and head_dim must be >= 1")
    shape = packed.shape
    if packed.dtype != torch.uint8 or len(shape) != 5 or shape[1] != 2 or shape[4] != (head_dim + 1) // 2:
        raise ValueError("packed must be uint8 [pages, 2, heads, page_size, ceil(head_dim/2)]")
    want = (*shape[:4], -(-head_dim // group))
    if scales.dtype != torch.float16 or scales.shape != want:
        raise ValueError("scales must be float16 [pages, 2, heads, page_size, ceil(head_dim/group)]")
    if zeros is not None and (zeros.dtype != torch.uint8 or zeros.shape != want):
        raise ValueError("zeros must be uint8, shaped as scales")
    _need_cuda("packed", packed)
    _need_cuda("scales", scales)
    device = packed.get_device()
    if scales.get_device() != device:
        raise ValueError("scales must be on packed's device")
    if zeros is not None:
        _need_cuda("zeros", zeros)
        if zeros.get_device() != device:
            raise ValueError("zeros must be on packed's device")
    return _Cache(packed.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(),
                  shape[0], shape[3], shape[2], head_dim, min(int(group), 1 << 30))


def _rows(name: str, x, like: torch.Tensor, heads: int | None, head_dim: int) -> torch.Tensor:
    """x checked as [tokens, heads, head_dim] with a dense last dimension, on like's device."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dim() != 3 or x.shape[2] != head_dim or (heads is not None and x.shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    if x.dtype not in _DTYPE_CODE:
        raise TypeError(f"{name} must be float32, bfloat16 or float16")
    if not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if x.stride(2) != 1 and head_dim > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    if x.get_device() != like.get_device():
        raise ValueError(f"{name} must be on the cache's device")
    return x


def _index(name: str, x, like: torch.Tensor, dtype: torch.dtype, shape: tuple) -> torch.Tensor:
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype != dtype or tuple(x.shape) != shape:
        raise ValueError(f"{name} must be {str(dtype).removeprefix('torch.')} {list(shape)}")
    _need_cuda(name, x)
    if x.get_device() != like.get_device():
        raise ValueError(f"{name} must be on the cache's device")
    return x


def _on(device: int):
    return _nullctx() if device == torch.cuda.current_device() else torch.cuda.device(device)


def int4_cache_write(k: torch.Tensor, v: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                     slots: torch.Tensor, group: int = 128, *,
                     zeros: torch.Tensor | None = None) -> None:
    """Quantize k and v [tokens, heads, head_dim] (fp32/bf16/fp16, any token
    and head stride) into the cache at ``slots`` (int64 [tokens], page *
    page_size + offset).  A token whose slot is negative or past the cache is
    not written; the other slots must be distinct."""
    head_dim = k.shape[-1] if isinstance(k, torch.Tensor) and k.dim() == 3 else 0
    cache = _cache_of(packed, scales, zeros, max(head_dim, 1), group)
    _rows("k", k, packed, cache.heads, cache.head_dim)
    _rows("v", v, packed, cache.heads, cache.head_dim)
    if v.shape[0] != k.shape[0] or v.dtype != k.dtype:
        raise ValueError("v must have k's shape and dtype")
    _index("slots", slots, packed, torch.int64, (k.shape[0],))
    device = packed.get_device()
    with _on(device):
        _check(lib().int4_cache_write(ctypes.byref(cache), k.data_ptr(), k.stride(0), k.stride(1),
                                      v.data_ptr(), v.stride(0), v.stride(1), _DTYPE_CODE[k.dtype],
                                      k.shape[0], slots.data_ptr(), _raw_stream(device)))


def int4_cache_read(packed: torch.Tensor, scales: torch.Tensor, slots: torch.Tensor, head_dim: int,
                    group: int = 128, dtype: torch.dtype = torch.bfloat16, *,
                    zeros: torch.Tensor | None = None,
                    out: tuple[torch.Tensor, torch.Tensor] | None = None):
    """The keys and values of ``slots`` (int64 [tokens]) as dense
    (k, v) [tokens, heads, head_dim] of ``dtype``; zeros for a slot that is
    negative or past the cache.  ``out``, if given, is written in place."""
    cache = _cache_of(packed, scales, zeros, head_dim, group)
    if dtype not in _DTYPE_CODE:
        raise TypeError("dtype must be float32, bfloat16 or float16")
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be int64 [tokens]")
    tokens = slots.shape[0]
    _index("slots", slots, packed, torch.int64, (tokens,))
    shape = (tokens, cache.heads, head_dim)
    if out is None:
        k, v = packed.new_empty(shape, dtype=dtype), packed.new_empty(shape, dtype=dtype)
    else:
        k, v = out
        for x in (k, v):
            if not isinstance(x, torch.Tensor) or x.dtype != dtype or tuple(x.shape) != shape:
                raise ValueError("out must be two tensors [tokens, heads, head_dim] of dtype")
            _need_cuda("out", x)
            if x.get_device() != packed.get_device():
                raise ValueError("out must be on the cache's device")
    device = packed.get_device()
    with _on(device):
        _check(lib().int4_cache_read(ctypes.byref(cache), slots.data_ptr(), tokens, k.data_ptr(),
                                     v.data_ptr(), _DTYPE_CODE[dtype], _raw_stream(device)))
    return k, v


def cache_attention_workspace_size(q: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                                   page_table: torch.Tensor, group: int = 128, *,
                                   zeros: torch.Tensor | None = None, path: int = PATH_AUTO) -> int:
    """Bytes of workspace that int4_cache_attention needs for these operands."""
    cache = _cache_of(packed, scales, zeros, q.shape[-1], group)
    return _workspace_size(cache, q, page_table, path, packed.get_device())


def _workspace_size(cache: _Cache, q, page_table, path: int, device: int) -> int:
    out = ctypes.c_size_t(0)
    with _on(device):
        _check(lib().int4_cache_attention_workspace_size(
            ctypes.byref(cache), _DTYPE_CODE[q.dtype], q.shape[0], q.shape[1], page_table.shape[0],
            page_table.shape[1], int(path), ctypes.byref(out)))
    return out.value


def int4_cache_attention(q: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                         page_table: torch.Tensor, kv_lens: torch.Tensor, group: int = 128, *,
                         zeros: torch.Tensor | None = None, q_starts: torch.Tensor | None = None,
                         causal: bool = True, window: int | None = None,
                         sm_scale: float | None = None, return_lse: bool = False,
                         out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                         path: int = PATH_AUTO, workspace: torch.Tensor | None = None):
    """Attention of q [rows, q_heads, head_dim] (bf16/fp16/fp32, any token and
    head stride) over a cache: ``out`` of q's shape and dtype, and with
    ``return_lse`` also lse float32 [rows, q_heads] (natural logarithm).

    Sequence b has kv_lens[b] cached tokens (int32 [batch]) in the pages
    page_table[b] (int32 [batch, max_pages]) and the rows q_starts[b] to
    q_starts[b + 1] of q (int32 [batch + 1]; None: rows / batch each), the last
    of which stands at its last token.  ``causal``: a query sees no token after
    its own.  ``window``: it sees the last ``window`` tokens up to its own.
    ``sm_scale``: None is head_dim ** -0.5.  A query that sees nothing gets 0
    and -inf; rows of no sequence are left as they were.

    ``workspace``: None takes one from torch's allocator for this call; a uint8
    CUDA tensor of cache_attention_workspace_size bytes is used as given."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [rows, q_heads, head_dim]")
    rows, q_heads, head_dim = q.shape
    cache = _cache_of(packed, scales, zeros, head_dim, group)
    _rows("q", q, packed, None, head_dim)
    if q_heads < 1 or q_heads % cache.heads:
        raise ValueError("q_heads must be a multiple of the cache's heads")
    device = packed.get_device()
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2 or page_table.dtype != torch.int32:
        raise ValueError("page_table must be int32 [batch, max_pages]")
    batch, max_pages = page_table.shape
    if not page_table.is_cuda or page_table.get_device() != device:
        raise ValueError("page_table must be on the cache's device")
    if max_pages > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table's rows must be contiguous")
    _index("kv_lens", kv_lens, packed, torch.int32, (batch,))
    if q_starts is not None:
        _index("q_starts", q_starts, packed, torch.int32, (batch + 1,))
    elif rows and (batch == 0 or rows % batch):
        raise ValueError("without q_starts, the batch must divide q's rows")
    window = 0 if window is None else min(int(window), 0x7FFFFFFF)
    if window < 0:
        raise ValueError("window must be None or >= 0")
    scale = head_dim ** -0.5 if sm_scale is None else float(sm_scale)
    if not math.isfinite(scale):
        raise ValueError("sm_scale must be finite")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        if not isinstance(out, torch.Tensor) or out.dtype != q.dtype or out.shape != q.shape:
            raise ValueError("out must have q's shape and dtype")
        _need_cuda("out", out)
        if out.get_device() != device:
            raise ValueError("out must be on the cache's device")
    if lse is not None:
        _index("lse", lse, packed, torch.float32, (rows, q_heads))
    elif return_lse:
        lse = torch.empty((rows, q_heads), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = _workspace_size(cache, q, page_table, path, device)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _need_cuda("workspace", workspace)
        if workspace.dtype != torch.uint8 or workspace.get_device() != device:
            raise ValueError("workspace must be a uint8 tensor on the cache's device")
    with _on(device):
        _check(lib().int4_cache_attention(
            ctypes.byref(cache), q.data_ptr(), q.stride(0), q.stride(1), _DTYPE_CODE[q.dtype], rows,
            q_heads, page_table.data_ptr(), page_table.stride(0), max_pages, kv_lens.data_ptr(),
            None if q_starts is None else q_starts.data_ptr(), batch, int(bool(causal)), window, scale,
            out.data_ptr(), None if lse is None else lse.data_ptr(), int(path),
            None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel(), _raw_stream(device)))
    return (out, lse) if return_lse else out


class Int4KVCache(torch.nn.Module):
    """A paged key/value cache of one layer in 4-bit codes, beside Int4Linear.

    scheme: "symmetric" or "affine", as for Int4Linear.  The codes, scales and
    zero points are buffers, so state_dict() carries them; which pages belong
    to which sequence is the caller's, who passes slots and page tables.
    """

    def __init__(self, pages: int, page_size: int, heads: int, head_dim: int, *, group: int = 128,
                 scheme: str = "symmetric", device=None):
        super().__init__()
        if scheme not in ("symmetric", "affine"):
            raise ValueError("scheme must be 'symmetric' or 'affine'")
        if pages < 0 or page_size < 1 or heads < 1 or not 1 <= head_dim <= 512 or group < 1:
            raise ValueError("need pages >= 0, page_size, heads, group >= 1 and head_dim in [1, 512]")
        self.head_dim, self.group, self.scheme = int(head_dim), min(int(group), int(head_dim)), scheme
        dev = torch.device("cuda") if device is None else torch.device(device)
        lead = (int(pages), 2, int(heads), int(page_size))
        groups = -(-self.head_dim // self.group)
        self.register_buffer("packed", torch.zeros((*lead, (self.head_dim + 1) // 2), dtype=torch.uint8, device=dev))
        self.register_buffer("scales", torch.zeros((*lead, groups), dtype=torch.float16, device=dev))
        if scheme == "affine":
            self.register_buffer("zeros", torch.zeros((*lead, groups), dtype=torch.uint8, device=dev))
        else:
            self.zeros = None

    def write(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
        """int4_cache_write into this cache."""
        int4_cache_write(k, v, self.packed, self.scales, slots, self.group, zeros=self.zeros)

    def read(self, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16):
        """int4_cache_read from this cache."""
        return int4_cache_read(self.packed, self.scales, slots, self.head_dim, self.group, dtype,
                               zeros=self.zeros)

    def attend(self, q: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor, **options):
        """int4_cache_attention over this cache (its keyword arguments as ``options``)."""
        return int4_cache_attention(q, self.packed, self.scales, page_table, kv_lens, self.group,
                                    zeros=self.zeros, **options)

    def extra_repr(self) -> str:
        pages, _, heads, page_size, _ = self.packed.shape
        return (f"pages={pages}, page_size={page_size}, heads={heads}, head_dim={self.head_dim}, "
                f"group={self.group}, scheme={self.scheme}")
