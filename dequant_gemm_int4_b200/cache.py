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
import importlib.machinery
import importlib.util
import os

import torch

from . import _DTYPE_CODE, PATH_AUTO, _check, lib

__all__ = ["int4_cache_write", "int4_cache_read", "int4_cache_attention",
           "cache_attention_workspace_size", "Int4KVCache"]

_BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_cache_binding.so")
_binding = None


def _native():
    """The extension module built from cache_binding.cpp, bound to libint4.so once."""
    global _binding
    if _binding is None:
        if not os.path.exists(_BINDING_PATH):
            raise RuntimeError(
                f"{_BINDING_PATH} is missing: build it with `python -m dequant_gemm_int4_b200.build`")
        L = lib()
        loader = importlib.machinery.ExtensionFileLoader("_cache_binding", _BINDING_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_cache_binding", loader))
        loader.exec_module(module)
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.int4_cache_write, L.int4_cache_read, L.int4_cache_attention,
            L.int4_cache_attention_workspace_size)))
        _binding = module
    return _binding


def int4_cache_write(k: torch.Tensor, v: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                     slots: torch.Tensor, group: int = 128, *,
                     zeros: torch.Tensor | None = None) -> None:
    """Quantize k and v [tokens, heads, head_dim] (fp32/bf16/fp16, any token
    and head stride) into the cache at ``slots`` (int64 [tokens], page *
    page_size + offset).  A token whose slot is negative or past the cache is
    not written; the other slots must be distinct."""
    r = (_binding or _native()).write(k, v, packed, scales, slots, group, zeros)
    if r is not None:
        _check(r)


def int4_cache_read(packed: torch.Tensor, scales: torch.Tensor, slots: torch.Tensor, head_dim: int,
                    group: int = 128, dtype: torch.dtype = torch.bfloat16, *,
                    zeros: torch.Tensor | None = None,
                    out: tuple[torch.Tensor, torch.Tensor] | None = None):
    """The keys and values of ``slots`` (int64 [tokens]) as dense
    (k, v) [tokens, heads, head_dim] of ``dtype``; zeros for a slot that is
    negative or past the cache.  ``out``, if given, is written in place."""
    code = _DTYPE_CODE.get(dtype)
    if code is None:
        raise TypeError("dtype must be float32, bfloat16 or float16")
    k, v = (None, None) if out is None else out
    r = (_binding or _native()).read(packed, scales, slots, head_dim, group, code, zeros, k, v)
    if type(r) is int:
        _check(r)
    return r


def cache_attention_workspace_size(q: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                                   page_table: torch.Tensor, group: int = 128, *,
                                   zeros: torch.Tensor | None = None, path: int = PATH_AUTO) -> int:
    """Bytes of workspace that int4_cache_attention needs for these operands."""
    r = _native().workspace_size(q, packed, scales, page_table, group, zeros, path)
    if r < 0:
        _check(-r)
    return r


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

    ``path``: PATH_AUTO takes a tensor-core kernel where one can run (16-bit q;
    weights rounded to fp16); PATH_SIMT the general kernel, in fp32 throughout;
    PATH_DECODE and PATH_PREFILL a given tensor-core kernel.
    ``workspace``: None takes one from torch's allocator for this call; a uint8
    CUDA tensor of cache_attention_workspace_size bytes is used as given."""
    r = (_binding or _native()).attention(q, packed, scales, page_table, kv_lens, group, zeros, q_starts,
                                          causal, window, sm_scale, return_lse, out, lse, path, workspace)
    if type(r) is int:
        _check(r)
    return r


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
