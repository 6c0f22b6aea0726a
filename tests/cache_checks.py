"""Attention over the 4-bit cache in 64 bits, and checks on norms that are
sharp enough to see one missing token, beside the bounds for each element in
cache_util.py.  Works on the device of its tensors."""

import math

import torch


def made_cache(pages, page_size, heads, D, group, affine, *, seed=0, device="cuda"):
    """A cache of random codes, scales around 0.4 and, if affine, zero points around 8."""
    gen = torch.Generator(device=device).manual_seed(seed)
    lead, G = (pages, 2, heads, page_size), -(-D // group)
    packed = torch.randint(0, 256, (*lead, (D + 1) // 2), dtype=torch.uint8, generator=gen, device=device)
    scales = (0.4 * torch.exp(0.3 * torch.randn((*lead, G), generator=gen, device=device))).half()
    zeros = torch.randint(5, 12, (*lead, G), dtype=torch.uint8, generator=gen, device=device) if affine else None
    return packed, scales, zeros


def made_table(lens, page_size, *, seed=0, spare=2, device="cuda"):
    """(table, pages): the sequences' distinct pages in random order, -1 past each one's last."""
    need = [-(-n // page_size) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return table.to(device), pages


def token_rows(packed, scales, zeros, page, kv, offset, D, group):
    """Values [tokens, H, D] in 64 bits of the tokens at (page, offset), and the
    size s (n + z) of each element's terms in the products (n from 0 to 15)."""
    d = torch.arange(D, device=packed.device)
    n = (packed[page, kv, :, offset].long()[..., d // 2] >> (4 * (d % 2))) & 15
    s = scales[page, kv, :, offset].double()[..., d // group]
    if zeros is None:
        n, z = (n + 8) & 15, torch.full_like(n, 8)
    else:
        z = zeros[page, kv, :, offset].long()[..., d // group]
    return (n - z).double() * s, (n + z).double() * s


def attention_64(q, packed, scales, zeros, table, lens, counts, group, *, causal=True, window=0, sm_scale=None):
    """out, lse, sum_j (p_j V_j)^2 and sum_j p_j A_j, A_j = |sm_scale| |q| |s (n + z)|
    (2-norms: no partial sum of the products that make S_j is larger)."""
    rows, q_heads, D = q.shape
    H, S = packed.shape[2], packed.shape[3]
    ratio = q_heads // H
    scale = D ** -0.5 if sm_scale is None else sm_scale
    dev = q.device
    out = torch.zeros((rows, q_heads, D), dtype=torch.float64, device=dev)
    spread = torch.zeros_like(out)
    lse = torch.full((rows, q_heads), -math.inf, dtype=torch.float64, device=dev)
    size = torch.zeros_like(lse)
    row = 0
    for b, (n, m) in enumerate(zip(lens, counts)):
        at, row = slice(row, row + m), row + m
        if n == 0 or m == 0:
            continue
        j = torch.arange(n, device=dev)
        page = table[b, j // S].long()
        k, k_size = token_rows(packed, scales, zeros, page, 0, j % S, D, group)
        v, _ = token_rows(packed, scales, zeros, page, 1, j % S, D, group)
        pos = n - m + torch.arange(m, device=dev)
        hidden = torch.zeros((m, n), dtype=torch.bool, device=dev)
        if causal:
            hidden |= j[None] > pos[:, None]
        if window:
            hidden |= j[None] <= pos[:, None] - window
        empty = hidden.all(1)
        x = q[at].double()
        for h in range(q_heads):
            kv = h // ratio
            s = (x[:, h] @ k[:, kv].T * scale).masked_fill_(hidden, -math.inf)
            a = torch.logsumexp(s, 1)
            lse[at, h] = a
            p = torch.exp(s - a[:, None]).masked_fill_(empty[:, None], 0.0)
            out[at, h] = p @ v[:, kv]
            spread[at, h] = (p * p) @ (v[:, kv] * v[:, kv])
            size[at, h] = abs(scale) * x[:, h].norm(dim=1) * (p @ k_size[:, kv].norm(dim=1))
    return out, lse, spread, size


def assert_attention_sharp(got, want):
    """Root mean squares over all rows, of at least 32 (row, head) pairs:

    * lse: 2^-22 A for S (fp32 steps, or the tensor core's truncations, of
      partial sums whose root mean square is about A / sqrt(D): D / 16 chained
      instructions of some units of 2^-24 each), 2^-19 for the exponentials
      and the sums, 2^-22 for the logarithm.
    * out: two roundings of each weight (or of weight and value) to fp16,
      uniform in a step: at most 2^-11 / sqrt(3) each, independent from token
      to token; twice lse's error; half a unit of the output's type over sqrt(3)."""
    (out, lse), (ref, ref_lse, spread, size) = got, want
    assert lse.numel() >= 32
    none = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), none)
    assert (out[none] == 0).all()
    held = ~none
    o, r, a, b = out.double()[held], ref[held], lse.double()[held], ref_lse[held]
    assert torch.isfinite(o).all() and torch.isfinite(a).all()
    tol = 2.0 ** -22 * size[held] + 2.0 ** -19 + 2.0 ** -22 * b.abs()
    worst = ((a - b) / tol).square().mean().sqrt().item()
    assert worst <= 1.0, f"lse is {worst:.3g} times its root mean square off"
    two = 0.0 if out.dtype == torch.float32 else 2 * (2.0 ** -11) ** 2 / 3
    unit = (torch.finfo(out.dtype).eps / 2) ** 2 / 3
    bound = (two * spread[held] + (unit + (2 * tol[:, None]) ** 2) * r * r).sum().sqrt().item()
    off = (o - r).norm().item()
    assert off <= bound, f"out is {off / bound:.3g} times its root mean square off"
