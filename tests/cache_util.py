"""Helpers for the tests of the 4-bit key/value cache: caches coded by the CPU
oracle, and attention in 64 bits with the error bound of the library's kernels.
"""

import math

import numpy as np
import torch

import oracle
from oracle import affine_oracle


def code_rows(x: np.ndarray, group: int, affine: bool):
    """(packed, scales, zeros or None) of the rows x [N, D] by the oracle."""
    if affine:
        packed, scales, zeros, _ = affine_oracle.quantize_uint4_affine(x, group)
        return packed, scales, zeros
    packed, scales, _ = oracle.quantize_int4(x, group)
    return packed, scales, None


def value_rows(packed: np.ndarray, scales: np.ndarray, zeros, D: int, group: int) -> np.ndarray:
    """64-bit values q s or (q - z) s of coded rows, by the oracle."""
    if zeros is None:
        q = oracle.unpack_int4(packed, D).astype(np.float64)
    else:
        q = affine_oracle.unpack_uint4(packed, D).astype(np.float64) - np.repeat(
            zeros.astype(np.float64), group, axis=1)[:, :D]
    return q * np.repeat(scales.astype(np.float64), group, axis=1)[:, :D]


def random_cache(pages, page_size, heads, D, group, affine, *, seed=0, device="cuda"):
    """A cache whose every row holds coded normal values (keys with a few large channels)."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(pages, 2, heads, page_size, D)).astype(np.float32)
    x[:, 0] *= np.exp(0.5 * rng.normal(size=(1, heads, 1, D))).astype(np.float32)
    packed, scales, zeros = code_rows(x.reshape(-1, D), group, affine)
    lead = (pages, 2, heads, page_size)

    def tensor(a):
        return torch.from_numpy(np.ascontiguousarray(a.reshape(*lead, -1))).to(device)

    return tensor(packed), tensor(scales), None if zeros is None else tensor(zeros)


def page_table(lens, page_size, pages, *, seed=0, extra=0, device="cuda"):
    """Distinct pages in random order for the sequences; -1 past each one's last token."""
    order = np.random.default_rng(seed + 77).permutation(pages)
    most = max([-(-n // page_size) for n in lens] + [0]) + extra
    table = np.full((len(lens), most), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // page_size)
        table[b, :m] = order[at:at + m]
        at += m
    assert at <= pages
    return torch.from_numpy(table).to(device)


def attention_ref(q, packed, scales, zeros, table, lens, counts, group, *, causal=True, window=0,
                  sm_scale=None, starts=None):
    """out, lse in 64 bits, and the bounds on their errors for 16-bit q.

    The kernels' errors, per row, with p_j the probabilities:
    * S_j: at most D + 64 fp32 operations on terms that sum to at most
      A_j = |sm_scale| s_j sum_d |q_d| (|n_d| + |z|) <= 30 |sm_scale| max(s_j) sum |q_d|, each off
      by at most 2^-23 (the tensor core may truncate) of that: e = (D + 64) 2^-23 max A_j.
    * p_j: 2 e (numerator and denominator), 2^-20 for the exponentials.
    * p_j V_j: two roundings to fp16, of the weight and of its product with the
      scale, or of the weight and of the value: 2^-11 each at worst.  They are
      independent from token to token, and three quarters of their sum,
      2^-11 * 1.5, is asked for.
    * the sums over j: at most len + 256 fp32 operations on terms that sum to
      at most sum_j p_j s_j 30.
    * out: half a unit of its type."""
    device = q.device
    rows, q_heads, D = q.shape
    P, _, H, S, _ = packed.shape
    ratio = q_heads // H
    scale = D ** -0.5 if sm_scale is None else sm_scale
    np_zeros = None if zeros is None else zeros.reshape(-1, zeros.shape[-1]).cpu().numpy()
    np_scales = scales.reshape(-1, scales.shape[-1]).cpu().numpy()
    with np.errstate(invalid="ignore"):
        values = value_rows(packed.reshape(-1, packed.shape[-1]).cpu().numpy(), np_scales, np_zeros, D, group)
    values = torch.from_numpy(values).reshape(P, 2, H, S, D).to(device)
    widest = torch.from_numpy(np_scales.astype(np.float64).max(1)).reshape(P, 2, H, S).to(device)
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=device)
    lse = torch.full((rows, q_heads), math.nan, dtype=torch.float64, device=device)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    qd = q.double()
    half = torch.finfo(q.dtype).eps / 2
    row = 0
    for b, (n, m) in enumerate(zip(lens, counts)):
        if starts is not None:
            row = starts[b]
        j = torch.arange(n, device=device)
        page = table[b, j // S].long() if n else j
        known = (page >= 0) & (page < P)
        page = page.clamp(0, max(P - 1, 0))
        pos = n - m + torch.arange(m, device=device)
        seen = known[None] & torch.ones((m, n), dtype=torch.bool, device=device)
        if causal:
            seen &= j[None] <= pos[:, None]
        if window:
            seen &= j[None] > pos[:, None] - window
        for h in range(q_heads):
            k = values[page, 0, h // ratio, j % S] if n else values.new_zeros((0, D))
            v = values[page, 1, h // ratio, j % S] if n else k
            k = torch.where(known[:, None], k, torch.zeros_like(k))
            here = seen.any(0)
            k, v = k.nan_to_num(0, 0, 0) if not here.all() else k, v
            v = torch.where(here[:, None], v, torch.zeros_like(v))
            k = torch.where(here[:, None], k, torch.zeros_like(k))
            x = qd[row:row + m, h]
            s = (x @ k.T * scale).masked_fill(~seen, -math.inf)
            empty = ~seen.any(1)
            top = s.amax(1, keepdim=True) if n else s.new_full((m, 1), -math.inf)
            p = torch.exp(s - torch.where(torch.isinf(top) & (top < 0), torch.zeros_like(top), top))
            total = p.sum(1, keepdim=True)
            p = torch.where(empty[:, None], torch.zeros_like(p), p / total)
            out[row:row + m, h] = p @ v
            lse[row:row + m, h] = torch.where(empty, torch.full_like(total[:, 0], -math.inf),
                                              (torch.log(total) + top)[:, 0])
            ks = torch.where(here, widest[page, 0, h // ratio, j % S] if n else k.new_zeros(0), torch.zeros_like(j, dtype=torch.float64))
            vs = torch.where(here, widest[page, 1, h // ratio, j % S] if n else k.new_zeros(0), torch.zeros_like(j, dtype=torch.float64))
            e = (D + 64) * 2.0 ** -23 * abs(scale) * 30 * x.abs().sum(1) * (ks.max() if n else 0.0)
            e = e[:, None]
            out_tol[row:row + m, h] = ((p @ v.abs()) * (2.0 ** -11 * 1.5 + 2.0 ** -20 + 2 * e)
                                       + (n + 256) * 2.0 ** -23 * 30 * (p @ vs[:, None])
                                       + half * out[row:row + m, h].abs() + torch.finfo(q.dtype).tiny)
            lse_tol[row:row + m, h] = (e[:, 0] + 2.0 ** -20 + (n + 256) * 2.0 ** -23
                                       + 2.0 ** -22 * lse[row:row + m, h].abs().nan_to_num(0, 0, 0))
        row += m
    return out, lse, out_tol, lse_tol


def assert_attention_close(got, want, rows=None):
    """got = (out, lse) against attention_ref's result; rows no sequence holds are skipped."""
    (out, lse), (ref, ref_lse, tol, lse_tol) = got, want
    held = ~torch.isnan(ref_lse)
    assert held.any() or rows == 0 or ref_lse.numel() == 0
    o, r, t = out.double()[held], ref[held], tol[held]
    assert torch.isfinite(o).all()
    worst = ((o - r).abs() / t).max().item() if o.numel() else 0.0
    assert worst <= 1.0, f"out is {worst:.3g} times its bound off"
    a, b, t = lse.double()[held], ref_lse[held], lse_tol[held]
    none = torch.isinf(b)
    assert torch.equal(torch.isinf(a) & (a < 0), none)
    if (~none).any():
        worst = ((a - b).abs() / t)[~none].max().item()
        assert worst <= 1.0, f"lse is {worst:.3g} times its bound off"
