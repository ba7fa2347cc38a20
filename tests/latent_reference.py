"""Latent attention in 64 bits, from the formulas in include/kda.h, with error bounds for the GPU results.

Everything is computed one sequence at a time with torch in float64, on the inputs' device.

Bounds.  u = 2^-8 is half a bf16 step (eps / 2).  An output is rounded to bf16 once (u |o|), and the weights
p_j enter the value product as bf16 (u sum_j p_j |v_j|, in proportions of the row's sum).  A score is a sum of
D products of bf16 numbers in fp32, off by at most D 2^-24 sum_i |q_i k_i| scale, and the exponential's argument
and result are off by a few 2^-24 of the argument: together delta, which moves p_j by a share delta and the
quotient by at most 2 delta sum_j p_j |v_j|.  The row's sum of `len` positive terms in fp32 is off by a share of
at most len 2^-24, in the quotient and in lse.
"""
import math

import torch

U = 2.0 ** -8


def rows_of(cache, table, n, count):
    """The first `count` rows of sequence n, entries outside the cache as zeros (float64)."""
    page = cache.shape[1]
    pos = torch.arange(count, device=cache.device)
    pages = table[n].long()[pos // page]
    ok = (pages >= 0) & (pages < cache.shape[0])
    x = cache[pages.clamp(0, max(cache.shape[0] - 1, 0)), pos % page].double()
    return torch.where(ok[:, None], x, torch.zeros_like(x))


def attend(q, k, v, scale, seen):
    """One softmax row per q [R, D] over k [L, D], v [L, V]; row i sees keys 0 .. seen[i] - 1.
    Returns (out, lse, bound of out, bound of lse), all [R, ...]."""
    L = k.shape[0]
    s = (q @ k.T) * scale
    hidden = torch.arange(L, device=q.device)[None, :] >= seen[:, None]
    s = s.masked_fill(hidden, -math.inf)
    none = seen <= 0
    lse = torch.logsumexp(s, -1) if L else torch.full((q.shape[0],), -math.inf, dtype=q.dtype, device=q.device)
    p = torch.exp(s - torch.where(none, torch.zeros_like(lse), lse)[:, None])
    p = p.masked_fill(hidden, 0.0)
    out = p @ v
    mass = p @ v.abs()
    size = ((q.abs() @ k.abs().T) * scale).masked_fill(hidden, 0.0)
    size = size.amax(-1) if L else torch.zeros_like(lse)
    delta = q.shape[1] * 2.0 ** -24 * size + 2.0 ** -21 * (1 + size)
    total = seen.clamp_min(1) * 2.0 ** -24
    b_out = U * out.abs() + (U + 2 * delta + total)[:, None] * mass + 1e-30
    return out, lse, b_out, delta + total + 2.0 ** -22 * lse.abs().nan_to_num(0.0, 0.0, 0.0)


def decode(q_latent, q_rope, cache, table, lens, scale):
    """Returns (out, lse, bound of out, bound of lse) of kda_latent_decode's arguments."""
    n, most = table.shape[0], table.shape[1] * cache.shape[1]
    T, H = q_latent.shape[0] // n, q_latent.shape[1]
    q = q_latent.double() if q_rope is None else torch.cat([q_latent, q_rope], -1).double()
    parts = []
    for i, length in enumerate(lens.tolist()):
        length = min(max(length, 0), most)
        c = rows_of(cache, table, i, length)
        seen = torch.arange(length - T + 1, length + 1, device=q.device).repeat_interleave(H)
        parts.append(attend(q[i * T:(i + 1) * T].reshape(T * H, -1), c, c[:, :512], scale, seen))
    out, lse, b_out, b_lse = (torch.cat(x) for x in zip(*parts))
    return out.view(n * T, H, 512), lse.view(n * T, H), b_out.view(n * T, H, 512), b_lse.view(n * T, H)


def prefill(q, k, v, k_rope, scale, cu, cu_k):
    """Returns (out, lse, bound of out, bound of lse) over the rows of the sequences cu names."""
    T, H = q.shape[0], q.shape[1]
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device=q.device)  # noqa: E731
    out, lse, b_out, b_lse = z(T, H, 128), z(T, H), z(T, H, 128), z(T, H)
    for n in range(len(cu) - 1):
        a, b, c, d = cu[n], cu[n + 1], cu_k[n], cu_k[n + 1]
        seen = torch.arange(b - a, device=q.device) + 1 + (d - c) - (b - a)
        for h in range(H):
            kk = k[c:d, h].double()
            if k_rope is not None:
                kk = torch.cat([kk, k_rope[c:d].double()], -1)
            out[a:b, h], lse[a:b, h], b_out[a:b, h], b_lse[a:b, h] = attend(
                q[a:b, h].double(), kk, v[c:d, h].double(), scale, seen)
    return out, lse, b_out, b_lse


def rotate(x, pos, freq, interleaved):
    """R(p) x [..., 64] for positions pos (broadcast over the axes behind the first), in 64 bits, and its bound:
    one rounding, and sines and cosines good to 2^-21 in fp32 products."""
    x = x.double()
    angle = pos.double()[:, None] * freq.double()
    angle = angle.view(angle.shape[0], *([1] * (x.dim() - 2)), 32)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    y = (a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos())
    w = (a.abs() + b.abs(),) * 2
    join = (lambda t: torch.stack(t, -1).flatten(-2)) if interleaved else (lambda t: torch.cat(t, -1))
    return join(y), U * join(y).abs() + 2.0 ** -20 * join(w)


def assert_within(got, want, bound, name):
    got = got.double()
    same = (got == want) | ((got - want).abs() <= bound)
    if not bool(same.all()):
        bad = (~same).nonzero()[0].tolist()
        i = tuple(bad)
        raise AssertionError(f"{name}: {int((~same).sum())} of {same.numel()} outside, first at {bad}: "
                             f"{got[i].item()} for {want[i].item()} +- {bound[i].item()}")
