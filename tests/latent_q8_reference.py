"""The 8-bit latent cache in 64 bits, from the formulas in include/kda.h, with error bounds for the GPU results.

Bounds, beside those of tests/latent_reference.py.
- A quantised number is off by at most half a step: 2^-4 of itself, or 2^-10 * 2^e near zero.
- The tensor cores take a query as the sum of two e4m3 numbers under one power of two.  Two e4m3 numbers hold eight
  significant bits; the last step is 2^-9 of the power, so a channel is off by at most 2^-10 * 2^e_q, with
  2^e_q <= max |q| / 224: a score is off by that times sum_i |k_i|, on top of its products' rounding.
- A softmax weight, times the row's 2^e_j, goes in as an e4m3 and a second 8-bit number, under a reference that is the
  row's and changes from tile to tile (128 cached rows).  e4m3 leaves at most 2^-4 of a weight of 2^-6 or more (in units of
  the reference).  Of that the second number, e5m2 with three significant bits, leaves 2^-3 / 2 and so 2^-8 in all (U);
  e4m3 of 2^7 times the rest, with four bits, leaves half as much.  Of a smaller weight e4m3 leaves at most 2^-10, of which
  e5m2 leaves 2^-13 (e4m3 of 2^7 times it: 2^-14); both end at 2^-17.  A row's weights together are off by at most 2^-7 of
  their sum.  The bound here is looser: 2^-8 of the largest weight among a tile and the two before it for every weight,
  which is 2^-8 of the sum where all weights are alike and more where a few are bright.  What faint weights beside bright
  ones may lose is tested in tests/test_latent_q8_weights_gpu.py, with 2^-7 of the sum.
- The reference is not the maximum: the exponent of the largest weight lies in -5 .. 9 and not at 0, is rounded to 2^-21 at
  most, and the exponential of it is good to 2^-22.  A weight moves by a share of 2^-21 ln 2 + 2^-22, and so does the sum:
  2^-20 bounds the two logarithms' roundings with it (lse near 0 would otherwise have no room for them).
"""
import math

import torch

from tests import latent_reference as ref

U, TILE = ref.U, 128
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def two(k):
    """2^k exactly, for whole k (float64)."""
    return ((torch.as_tensor(k).long() + 1023) << 52).view(torch.float64)


def power_of_rows(x):
    """e of rows x [..., channels] (float64, finite), by the definition."""
    most = x.abs().amax(-1)
    e = torch.ceil(torch.log2(most.clamp_min(2.0 ** -300) / 448))
    e = e + (448 * two(e) < most).double() - (448 * two(e - 1) >= most).double()
    return torch.where(most == 0, torch.full_like(e, -64), e).clamp(-64, 120)


def to_e4m3(x):
    """The nearest e4m3 number, ties to even, of |x| <= 448 (float64): steps of 2^(k - 3) in [2^k, 2^(k + 1)), k >= -6."""
    size = x.abs().clamp_min(2.0 ** -6)
    k = torch.floor(torch.log2(size))
    k = k + (two(k + 1) <= size).double() - (two(k) > size).double()
    return torch.round(x * two(3 - k)) * two(k - 3)


def quantise(x):
    """(numbers, e) of rows x (float64)."""
    e = power_of_rows(x)
    return to_e4m3(x * two(-e)[..., None]), e


def bytes_of(y):
    """e4m3 numbers (float64, exact) as torch's 8-bit type."""
    return y.float().to(E4M3)


def powers_of(e):
    return (e + 127).to(torch.uint8).view(E8M0)


def values(cache, scales):
    """What a cache stands for (float64); bytes of scales outside 63 .. 247 count as the nearest of them."""
    return cache.double() * two(scales.view(torch.uint8).long().clamp(63, 247) - 127)[..., None]


def rows_of(cache, scales, table, n, count):
    """The first `count` rows of sequence n as (numbers, e), entries outside the cache as rows of zeros."""
    page = cache.shape[1]
    pos = torch.arange(count, device=cache.device)
    pages = table[n].long()[pos // page]
    ok = (pages >= 0) & (pages < cache.shape[0])
    pages = pages.clamp(0, max(cache.shape[0] - 1, 0))
    y = cache.view(torch.uint8)[pages, pos % page].view(E4M3).double()
    e = scales.view(torch.uint8)[pages, pos % page].double().clamp(63, 247) - 127
    return torch.where(ok[:, None], y, torch.zeros_like(y)), torch.where(ok, e, torch.full_like(e, -64))


def decode(q_latent, q_rope, cache, scales, table, lens, scale):
    """Returns (out, lse, bound of out, bound of lse) of kda_latent_decode_q8's arguments."""
    n, most = table.shape[0], table.shape[1] * cache.shape[1]
    T, H = q_latent.shape[0] // n, q_latent.shape[1]
    q = q_latent.double() if q_rope is None else torch.cat([q_latent, q_rope], -1).double()
    parts = []
    for i, length in enumerate(lens.tolist()):
        length = min(max(length, 0), most)
        y, e = rows_of(cache, scales, table, i, length)
        c = y * two(e)[:, None]
        seen = torch.arange(length - T + 1, length + 1, device=q.device).repeat_interleave(H)
        x = q[i * T:(i + 1) * T].reshape(T * H, -1)
        o, lse, bo, bs = ref.attend(x, c, c[:, :512], scale, seen)
        if length:
            off = 2.0 ** -10 * (x.abs().amax(-1) / 224).clamp_min(2.0 ** -64) * scale * c.abs().sum(-1).amax()   # of a score
            s = (x @ c.T) * scale
            hidden = torch.arange(length, device=q.device)[None, :] >= seen[:, None]
            s = s.masked_fill(hidden, -math.inf)
            z = torch.where(seen <= 0, torch.zeros_like(lse), lse)
            p = torch.exp(s - z[:, None]).masked_fill(hidden, 0.0)
            w = torch.nn.functional.pad(p * two(e), (0, -length % TILE)).view(p.shape[0], -1, TILE)
            top = torch.nn.functional.pad(w.amax(-1), (2, 0))
            top = torch.maximum(torch.maximum(top[:, 2:], top[:, 1:-1]), top[:, :-2])        # of a tile and the two before it
            top = top[:, :, None].expand_as(w).reshape(p.shape[0], -1)[:, :length]
            low = torch.where(hidden, torch.zeros_like(top), U * top) @ y[:, :512].abs()
            off = off + 2.0 ** -20
            bo = bo + 2 * off[:, None] * (p @ c[:, :512].abs()) + low
            bs = bs + off
        parts.append((o, lse, bo, bs))
    out, lse, b_out, b_lse = (torch.cat(x) for x in zip(*parts))
    return out.view(n * T, H, 512), lse.view(n * T, H), b_out.view(n * T, H, 512), b_lse.view(n * T, H)
