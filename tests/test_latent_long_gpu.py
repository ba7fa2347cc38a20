"""Absorbed latent attention over long contexts on the GPU, where many partial results are joined: bounds that a lost or
twice-counted piece cannot meet.

lse: the sum of n positive terms goes through n / (128 or 64) / 152 additions in a thread and 30 more at most (a warp, a
team, the join), each off by 2^-24 of what it adds up, and the scores by D 2^-24 sum_i |q_i k_i| at most (tests/
latent_reference.py).  out: its rounding is 2^-8 of each channel at most, and so are the weights'.  A run of blocks that is
left out is 1/152 of lse's sum, 6.6e-3.  out is a mean and would hardly move, but for 128 channels that a page's rows have
for themselves and few others: each is the share of the weights that its pages have."""
import math

import pytest
import torch

import linear_attention_06_gb300 as kda
from tests import latent_q8_reference as q8

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16
RUNS, MARK = 152, 384                         # blocks of the card; the first of the pages' channels


def parts(q, read, pages, scale):
    """Softmax rows q [R, D] over some pages' rows in 64 bits: their largest score, sum and weighted values."""
    top = torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=DEV)
    total, out = torch.zeros_like(top), torch.zeros(q.shape[0], 512, dtype=torch.float64, device=DEV)
    for k in range(0, pages.shape[0], 64):
        v = read(pages[k:k + 64]).flatten(0, 1)
        s = q @ v.T * scale
        new = torch.maximum(top, s.amax(-1))
        p = torch.exp(s - new[:, None])
        f = torch.exp(top - new)
        top, total, out = new, total * f + p.sum(-1), out * f[:, None] + p @ v[:, :512]
    return top, total, out


@pytest.mark.parametrize("cache_type", ["bf16", "8 bits"])
@pytest.mark.parametrize("H,pages", [(16, 1024), (32, 1024), (64, 256), (3, 2048)])
def test_a_long_context_is_seen_whole(cache_type, H, pages):
    """Up to 2^21 tokens on pages of 1024 tokens in random order, a short neighbour before and behind."""
    g = torch.Generator(device=DEV)
    g.manual_seed(H + pages)
    order = torch.randperm(pages, generator=g, device=DEV)
    table = torch.zeros(3, pages, dtype=torch.int32, device=DEV)
    table[1] = order.to(torch.int32)
    lens = torch.tensor([77, pages * 1024, 1], dtype=torch.int32, device=DEV)
    q, qr = (torch.randn(3, H, d, generator=g, device=DEV).to(BF) for d in (512, 64))
    scale = 0.07
    cache = torch.empty(pages, 1024, 576, dtype=BF if cache_type == "bf16" else q8.E4M3, device=DEV)
    for k in range(0, pages, 64):
        x = torch.randn(cache[k:k + 64].shape, generator=g, device=DEV)
        x[..., MARK:MARK + 128] = (torch.arange(k, min(k + 64, pages), device=DEV)[:, None, None] % 128
                                   == torch.arange(128, device=DEV)).float()
        cache[k:k + 64] = x.to(BF) if cache_type == "bf16" else x.mul_(100).clamp_(-448, 448).to(q8.E4M3)
    if cache_type == "bf16":
        read = lambda at: cache[at].double()  # noqa: E731
        out, lse = kda.kda_latent_decode(q, qr, cache, table, lens, scale, lse=True)
        tile = 64
    else:
        scales = torch.randint(120, 122, (pages, 1024), generator=g, device=DEV).to(torch.uint8)
        read = lambda at: q8.values(cache.view(torch.uint8)[at].view(q8.E4M3), scales[at])  # noqa: E731
        out, lse = kda.kda_latent_decode_q8(q, qr, cache, scales.view(q8.E8M0), table, lens, scale, lse=True)
        tile = 128
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0
    x = torch.cat([q[1], qr[1]], -1).double()
    top, total, o = parts(x, read, order, scale)
    z = top + total.log()
    some = read(order[:8]).abs().flatten(0, 1)                 # sizes, with room for larger rows among the others
    size = 1.25 * float((x.abs() @ some.T * scale).amax())
    near = (pages * 1024 / tile / RUNS + 30) * 2.0 ** -24 + 576 * 2.0 ** -24 * size + 2.0 ** -20 * (1 + float(z.abs().amax()))
    if cache_type != "bf16":                                   # a channel of a query: 2^-10 of its power of two
        near += 2.0 ** -10 * float(x.abs().amax()) / 224 * scale * 1.25 * float(some.sum(-1).amax())
    far = 2 * 2.0 ** -8 + 2 * near
    o = o / total[:, None]
    share = lambda a: ((a.double() - o) / o)[:, MARK:MARK + 128].abs().amax(-1)  # noqa: E731
    assert float((lse[1].double() - z).abs().amax()) <= near
    assert float(share(out[1]).amax()) <= far
    assert float(((out[1].double() - o).norm(dim=-1) / o.norm(dim=-1)).amax()) <= far
    # one run of blocks less would be told apart (by lse too, where a page is not all of a run)
    t, l, r = parts(x, read, order[pages // 2: pages // 2 + max(1, pages // RUNS)], scale)
    f = torch.exp(t - top)
    less = (o * total[:, None] - r * f[:, None]) / (total - l * f)[:, None]
    assert float(share(less).amin()) > 2 * far
    assert pages < 1024 or float(-torch.log1p(-l * f / total).amax()) > near


def test_the_longest_context_is_counted_to_the_token():
    """2^31 - 21 rows of zeros in 8 bits: equal weights, a power of two each, so that the sums are whole numbers and exact."""
    page, per = 16, 2 ** 27 - 1
    table = torch.zeros((1, per), dtype=torch.int32, device=DEV)
    length = per * page - 5
    cache = torch.zeros(1, page, 512, dtype=torch.uint8, device=DEV).view(q8.E4M3)
    scales = torch.full((1, page), 127, dtype=torch.uint8, device=DEV).view(q8.E8M0)
    out, lse = kda.kda_latent_decode_q8(torch.ones(1, 1, 512, dtype=BF, device=DEV), None, cache, scales, table,
                                        torch.tensor([length], dtype=torch.int32, device=DEV), 0.01, lse=True)
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0
    # the sum is exact; lse is rounded three times, near 21.5
    assert bool((out == 0).all()) and abs(float(lse) - math.log(length)) <= 3 * 2.0 ** -24 * 32
