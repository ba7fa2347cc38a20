"""The 8-bit latent cache on the GPU against the 64-bit formulas of tests/latent_q8_reference.py: rows quantised in, rows
out, the absorbed decode over them, and a run of them together."""
import math
import os
import subprocess
import sys

import pytest
import torch

import linear_attention_06_gb300 as kda
from tests import latent_q8_reference as q8
from tests import latent_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, U8 = torch.bfloat16, torch.uint8


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(BF)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def freqs():
    return (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().to(DEV)


def offsets(counts):
    return [0] + torch.tensor(counts, dtype=torch.int64).cumsum(0).tolist()


def paged(lens, page, rope, g, extra_pages=3, per=None, make=None):
    """A cache of quantised N(0, 1) rows (of make(n, count) where given) on pages in random order.  Rows behind the
    sequences' ends hold NaN bytes and scale bytes of every kind; table entries behind a sequence's last page are nonsense."""
    used = [-(-max(n, 0) // page) for n in lens]
    per = max(used + [1]) + 1 if per is None else per
    total = sum(used) + extra_pages
    order = torch.randperm(total, generator=g, device=DEV).tolist()
    cache = torch.full((total, page, 512 + rope), 0x7F, dtype=U8, device=DEV)
    scales = torch.randint(0, 256, (total, page), generator=g, device=DEV).to(U8)
    table = torch.full((len(lens), per), -1, dtype=torch.int32)
    at = 0
    for n, length in enumerate(lens):
        for j in range(per):
            table[n, j] = order[at + j] if j < used[n] else [-1, 2 ** 31 - 1, total, -2 ** 31][(n + j) % 4]
        if used[n]:
            x = randn(g, length, 512 + rope).double() if make is None else make(n, length)
            y, e = q8.quantise(x)
            pos = torch.arange(length, device=DEV)
            pages = torch.tensor(order[at:at + used[n]], device=DEV)[pos // page]
            cache[pages, pos % page] = q8.bytes_of(y).view(U8)
            scales[pages, pos % page] = (e + 127).to(U8)
        at += used[n]
    return cache.view(q8.E4M3), scales.view(q8.E8M0), table.to(DEV)


def clean():
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0


def positions(counts, lens, table, page):
    """(sequence, position, cache row) of every new token."""
    pos = torch.cat([torch.arange(n - c, n, device=DEV) for c, n in zip(counts, lens)])
    seq = torch.repeat_interleave(torch.arange(len(counts), device=DEV), torch.tensor(counts, device=DEV))
    return seq, pos, table.long()[seq, pos // page] * page + pos % page


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("counts,past,H,page,rope", [
    ([1], [0], 1, 16, 64), ([1, 1, 1], [5, 0, 63], 32, 64, 64), ([3, 0, 70, 1], [14, 9, 100, 0], 5, 16, 64),
    ([2, 5], [1, 30], 4, 32, 0), ([1500, 7, 900], [3, 0, 77], 3, 128, 64), ([2100], [9], 1, 1024, 0)])
def test_append(counts, past, H, page, rope, interleaved):
    g = gen(len(counts) + page)
    lens = [c + p for c, p in zip(counts, past)]
    cache, scales, table = paged(lens, page, rope, g)
    T, extra = sum(counts), 2
    size = torch.exp2(torch.randint(-9, 9, (T + extra, 1), generator=g, device=DEV).float()).to(BF)
    both = randn(g, T + extra, 576) * size                     # one projection: latent and key part side by side
    both[T // 2] = 0
    both[0, :3] = torch.tensor([448.0, -448.0, 450.0], device=DEV).to(BF)
    q = randn(g, T + extra, H, 192)                            # the queries' part is the end of each row
    seq, pos, slot = positions(counts, lens, table, page)
    width = 512 + rope
    want, want_scales = cache.view(U8).clone(), scales.view(U8).clone()
    q_out = torch.full((T + extra, H, 64), 7.0, dtype=BF, device=DEV) if rope else None
    got = kda.kda_latent_append_q8(both[:, :512], both[:, 512:] if rope else None, cache, scales, table, i32(lens),
                                   inv_freq=freqs(), interleaved=interleaved, q_rope=q[..., 128:] if rope else None,
                                   q_rope_out=q_out, cu_seqlens=i32(offsets(counts)))
    clean()
    x, off = both[:T, :512].double(), torch.zeros(T, 0, device=DEV, dtype=torch.float64)
    if rope:
        turned, _ = ref.rotate(both[:T, 512:], pos, freqs(), interleaved)
        part = both[:T, 512:].double()
        a, b = (part[:, 0::2], part[:, 1::2]) if interleaved else (part[:, :32], part[:, 32:])
        off = a.abs() + b.abs()                                # sines and cosines good to 2^-21 in fp32 products
        off = 2.0 ** -20 * (torch.stack((off, off), -1).flatten(-2) if interleaved else torch.cat((off, off), 1))
        x = torch.cat([x, turned], 1)
    y = cache.view(U8).view(-1, width)[slot].view(q8.E4M3).double()
    e = scales.view(U8).view(-1)[slot].double() - 127
    exact = q8.power_of_rows(x)
    if rope:                                                   # a largest channel at a border may fall on either side of it
        lo, hi = q8.power_of_rows((x.abs() - torch.cat([torch.zeros_like(x[:, :512]), off], 1)).clamp_min(0)), \
            q8.power_of_rows(x.abs() + torch.cat([torch.zeros_like(x[:, :512]), off], 1))
        assert bool(((e >= lo) & (e <= hi)).all())
    else:
        assert torch.equal(e, exact)
    assert torch.equal(y[:, :512], q8.to_e4m3(x[:, :512] * q8.two(-e)[:, None]))            # not rotated: bit for bit
    if rope:
        v, b = y[:, 512:] * q8.two(e)[:, None], off + 2.0 ** -4 * (x[:, 512:].abs() + off) + 2.0 ** -10 * q8.two(e)[:, None]
        ref.assert_within(v, x[:, 512:], b, "cached key part")
        w, b = ref.rotate(q[:T, :, 128:], pos, freqs(), interleaved)
        ref.assert_within(got[:T], w, b, "queries")
        assert bool((got[T:] == 7.0).all())                    # rows of no sequence are left alone
    else:
        assert got is None
    want.view(-1, width)[slot] = cache.view(U8).view(-1, width)[slot]
    want_scales.view(-1)[slot] = scales.view(U8).view(-1)[slot]
    assert torch.equal(cache.view(U8), want) and torch.equal(scales.view(U8), want_scales)  # the rest is left as it was


def test_append_borders_of_the_format():
    """Every bf16 magnitude of a row alone beside small ones, ties, the format's ends, and what is not finite."""
    edges = torch.tensor([448.0, 450.0, 224.0, 226.0, 449.0 * 2.0 ** -56, 448 * 2.0 ** -64, 2.0 ** -70, 2.0 ** -80, 2.0 ** -133,
                          448 * 2.0 ** 118, 2.0 ** 127, 1.0, 1.75, 1.7578125, 0.0], device=DEV).to(BF)
    n = edges.numel() + 2
    lat = torch.zeros(n, 512, dtype=BF, device=DEV)
    lat[:-2] = edges[:, None] * torch.linspace(-1, 1, 512, device=DEV).to(BF)
    lat[:-2, 7] = edges
    lat[-2, 3], lat[-1, 5] = math.inf, math.nan
    lat[-2, 4] = lat[-1, 4] = 1.0
    cache = torch.zeros(2, 16, 512, dtype=U8, device=DEV).view(q8.E4M3)
    scales = torch.zeros(2, 16, dtype=U8, device=DEV).view(q8.E8M0)
    kda.kda_latent_append_q8(lat, None, cache, scales, i32([[1, 0]]), i32([n]))
    clean()
    y = torch.cat([cache[1], cache[0]])[:n].double()
    e = torch.cat([scales.view(U8)[1], scales.view(U8)[0]])[:n].double() - 127
    want, power = q8.quantise(lat[:-2].double())
    assert torch.equal(e[:-2], power) and torch.equal(y[:-2], want)
    assert float(e[-2]) == 120 and float(y[-2, 3]) == 448 and float(y[-2, 4]) == 0
    assert float(e[-1]) == 120 and math.isnan(float(y[-1, 5])) and float(y[-1, 4]) == 0
    got, _ = kda.kda_latent_gather_q8(cache, scales, i32([[1, 0]]), [0, n - 2], n - 2)
    assert torch.equal(got.double(), want * q8.two(power)[:, None])


def test_append_in_place_and_without_rotation():
    g = gen(3)
    cache, scales, table = paged([40, 33], 16, 64, g)
    q = randn(g, 6, 4, 192)
    before = q.clone()
    lat, kr = randn(g, 6, 512), randn(g, 6, 64)
    kda.kda_latent_append_q8(lat, kr, cache, scales, table, i32([40, 33]), inv_freq=freqs(), q_rope=q[..., 128:],
                             q_rope_out=q[..., 128:])          # three tokens a sequence
    pos = torch.tensor([37, 38, 39, 30, 31, 32], device=DEV)
    y, b = ref.rotate(before[..., 128:], pos, freqs(), False)
    ref.assert_within(q[..., 128:], y, b, "in place")
    assert torch.equal(q[..., :128], before[..., :128])
    for interleaved in (False, True):
        kept = kda.kda_latent_append_q8(lat, kr, cache, scales, table, i32([40, 33]), interleaved=interleaved, q_rope=before[..., 128:])
        assert torch.equal(kept, before[..., 128:])
        y, e = q8.rows_of(cache, scales, table, 0, 40)
        want, power = q8.quantise(torch.cat([lat, kr], 1)[:3].double())
        assert torch.equal(y[37:], want) and torch.equal(e[37:], power)
    clean()


def test_append_leaves_out_what_has_no_row():
    """A padded batch: an empty slot whose length is shorter than its tokens, a page outside the cache."""
    g = gen(5)
    cache, scales, table = paged([20, 20, 20], 16, 64, g)
    table[1, 1] = cache.shape[0]                               # sequence 1's second page is outside
    before, before_scales = cache.view(U8).clone(), scales.view(U8).clone()
    lat, kr, q = randn(g, 6, 512), randn(g, 6, 64), randn(g, 6, 2, 64)
    for lens, rows in (([20, 20, 1], [(0, 18, 0), (0, 19, 1), (2, 0, 5)]), ([10 ** 9, -5, 1], [(2, 0, 5)])):
        out = kda.kda_latent_append_q8(lat, kr, cache, scales, table, i32(lens), q_rope=q, inv_freq=freqs())
        clean()
        for n, p, t in rows:
            at = (int(table[n, p // 16]), p % 16)
            y, e = q8.to_e4m3(lat[t].double() * q8.two(127 - scales.view(U8)[at].long())), scales.view(U8)[at]
            assert torch.equal(cache[at][:512].double(), y) and int(e) != 0
            before[at], before_scales[at] = cache.view(U8)[at], scales.view(U8)[at]
        assert torch.equal(cache.view(U8), before) and torch.equal(scales.view(U8), before_scales)
        assert bool(out.isfinite().all())


# ---------------------------------------------------------------- gather

@pytest.mark.parametrize("counts,starts,page,rope", [
    ([1], None, 16, 64), ([5, 0, 70], [3, 1, 16], 16, 64), ([300, 1], None, 64, 0), ([9000, 500], [7, 0], 128, 64)])
def test_gather(counts, starts, page, rope):
    g = gen(page + rope)
    at = [0] * len(counts) if starts is None else starts
    cache, scales, table = paged([c + s for c, s in zip(counts, at)], page, rope, g)
    cu = offsets(counts)
    T = cu[-1] + 3
    out = (torch.full((T, 512), 7.0, dtype=BF, device=DEV), torch.full((T, 64), 7.0, dtype=BF, device=DEV) if rope else None)
    lat, kr = kda.kda_latent_gather_q8(cache, scales, table, i32(cu), T, None if starts is None else i32(starts), out=out)
    clean()
    want = []
    for n, (c, s) in enumerate(zip(counts, at)):
        y, e = q8.rows_of(cache, scales, table, n, c + s)
        want.append((y * q8.two(e)[:, None])[s:])
    want = torch.cat(want)
    assert torch.equal(lat[:cu[-1]].double(), want[:, :512]) and bool((lat[cu[-1]:] == 7.0).all())
    if rope:
        assert torch.equal(kr[:cu[-1]].double(), want[:, 512:]) and bool((kr[cu[-1]:] == 7.0).all())
    else:
        assert kr is None


def test_gather_of_missing_rows_is_zero_and_of_every_byte_exact():
    g = gen(6)
    cache, scales, table = paged([40], 16, 64, g, per=3)
    table[0, 1] = -1
    lat, kr = kda.kda_latent_gather_q8(cache, scales, table, [0, 50], 50, i32([-2]))
    y, e = q8.rows_of(cache, scales, table, 0, 40)
    want = torch.zeros(50, 576, dtype=torch.float64, device=DEV)
    want[2:42] = y * q8.two(e)[:, None]
    got = torch.cat([lat, kr], 1).double()
    ok = torch.ones(50, dtype=torch.bool, device=DEV)
    ok[42:] = False                                            # rows behind the end: as they lie there
    assert torch.equal(got[ok], want[ok])
    # all 256 numbers under all 256 scale bytes
    page = torch.arange(512, device=DEV).to(U8).expand(256, 1, 512).repeat(1, 16, 1)
    powers = torch.arange(256, device=DEV).to(U8)[:, None].repeat(1, 16)
    every = page.view(q8.E4M3)
    got, _ = kda.kda_latent_gather_q8(every, powers.view(q8.E8M0), torch.arange(256, dtype=torch.int32, device=DEV)[None], [0, 4096], 4096)
    clean()
    want = q8.values(every, powers).view(4096, 512)
    fine = want.abs() < 2.0 ** 128
    assert torch.equal(got.double()[fine], want[fine]) and bool(got[want.isnan()].isnan().all())


# ---------------------------------------------------------------- decode

def check_decode(lens, T, H, page, rope, seed, scale=None, std=1.0, make=None, **kw):
    g = gen(seed)
    cache, scales, table = paged(lens, page, rope, g, make=make)
    q = randn(g, len(lens) * T, H, 512, std=std)
    qr = randn(g, len(lens) * T, H, 64, std=std) if rope else None
    scale = (128 + rope) ** -0.5 if scale is None else scale
    args = (q, qr, cache, scales, table, i32(lens), scale)
    out, lse = kda.kda_latent_decode_q8(*args, lse=True, **kw)
    clean()
    against(out, lse, args)
    return out, lse, args


def against(out, lse, args):
    o, s, bo, bs = q8.decode(*args)
    ref.assert_within(lse, s, bs, "lse")
    ref.assert_within(out, o, bo, "out")


@pytest.mark.parametrize("rope", [0, 64])
@pytest.mark.parametrize("H,T,page", [(1, 1, 16), (3, 1, 64), (16, 1, 32), (17, 1, 128), (32, 1, 64), (64, 1, 16),
                                      (96, 1, 64), (128, 1, 1024), (8, 2, 64), (5, 7, 16), (16, 4, 32), (32, 16, 256)])
def test_decode_shapes(H, T, page, rope):
    check_decode([T, 64, 127 + T, 129, 300, 1000], T, H, page, rope, seed=H + T)


def test_decode_lengths_of_one_sequence():
    for n in (1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 192, 255, 256, 257, 640, 4097):
        check_decode([n], 1, 32, 16, 64, seed=n)


def test_decode_sequences_that_see_nothing():
    """Empty sequences, sequences shorter than the step, and tokens of a step that see nothing."""
    out, lse, _ = check_decode([0, 5, 2, 0, 1, 300, -7], 4, 8, 16, 64, seed=9)
    assert bool((out[:4] == 0).all()) and bool((lse[:4] == -math.inf).all())
    assert bool((out[8:10] == 0).all()) and bool((lse[8:10] == -math.inf).all()) and bool(lse[10:12].isfinite().all())


def test_decode_lengths_beyond_the_table_are_clamped():
    g = gen(10)
    cache, scales, table = paged([64, 64], 16, 64, g, per=4)
    q, qr = randn(g, 2, 4, 512), randn(g, 2, 4, 64)
    out, lse = kda.kda_latent_decode_q8(q, qr, cache, scales, table, i32([2 ** 31 - 1, 65]), 0.07, lse=True)
    clean()
    against(out, lse, (q, qr, cache, scales, table, i32([64, 64]), 0.07))


def test_decode_pages_outside_the_cache_read_as_zero_rows():
    g = gen(11)
    cache, scales, table = paged([300, 70], 16, 64, g, per=19)
    for j, bad in ((0, -1), (5, cache.shape[0]), (6, 2 ** 31 - 1), (18, -2 ** 31)):
        table[0, j] = bad
    table[1, 4] = -9
    args = (randn(g, 2, 32, 512), randn(g, 2, 32, 64), cache, scales, table, i32([300, 70]), 0.07)
    out, lse = kda.kda_latent_decode_q8(*args, lse=True)
    clean()
    against(out, lse, args)


@pytest.mark.parametrize("factor", [0.02, 0.8])
@pytest.mark.parametrize("falling", [False, True])
def test_decode_rising_and_falling_scores(factor, falling):
    """Keys that grow, or shrink, with the position move the tiles' maxima all the way; with the large factor one key
    takes all the weight."""
    h = gen(99)

    def make(n, count):
        size = torch.arange(count, device=DEV) // 64 + 1.0
        return randn(h, count, 576).double() * factor * (size.flip(0) if falling else size)[:, None]
    check_decode([13 * 64, 13 * 64 - 5, 129], 2, 16, 64, 64, seed=12, make=make)


def test_decode_a_sink_and_a_long_faint_tail():
    """The first key takes far more weight than any other, but the others together count: e^11 against 20000 keys of
    about 1.  Their values share a direction, so that weights lost or rounded to one side would show."""
    n = 20000

    def make(i, count):
        x = torch.zeros(count, 512, dtype=torch.float64, device=DEV)
        x[:, 100:] = 1 + 0.1 * torch.randn(count, 412, generator=gen(5), device=DEV)
        x[0, 100:] = -1
        x[0, 0] = 11 * (i + 1)                                 # sequence 1: e^22, where the tail no longer counts
        return x
    g = gen(6)
    cache, scales, table = paged([n, n], 64, 0, g, make=make)
    q = torch.zeros(2, 16, 512, dtype=BF, device=DEV)
    q[..., 0] = 1
    args = (q, None, cache, scales, table, i32([n, n]), 1.0)
    out, lse = kda.kda_latent_decode_q8(*args, lse=True)
    clean()
    o, s, bo, _ = q8.decode(*args)
    ref.assert_within(lse, s, 1e-5 * s.abs(), "lse")
    # rounding weights: 2^-8 of each (independent in the mean), and once more the output
    ref.assert_within(out, o, 2 * q8.U * o.abs().amax() + torch.zeros_like(o), "out")
    assert float((out[0, :, 100:].double() - o[0, :, 100:]).abs().max()) < 4 * q8.U


def test_decode_rows_of_very_different_sizes():
    """Scale bytes over the whole format, rows of zeros and tiny rows beside large ones."""
    h = gen(41)

    def make(n, count):
        size = torch.exp2(torch.randint(-70, 4, (count, 1), generator=h, device=DEV).double())
        size[::7] = 0
        return randn(h, count, 576).double() * size
    check_decode([700, 129, 3], 1, 32, 64, 64, seed=42, make=make)
    check_decode([300], 1, 4, 16, 0, seed=43, make=lambda n, c: torch.zeros(c, 512, dtype=torch.float64, device=DEV))


def test_decode_queries_of_very_different_channels():
    g = gen(44)
    cache, scales, table = paged([500, 65], 64, 64, g)
    size = torch.exp2(torch.randint(-30, 6, (2, 8, 576), generator=g, device=DEV).float()).to(BF)
    q = randn(g, 2, 8, 576) * size
    q[0, 3] = 0
    args = (q[..., :512].contiguous(), q[..., 512:].contiguous(), cache, scales, table, i32([500, 65]), 0.02)
    out, lse = kda.kda_latent_decode_q8(*args, lse=True)
    clean()
    against(out, lse, args)


def test_decode_large_values():
    check_decode([500, 65], 1, 32, 64, 64, seed=13, scale=1.0, std=4.0)


def test_decode_many_sequences_and_few_long_ones():
    g = torch.Generator().manual_seed(1)
    check_decode(torch.randint(1, 400, (700,), generator=g).tolist(), 1, 8, 64, 64, seed=14)
    check_decode([20000, 3, 9000], 1, 32, 64, 0, seed=15)
    check_decode([0] * 40 + [5000] + [1] * 40, 1, 16, 64, 64, seed=16)


@pytest.mark.parametrize("seed", range(12))
def test_decode_cuts_of_mixed_batches(seed):
    """Batches of short and long sequences in random order: whole sequences, cut ones and empty ones side by side."""
    g = torch.Generator().manual_seed(1000 + seed)
    pick = lambda xs: xs[int(torch.randint(len(xs), (1,), generator=g))]  # noqa: E731
    H, T, rope = pick([4, 32, 40, 64]), pick([1, 2, 8]), pick([0, 64])
    choices = [0, 1, 63, 64, 65, 128, 300, 384, 385, 1000, 3001][:pick([6, 9, 11])]
    lens = [pick(choices) for _ in range(pick([2, 9, 37, 150, 400]))]
    check_decode(lens, T, H, pick([16, 64, 256]), rope, seed=2000 + seed)


def test_decode_repeats_bit_for_bit_and_shares_pages():
    out, lse, args = check_decode([3000, 129, 64, 3000], 1, 32, 64, 64, seed=17)
    q, qr, cache, scales, table, lens, scale = args
    again, lse2 = kda.kda_latent_decode_q8(*args, lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    table[3] = table[0]                                        # two sequences over one set of pages
    shared, lse2 = kda.kda_latent_decode_q8(*args, lse=True)
    against(shared, lse2, args)


def test_cache_beyond_32_bit_offsets():
    """Pages at the end of a cache of more than 2^32 bytes."""
    g = gen(18)
    page = 64
    pages = 2 ** 32 // (page * 576) + 100
    cache = torch.empty((pages, page, 576), dtype=U8, device=DEV).view(q8.E4M3)
    scales = torch.zeros((pages, page), dtype=U8, device=DEV).view(q8.E8M0)
    lens = [300, 150]
    table = torch.tensor([[pages - 1 - j for j in range(5)], [pages - 9 - j for j in range(5)]], dtype=torch.int32, device=DEV)
    lat, kr = randn(g, 450, 512), randn(g, 450, 64)
    kda.kda_latent_append_q8(lat, kr, cache, scales, table, i32(lens), cu_seqlens=[0, 300, 450])
    y, e = q8.quantise(torch.cat([lat, kr], 1).double())
    for n, (a, b) in enumerate(((0, 300), (300, 450))):
        got = q8.rows_of(cache, scales, table, n, b - a)
        assert torch.equal(got[0], y[a:b]) and torch.equal(got[1], e[a:b])
    args = (randn(g, 2, 32, 512), randn(g, 2, 32, 64), cache, scales, table, i32(lens), 0.07)
    out, lse = kda.kda_latent_decode_q8(*args, lse=True)
    got, _ = kda.kda_latent_gather_q8(cache, scales, table, [0, 300, 450], 450)
    clean()
    against(out, lse, args)
    assert torch.equal(got.double(), (y * q8.two(e)[:, None])[:, :512])


def test_decode_a_context_of_a_million_tokens():
    """2^20 tokens over 64 distinct pages, and a short neighbour."""
    g = gen(20)
    y, e = q8.quantise(randn(g, 64, 1024, 576).double())
    cache, scales = q8.bytes_of(y), q8.powers_of(e)
    table = torch.randint(0, 64, (2, 1024), generator=g, device=DEV).to(torch.int32)
    args = (randn(g, 2, 16, 512), randn(g, 2, 16, 64), cache, scales, table, i32([2 ** 20, 77]), 0.07)
    out, lse = kda.kda_latent_decode_q8(*args, lse=True)
    clean()
    against(out, lse, args)


def test_decode_without_pages():
    """No pages, no table entries: nothing is seen."""
    q, qr = torch.ones(3, 4, 512, dtype=BF, device=DEV), torch.ones(3, 4, 64, dtype=BF, device=DEV)
    empty = torch.empty(0, 64, 576, dtype=U8, device=DEV).view(q8.E4M3)
    powers = torch.empty(0, 64, dtype=U8, device=DEV).view(q8.E8M0)
    for per, lens, want in ((0, [5, 0, 9], [-math.inf] * 3), (2, [5, 0, 128], [math.log(5), -math.inf, math.log(128)])):
        out, lse = kda.kda_latent_decode_q8(q, qr, empty, powers, torch.zeros(3, per, dtype=torch.int32, device=DEV), i32(lens),
                                            0.07, lse=True)
        clean()
        assert bool((out == 0).all())                          # rows of pages that are not there are zeros
        torch.testing.assert_close(lse[:, 0].cpu(), torch.tensor(want), rtol=1e-6, atol=1e-6)


def test_decode_writes_no_row_but_its_own():
    g = gen(19)
    cache, scales, table = paged([100, 40, 7], 16, 64, g)
    q, qr = randn(g, 3, 5, 512), randn(g, 3, 5, 64)
    big = torch.full((5, 5, 512), 7.0, dtype=BF, device=DEV)
    lse = torch.full((5, 5), 7.0, device=DEV)
    kda.kda_latent_decode_q8(q, qr, cache, scales, table, i32([100, 40, 7]), 0.07, out=big[1:4], lse=lse[1:4])
    clean()
    for x in (big[0], big[4], lse[0], lse[4]):
        assert bool((x == 7.0).all())


# ---------------------------------------------------------------- what the binding refuses

def test_binding_refusals():
    g = gen(22)
    cache, scales, table = paged([70, 40], 16, 64, g)
    lens = i32([70, 40])
    lat, kr, q, qr = randn(g, 2, 512), randn(g, 2, 64), randn(g, 2, 4, 512), randn(g, 2, 4, 64)
    ok = dict(q_latent=q, q_rope=qr, cache=cache, scales=scales, block_table=table, seq_lens=lens, scale=0.07)
    kda.kda_latent_decode_q8(**ok)
    plain = torch.zeros(cache.shape, dtype=BF, device=DEV)
    for bad, error in ((dict(cache=plain), TypeError), (dict(cache=cache.view(U8)), TypeError), (dict(scales=scales.view(U8)), TypeError),
                       (dict(scales=scales[:-1]), ValueError), (dict(scales=scales.view(-1)), ValueError), (dict(scales=scales.cpu()), ValueError),
                       (dict(scales=None), TypeError), (dict(q_rope=None), ValueError), (dict(cache=cache[..., :512]), ValueError),
                       (dict(q_latent=q.float()), TypeError), (dict(out=q[:1]), ValueError)):
        with pytest.raises(error):
            kda.kda_latent_decode_q8(**{**ok, **bad})
    with pytest.raises(TypeError):
        kda.kda_latent_decode(q, qr, cache, table, lens, 0.07)            # the bf16 call on an 8-bit cache
    with pytest.raises(kda.KdaError) as e:
        kda.kda_latent_decode_q8(**{**ok, "scale": -1.0})
    assert e.value.status == 1
    for bad, error in ((dict(cache=plain), TypeError), (dict(scales=scales[:1]), ValueError), (dict(k_rope=None), ValueError),
                       (dict(latent=lat.float()), TypeError)):
        with pytest.raises(error):
            kda.kda_latent_append_q8(**{**dict(latent=lat, k_rope=kr, cache=cache, scales=scales, block_table=table, seq_lens=lens), **bad})
    with pytest.raises(TypeError):
        kda.kda_latent_gather_q8(plain, scales, table, [0, 1, 2], 2)
    with pytest.raises(ValueError):
        kda.kda_latent_gather_q8(cache, scales[:, :8], table, [0, 1, 2], 2)
    clean()


# ---------------------------------------------------------------- streams, graphs, the run of them

def test_side_stream_and_captured_graph():
    """The calls on another stream, and captured once and replayed with new lengths and queries."""
    g = gen(12)
    lens = i32([130, 900, 64])
    cache, scales, table = paged([2000, 2000, 2000], 64, 64, g)
    q, qr = randn(g, 3, 32, 512), randn(g, 3, 32, 64)
    lat, kr, qn = randn(g, 3, 512), randn(g, 3, 64), randn(g, 3, 32, 64)
    ws = torch.empty(kda.kda_latent_decode_q8_workspace_size(3, 3, 32), dtype=U8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(3, 32, device=DEV)
    freq = freqs()

    def step():
        kda.kda_latent_append_q8(lat, kr, cache, scales, table, lens, inv_freq=freq, q_rope=qn, q_rope_out=qr)
        kda.kda_latent_decode_q8(q, qr, cache, scales, table, lens, 0.07, out=out, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, new in ((1, [131, 901, 65]), (2, [1, 2000, 300])):
        h = gen(seed)
        q.copy_(randn(h, 3, 32, 512))
        lat.copy_(randn(h, 3, 512))
        lens.copy_(i32(new))
        graph.replay()
        torch.cuda.synchronize()
        against(out, lse, (q, qr, cache, scales, table, lens, 0.07))
    clean()


def test_two_streams_at_once():
    """Two decodes in flight together, each with its own workspace, and calls with a stream argument."""
    g = gen(13)
    sets = []
    for k in range(2):
        cache, scales, table = paged([3000, 1700, 64], 64, 64, g)
        sets.append((randn(g, 3, 32, 512), randn(g, 3, 32, 64), cache, scales, table, i32([3000, 1700, 64]), 0.07))
    alone = [kda.kda_latent_decode_q8(*x)[0] for x in sets]
    rows = [kda.kda_latent_gather_q8(x[2], x[3], x[4], [0, 3000, 4700, 4764], 4764)[0] for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    together = []
    for x, st in zip(sets, streams):
        for _ in range(3):
            a = kda.kda_latent_decode_q8(*x, stream=st)[0]
            b = kda.kda_latent_gather_q8(x[2], x[3], x[4], [0, 3000, 4700, 4764], 4764, stream=st.cuda_stream)[0]
        together.append((a, b))
    torch.cuda.synchronize()
    for k in range(2):
        assert torch.equal(together[k][0], alone[k]) and torch.equal(together[k][1], rows[k])
    lat, kr, qn = randn(g, 3, 512), randn(g, 3, 64), randn(g, 3, 4, 64)
    kda.kda_latent_append_q8(lat, kr, *sets[0][2:6], q_rope=qn, stream=streams[0])
    streams[0].synchronize()
    y, e = q8.rows_of(*sets[0][2:5], 0, 3000)
    want, power = q8.quantise(torch.cat([lat, kr], 1)[:1].double())
    assert torch.equal(y[2999:], want) and torch.equal(e[2999:], power)
    clean()


FIRST_CAPTURE = """
import torch, linear_attention_06_gb300 as kda
BF, d = torch.bfloat16, "cuda"
z = lambda *s: torch.randn(*s, device=d).to(BF)
i = lambda x: torch.tensor(x, dtype=torch.int32, device=d)
def call(H, T, rope, nk, n):
    page = 64
    cache, table = z(40 * n, page, 512 + rope).to(torch.float8_e4m3fn), torch.arange(n * 40, dtype=torch.int32, device=d).view(n, 40)
    scales = torch.full((40 * n, page), 127, dtype=torch.uint8, device=d).view(torch.float8_e8m0fnu)
    lens, f = i([min(2500, nk)] * n), torch.rand(32, device=d)
    lat, kr, q = z(n * T, 512), z(n * T, 64) if rope else None, z(n * T, H, 64) if rope else None
    ql = z(n * T, H, 512)
    cu = torch.arange(n + 1, dtype=torch.int32, device=d) * 100
    def run():
        kda.kda_latent_append_q8(lat, kr, cache, scales, table, lens, inv_freq=f if rope else None, q_rope=q)
        return (kda.kda_latent_gather_q8(cache, scales, table, cu, 100 * n)[0],
                kda.kda_latent_decode_q8(ql, q, cache, scales, table, lens, 0.1)[0])
    return run
call(4, 1, 64, 20, 1)()
call(4, 1, 0, 20, 1)()
torch.cuda.synchronize()
for args in ((4, 1, 64, 4000, 1), (32, 2, 0, 8000, 40), (64, 1, 64, 700, 2), (20, 1, 0, 30, 3)):
    run = call(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    torch.cuda.synchronize()
    first = [x.clone() for x in got]
    for a, b in zip(first, run()):
        assert torch.equal(a, b), args
assert kda.kda_device_status() == 0
"""


def test_forms_first_met_in_a_capture():
    """One call of each operator and row width loads its kernels: every other form may then first be met in a capture."""
    done = subprocess.run([sys.executable, "-c", FIRST_CAPTURE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_prompt_then_steps_over_one_cache():
    """A prompt quantised into the cache, read back, up-projected and attended in the expanded form; then a step whose
    rows join the cache, in the absorbed form and in the expanded form: one model, two forms, one result."""
    g = gen(14)
    H, page, nq = 8, 16, [90, 33]
    w_k = (torch.randn(H, 512, 128, generator=g, device=DEV) / 512 ** 0.5).to(BF)
    w_v = (torch.randn(H, 512, 128, generator=g, device=DEV) / 512 ** 0.5).to(BF)
    step, scale, freq = 3, 192 ** -0.5, freqs()
    top = [n + step for n in nq]
    cache, scales, table = paged(top, page, 64, g)
    cache.view(U8).fill_(0x7F)
    scales.view(U8).fill_(255)

    def tokens(counts, lens):
        T = sum(counts)
        cu = i32(offsets(counts))
        q = randn(g, T, H, 192)
        kda.kda_latent_append_q8(randn(g, T, 512), randn(g, T, 64), cache, scales, table, i32(lens), inv_freq=freq,
                                 q_rope=q[..., 128:], q_rope_out=q[..., 128:], cu_seqlens=cu)
        return q, cu

    def expanded(q, cu, lens):
        ck = i32(offsets(lens))
        lat, kr = kda.kda_latent_gather_q8(cache, scales, table, ck, sum(lens))
        k = torch.einsum("tc,hcd->thd", lat.float(), w_k.float()).to(BF).contiguous()
        v = torch.einsum("tc,hcd->thd", lat.float(), w_v.float()).to(BF).contiguous()
        out, _ = kda.kda_latent_prefill(q, k, v, kr, scale, cu, ck)
        o, _, bo, _ = ref.prefill(q, k, v, kr, scale, cu.tolist(), ck.tolist())
        ref.assert_within(out, o, bo, "expanded")
        return out

    q, cu = tokens(nq, nq)
    expanded(q, cu, nq)
    q, cu = tokens([step, step], top)                          # the step's rows join the cache
    want = expanded(q, cu, top)
    q_lat = torch.einsum("thd,hcd->thc", q[..., :128].float(), w_k.float()).to(BF).contiguous()
    o_lat, _ = kda.kda_latent_decode_q8(q_lat, q[..., 128:].contiguous(), cache, scales, table, i32(top), scale)
    got = torch.einsum("thc,hcd->thd", o_lat.double(), w_v.double())
    clean()
    # both forms read the same quantised rows; they round k, v, q_lat and o_lat at different places, each by at most
    # 2^-8 of its value; of independent roundings over 128 and 512 terms about as much is left in the norm
    assert float((got - want.double()).norm() / want.double().norm()) < 4 * ref.U


def test_no_index_leaves_its_buffer():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "latent_q8_bounds_run.py")], capture_output=True,
                         text=True, timeout=1200, cwd=ROOT)
    assert out.returncode == 0, out.stdout[-3000:] + out.stderr[-3000:]
    assert "bounds ok" in out.stdout
