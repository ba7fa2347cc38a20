"""Latent attention on the GPU against the 64-bit formulas of tests/latent_reference.py: the cache, the
absorbed decode, the expanded prefill, and a run of them together."""
import math
import os
import subprocess
import sys

import pytest
import torch

import linear_attention_06_gb300 as kda
from tests import latent_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16
NAN = float("nan")


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


def paged(lens, page, rope, g, extra_pages=3, per=None, std=1.0):
    """A cache whose rows behind the sequences' ends hold NaN, on pages in random order; the table's entries
    behind a sequence's last page are nonsense."""
    used = [-(-n // page) for n in lens]
    per = max(used + [1]) + 1 if per is None else per
    total = sum(used) + extra_pages
    order = torch.randperm(total, generator=g, device=DEV).tolist()
    cache = torch.full((total, page, 512 + rope), NAN, dtype=BF, device=DEV)
    table = torch.full((len(lens), per), -1, dtype=torch.int32)
    at = 0
    for n, length in enumerate(lens):
        for j in range(per):
            table[n, j] = order[at + j] if j < used[n] else [-1, 2 ** 31 - 1, total, -2 ** 31][(n + j) % 4]
        for j in range(used[n]):
            m = min(page, length - j * page)
            cache[order[at + j], :m] = randn(g, m, 512 + rope, std=std)
        at += used[n]
    return cache, table.to(DEV)


def clean():
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("counts,past,H,page,rope", [
    ([1], [0], 1, 16, 64), ([1, 1, 1], [5, 0, 63], 32, 64, 64), ([3, 0, 70, 1], [14, 9, 100, 0], 5, 16, 64),
    ([2, 5], [1, 30], 4, 32, 0), ([1500, 7, 900], [3, 0, 77], 3, 128, 64)])
def test_append(counts, past, H, page, rope, interleaved):
    g = gen(len(counts) + page)
    lens = [c + p for c, p in zip(counts, past)]
    cache, table = paged(lens, page, rope, g)
    T, extra = sum(counts), 2
    both = randn(g, T + extra, 512 + 64)                       # one projection: latent and key part side by side
    q = randn(g, T + extra, H, 192)                            # the queries' part is the end of each row
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    want = cache.clone()
    pos = torch.cat([torch.arange(p, p + c, device=DEV) for c, p in zip(counts, past)] + [torch.zeros(0, device=DEV)]).long()
    seq = torch.repeat_interleave(torch.arange(len(counts), device=DEV), torch.tensor(counts, device=DEV))
    slot = table.long()[seq, pos // page] * page + pos % page
    want.view(-1, 512 + rope)[slot, :512] = both[:T, :512]
    q_out = torch.full((T + extra, H, 64), 7.0, dtype=BF, device=DEV) if rope else None
    got = kda.kda_latent_append(both[:, :512], both[:, 512:] if rope else None, cache, table, i32(lens),
                                inv_freq=freqs(), interleaved=interleaved, q_rope=q[..., 128:] if rope else None,
                                q_rope_out=q_out, cu_seqlens=i32(cu))
    clean()
    if rope:
        y, b = ref.rotate(both[:T, 512:], pos, freqs(), interleaved)
        ref.assert_within(cache.view(-1, 576)[slot, 512:], y, b, "cached key part")
        want.view(-1, 576)[slot, 512:] = cache.view(-1, 576)[slot, 512:]
        y, b = ref.rotate(q[:T, :, 128:], pos, freqs(), interleaved)
        ref.assert_within(got[:T], y, b, "queries")
        assert bool((got[T:] == 7.0).all())                    # rows of no sequence are left alone
    else:
        assert got is None
    assert torch.equal(cache.view(torch.int16), want.view(torch.int16))   # the rest is left as it was, bit for bit


def test_append_in_place_and_without_rotation():
    g = gen(3)
    cache, table = paged([40, 33], 16, 64, g)
    q = randn(g, 6, 4, 192)
    before = q.clone()
    lat, kr = randn(g, 6, 512), randn(g, 6, 64)
    kda.kda_latent_append(lat, kr, cache, table, i32([40, 33]), inv_freq=freqs(), q_rope=q[..., 128:],
                          q_rope_out=q[..., 128:])             # three tokens a sequence
    pos = torch.tensor([37, 38, 39, 30, 31, 32], device=DEV)
    y, b = ref.rotate(before[..., 128:], pos, freqs(), False)
    ref.assert_within(q[..., 128:], y, b, "in place")
    assert torch.equal(q[..., :128], before[..., :128])
    kept = kda.kda_latent_append(lat, kr, cache, table, i32([40, 33]), q_rope=before[..., 128:])
    assert torch.equal(kept, before[..., 128:])
    assert torch.equal(ref.rows_of(cache, table, 0, 40)[37:, 512:], kr[:3].double())
    clean()


def test_append_far_positions_keep_their_angles():
    """Positions near 2^20 and 2^30: a table row of few distinct pages stands for a long context."""
    g = gen(4)
    lens = [2 ** 20 + 5, 2 ** 30 - 3]
    page, per = 1024, 2 ** 20
    table = torch.zeros((2, per), dtype=torch.int32, device=DEV)
    table[1] = 1
    cache = torch.zeros((2, page, 576), dtype=BF, device=DEV)
    kr, q = randn(g, 4, 64), randn(g, 4, 2, 64)
    out = kda.kda_latent_append(randn(g, 4, 512), kr, cache, table, i32(lens), inv_freq=freqs(), q_rope=q)
    pos = torch.tensor([lens[0] - 2, lens[0] - 1, lens[1] - 2, lens[1] - 1], device=DEV)
    y, b = ref.rotate(q, pos, freqs(), False)
    ref.assert_within(out, y, b, "far queries")
    y, b = ref.rotate(kr, pos, freqs(), False)
    slot = torch.tensor([0, 0, 1, 1], device=DEV) * page + pos % page
    ref.assert_within(cache.view(-1, 576)[slot, 512:], y, b, "far keys")
    clean()


def test_append_leaves_out_what_has_no_row():
    """A padded batch: an empty slot whose length is shorter than its tokens, a page outside the cache."""
    g = gen(5)
    cache, table = paged([20, 20, 20], 16, 64, g)
    table[1, 1] = cache.shape[0]                               # sequence 1's second page is outside
    before = cache.clone()
    lat, kr, q = randn(g, 6, 512), randn(g, 6, 64), randn(g, 6, 2, 64)
    out = kda.kda_latent_append(lat, kr, cache, table, i32([20, 20, 1]), q_rope=q, inv_freq=freqs())
    clean()
    rows = ref.rows_of(cache, table, 0, 20)
    assert torch.equal(rows[18:, :512], lat[:2].double())
    assert torch.equal(ref.rows_of(cache, table, 2, 1)[0, :512], lat[5].double())   # position 0; position -1 has no row
    changed = (cache.view(torch.int16) != before.view(torch.int16)).any(-1).sum()
    assert int(changed) == 3
    assert bool(out.isfinite().all())
    # lengths beyond the table, and below zero, give positions without a row
    before = cache.clone()
    out = kda.kda_latent_append(lat, kr, cache, table, i32([10 ** 9, -5, 1]), q_rope=q, inv_freq=freqs())
    clean()
    before[table[2, 0].long(), 0] = cache[table[2, 0].long(), 0]
    assert torch.equal(cache.view(torch.int16), before.view(torch.int16))
    pos = torch.tensor([10 ** 9 - 2, 10 ** 9 - 1, -7, -6, -1, 0], device=DEV)
    y, b = ref.rotate(q, pos, freqs(), False)
    ref.assert_within(out, y, b, "queries without a row")


# ---------------------------------------------------------------- gather

@pytest.mark.parametrize("counts,starts,page,rope", [
    ([1], None, 16, 64), ([5, 0, 70], [3, 1, 16], 16, 64), ([300, 1], None, 64, 0), ([9000, 500], [7, 0], 128, 64)])
def test_gather(counts, starts, page, rope):
    g = gen(page + rope)
    at = [0] * len(counts) if starts is None else starts
    cache, table = paged([c + s for c, s in zip(counts, at)], page, rope, g)
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    T = cu[-1] + 3
    out = (torch.full((T, 512), 7.0, dtype=BF, device=DEV), torch.full((T, 64), 7.0, dtype=BF, device=DEV) if rope else None)
    lat, kr = kda.kda_latent_gather(cache, table, i32(cu), T, None if starts is None else i32(starts), out=out)
    clean()
    want = torch.cat([ref.rows_of(cache, table, n, c + s)[s:] for n, (c, s) in enumerate(zip(counts, at))])
    assert torch.equal(lat[:cu[-1]].double(), want[:, :512]) and bool((lat[cu[-1]:] == 7.0).all())
    if rope:
        assert torch.equal(kr[:cu[-1]].double(), want[:, 512:]) and bool((kr[cu[-1]:] == 7.0).all())
    else:
        assert kr is None


def test_gather_of_missing_rows_is_zero():
    g = gen(6)
    cache, table = paged([40], 16, 64, g, per=3)
    table[0, 1] = -1
    lat, kr = kda.kda_latent_gather(cache, table, [0, 50], 50, i32([-2]))
    clean()
    want = torch.zeros(50, 576, dtype=torch.float64, device=DEV)
    want[2:42] = ref.rows_of(cache, table, 0, 40)
    got = torch.cat([lat, kr], 1).double()
    ok = torch.ones(50, dtype=torch.bool, device=DEV)
    ok[42:] = False                                            # row 40.. of the last page are NaN, as they lie there
    assert torch.equal(got[ok], want[ok])
    assert bool((got[:2] == 0).all())                          # rows -2 and -1


# ---------------------------------------------------------------- decode

def check_decode(lens, T, H, page, rope, seed, scale=None, std=1.0, grow=None, **kw):
    g = gen(seed)
    cache, table = paged(lens, page, rope, g, std=std)
    if grow is not None:                                       # scores that rise with the position
        grow(cache, table)
    q = randn(g, len(lens) * T, H, 512)
    qr = randn(g, len(lens) * T, H, 64) if rope else None
    scale = (128 + rope) ** -0.5 if scale is None else scale
    out, lse = kda.kda_latent_decode(q, qr, cache, table, i32(lens), scale, lse=True, **kw)
    clean()
    o, s, bo, bs = ref.decode(q, qr, cache, table, i32(lens), scale)
    ref.assert_within(out, o, bo, "out")
    ref.assert_within(lse, s, bs, "lse")
    return out, lse, (q, qr, cache, table, i32(lens), scale)


@pytest.mark.parametrize("rope", [0, 64])
@pytest.mark.parametrize("H,T,page", [(1, 1, 16), (3, 1, 64), (16, 1, 32), (17, 1, 128), (32, 1, 64), (64, 1, 16),
                                      (96, 1, 64), (128, 1, 1024), (8, 2, 64), (5, 7, 16), (16, 4, 32), (32, 16, 64)])
def test_decode_shapes(H, T, page, rope):
    lens = [T, 64, 63 + T, 129, 200, 1000]
    check_decode(lens, T, H, page, rope, seed=H + T)


def test_decode_lengths_of_one_sequence():
    for n in (1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 192, 193, 640, 4097):
        check_decode([n], 1, 32, 16, 64, seed=n)


def test_decode_sequences_that_see_nothing():
    """Empty sequences, sequences shorter than the step, and tokens of a step that see nothing."""
    out, lse, _ = check_decode([0, 5, 2, 0, 1, 300, -7], 4, 8, 16, 64, seed=9)
    assert bool((out[:4] == 0).all()) and bool((lse[:4] == -math.inf).all())
    assert bool((out[8:10] == 0).all()) and bool((lse[8:10] == -math.inf).all()) and bool(lse[10:12].isfinite().all())


def test_decode_lengths_beyond_the_table_are_clamped():
    g = gen(10)
    cache, table = paged([64, 64], 16, 64, g, per=4)
    q, qr = randn(g, 2, 4, 512), randn(g, 2, 4, 64)
    out, lse = kda.kda_latent_decode(q, qr, cache, table, i32([2 ** 31 - 1, 65]), 0.07, lse=True)
    clean()
    o, s, bo, bs = ref.decode(q, qr, cache, table, i32([64, 64]), 0.07)
    ref.assert_within(out, o, bo, "out")
    ref.assert_within(lse, s, bs, "lse")


def test_decode_pages_outside_the_cache_read_as_zero_rows():
    g = gen(11)
    cache, table = paged([300, 70], 16, 64, g, per=19)
    for j, bad in ((0, -1), (5, cache.shape[0]), (6, 2 ** 31 - 1), (18, -2 ** 31)):
        table[0, j] = bad
    table[1, 4] = -9
    q, qr = randn(g, 2, 32, 512), randn(g, 2, 32, 64)
    out, lse = kda.kda_latent_decode(q, qr, cache, table, i32([300, 70]), 0.07, lse=True)
    clean()
    o, s, bo, bs = ref.decode(q, qr, cache, table, i32([300, 70]), 0.07)
    ref.assert_within(out, o, bo, "out")
    ref.assert_within(lse, s, bs, "lse")


@pytest.mark.parametrize("factor", [1.0, 40.0])
def test_decode_rising_and_peaked_scores(factor):
    """Keys that grow with the position make the running maximum rise in every tile; the large factor makes
    one key take all the weight."""
    def grow(cache, table):
        for n in range(2):
            for j in range(13):
                x = cache[table[n, j].long()]
                cache[table[n, j].long()] = x * (0.02 * factor * (j + 1))
    check_decode([13 * 64, 13 * 64 - 5], 2, 16, 64, 64, seed=12, grow=grow)


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
    choices = [0, 1, 63, 64, 65, 128, 300, 384, 385, 1000, 3000][:pick([6, 9, 11])]
    lens = [pick(choices) for _ in range(pick([2, 9, 37, 150, 400]))]
    check_decode(lens, T, H, pick([16, 64, 256]), rope, seed=2000 + seed)


def test_decode_repeats_bit_for_bit_and_shares_pages():
    out, lse, args = check_decode([3000, 129, 64, 3000], 1, 32, 64, 64, seed=17)
    q, qr, cache, table, lens, scale = args
    again, lse2 = kda.kda_latent_decode(*args, lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    table[3] = table[0]                                        # two sequences over one set of pages
    shared, _ = kda.kda_latent_decode(*args)
    o, _, bo, _ = ref.decode(q, qr, cache, table, lens, scale)
    ref.assert_within(shared, o, bo, "shared pages")


def test_decode_cache_beyond_32_bit_offsets():
    """Pages at the end of a cache of more than 2^32 bytes and 2^31 elements."""
    g = gen(18)
    page, rope = 64, 64
    pages = 2 ** 31 // (page * 576) + 100
    cache = torch.empty((pages, page, 576), dtype=BF, device=DEV)
    lens = [300, 150]
    table = torch.tensor([[pages - 1 - j for j in range(5)], [pages - 9 - j for j in range(5)]], dtype=torch.int32, device=DEV)
    for n in range(2):
        for j in range(5):
            cache[table[n, j].long()] = randn(g, page, 576)
    lat, kr = randn(g, 2, 512), randn(g, 2, 64)
    kda.kda_latent_append(lat, kr, cache, table, i32(lens))
    assert torch.equal(ref.rows_of(cache, table, 0, 300)[299], torch.cat([lat[0], kr[0]]).double())
    q, qr = randn(g, 2, 32, 512), randn(g, 2, 32, 64)
    out, lse = kda.kda_latent_decode(q, qr, cache, table, i32(lens), 0.07, lse=True)
    clean()
    o, s, bo, bs = ref.decode(q, qr, cache, table, i32(lens), 0.07)
    ref.assert_within(out, o, bo, "out")
    ref.assert_within(lse, s, bs, "lse")
    got, _ = kda.kda_latent_gather(cache, table, [0, 300, 450], 450)
    assert torch.equal(got[:300].double(), ref.rows_of(cache, table, 0, 300)[:, :512])


def test_decode_a_context_of_a_million_tokens():
    """2^20 tokens over 64 distinct pages, and a short neighbour."""
    g = gen(20)
    cache = randn(g, 64, 1024, 576)
    table = torch.randint(0, 64, (2, 1024), generator=g, device=DEV).to(torch.int32)
    check = (randn(g, 2, 16, 512), randn(g, 2, 16, 64), cache, table, i32([2 ** 20, 77]), 0.07)
    out, lse = kda.kda_latent_decode(*check, lse=True)
    clean()
    o, s, bo, bs = ref.decode(*check)
    ref.assert_within(out, o, bo, "out")
    ref.assert_within(lse, s, bs, "lse")


def test_decode_without_pages():
    """No pages, no table entries: nothing is seen."""
    q, qr = torch.ones(3, 4, 512, dtype=BF, device=DEV), torch.ones(3, 4, 64, dtype=BF, device=DEV)
    empty = torch.empty(0, 64, 576, dtype=BF, device=DEV)
    out, lse = kda.kda_latent_decode(q, qr, empty, torch.empty(3, 0, dtype=torch.int32, device=DEV), i32([5, 0, 9]), 0.07, lse=True)
    clean()
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    out, lse = kda.kda_latent_decode(q, qr, empty, torch.zeros(3, 2, dtype=torch.int32, device=DEV), i32([5, 0, 128]), 0.07, lse=True)
    clean()                                                    # rows of pages that are not there are zeros
    assert bool((out == 0).all())
    torch.testing.assert_close(lse[:, 0].cpu(), torch.tensor([math.log(5), -math.inf, math.log(128)]), rtol=1e-6, atol=0)


def test_decode_writes_no_row_but_its_own():
    g = gen(19)
    cache, table = paged([100, 40, 7], 16, 64, g)
    q, qr = randn(g, 3, 5, 512), randn(g, 3, 5, 64)
    big = torch.full((5, 5, 512), 7.0, dtype=BF, device=DEV)
    lse = torch.full((5, 5), 7.0, device=DEV)
    kda.kda_latent_decode(q, qr, cache, table, i32([100, 40, 7]), 0.07, out=big[1:4], lse=lse[1:4])
    clean()
    for x in (big[0], big[4], lse[0], lse[4]):
        assert bool((x == 7.0).all())


# ---------------------------------------------------------------- prefill

def check_prefill(nq, nk, H, rope, seed, fused=True, tail=0, scale=None, host=False, std=1.0):
    g = gen(seed)
    cu, ck = [0], [0]
    for a, b in zip(nq, nk):
        cu.append(cu[-1] + a)
        ck.append(ck[-1] + b)
    T, S = cu[-1] + tail, ck[-1] + tail
    q = randn(g, T, H, 128 + rope, std=std)
    if fused:
        kv = randn(g, S, H, 256)
        k, v = kv[..., :128], kv[..., 128:]
    else:
        k, v = randn(g, S, H, 128), randn(g, S, H, 128)
    kr = randn(g, S, 64) if rope else None
    if tail:                                                   # rows behind the last sequence
        for x in (q, k, v) + ((kr,) if rope else ()):
            x[-tail:] = NAN
    out = torch.full((T, H, 128), 7.0, dtype=BF, device=DEV)
    lse = torch.full((T, H), 7.0, device=DEV)
    scale = (128 + rope) ** -0.5 if scale is None else scale
    tables = (cu, ck) if host else (i32(cu), i32(ck))
    kda.kda_latent_prefill(q, k, v, kr, scale, *tables, out=out, lse=lse)
    clean()
    o, s, bo, bs = ref.prefill(q[:cu[-1]], k, v, kr, scale, cu, ck)
    ref.assert_within(out[:cu[-1]], o, bo, "out")
    ref.assert_within(lse[:cu[-1]], s, bs, "lse")
    assert bool((out[cu[-1]:] == 7.0).all()) and bool((lse[cu[-1]:] == 7.0).all())
    return out, lse


@pytest.mark.parametrize("rope", [0, 64])
@pytest.mark.parametrize("n", [1, 2, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 385, 640, 1025])
def test_prefill_one_sequence(n, rope):
    check_prefill([n], [n], 2, rope, seed=n, fused=n % 2 == 0)


@pytest.mark.parametrize("rope", [0, 64])
def test_prefill_ragged_batches(rope):
    check_prefill([1, 0, 130, 77, 300, 256], [1, 0, 130, 77, 300, 256], 3, rope, seed=1, tail=5)
    check_prefill([200] * 3, [200] * 3, 4, rope, seed=2, host=True)


@pytest.mark.parametrize("rope", [0, 64])
def test_prefill_over_a_prefix(rope):
    check_prefill([1, 100, 300, 7], [1000, 228, 301, 7], 2, rope, seed=3, tail=9)
    check_prefill([128], [1153], 1, rope, seed=4)
    check_prefill([513], [2049], 2, rope, seed=5)


@pytest.mark.parametrize("rope", [0, 64])
@pytest.mark.parametrize("nq,past,H", [
    ([100], [1948], 32), ([1], [1300], 3), ([128], [2048], 16), ([129], [5000], 4), ([256], [4096], 1), ([700], [8000], 6),
    ([40, 3], [3000, 2500], 9), ([300, 1, 0, 257], [1, 6000, 900, 2222], 4), ([5, 5, 5], [0, 9000, 130], 7)])
def test_prefill_few_queries_over_many_keys(nq, past, H, rope):
    """Queries too few for all SMs, whose keys several blocks share."""
    check_prefill(nq, [a + b for a, b in zip(nq, past)], H, rope, seed=sum(past) + H)


def test_prefill_shared_keys_repeat_bit_for_bit_and_rising_scores():
    g = gen(77)
    q, kv, kr = randn(g, 60, 8, 192), randn(g, 4060, 8, 256), randn(g, 4060, 64)
    kv[..., :128] *= torch.linspace(0.01, 6, 4060, device=DEV)[:, None, None].to(BF)     # the maximum rises with the keys
    call = lambda: kda.kda_latent_prefill(q, kv[..., :128], kv[..., 128:], kr, 0.3, lse=True, num_seqs=1)  # noqa: E731
    out, lse = call()
    again = call()
    clean()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    o, s, bo, bs = ref.prefill(q, kv[..., :128], kv[..., 128:], kr, 0.3, [0, 60], [0, 4060])
    ref.assert_within(out, o, bo, "out")
    ref.assert_within(lse, s, bs, "lse")


def test_prefill_with_fewer_keys_than_queries():
    out, lse = check_prefill([10, 300, 5, 140], [4, 20, 0, 139], 2, 64, seed=6, tail=3)
    assert bool((out[:6] == 0).all()) and bool((lse[:6] == -math.inf).all())


def test_prefill_neighbours_do_not_reach_each_other():
    """NaN in one sequence leaves the sequences beside it finite and right."""
    g = gen(7)
    cu = [0, 100, 170, 400]
    q, kv, kr = randn(g, 400, 2, 192), randn(g, 400, 2, 256), randn(g, 400, 64)
    clean_out, _ = kda.kda_latent_prefill(q, kv[..., :128], kv[..., 128:], kr, 0.07, i32(cu))
    for x in (q, kv, kr):
        x[100:170] = NAN
    out, _ = kda.kda_latent_prefill(q, kv[..., :128], kv[..., 128:], kr, 0.07, i32(cu))
    assert torch.equal(out[:100], clean_out[:100]) and torch.equal(out[170:], clean_out[170:])


def test_prefill_heads_and_scale():
    check_prefill([150, 40], [150, 40], 33, 64, seed=8)
    check_prefill([300], [300], 2, 64, seed=9, scale=1.0, std=3.0)         # peaked, a maximum that moves
    check_prefill([300], [700], 1, 0, seed=10, scale=1e-4)


def test_prefill_repeats_bit_for_bit():
    g = gen(11)
    q, kv, kr = randn(g, 700, 4, 192), randn(g, 700, 4, 256), randn(g, 700, 64)
    args = (q, kv[..., :128], kv[..., 128:], kr, 0.07, i32([0, 300, 700]))
    a, la = kda.kda_latent_prefill(*args, lse=True)
    b, lb = kda.kda_latent_prefill(*args, lse=True)
    assert torch.equal(a, b) and torch.equal(la, lb)


# ---------------------------------------------------------------- what the binding refuses

def test_binding_refusals():
    g = gen(22)
    cache, table = paged([70, 40], 16, 64, g)
    lens = i32([70, 40])
    lat, kr, q, qr = randn(g, 2, 512), randn(g, 2, 64), randn(g, 2, 4, 512), randn(g, 2, 4, 64)
    ok = dict(q_latent=q, q_rope=qr, cache=cache, block_table=table, seq_lens=lens, scale=0.07)
    kda.kda_latent_decode(**ok)
    for bad, error in ((dict(q_latent=q.float()), TypeError), (dict(q_latent=q[0]), ValueError), (dict(q_rope=None), ValueError),
                       (dict(q_rope=qr[:, :3]), ValueError), (dict(cache=cache[0]), ValueError), (dict(cache=cache[..., :500]), ValueError),
                       (dict(cache=cache[:, ::2]), ValueError), (dict(block_table=table.long()), TypeError),
                       (dict(block_table=table[0]), ValueError), (dict(seq_lens=lens[:1]), ValueError), (dict(seq_lens=lens.cpu()), ValueError),
                       (dict(out=q[:1]), ValueError), (dict(lse=torch.empty(2, 4, dtype=BF, device=DEV)), TypeError),
                       (dict(workspace=torch.empty(9, device=DEV)), TypeError), (dict(q_latent=q.transpose(0, 1).contiguous().transpose(0, 1)), ValueError)):
        with pytest.raises(error):
            kda.kda_latent_decode(**{**ok, **bad})
    for bad, status in ((dict(scale=-1.0), 1), (dict(workspace=torch.empty(256, dtype=torch.uint8, device=DEV)), 1),
                        (dict(cache=cache.view(-1, 4, 576)), 2)):
        with pytest.raises(kda.KdaError) as e:
            kda.kda_latent_decode(**{**ok, **bad})
        assert e.value.status == status
    for bad, error in ((dict(latent=lat.float()), TypeError), (dict(k_rope=None), ValueError), (dict(inv_freq=freqs()[:5]), ValueError),
                       (dict(cu_seqlens=i32([0, 1])), ValueError), (dict(cu_seqlens=[0, 2, 1]), kda.KdaError),
                       (dict(q_rope=qr[:, :3]), ValueError), (dict(latent=lat.t().contiguous().t()), ValueError)):
        with pytest.raises(error):
            kda.kda_latent_append(**{**dict(latent=lat, k_rope=kr, cache=cache, block_table=table, seq_lens=lens), **bad})
    p = dict(q=randn(g, 10, 2, 192), k=randn(g, 10, 2, 128), v=randn(g, 10, 2, 128), k_rope=randn(g, 10, 64), scale=0.07)
    kda.kda_latent_prefill(**p)
    for bad, error in ((dict(q=p["q"][..., :100]), ValueError), (dict(k_rope=None), ValueError), (dict(v=randn(g, 10, 2, 256)[..., :128]), ValueError),
                       (dict(k=p["k"][:9]), ValueError), (dict(cu_seqlens=i32([0, 10]), cu_seqlens_k=i32([0, 5, 10])), ValueError),
                       (dict(num_seqs=3), kda.KdaError), (dict(q=p["q"].half()), TypeError), (dict(lse=torch.empty(3, device=DEV)), ValueError)):
        with pytest.raises(error):
            kda.kda_latent_prefill(**{**p, **bad})
    with pytest.raises(ValueError):
        kda.kda_latent_gather(cache, table, i32([0, 1]), 1)
    clean()


# ---------------------------------------------------------------- streams, graphs, the run of them

def test_side_stream_and_captured_graph():
    """The calls on another stream, and captured once and replayed with new lengths and queries."""
    g = gen(12)
    lens = i32([130, 900, 64])
    cache, table = paged([2000, 2000, 2000], 64, 64, g)
    q, qr = randn(g, 3, 32, 512), randn(g, 3, 32, 64)
    lat, kr, qn = randn(g, 3, 512), randn(g, 3, 64), randn(g, 3, 32, 64)
    ws = torch.empty(kda.kda_latent_decode_workspace_size(3, 3, 32), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(3, 32, device=DEV)

    def step():
        kda.kda_latent_append(lat, kr, cache, table, lens, inv_freq=freq, q_rope=qn, q_rope_out=qr)
        kda.kda_latent_decode(q, qr, cache, table, lens, 0.07, out=out, lse=lse, workspace=ws)

    freq = freqs()
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
        o, s, bo, bs = ref.decode(q, qr, cache, table, lens, 0.07)
        ref.assert_within(out, o, bo, "replayed out")
        ref.assert_within(lse, s, bs, "replayed lse")
    clean()


FIRST_CAPTURE = """
import torch, linear_attention_06_gb300 as kda
BF, d = torch.bfloat16, "cuda"
z = lambda *s: torch.randn(*s, device=d).to(BF)
i = lambda x: torch.tensor(x, dtype=torch.int32, device=d)
def call(H, T, rope, nq, nk, n):
    page = 64
    cache, table = z(40 * n, page, 512 + rope), torch.arange(n * 40, dtype=torch.int32, device=d).view(n, 40)
    lens, f = i([min(2500, nk)] * n), torch.rand(32, device=d)
    lat, kr, q = z(n * T, 512), z(n * T, 64) if rope else None, z(n * T, H, 64) if rope else None
    ql, k, v = z(n * T, H, 512), z(nk, H, 128), z(nk, H, 128)
    qq, kr2 = z(nq, H, 128 + rope), z(nk, 64) if rope else None
    cu = torch.arange(n + 1, dtype=torch.int32, device=d) * 100
    def run():
        kda.kda_latent_append(lat, kr, cache, table, lens, inv_freq=f if rope else None, q_rope=q)
        return (kda.kda_latent_gather(cache, table, cu, 100 * n)[0],
                kda.kda_latent_decode(ql, q, cache, table, lens, 0.1)[0],
                kda.kda_latent_prefill(qq, k, v, kr2, 0.1, num_seqs=1)[0])
    return run
call(4, 1, 64, 20, 20, 1)()
call(4, 1, 0, 20, 20, 1)()
torch.cuda.synchronize()
for args in ((4, 1, 64, 100, 4000, 1), (32, 2, 0, 100, 8000, 40), (64, 1, 64, 700, 700, 2), (20, 1, 0, 30, 30, 3)):
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


def test_a_stream_argument_carries_the_whole_call():
    """Outputs, workspaces and table copies of a call with stream= belong to that stream; a raw handle works too."""
    g = gen(21)
    cache, table = paged([700, 65], 64, 64, g)
    q, qr, lens = randn(g, 2, 32, 512), randn(g, 2, 32, 64), i32([700, 65])
    p = (randn(g, 300, 2, 192), randn(g, 300, 2, 128), randn(g, 300, 2, 128), randn(g, 300, 64), 0.07)
    lat, kr, qn = randn(g, 2, 512), randn(g, 2, 64), randn(g, 2, 4, 64)
    want = (kda.kda_latent_decode(q, qr, cache, table, lens, 0.07)[0], kda.kda_latent_prefill(*p, cu_seqlens=[0, 100, 300])[0],
            kda.kda_latent_gather(cache, table, [0, 700, 765], 765)[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = []
        for _ in range(20):                                    # memory is reused from call to call
            got = [kda.kda_latent_decode(q, qr, cache, table, lens, 0.07, stream=stream)[0],
                   kda.kda_latent_prefill(*p, cu_seqlens=[0, 100, 300], stream=stream)[0],
                   kda.kda_latent_gather(cache, table, [0, 700, 765], 765, stream=stream)[0]]
            torch.full((1 << 22,), 7.0, device=DEV)            # on the default stream
        kda.kda_latent_append(lat, kr, cache.clone(), table, lens, q_rope=qn, stream=stream)
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    clean()


def test_two_streams_at_once():
    """Two decodes and two prefills in flight together, each with its own workspace."""
    g = gen(13)
    sets = []
    for k in range(2):
        cache, table = paged([3000, 1700, 64], 64, 64, g)
        sets.append((randn(g, 3, 32, 512), randn(g, 3, 32, 64), cache, table, i32([3000, 1700, 64]), 0.07))
    qs = [(randn(g, 900, 4, 192), randn(g, 900, 4, 128), randn(g, 900, 4, 128), randn(g, 900, 64), 0.07) for _ in range(2)]
    alone = [kda.kda_latent_decode(*x)[0] for x in sets] + [kda.kda_latent_prefill(*x)[0] for x in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    together = []
    for x, y, st in zip(sets, qs, streams):
        with torch.cuda.stream(st):
            for _ in range(3):
                a, b = kda.kda_latent_decode(*x)[0], kda.kda_latent_prefill(*y)[0]
            together.append((a, b))
    torch.cuda.synchronize()
    for k in range(2):
        assert torch.equal(together[k][0], alone[k]) and torch.equal(together[k][1], alone[2 + k])


def test_prompt_then_steps_agree_in_both_forms():
    """A prompt through append, gather, the up-projections and the expanded form; then a step of the absorbed
    form over the same cache, and the expanded form over everything: one model, two forms, one result."""
    g = gen(14)
    H, page, nq = 8, 16, [90, 33]
    w_k = (torch.randn(H, 512, 128, generator=g, device=DEV) / 512 ** 0.5).to(BF)
    w_v = (torch.randn(H, 512, 128, generator=g, device=DEV) / 512 ** 0.5).to(BF)
    step, scale, freq = 3, 192 ** -0.5, freqs()
    top = [n + step for n in nq]
    cache, table = paged(top, page, 64, g)
    cache.fill_(NAN)

    def tokens(counts, lens):
        T = sum(counts)
        cu = i32([0] + torch.tensor(counts).cumsum(0).tolist())
        q = randn(g, T, H, 192)
        kda.kda_latent_append(randn(g, T, 512), randn(g, T, 64), cache, table, i32(lens), inv_freq=freq,
                              q_rope=q[..., 128:], q_rope_out=q[..., 128:], cu_seqlens=cu)
        return q, cu

    def expanded(q, cu, lens):
        ck = i32([0] + torch.tensor(lens).cumsum(0).tolist())
        lat, kr = kda.kda_latent_gather(cache, table, ck, sum(lens))
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
    o_lat, _ = kda.kda_latent_decode(q_lat, q[..., 128:].contiguous(), cache, table, i32(top), scale)
    got = torch.einsum("thc,hcd->thd", o_lat.double(), w_v.double())
    clean()
    # the forms round k, v, q_lat and o_lat at different places, each by at most 2^-8 of its value; of
    # independent roundings over 128 and 512 terms about as much is left in the norm
    assert float((got - want.double()).norm() / want.double().norm()) < 4 * ref.U


def test_no_index_leaves_its_buffer():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "latent_bounds_run.py")], capture_output=True,
                         text=True, timeout=1200, cwd=ROOT)
    assert out.returncode == 0, out.stdout[-3000:] + out.stderr[-3000:]
    assert "bounds ok" in out.stdout
