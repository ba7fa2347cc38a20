"""The 8-bit latent decode's softmax weights on the GPU: faint ones beside bright ones, against 64 bits.

The weights of a row are multiplied as 8-bit numbers.  Together they are off by at most 2^-7 of their sum, each counted
times its cached row's 2^e (include/kda.h); an output is off by that times the largest of the rows' numbers in its channel,
beside its own rounding and what the scores' arithmetic leaves (tests/latent_q8_reference.py)."""
import math

import pytest
import torch

import linear_attention_06_gb300 as kda
from tests import latent_q8_reference as q8
from tests import latent_reference as ref

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def clean():
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0


def paged(y, e, page):
    """Numbers and powers of one sequence's rows on consecutive pages, NaN bytes behind its end."""
    pages = -(-y.shape[0] // page)
    cache = torch.full((pages * page, 512), 0x7F, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(pages * page, dtype=torch.uint8, device=DEV)
    cache[:y.shape[0]] = q8.bytes_of(y).view(torch.uint8)
    scales[:y.shape[0]] = (e + 127).to(torch.uint8)
    return cache.view(q8.E4M3).view(pages, page, 512), scales.view(q8.E8M0).view(pages, page)


def exact(q, y, e, scale):
    """Outputs, lse and bounds of rows q [R, 512] over cached rows (numbers y, powers e), all in 64 bits."""
    c = y * q8.two(e)[:, None]
    s = (q @ c.T) * scale
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    out = p @ c
    held = (p * q8.two(e)).sum(-1, keepdim=True)               # the weights' sum, each times its row's 2^e
    size = ((q.abs() @ c.abs().T) * scale).amax(-1)
    delta = 512 * 2.0 ** -24 * size + 2.0 ** -20 * (1 + size) + 2.0 ** -10 * (q.abs().amax(-1) / 224) * scale * c.abs().sum(-1).amax()
    bound = q8.U * out.abs() + 2.0 ** -7 * held * y.abs().amax(0) + 2 * delta[:, None] * (p @ c.abs())
    return out, lse, bound, delta + 2.0 ** -20 * (1 + lse.abs())


def tail(length, period, sink, H, spread, seed):
    """Rows with one direction in common, and queries that weigh them so: 2^sink the first, 2^-4 one token of every
    `period` tiles of 128, the others 2^-8 (the first head) to 2^-20 (the last) of the first's usual weight, spread by
    `spread` bits."""
    g = gen(seed)
    x = torch.zeros(length, 512, dtype=torch.float64, device=DEV)
    x[:, 100:] = 1 + 0.1 * torch.randn(length, 412, generator=g, device=DEV)
    x[:, 0] = -8 * math.log(2)
    x[:, 2] = torch.randn(length, generator=g, device=DEV)
    x[0, 0], x[0, 2] = 0, sink * math.log(2)
    bright = torch.arange(128 * (period // 2) + 5, length, 128 * period, device=DEV)
    x[bright, 0], x[bright, 1], x[bright, 2] = 0, -4 * math.log(2), 0
    q = torch.zeros(H, 512, device=DEV)
    q[:, 0] = torch.linspace(1, 2.5, H, device=DEV)
    q[:, 1] = 1
    q[:, 2] = spread * math.log(2)
    if sink:
        q[:, 3] = 1
        x[0, 2], x[0, 3] = 0, sink * math.log(2)
    elif not spread:
        x[:, 2] = 0
    y, e = q8.quantise(x)
    return q.to(BF), y, e


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("sequences", [152, 3])                # whole sequences in a block each, and cut ones
@pytest.mark.parametrize("period", [1, 2, 3, 5])
@pytest.mark.parametrize("sink,spread", [(0, 0.0), (0, 0.7), (8, 0.0), (20, 1.0)])
def test_faint_weights_beside_bright_ones(H, sequences, period, sink, spread):
    length, page = 8192, 64
    q, y, e = tail(length, period, sink, H, spread, seed=period)
    cache = q8.bytes_of(y).view(-1, page, 512)
    scales = q8.powers_of(e).view(-1, page)
    table = torch.arange(length // page, dtype=torch.int32, device=DEV).expand(sequences, -1).contiguous()
    out, lse = kda.kda_latent_decode_q8(q.expand(sequences, -1, -1).contiguous(), None, cache, scales, table,
                                        torch.full((sequences,), length, dtype=torch.int32, device=DEV), 1.0, lse=True)
    clean()
    o, s, bo, bs = exact(q.double(), y, e, 1.0)
    for n in (0, sequences - 1):
        ref.assert_within(lse[n], s, bs, "lse")
        ref.assert_within(out[n], o, bo, "out")
        # What is lost has one sign in the common direction.  The kernel's conversions and its rule, taken step by step on
        # the host, leave at most 3.6e-3 of such rows; 412 outputs' roundings of 2^-8 at most have a mean within 2^-11.
        off = (out[n, :, 100:].double() - o[:, 100:]).mean(-1) / o[:, 100:].mean(-1)
        assert float(off.abs().max()) <= 2.0 ** -8 + 2.0 ** -11, off


@pytest.mark.parametrize("H,T", [(8, 1), (16, 2), (16, 4), (32, 3)])
@pytest.mark.parametrize("rate", [0.25, 1.0, 4.0])
@pytest.mark.parametrize("rising", [False, True])
def test_weights_that_fall_and_rise(H, T, rate, rising):
    """Weights that fall, or rise, by so many bits a tile, with a few bright tokens on the way."""
    length, page, n = 5000, 16, 2
    g = gen(int(16 * rate) + H)
    x = torch.zeros(length, 512, dtype=torch.float64, device=DEV)
    x[:, 100:] = 1 + 0.2 * torch.randn(length, 412, generator=g, device=DEV)
    at = torch.arange(length, device=DEV)
    x[:, 0] = -rate * math.log(2) * ((length - 1 - at if rising else at) // 128)
    x[::700, 0] += 6 * math.log(2)
    y, e = q8.quantise(x)
    cache, scales = paged(y, e, page)
    table = torch.arange(cache.shape[0], dtype=torch.int32, device=DEV).expand(n, -1).contiguous()
    q = torch.zeros(n * T, H, 512, device=DEV)
    q[..., 0] = torch.linspace(0.5, 1.0, H, device=DEV)
    q = q.to(BF)
    lens = [length, length - 130]
    out, lse = kda.kda_latent_decode_q8(q, None, cache, scales, table, torch.tensor(lens, dtype=torch.int32, device=DEV), 1.0, lse=True)
    clean()
    for i, m in enumerate(lens):
        for t in range(T):
            seen = m - T + 1 + t
            o, s, bo, bs = exact(q[i * T + t].double(), y[:seen], e[:seen], 1.0)
            ref.assert_within(lse[i * T + t], s, bs, "lse")
            ref.assert_within(out[i * T + t], o, bo, "out")


# ---------------------------------------------------------------- rows of very different powers

def numbers(g, count):
    """e4m3 numbers of 64 .. 200, no channel that a query sees."""
    y = q8.to_e4m3((64 + 136 * torch.rand(count, 512, generator=g, device=DEV, dtype=torch.float64)))
    y[:, :2] = 0
    return y


def check_powers(y, e, score, H, sequences, page=64, T=1):
    """Decodes rows of numbers y and powers e under scores `score` (natural logarithms; only rows of e <= 0 may have one),
    seen by queries that weigh them by 1/2 to 1.  Zero channels of a query and of a row multiply to exact zeros, so the
    scores are good to a few 2^-24 of themselves whatever the other channels are."""
    y = y.clone()
    y[:, 0] = q8.to_e4m3(score * q8.two(-e))
    score = y[:, 0] * q8.two(e)
    n = y.shape[0]
    cache, scales = paged(y, e, page)
    table = torch.arange(cache.shape[0], dtype=torch.int32, device=DEV).expand(sequences, -1).contiguous()
    q = torch.zeros(sequences * T, H, 512, device=DEV)
    q[..., 0] = torch.linspace(0.5, 1.0, H, device=DEV)
    q[:, -1] = 0                                               # and one that weighs all alike
    q = q.to(BF)
    out, lse = kda.kda_latent_decode_q8(q, None, cache, scales, table,
                                        torch.full((sequences,), n, dtype=torch.int32, device=DEV), 1.0, lse=True)
    clean()
    for i in (0, sequences - 1):
        for t in range(T):
            seen = n - T + 1 + t
            row = i * T + t
            c = y[:seen] * q8.two(e[:seen])[:, None]
            s = q[row, :, 0].double()[:, None] * score[None, :seen]
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[:, None])
            size = s.abs().amax(-1)
            # the sum: 2^-20 holds its 2^4 roundings a thread, the exponential's and the logarithms'
            delta = 2.0 ** -22 * size + 2.0 ** -20 * (1 + size + z.abs())
            ref.assert_within(lse[row], z, delta, "lse")
            o = p @ c
            held = (p * q8.two(e[:seen])).sum(-1, keepdim=True)
            bound = q8.U * o.abs() + 2.0 ** -7 * held * y[:seen].abs().amax(0) + 4 * delta[:, None] * (p @ c.abs())
            ref.assert_within(out[row], o, bound, "out")


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("top", [6, 16, 60, 70, 100, 120])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed", "late"])
def test_rows_of_powers_far_apart(H, top, order):
    """Rows of zeros and rows of the largest powers beside each other, in one tile and tiles apart."""
    g = gen(top + H)
    count = 700
    y = numbers(g, count)
    if order == "mixed":
        e = torch.randint(-64, top + 1, (count,), generator=g, device=DEV).double()
    else:
        e = torch.full((count,), float(top), dtype=torch.float64, device=DEV)
        zeros = {"rising": slice(0, 256), "falling": slice(444, count), "late": slice(0, 650)}[order]
        e[zeros] = -64
        y[zeros] = 0
    score = torch.zeros(count, dtype=torch.float64, device=DEV)
    for sequences in (1, 152):
        check_powers(y, e, score, H, sequences)


@pytest.mark.parametrize("H,T", [(16, 1), (8, 4), (32, 2), (64, 1)])
@pytest.mark.parametrize("seed", range(6))
def test_rows_of_any_power_under_scores(H, T, seed):
    """Powers of the whole format in random order, the small rows under scores that move the sums' reference."""
    g = gen(100 + seed)
    count = [300, 1000, 2500][seed % 3]
    y = numbers(g, count)
    e = torch.randint(-64, 121, (count,), generator=g, device=DEV).double()
    steady = torch.arange(count, device=DEV) % 400 < [150, 390, 250][seed // 2]        # stretches of ordinary rows
    e = torch.where(steady, torch.randint(-9, -4, (count,), generator=g, device=DEV).double(), e)
    score = torch.where(steady, 3 * torch.randn(count, generator=g, device=DEV, dtype=torch.float64), 0.0)
    score = score + torch.where(steady, 2.0 * (torch.arange(count, device=DEV) // 400), 0.0)
    score = score.clamp(-448 * 2.0 ** -9, 448 * 2.0 ** -9) * (8 if seed % 2 else 1)
    e = torch.where(steady & (score.abs() > 0), torch.maximum(e, torch.full_like(e, -6 if seed % 2 else -9)), e)
    check_powers(y, e, score, H, 2, T=T)


def test_missing_pages_before_large_rows():
    """Pages outside the cache count as rows of zeros: 2 x 128 of them, then rows of the largest power."""
    for top, H, N in ((70, 4, 152), (119, 32, 1), (119, 32, 152), (119, 64, 152)):
        g = gen(top)
        y, e = numbers(g, 256), torch.full((256,), float(top), dtype=torch.float64, device=DEV)
        cache, scales = paged(y, e, 64)
        table = torch.tensor([[-1, -1, 9, 9, 0, 1, 2, 3]] * N, dtype=torch.int32, device=DEV)
        q = torch.zeros(N, H, 512, dtype=BF, device=DEV)
        out, lse = kda.kda_latent_decode_q8(q, None, cache, scales, table, torch.tensor([512] * N, dtype=torch.int32, device=DEV),
                                            1.0, lse=True)
        clean()
        o = (y * q8.two(e)[:, None]).sum(0) / 512
        assert float((lse.double() - math.log(512)).abs().max()) <= 2.0 ** -20 * 8
        for n in (0, N - 1):
            ref.assert_within(out[n], o.expand(H, -1), (2 * q8.U + 2.0 ** -7) * o.abs().expand(H, -1), "out")
