"""The 8-bit latent cache on the GPU: promises about order, memory and neighbours."""
import pytest
import torch

import linear_attention_06_gb300 as kda
from tests import latent_q8_reference as q8
from tests import latent_reference as ref

pytestmark = pytest.mark.gpu
DEV, BF, U8 = "cuda", torch.bfloat16, torch.uint8


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(BF)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def clean():
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0


def full_cache(g, pages, page, rope):
    y, e = q8.quantise(randn(g, pages, page, 512 + rope).double())
    return q8.bytes_of(y), q8.powers_of(e)


def stored(latent, k_rope):
    """What rows without rotation are held as (bf16, exact)."""
    y, e = q8.quantise((latent if k_rope is None else torch.cat([latent, k_rope], 1)).double())
    x = (y * q8.two(e)[:, None]).to(BF)
    return x[:, :512], x[:, 512:]


@pytest.mark.parametrize("rope", [0, 64])
def test_rows_gathered_before_and_after_they_are_replaced(rope):
    """Gathers and appends of the same rows in turn on one stream, each long enough to start while the one before it
    ends: every gather reads what the append before it wrote."""
    g = gen(rope)
    n, each, page, rounds = 3, 4000, 64, 12
    per = -(-each // page)
    cache, scales = full_cache(g, n * per, page, rope)
    table = torch.randperm(n * per, generator=g, device=DEV).to(torch.int32).view(n, per)
    lens, cu = i32([each] * n), i32([each * k for k in range(n + 1)])
    T = n * each
    new = [(randn(g, T, 512) * 2.0 ** k, randn(g, T, 64) if rope else None) for k in range(rounds)]
    empty = lambda: (torch.empty(T, 512, dtype=BF, device=DEV), torch.empty(T, 64, dtype=BF, device=DEV) if rope else None)  # noqa: E731
    got = [empty() for _ in range(rounds)]
    torch.cuda.synchronize()
    kda.kda_latent_gather_q8(cache, scales, table, cu, T, out=empty())
    for x, y in zip(new, got):
        kda.kda_latent_append_q8(x[0], x[1], cache, scales, table, lens, cu_seqlens=cu)
        kda.kda_latent_gather_q8(cache, scales, table, cu, T, out=y)
    clean()
    for x, y in zip(new, got):
        want = stored(*x)
        assert torch.equal(want[0], y[0])
        assert not rope or torch.equal(want[1], y[1])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (37, 300), (2500, 40)])
def test_queries_without_rotation_are_copied_bit_for_bit(T, H, interleaved):
    g = gen(T + H)
    page = 16
    per = -(-T // page)
    cache, scales = full_cache(g, per, page, 64)
    table = torch.randperm(per, generator=g, device=DEV).to(torch.int32).view(1, per)
    q = torch.randint(-2 ** 15, 2 ** 15, (T, H, 192), generator=g, device=DEV).to(torch.int16).view(BF)
    got = kda.kda_latent_append_q8(randn(g, T, 512), randn(g, T, 64), cache, scales, table, i32([T]), interleaved=interleaved,
                                   q_rope=q[..., 128:])
    clean()
    assert torch.equal(got.view(torch.int16), q[..., 128:].contiguous().view(torch.int16))


@pytest.mark.parametrize("T,H,rope", [(7, 640, 64), (5, 1024, 0), (16, 1024, 64)])
def test_decode_of_so_many_rows_that_few_runs_are_left(T, H, rope):
    """Two runs and one run over the sequences, with a workspace of exactly the size asked for: bytes behind it stay."""
    g = gen(T)
    page, lens = 16, [T, 200, 0, 700, 65, T - 1]
    per = -(-max(lens) // page)
    cache, scales = full_cache(g, len(lens) * per, page, rope)
    table = torch.randperm(len(lens) * per, generator=g, device=DEV).to(torch.int32).view(len(lens), per)
    rows = len(lens) * T
    q, qr = randn(g, rows, H, 512), randn(g, rows, H, 64) if rope else None
    size = kda.kda_latent_decode_q8_workspace_size(len(lens), rows, H, rope)
    ws = torch.full((size + 4096,), 7, dtype=U8, device=DEV)
    args = (q, qr, cache, scales, table, i32(lens), 0.07)
    out, lse = kda.kda_latent_decode_q8(*args, lse=True, workspace=ws[:size])
    clean()
    assert bool((ws[size:] == 7).all())
    o, s, bo, bs = q8.decode(*args)
    ref.assert_within(out, o, bo, "out")
    ref.assert_within(lse, s, bs, "lse")


def test_nan_reaches_no_neighbour():
    """A NaN query channel reaches its own row of the output, a NaN in a cached row its own sequence."""
    g = gen(51)
    cache, scales = full_cache(g, 60, 64, 64)
    table = torch.arange(60, dtype=torch.int32, device=DEV).view(3, 20)
    q, qr = randn(g, 3, 32, 512), randn(g, 3, 32, 64)
    args = (q, qr, cache, scales, table, i32([1200, 700, 130]), 0.07)
    want, wl = kda.kda_latent_decode_q8(*args, lse=True)
    q[1, 5, 300] = float("nan")
    out, lse = kda.kda_latent_decode_q8(*args, lse=True)
    clean()
    keep = torch.ones(3, 32, dtype=torch.bool, device=DEV)
    keep[1, 5] = False
    assert bool(out[1, 5].isnan().all()) and torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], wl[keep])
    q[1, 5, 300] = 0
    want, _ = kda.kda_latent_decode_q8(*args)
    cache.view(U8)[25, 10, 77] = 0x7F                          # a row of sequence 1
    out, _ = kda.kda_latent_decode_q8(*args)
    clean()
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2]) and bool(out[1].isnan().any())


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("H", [16, 32, 64])
def test_an_infinite_query_is_not_answered(H, value):
    """An infinite channel has no 8-bit number: its row of the results is NaN, as a NaN channel's is, the others as before; a
    row that sees nothing stays empty."""
    g = gen(52)
    cache, scales = full_cache(g, 60, 64, 64)
    table = torch.arange(60, dtype=torch.int32, device=DEV).view(3, 20)
    q, qr = randn(g, 3, H, 512), randn(g, 3, H, 64)
    args = (q, qr, cache, scales, table, i32([1200, 100, 0]), 0.07)
    want, wl = kda.kda_latent_decode_q8(*args, lse=True)
    keep = torch.ones(3, H, dtype=torch.bool, device=DEV)
    for x, n, h, i in ((q, 0, 5, 300), (qr, 0, H - 1, 63), (q, 1, 0, 0), (q, 2, 3, 9)):
        x[n, h, i] = value
        keep[n, h] = n == 2
    out, lse = kda.kda_latent_decode_q8(*args, lse=True)
    clean()
    assert bool(out[~keep].isnan().all()) and bool(lse[~keep].isnan().all())
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], wl[keep])
    assert bool((out[2] == 0).all()) and bool((lse[2] == -float("inf")).all())


def test_captured_calls_behind_two_branches():
    """A capture that forks and joins: calls that may start early behind work of two streams, replayed with new rows."""
    g = gen(41)
    n, each, page = 3, 4000, 64
    per = -(-each // page)
    held = [full_cache(g, n * per, page, 64) for _ in range(2)]
    table = torch.arange(n * per, dtype=torch.int32, device=DEV).view(n, per)
    lens, cu = i32([each] * n), i32([each * k for k in range(n + 1)])
    T = n * each
    new = [(randn(g, T, 512), randn(g, T, 64)) for _ in range(2)]
    q, qr = randn(g, n, 32, 512), randn(g, n, 32, 64)
    rows = [(torch.empty(T, 512, dtype=BF, device=DEV), torch.empty(T, 64, dtype=BF, device=DEV)) for _ in range(3)]
    ws = [torch.empty(kda.kda_latent_decode_q8_workspace_size(n, n, 32), dtype=U8, device=DEV) for _ in range(2)]
    out = [torch.empty_like(q) for _ in range(2)]
    lse = [torch.empty(n, 32, device=DEV) for _ in range(2)]
    side = torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        for k, stream in enumerate((main, side)):
            with torch.cuda.stream(stream):
                kda.kda_latent_append_q8(*new[k], *held[k], table, lens, cu_seqlens=cu)
                kda.kda_latent_decode_q8(q, qr, *held[k], table, lens, 0.07, out=out[k], lse=lse[k], workspace=ws[k])
                kda.kda_latent_gather_q8(*held[k], table, cu, T, out=rows[k])
        main.wait_stream(side)
        kda.kda_latent_append_q8(*new[0], *held[1], table, lens, cu_seqlens=cu)   # behind both branches
        kda.kda_latent_gather_q8(*held[1], table, cu, T, out=rows[2])

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in range(3):
        h = gen(100 + seed)
        for x in new:
            for y in x:
                y.copy_(randn(h, *y.shape))
        graph.replay()
        clean()
        for got, want in zip(rows, (new[0], new[1], new[0])):
            for a, b in zip(got, stored(*want)):
                assert torch.equal(a, b)
        o, s, bo, bs = q8.decode(q, qr, *held[0], table, lens, 0.07)               # held[0] keeps new[0]
        ref.assert_within(out[0], o, bo, "out")
        ref.assert_within(lse[0], s, bs, "lse")
        y, e = q8.quantise(torch.cat(new[1], 1).double())
        o, s, bo, bs = q8.decode(q, qr, q8.bytes_of(y).view(-1, 4000, 576)[:, :], q8.powers_of(e).view(-1, 4000),
                                 torch.arange(n, dtype=torch.int32, device=DEV)[:, None], lens, 0.07)
        ref.assert_within(out[1], o, bo, "out")
        ref.assert_within(lse[1], s, bs, "lse")


def test_the_longest_context():
    """A table row of nearly 2^31 rows, whose last tile ends at 2^31 - 16: what lies behind the end is not seen."""
    page, per = 16, 2 ** 27 - 1
    table = torch.zeros((1, per), dtype=torch.int32, device=DEV)
    table[0, -1] = 1
    length = per * page - 5
    cache = torch.zeros(2, page, 512, dtype=U8, device=DEV)
    scales = torch.full((2, page), 127, dtype=U8, device=DEV)
    cache[1, page - 5:] = 0x78                                 # 256 in every channel, behind the end
    out, lse = kda.kda_latent_decode_q8(torch.ones(1, 1, 512, dtype=BF, device=DEV), None, cache.view(q8.E4M3), scales.view(q8.E8M0),
                                        table, i32([length]), 0.01, lse=True)
    clean()
    # every thread adds 2^31 / 128 / 152 equal terms in fp32, each sum off by at most 2^-24 of itself
    steps = 2 ** 31 / 128 / 152
    assert bool((out == 0).all()) and abs(float(lse) - torch.tensor(float(length), dtype=torch.float64).log()) < 1.1 * steps * 2.0 ** -24
