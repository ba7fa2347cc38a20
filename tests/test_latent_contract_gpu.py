"""Latent attention on the GPU: calls that the documentation allows, in orders and with values of their own."""
import pytest
import torch

import linear_attention_06_gb300 as kda
from tests import latent_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


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


@pytest.mark.parametrize("rope", [0, 64])
def test_rows_gathered_before_and_after_they_are_replaced(rope):
    """Gathers and appends of the same rows in turn on one stream, each long enough to start while the one before it
    ends: every gather reads what the append before it wrote."""
    g = gen(rope)
    n, each, page, rounds = 3, 4000, 64, 24
    per = -(-each // page)
    cache = randn(g, n * per, page, 512 + rope)
    table = torch.randperm(n * per, generator=g, device=DEV).to(torch.int32).view(n, per)
    lens, cu = i32([each] * n), i32([each * k for k in range(n + 1)])
    T = n * each
    new = [(randn(g, T, 512), randn(g, T, 64) if rope else None) for _ in range(rounds)]
    empty = lambda: (torch.empty(T, 512, dtype=BF, device=DEV), torch.empty(T, 64, dtype=BF, device=DEV) if rope else None)  # noqa: E731
    got = [empty() for _ in range(rounds)]
    torch.cuda.synchronize()
    kda.kda_latent_gather(cache, table, cu, T, out=empty())
    for x, y in zip(new, got):
        kda.kda_latent_append(x[0], x[1], cache, table, lens, cu_seqlens=cu)
        kda.kda_latent_gather(cache, table, cu, T, out=y)
    clean()
    for x, y in zip(new, got):
        assert torch.equal(x[0], y[0])
        assert not rope or torch.equal(x[1], y[1])


def bits(g, *shape):
    """Every bit pattern alike: infinities, NaN, negative zeros and subnormals among them."""
    return torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, device=DEV).to(torch.int16).view(BF)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,rope", [(1, 1, 64), (37, 300, 64), (37, 4, 0), (2500, 40, 64), (2500, 3, 0)])
def test_rows_without_rotation_are_copied_bit_for_bit(T, H, rope, interleaved):
    """Without inv_freq: a few tokens a block and many, queries within a thread's first loads and behind them."""
    g = gen(T + H)
    page = 16
    per = -(-T // page)
    table = torch.randperm(per, generator=g, device=DEV).to(torch.int32).view(1, per)
    cache = bits(g, per, page, 512 + rope)
    both, q = bits(g, T, 576), bits(g, T, H, 192)
    pos = torch.arange(T, device=DEV)
    slot = table.long()[0, pos // page] * page + pos % page
    want = cache.clone().view(torch.int16)
    want.view(-1, 512 + rope)[slot] = both[:, :512 + rope].view(torch.int16)
    before = q.clone()
    args = (both[:, :512], both[:, 512:] if rope else None, cache, table, i32([T]))
    got = kda.kda_latent_append(*args, interleaved=interleaved, q_rope=q[..., 128:] if rope else None)
    clean()
    assert torch.equal(cache.view(torch.int16), want)
    if rope:
        assert torch.equal(got.view(torch.int16), q[..., 128:].contiguous().view(torch.int16))
        kda.kda_latent_append(*args, interleaved=interleaved, q_rope=q[..., 128:], q_rope_out=q[..., 128:])
        clean()
        assert torch.equal(q.view(torch.int16), before.view(torch.int16))
        assert torch.equal(cache.view(torch.int16), want)
    else:
        assert got is None


@pytest.mark.parametrize("T,H,rope", [(7, 640, 64), (5, 1024, 0), (16, 1024, 64)])
def test_decode_of_so_many_rows_that_few_runs_are_left(T, H, rope):
    """Two runs and one run over the sequences, with a workspace of exactly the size asked for: bytes behind it stay."""
    g = gen(T)
    page, lens = 16, [T, 200, 0, 700, 65, T - 1]
    per = -(-max(lens) // page)
    cache = randn(g, len(lens) * per, page, 512 + rope)
    table = torch.randperm(len(lens) * per, generator=g, device=DEV).to(torch.int32).view(len(lens), per)
    rows = len(lens) * T
    q, qr = randn(g, rows, H, 512), randn(g, rows, H, 64) if rope else None
    size = kda.kda_latent_decode_workspace_size(len(lens), rows, H, rope)
    ws = torch.full((size + 4096,), 7, dtype=torch.uint8, device=DEV)
    out, lse = kda.kda_latent_decode(q, qr, cache, table, i32(lens), 0.07, lse=True, workspace=ws[:size])
    clean()
    assert bool((ws[size:] == 7).all())
    o, s, bo, bs = ref.decode(q, qr, cache, table, i32(lens), 0.07)
    ref.assert_within(out, o, bo, "out")
    ref.assert_within(lse, s, bs, "lse")


def test_the_binding_drops_no_argument():
    """A rotated part for rows that have none, an output without its input, a number of sequences that the offsets
    contradict: refused with the argument's name, and nothing is written."""
    g = gen(31)
    cache, table, lens = randn(g, 4, 16, 512), i32([[0, 1], [2, 3]]), i32([20, 32])
    full = randn(g, 4, 16, 576)
    before = cache.clone(), full.clone()
    lat, kr, q, qr = randn(g, 2, 512), randn(g, 2, 64), randn(g, 2, 4, 512), randn(g, 2, 4, 64)
    p = (randn(g, 10, 2, 128), randn(g, 10, 2, 128), randn(g, 10, 2, 128))
    wide, cu = randn(g, 10, 2, 192), i32([0, 4, 10])
    new = lambda: torch.empty(2, 512, dtype=BF, device=DEV)    # noqa: E731
    freq = torch.ones(32, device=DEV)
    for name, call in (
            ("k_rope", lambda: kda.kda_latent_append(lat, kr, cache, table, lens)),
            ("q_rope", lambda: kda.kda_latent_append(lat, None, cache, table, lens, inv_freq=freq, q_rope=qr)),
            ("q_rope_out", lambda: kda.kda_latent_append(lat, kr, full, table, lens, q_rope_out=qr)),
            ("k_rope", lambda: kda.kda_latent_gather(cache, table, [0, 1, 2], 2, out=(new(), kr))),
            ("k_rope", lambda: kda.kda_latent_gather(cache, table, [0, 1, 2], 2, out=(None, kr))),
            ("k_rope", lambda: kda.kda_latent_gather(full, table, [0, 1, 2], 2, out=(None, kr))),
            ("q_rope", lambda: kda.kda_latent_decode(q, qr, cache, table, lens, 0.07)),
            ("k_rope", lambda: kda.kda_latent_prefill(*p, randn(g, 10, 64), 0.07)),
            ("num_seqs", lambda: kda.kda_latent_prefill(*p, None, 0.07, cu_seqlens=cu, num_seqs=5)),
            ("num_seqs", lambda: kda.kda_latent_prefill(wide, *p[1:], randn(g, 10, 64), 0.07, cu_seqlens_k=cu, num_seqs=1))):
        with pytest.raises((ValueError, kda.KdaError), match=name if name != "q_rope" else "q_rope|INVALID_ARG"):
            call()
    clean()
    assert torch.equal(cache, before[0]) and torch.equal(full, before[1])
    # the same calls as they belong
    kda.kda_latent_append(lat, None, cache, table, lens, inv_freq=freq)
    kda.kda_latent_append(lat, kr, full, table, lens, q_rope=qr, q_rope_out=qr)
    kda.kda_latent_gather(cache, table, [0, 1, 2], 2, out=(new(), None))
    kda.kda_latent_decode(q, None, cache, table, lens, 0.07)
    kda.kda_latent_prefill(*p, None, 0.07, cu_seqlens=cu, num_seqs=2)
    clean()


def test_captured_calls_behind_two_branches():
    """A capture that forks and joins: calls that may start early behind work of two streams, replayed with new rows."""
    g = gen(41)
    n, each, page = 3, 4000, 64
    per = -(-each // page)
    cache = [randn(g, n * per, page, 576) for _ in range(2)]
    table = torch.arange(n * per, dtype=torch.int32, device=DEV).view(n, per)
    lens, cu = i32([each] * n), i32([each * k for k in range(n + 1)])
    T = n * each
    new = [(randn(g, T, 512), randn(g, T, 64)) for _ in range(2)]
    q, qr = randn(g, n, 32, 512), randn(g, n, 32, 64)
    rows = [(torch.empty(T, 512, dtype=BF, device=DEV), torch.empty(T, 64, dtype=BF, device=DEV)) for _ in range(3)]
    ws = [torch.empty(kda.kda_latent_decode_workspace_size(n, n, 32), dtype=torch.uint8, device=DEV) for _ in range(2)]
    out = [torch.empty_like(q) for _ in range(2)]
    side = torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        for k, stream in enumerate((main, side)):
            with torch.cuda.stream(stream):
                kda.kda_latent_append(*new[k], cache[k], table, lens, cu_seqlens=cu)
                kda.kda_latent_decode(q, qr, cache[k], table, lens, 0.07, out=out[k], workspace=ws[k])
                kda.kda_latent_gather(cache[k], table, cu, T, out=rows[k])
        main.wait_stream(side)
        kda.kda_latent_append(*new[0], cache[1], table, lens, cu_seqlens=cu)      # behind both branches
        kda.kda_latent_gather(cache[1], table, cu, T, out=rows[2])

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in range(4):
        h = gen(100 + seed)
        for x in new:
            for y in x:
                y.copy_(randn(h, *y.shape))
        graph.replay()
        clean()
        for got, want in zip(rows, (new[0], new[1], new[0])):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for k in range(2):
            c = torch.cat(new[k], 1).view(n, each, 576)
            for i in range(n):
                o, _, bo, _ = ref.attend(torch.cat([q[i], qr[i]], -1).double(), c[i].double(), c[i, :, :512].double(), 0.07,
                                         torch.full((32,), each, device=DEV))
                ref.assert_within(out[k][i], o, bo, "out")
