"""Latent attention on the GPU: calls that the documentation allows, in orders and with values of their own."""
import pytest
import torch

import linear_attention_06_gb300 as kda

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
