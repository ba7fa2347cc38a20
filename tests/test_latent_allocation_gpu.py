"""Memory that the latent calls allocate is seen by torch's dispatch modes and profilers."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import linear_attention_06_gb300 as kda

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.shapes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func.overloadpacket is torch.ops.aten.empty:
            self.shapes.append(tuple(out.shape))
        return out


def test_allocations_go_through_the_dispatcher():
    n, H, page = 2, 4, 16
    z = lambda *s: torch.zeros(*s, dtype=BF, device=DEV)  # noqa: E731
    cache, table = z(4, page, 576), torch.arange(4, dtype=torch.int32, device=DEV).view(n, 2)
    c8, s8 = cache.to(torch.float8_e4m3fn), torch.full((4, page), 127, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)
    lens, cu = torch.tensor([20, 3], dtype=torch.int32, device=DEV), torch.tensor([0, 5, 8], dtype=torch.int32, device=DEV)
    q, qr = z(n, H, 512), z(n, H, 64)
    size, size8 = kda.kda_latent_decode_workspace_size(n, n, H), kda.kda_latent_decode_q8_workspace_size(n, n, H)
    calls = [
        (lambda: kda.kda_latent_append(z8, k8, cache, table, lens, q_rope=qr), [(n, H, 64)]),
        (lambda: kda.kda_latent_append_q8(z8, k8, c8, s8, table, lens, q_rope=qr), [(n, H, 64)]),
        (lambda: kda.kda_latent_gather(cache, table, cu, 8), [(8, 512), (8, 64)]),
        (lambda: kda.kda_latent_gather_q8(c8, s8, table, cu, 8), [(8, 512), (8, 64)]),
        (lambda: kda.kda_latent_decode(q, qr, cache, table, lens, 0.1, lse=True), [(n, H, 512), (n, H), (size,)]),
        (lambda: kda.kda_latent_decode_q8(q, qr, c8, s8, table, lens, 0.1, lse=True), [(n, H, 512), (n, H), (size8,)]),
        (lambda: kda.kda_latent_prefill(z(8, H, 192), z(8, H, 128), z(8, H, 128), z(8, 64), 0.1, cu_seqlens=cu, lse=True),
         [(8, H, 128), (8, H)]),
    ]
    z8, k8 = z(n, 512), z(n, 64)
    for call, shapes in calls:
        with Seen() as seen:
            call()
        for shape in shapes:
            assert shape in seen.shapes, (shape, seen.shapes)
        with torch.autograd.profiler.profile() as events:
            call()
        assert sum(e.name == "aten::empty" for e in events.function_events) >= len(shapes)
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0


def test_rows_of_no_sequence_are_filled_in_deterministic_mode():
    """torch's deterministic mode fills new memory with NaN; what a call leaves alone shows it."""
    cache, table = torch.zeros(4, 16, 512, dtype=BF, device=DEV), torch.arange(4, dtype=torch.int32, device=DEV).view(2, 2)
    cu = torch.tensor([0, 5, 8], dtype=torch.int32, device=DEV)
    torch.use_deterministic_algorithms(True)
    try:
        rows, _ = kda.kda_latent_gather(cache, table, cu, 11)
    finally:
        torch.use_deterministic_algorithms(False)
    torch.cuda.synchronize()
    assert bool((rows[:8] == 0).all()) and bool(rows[8:].isnan().all())
