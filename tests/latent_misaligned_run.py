"""Run the latent decodes on a library built with -DKDA_TEST_MISALIGNED, whose blocks all take their shared memory for
misaligned: they must report it and leave the join nothing to do, whatever the workspace held before.

Executed in a child process by tests/test_latent_misaligned_gpu.py (so that it loads its own copy of the library); prints
"left alone" at the end.
"""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def main() -> int:
    from linear_attention_06_gb300 import _lib
    from linear_attention_06_gb300 import build as _build
    _lib.LIB_PATH = _build.build(extra_flags=["-DKDA_TEST_MISALIGNED"], tag="misaligned")
    _lib._lib = _lib._native = None

    import torch

    import linear_attention_06_gb300 as kda

    bf, u8, dev = torch.bfloat16, torch.uint8, "cuda"
    for H, T, rope in ((4, 1, 64), (32, 1, 0), (64, 1, 64), (32, 16, 64)):
        n, page = 5, 64
        table = torch.arange(n * 20, dtype=torch.int32, device=dev).view(n, 20)
        lens = torch.tensor([1200, 5, 0, 700, 129], dtype=torch.int32, device=dev)
        q = torch.ones(n * T, H, 512, dtype=bf, device=dev)
        qr = torch.ones(n * T, H, 64, dtype=bf, device=dev) if rope else None
        rows = torch.zeros(n * 20, page, 512 + rope, dtype=bf, device=dev)
        held = (rows.to(torch.float8_e4m3fn), torch.full((n * 20, page), 127, dtype=u8, device=dev).view(torch.float8_e8m0fnu))
        for name, cache, size in (("kda_latent_decode", (rows,), kda.kda_latent_decode_workspace_size),
                                  ("kda_latent_decode_q8", held, kda.kda_latent_decode_q8_workspace_size)):
            # headers of zeros name sequence 0, an index that is in range: a join that believed them would write its rows
            ws = torch.zeros(size(n, n * T, H, rope), dtype=u8, device=dev)
            out, lse = torch.full_like(q, 7.0), torch.full((n * T, H), 7.0, device=dev)
            getattr(kda, name)(q, qr, *cache, table, lens, 0.07, out=out, lse=lse, workspace=ws)
            torch.cuda.synchronize()
            assert kda.kda_device_status() != _lib.KDA_OK, "not reported"
            assert bool((out == 7.0).all()) and bool((lse == 7.0).all()), f"{name}, {H} heads: rows were written"
    print("left alone")
    return 0


if __name__ == "__main__":
    sys.exit(main())
