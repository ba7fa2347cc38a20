"""Run the entry points of the 8-bit latent cache on a library built with -DKDA_CHECK_BOUNDS and check that no kernel
skipped a global-memory access because its index left its buffer.

Executed in a child process by tests/test_latent_q8_gpu.py (so that it loads its own copy of the library); prints
one line per case and "bounds ok" at the end, and exits non-zero if a case's status is not KDA_OK.
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
    _lib.LIB_PATH = _build.build(extra_flags=["-DKDA_CHECK_BOUNDS"], tag="bounds")
    _lib._lib = _lib._native = None

    import torch

    import linear_attention_06_gb300 as kda

    bf, dev = torch.bfloat16, "cuda"
    failures = []

    def check(name):
        st = kda.kda_device_status()
        print(f"{name}: {_lib.status_string(st)}", flush=True)
        if st != _lib.KDA_OK:
            failures.append(name)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    torch.manual_seed(1)
    freq = torch.rand(32, device=dev)
    for rope in (0, 64):
        for page in (16, 64, 256):
            for T, H in ((1, 1), (1, 32), (3, 16), (16, 32), (2, 64)):
                lens = [0, T, 1, 64, 129, 700, 1500, -3, 10 ** 9]
                n, per = len(lens), 2048 // page
                cache = torch.randn(n * per, page, 512 + rope, device=dev).to(torch.float8_e4m3fn)
                scales = torch.randint(110, 130, (n * per, page), device=dev).to(torch.uint8).view(torch.float8_e8m0fnu)
                table = torch.randperm(n * per, device=dev).to(torch.int32).view(n, per).contiguous()
                table[3, 0], table[5, 2], table[5, 1] = -1, n * per, 2 ** 31 - 1
                rows = n * T
                q = torch.randn(rows, H, 512, device=dev).to(bf)
                qr = torch.randn(rows, H, 64, device=dev).to(bf) if rope else None
                for inter in (False, True):
                    kda.kda_latent_append_q8(q[:, 0].contiguous(), qr[:, 0].contiguous() if rope else None, cache, scales,
                                             table, i32(lens), inv_freq=freq, interleaved=inter, q_rope=qr, q_rope_out=qr)
                check(f"append rope={rope} page={page} T={T} H={H}")
                kda.kda_latent_decode_q8(q, qr, cache, scales, table, i32(lens), 0.07, lse=True)
                check(f"decode rope={rope} page={page} T={T} H={H}")
            cu = i32([0, 5, 5, 900, 1000, 9000, 9001, 9002, 9003, 9004])
            kda.kda_latent_gather_q8(cache, scales, table, cu, 9010, i32([0, 3, 0, -7, 0, 2040, 0, 1, 2]))
            kda.kda_latent_gather_q8(cache, scales, table, i32([0, 1, 2, 3, 4, 5, 6, 7, 8, 900]), 1000)
            check(f"gather rope={rope} page={page}")
            T = 3000                                           # a long append: many tokens a block
            kda.kda_latent_append_q8(torch.randn(T, 512, device=dev).to(bf),
                                     torch.randn(T, 64, device=dev).to(bf) if rope else None, cache, scales, table,
                                     i32(lens), inv_freq=freq,
                                     cu_seqlens=i32([0, 5, 5, 900, 1000, 2000, 2900, 2900, 2901, 2990]))
            check(f"long append rope={rope} page={page}")
    if failures:
        print("failed:", failures)
        return 1
    print("bounds ok")
    return 0


if __name__ == "__main__":
    sys.exit(main())
