"""Run the latent-attention entry points on a library built with -DKDA_CHECK_BOUNDS and check that no kernel
skipped a global-memory access because its index left its buffer.

Executed in a child process by tests/test_latent_gpu.py (so that it loads its own copy of the library); prints
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
                lens = [0, T, 1, 64, 65, 700, 1500, -3, 10 ** 9]
                n, per = len(lens), 2048 // page
                cache = torch.randn(n * per, page, 512 + rope, device=dev).to(bf)
                table = torch.randperm(n * per, device=dev).to(torch.int32).view(n, per).contiguous()
                table[3, 0], table[5, 2], table[5, 1] = -1, n * per, 2 ** 31 - 1
                rows = n * T
                q = torch.randn(rows, H, 512, device=dev).to(bf)
                qr = torch.randn(rows, H, 64, device=dev).to(bf) if rope else None
                for inter in (False, True):
                    kda.kda_latent_append(q[:, 0].contiguous(), qr[:, 0].contiguous() if rope else None, cache, table,
                                          i32(lens), inv_freq=freq, interleaved=inter, q_rope=qr, q_rope_out=qr)
                check(f"append rope={rope} page={page} T={T} H={H}")
                kda.kda_latent_decode(q, qr, cache, table, i32(lens), 0.07, lse=True)
                check(f"decode rope={rope} page={page} T={T} H={H}")
            cu = i32([0, 5, 5, 900, 1000, 9000, 9001, 9002, 9003, 9004])
            kda.kda_latent_gather(cache, table, cu, 9010, i32([0, 3, 0, -7, 0, 2040, 0, 1, 2]))
            kda.kda_latent_gather(cache, table, i32([0, 1, 2, 3, 4, 5, 6, 7, 8, 900]), 1000)
            check(f"gather rope={rope} page={page}")
            T = 3000                                           # a long append: many tokens a block
            kda.kda_latent_append(torch.randn(T, 512, device=dev).to(bf),
                                  torch.randn(T, 64, device=dev).to(bf) if rope else None, cache, table, i32(lens),
                                  inv_freq=freq, cu_seqlens=i32([0, 5, 5, 900, 1000, 2000, 2900, 2900, 2901, 2990]))
            check(f"long append rope={rope} page={page}")
        cq, ck = i32([0, 1, 1, 300, 700, 701]), i32([0, 1, 40, 100, 1200, 1201])
        q = torch.randn(705, 3, 128 + rope, device=dev).to(bf)
        kv = torch.randn(1210, 3, 256, device=dev).to(bf)
        kr = torch.randn(1210, 64, device=dev).to(bf) if rope else None
        kda.kda_latent_prefill(q, kv[..., :128], kv[..., 128:], kr, 0.07, cq, ck, lse=True)
        check(f"prefill rope={rope}")
        # offsets that are no table: reversed, negative and beyond the batch
        kda.kda_latent_prefill(q, kv[..., :128], kv[..., 128:], kr, 0.07, i32([0, 50, 20, 900, -4, 10 ** 9]),
                               i32([3, 2000, 5, 10, 10, 1210]), lse=True)
        check(f"prefill, bad tables rope={rope}")
        # few queries over many keys, which blocks share
        kv = torch.randn(9000, 3, 256, device=dev).to(bf)
        kr = torch.randn(9000, 64, device=dev).to(bf) if rope else None
        for qs, ks in (([0, 90, 90, 700], [0, 3000, 3001, 9000]), ([0, 50, 20, 10 ** 9], [3, 20000, 5, 9000])):
            kda.kda_latent_prefill(q, kv[..., :128], kv[..., 128:], kr, 0.07, i32(qs), i32(ks), lse=True)
            check(f"prefill, shared keys rope={rope}")
    if failures:
        print("index checks failed:", ", ".join(failures))
        return 1
    print("bounds ok")
    return 0


if __name__ == "__main__":
    sys.exit(main())
