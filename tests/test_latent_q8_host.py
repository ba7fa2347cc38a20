"""The 8-bit latent cache on the host: what the C ABI and the binding refuse, before any CUDA call."""
import ctypes
import os
import subprocess

import pytest
import torch

import linear_attention_06_gb300 as kda
from linear_attention_06_gb300 import _lib
from linear_attention_06_gb300 import build as kbuild
from tests import latent_q8_reference as q8
from tests.test_latent_host import ARG, BAD_SHAPES, FAKE, MIS, OK, UNS, shape


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return _lib.lib()


def append(L, sh=None, lat=FAKE, lat_s=512, kr=FAKE, kr_s=64, freq=FAKE, inter=0, q=FAKE, q_s=64, qo=FAKE, qo_s=64,
           cu=None, lens=FAKE, table=FAKE, cache=FAKE, scales=FAKE + 1):
    return L.kda_latent_append_q8(shape() if sh is None else sh, lat, lat_s, kr, kr_s, freq, inter, q, q_s, qo, qo_s, cu,
                                  lens, table, cache, scales, None)


def gather(L, sh=None, cache=FAKE, scales=FAKE + 1, table=FAKE, cu=FAKE, starts=None, lat=FAKE, kr=FAKE):
    return L.kda_latent_gather_q8(shape() if sh is None else sh, cache, scales, table, cu, starts, lat, kr, None)


def decode(L, sh=None, q=FAKE, qr=FAKE, cache=FAKE, scales=FAKE + 1, table=FAKE, lens=FAKE, scale=1.0, out=FAKE, lse=None,
           ws=FAKE, size=1 << 40):
    return L.kda_latent_decode_q8(shape() if sh is None else sh, q, qr, cache, scales, table, lens, scale, out, lse, ws, size, None)


@pytest.mark.parametrize("kw,code", BAD_SHAPES)
def test_shapes_refused_by_every_call(L, kw, code):
    for f in (append, gather, decode):
        assert f(L, shape(**kw)) == code
    size = ctypes.c_size_t(5)
    assert L.kda_latent_decode_q8_workspace_size(shape(**kw), ctypes.byref(size)) == code and size.value == 0


def test_null_shape(L):
    for f in (append, gather, decode):
        assert f(L, ctypes.POINTER(_lib.KdaLatentShape)()) == ARG
    assert L.kda_latent_decode_q8_workspace_size(shape(), None) == ARG


def test_append_refusals(L):
    for kw in (dict(lat=None), dict(kr=None), dict(lens=None), dict(table=None), dict(cache=None), dict(scales=None), dict(qo=None),
               dict(lat_s=511), dict(kr_s=63), dict(q_s=0), dict(qo_s=8), dict(inter=2), dict(sh=shape(n=3, T=4)),
               dict(sh=shape(n=0, T=4)), dict(sh=shape(rope=0))):
        assert append(L, **kw) == ARG, kw
    for kw in (dict(lat=MIS), dict(kr=MIS), dict(q=MIS), dict(qo=MIS), dict(cache=MIS), dict(table=FAKE + 2),
               dict(lens=FAKE + 1), dict(freq=FAKE + 2), dict(cu=FAKE + 2), dict(lat_s=513), dict(kr_s=65),
               dict(q_s=68), dict(qo_s=67), dict(sh=shape(T=2 ** 31))):
        assert append(L, **kw) == UNS, kw
    assert append(L, shape(n=0, T=0), lat=None, lens=None, cache=None, scales=None, table=None) == OK
    assert append(L, shape(T=0), lat=None) == OK


def test_gather_refusals(L):
    for kw in (dict(lat=None), dict(kr=None), dict(table=None), dict(cache=None), dict(scales=None), dict(sh=shape(n=0)),
               dict(sh=shape(T=3), cu=None), dict(sh=shape(rope=0))):
        assert gather(L, **kw) == ARG, kw
    for kw in (dict(lat=MIS), dict(kr=MIS), dict(cache=MIS), dict(table=FAKE + 1), dict(cu=FAKE + 2), dict(starts=FAKE + 2)):
        assert gather(L, **kw) == UNS, kw
    assert gather(L, shape(T=0), lat=None, kr=None, cache=None, scales=None) == OK


def test_decode_refusals(L):
    for kw in (dict(q=None), dict(qr=None), dict(cache=None), dict(scales=None), dict(table=None), dict(lens=None), dict(out=None),
               dict(ws=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(sh=shape(n=4, T=6)), dict(sh=shape(T=0)), dict(sh=shape(n=0, T=2)), dict(size=0), dict(sh=shape(rope=0))):
        assert decode(L, **kw) == ARG, kw
    for kw in (dict(q=MIS), dict(qr=MIS), dict(cache=MIS), dict(out=MIS), dict(lse=FAKE + 2), dict(table=FAKE + 3),
               dict(lens=FAKE + 2), dict(ws=FAKE + 128), dict(sh=shape(n=2, T=34)), dict(sh=shape(n=2 ** 22, T=2 ** 22, H=512))):
        assert decode(L, **kw) == UNS, kw
    assert decode(L, shape(n=0, T=0), q=None, qr=None, cache=None, scales=None, ws=None) == OK


def test_decode_workspace(L):
    for T, H in ((1, 1), (1, 32), (16, 32), (1, 128), (16, 1024)):
        size = kda.kda_latent_decode_q8_workspace_size(3, 3 * T, H)
        assert 0 < size <= 48 << 20
        assert decode(L, shape(n=3, T=3 * T, H=H), size=size - 1) == ARG
        assert size == kda.kda_latent_decode_q8_workspace_size(1000, 1000 * T, H, rope_dim=0)
    assert kda.kda_latent_decode_q8_workspace_size(0, 0, 4) == 0


def test_valid_calls_without_a_gpu_report_a_cuda_error(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for f in (append, gather, decode):
        assert f(L) == _lib.KDA_ERR_CUDA
        assert f(L, shape(pages=0), cache=None, scales=None) == _lib.KDA_ERR_CUDA


def test_binding_refuses_cpu_tensors_and_streams_of_another_device(L):
    class Stream:
        cuda_stream, device = FAKE, torch.device("cuda", 1)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    cache = torch.zeros(1, 16, 576, dtype=torch.uint8).view(q8.E4M3)
    scales = torch.zeros(1, 16, dtype=torch.uint8).view(q8.E8M0)
    t = torch.zeros(1, 1, dtype=torch.int32)
    calls = (lambda **kw: kda.kda_latent_append_q8(z(1, 512), z(1, 64), cache, scales, t, t[0], **kw),
             lambda **kw: kda.kda_latent_decode_q8(z(1, 1, 512), z(1, 1, 64), cache, scales, t, t[0], 1.0, **kw),
             lambda **kw: kda.kda_latent_gather_q8(cache, scales, t, [0, 1], 1, **kw))
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call(stream=Stream())


def test_the_reference_rounds_as_the_format_does():
    """The tests' own quantisation against torch's conversion, over every bf16 number that e4m3 covers, and the power of
    two against its definition."""
    x = torch.arange(2 ** 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()
    x = x[x.isfinite() & (x.abs() <= 448)]
    assert torch.equal(q8.to_e4m3(x), x.float().to(q8.E4M3).double())
    most = torch.tensor([448.0, 449, 447, 224, 224.5, 1.75, 1.7500001, 2.0 ** -60, 2.0 ** -100, 0.0], dtype=torch.float64)
    e = q8.power_of_rows(most[:, None])
    assert e.tolist() == [0, 1, 0, -1, 0, -8, -7, -64, -64, -64]
    assert torch.equal(q8.two(torch.tensor([-64, 0, 120])), torch.tensor([2.0 ** -64, 1.0, 2.0 ** 120], dtype=torch.float64))


def test_runs_of_the_line_take_every_tile_once(tmp_path):
    """The walk of kda_latent_runs.h with the 8-bit decode's tiles and start places: every tile of every sequence in
    exactly one run, whatever the lengths, and no part for the workspace where one run is all there is."""
    src, exe = tmp_path / "runs.cpp", tmp_path / "runs"
    src.write_text(RUNS)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-I", kbuild.CSRC, str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0 and done.stdout == "ok\n", done.stdout


RUNS = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "kda_latent_runs.h"
using namespace kda::latent;
constexpr int TILE = 128, START = 3;

static int walk(const std::vector<int>& lens, int runs, std::vector<int>& tiles) {
    const int count = (int)lens.size();
    int64_t total = 0;
    std::vector<int64_t> first;
    for (int x : lens) { first.push_back(total); total += START + tiles_of<TILE>(x); }
    if (total < runs) runs = (int)total;
    int partial = 0;
    for (int r = 0; r < runs; ++r) {
        const int64_t begin = run_begin(total, runs, r), end = run_begin(total, runs, r + 1);
        int n = count - 1;
        while (first[n] > begin) --n;
        const int into = (int)(begin - first[n]);
        RunWalkOf<TILE, START> w{n, into < START ? 0 : into - START, into < START ? START - into : 0, lens[n], end - begin};
        Piece p;
        int64_t at = begin + w.lead;          // the piece's first tile in the line, as the kernel follows it
        while (w.next(count, [&](int n) { return lens[n]; }, p)) {
            if (p.off < 0 || p.tiles <= 0 || p.off + p.tiles > p.all) return -1;
            if (at != first[p.n] + START + p.off || run_of(total, runs, at) != r) return -2;
            tiles[p.n] += p.tiles;
            settle(p, runs);
            partial += !is_whole(p);
            at += p.tiles + START;
        }
    }
    return partial;
}

int main() {
    srand(2);
    for (int round = 0; round < 4000; ++round) {
        std::vector<int> lens(1 + rand() % 12);
        for (int& x : lens) x = rand() % 4 ? rand() % 700 : rand() % 20000;
        for (int runs : {1, 2 + rand() % 150, 152}) {
            std::vector<int> tiles(lens.size());
            const int partial = walk(lens, runs, tiles);
            if (partial < 0 || (runs == 1 && partial)) return printf("runs %d: %d\n", runs, partial), 1;
            for (size_t n = 0; n < lens.size(); ++n)
                if (tiles[n] != tiles_of<TILE>(lens[n])) return printf("tiles missed or taken twice\n"), 1;
        }
    }
    printf("ok\n");
    return 0;
}
"""


@pytest.mark.parametrize("total", [2, torch.tensor(2), torch.tensor([2])])
@pytest.mark.parametrize("gather", [kda.kda_latent_gather, kda.kda_latent_gather_q8])
def test_a_host_table_takes_its_total_from_a_tensor_too(gather, total, monkeypatch):
    """total_tokens as the table's own last entry, a number or a tensor of one: validated and handed on as it is."""
    class Cuda:                                                # a cache that says it is on a device
        is_cuda, device = True, torch.device("cpu")

    class Native:
        @staticmethod
        def gather(cache, table, cu, tokens, *rest):
            return cu, tokens

        @staticmethod
        def gather_q8(cache, scales, table, cu, tokens, *rest):
            return cu, tokens

    monkeypatch.setattr(_lib, "_native", Native)
    cache = (Cuda(),) if gather is kda.kda_latent_gather else (Cuda(), None)
    cu, tokens = gather(*cache, None, [0, 1, 2], total)
    assert cu.tolist() == [0, 1, 2] and tokens is total
    with pytest.raises(kda.KdaError):
        gather(*cache, None, [0, 1, 3], total)
