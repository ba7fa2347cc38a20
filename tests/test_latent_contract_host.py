"""Latent attention on the host: promises of the calls that need no GPU to be checked."""
import ctypes
import glob
import os
import re
import subprocess

import pytest
import torch

import linear_attention_06_gb300 as kda
from linear_attention_06_gb300 import _lib
from linear_attention_06_gb300 import build as kbuild


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(kbuild.CSRC, "kda_latent_*.cu*"))), ids=os.path.basename)
def test_overlapped_kernels_read_nothing_as_read_only_data(path):
    """These kernels may be resident while the kernel before them still writes what they read, so no load of theirs
    may go through the read-only path, which promises memory that nobody writes while the kernel lives."""
    with open(path) as f:
        code = re.sub(r"//.*", "", f.read())
    assert not re.search(r"__ldg\b|ld\.global(\.\w+)*\.nc|__restrict__", code)


RUNS = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "kda_latent_runs.h"
using namespace kda::latent;

// A line in `runs` runs over sequences of the given lengths; length(n) is what the walk reads.  Returns the pieces that
// go to the workspace, -1 if a piece leaves its sequence, and counts the tiles of each sequence.
template <typename Length>
static int walk(const std::vector<int>& lens, int runs, const Length& length, std::vector<int>& tiles) {
    const int count = (int)lens.size();
    int64_t total = 0;
    std::vector<int64_t> first;
    for (int x : lens) { first.push_back(total); total += kStart + tiles_of(x); }
    if (total < runs) runs = (int)total;
    int partial = 0;
    for (int r = 0; r < runs; ++r) {
        const int64_t begin = run_begin(total, runs, r), end = run_begin(total, runs, r + 1);
        int n = count - 1;
        while (first[n] > begin) --n;
        const int into = (int)(begin - first[n]);
        RunWalk w{n, into < kStart ? 0 : into - kStart, into < kStart ? kStart - into : 0, lens[n], end - begin};
        Piece p;
        while (w.next(count, length, p)) {
            if (p.n < 0 || p.n >= count || p.off < 0 || p.tiles <= 0 || p.off + p.tiles > p.all) return -1;
            tiles[p.n] += p.tiles;
            settle(p, runs);
            partial += !is_whole(p);
        }
    }
    return partial;
}

int main() {
    srand(1);
    for (int round = 0; round < 4000; ++round) {
        std::vector<int> lens(1 + rand() % 12);
        for (int& x : lens) x = rand() % 4 ? rand() % 700 : rand() % 9000;
        std::vector<int> tiles(lens.size());
        if (walk(lens, 1, [&](int n) { return lens[n]; }, tiles) != 0) return printf("one run leaves a part\n"), 1;
        for (size_t n = 0; n < lens.size(); ++n)
            if (tiles[n] != tiles_of(lens[n])) return printf("tiles missed\n"), 1;
        // lengths that change after the line was measured: nothing may go to the workspace, which has no room for it
        if (walk(lens, 1, [&](int n) { return rand() % 2 ? lens[n] + rand() % 5000 : rand() % (lens[n] + 1); }, tiles) != 0)
            return printf("one run leaves a part when lengths change\n"), 1;
        std::vector<int> again(lens.size());
        if (walk(lens, 2 + rand() % 150, [&](int n) { return lens[n]; }, again) < 0) return printf("a piece leaves its sequence\n"), 1;
        for (size_t n = 0; n < lens.size(); ++n)
            if (again[n] != tiles_of(lens[n])) return printf("tiles missed or taken twice\n"), 1;
    }
    printf("ok\n");
    return 0;
}
"""


def test_a_line_in_one_run_never_uses_the_workspace(tmp_path):
    """With so many rows a step that one run is all the grid holds, the workspace has no room for partial results: the
    walk of the run asks for none, not even where lengths change while the call runs."""
    kbuild.build()
    per_row = 512 * 4
    for T, H in ((5, 1024), (16, 1024)):
        assert kda.kda_latent_decode_workspace_size(2, 2 * T, H) < 64 * per_row
    src, exe = tmp_path / "runs.cpp", tmp_path / "runs"
    src.write_text(RUNS)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-I", kbuild.CSRC, str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0 and done.stdout == "ok\n", done.stdout


FAKE = 0x10000                          # never dereferenced


def test_data_without_a_place_is_refused():
    """Rotated parts beside a cache or queries that have none, and an output without its input: all refused before any
    CUDA call; the same calls without them get as far as the device."""
    kbuild.build()
    L = kda.lib()
    bare = ctypes.byref(kda.KdaLatentShape(2, 2, 4, 512, 0, 64, 8, 4, _lib.KDA_BF16))
    full = ctypes.byref(kda.KdaLatentShape(2, 2, 4, 512, 64, 64, 8, 4, _lib.KDA_BF16))
    narrow = ctypes.byref(kda.KdaShape(2, 4, 3, 128, 128, _lib.KDA_BF16))
    ends = (None, FAKE, FAKE, FAKE, None)                      # cu_seqlens, seq_lens, block_table, cache, stream

    def append(shape, k_rope, freq, q, q_out):
        return L.kda_latent_append(shape, FAKE, 512, k_rope, 64, freq, 0, q, 64, q_out, 64, *ends)

    def gather(k_rope):
        return L.kda_latent_gather(bare, FAKE, FAKE, FAKE, None, FAKE, k_rope, None)

    def decode(q_rope):
        return L.kda_latent_decode(bare, FAKE, q_rope, FAKE, FAKE, FAKE, 1.0, FAKE, None, FAKE, 1 << 40, None)

    def prefill(k_rope, total_kv=4):
        return L.kda_latent_prefill(narrow, total_kv, FAKE, FAKE, FAKE, 128, k_rope, 1.0, None, None, FAKE, None, None)

    for st in (append(bare, FAKE, None, None, None), append(bare, FAKE, FAKE, None, None), append(bare, None, None, FAKE, FAKE),
               append(full, FAKE, FAKE, None, FAKE), gather(FAKE), decode(FAKE), prefill(FAKE), prefill(FAKE, 0)):
        assert st == _lib.KDA_ERR_INVALID_ARG
    if torch.cuda.is_available():
        return                                                 # the calls below would run on the addresses
    for st in (append(bare, None, None, None, None), append(bare, None, FAKE, None, None), append(full, FAKE, FAKE, None, None),
               gather(None), decode(None), prefill(None), prefill(None, 0)):
        assert st == _lib.KDA_ERR_CUDA


SPLIT = r"""
#include <cstdio>
#include <cstdlib>
#include "kda_latent_split.h"
int main(int argc, char** argv) {
    // tiles, clusters with queries, clusters, and how many of two, four and eight blocks run at once
    const int room[3] = {atoi(argv[4]), atoi(argv[5]), atoi(argv[6])};
    printf("%d", kda::latent::split_of(atoll(argv[1]), atoll(argv[2]), atoll(argv[3]),
                                       [&](int parts) { return room[parts == 2 ? 0 : parts == 4 ? 1 : 2]; }));
    return 0;
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    (d / "split.cpp").write_text(SPLIT)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-I", kbuild.CSRC, str(d / "split.cpp"), "-o", str(d / "split")],
                   check=True)

    def call(n, nq, nk, H, room=(76, 36, 15)):
        busy, slots = -(-nq // 256) * n * H, (-(-n * nq // 256) + n - 1) * H
        args = [nk // 128, busy, slots, *room]
        return int(subprocess.run([str(d / "split"), *map(str, args)], capture_output=True, text=True, check=True).stdout)
    return call


@pytest.mark.parametrize("n,nq,nk,H,good", [
    # more slots than clusters that start together: the times of 1, 2 and 4 blocks (us) stand behind each
    (4, 512, 512, 4, (1,)),                                    # 12.6, 15.0, 15.6
    (9, 256, 512, 4, (1,)),                                    # 12.7, 15.6, 25.0
    (12, 100, 512, 3, (1,)),                                   # 11.3, 11.7, 16.2
    (8, 256, 1024, 4, (1, 2)),                                 # 18.2, 18.1, 21.1
    (4, 256, 1024, 16, (1,)),                                  # 18.6, 23.3, 34.5
    (9, 256, 2048, 4, (2,)),                                   # 29.3, 23.8, 29.4
    (4, 256, 4096, 8, (4,)),                                   # 50.7, 34.0, 29.1
    (8, 256, 4096, 8, (2,)),                                   # 57.4, 45.0, 56.7
    # one sequence, all its clusters at work together
    (1, 100, 16384, 32, (4,)), (1, 128, 8192, 1, (8,)), (1, 64, 600, 8, (4,)), (1, 200, 4096, 18, (4,)),
    (1, 512, 512, 8, (1, 4)), (1, 512, 512, 32, (1,)), (1, 1024, 1024, 1, (8,)), (1, 2048, 2048, 8, (2,)),
    (3, 100, 100, 32, (1,)), (4, 8192, 8192, 32, (1,))])
def test_blocks_share_keys_only_where_that_is_faster(split, n, nq, nk, H, good):
    """The number of blocks that share a block's keys, against what was measured on a card that runs 76 clusters of
    two, 36 of four and 15 of eight at once."""
    assert split(n, nq, nk, H) in good


def test_no_sharing_where_no_cluster_runs(split):
    assert split(1, 100, 16384, 32, room=(0, 0, 0)) == 1
