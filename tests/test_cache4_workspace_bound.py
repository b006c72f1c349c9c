"""The workspace that dash_attn_paged asks for holds the partial rows that its cutting rules make of caches of 4 bits, too:
the rules themselves, compiled for the host, over random batches."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from tile_scheduling_persistent_gb300 import build, dash

from test_paged_workspace_bound import batch, seen

SOURCE = r"""
#include "dash_paged.cuh"
using namespace dash;
extern "C" int header_bytes() { return (256 + (int)sizeof(Plan) + 255) / 256 * 256; }
extern "C" int ranges(int lo, int hi, int n, int G, int Hkv, int D, int type) {
    int ns, st;
    if (few_rows(n, G, type)) {
        const int keys = few_keys(type);
        few_split(hi > lo ? (hi - 1) / keys - lo / keys + 1 : 0, few_workers(D, type), Hkv * few_parts(n, G), ns, st, type, n * G);
        return ns;
    }
    const int tiles = hi > lo ? (hi - 1) / 128 - lo / 128 + 1 : 0, tpi = tokens_per_item(G);
    ns = many_split(tiles, (long long)((n + tpi - 1) / tpi) * Hkv);
    st = (tiles + ns - 1) / ns;
    return st > 0 ? (tiles + st - 1) / st : 1;
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    d = tmp_path_factory.mktemp("rules4")
    (d / "rules.cu").write_text(SOURCE)
    subprocess.run([nvcc, *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-I", build.CSRC, "-I",
                    build.INCLUDE, "-shared", "-o", str(d / "rules.so"), str(d / "rules.cu")], check=True)
    return ctypes.CDLL(str(d / "rules.so"))


def test_partial_rows_of_a_cache_of_4_bits_fit_the_workspace(rules):
    if not os.path.exists(dash.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    r = random.Random(1)
    split = closest = 0
    for _ in range(4000):
        Hq, Hkv, D, _, causal, window, n, lens = batch(r)
        T, G = sum(n), Hq // Hkv
        if T == 0 or T * Hq >= 2 ** 31:
            continue
        rows = 0
        for m, ln in zip(n, lens):
            if m:
                ns = rules.ranges(*seen(m, ln, causal, window), m, G, Hkv, D, 2)
                rows += m * Hq * ns if ns > 1 else 0
        try:
            need = dash.attn_paged_workspace(len(n), T, Hq, Hkv, D, max(n), max(lens))
        except dash.DashError:   # a bound past 32 bits is refused
            continue
        held = (need - rules.header_bytes()) // (4 * D + 8) if need else 0
        assert rows <= held, (Hq, Hkv, D, causal, window, n, lens)
        split += rows > 0
        closest = max(closest, rows / max(held, 1))
    assert split > 1000 and closest > 0.4   # the sweep reaches split sequences (and bounds that other types meet by half as many stages)
