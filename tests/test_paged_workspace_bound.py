"""The workspace that dash_attn_paged asks for holds the partial rows that its cutting rules make: the rules themselves,
compiled for the host, over random batches."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from tile_scheduling_persistent_gb300 import build, dash

SOURCE = r"""
#include "dash_paged.cuh"
using namespace dash;
extern "C" int header_bytes() { return (256 + (int)sizeof(Plan) + 255) / 256 * 256; }
extern "C" int most_few(int type) { return few_most(type); }
// key ranges of a sequence of n tokens that sees keys [lo, hi)
extern "C" int ranges(int lo, int hi, int n, int G, int Hkv, int D, int type) {
    int ns, st;
    if (few_rows(n, G, type)) {
        few_split(hi > lo ? (hi - 1) / kFewKeys - lo / kFewKeys + 1 : 0, few_workers(D, type), Hkv * few_parts(n, G), ns, st);
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
    d = tmp_path_factory.mktemp("rules")
    (d / "rules.cu").write_text(SOURCE)
    subprocess.run([nvcc, *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-I", build.CSRC, "-I",
                    build.INCLUDE, "-shared", "-o", str(d / "rules.so"), str(d / "rules.cu")], check=True)
    return ctypes.CDLL(str(d / "rules.so"))


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dash.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dash.lib()


def seen(n, length, causal, window):
    p0 = length - n
    hi = max(length, 0) if causal else length
    lo = p0 + 1 - window if window and p0 + 1 > window else 0
    return lo, hi


def batch(r):
    """Hq, Hkv, D, type, causal, window, new tokens and lengths of each sequence."""
    G = r.choice([1, 1, 2, 3, 4, 4, 7, 8, 16, 17, 32, 33, 64, 128])
    Hkv = r.choice([1, 1, 2, 3, 4, 8, 8, 16, 32, 100, 500])
    D, typ = r.choice([64, 128]), r.choice([0, 1])
    causal = r.random() < 0.8
    window = r.choice([0, 0, int(2 ** r.uniform(0, 17))]) if causal else 0
    B = r.choice([1, 1, 2, 3, 16, 64, 200, 512])
    longest, wide = int(2 ** r.uniform(4, 21)), int(2 ** r.uniform(0, 13))
    same_n, same_len = r.random() < 0.4, r.random() < 0.4
    n, lens = [], []
    for _ in range(B):
        n.append(wide if same_n else r.choice([0, 1, 1, 1, r.randint(1, wide)]))
        lens.append(longest if same_len else r.choice([0, 1, r.randint(0, longest), longest]))
    return Hkv * G, Hkv, D, typ, causal, window, n, lens


def test_partial_rows_fit_the_workspace(L, rules):
    r = random.Random(0)
    split = closest = 0
    for _ in range(4000):
        Hq, Hkv, D, typ, causal, window, n, lens = batch(r)
        T, G = sum(n), Hq // Hkv
        if T == 0 or T * Hq >= 2 ** 31:
            continue
        rows = 0
        for m, ln in zip(n, lens):
            if m:
                ns = rules.ranges(*seen(m, ln, causal, window), m, G, Hkv, D, typ)
                rows += m * Hq * ns if ns > 1 else 0
        try:
            need = dash.attn_paged_workspace(len(n), T, Hq, Hkv, D, max(n), max(lens))
        except dash.DashError:   # a bound past 32 bits is refused
            continue
        held = (need - rules.header_bytes()) // (4 * D + 8) if need else 0
        assert rows <= held, (Hq, Hkv, D, typ, causal, window, n, lens)
        split += rows > 0
        closest = max(closest, rows / max(held, 1))
    assert split > 1000 and closest > 0.9   # the sweep reaches split sequences, and bounds that are nearly met


def test_a_workspace_is_asked_for_and_a_smaller_one_refused(L):
    import test_serving_cpu as S
    c = dict(c=S.cache(H=8, D=128, page=16), Hq=32, T=2, max_q=1, pages=1 << 13, cu=None)
    need = dash.attn_paged_workspace(2, 2, 32, 8, 128, 1, 1 << 17)
    assert need > 0
    assert S.call_attn(L, wn=need - 1, **c) == dash.ERR_SCRATCH
    assert S.call_attn(L, ws=None, **c) == dash.ERR_ARG
