"""dash_packed: every word reaches the argument of its place, and words out of an int's range are refused."""
import ctypes
import os
import re
import shutil
import struct
import subprocess

import pytest

from tile_scheduling_persistent_gb300 import build, dash

CALLS = ("dash_kv_write", "dash_kv_read", "dash_attn_paged", "dash_pages_fork", "dash_pages_extend", "dash_pages_compact")
OK = 4096   # an aligned address, never dereferenced


def parameters(name):
    """The types and names of a call's parameters, from the header."""
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(build.INCLUDE, "dash.h")).read(), flags=re.S)
    args = re.search(r"\bint %s\((.*?)\);" % name, text, flags=re.S).group(1)
    return [re.match(r"\s*(.*?[\s*])(\w+)\s*$", a, flags=re.S).groups() for a in args.split(",")]


@pytest.fixture(scope="module")
def recorded(tmp_path_factory):
    """dash_packed over calls that write down what they get."""
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("packed")
    src = '#include "dash.h"\nextern "C" int64_t got[32];\nint64_t got[32];\n'
    for n, name in enumerate(CALLS):
        ps = parameters(name)
        body = "".join("got[%d] = (int64_t)%s;" % (i, p) for i, (_, p) in enumerate(ps))
        src += 'extern "C" int %s(%s) { %s return %d; }\n' % (name, ", ".join(t + p for t, p in ps), body, 100 + n)
    (d / "calls.cpp").write_text(src)
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I", build.INCLUDE, "-o", str(d / "packed.so"), str(d / "calls.cpp"),
                    os.path.join(build.CSRC, "dash_packed.cpp")], check=True)
    L = ctypes.CDLL(str(d / "packed.so"))
    L.dash_packed.argtypes = [ctypes.c_int] + [ctypes.c_void_p] * 3
    return L, (ctypes.c_int64 * 32).in_dll(L, "got")


@pytest.mark.parametrize("call", range(6))
def test_words_arrive_in_order(recorded, call):
    L, got = recorded
    ps = parameters(CALLS[call])
    own = {"cache": 7 << 40, "rope": 9 << 40}
    wide = [t.strip() != "int" for t, p in ps if p not in own]
    words = [((i + 1) << 35) + i if w else -1000 - i for i, w in enumerate(wide)]
    assert L.dash_packed(call, struct.pack("@%dq" % len(words), *words), own["cache"], own["rope"]) == 100 + call
    rest = iter(words)
    assert list(got[:len(ps)]) == [own[p] if p in own else next(rest) for _, p in ps]
    for i, w in enumerate(wide):   # an int that does not fit, alone
        for bad in (1 << 31, -(1 << 31) - 1, 1 << 40):
            x = list(words)
            x[i] = bad
            assert L.dash_packed(call, struct.pack("@%dq" % len(x), *x), own["cache"], own["rope"]) == (100 + call if w else dash.ERR_ARG)


def test_the_bindings_blocks_have_a_word_for_each_argument():
    blocks = (dash._KV_WRITE, dash._KV_READ, dash._ATTN_PAGED, dash._FORK, dash._EXTEND, dash._COMPACT)
    for name, block in zip(CALLS, blocks):
        assert block.size == 8 * sum(p not in ("cache", "rope") for _, p in parameters(name))


def test_refusals():
    if not os.path.exists(dash.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    L = dash.lib()
    words = bytes(8 * 20)
    assert L.dash_packed(-1, words, None, None) == dash.ERR_ARG and L.dash_packed(6, words, None, None) == dash.ERR_ARG
    for call in range(6):
        assert L.dash_packed(call, None, None, None) == dash.ERR_ARG
    for call in range(3):
        assert L.dash_packed(call, words, None, None) == dash.ERR_ARG      # no cache
    for call in (4, 5):
        assert L.dash_packed(call, words, None, None) == dash.ERR_ARG      # no pool
    assert L.dash_packed(3, dash._FORK.pack(OK, 8, OK, -1, OK, 2 * OK, 8, 2 * OK, 4, 8, OK, 10, 16, 0), None, None) == dash.ERR_ARG
