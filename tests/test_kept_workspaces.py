"""The workspaces that the binding keeps between calls of attn_paged: bounded, and given back by any thread."""
import gc
import threading
import weakref

import pytest
import torch

from tile_scheduling_persistent_gb300 import dash

MIB = 1 << 20


class Library:
    """In place of the loaded library: nothing of its own to release."""

    @staticmethod
    def dash_release_workspaces():
        return dash.OK


class Kept:
    """Workspaces asked for, by address alone: those that are still alive are kept by the binding."""

    def __init__(self):
        self.seen = {}

    def __call__(self, n, stream):
        w = dash._workspace(n, "cpu", stream)
        assert w.numel() >= n
        self.seen[id(w)] = weakref.ref(w)
        return id(w)

    def held(self):
        gc.collect()
        return sum(t.numel() for t in (r() for r in self.seen.values()) if t is not None)


@pytest.fixture
def kept(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(dash, "lib", Library)
    dash.release_workspaces()
    yield Kept()
    dash.release_workspaces()


def test_a_stream_keeps_its_workspace(kept):
    a, b = kept(1000, 1), kept(1000, 2)
    assert a != b and kept(500, 1) == a and kept(1000, 2) == b
    c = kept(3 * MIB, 1)
    assert kept(1000, 1) == c and kept(1000, 2) == b
    assert 4 * MIB <= kept.held() < 5 * MIB


def test_a_pool_of_streams_stays_bounded(kept):
    for i in range(40):
        kept(32 * MIB, 1000 + i)
    assert 32 * MIB <= kept.held() <= 256 * MIB
    last = kept(32 * MIB, 1039)
    assert kept(32 * MIB, 1039) == last
    before = kept.held()
    kept(32 * MIB + 1, 5)              # too large to be kept
    assert kept.held() == before


def test_one_thread_gives_back_the_workspaces_of_all(kept):
    got, asked, done = [], threading.Barrier(5), threading.Barrier(5)

    def work():
        got.append(kept(MIB, 7))
        asked.wait()
        done.wait()

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    asked.wait()
    assert len(set(got)) == 4 and kept.held() == 4 * MIB   # one for each thread that runs at the same time
    dash.release_workspaces()
    left = kept.held()
    done.wait()
    for t in threads:
        t.join()
    assert left == 0
