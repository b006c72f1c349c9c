"""Paged attention at the edges of its protocol and its arithmetic: runs of the smallest items, weights far apart,
errors of several kernels at once, workspaces of exactly the size asked for, long contexts."""
import numpy as np
import pytest
import torch

from oracle import serving as V
from tile_scheduling_persistent_gb300 import dash

from serving_helpers import DEV, check_attn, no_error, paged, randn, run_attn, same

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("quant", [False, True])
def test_many_items_of_one_row_tile_and_one_key_tile(D, quant):
    # Some 25 items for each SM, every one of them a single row tile (33 to 128 rows) over a single key tile: queries, keys
    # and values of two items are staged at once, and the roles that stage them run as far ahead of the products as they can.
    g = gen(60)
    B = 480
    lens = [17 + 37 * i % 112 for i in range(B)]
    n = [9 + i % 8 if i % 16 else 12 for i in range(B)]
    c = paged(g, lens, 8, D, 16, quant)
    q = randn(g, sum(n), 32, D)
    o, lse = run_attn(c, q, n)
    no_error()
    check_attn(c, q, n, o, lse)
    for _ in range(20):
        again = run_attn(c, q, n)
        no_error()
        assert same(o, again[0]) and same(lse, again[1])
