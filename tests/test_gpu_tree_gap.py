"""paged_tree_attention and paged_attention behind a window with sinks, the pages between the two given up (-1, or any
other number outside the cache), as a server does with a sequence that has outgrown its window (bounds: tree_cases.py)."""
import numpy as np
import pytest
import torch

from block_cases import DTYPES, check
from tree_cases import Case, tree_mask

pytestmark = pytest.mark.gpu

FORMS = [("bf16", "bf16"), ("f16", "int8")]


def give_up(c):
    """Takes the pages that no token of their request sees out of the table; how many."""
    gone = 0
    for b, (length, n) in enumerate(c.requests):
        for p in range(c.table64.shape[1]):
            if p * c.page >= c.sinks and (p + 1) * c.page <= length - n - c.window:
                c.table64[b, p] = (-1, 2 ** 31 - 1, -2 ** 31)[p % 3]
                gone += 1
    c.table = torch.from_numpy(c.table64).cuda()
    return gone


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(100, 4), (64, 64), (333, 1), (129, 70), (200, 0)])
def test_pages_between_sinks_and_window(gpu_lib, window, sinks, D, xt, fmt):
    rng = np.random.default_rng(window + D)
    for requests in ([(3000, 2), (90, 3), (700, 1)], [(3000, 90), (700, 333), (40, 40)]):
        for masks in (None, [tree_mask(rng, n) for _, n in requests]):
            c = Case(window, requests, H=4, KV=2, D=D, page=8, xt=xt, fmt=fmt, window=window, sinks=sinks, masks=masks)
            assert give_up(c) > 100
            c.check(gpu_lib)


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("page", [4, 16, 64, 1024])
def test_single_tokens(gpu_lib, page, xt, fmt):
    c = Case(page, [(n, 1) for n in (0, 1, 130, 5000, 20000)], page=page, xt=xt, fmt=fmt, window=500, sinks=5)
    assert give_up(c) > 10
    want, want_lse, omag, lmag = c.reference()
    out, lse = gpu_lib.paged_attention(c.q, c.k, c.v, c.table, c.lengths, scale=c.scale, window=500, sinks=5, return_lse=True, **c.kw)
    check(out, want, DTYPES[xt], omag, "out")
    check(lse, want_lse, torch.float32, lmag, "lse")


def test_pages_that_are_seen_may_be_missing_beside_them(gpu_lib):
    c = Case(1, [(3000, 90), (700, 333)], H=4, KV=2, page=8, window=300, sinks=20)
    give_up(c)
    c.table64[0, 1], c.table64[0, 3000 // 8 - 20], c.table64[1, 0], c.table64[1, 50] = -1, -7, 10 ** 6, -1
    c.table = torch.from_numpy(c.table64).cuda()
    c.check(gpu_lib)


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("window,sinks", [(1000, 4), (100, 4), (60, 30), (100, 70), (333, 200)])
def test_pages_missing_where_window_and_sinks_share_a_tile(gpu_lib, window, sinks, D, xt, fmt):
    """Every page in its turn is missing, those that a window sees in a tile of the sinks among them."""
    rng = np.random.default_rng(window)
    for requests in ([(120, 2)] * 15, [(120, 70)] * 15):
        for masks in (None, [tree_mask(rng, n) for _, n in requests]):
            c = Case(sinks, requests, H=4, KV=2, D=D, page=8, xt=xt, fmt=fmt, window=window, sinks=sinks, masks=masks)
            for b in range(15):
                c.table64[b, b] = -1 - b
            c.table = torch.from_numpy(c.table64).cuda()
            c.check(gpu_lib)
