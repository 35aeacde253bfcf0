"""paged_attention where a wave goes over several tiles of a piece (the running
maximum is corrected, the next tile's loads are in flight while one is used),
and where a table is much wider than the contexts (captured graphs, padded
tables).  Bounds as in test_gpu_paged_attention.py.

A wave takes every fourth tile of 32 tokens, so a piece of more than 128 tokens
is more than one tile to a wave.  How many pieces a call has follows from its
workspace: per query head and piece, an output and two sums in float32.
"""
import numpy as np
import pytest
import torch

import oracle
from block_cases import DTYPES, E, check, draw, f64
from test_gpu_paged_attention import FORMS, _bound, _make

pytestmark = pytest.mark.gpu


def _pieces(rbp, batch, H, KV, D, page, width, window, fmt):
    need = rbp.lib.orbit_paged_attention_workspace(batch, H, KV, D, page, width, window, {"bf16": 1, "f16": 2, "int8": 3}[fmt])
    assert need >= 0
    return max(1, need // (batch * H * (D + 2) * 4))


def _pool(rng, pages, KV, page, D, fmt):
    """A cache of `pages` pages that requests share; the scores of page p's tokens rise with p."""
    lift = np.linspace(-1.0, 1.0, pages)[:, None, None]
    kw = {}
    if fmt == "int8":
        k, v = (rng.integers(-127, 128, (pages, KV, page, D)) for _ in "kv")
        k[..., 0] = np.round(127 * lift)
        scales = [rng.uniform(0.5, 1.5, (pages, KV, page)) / 73 for _ in "kv"]
        scales[0][:] = 1 / 64
        kw = {n: torch.from_numpy(s).half().cuda() for n, s in zip(("k_scale", "v_scale"), scales)}
        k, v = (torch.from_numpy(t.astype(np.int8)).cuda() for t in (k, v))
        k64, v64 = (f64(t) * f64(s)[..., None] for t, s in zip((k, v), kw.values()))
    else:
        k, v = rng.standard_normal((2, pages, KV, page, D))
        k[..., 0] = 2 * lift
        k, v = (torch.from_numpy(t).to(DTYPES[fmt]).cuda() for t in (k, v))
        k64, v64 = f64(k), f64(v)
    return k, v, kw, k64, v64


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("D,page", [(64, 8), (64, 16), (128, 8), (128, 64), (256, 16), (256, 8), (80, 16)])
@pytest.mark.parametrize("trend", ["rising", "falling", "both", "none"])
def test_several_tiles_to_a_wave(gpu_lib, xt, fmt, D, page, trend):
    batch, H, KV, pages = 520, 8, 8, 128
    rng = np.random.default_rng(D + page)
    width = -(-700 // page)
    assert _pieces(gpu_lib, batch, H, KV, D, page, width, 0, fmt) < -(-700 // 128)
    k, v, kw, k64, v64 = _pool(rng, pages, KV, page, D, fmt)
    lengths = rng.integers(0, 701, batch)
    lengths[:6] = 700, 0, 1, 257, 129, 640
    order = np.stack([np.sort(rng.choice(pages, width, replace=width > pages)) for _ in range(batch)])
    if trend == "falling":
        order = order[:, ::-1]
    elif trend == "both":
        order = np.concatenate([order[:, ::2], order[:, 1::2][:, ::-1]], 1)
    elif trend == "none":
        order = rng.permuted(order, axis=1)
    table = np.ascontiguousarray(order).astype(np.int32)
    q, q64 = draw(rng, (batch, H, D), DTYPES[xt])
    q[..., 0] = q[..., 0].abs() + 8  # the lifted coordinate carries the trend: scores go over ~ 30 / sqrt(D / 64)
    q64 = f64(q)
    check_rows = np.r_[0:24, 500:520]
    for window in (0, 300):
        out, lse = gpu_lib.paged_attention(q, k, v, torch.from_numpy(table).cuda(), torch.from_numpy(lengths).int().cuda(),
                                           window=window, scale=0.25, return_lse=True, **kw)
        args = q64[check_rows], k64, v64, table[check_rows], lengths[check_rows], 0.25, window
        ref, ref_lse = oracle.paged_attention(*args)
        o_mag, l_mag = _bound(*args, fmt, D)
        check(out[check_rows], ref, DTYPES[xt], o_mag, "out")
        check(lse[check_rows], ref_lse, torch.float32, l_mag + 4 * E * np.abs(np.where(np.isfinite(ref_lse), ref_lse, 0)), "lse")


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("page", [8, 16])
def test_hidden_pages_and_tokens_in_later_tiles(gpu_lib, xt, fmt, page):
    batch, H, KV, D, pages, n = 520, 8, 8, 64, 128, 900
    rng = np.random.default_rng(page)
    width = -(-n // page)
    assert _pieces(gpu_lib, batch, H, KV, D, page, width, 0, fmt) < -(-n // 128)
    k, v, kw, k64, v64 = _pool(rng, pages, KV, page, D, fmt)
    table = rng.integers(0, pages, (batch, width)).astype(np.int32)
    for b in range(batch):
        table[b, rng.integers(0, width, 1 + b % 20)] = (-1, pages, 2 ** 31 - 1)[b % 3]
    table[3] = -1
    table[4, 3:] = -1  # nothing is seen after the first tiles
    lengths = np.full(batch, n)
    lengths[5:8] = 870, 871, 897
    q, q64 = draw(rng, (batch, H, D), DTYPES[xt], 2.0)
    rows = np.r_[0:30, 510:520]
    for window in (0, 400, 33):
        out, lse = gpu_lib.paged_attention(q, k, v, torch.from_numpy(table).cuda(), torch.from_numpy(lengths).int().cuda(),
                                           window=window, return_lse=True, **kw)
        args = q64[rows], k64, v64, table[rows], lengths[rows], 0.125, window
        ref, ref_lse = oracle.paged_attention(*args)
        o_mag, l_mag = _bound(*args, fmt, D)
        check(out[rows], ref, DTYPES[xt], o_mag, "out")
        check(lse[rows], ref_lse, torch.float32, l_mag + 4 * E * np.abs(np.where(np.isfinite(ref_lse), ref_lse, 0)), "lse")


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("batch,H,KV,D,page,chunk", [(128, 8, 8, 128, 64, 1024), (64, 8, 8, 64, 256, 2048)])
def test_long_pieces_of_long_contexts(gpu_lib, xt, fmt, batch, H, KV, D, page, chunk):
    # pieces of a thousand tokens and more, several to a context
    rng = np.random.default_rng(chunk)
    pages, n = 96, 6 * chunk - 50
    width = -(-n // page) * (5 if batch == 64 else 2)
    pieces = _pieces(gpu_lib, batch, H, KV, D, page, width, 0, fmt)
    assert pieces > 1 and width * page / pieces > chunk / 2
    k, v, kw, k64, v64 = _pool(rng, pages, KV, page, D, fmt)
    table = rng.integers(0, pages, (batch, width)).astype(np.int32)
    lengths = rng.integers(0, n, batch)
    lengths[:4] = n, chunk, chunk + 1, width * page
    q, q64 = draw(rng, (batch, H, D), DTYPES[xt], 2.0)
    out, lse = gpu_lib.paged_attention(q, k, v, torch.from_numpy(table).cuda(), torch.from_numpy(lengths).int().cuda(),
                                       return_lse=True, **kw)
    args = q64[:6], k64, v64, table[:6], lengths[:6], D ** -0.5, 0
    ref, ref_lse = oracle.paged_attention(*args)
    o_mag, l_mag = _bound(*args, fmt, D)
    check(out[:6], ref, DTYPES[xt], o_mag, "out")
    check(lse[:6], ref_lse, torch.float32, l_mag + 4 * E * np.abs(np.where(np.isfinite(ref_lse), ref_lse, 0)), "lse")


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("batch,width", [(1, 8192), (4, 8192), (16, 8192), (16, 700)])
@pytest.mark.parametrize("window", [0, 100])
def test_tables_wider_than_the_contexts(gpu_lib, xt, fmt, batch, width, window):
    rng = np.random.default_rng(batch + width)
    H, KV, D, page = 8, 2, 64, 16
    lengths = [int(n) for n in rng.integers(0, 3000, batch)]
    lengths[0] = 2000
    q, k, v, table, kw, (q64, k64, v64, t64) = _make(rng, lengths, H, KV, D, page, xt, fmt, width=width)
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = gpu_lib.paged_attention(q, k, v, table, ln, window=window, return_lse=True, **kw)
    ref, ref_lse = oracle.paged_attention(q64, k64, v64, t64, lengths, D ** -0.5, window)
    o_mag, l_mag = _bound(q64, k64, v64, t64, lengths, D ** -0.5, window, fmt, D)
    check(out, ref, DTYPES[xt], o_mag, "out")
    check(lse, ref_lse, torch.float32, l_mag + 4 * E * np.abs(np.where(np.isfinite(ref_lse), ref_lse, 0)), "lse")


@pytest.mark.parametrize("xt,fmt", [("bf16", "bf16"), ("f16", "int8")])
def test_lengths_that_grow_in_a_replayed_graph(gpu_lib, xt, fmt):
    rng = np.random.default_rng(1)
    H, KV, D, page, width, batch = 8, 2, 128, 16, 8192, 4
    most = [40000, 9000, 300, 5000]
    q, k, v, table, kw, (q64, k64, v64, t64) = _make(rng, most, H, KV, D, page, xt, fmt, width=width)
    ln = torch.tensor([1] * batch, dtype=torch.int32, device="cuda")
    out = gpu_lib.paged_attention(q, k, v, table, ln, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.paged_attention(q, k, v, table, ln, out=out, **kw)
    for lengths in ([0, 1, 2, 3], [100, 0, 300, 129], [5000, 9000, 0, 4096], most):
        ln.copy_(torch.tensor(lengths, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, gpu_lib.paged_attention(q, k, v, table, ln, **kw))
        ref, _ = oracle.paged_attention(q64, k64, v64, t64, lengths, D ** -0.5)
        o_mag, _ = _bound(q64, k64, v64, t64, lengths, D ** -0.5, 0, fmt, D)
        check(out, ref, DTYPES[xt], o_mag)
