"""paged_tree_attention, and paged_attention behind a window with sinks, against 64 bits (bounds: tree_cases.py)."""
import numpy as np
import pytest
import torch

from block_cases import DTYPES, check
from tree_cases import Case, pack, tree_mask

pytestmark = pytest.mark.gpu

FORMS = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "int8"), ("f16", "int8")]


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("length,n", [(0, 0), (0, 1), (1, 1), (1, 0), (3, 5), (2, 2), (31, 1), (32, 3), (33, 33), (128, 4), (129, 128), (130, 17), (257, 64),
                                      (700, 8), (1000, 300), (5000, 2)])
def test_every_length_of_a_run(gpu_lib, length, n, xt, fmt):
    Case(length + n, [(length, n)], xt=xt, fmt=fmt).check(gpu_lib)


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("n", [1, 2, 7, 16, 33, 63, 64, 65, 100, 130])
def test_every_size_of_a_tree(gpu_lib, n, xt, fmt):
    rng = np.random.default_rng(n)
    masks = [tree_mask(rng, n), tree_mask(rng, n)]
    Case(n, [(n + 200, n), (n, n)], xt=xt, fmt=fmt, masks=masks).check(gpu_lib)


@pytest.mark.parametrize("xt,fmt", FORMS)
def test_any_mask(gpu_lib, xt, fmt):
    """Rows with any bits, with none, with later tokens; more words than needed, and fewer (later tokens unseen)."""
    rng = np.random.default_rng(4)
    for n, words, window in ((5, 1, 0), (40, 3, 0), (70, 1, 0), (150, 4, 0), (40, 1, 20)):
        masks = [rng.random((n, n)) < 0.4, rng.random((n, n)) < 0.1, np.zeros((n, n), bool)]
        masks[1][3] = False
        for m in masks:
            m[:, words * 64:] = False
        Case(n, [(300, n), (n, n), (n, n)], xt=xt, fmt=fmt, masks=masks, words=words, window=window, sinks=3, H=4, KV=2).check(gpu_lib)


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 112, 128, 144, 192, 256])
def test_every_head_dimension(gpu_lib, D, xt, fmt):
    Case(D, [(1, 1), (0, 0), (77, 20), (300, 70)], D=D, xt=xt, fmt=fmt).check(gpu_lib)


@pytest.mark.parametrize("D", [8, 24, 40, 72, 136, 248])
def test_head_dimensions_of_whole_vectors(gpu_lib, D):
    Case(D, [(1, 1), (77, 3), (300, 40)], D=D).check(gpu_lib)


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("H,KV", [(1, 1), (4, 4), (3, 1), (12, 4), (40, 8), (17, 1), (64, 2), (300, 1)])
def test_every_head_layout(gpu_lib, H, KV, xt, fmt):
    Case(H, [(130, 9), (1, 1), (200, 2)], H=H, KV=KV, D=64, xt=xt, fmt=fmt).check(gpu_lib)


# rows of a request (tokens * group): each shape of a workgroup, whole and not
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [3, 4, 5, 8, 9, 16, 17, 31, 33, 64, 100])
def test_every_number_of_rows(gpu_lib, n, D):
    Case(n, [(400, n), (n + 1, n), (260, n)], H=4, KV=1, D=D).check(gpu_lib)


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("page", [1, 2, 4, 8, 32, 64, 256, 1024])
def test_every_page_size(gpu_lib, page, xt, fmt):
    if fmt == "int8" and page < 4:
        pytest.skip("an int8 cache has pages of four tokens or more")
    Case(page, [(1, 1), (31, 10), (500, 3), (0, 0), (1500, 40)], page=page, xt=xt, fmt=fmt, H=4, KV=2).check(gpu_lib)


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (31, 4), (32, 32), (33, 100), (100, 0), (128, 200), (1000, 5), (10 ** 6, 3), (0, 7)])
def test_windows_and_sinks(gpu_lib, window, sinks, xt, fmt):
    requests = [(0, 0), (1, 1), (40, 33), (131, 4), (2000, 50), (700, 300)]
    Case(window, requests, window=window, sinks=sinks, xt=xt, fmt=fmt, H=4, KV=2).check(gpu_lib)
    rng = np.random.default_rng(window)
    Case(window, requests[:5], window=window, sinks=sinks, xt=xt, fmt=fmt, H=4, KV=2, masks=[tree_mask(rng, n) for _, n in requests[:5]]).check(gpu_lib)


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("window,sinks", [(1, 1), (33, 4), (100, 130), (333, 40), (4096, 4)])
def test_single_tokens_with_sinks(gpu_lib, window, sinks, xt, fmt):
    lengths = [0, 1, 5, 33, 130, 700, 6000]
    c = Case(sinks, [(n, 1) for n in lengths], window=window, sinks=sinks, xt=xt, fmt=fmt)
    want, want_lse, omag, lmag = c.reference()
    out, lse = gpu_lib.paged_attention(c.q, c.k, c.v, c.table, c.lengths, scale=c.scale, window=window, sinks=sinks, return_lse=True, **c.kw)
    check(out, want, DTYPES[xt], omag, "out")
    check(lse, want_lse, torch.float32, lmag, "lse")


def test_sinks_do_nothing_without_a_window(gpu_lib):
    c = Case(1, [(50, 1), (700, 1)])
    a, b = (gpu_lib.paged_attention(c.q, c.k, c.v, c.table, c.lengths, sinks=s) for s in (0, 9))
    assert torch.equal(a, b)


@pytest.mark.parametrize("xt,fmt", FORMS)
def test_ragged_batches(gpu_lib, xt, fmt):
    rng = np.random.default_rng(7)
    for batch, most in ((2, 100), (65, 9), (300, 4)):
        requests = [(int(rng.integers(0, 400)), int(rng.integers(0, most))) for _ in range(batch)]
        Case(batch, requests, H=4, KV=1, D=64, xt=xt, fmt=fmt).check(gpu_lib)
    requests = [(int(rng.integers(0, 300)), 1) for _ in range(200)]
    Case(3, requests, H=40, KV=2, D=64, xt=xt, fmt=fmt, window=50, sinks=2).check(gpu_lib)


@pytest.mark.parametrize("xt,fmt", FORMS)
def test_long_contexts_in_pieces(gpu_lib, xt, fmt):
    Case(1, [(20000, 3), (129, 2), (9000, 5)], xt=xt, fmt=fmt, H=4, KV=2).check(gpu_lib)
    Case(2, [(9000, 90)], xt=xt, fmt=fmt, H=8, KV=2, width=4000).check(gpu_lib)
    Case(3, [(30000, 2)], xt=xt, fmt=fmt, H=4, KV=1, window=5000, sinks=300).check(gpu_lib)


@pytest.mark.parametrize("requests", [64, 65, 100, 513])  # counted by 64 lanes; from 513 on contexts stay whole
@pytest.mark.parametrize("xt,fmt", [("bf16", "bf16"), ("f16", "int8")])
def test_many_requests(gpu_lib, requests, xt, fmt):
    rng = np.random.default_rng(requests)
    ns = [int(n) for n in rng.integers(0, 6, requests)]
    lengths = [n + int(x) for n, x in zip(ns, rng.integers(0, 90, requests))]
    for b in (0, requests // 2, requests - 1):
        lengths[b] += 1500
    Case(requests, list(zip(lengths, ns)), H=4, KV=1, D=64, xt=xt, fmt=fmt, masks=[tree_mask(rng, n) if n else np.zeros((0, 0), bool) for n in ns]).check(gpu_lib)


@pytest.mark.parametrize("D", [48, 80, 128, 256])
@pytest.mark.parametrize("xt,fmt", [("bf16", "bf16"), ("f16", "int8")])
def test_many_rows_in_pieces(gpu_lib, D, xt, fmt):
    Case(D, [(2500, 131), (40, 0), (1500, 7)], H=32, KV=1, D=D, xt=xt, fmt=fmt, lead=1, tail=2).check(gpu_lib)  # 4512 rows


def test_rows_outside_the_requests_stay(gpu_lib):
    c = Case(5, [(40, 3), (0, 0), (200, 70)], lead=4, tail=9)
    before = torch.full_like(c.q, 7.0)
    out = before.clone()
    assert c.run(gpu_lib, out=out).data_ptr() == out.data_ptr()
    assert torch.equal(out[:4], before[:4]) and torch.equal(out[77:], before[77:])
    c.check(gpu_lib)
    c = Case(6, [(20000, 2)], H=4, KV=1, lead=1, tail=1)  # in pieces
    out = torch.full_like(c.q, 7.0)
    c.run(gpu_lib, out=out)
    assert (out[0] == 7).all() and (out[3] == 7).all()
    c.check(gpu_lib)


def test_lengths_and_tables_at_their_ends(gpu_lib):
    c = Case(7, [(500, 10), (-3, 2), (90, 4)], width=3)  # 500 and 90 tokens in a table of 48
    c.check(gpu_lib)
    c = Case(8, [(300, 20), (64, 64)])
    for i, bad in ((2, -1), (5, 10 ** 6), (18, 2 ** 31 - 1)):
        c.table64[0, i] = bad
    c.table64[1, 0] = -5
    c.table = torch.from_numpy(c.table64).cuda()
    c.check(gpu_lib)


def test_no_pages_no_tokens_no_requests(gpu_lib):
    c = Case(9, [(5, 2)])
    empty = c.k[:0]
    out, lse = gpu_lib.paged_tree_attention(c.q, empty, empty, c.table, c.lengths, c.starts, return_lse=True)
    assert (out == 0).all() and (lse == float("-inf")).all()
    assert gpu_lib.paged_tree_attention(c.q[:0], c.k, c.v, c.table, c.lengths, c.starts * 0).shape == (0, 8, 128)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert gpu_lib.paged_tree_attention(c.q, c.k, c.v, c.table[:0], none, c.starts[:1]).shape == c.q.shape


def test_unsorted_starts_stay_in_bounds(gpu_lib):
    c = Case(10, [(50, 3), (60, 4), (70, 5)])
    for s in ([0, 9, 2, 12], [12, 0, 5, 7], [-4, 100, 3, 2 ** 31 - 1], [5, 5, 5, 5]):
        gpu_lib.paged_tree_attention(c.q, c.k, c.v, c.table, c.lengths, torch.tensor(s, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    c.check(gpu_lib)


@pytest.mark.parametrize("xt,fmt", [("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_hidden_and_infinite_values(gpu_lib, xt, fmt, D):
    """NaN and infinite values, keys too, reach those rows alone that see their token."""
    rng = np.random.default_rng(D)
    n = 12
    for masks in (None, [tree_mask(rng, n), tree_mask(rng, n)]):
        c = Case(D, [(90, n), (n, n)], xt=xt, fmt=fmt, D=D, masks=masks, H=4, KV=2)
        page = c.page
        for b, (length, _) in enumerate(c.requests):
            for j, x, y in ((3, float("inf"), 1), (6, float("-inf"), D - 1), (9, float("nan"), 5)):
                t = length - n + j
                c.v[c.table64[b, t // page], :, t % page, y] = x
        t = 20
        c.v[c.table64[0, t // page], :, t % page, 2] = float("inf")  # in the prefix: all see it
        c.check(gpu_lib)
    c = Case(D, [(90, n)], xt=xt, fmt=fmt, D=D, H=4, KV=2)
    t = 90 - n + 8
    c.k[c.table64[0, t // 16], :, t % 16] = float("nan")
    out = c.run(gpu_lib)
    assert out[:8].isfinite().all() and out[8:].isnan().all()


def test_hidden_scales(gpu_lib):
    c = Case(11, [(90, 12)], xt="f16", fmt="int8")
    t = 90 - 12 + 8
    for s, x in (("k_scale", float("nan")), ("v_scale", float("inf"))):
        c.kw[s][c.table64[0, t // 16], :, t % 16] = x
    out = c.run(gpu_lib)
    assert out[:8].isfinite().all() and not out[8:].isfinite().any()


def test_strided_queries_scales_and_a_wide_table(gpu_lib):
    c = Case(12, [(50, 3), (200, 70)])
    wide = torch.full((c.tokens, 13, 128), float("nan"), dtype=c.q.dtype, device="cuda")
    wide[:, 2:10] = c.q
    c.q = wide[:, 2:10]
    big = torch.zeros(2, 40, dtype=torch.int32, device="cuda")
    big[:, :c.table.shape[1]] = c.table
    c.table = big[:, :c.table.shape[1]]
    c.check(gpu_lib)
    for scale in (0.0, 1.0, -0.1):
        Case(13, [(50, 3), (200, 7)], scale=scale).check(gpu_lib)


def test_a_run_equals_its_tokens_one_by_one(gpu_lib):
    """The same bits need not come out: both are within the bound of the same result."""
    c = Case(14, [(300, 20)])
    want, _, omag, _ = c.reference()
    lengths = torch.arange(281, 301, dtype=torch.int32, device="cuda")
    one = gpu_lib.paged_attention(c.q, c.k, c.v, c.table.expand(20, -1).contiguous(), lengths)
    check(one, want, torch.bfloat16, omag, "one by one")
    check(c.run(gpu_lib), want, torch.bfloat16, omag, "at once")


def test_stream_and_graph(gpu_lib):
    c = Case(15, [(5000, 3), (40, 2)], H=4, KV=1)  # two launches
    want = c.run(gpu_lib)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.stream(side):
        assert torch.equal(c.run(gpu_lib), want)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            c.run(gpu_lib, out=out)
    for i in range(3):
        c.lengths.copy_(torch.tensor([5000 - 700 * i, 40], dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.run(gpu_lib))


def test_cache_past_two_to_the_31_elements(gpu_lib):
    pages, KV, page, D = 66000, 4, 64, 128  # 2.16e9 elements
    k = torch.zeros(pages, KV, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.tensor([[65999, 0, 65998]], dtype=torch.int32, device="cuda")
    small = Case(16, [(180, 5)], H=8, KV=4, page=64)
    for i in range(3):
        k[table[0, i]], v[table[0, i]] = small.k[small.table[0, i]], small.v[small.table[0, i]]
    got = gpu_lib.paged_tree_attention(small.q, k, v, table, small.lengths, small.starts)
    assert torch.equal(got, small.run(gpu_lib))


def test_refusals(gpu_lib):
    rbp, c = gpu_lib, Case(17, [(50, 3), (60, 2)])
    tree = torch.from_numpy(pack(np.ones((5, 64), bool))).cuda()
    call = lambda **kw: rbp.paged_tree_attention(**{**dict(  # noqa: E731
        q=c.q, k_cache=c.k, v_cache=c.v, block_table=c.table, lengths=c.lengths, starts=c.starts, tree=tree), **kw})
    call()
    for bad in (dict(starts=None), dict(starts=c.starts[:2]), dict(starts=c.starts.long()), dict(tree=tree[:3]), dict(tree=tree.int()),
                dict(tree=tree[:, :0]), dict(lengths=c.lengths[:1]), dict(block_table=c.table[:1]), dict(q=c.q.half()), dict(q=c.q[:, :7]),
                dict(q=c.q[..., :64]), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(out=c.q[:2].clone()),
                dict(k_scale=c.q), dict(q=c.q.cpu()), dict(tree=tree.repeat(1, 1025)), dict(sinks=1 << 31)):
        with pytest.raises(rbp.OrbitError):
            call(**bad)
    one = dict(q=c.q[:2], k_cache=c.k, v_cache=c.v, block_table=c.table, lengths=c.lengths)
    rbp.paged_attention(**one, window=8, sinks=2)
    for bad in (dict(window=8, sinks=-2), dict(sinks=-2), dict(window=-8, sinks=2), dict(q=c.q[:3], window=8, sinks=2)):
        with pytest.raises(rbp.OrbitError):
            rbp.paged_attention(**{**one, **bad})
