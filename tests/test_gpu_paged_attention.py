"""Attention of one token over the paged cache against the fp64 definition.

Bounds: a score is a sum of D <= 256 products (depth D / 32 + 32 on the matrix
cores) and two scalings; dz bounds its error, so probabilities are within a
relative 2 dz + 2^-20 of their values (exponential, running maxima), and as
pairs of 16-bit operands within 2^-16 (bfloat16) or 2^-20 (float16, of the
largest).  Sums over L tokens add (L / 128 + 40) E.  The output's error is
that times sum p |v| / sum p.
"""
import numpy as np
import pytest
import torch

import oracle
from block_cases import DTYPES, E, check, draw, f64

pytestmark = pytest.mark.gpu

PAIR = {"bf16": 2.0 ** -15, "f16": 2.0 ** -19, "int8": 2.0 ** -19}


def _make(rng, lengths, H, KV, D, page, xt, fmt, spare=3, width=None, std=1.0):
    need = [max(0, -(-n // page)) for n in lengths]
    width = width or max(1, max(need, default=1))
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = rng.integers(0, pages, (len(lengths), width)).astype(np.int32)  # what lies past a request's pages is anything
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n][:width]
        at += n
    q, q64 = draw(rng, (len(lengths), H, D), DTYPES[xt], 2.0)
    kw = {}
    if fmt == "int8":
        k, v = (torch.from_numpy(rng.integers(-127, 128, (pages, KV, page, D)).astype(np.int8)).cuda() for _ in "kv")
        scales = [torch.from_numpy((std * rng.uniform(0.5, 1.5, (pages, KV, page)) / 73).astype(np.float16)).cuda() for _ in "kv"]
        kw = dict(k_scale=scales[0], v_scale=scales[1])
        k64, v64 = (f64(t) * f64(s)[..., None] for t, s in zip((k, v), scales))
    else:
        k, k64 = draw(rng, (pages, KV, page, D), DTYPES[fmt], std)
        v, v64 = draw(rng, (pages, KV, page, D), DTYPES[fmt], std)
    return q, k, v, torch.from_numpy(table).cuda(), kw, (q64, k64, v64, table)


def _bound(q64, k64, v64, table, lengths, sm, window, fmt, D):
    """(output's, lse's) float32 error by the bounds above."""
    zero = lambda t: np.where(np.isfinite(t), t, 0.0)  # noqa: E731
    av, _ = oracle.paged_attention(q64, zero(k64), np.abs(zero(v64)), table, lengths, sm, window)
    dz = (D / 32 + 36) * E * abs(sm) * (np.abs(q64).sum(-1) * 1.0) * np.abs(zero(k64)).max()
    # sum |q||k| <= sum |q| max |k|; the exponential turns dz into a relative error
    rel = 2 * dz + PAIR[fmt] + (min(max(lengths, default=1), table.shape[1] * k64.shape[2]) / 128 + 60) * E
    return rel[..., None] * av, rel


def _run(rbp, seed, lengths, H=8, KV=2, D=128, page=16, xt="bf16", fmt="bf16", window=0, scale=None, width=None, std=1.0,
         strided_q=False):
    rng = np.random.default_rng(seed)
    q, k, v, table, kw, (q64, k64, v64, t64) = _make(rng, lengths, H, KV, D, page, xt, fmt, width=width, std=std)
    if strided_q:  # heads of a fused projection's output
        wide = torch.full((len(lengths), H + 3, D), float("nan"), dtype=q.dtype, device="cuda")
        wide[:, 1:1 + H] = q
        q = wide[:, 1:1 + H]
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = rbp.paged_attention(q, k, v, table, ln, scale=scale, window=window, return_lse=True, **kw)
    sm = D ** -0.5 if scale is None else scale
    ref, ref_lse = oracle.paged_attention(q64, k64, v64, t64, lengths, sm, window)
    o_mag, l_mag = _bound(q64, k64, v64, t64, lengths, sm, window, fmt, D)
    check(out, ref, DTYPES[xt], o_mag, "out")
    check(lse, ref_lse, torch.float32, l_mag + 4 * E * np.abs(np.where(np.isfinite(ref_lse), ref_lse, 0)), "lse")
    alone = rbp.paged_attention(q, k, v, table, ln, scale=scale, window=window, **kw)
    assert torch.equal(alone, out)


FORMS = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "int8"), ("f16", "int8")]


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 257, 1000, 5000])
def test_every_length(gpu_lib, n, xt, fmt):
    _run(gpu_lib, n, [n], xt=xt, fmt=fmt)


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 240, 256])
def test_every_head_dimension(gpu_lib, D, xt, fmt):
    _run(gpu_lib, D, [1, 0, 77, 300], D=D, xt=xt, fmt=fmt)


@pytest.mark.parametrize("D", [8, 24, 40, 72, 136, 248])
def test_head_dimensions_of_whole_vectors(gpu_lib, D):
    _run(gpu_lib, D, [1, 0, 77, 300], D=D)


@pytest.mark.parametrize("H,KV", [(1, 1), (4, 4), (3, 1), (12, 4), (40, 8), (16, 1), (17, 1), (40, 2), (64, 2), (128, 1)])
@pytest.mark.parametrize("xt,fmt", FORMS)
def test_every_head_layout(gpu_lib, H, KV, xt, fmt):
    _run(gpu_lib, H, [130, 1, 600], H=H, KV=KV, D=64, xt=xt, fmt=fmt)


@pytest.mark.parametrize("page", [1, 2, 4, 8, 32, 64, 256, 1024])
@pytest.mark.parametrize("xt,fmt", FORMS)
def test_every_page_size(gpu_lib, page, xt, fmt):
    if fmt == "int8" and page < 4:
        pytest.skip("scales of an int8 cache are read by fours")
    _run(gpu_lib, page, [1, 31, 500, 0, 1500], page=page, xt=xt, fmt=fmt)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 128, 1000, 10 ** 6])
@pytest.mark.parametrize("xt,fmt", FORMS)
def test_every_window(gpu_lib, window, xt, fmt):
    _run(gpu_lib, window, [0, 1, 32, 33, 100, 131, 2000], window=window, xt=xt, fmt=fmt)


@pytest.mark.parametrize("xt,fmt", FORMS)
def test_ragged_batches(gpu_lib, xt, fmt):
    rng = np.random.default_rng(7)
    for batch in (2, 33, 300):
        _run(gpu_lib, batch, [int(x) for x in rng.integers(0, 400, batch)], H=4, KV=1, D=64, xt=xt, fmt=fmt)


def test_strided_queries_and_scales(gpu_lib):
    _run(gpu_lib, 1, [50, 200], strided_q=True)
    for scale in (0.0, 1.0, -0.1):
        _run(gpu_lib, 2, [50, 200], scale=scale)


@pytest.mark.parametrize("xt", ["bf16", "f16"])
def test_scales_of_every_size_in_an_int8_cache(gpu_lib, xt):
    # values of 1e-4 and of 1e3 keep their accuracy although products run in float16
    for std in (1e-4, 1e3):
        rng = np.random.default_rng(3)
        q, k, v, table, kw, (q64, k64, v64, t64) = _make(rng, [300, 40], 8, 2, 128, 16, xt, "int8")
        kw["v_scale"] = (kw["v_scale"].float() * std).half()
        v64 = f64(v) * f64(kw["v_scale"])[..., None]
        ln = torch.tensor([300, 40], dtype=torch.int32, device="cuda")
        out = gpu_lib.paged_attention(q, k, v, table, ln, **kw)
        ref, _ = oracle.paged_attention(q64, k64, v64, t64, [300, 40], 128 ** -0.5)
        mag, _ = _bound(q64, k64, v64, t64, [300, 40], 128 ** -0.5, 0, "int8", 128)
        check(out, ref, DTYPES[xt], mag, f"values of {std}")
    for qstd in (1e-6, 1e4):  # and queries past float16's range either way
        q2 = (q.float() * qstd).to(q.dtype)
        got = gpu_lib.paged_attention(q2, k, v, table, ln, scale=128 ** -0.5 / qstd, **kw)
        ref, _ = oracle.paged_attention(f64(q2), k64, v64, t64, [300, 40], 128 ** -0.5 / qstd)
        mag, _ = _bound(f64(q2), k64, v64, t64, [300, 40], 128 ** -0.5 / qstd, 0, "int8", 128)
        check(got, ref, DTYPES[xt], mag, f"queries of {qstd}")


@pytest.mark.parametrize("xt,fmt", FORMS)
def test_what_lies_outside_the_seen_tokens_is_never_used(gpu_lib, xt, fmt):
    rng = np.random.default_rng(5)
    lengths, page = [1, 0, 45, 200, 515], 16
    q, k, v, table, kw, (q64, k64, v64, t64) = _make(rng, lengths, 8, 2, 64, page, xt, fmt)
    seen = np.zeros((k.shape[0], page), dtype=bool)
    for b, n in enumerate(lengths):
        for t in range(max(0, n - 100), n):
            seen[t64[b, t // page], t % page] = True
    hide = torch.from_numpy(~seen).cuda()
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    good = gpu_lib.paged_attention(q, k, v, table, ln, window=100, return_lse=True, **kw)
    for bad in (float("nan"), float("inf"), float("-inf")):
        if fmt == "int8":
            kw = {n: torch.where(hide[:, None, :], torch.tensor(bad, dtype=torch.float16, device="cuda"), s) for n, s in kw.items()}
        else:
            k, v = (torch.where(hide[:, None, :, None], torch.tensor(bad, dtype=t.dtype, device="cuda"), t) for t in (k, v))
        got = gpu_lib.paged_attention(q, k, v, table, ln, window=100, return_lse=True, **kw)
        assert torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])


@pytest.mark.parametrize("xt,fmt", FORMS)
def test_table_entries_and_lengths_outside(gpu_lib, xt, fmt):
    rng = np.random.default_rng(6)
    lengths = [100, 64, 300, 40]
    q, k, v, table, kw, (q64, k64, v64, t64) = _make(rng, lengths, 4, 2, 64, 16, xt, fmt)
    t64 = t64.copy()
    t64[0, 2] = -1
    t64[0, 4] = k.shape[0]
    t64[1, :] = 2 ** 31 - 1  # nothing of this request is in the cache
    t64[3, 0] = -2 ** 31
    lengths = [100, 64, 10 ** 9, -5]
    out, lse = gpu_lib.paged_attention(q, k, v, torch.from_numpy(t64).cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                                       return_lse=True, **kw)
    ref, ref_lse = oracle.paged_attention(q64, k64, v64, t64, lengths, 0.125)
    o_mag, l_mag = _bound(q64, k64, v64, t64, lengths, 0.125, 0, fmt, 64)
    check(out, ref, DTYPES[xt], o_mag)
    check(lse, ref_lse, torch.float32, l_mag)
    assert (out[1] == 0).all() and (lse[1] == float("-inf")).all() and (out[3] == 0).all()


def test_infinite_and_nan_tokens_that_are_seen(gpu_lib):
    rng = np.random.default_rng(8)
    q, k, v, table, kw, (_, _, _, t64) = _make(rng, [300, 300, 300], 4, 1, 64, 16, "bf16", "bf16")
    good = gpu_lib.paged_attention(q, k, v, table, torch.full((3,), 300, dtype=torch.int32, device="cuda"))
    v[t64[1, 4], 0, 3, 7] = float("nan")
    k[t64[2, 9], 0, 2, 1] = float("nan")
    got = gpu_lib.paged_attention(q, k, v, table, torch.full((3,), 300, dtype=torch.int32, device="cuda"))
    assert torch.equal(got[0], good[0])
    assert torch.isnan(got[1, :, 7]).all() and torch.equal(got[1, :, :7], good[1, :, :7])
    assert torch.isnan(got[2]).all()


def test_large_scores_do_not_overflow(gpu_lib):
    _run(gpu_lib, 9, [700, 33], std=1.0, scale=30.0)


def test_parts_of_a_context_join_by_their_lse(gpu_lib):
    rng = np.random.default_rng(10)
    q, k, v, table, kw, _ = _make(rng, [640], 8, 2, 64, 32, "bf16", "bf16")
    full = gpu_lib.paged_attention(q, k, v, table, torch.tensor([640], dtype=torch.int32, device="cuda"))
    n = torch.tensor([320], dtype=torch.int32, device="cuda")
    a, la = gpu_lib.paged_attention(q, k, v, table[:, :10], n, return_lse=True)
    b, lb = gpu_lib.paged_attention(q, k, v, table[:, 10:], n, return_lse=True)
    w = torch.softmax(torch.stack([la, lb]), 0)[..., None]
    joined = w[0] * a.float() + w[1] * b.float()
    assert (joined - full.float()).abs().max() <= 3 * 2.0 ** -8 * full.float().abs().max()


def test_a_cache_of_more_than_two_to_the_thirty_one_bytes(gpu_lib):
    # rows past 2^31 elements and 2^32 bytes: the last pages of a 5 GiB cache
    pages, KV, page, D = 10240, 8, 256, 128
    k = torch.zeros(pages, KV, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    rng = np.random.default_rng(11)
    last = [pages - 1, pages - 2, 5, pages // 2 + 1]
    small, s64 = draw(rng, (2, 4, KV, page, D), torch.bfloat16)
    for i, p in enumerate(last):
        k[p], v[p] = small[0, i], small[1, i]
    q, q64 = draw(rng, (1, 16, D), torch.bfloat16, 2.0)
    table = torch.tensor([last], dtype=torch.int32, device="cuda")
    out = gpu_lib.paged_attention(q, k, v, table, torch.tensor([1000], dtype=torch.int32, device="cuda"))
    t4 = np.array([[0, 1, 2, 3]])
    ref, _ = oracle.paged_attention(q64, s64[0], s64[1], t4, [1000], D ** -0.5)
    mag, _ = _bound(q64, s64[0], s64[1], t4, [1000], D ** -0.5, 0, "bf16", D)
    check(out, ref, torch.bfloat16, mag)
    # and the append and the read reach them
    slot = torch.tensor([(pages - 1) * page + 255, 3], device="cuda")
    new, n64 = draw(rng, (2, KV, D), torch.bfloat16)
    gpu_lib.kv_append(new, new, k, v, slot)
    assert torch.equal(k[pages - 1, :, 255], new[0]) and torch.equal(v[0, :, 3], new[1])
    back, _ = gpu_lib.kv_read(k, v, slot)
    assert torch.equal(back, new)


def test_after_an_append(gpu_lib):
    """Append into the int8 cache, attend with the rotated queries: q . k of the rotated pair is the plain one's."""
    rng = np.random.default_rng(12)
    T, H, KV, D, page = 200, 8, 2, 128, 16
    k, k64 = draw(rng, (T, KV, D), torch.bfloat16)
    v, v64 = draw(rng, (T, KV, D), torch.bfloat16)
    q, q64 = draw(rng, (T, H, D), torch.bfloat16)
    pages = T // page + 2
    kc, vc = (torch.zeros(pages, KV, page, D, dtype=torch.int8, device="cuda") for _ in "kv")
    sc = {n: torch.zeros(pages, KV, page, dtype=torch.float16, device="cuda") for n in ("k_scale", "v_scale")}
    q2 = gpu_lib.kv_append(k, v, kc, vc, torch.arange(T, device="cuda"), q=q, hadamard=True, **sc)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    out = gpu_lib.paged_attention(q2[-1:], kc, vc, table, torch.tensor([T], dtype=torch.int32, device="cuda"), **sc)
    kv = [np.concatenate([t, np.zeros((pages * page - T, KV, D))]).reshape(pages, page, KV, D).transpose(0, 2, 1, 3) for t in (k64, v64)]
    ref, _ = oracle.paged_attention(q64[-1:], *kv, np.arange(pages)[None], [T], D ** -0.5)
    # codes are within half a step, 1 / 254 of a head's largest (~ 2.5 to 4 of N(0, 1)): ~1 % of the values
    assert np.linalg.norm(f64(out) - ref) <= 0.03 * np.linalg.norm(ref)


def test_another_stream_and_a_graph(gpu_lib):
    rng = np.random.default_rng(13)
    lengths = [700, 3, 0, 4000]
    q, k, v, table, kw, _ = _make(rng, lengths, 8, 2, 128, 16, "bf16", "bf16")
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    first = gpu_lib.paged_attention(q, k, v, table, ln)
    out = torch.empty_like(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gpu_lib.paged_attention(q, k, v, table, ln, out=out)
    side.synchronize()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.paged_attention(q, k, v, table, ln, out=out)
    for step in range(3):
        ln.copy_(torch.tensor([[1, 2, 3, 4], [700, 0, 9, 3999], [64, 64, 64, 64]][step], dtype=torch.int32))
        ln.clamp_(max=int(table.shape[1]) * 16)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, gpu_lib.paged_attention(q, k, v, table, ln))


def test_refusals(gpu_lib):
    rbp = gpu_lib
    q = torch.zeros(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    kc = torch.zeros(3, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
    k8, s8 = kc.to(torch.int8), torch.ones(3, 2, 16, device="cuda", dtype=torch.float16)
    table = torch.zeros(2, 3, device="cuda", dtype=torch.int32)
    ln = torch.ones(2, device="cuda", dtype=torch.int32)
    rbp.paged_attention(q, kc, kc, table, ln)
    bad = [
        lambda: rbp.paged_attention(q.float(), kc, kc, table, ln),
        lambda: rbp.paged_attention(q.half(), kc, kc, table, ln),
        lambda: rbp.paged_attention(q, kc.half(), kc.half(), table, ln),
        lambda: rbp.paged_attention(q[:, :3], kc, kc, table, ln),       # 3 query heads on 2
        lambda: rbp.paged_attention(q[:, :, :32], kc, kc, table, ln),
        lambda: rbp.paged_attention(q, kc, kc[:2], table, ln),
        lambda: rbp.paged_attention(q, kc, kc, table.long(), ln),
        lambda: rbp.paged_attention(q, kc, kc, table[:1], ln),
        lambda: rbp.paged_attention(q, kc, kc, table, ln.long()),
        lambda: rbp.paged_attention(q, kc, kc, table, ln[:1]),
        lambda: rbp.paged_attention(q, kc, kc, table, ln, window=-1),
        lambda: rbp.paged_attention(q, kc, kc, table, ln, scale=float("inf")),
        lambda: rbp.paged_attention(q, kc, kc, table, ln, out=q.float()),
        lambda: rbp.paged_attention(q, k8, k8, table, ln),
        lambda: rbp.paged_attention(q, k8, k8, table, ln, k_scale=s8, v_scale=s8[:2]),
        lambda: rbp.paged_attention(q, kc, kc, table, ln, k_scale=s8, v_scale=s8),
        lambda: rbp.paged_attention(q.cpu(), kc, kc, table, ln),
        lambda: rbp.paged_attention(q, kc, kc, table.cpu(), ln),
    ]
    for f in bad:
        with pytest.raises(rbp.OrbitError):
            f()
    wide = torch.zeros(2, 4, 66, device="cuda", dtype=torch.bfloat16)[:, :, 1:65]  # heads that are not 16-byte aligned
    with pytest.raises(rbp.OrbitError):
        rbp.paged_attention(wide, kc, kc, table, ln)
