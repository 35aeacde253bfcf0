"""Low-rank adapters of many requests (adapter_add) against the fp64 definition.

Bounds: A x is summed in chains of at most K / 32 steps of 32 products and at
most 64 partial sums: depth <= K / 32 + 96; B v has at most 128 terms.  The
factor v may enter the second product as a pair of 16-bit numbers: bfloat16
pairs keep 2^-16 of it, float16 pairs 2^-21.
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from block_cases import DTYPES, E, check, draw, strided
from parity import as_f64, to_dev

pytestmark = pytest.mark.gpu

PAIR = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -21}


def _mag(y, x, A, B, ids, scale, ranks, xt):
    """What float32 errors of the two products scale with."""
    K, R = A.shape[2], A.shape[1]
    mag = 4 * E * np.abs(y)
    for m, a in enumerate(ids):
        if 0 <= a < len(A):
            r = R if ranks is None else int(np.clip(ranks[a], 0, R))
            s = 1.0 if scale is None else abs(float(scale[a]))
            if r:
                dv = (K / 32 + 96) * E * (np.abs(A[a, :r]) @ np.abs(x[m])) + PAIR[xt] * np.abs(A[a, :r] @ x[m])
                mag[m] += s * (np.abs(B[a, :, :r]) @ (dv + 136 * E * np.abs(A[a, :r] @ x[m])))
    return mag


def _run(rbp, seed, M, K, N, R, L, ids, xt="bf16", yt="bf16", ranks=None, scale=True, pad=0, inplace=False, lead=0):
    rng = np.random.default_rng(seed)
    xt, yt = DTYPES[xt], DTYPES[yt]
    x, x64 = draw(rng, (M, K), xt)
    y, y64 = draw(rng, (M, N), yt)
    A, A64 = draw(rng, (L, R, K), xt, K ** -0.5)
    B, B64 = draw(rng, (L, N, R), xt, 0.5)
    kw, s = {}, None
    if scale:
        s = (rng.uniform(0.25, 4.0, L)).astype(np.float32)
        kw["scale"] = torch.from_numpy(s).cuda()
    if ranks is not None:
        kw["ranks"] = torch.tensor(ranks, dtype=torch.int32, device="cuda")
        for a, r in enumerate(ranks):  # what lies past an adapter's rank is never used
            A[a, max(0, r):] = float("nan")
            B[a, :, max(0, r):] = float("inf")
    if pad:
        x, y = strided(x, pad), strided(y, pad, lead)
    if inplace:
        kw["out"] = y
    got = rbp.adapter_add(y, x, A, B, torch.tensor(ids, dtype=torch.int32, device="cuda"), **kw)
    if inplace:
        assert got.data_ptr() == y.data_ptr()
    ref = oracle.adapter_add(y64, x64, A64, B64, ids, s, ranks)
    check(got, ref, yt, _mag(y64, x64, A64, B64, ids, s, ranks, xt))
    return got


def _mixed(rng, M, L):
    """A few long runs, single tokens, tokens without an adapter."""
    ids = []
    while len(ids) < M:
        ids += [int(rng.integers(-1, L))] * int(rng.choice([1, 1, 2, 5, 17, 40]))
    return ids[:M]


@pytest.mark.parametrize("M", [0, 1, 2, 3, 15, 16, 17, 63, 64, 65, 130, 300, 1025])
@pytest.mark.parametrize("xt", ["bf16", "f16"])
def test_every_number_of_tokens(gpu_lib, M, xt):
    rng = np.random.default_rng(M)
    _run(gpu_lib, M, M, 256, 200, 16, 7, _mixed(rng, M, 7), xt=xt, ranks=[16, 1, 0, 7, 8, 15, 9])


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 96, 128])
@pytest.mark.parametrize("M", [5, 300])
def test_every_rank(gpu_lib, R, M):
    rng = np.random.default_rng(R)
    _run(gpu_lib, R, M, 384, 136, R, 3, _mixed(rng, M, 3), xt="f16", yt="f32", ranks=[R, R - 3, 1])


@pytest.mark.parametrize("K", [8, 16, 24, 40, 64, 120, 136, 264, 520, 1000, 4096, 12288])
@pytest.mark.parametrize("M", [4, 150])
def test_every_inner_length(gpu_lib, K, M):
    rng = np.random.default_rng(K)
    _run(gpu_lib, K, M, K, 72, 16, 4, _mixed(rng, M, 4))


@pytest.mark.parametrize("N", [0, 1, 3, 8, 12, 63, 64, 65, 255, 256, 257, 260, 1000, 4100])
@pytest.mark.parametrize("yt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [3, 100])
def test_every_width(gpu_lib, N, yt, M):
    rng = np.random.default_rng(N)
    _run(gpu_lib, N, M, 128, N, 8, 5, _mixed(rng, M, 5), yt=yt)


@pytest.mark.parametrize("order", ["one", "none", "each", "alternating", "blocks", "outside"])
@pytest.mark.parametrize("M", [33, 129, 700])
def test_every_order_of_requests(gpu_lib, order, M):
    L = 40
    ids = {"one": [3] * M, "none": [-1] * M, "each": [m % L for m in range(M)], "alternating": [m % 2 for m in range(M)],
           "blocks": [m // 16 % L for m in range(M)],
           "outside": [(-2, L, 2 ** 31 - 1, -2 ** 31, 5)[m % 5] for m in range(M)]}[order]
    _run(gpu_lib, M, M, 320, 264, 32, L, ids, xt="f16")


@pytest.mark.parametrize("M", [2047, 2049, 2500, 4113])
@pytest.mark.parametrize("R,K,xt", [(16, 200, "bf16"), (24, 1032, "f16"), (64, 520, "bf16"), (104, 136, "f16")])
def test_many_tokens(gpu_lib, M, R, K, xt):
    rng = np.random.default_rng(M + R)
    L, N = 70, 72
    ranks = [int(r) for r in rng.integers(0, R + 1, L)]
    long_runs = sorted(int(i) for i in rng.integers(-1, 5, M - 200))
    ids = long_runs + [int(i) for i in rng.integers(-1, L, 200)]  # prompts, then single tokens
    _run(gpu_lib, M, M, K, N, R, L, ids, xt=xt, ranks=ranks)


def test_many_tokens_into_wide_rows(gpu_lib):
    rng = np.random.default_rng(1)
    for N in (1001, 2052, 4096):  # tiles of 64 rows and of 16; single elements, fours, eights
        for order in (sorted(int(i) for i in rng.integers(-1, 3, 2100)), [m % 33 for m in range(2100)]):
            _run(gpu_lib, N, 2100, 64, N, 16, 33, order, ranks=[16 - i % 9 for i in range(33)])


def test_no_scale_no_ranks_no_adapters(gpu_lib):
    _run(gpu_lib, 1, 20, 128, 64, 8, 2, [0, 1] * 10, scale=False)
    x = torch.ones(4, 128, device="cuda", dtype=torch.bfloat16)
    y = torch.randn(4, 64, device="cuda")
    empty = torch.zeros(0, 8, 128, device="cuda", dtype=torch.bfloat16), torch.zeros(0, 64, 8, device="cuda", dtype=torch.bfloat16)
    got = gpu_lib.adapter_add(y, x, *empty, torch.zeros(4, device="cuda", dtype=torch.int32))
    assert torch.equal(got, y)


@pytest.mark.parametrize("M", [9, 200])
def test_strided_and_in_place(gpu_lib, M):
    rng = np.random.default_rng(8)
    ids = _mixed(rng, M, 4)
    for pad, lead in ((8, 0), (16, 8), (8, 1), (8, 3), (8, 4)):
        _run(gpu_lib, pad, M, 256, 248, 16, 4, ids, pad=pad, lead=lead)
        _run(gpu_lib, pad, M, 256, 248, 16, 4, ids, pad=pad, lead=lead, yt="f32", inplace=True)


@pytest.mark.parametrize("M", [24, 200])
@pytest.mark.parametrize("xt", ["bf16", "f16"])
def test_a_broken_adapter_or_token_stays_alone(gpu_lib, M, xt):
    # requests of one batch share tiles: one of NaN weights, one with an
    # infinite token, must leave the others' bits as they are
    rng = np.random.default_rng(3)
    t = DTYPES[xt]
    x, _ = draw(rng, (M, 256), t)
    y, _ = draw(rng, (M, 128), torch.float32)
    A, _ = draw(rng, (4, 16, 256), t, 1 / 16)
    B, _ = draw(rng, (4, 128, 16), t)
    ids = torch.tensor([m % 5 - 1 for m in range(M)], dtype=torch.int32, device="cuda")
    good = gpu_lib.adapter_add(y, x, A, B, ids)
    A2, B2, x2 = A.clone(), B.clone(), x.clone()
    A2[2] = float("nan")
    B2[1, :, 3] = float("inf")
    x2[8] = float("inf")  # token 8: adapter 2
    got = gpu_lib.adapter_add(y, x2, A2, B2, ids)
    keep = (ids != 2) & (ids != 1)
    assert torch.equal(got[keep], good[keep])
    assert torch.isnan(got[ids == 2]).all() and not torch.isfinite(got[ids == 1]).any()


@pytest.mark.parametrize("M", [400, 1100, 2100])
@pytest.mark.parametrize("run", [1, 3, 9, 50])
def test_a_broken_adapter_stays_alone_among_many_tokens(gpu_lib, M, run):
    # runs of `run` tokens of each of 13 adapters: tiles of one, a few and many
    # of them, borders inside tiles; R 40: three blocks of ranks, one not whole
    rng = np.random.default_rng(M + run)
    L, R, t = 13, 40, torch.float16
    x, _ = draw(rng, (M, 264), t)
    y, _ = draw(rng, (M, 136), torch.float32)
    A, _ = draw(rng, (L, R, 264), t, 1 / 16)
    B, _ = draw(rng, (L, 136, R), t)
    ids = torch.tensor([m // run % (L + 1) - 1 for m in range(M)], dtype=torch.int32, device="cuda")
    good = gpu_lib.adapter_add(y, x, A, B, ids)
    A2, B2, x2 = A.clone(), B.clone(), x.clone()
    A2[2] = float("inf")
    A2[5] = float("nan")
    B2[7] = float("nan")
    x2[ids == 9] = float("nan")
    got = gpu_lib.adapter_add(y, x2, A2, B2, ids)
    bad = (ids == 2) | (ids == 5) | (ids == 7) | (ids == 9)
    assert torch.equal(got[~bad], good[~bad])
    assert torch.isfinite(good).all() and not torch.isfinite(got[bad]).any()


@pytest.mark.parametrize("M", [10, 150])
def test_large_values_do_not_overflow_between_the_products(gpu_lib, M):
    # A x reaches 4e6, past float16's largest number; B brings it back
    rng = np.random.default_rng(4)
    x, x64 = draw(rng, (M, 512), torch.float16, 2000.0)
    A, A64 = draw(rng, (1, 8, 512), torch.float16, 100.0)
    B, B64 = draw(rng, (1, 64, 8), torch.float16, 1e-4)
    y, y64 = draw(rng, (M, 64), torch.float32)
    ids = [0] * M
    got = gpu_lib.adapter_add(y, x, A, B, torch.zeros(M, dtype=torch.int32, device="cuda"))
    ref = oracle.adapter_add(y64, x64, A64, B64, ids)
    check(got, ref, torch.float32, _mag(y64, x64, A64, B64, ids, None, None, torch.float16))


def test_beside_a_rotated_quantized_projection(gpu_lib):
    """The adapter absorbed once (A Pi^T) reads the x' that int8_linear reads."""
    rbp = gpu_lib
    inp = synth.make(3, M=48, N=256)
    rot = rbp.Rotation(inp["perm"], inp["signs"], inp["h"])
    X, W = to_dev(inp["X"]), to_dev(inp["W"])
    K = X.shape[1]
    rng = np.random.default_rng(5)
    A, A64 = draw(rng, (3, 16, K), torch.bfloat16, K ** -0.5)
    B, B64 = draw(rng, (3, 256, 16), torch.float16, 0.5)
    ids = [m % 4 - 1 for m in range(48)]
    xr = rbp.rotate(rot, X)
    absorbed = rbp.rotate(rot, A.reshape(-1, K)).reshape(3, 16, K)
    q, sc = rbp.int8_pack_weights(rot, W)
    y = rbp.int8_linear(xr, q, sc, out_dtype=torch.float32)
    got = rbp.adapter_add(y, xr, absorbed, B, torch.tensor(ids, dtype=torch.int32, device="cuda"))
    ref = oracle.adapter_add(y.double().cpu().numpy(), as_f64(inp["X"]), A64, B64, ids)
    delta, want = got.double().cpu().numpy() - y.double().cpu().numpy(), ref - y.double().cpu().numpy()
    # x' and A Pi^T are each rounded to float16 (2^-11): two such errors, independent over K terms
    assert np.linalg.norm(delta - want) <= 2e-3 * np.linalg.norm(want)


def test_repeats_are_identical_on_another_stream_and_in_a_graph(gpu_lib):
    rng = np.random.default_rng(6)
    for M in (16, 600):
        x, _ = draw(rng, (M, 1024), torch.float16)
        y, _ = draw(rng, (M, 512), torch.bfloat16)
        A, _ = draw(rng, (5, 32, 1024), torch.float16, 1 / 32)
        B, _ = draw(rng, (5, 512, 32), torch.float16)
        ids = torch.tensor(_mixed(rng, M, 5), dtype=torch.int32, device="cuda")
        first = gpu_lib.adapter_add(y, x, A, B, ids)
        out = torch.empty_like(y)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = gpu_lib.adapter_add(y, x, A, B, ids, out=out)
        side.synchronize()
        assert torch.equal(first, again)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gpu_lib.adapter_add(y, x, A, B, ids, out=out)
        for seed in range(3):
            x.copy_(draw(np.random.default_rng(seed), (M, 1024), torch.float16)[0])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, gpu_lib.adapter_add(y, x, A, B, ids))


def test_refusals(gpu_lib):
    rbp = gpu_lib
    x = torch.zeros(4, 128, device="cuda", dtype=torch.bfloat16)
    y = torch.zeros(4, 64, device="cuda")
    A = torch.zeros(2, 8, 128, device="cuda", dtype=torch.bfloat16)
    B = torch.zeros(2, 64, 8, device="cuda", dtype=torch.bfloat16)
    ids = torch.zeros(4, device="cuda", dtype=torch.int32)
    rbp.adapter_add(y, x, A, B, ids)
    bad = [
        lambda: rbp.adapter_add(y, x.float(), A, B, ids),
        lambda: rbp.adapter_add(y, x.half(), A, B, ids),
        lambda: rbp.adapter_add(y[:3], x, A, B, ids),
        lambda: rbp.adapter_add(y, x, A[:1], B, ids),
        lambda: rbp.adapter_add(y, x, A.transpose(1, 2), B, ids),
        lambda: rbp.adapter_add(y, x, A, B[:, :32], ids),
        lambda: rbp.adapter_add(y, x, A, B, ids.long()),
        lambda: rbp.adapter_add(y, x, A, B, ids[:2]),
        lambda: rbp.adapter_add(y, x, A, B, ids.cpu()),
        lambda: rbp.adapter_add(y, x, A, B, ids, scale=torch.ones(3, device="cuda")),
        lambda: rbp.adapter_add(y, x, A, B, ids, ranks=torch.ones(2, device="cuda")),
        lambda: rbp.adapter_add(y, x, A, B, ids, out=y.bfloat16()),
        lambda: rbp.adapter_add(y, x, A, B, ids, out=y[:1].expand(4, 64)),
        lambda: rbp.adapter_add(y, x, A[:, :4].contiguous(), B[:, :, :4].contiguous(), ids),  # rank not a multiple of 8
        lambda: rbp.adapter_add(y, x[:, :124], A[:, :, :124].contiguous(), B, ids),           # K not a multiple of 8
        lambda: rbp.adapter_add(y, strided(x, 8, 4), A, B, ids),                              # x's rows not 16-byte aligned
        lambda: rbp.adapter_add(y.int(), x, A, B, ids),
    ]
    for f in bad:
        with pytest.raises(rbp.OrbitError):
            f()
