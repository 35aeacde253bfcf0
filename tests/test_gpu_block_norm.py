"""Norms around a residual sum (block_norm) against the fp64 definition.

Bounds: a row of D <= 16384 is summed by at most 16 serial terms per lane and
16 pairwise steps (lanes, waves): depth <= 40, so mean and mean square are
within 40 E of their magnitudes, the inverse root within 20 E + 4 E, and the
chain of products around them adds less than 10 E: 64 E of the magnitudes
below covers both norms.
"""
import numpy as np
import pytest
import torch

import oracle
from block_cases import DTYPES, E, check, draw, strided

pytestmark = pytest.mark.gpu


def _mags(x, b, o):
    """Magnitudes of r and y that float32 errors scale with."""
    row = lambda v: np.abs(v).mean(axis=-1, keepdims=True)  # noqa: E731
    r, _ = oracle.block_norm(x, b, **o)
    gain = np.ones(x.shape)
    if b is not None:
        if o.get("post"):
            inv = 1.0 / np.sqrt(np.var(b, -1, keepdims=True) * (o["post"] == "layer")
                                + (b * b).mean(-1, keepdims=True) * (o["post"] == "rms") + o.get("eps", 1e-6))
            b_mag = (np.abs(b) + row(b)) * inv
        else:
            b_mag = np.abs(b)
        lift, _ = oracle.block_norm(np.zeros_like(x), np.ones_like(x), **{**o, "post": None, "norm": None, "weight": None,
                                                                            "scale": None, "shift": None})
        r_mag = np.abs(o.get("residual_scale", 1.0) * x) + np.abs(lift) * b_mag
    else:
        r_mag = np.abs(x)
    if o.get("norm", "rms") is None:
        return r_mag, None
    kind = o.get("norm", "rms")
    c = r - r.mean(-1, keepdims=True) if kind == "layer" else r
    inv = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + o.get("eps", 1e-6))
    _, plus = oracle.block_norm(gain, None, **{**o, "post": None, "post_weight": None, "gate": None, "shift": None,
                                               "norm": "rms", "eps": 0.0})
    _, sh = oracle.block_norm(np.zeros_like(x), None, **{**o, "post": None, "post_weight": None, "gate": None,
                                                         "weight": None, "scale": None, "norm": "rms", "eps": 1.0})
    # an error of the mean square moves the whole row by its relative size
    worst = (r_mag * np.abs(c)).mean(-1, keepdims=True) * inv * inv
    return r_mag, np.abs(plus) * inv * (r_mag + row(r_mag) + np.abs(c) * (1 + worst)) + np.abs(sh)


def _run(rbp, seed, M, D, xt="bf16", bt="bf16", yt=None, pt="f32", G=1, norm="rms", post=None, weight=True,
         post_weight=False, gate=True, mod=True, branch=True, ids=None, rho=1.0, eps=1e-6, pad=0, std=1.0, mean=0.0):
    rng = np.random.default_rng(seed)
    xt, bt, pt = DTYPES[xt], DTYPES[bt], DTYPES[pt]
    yt = xt if yt is None else DTYPES[yt]
    x, x64 = draw(rng, (M, D), xt, std)
    if mean:
        x = (x.float() + mean).to(xt)
        x64 = x.cpu().double().numpy()
    b, b64 = draw(rng, (M, D), bt) if branch else (None, None)
    ada, ada64 = draw(rng, (G, 6 * D), pt, 0.5)
    kw, o = {}, dict(norm=norm, post=post, residual_scale=rho, eps=eps)
    for name, on, part in (("shift", mod and norm, 0), ("scale", mod and norm, 1), ("gate", gate and branch, 2)):
        if on:
            kw[name], o[name] = ada[:, part * D:(part + 1) * D], ada64[:, part * D:(part + 1) * D]
    for name, on in (("weight", weight and norm), ("post_weight", post_weight and branch)):
        if on:
            kw[name], o[name] = draw(rng, (D,), pt)
    if ids is not None:
        kw["groups"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
        o["groups"] = ids
    if pad:
        x, b = strided(x, pad), None if b is None else strided(b, pad)
    got = rbp.block_norm(x, b, norm=norm, post=post, residual_scale=rho, eps=eps, out_dtype=yt if norm else None, **kw)
    r, y = (got if branch and norm else (got, None) if branch else (None, got))
    ref_r, ref_y = oracle.block_norm(x64, b64, **o)
    r_mag, y_mag = _mags(x64, b64, o)
    if branch:
        assert r.dtype == xt
        check(r, ref_r, xt, 64 * E * r_mag, "r")
    if norm:
        assert y.dtype == yt
        check(y, ref_y, yt, 64 * E * y_mag, "y")


@pytest.mark.parametrize("D", [1, 2, 7, 8, 64, 100, 303, 511, 512, 513, 520, 1000, 1024, 2048, 3072, 4096, 4097, 4104,
                               6328, 8192, 12288, 16383, 16384])
@pytest.mark.parametrize("norm,post", [("rms", "rms"), ("layer", "layer"), ("layer", None)])
def test_every_width(gpu_lib, D, norm, post):
    _run(gpu_lib, D, M=5, D=D, norm=norm, post=post, post_weight=post is not None)


@pytest.mark.parametrize("M", [0, 1, 3, 4, 5, 64, 1001])
@pytest.mark.parametrize("D", [256, 2048])
def test_every_number_of_rows(gpu_lib, M, D):
    _run(gpu_lib, M, M=M, D=D, G=3, post="rms")


@pytest.mark.parametrize("xt,bt,yt", [("f32", "f32", "f32"), ("f32", "bf16", "bf16"), ("f32", "f16", "f16"),
                                      ("f32", "bf16", "f32"), ("f32", "f32", "bf16"), ("f32", "bf16", "f16"),
                                      ("bf16", "bf16", "bf16"), ("f16", "f16", "f16")])
@pytest.mark.parametrize("pt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [99, 1536, 2048, 5000, 8192])
def test_every_type(gpu_lib, xt, bt, yt, pt, D):
    _run(gpu_lib, 3, M=9, D=D, xt=xt, bt=bt, yt=yt, pt=pt, G=3, norm="rms", post="layer", post_weight=True, rho=0.5)


@pytest.mark.parametrize("part", range(8))
@pytest.mark.parametrize("D", [320, 2048, 8192])
def test_every_part_alone(gpu_lib, part, D):
    none = dict(weight=False, gate=False, mod=False)
    kw = [dict(none, branch=False), dict(none, branch=False, weight=True), dict(none, branch=False, mod=True, G=2),
          dict(none), dict(none, gate=True, G=4), dict(none, post="rms"), dict(none, norm=None, gate=True),
          dict(none, norm=None, post="layer", post_weight=True)][part]
    _run(gpu_lib, part, M=8, D=D, **kw)


@pytest.mark.parametrize("D", [1024, 2048, 4096])
def test_unequal_and_unknown_groups(gpu_lib, D):
    _run(gpu_lib, 1, M=10, D=D, G=4)  # ceil(10 / 4) = 3 rows to a group, the last one short
    _run(gpu_lib, 2, M=10, D=D, G=4, ids=[3, 0, 0, 2, 1, -1, 4, 3, 2 ** 31 - 1, -2 ** 31])


@pytest.mark.parametrize("pad", [1, 3, 8, 24])
def test_strided_rows(gpu_lib, pad):
    _run(gpu_lib, pad, M=7, D=1024, pad=pad, post="rms")


def test_rows_read_at_an_odd_place(gpu_lib):
    rng = np.random.default_rng(1)
    x, x64 = draw(rng, (6, 640), torch.bfloat16)
    b, b64 = draw(rng, (6, 640), torch.bfloat16)
    for lead in (1, 2, 4, 8):
        r, y = gpu_lib.block_norm(strided(x, 3, lead), strided(b, 3, lead))
        r0, y0 = oracle.block_norm(x64, b64)
        r_mag, y_mag = _mags(x64, b64, {})
        check(r, r0, torch.bfloat16, 64 * E * r_mag, "r")
        check(y, y0, torch.bfloat16, 64 * E * y_mag, "y")


def test_a_layer_norm_keeps_a_large_mean_apart(gpu_lib):
    # mean 300 standard deviations away: E[v^2] - mean^2 in float32 would lose
    # 2 log2(300) = 16 bits of the variance
    _run(gpu_lib, 9, M=4, D=4096, xt="f32", bt="f32", yt="f32", norm="layer", mean=300.0, gate=False)


def test_zero_rows_and_no_epsilon(gpu_lib):
    x = torch.zeros(3, 768, device="cuda")
    x[1] = 1.0
    y = gpu_lib.block_norm(x, norm="rms", eps=1e-6)
    assert torch.equal(y[0], torch.zeros(768, device="cuda")) and torch.equal(y[2], y[0])
    assert torch.allclose(y[1], torch.full((768,), 1 / np.sqrt(1 + 1e-6), device="cuda", dtype=torch.float32), rtol=1e-6)
    y = gpu_lib.block_norm(x, norm="layer", eps=1e-6)
    assert torch.equal(y, torch.zeros_like(x))
    assert torch.isnan(gpu_lib.block_norm(x, norm="rms", eps=0.0)[0]).all()  # 0 / 0, as the formula has it


def test_a_row_that_is_not_finite_stays_alone(gpu_lib):
    rng = np.random.default_rng(2)
    for D in (256, 2048, 8192):
        x, _ = draw(rng, (8, D), torch.bfloat16)
        b, _ = draw(rng, (8, D), torch.bfloat16)
        r0, y0 = gpu_lib.block_norm(x, b, post="rms")
        b[3, D // 2] = float("nan")
        x[5, 1] = float("inf")
        r, y = gpu_lib.block_norm(x, b, post="rms")
        keep = [0, 1, 2, 4, 6, 7]
        assert torch.equal(r[keep], r0[keep]) and torch.equal(y[keep], y0[keep])
        assert torch.isnan(y[3]).all() and torch.isnan(y[5, 1])


def test_in_place(gpu_lib):
    rng = np.random.default_rng(4)
    for D in (300, 1024, 6144):
        x, _ = draw(rng, (11, D), torch.bfloat16)
        b, _ = draw(rng, (11, D), torch.bfloat16)
        r0, y0 = gpu_lib.block_norm(x, b, post="layer", residual_scale=0.7)
        r, y = gpu_lib.block_norm(x, b, post="layer", residual_scale=0.7, r_out=x, out=b)
        assert r.data_ptr() == x.data_ptr() and y.data_ptr() == b.data_ptr()
        assert torch.equal(x, r0) and torch.equal(b, y0)


def test_repeats_are_identical_and_streams_are_kept(gpu_lib):
    rng = np.random.default_rng(5)
    x, _ = draw(rng, (513, 3072), torch.float32)
    b, _ = draw(rng, (513, 3072), torch.bfloat16)
    first = gpu_lib.block_norm(x, b, post="rms", out_dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = gpu_lib.block_norm(x, b, post="rms", out_dtype=torch.bfloat16)
    side.synchronize()
    for p, q in zip(first, again):
        assert torch.equal(p, q)


def test_refusals(gpu_lib):
    rbp = gpu_lib
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    mod = torch.zeros(2, 64, device="cuda")
    bad = [
        lambda: rbp.block_norm(x.cpu()),
        lambda: rbp.block_norm(x[0]),
        lambda: rbp.block_norm(x.t()),
        lambda: rbp.block_norm(x.to(torch.int32)),
        lambda: rbp.block_norm(x, norm="batch"),
        lambda: rbp.block_norm(x, norm=None),
        lambda: rbp.block_norm(x, gate=mod),
        lambda: rbp.block_norm(x, x, norm=None, scale=mod),
        lambda: rbp.block_norm(x, x[:3]),
        lambda: rbp.block_norm(x, x.float()),                        # branch of another type than a 16-bit x
        lambda: rbp.block_norm(x, x, out_dtype=torch.float32),
        lambda: rbp.block_norm(x, scale=mod, shift=mod.bfloat16()),  # parameters of two types
        lambda: rbp.block_norm(x, scale=mod, shift=mod[:1]),
        lambda: rbp.block_norm(x, scale=mod[:0], shift=mod[:0]),     # no group at all
        lambda: rbp.block_norm(x, weight=mod),
        lambda: rbp.block_norm(x, scale=mod, groups=torch.zeros(4, device="cuda", dtype=torch.int64)),
        lambda: rbp.block_norm(x, scale=mod, groups=torch.zeros(3, device="cuda", dtype=torch.int32)),
        lambda: rbp.block_norm(x, eps=-1.0),
        lambda: rbp.block_norm(x, eps=float("nan")),
        lambda: rbp.block_norm(torch.zeros(2, 16385, device="cuda")),
        lambda: rbp.block_norm(x, x, r_out=x[:1].expand(4, 64)),     # output rows on top of each other
    ]
    for f in bad:
        with pytest.raises(rbp.OrbitError):
            f()


def test_in_a_graph(gpu_lib):
    rng = np.random.default_rng(6)
    x, _ = draw(rng, (32, 4096), torch.bfloat16)
    b, _ = draw(rng, (32, 4096), torch.bfloat16)
    r, y = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        gpu_lib.block_norm(x, b, r_out=r, out=y)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.block_norm(x, b, r_out=r, out=y)
    for seed in range(3):
        x.copy_(draw(np.random.default_rng(seed), (32, 4096), torch.bfloat16)[0])
        graph.replay()
        torch.cuda.synchronize()
        r0, y0 = gpu_lib.block_norm(x, b)
        assert torch.equal(r, r0) and torch.equal(y, y0)
