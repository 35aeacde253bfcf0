"""Norms of queries and keys for each head with the position rotation, alone (qk_norm) and into the cache (kv_append),
against 64 bits.

Bounds.  The mean is a sum of at most 256 terms, eight in turn and five levels of a tree: within 14 E mean|x|.  The centred
squares' sum is within (14 + 2) E of itself beside what the mean's error does (second order), so the factor is within 10 E
with the root and the division; x^ = ((x - mean) factor) w adds 3 roundings: 14 E |x^| + 16 E mean|x| factor |w| (layer
alone).  A rotated pair is two products and a sum of those: the magnitudes rotated, and 3 E.  The Hadamard transform adds
12 E sum|x| / sqrt(D) (eight levels, a scaling, the rounding before).
"""
import numpy as np
import pytest
import torch

import oracle
from block_cases import DTYPES, E, check, draw, f64

pytestmark = pytest.mark.gpu
EPS = 1e-6


def table(P, rot):
    angle = np.arange(P)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()


def normed(x, w, kind, eps=EPS):
    mean = x.mean(-1, keepdims=True) if kind == "layer" else 0.0
    factor = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    y = (x - mean) * factor * w
    mag = 14 * E * np.abs(y)
    if kind == "layer":
        mag = mag + 16 * E * np.abs(x).mean(-1, keepdims=True) * factor * np.abs(w)
    return y, mag


def turned(y, mag, cs, rot, interleaved, hadamard):
    c, s = cs[:, :rot // 2], cs[:, rot // 2:]

    def spread(v):
        return np.maximum(oracle.turn(v, np.abs(c), -np.abs(s), interleaved), oracle.turn(v, np.abs(c), np.abs(s), interleaved))

    z, m = oracle.turn(y, c, s, interleaved), spread(mag) + 3 * E * spread(np.abs(y))
    if hadamard:
        D = y.shape[-1]
        m = (m.sum(-1, keepdims=True) + 12 * E * np.abs(z).sum(-1, keepdims=True)) / np.sqrt(D) * np.ones(z.shape)
        z = oracle.hadamard_heads(z)
    return z, m


class Case:
    def __init__(self, seed, T=19, H=3, KV=2, D=64, xt="bf16", wt="f32", kind="rms", rot=None, interleaved=False, hadamard=False, each=False,
                 shift=0, mean=0.0, weights=True, eps=EPS):
        rng = np.random.default_rng(seed)
        self.rot = D if rot is None else rot
        qkv, _ = draw(rng, (T, H + 2 * KV, D + shift), DTYPES[xt], 2.0)
        qkv = (qkv.float() + mean).to(DTYPES[xt])[:, :, shift:]
        self.q, self.k, self.v = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
        ws = [draw(rng, (n, D) if each else (D,), DTYPES[wt]) for n in (H, KV)]
        self.cos_sin = table(300, self.rot) if self.rot else None
        pos = rng.integers(0, 300, T)
        self.positions = torch.from_numpy(pos).cuda()
        cs = f64(self.cos_sin)[pos] if self.rot else np.zeros((T, 0))
        self.kw = dict(norm=kind, positions=self.positions, cos_sin=self.cos_sin, interleaved=interleaved, hadamard=hadamard, eps=eps)
        if weights:
            self.kw.update(q_weight=ws[0][0], k_weight=ws[1][0])
        self.want = [turned(*normed(f64(x), w[1] if weights else 1.0, kind, eps), cs, self.rot, interleaved, hadamard)
                     for x, w in ((self.q, ws[0]), (self.k, ws[1]))]
        self.xt, self.shape = xt, (T, H, KV, D)

    def rows(self, rbp):
        q, k = rbp.qk_norm(self.q, self.k, **self.kw)
        for n, got, (ref, mag) in (("q", q, self.want[0]), ("k", k, self.want[1])):
            check(got, ref, DTYPES[self.xt], mag, n)
        assert torch.equal(rbp.qk_norm(self.q, **{n: x for n, x in self.kw.items() if n != "k_weight"}), q)
        return q, k

    def cache(self, rbp, fmt, page=8):
        T, H, KV, D = self.shape
        pages = -(-T // page) + 1
        t = torch.int8 if fmt == "int8" else DTYPES[fmt]
        kc, vc = (torch.zeros(pages, KV, page, D, dtype=t, device="cuda") for _ in "kv")
        sc = {n: torch.zeros(pages, KV, page, dtype=torch.float16, device="cuda") for n in ("k_scale", "v_scale")} if fmt == "int8" else {}
        slots = torch.randperm(pages * page, device="cuda")[:T]
        if T > 2:
            slots[2] = -1
        q = rbp.kv_append(self.k, self.v, kc, vc, slots, q=self.q, **self.kw, **sc)
        check(q, self.want[0][0], DTYPES[self.xt], self.want[0][1], "q")
        kept = (slots >= 0).cpu().numpy()
        pg, off = slots[slots >= 0] // page, slots[slots >= 0] % page
        got, ref, mag = f64(kc[pg, :, off]), self.want[1][0][kept], self.want[1][1][kept]
        v = f64(vc[pg, :, off])
        if fmt == "int8":
            s, sv = f64(sc["k_scale"][pg, :, off])[..., None], f64(sc["v_scale"][pg, :, off])[..., None]
            top = np.abs(ref).max(-1, keepdims=True) / 127
            assert (np.abs(s - top) <= top * 2.0 ** -11 * (1 + 2.0 ** -9) + mag.max(-1, keepdims=True) / 127 + 2.0 ** -25).all()
            # half a step, and what the rounded scale cuts off the largest
            assert (np.abs(got * s - ref) <= s * 0.5 * (1 + 2.0 ** -10) + 127 * np.abs(s - top) + mag).all()
            assert (np.abs(v * sv - f64(self.v)[kept]) <= sv * 0.5 * (1 + 2.0 ** -3)).all()
        else:
            check(torch.from_numpy(got), ref, DTYPES[fmt], mag, "k")
            assert np.array_equal(v, f64(self.v.to(DTYPES[fmt]))[kept])


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [8, 16, 24, 40, 64, 72, 80, 96, 120, 128, 136, 192, 256])
def test_every_head_dimension(gpu_lib, D, xt, kind):
    for interleaved in (False, True):
        for rot in sorted({D, D // 2 // 2 * 2, 2, 0}):
            Case(D + rot, D=D, xt=xt, kind=kind, rot=rot, interleaved=interleaved, hadamard=D & (D - 1) == 0).rows(gpu_lib)


@pytest.mark.parametrize("wt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("each", [False, True])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_weights(gpu_lib, wt, each, shift):
    Case(1, wt=wt, each=each, shift=shift, D=128).rows(gpu_lib)
    Case(2, wt=wt, each=each, shift=shift, D=80, kind="layer", xt="f16").rows(gpu_lib)
    c = Case(3, wt=wt, D=64)
    wide = torch.full((130,), float("nan"), dtype=DTYPES[wt], device="cuda")
    wide[1:65] = c.kw["q_weight"]
    c.kw["q_weight"] = wide[1:65]  # at an odd place
    c.rows(gpu_lib)


@pytest.mark.parametrize("T", [0, 1, 2, 7, 64, 333])
@pytest.mark.parametrize("H,KV", [(1, 1), (32, 8), (5, 5), (40, 1)])
def test_tokens_and_heads(gpu_lib, T, H, KV):
    Case(T, T=T, H=H, KV=KV, D=128, weights=T != 7).rows(gpu_lib)


@pytest.mark.parametrize("xt,fmt", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "int8"), ("f32", "bf16"), ("f32", "int8"), ("f16", "bf16")])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_into_the_cache(gpu_lib, xt, fmt, kind):
    for D in (16, 64, 80, 128, 256):
        Case(D, T=29, D=D, xt=xt, kind=kind, hadamard=D != 80 and fmt == "int8").cache(gpu_lib, fmt)
        Case(D, T=29, D=D, xt=xt, kind=kind, each=True, interleaved=True, rot=D // 2, shift=8).cache(gpu_lib, fmt)


def test_large_means(gpu_lib):
    """Centred sums: a mean a hundred times the spread keeps its digits."""
    Case(4, mean=200.0, kind="layer", xt="f32", D=128).rows(gpu_lib)
    Case(5, mean=200.0, kind="rms", xt="f32", D=128).rows(gpu_lib)


def test_in_place_and_strided_outputs(gpu_lib):
    for D, xt, shift in ((128, "bf16", 0), (80, "f16", 0), (64, "f32", 3), (256, "bf16", 8)):
        c = Case(6, T=150, H=9, KV=4, D=D, xt=xt, shift=shift, kind="layer", each=True)
        want = c.rows(gpu_lib)
        got = gpu_lib.qk_norm(c.q, c.k, q_out=c.q, k_out=c.k, **c.kw)
        assert got[0].data_ptr() == c.q.data_ptr() and torch.equal(c.q, want[0]) and torch.equal(c.k, want[1])


def test_zero_rows_infinities_and_unknown_positions(gpu_lib):
    c = Case(7, T=6, D=64, eps=0.0, weights=False)
    q = c.q.clone()
    q[0] = 0
    q[1, 0, 5] = float("inf")
    q[2, 1, 6] = float("nan")
    c.positions[4], c.positions[5] = 300, -1
    out = gpu_lib.qk_norm(q, **c.kw)
    assert out[0].isnan().all() and out[2, 1].isnan().all() and out[4:].isnan().all()
    # by the formula: a finite coordinate over an infinite root is 0, the infinite one NaN, and its partner with it
    lost = torch.zeros(64, dtype=torch.bool, device="cuda")
    lost[[5, 37]] = True
    assert torch.equal(out[1, 0].isnan(), lost) and (out[1, 0][~lost] == 0).all()
    assert out[1, 1:].isfinite().all() and out[3].isfinite().all()
    c.kw["eps"] = 1e-6
    assert (gpu_lib.qk_norm(q, **c.kw)[0] == 0).all()


def test_stream_and_graph(gpu_lib):
    c = Case(8, T=40, H=8, KV=2, D=128)
    want = gpu_lib.qk_norm(c.q, c.k, **c.kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, qo, ko = torch.cuda.CUDAGraph(), *(torch.empty_like(x) for x in want)
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            gpu_lib.qk_norm(c.q, c.k, q_out=qo, k_out=ko, **c.kw)
    for i in range(3):
        c.positions.add_(1).remainder_(300)
        graph.replay()
        torch.cuda.synchronize()
        want = gpu_lib.qk_norm(c.q, c.k, **c.kw)
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


def test_refusals(gpu_lib):
    rbp, c = gpu_lib, Case(9, D=64)
    call = lambda **kw: rbp.qk_norm(**{**dict(q=c.q, k=c.k), **c.kw, **kw})  # noqa: E731
    call()
    for bad in (dict(norm=None), dict(norm="batch"), dict(q=c.q[..., :60]), dict(k=c.k[:3]), dict(k=c.k.float()), dict(q=c.q.cpu()),
                dict(q_weight=c.kw["q_weight"][:8]), dict(q_weight=c.kw["q_weight"].half()), dict(k_weight=c.kw["k_weight"].long()),
                dict(k_weight=c.kw["k_weight"].expand(3, 64)), dict(eps=-1.0), dict(eps=float("nan")), dict(positions=None),
                dict(positions=c.positions[:2]), dict(cos_sin=c.cos_sin.repeat(1, 2)), dict(q_out=c.q[:2]), dict(k=None, k_out=c.k),
                dict(q_weight=c.kw["q_weight"].cpu())):
        with pytest.raises(rbp.OrbitError):
            call(**bad)
    kc = torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(19, device="cuda")
    kw = {n: x for n, x in c.kw.items()}
    rbp.kv_append(c.k, c.v, kc, kc.clone(), slots, q=c.q, **kw)
    for bad in (dict(norm=None), dict(norm="l2"), dict(eps=-1.0), dict(q=None), dict(k_weight=kw["k_weight"][:3])):
        with pytest.raises(rbp.OrbitError):
            rbp.kv_append(c.k, c.v, kc, kc.clone(), slots, **{**dict(q=c.q), **kw, **bad})
