"""The paged key-value cache (kv_append, kv_read) against the fp64 definition.

Bounds: a rotated pair is two products and a sum (3 E of their magnitudes);
the Hadamard transform of D <= 256 coordinates is 8 pairwise steps and one
scaling: 12 E of sum |x| / sqrt(D) with the rounding before it.  Codes and
scales follow the rule of the weights' group codes (parity.check_group_codes).
"""
import numpy as np
import pytest
import torch

import oracle
from block_cases import DTYPES, E, U, check, draw, f64
from parity import bits_of, check_group_codes

pytestmark = pytest.mark.gpu


def _table(P, rot, base=10000.0):
    angle = np.arange(P)[:, None] * base ** (-np.arange(0, rot, 2) / max(rot, 1))
    t = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    return torch.from_numpy(t).cuda(), t.astype(np.float64)


def _cache(pages, KV, page, D, fmt):
    t = torch.int8 if fmt == "int8" else DTYPES[fmt]
    kw = {}
    k, v = (torch.full((pages, KV, page, D), 77, dtype=t, device="cuda") for _ in "kv")
    if fmt == "int8":
        kw = {n: torch.full((pages, KV, page), 0.5, dtype=torch.float16, device="cuda") for n in ("k_scale", "v_scale")}
    return k, v, kw


def _run(rbp, seed, T, H, KV, D, page, xt, fmt, rot, interleaved=False, hadamard=False, slots=None, fused=True, shift=0):
    rng = np.random.default_rng(seed)
    t = DTYPES[xt]
    pages = -(-T // page) + 2
    qkv, qkv64 = draw(rng, (T, H + 2 * KV, D + shift), t)
    qkv[:, :, shift + 1] *= 8  # an outlier channel
    qkv64 = f64(qkv)[:, :, shift:]
    qkv = qkv[:, :, shift:]  # heads that begin at an odd place when shift is odd
    q, k, v = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    if slots is None:
        slots = rng.permutation(pages * page)[:T]
        slots[::7] = -1
    slots = np.asarray(slots)
    pos = rng.integers(0, 5000, T)
    cos_sin, cs = _table(5000, rot) if rot else (None, np.zeros((5000, 0)))
    kc, vc, scales = _cache(pages, KV, page, D, fmt)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    q_out = rbp.kv_append(k, v, kc, vc, dev(slots.astype(np.int64)), positions=dev(pos.astype(np.int64)), cos_sin=cos_sin,
                          interleaved=interleaved, q=q if H else None, hadamard=hadamard, **scales)
    c, s = cs[pos][:, :rot // 2], cs[pos][:, rot // 2:]
    turned = oracle.turn(qkv64[:, :H + KV], c, s, interleaved)
    mag = 3 * E * oracle.turn(np.abs(qkv64[:, :H + KV]), np.abs(c), -np.abs(s), interleaved)
    mag = np.maximum(mag, 3 * E * oracle.turn(np.abs(qkv64[:, :H + KV]), np.abs(c), np.abs(s), interleaved))
    if hadamard:
        mag = 12 * E * np.abs(turned).sum(-1, keepdims=True) / np.sqrt(D) * np.ones(turned.shape)
        turned = oracle.hadamard_heads(turned)
    if H:
        assert q_out.dtype == t and q_out.is_contiguous()
        check(q_out, turned[:, :H], t, mag[:, :H], "q")
    else:
        assert q_out is None
    kept = (slots >= 0) & (slots < pages * page)
    pg, off = slots[kept] // page, slots[kept] % page
    ref = {"k": turned[kept][:, H:], "v": qkv64[kept][:, H + KV:]}
    untouched = np.ones((pages, page), dtype=bool)
    untouched[pg, off] = False
    for n, cache in (("k", kc), ("v", vc)):
        got = cache.cpu()
        assert (got.transpose(1, 2)[torch.from_numpy(untouched)] == 77).all(), "a slot that was not named was written"
        rows = got.transpose(1, 2)[torch.from_numpy(pg), torch.from_numpy(off)]  # [T', KV, D]
        if not kept.any():
            continue
        if fmt == "int8":
            sc = scales[n + "_scale"].cpu().transpose(1, 2)
            assert (sc[torch.from_numpy(untouched)] == 0.5).all()
            bits = bits_of(sc[torch.from_numpy(pg), torch.from_numpy(off)].contiguous())
            check_group_codes(rows.numpy().reshape(-1, D), bits.reshape(-1, 1), ref[n].reshape(-1, D), D, 127, n)
        else:
            check(rows, ref[n], DTYPES[fmt], mag[kept][:, H:] if n == "k" else 0.0, n)
    # reading back: the cache's values, rounded once
    back = rbp.kv_read(kc, vc, dev(slots.astype(np.int64)), dtype=t, **scales)
    for n, cache, got in (("k", kc, back[0]), ("v", vc, back[1])):
        vals = f64(cache)
        if fmt == "int8":
            vals = vals * f64(scales[n + "_scale"])[..., None]
        want = np.zeros((T, KV, D))
        want[kept] = vals.transpose(0, 2, 1, 3)[pg, off]
        assert got.dtype == t
        check(got, want, t, 0.0, "read " + n)


@pytest.mark.parametrize("T", [0, 1, 2, 7, 64, 333])
@pytest.mark.parametrize("fmt,had", [("bf16", False), ("int8", True)])
def test_every_number_of_tokens(gpu_lib, T, fmt, had):
    _run(gpu_lib, T, T, 8, 2, 128, 16, "bf16", fmt, 128, hadamard=had)


@pytest.mark.parametrize("D", [8, 16, 24, 32, 40, 64, 72, 80, 96, 120, 128, 160, 192, 248, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_every_head_dimension(gpu_lib, D, interleaved):
    had = D & (D - 1) == 0
    for rot in sorted({D, D // 2 // 2 * 2, 2, 0}):
        _run(gpu_lib, D, 19, 3, 2, D, 8, "bf16", "bf16", rot, interleaved, had)
        if D % 16 == 0:
            _run(gpu_lib, D, 19, 3, 2, D, 8, "f16", "int8", rot, interleaved, had)


@pytest.mark.parametrize("xt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8"])
@pytest.mark.parametrize("had", [False, True])
def test_every_type(gpu_lib, xt, fmt, had):
    _run(gpu_lib, 5, 50, 4, 2, 128, 16, xt, fmt, 128, hadamard=had)
    _run(gpu_lib, 6, 50, 4, 2, 64, 16, xt, fmt, 32, interleaved=True, hadamard=had, fused=False)


@pytest.mark.parametrize("H,KV", [(0, 1), (1, 1), (5, 1), (32, 8), (40, 8), (16, 16), (128, 1), (7, 3)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_head_layout(gpu_lib, H, KV, D):
    _run(gpu_lib, H, 21, H, KV, D, 4, "bf16", "bf16", D)
    _run(gpu_lib, H, 21, H, KV, D, 4, "bf16", "int8", D, hadamard=True)


@pytest.mark.parametrize("page", [1, 2, 4, 16, 64, 1024])
def test_every_page_size(gpu_lib, page):
    _run(gpu_lib, page, 100, 2, 2, 64, page, "f16", "f16", 64)
    if page >= 4:
        _run(gpu_lib, page, 100, 2, 2, 64, page, "f16", "int8", 64, hadamard=True)


@pytest.mark.parametrize("shift", [1, 2, 4, 8])
def test_heads_that_begin_at_an_odd_place(gpu_lib, shift):
    for rot, inter in ((128, False), (128, True), (36, False)):
        _run(gpu_lib, shift, 30, 3, 2, 128, 16, "bf16", "bf16", rot, inter, shift=shift)


def test_slots_outside_the_cache(gpu_lib):
    slots = [-1, -2 ** 63, 2 ** 62, 2 ** 32, 2 ** 32 + 3, 96, 95, 0, 31, -5, 64, 2 ** 31]  # 96 slots
    _run(gpu_lib, 1, 12, 2, 1, 64, 16, "bf16", "bf16", 64, slots=slots)


def test_positions_outside_the_table(gpu_lib):
    rng = np.random.default_rng(2)
    q, _ = draw(rng, (5, 2, 64), torch.float32)
    k, _ = draw(rng, (5, 1, 64), torch.float32)
    kc, vc, _ = _cache(2, 1, 8, 64, "bf16")
    cs, _ = _table(100, 64)
    pos = torch.tensor([0, 100, -1, 99, 2 ** 40], device="cuda")
    out = gpu_lib.kv_append(k, k, kc, vc, torch.arange(5, device="cuda"), positions=pos, cos_sin=cs, q=q)
    assert torch.isnan(out[[1, 2, 4]]).all() and torch.isfinite(out[[0, 3]]).all()
    assert (kc[0, 0, [1, 2, 4]] == 77).all() and (vc[0, 0, [1, 2, 4]] == 77).all() and not (kc[0, 0, [0, 3]] == 77).all()
    assert torch.equal(out[0], q[0])  # position 0 turns nothing


def test_rotation_keeps_products_and_spreads_outliers(gpu_lib):
    """q' . k' = q . k, and one outlier channel no longer costs the others their codes."""
    rng = np.random.default_rng(3)
    T, D = 64, 128
    k, k64 = draw(rng, (T, 1, D), torch.float32)
    k[:, :, 17] *= 100
    k64 = f64(k)
    q, q64 = draw(rng, (T, 1, D), torch.float32)
    off = {}
    for had in (False, True):
        kc, vc, sc = _cache(4, 1, 16, D, "int8")
        slots = torch.arange(T, device="cuda")
        q2 = gpu_lib.kv_append(k, k, kc, vc, slots, q=q, hadamard=had, **sc)
        k2, _ = gpu_lib.kv_read(kc, vc, slots, dtype=torch.float32, **sc)
        got = np.einsum("thd,thd->t", f64(q2), f64(k2))
        off[had] = np.sqrt(np.mean((got - np.einsum("thd,thd->t", q64, k64)) ** 2))
    # uniform rounding error of step / sqrt(12) per coordinate: the step is max|k| / 127, and the
    # Hadamard brings max|k| from ~100 |x| to ~100 |x| / sqrt(128) * a few
    assert off[True] < 0.5 * off[False]


def test_zero_infinite_and_nan_heads(gpu_lib):
    k = torch.randn(4, 1, 64, device="cuda")
    k[0] = 0
    k[1, 0, 5] = float("inf")
    k[2, 0, 9] = float("nan")
    kc, vc, sc = _cache(1, 1, 4, 64, "int8")
    slots = torch.arange(4, device="cuda")
    gpu_lib.kv_append(k, k, kc, vc, slots, **sc)
    back, _ = gpu_lib.kv_read(kc, vc, slots, **sc)
    assert torch.equal(back[0], torch.zeros_like(back[0])) and torch.isfinite(back[3]).all()
    assert not torch.isfinite(back[1]).any() and not torch.isfinite(back[2]).any()  # seen, not hidden
    assert torch.allclose(back[3].float(), k[3], atol=float(k[3].abs().max()) / 127)


def test_another_stream_and_a_graph(gpu_lib):
    rng = np.random.default_rng(4)
    k, _ = draw(rng, (33, 2, 128), torch.bfloat16)
    q, _ = draw(rng, (33, 8, 128), torch.bfloat16)
    cs, _ = _table(64, 128)
    slots, pos = torch.arange(33, device="cuda"), torch.arange(33, device="cuda")
    a, b = _cache(5, 2, 8, 128, "int8"), _cache(5, 2, 8, 128, "int8")
    first = gpu_lib.kv_append(k, k, a[0], a[1], slots, positions=pos, cos_sin=cs, q=q, hadamard=True, **a[2])
    out = torch.empty_like(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gpu_lib.kv_append(k, k, b[0], b[1], slots, positions=pos, cos_sin=cs, q=q, q_out=out, hadamard=True, **b[2])
    side.synchronize()
    assert torch.equal(out, first) and torch.equal(a[0], b[0]) and torch.equal(a[2]["v_scale"], b[2]["v_scale"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.kv_append(k, k, b[0], b[1], slots, positions=pos, cos_sin=cs, q=q, q_out=out, hadamard=True, **b[2])
    for step in range(3):
        pos += 1
        slots.copy_(torch.roll(slots, 1))
        graph.replay()
        torch.cuda.synchronize()
        want = gpu_lib.kv_append(k, k, a[0], a[1], slots, positions=pos, cos_sin=cs, q=q, hadamard=True, **a[2])
        assert torch.equal(out, want) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals(gpu_lib):
    rbp = gpu_lib
    k = torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    slots = torch.zeros(4, device="cuda", dtype=torch.int64)
    kc, vc, _ = _cache(2, 2, 8, 64, "bf16")
    k8, v8, sc = _cache(2, 2, 8, 64, "int8")
    cs, _ = _table(10, 64)
    bad = [
        lambda: rbp.kv_append(k.cpu(), k, kc, vc, slots),
        lambda: rbp.kv_append(k, k[:, :1], kc, vc, slots),
        lambda: rbp.kv_append(k, k.float(), kc, vc, slots),
        lambda: rbp.kv_append(k.int(), k.int(), kc, vc, slots),
        lambda: rbp.kv_append(k, k, kc, vc, slots.int()),
        lambda: rbp.kv_append(k, k, kc, vc, slots[:3]),
        lambda: rbp.kv_append(k, k, kc, vc.half(), slots),
        lambda: rbp.kv_append(k, k, kc.float(), vc.float(), slots),
        lambda: rbp.kv_append(k, k, kc.transpose(2, 3), vc.transpose(2, 3), slots),
        lambda: rbp.kv_append(k, k, kc, vc, slots, cos_sin=cs),
        lambda: rbp.kv_append(k, k, kc, vc, slots, cos_sin=cs.double(), positions=slots),
        lambda: rbp.kv_append(k, k, kc, vc, slots, cos_sin=cs[:0], positions=slots),
        lambda: rbp.kv_append(k, k, kc, vc, slots, cos_sin=torch.zeros(10, 66, device="cuda"), positions=slots),
        lambda: rbp.kv_append(k, k, kc, vc, slots, cos_sin=torch.zeros(10, 31, device="cuda"), positions=slots),
        lambda: rbp.kv_append(k, k, kc, vc, slots, q=k, q_out=k),
        lambda: rbp.kv_append(k, k, kc, vc, slots, q_out=k),
        lambda: rbp.kv_append(k, k, kc, vc, slots, **sc),
        lambda: rbp.kv_append(k, k, k8, v8, slots),
        lambda: rbp.kv_append(k, k, k8, v8, slots, k_scale=sc["k_scale"].float(), v_scale=sc["v_scale"]),
        lambda: rbp.kv_append(k[:, :, :24], k[:, :, :24], kc[..., :24].contiguous(), vc[..., :24].contiguous(), slots, hadamard=True),
        lambda: rbp.kv_append(k, k, kc[:, :, :3].contiguous(), vc[:, :, :3].contiguous(), slots),  # page not a power of two
        lambda: rbp.kv_append(k[:, :, :8], k[:, :, :8], k8[..., :8].contiguous(), v8[..., :8].contiguous(), slots, **sc),
        lambda: rbp.kv_read(kc, vc, slots, dtype=torch.int8),
        lambda: rbp.kv_read(k8, v8, slots),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(rbp.OrbitError):
            f()
            print("not refused:", i)
