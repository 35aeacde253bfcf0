"""int8_qlinear against 64 bits.

Tolerances.  The integer sums are exact.  y = (float(sum)) (sx sw) + b takes four roundings: within 4 E |sx sw sum| + E
(|b| + |y|).  GELU y/2 (1 + erf(y / sqrt 2)): erff and its argument are within 2^-21 of erf's slope and value, which
adds |y| 2^-21; the slope of the whole is at most 1.13.  Then one rounding to the output's type.
"""
import math

import numpy as np
import pytest
import torch

from block_cases import DTYPES, E, check, f64

pytestmark = pytest.mark.gpu


def codes(rng, rows, K, extreme=False):
    if extreme:
        return torch.from_numpy(rng.choice(np.array([-128, -127, 127], np.int8), (rows, K))).cuda()
    return torch.from_numpy(rng.integers(-128, 128, (rows, K)).astype(np.int8)).cuda()


def scales(rng, n, K):
    return torch.from_numpy((np.exp(rng.standard_normal(n)) / (74 * K ** 0.5)).astype(np.float32)).cuda()


def reference(qx, sx, qw, sw, bias, act):
    total = qx.double() @ qw.double().t()  # exact: below 2^53
    y = f64(total) * f64(sx)[:, None] * f64(sw)
    mag = 4 * E * np.abs(y)
    if bias is not None:
        y = y + f64(bias)
        mag = mag + E * (np.abs(f64(bias)) + np.abs(y))
    if act == "gelu":
        mag = 1.13 * mag + np.abs(y) * 2.0 ** -21
        y = 0.5 * y * (1 + np.vectorize(math.erf)(y / math.sqrt(2)) if y.size < 5000 else 1 + f64(torch.erf(torch.from_numpy(y) / math.sqrt(2))))
    return y, mag


def run(rbp, M, N, K, out="bf16", bias=None, act=None, extreme=False, seed=0):
    rng = np.random.default_rng(seed + M + 7 * N + 11 * K)
    qx, qw, sx, sw = codes(rng, M, K, extreme), codes(rng, N, K, extreme), scales(rng, M, K), scales(rng, N, K)
    b = torch.from_numpy(rng.standard_normal(N)).to(DTYPES[bias]).cuda() if bias else None
    got = rbp.int8_qlinear(qx, sx, qw, sw, bias=b, out_dtype=DTYPES[out], act=act)
    ref, mag = reference(qx, sx, qw, sw, b, act)
    check(got, ref, DTYPES[out], mag, f"{M} x {K} -> {N}")


SIZES = [(1, 1, 16), (1, 7, 16), (1, 300, 4096), (2, 8, 48), (5, 33, 64), (16, 16, 112), (16, 200, 128), (17, 264, 144), (33, 40, 1040),
         (64, 129, 256), (65, 96, 272), (100, 1000, 2064), (257, 31, 512), (300, 520, 96), (1000, 9, 640), (3, 4112, 1536)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out", ["bf16", "f32", "f16"])
def test_sizes(gpu_lib, M, N, K, out):
    run(gpu_lib, M, N, K, out)


@pytest.mark.parametrize("M,N,K", [(3, 100, 128), (70, 72, 80), (130, 256, 320), (600, 513, 192)])
@pytest.mark.parametrize("bias", [None, "f32", "bf16", "f16"])
@pytest.mark.parametrize("act", [None, "gelu"])
def test_bias_and_activation(gpu_lib, M, N, K, bias, act):
    run(gpu_lib, M, N, K, "f32", bias, act)
    run(gpu_lib, M, N, K, "bf16", bias, act)


# enough tiles for the tiled kernel: whole and ragged tiles, one chunk of K, part of a chunk, odd rows of the output
@pytest.mark.parametrize("M,N,K", [(4096, 3072, 64), (4096, 3072, 16), (4097, 3000, 80), (2049, 4104, 208), (5000, 1001, 4096),
                                   (16384, 1024, 144), (1025, 9000, 336), (257, 33000, 128), (33000, 257, 112)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_many_tiles(gpu_lib, M, N, K, out):
    run(gpu_lib, M, N, K, out, "f32", "gelu" if K == 80 else None)


@pytest.mark.parametrize("M,N,K", [(16, 64, 65536), (128, 128, 65536), (2048, 2048, 16384)])
def test_extreme_codes_and_long_rows(gpu_lib, M, N, K):
    """Sums up to 2^30."""
    run(gpu_lib, M, N, K, "f32", extreme=True)


def test_non_finite_scales_and_zero_rows(gpu_lib):
    for M in (5, 1500):
        rng = np.random.default_rng(M)
        qx, qw, sx, sw = codes(rng, M, 256), codes(rng, 1500, 256), scales(rng, M, 256), scales(rng, 1500, 256)
        sx[1], sx[2], qx[2], sx[3], sw[9] = float("nan"), float("nan"), 0, 0, float("nan")
        y = gpu_lib.int8_qlinear(qx, sx, qw, sw, out_dtype=torch.float32)
        assert y[1].isnan().all() and y[2].isnan().all() and y[:, 9].isnan().all()
        keep = [i for i in range(1500) if i != 9]
        assert (y[3, keep] == 0).all() and y[0, keep].isfinite().all() and y[4, keep].isfinite().all()


@pytest.mark.parametrize("M,N,K", [(4, 96, 512), (3000, 3000, 256)])
def test_out_repeat_stream_and_graph(gpu_lib, M, N, K):
    rng = np.random.default_rng(5)
    qx, qw, sx, sw = codes(rng, M, K), codes(rng, N, K), scales(rng, M, K), scales(rng, N, K)
    want = gpu_lib.int8_qlinear(qx, sx, qw, sw)
    out = torch.full_like(want, float("nan"))
    assert gpu_lib.int8_qlinear(qx, sx, qw, sw, out=out) is not None and torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, mine = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.stream(side):
        assert torch.equal(gpu_lib.int8_qlinear(qx, sx, qw, sw), want)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            gpu_lib.int8_qlinear(qx, sx, qw, sw, out=mine)
    for i in range(3):
        new = codes(rng, M, K)
        qx.copy_(new)
        mine.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(mine, gpu_lib.int8_qlinear(new, sx, qw, sw))


def test_unaligned_out(gpu_lib):
    rng = np.random.default_rng(6)
    for M, N in ((4, 64), (2048, 1024)):
        qx, qw, sx, sw = codes(rng, M, 64), codes(rng, N, 64), scales(rng, M, 64), scales(rng, N, 64)
        flat = torch.zeros(M * N + 1, dtype=torch.bfloat16, device="cuda")
        gpu_lib.int8_qlinear(qx, sx, qw, sw, out=flat[1:].view(M, N))
        assert flat[0] == 0 and torch.equal(flat[1:].view(M, N), gpu_lib.int8_qlinear(qx, sx, qw, sw))


def test_layer_from_float_rows(gpu_lib):
    """Both quantizers and the product: W x within the distortion of two 8-bit codes (steps of max / 127 each, errors of at
    most half a step, independent over 1024 coordinates)."""
    import synth
    rng = np.random.default_rng(8)
    K, M, N = 1024, 40, 96
    rot = gpu_lib.Rotation(*synth.rotation_params(K, seed=1), 128)
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    w = torch.from_numpy((rng.standard_normal((N, K)) / 32).astype(np.float32)).to(torch.bfloat16).cuda()
    (qx, sx), (qw, sw) = gpu_lib.int8_quant_rows(rot, x), gpu_lib.int8_quant_rows(rot, w)
    y = f64(gpu_lib.int8_qlinear(qx, sx, qw, sw, out_dtype=torch.float32))
    ref = f64(x) @ f64(w).T
    xs, ws = f64(sx)[:, None], f64(sw)
    # Cauchy-Schwarz with |x' - s q| <= s / 2 (1 + 2^-10) per coordinate
    nx, nw = np.linalg.norm(f64(x), axis=1)[:, None], np.linalg.norm(f64(w), axis=1)
    half = 0.5 * (1 + 2.0 ** -10) * math.sqrt(K)
    assert (np.abs(y - ref) <= half * (xs * nw + ws * nx) + half ** 2 * xs * ws).all()


def test_refusals(gpu_lib):
    rbp = gpu_lib
    q, s = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    o = torch.empty(4, 4, device="cuda")
    for bad in (lambda: rbp.int8_qlinear(q, s, q[:, :48], s), lambda: rbp.int8_qlinear(q, s[:3], q, s),
                lambda: rbp.int8_qlinear(q, s, q, s.half()), lambda: rbp.int8_qlinear(q.float(), s, q, s),
                lambda: rbp.int8_qlinear(q[:, :24].contiguous(), s, q[:, :24].contiguous(), s),
                lambda: rbp.int8_qlinear(q.t(), s, q, s), lambda: rbp.int8_qlinear(q, s, q.cpu(), s),
                lambda: rbp.int8_qlinear(q, s, q, s, bias=s[:2]), lambda: rbp.int8_qlinear(q, s, q, s, bias=s.long()),
                lambda: rbp.int8_qlinear(q, s, q, s, out=o, out_dtype=torch.bfloat16), lambda: rbp.int8_qlinear(q, s, q, s, out=o.t()[:, :]),
                lambda: rbp.int8_qlinear(q, s, q, s, act="relu"), lambda: rbp.int8_qlinear(q, s, q, s, out_dtype=torch.int8)):
        with pytest.raises(rbp.OrbitError):
            bad()
    assert rbp.int8_qlinear(q[:0], s[:0], q, s).shape == (0, 4)
