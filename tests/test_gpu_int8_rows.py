"""int8_quant_rows against float64: x' = Pi x, s = max|x'| / 127, codes rounded to nearest.

Tolerances.  A coordinate of x' is a sum of h terms in log2(h) levels, scaled once: within e = (log2 h + 1) E sum|x| /
sqrt(h) over its block (e = 0 without a rotation).  s then is within max e / 127 + 3 E s.  A code is the nearest integer
to u = 127 x' / max|x'|, whose float32 form is within 127 (2 e / max) + 4 E 127 of it (x' and max, a division, the
fused product's one rounding at 1.5 * 2^23 + u is the rounding to an integer itself).
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from block_cases import DTYPES, E, draw, strided

pytestmark = pytest.mark.gpu


def rotation(rbp, d, h, plan=True, identity=False):
    perm, signs = synth.rotation_params(d, seed=d + h)
    if identity:
        perm = np.arange(d, dtype=np.int32)
    return rbp.Rotation(perm, signs, h, plan=plan), perm, signs


def against(q, s, x, perm, signs, h):
    """x: float64 [M, K]."""
    e = np.zeros(len(x))
    if h:
        y = oracle.rpbh_rotate(x, perm, signs, h)
        sums = np.abs(x[:, perm]).reshape(len(x), -1, h).sum(2).max(1)
        e = (np.log2(h) + 1) * E * sums / np.sqrt(h)
    else:
        y = x
    q, s = q.cpu().numpy().astype(np.float64), s.cpu().numpy().astype(np.float64)
    fine = np.isfinite(x).all(1)
    assert np.isnan(s[~fine]).all() and (q[~fine] == 0).all()
    y, q, s, e = y[fine], q[fine], s[fine], e[fine]
    top = np.abs(y).max(1)
    assert (np.abs(s - top / 127) <= e / 127 + 3 * E * top / 127 + 2.0 ** -149).all()
    zero = top <= e
    assert (q[zero & (top == 0)] == 0).all()
    y, q, top, e = y[~zero], q[~zero], top[~zero], e[~zero]
    off = np.abs(q - 127 * y / top[:, None])
    bound = 0.5 + (254 * e / top + 4 * E * 127)[:, None]
    assert (off <= bound).all(), f"a code is {off.max()} off"
    assert np.abs(q).max(initial=0) <= 127


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("d,h", [(16, 16), (48, 16), (96, 32), (320, 64), (1024, 1024), (1280, 256), (2048, 2048), (4096, 4096),
                                 (4096, 2048), (3072, 1024), (5120, 512), (8192, 64), (12288, 256), (16384, 128), (9216, 128)])
def test_rotated(gpu_lib, d, h, dtype):
    rng = np.random.default_rng(d + h)
    rot, perm, signs = rotation(gpu_lib, d, h)
    x, ref = draw(rng, (5, d), DTYPES[dtype])
    q, s = gpu_lib.int8_quant_rows(rot, x)
    against(q, s, ref, perm, signs, h)


# rows of whole words: every width, both blocks, with and without a plan, an identity, more rows than waves
@pytest.mark.parametrize("d", [1024, 2048, 3072, 4096, 8192, 12288, 16384])
@pytest.mark.parametrize("h", [128, 256])
@pytest.mark.parametrize("form", ["plan", "no plan", "identity"])
def test_bf16_blocks_of_128_and_256(gpu_lib, d, h, form):
    rng = np.random.default_rng(3 * d + h)
    rot, perm, signs = rotation(gpu_lib, d, h, plan=form != "no plan", identity=form == "identity")
    x, ref = draw(rng, (3, d), torch.bfloat16)
    x[1, 5::64] *= 100
    x[2] = 0
    ref = x.double().cpu().numpy()
    q, s = gpu_lib.int8_quant_rows(rot, x)
    against(q, s, ref, perm, signs, h)


@pytest.mark.parametrize("d,h", [(1024, 128), (3072, 128), (2048, 256), (8192, 256), (640, 64)])
def test_many_rows(gpu_lib, d, h):
    rng = np.random.default_rng(d)
    rot, perm, signs = rotation(gpu_lib, d, h)
    x, ref = draw(rng, (9001, d), torch.bfloat16)
    q, s = gpu_lib.int8_quant_rows(rot, x)
    at = np.r_[0:4, 4093:4101, 8190:8194, 8999:9001]
    against(q[at], s[at], ref[at], perm, signs, h)
    q2, s2 = gpu_lib.int8_quant_rows(rot, x[17:23])
    assert torch.equal(q[17:23], q2) and torch.equal(s[17:23], s2)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("K", [16, 32, 240, 1024, 1040, 4096, 4112, 8208, 16384])
def test_not_rotated(gpu_lib, K, dtype):
    rng = np.random.default_rng(K)
    x, ref = draw(rng, (7, K), DTYPES[dtype])
    against(*gpu_lib.int8_quant_rows(None, x), ref, None, None, 0)


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "f16"])
def test_strided_unaligned_rows(gpu_lib, rotated, dtype):
    rng = np.random.default_rng(1)
    x, ref = draw(rng, (6, 256), DTYPES[dtype])
    rot, perm, signs = rotation(gpu_lib, 256, 128)
    for view in (strided(x, 3, 1), strided(x, 8, 8), x[1:2].as_strided((1, 256), (3, 1), x[1:2].storage_offset())):
        r = ref if len(view) == 6 else ref[1:2]
        against(*gpu_lib.int8_quant_rows(rot if rotated else None, view), r, perm, signs, 128 if rotated else 0)


@pytest.mark.parametrize("d,h,dtype", [(256, 128, "f32"), (1024, 128, "bf16"), (2048, 256, "bf16"), (8192, 128, "bf16"), (96, 0, "f32"),
                                       (2048, 0, "bf16")])
def test_zeros_tiny_and_non_finite_rows(gpu_lib, d, h, dtype):
    rng = np.random.default_rng(d)
    rot, perm, signs = rotation(gpu_lib, d, h) if h else (None, None, None)
    x, _ = draw(rng, (9, d), DTYPES[dtype])
    x[0] = 0
    x[1, 3], x[2, 5], x[3, 7] = float("nan"), float("inf"), float("-inf")
    x[4] *= 2.0 ** -118  # 127 / max leaves float32's range below 2^-121
    x[5] *= 2.0 ** -104
    x[6] *= 2.0 ** 100
    x[7] = -0.0
    q, s = gpu_lib.int8_quant_rows(rot, x)
    against(q, s, x.double().cpu().numpy(), perm, signs, h)
    assert s[0] == 0 and s[7] == 0


def test_empty_and_other_stream(gpu_lib):
    rot, perm, signs = rotation(gpu_lib, 1024, 128)
    q, s = gpu_lib.int8_quant_rows(rot, torch.zeros(0, 1024, dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 1024) and s.shape == (0,)
    x, ref = draw(np.random.default_rng(0), (33, 1024), torch.bfloat16)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = gpu_lib.int8_quant_rows(rot, x)
    side.synchronize()
    against(*got, ref, perm, signs, 128)


def test_refusals(gpu_lib):
    rbp = gpu_lib
    rot, _, _ = rotation(rbp, 256, 128)
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: rbp.int8_quant_rows(rot, x[:, :128]), lambda: rbp.int8_quant_rows(rot, x.cpu()),
                lambda: rbp.int8_quant_rows(rot, x.to(torch.float64)), lambda: rbp.int8_quant_rows(None, x[:, :20]),
                lambda: rbp.int8_quant_rows(None, x.t()), lambda: rbp.int8_quant_rows(None, x[0]),
                lambda: rbp.int8_quant_rows(None, torch.zeros(1, 16400, device="cuda")), lambda: rbp.int8_quant_rows("rot", x)):
        with pytest.raises(rbp.OrbitError):
            bad()
