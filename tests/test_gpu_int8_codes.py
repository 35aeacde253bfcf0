"""int8_quant_rows: the codes and scales are those of the definition, s = max|x'| / 127 and q = 127 x' / max|x'| rounded
to the nearest integer.

The oracle rotates in float64 without the factor 1 / sqrt(h): sums of 16-bit values that lie within 2^33 of each other
are exact so, and those of float32 rows within log2(h) 2^-53 of the block's largest.  127 y / max is then within 1e-12 of
what it stands for, and codes are compared wherever it is not that near to a half (NEAR, a thousand times wider).  A scale
is rounded once, from float64: half a step of float32 (2^-24 of it), and what its computation in 64 bits adds (SLACK).
"""
import numpy as np
import pytest
import torch

import synth
from block_cases import DTYPES

pytestmark = pytest.mark.gpu

NEAR, SLACK = 1e-9, 1e-12


def turned(x, perm, signs, h):
    """Pi x sqrt(h), in float64."""
    y = (x.double().cpu()[:, torch.from_numpy(perm).long()] * torch.from_numpy(np.asarray(signs, np.float64))).reshape(-1, h)
    n = 1
    while n < h:
        y = y.reshape(-1, 2, n)
        y = torch.stack([y[:, 0] + y[:, 1], y[:, 0] - y[:, 1]], 1)
        n *= 2
    return y.reshape(x.shape[0], -1)


def coded(rbp, x, h, near=NEAR):
    """Checks the codes of x, rotated by blocks of h (0: not); the number of codes that were compared."""
    d = x.shape[1]
    perm, signs = synth.rotation_params(d, seed=d + h) if h else (None, None)
    q, s = rbp.int8_quant_rows(rbp.Rotation(perm, signs, h) if h else None, x)
    y = turned(x, perm, signs, h) if h else x.double().cpu()
    top = y.abs().amax(1, keepdim=True)
    assert torch.isfinite(top).all() and (top > 0).all()
    u = 127 * y / top
    sure = ((u - torch.floor(u)) - 0.5).abs() > near
    wrong = (q.cpu().double() != torch.round(u)) & (sure if near else torch.ones_like(sure))
    assert not wrong.any(), "%d of %d codes, the first at %s" % (int(wrong.sum()), u.numel(), wrong.nonzero()[0].tolist())
    scale = (top[:, 0] / (127 * max(h, 1) ** 0.5))
    assert ((s.cpu().double() - scale).abs() <= scale * (2.0 ** -24 + SLACK) + 2.0 ** -150).all()
    return int(sure.sum())


def rows(M, d, dtype, seed):
    """Tokens of different sizes, some channels far larger than the others."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    chan = torch.where(torch.rand(d, generator=g, device="cuda") < 0.005, 50.0, 1.0)
    size = torch.exp(0.5 * torch.randn(M, 1, generator=g, device="cuda"))
    return (torch.randn(M, d, generator=g, device="cuda") * chan * size).to(DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,d,h", [(1024, 3328, 64), (1024, 3328, 128), (3200, 3328, 256), (512, 4096, 512), (512, 4096, 1024),
                                   (512, 2048, 2048), (512, 4096, 4096), (64, 16384, 128), (2000, 48, 16), (2000, 96, 32)])
def test_codes_of_rotated_rows(gpu_lib, M, d, h, dtype):
    x = rows(M, d, dtype, seed=d + h)
    assert coded(gpu_lib, x, h) > 0.999 * M * d


# a block's sum of values near the type's largest is far above float32's, its scale is not
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,h", [(256, 16), (256, 128), (1024, 256), (1024, 1024), (4096, 4096)])
def test_rows_near_the_largest_value(gpu_lib, d, h, dtype):
    g = torch.Generator(device="cuda").manual_seed(h)
    x = torch.where(torch.rand(6, d, generator=g, device="cuda") < 0.5, -1.0, 1.0) * 2.0 ** 122
    x[1] = 2.0 ** 122
    x[2] = 2.0 ** 127
    x[3:] *= 31 * torch.rand(3, d, generator=g, device="cuda")
    coded(gpu_lib, x.to(DTYPES[dtype]), h)


def halves(d, dtype, seed):
    """Rows whose largest is b, with values (k + 1/2) b / 127 in every place where the type holds them, and their neighbours."""
    g = torch.Generator().manual_seed(seed)
    t = DTYPES[dtype]
    out = []
    for b in (127.0, 254.0, 1.0, 2.0, 127.0 * 2 ** -20, 63.5, 508.0, 100.0):
        k = torch.randint(-127, 127, (d,), generator=g).double()
        v = ((k + 0.5) * b / 127).to(t)
        step = torch.where(torch.rand(d, generator=g) < 0.3, 1, 0) * torch.where(torch.rand(d, generator=g) < 0.5, -1, 1)
        v = (v.view(torch.int32 if dtype == "f32" else torch.int16) + step.to(torch.int32 if dtype == "f32" else torch.int16)).view(t)
        v = torch.where(v.abs() > b, torch.zeros_like(v), v)
        v[torch.randint(0, d, (1,), generator=g)] = b
        out.append(v)
    return torch.stack(out).cuda()


# 127 x of a value of 24 bits or fewer is exact in float64, and its quotient by the maximum rounded once: a tie stays one, and
# no other value becomes one (two values of 24 bits whose quotient is no tie are 2^-33 away at least)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [16, 240, 1024, 1040, 4096, 16384])
def test_ties_go_to_the_even_code(gpu_lib, d, dtype):
    x = halves(d, dtype, d)
    coded(gpu_lib, x, 0, near=0)
    coded(gpu_lib, -x, 0, near=0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_every_code_of_rows_that_are_not_rotated(gpu_lib, dtype):
    x = rows(4000, 2512, dtype, 7)
    assert coded(gpu_lib, x, 0, near=0) > 0


# blocks of one value (and zeros) rotate to that value times +-1 everywhere: a block of half the largest is a tie
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,h", [(256, 16), (256, 64), (1024, 128), (2048, 256), (2048, 1024), (4096, 2048)])
def test_ties_of_rotated_rows(gpu_lib, d, h, dtype):
    perm, signs = synth.rotation_params(d, seed=d + h)
    blocks = torch.zeros(12, d // h, h)
    size = [3.0, 3.25, 5.0, 7.0, 9.5, 11.0, 13.0, 15.0, 17.0, 19.0, 21.0, 23.0]  # 127 / size is rounded either way
    g = torch.Generator().manual_seed(h)
    for r in range(12):
        for b in range(d // h):
            blocks[r, b, torch.randint(0, h, (1,), generator=g)] = float([1.0, 0.5, -0.5, 63.5 / 127, 1.5, -2.0][(r + b) % 6]) * size[r]
    blocks[:, 0] = 0
    blocks[:, 0, 5] = 2 * torch.tensor(size)
    x = torch.zeros(12, d)
    x[:, torch.from_numpy(perm).long()] = blocks.reshape(12, d)  # the gather brings them back
    coded(gpu_lib, x.to(DTYPES[dtype]).cuda(), h, near=0)
