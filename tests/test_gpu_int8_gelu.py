"""int8_qlinear's GELU, y Phi(y), alone: products of single codes and biases whose sums float32 holds exactly.

Tolerance.  With x = |y| / sqrt 2 and E = 2^-24: x^2 log2 e, from three factors and three products, is within 8 E of itself,
which is 8 x^2 E of exp(-x^2).  Its factor is a polynomial of degree 8 whose terms' magnitudes sum to twice its value, at
a t within 3 E (whose relative change is at most the polynomial's): 8 E; the exponential itself, two products and a
difference: 8 E; the fit 1.4e-8: a quarter of E.  So (8 x^2 + 20) E of the result, before it is rounded to its type.
"""
import numpy as np
import pytest
import torch
from scipy.special import log_ndtr

from block_cases import DTYPES, U

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def exact(y):
    return y * np.exp(log_ndtr(y))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N", [(8, 255), (8, 256), (300, 1024), (2048, 256), (4096, 256)])
def test_gelu_of_every_size(gpu_lib, M, N, dtype):
    qx = torch.zeros(M, 16, dtype=torch.int8, device="cuda")
    qx[:, 3] = 1
    qw = torch.zeros(N, 16, dtype=torch.int8, device="cuda")
    qw[:, 3] = (torch.arange(N) % 255 - 127).to(torch.int8).cuda()
    sx = 2.0 ** -(3 + torch.arange(M).float() % 24)
    bias = torch.round((torch.arange(N) % 7 - 3) * 2.0 ** 8 / 3) * 2.0 ** -10
    bias[::3] = 0
    y = sx.double()[:, None] * qw[:, 3].cpu().double() + bias.double()
    assert (y == y.float().double())[: 8].all()
    y = y.float().double().numpy()
    got = gpu_lib.int8_qlinear(qx, sx.cuda(), qw, torch.ones(N, device="cuda"), bias=bias.cuda(), out_dtype=DTYPES[dtype], act="gelu")
    want = exact(y)
    tiny = {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -25}[dtype]
    bound = np.abs(want) * ((4 * y * y + 20) * E + (U[DTYPES[dtype]] if dtype != "f32" else 0)) + tiny
    # the sum y is rounded once where float32 does not hold it: half a step, by a slope of at most 1.13
    bound = bound + 1.13 * E * np.abs(y)
    off = np.abs(got.cpu().double().numpy() - want)
    assert (off <= bound).all(), "%.3g times the bound at y = %r" % ((off / bound).max(), y[np.unravel_index((off / bound).argmax(), y.shape)])


def test_gelu_of_the_tail_keeps_its_digits(gpu_lib):
    """From -13 to 0 in steps of 1 / 512, exact in float32: the bound without the sum's own rounding."""
    y = -torch.arange(0, 13 * 512 + 1).float() / 512
    N = len(y)
    qx = torch.zeros(1, 16, dtype=torch.int8, device="cuda")
    got = gpu_lib.int8_qlinear(qx, torch.ones(1, device="cuda"), torch.zeros(N, 16, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda"),
                               bias=y.cuda(), out_dtype=torch.float32, act="gelu")[0].cpu().double().numpy()
    y = y.double().numpy()
    want = exact(y)
    assert (np.abs(got - want) <= np.abs(want) * (4 * y * y + 20) * E + 1e-37).all()
