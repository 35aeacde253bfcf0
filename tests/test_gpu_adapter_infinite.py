"""adapter_add with infinite weights and activations: its products are what the
fp64 definition gives (infinite of the right sign, or NaN where infinities
cancel or meet a zero), the same for few tokens and for many.
"""
import numpy as np
import pytest
import torch

import oracle
from block_cases import DTYPES, check, draw, f64
from test_gpu_adapter import _mag

pytestmark = pytest.mark.gpu

INF = float("inf")


def _orders(M, L):
    return {"one": [0] * M, "few": [m // 30 % (L + 1) - 1 for m in range(M)], "many": [m % (L + 1) - 1 for m in range(M)]}


@pytest.mark.parametrize("xt", ["bf16", "f16"])
@pytest.mark.parametrize("order", ["one", "few", "many"])
@pytest.mark.parametrize("M,R,N", [*((M, R, N) for M in (5, 200, 257, 700, 1100, 2100)
                                     for R, N in ((8, 136), (24, 71), (40, 300), (128, 64))),
                                   (1100, 8, 15008)])  # the last: tiles of 64 tokens
def test_infinite_weights(gpu_lib, xt, order, M, R, N):
    L, K, t = 12, 64, DTYPES[xt]
    rng = np.random.default_rng(M + R)
    ids = _orders(M, L)[order]
    x, x64 = draw(rng, (M, K), t)
    y, y64 = draw(rng, (M, N), torch.float32)
    A, A64 = draw(rng, (L, R, K), t, K ** -0.5)
    B, _ = draw(rng, (L, N, R), t)
    B[::2, 3, 0] = INF             # the first ranks: read again for the ranks past the last
    B[1::2, N - 1, R // 2] = -INF
    B[::3, 7, R - 1] = INF
    B[0, 9, 0], B[0, 9, 1] = INF, -INF
    ranks = [(R, max(1, R - 3), 5)[a % 3] for a in range(L)]
    kw = dict(scale=torch.linspace(0.5, 2.0, L, device="cuda"), ranks=torch.tensor(ranks, dtype=torch.int32, device="cuda"))
    got = gpu_lib.adapter_add(y, x, A, B, torch.tensor(ids, dtype=torch.int32, device="cuda"), **kw)
    B64, s = f64(B), f64(kw["scale"])
    with np.errstate(invalid="ignore"):
        ref = oracle.adapter_add(y64, x64, A64, B64, ids, s, ranks)
    assert np.isinf(ref).any() or set(ids) == {-1}
    mag = _mag(y64, x64, A64, np.where(np.isfinite(B64), B64, 0.0), ids, s, ranks, t)
    check(got, ref, torch.float32, mag)


@pytest.mark.parametrize("xt", ["bf16", "f16"])
@pytest.mark.parametrize("M", [5, 200, 257, 700, 1100, 2100])
@pytest.mark.parametrize("order", ["one", "few", "many"])
def test_infinite_activations(gpu_lib, xt, M, order):
    # one rank in use, so that the second product has one term
    L, K, R, N, t = 5, 64, 8, 136, DTYPES[xt]
    rng = np.random.default_rng(M)
    ids = _orders(M, L)[order]
    x, _ = draw(rng, (M, K), t)
    x[::4, 5] = INF
    x[1::4, 5] = -INF
    y, y64 = draw(rng, (M, N), torch.float32)
    A, A64 = draw(rng, (L, R, K), t, K ** -0.5)
    B, _ = draw(rng, (L, N, R), t)
    B[:, 4] = 0    # an infinite sum has no product with it
    B[:, 6] = INF
    ranks = [1] * L
    got = gpu_lib.adapter_add(y, x, A, B, torch.tensor(ids, dtype=torch.int32, device="cuda"),
                              ranks=torch.tensor(ranks, dtype=torch.int32, device="cuda"))
    x64, B64 = f64(x), f64(B)
    with np.errstate(invalid="ignore"):
        ref = oracle.adapter_add(y64, x64, A64, B64, ids, None, ranks)
    zero = lambda a: np.where(np.isfinite(a), a, 0.0)  # noqa: E731
    check(got, ref, torch.float32, _mag(y64, zero(x64), A64, zero(B64), ids, None, ranks, t))
