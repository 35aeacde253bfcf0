"""adapter_add keeps A x in float32's precision between its two products,
whatever the number of tokens and the types.

The inputs make both products exact: a token has three places (1, 2^-8, 2^-16)
where the adapter holds eight-bit numbers of one sign, so A x has up to 24 bits
and no rounding, and one row of B is 1.  What remains is the rounding of a
product with the scale, of the sum with y, and of the output.
"""
import numpy as np
import pytest
import torch

from block_cases import DTYPES, E, check, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt", ["bf16", "f16"])
@pytest.mark.parametrize("M", [3, 200, 257, 700, 1025, 2100])
@pytest.mark.parametrize("R", [8, 40, 64, 128])
@pytest.mark.parametrize("order", ["one", "few", "many"])
def test_no_bits_are_lost_between_the_products(gpu_lib, xt, M, R, order):
    K, N, L, t = 256, 72, 24, DTYPES[xt]
    rng = np.random.default_rng(M + R)
    ids = {"one": np.zeros(M, int), "few": np.arange(M) // 50 % L, "many": np.arange(M) % L}[order]
    x = np.zeros((M, K))
    A, B = rng.standard_normal((L, R, K)), np.zeros((L, N, R))
    places = np.arange(3) * 80 + 5
    step = 2.0 ** -8 if xt == "bf16" else 2.0 ** -6  # the third is a normal number in float16 too
    x[:, places] = step ** np.arange(3)
    A[:, :, places] = (1 + rng.integers(0, 128, (L, R, 3)) / 128) * rng.choice([-1.0, 1.0], (L, R, 1))
    for n in range(N):
        B[:, n, n % R] = 1
    dev = lambda a, d: torch.from_numpy(a).to(d).cuda()  # noqa: E731
    xd, Ad, Bd = dev(x, t), dev(A, t), dev(B, t)
    got = gpu_lib.adapter_add(torch.zeros(M, N, device="cuda"), xd, Ad, Bd, dev(ids, torch.int32))
    v = np.einsum("mk,mrk->mr", f64(xd)[:, places], f64(Ad)[:, :, places][ids])
    ref = v[:, np.arange(N) % R]
    # float16 operands are pairs of 11 bits against the token's largest of the
    # R sums (below 4); float32 itself would be exact
    check(got, ref, torch.float32, 2 * E * np.abs(ref) + (2 * E * 4 if xt == "f16" else 0))
