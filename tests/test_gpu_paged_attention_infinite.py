"""paged_attention with infinite keys and values among the seen tokens, against
the fp64 definition: a score of minus infinity is a weight of zero, an infinite
value makes its coordinate infinite (of its sign) wherever it has a weight, and
nothing else changes.  Bounds as in test_gpu_paged_attention.py.
"""
import numpy as np
import pytest
import torch

import oracle
from block_cases import DTYPES, E, check, f64
from test_gpu_paged_attention import _bound, _make

pytestmark = pytest.mark.gpu

INF = float("inf")
WIDE = [("bf16", "bf16"), ("f16", "f16")]


def _compare(rbp, made, lengths, xt, fmt, D, window=0, scale=None):
    q, k, v, table, kw, (_, _, _, t64) = made
    k64, v64 = f64(k), f64(v)
    sm = D ** -0.5 if scale is None else scale
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = rbp.paged_attention(q, k, v, table, ln, window=window, scale=scale, return_lse=True, **kw)
    with np.errstate(invalid="ignore"):
        ref, ref_lse = oracle.paged_attention(f64(q), k64, v64, t64, lengths, sm, window)
    o_mag, l_mag = _bound(f64(q), k64, v64, t64, lengths, sm, window, fmt, D)
    check(out, ref, DTYPES[xt], o_mag, "out")
    check(lse, ref_lse, torch.float32, l_mag + 4 * E * np.abs(np.where(np.isfinite(ref_lse), ref_lse, 0)), "lse")
    return ref


@pytest.mark.parametrize("xt,fmt", WIDE)
@pytest.mark.parametrize("D", [8, 24, 40, 64, 72, 80, 96, 112, 128, 144, 192, 248, 256])
@pytest.mark.parametrize("n", [3, 40, 700])
def test_infinite_keys(gpu_lib, xt, fmt, D, n):
    # one infinite coordinate in the last vector of a key: minus infinity for
    # the heads whose query has the other sign there, NaN for the others
    rng = np.random.default_rng(D + n)
    made = _make(rng, [n, n], 8, 2, D, 16, xt, fmt)
    q, k, _, _, _, (_, _, _, t64) = made
    for i, at in enumerate((1, n - 1)):
        k[t64[0, at // 16], :, at % 16, D - 1 - 3 * i] = INF if i else -INF
    q[0, :6, D - 1], q[0, :6, D - 4] = 1.0, -1.0  # these see minus infinity twice
    ref = _compare(gpu_lib, made, [n, n], xt, fmt, D)
    assert np.isfinite(ref[0, :6]).all()


@pytest.mark.parametrize("xt,fmt", WIDE)
@pytest.mark.parametrize("D", [40, 64, 96, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 31, 300, 1500])
def test_infinite_values(gpu_lib, xt, fmt, D, n):
    rng = np.random.default_rng(D * n)
    made = _make(rng, [n, n, n], 8, 2, D, 16, xt, fmt)
    _, _, v, _, _, (_, _, _, t64) = made
    for i, at in enumerate(sorted({0, n // 2, n - 1})):
        v[t64[0, at // 16], :, at % 16, i] = INF
        v[t64[0, at // 16], :, at % 16, D - 1] = -INF
        v[t64[1, at // 16], 1, at % 16, 5] = (-1) ** i * INF  # both signs: NaN
    ref = _compare(gpu_lib, made, [n, n, n], xt, fmt, D)
    assert (ref[0, :, 0] == INF).all() and (ref[0, :, D - 1] == -INF).all() and np.isfinite(ref[0, :, 3:D - 1]).all()
    assert np.isfinite(ref[2]).all()


@pytest.mark.parametrize("xt,fmt", WIDE)
@pytest.mark.parametrize("page", [4, 16])
@pytest.mark.parametrize("gap", [20, 60, 100])
@pytest.mark.parametrize("heavy,light", [(0, 1), (1, 0), (7, 40), (40, 7), (3, 600), (600, 3)])
@pytest.mark.parametrize("empty", [0, 4200])  # requests beside it: the context in pieces, or in one
def test_infinite_values_of_little_weight(gpu_lib, xt, fmt, page, gap, heavy, light, empty):
    # the weight e^-gap is far below what a 16-bit operand holds, and not zero
    D, n = 64, 700
    lengths = [n] + [0] * empty
    rng = np.random.default_rng(gap)
    made = _make(rng, lengths, 2, 1, D, page, xt, fmt, std=2.0 ** -7)
    pieces = gpu_lib.lib.orbit_paged_attention_workspace(len(lengths), 2, 1, D, page, made[3].shape[1], 0, 1) > 0
    assert pieces == (empty == 0)
    q, k, v, _, _, (_, _, _, t64) = made
    q[:], k[t64[0, heavy // page], 0, heavy % page] = 1.0, gap / 8
    k[t64[0, light // page], 0, light % page] = 0
    v[t64[0, light // page], 0, light % page, 9] = -INF
    ref = _compare(gpu_lib, made, lengths, xt, fmt, D, scale=0.125)
    assert (ref[0, :, 9] == -INF).all() and np.isfinite(np.delete(ref, 9, -1)).all()


@pytest.mark.parametrize("xt,fmt", WIDE)
@pytest.mark.parametrize("D", [96, 128])
def test_infinite_values_that_are_not_seen_or_have_no_weight(gpu_lib, xt, fmt, D):
    n, page = 200, 16
    rng = np.random.default_rng(D)
    made = _make(rng, [n, n], 4, 2, D, page, xt, fmt)
    q, k, v, _, _, (_, _, _, t64) = made
    v[t64[0, 0], :, 0] = INF         # before the window
    v[t64[0, n // page], :, n % page:] = -INF  # past the length
    # a weight of zero: finite values add nothing, infinite ones have no product
    q[1, :, 0] = 1.0
    k[t64[1, 9], :, 4, 0] = -INF
    v[t64[1, 9], :, 4, 3] = INF
    ref = _compare(gpu_lib, made, [n, n], xt, fmt, D, window=150)
    assert np.isfinite(ref[0]).all() and np.isnan(ref[1, :, 3]).all() and np.isfinite(ref[1, :, 4:]).all()
