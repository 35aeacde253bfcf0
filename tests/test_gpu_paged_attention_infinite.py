"""paged_attention with infinite keys among the seen tokens, against the fp64
definition: a score of minus infinity is a weight of zero.  Bounds as in test_gpu_paged_attention.py.
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
