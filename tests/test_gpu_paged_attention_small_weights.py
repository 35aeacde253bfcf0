"""paged_attention where small weights decide: a dominant token whose value is
zero (the place where attention that has nothing to attend to goes), so that
the output is made of the other tokens alone.

Bounds.  A score is a sum of D products on the matrix cores (depth D / 32 + 36)
and its error dz enters the weight as a relative 2 dz; sums over n tokens add
(n / 128 + 60) E, as in the other tests of the operator.  Weights are
multiplied as pairs of 16-bit numbers: within 2^-15 of themselves (bfloat16),
or 2^-19 and 2^-39 of the largest weight (float16 operands: float16 and int8
caches), whichever is more.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from block_cases import DTYPES, E, check

pytestmark = pytest.mark.gpu

FORMS = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "int8"), ("f16", "int8")]
PAIR = {"bf16": (2.0 ** -15, 0.0), "f16": (2.0 ** -19, 2.0 ** -39), "int8": (2.0 ** -19, 2.0 ** -39)}


@pytest.mark.parametrize("xt,fmt", FORMS)
@pytest.mark.parametrize("gap", [6, 9, 12, 15, 18, 20])  # of the scores; a weight of e^-20 is 2^-29
@pytest.mark.parametrize("n,sink", [(33, 0), (33, 32), (2000, 5), (2000, 1999)])
def test_a_dominant_token_of_zero_value(gpu_lib, xt, fmt, gap, n, sink):
    D, page, sm = 64, 16, 0.125
    rng = np.random.default_rng(n + gap)
    pages = -(-n // page)
    # scores: sm * 64 * gap / 8 = gap for the one token, 0 for the others, all of it exact
    k = np.zeros((pages * page, 1, D))
    k[sink] = gap / 8
    v = rng.integers(64, 128, k.shape) * 128.0  # 8192 .. 16256, exact in every format
    v[sink] = 0
    rows = lambda t: np.ascontiguousarray(t.reshape(pages, page, 1, D).transpose(0, 2, 1, 3))  # noqa: E731
    k64, v64 = rows(k), rows(v)
    kw = {}
    if fmt == "int8":
        # codes and a scale each; the dominant token's codes are zeros of the others' scale
        ks, vs = np.full(k64.shape[:3], gap / 512), np.full(k64.shape[:3], 128.0)
        kc, vc = (torch.from_numpy((t / s[..., None]).astype(np.int8)).cuda() for t, s in ((k64, ks), (v64, vs)))
        kw = dict(k_scale=torch.from_numpy(ks).half().cuda(), v_scale=torch.from_numpy(vs).half().cuda())
    else:
        kc, vc = (torch.from_numpy(t).to(DTYPES[fmt]).cuda() for t in (k64, v64))
    q = torch.ones(1, 2, D, dtype=DTYPES[xt], device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    out, lse = gpu_lib.paged_attention(q, kc, vc, table, torch.tensor([n], dtype=torch.int32, device="cuda"), scale=sm,
                                       return_lse=True, **kw)
    ref, ref_lse = oracle.paged_attention(np.ones((1, 2, D)), k64, v64, table.cpu().numpy(), [n], sm)
    dz = (D / 32 + 36) * E * gap
    rel = 2 * dz + PAIR[fmt][0] + (n / 128 + 60) * E
    # the largest weight is 1 of a sum of 1 + (n - 1) e^-gap
    lost = PAIR[fmt][1] * np.abs(v[:n]).sum() / D / (1 + (n - 1) * math.exp(-gap))
    check(out, ref, DTYPES[xt], rel * np.abs(ref) + lost, "out")
    check(lse, ref_lse, torch.float32, rel + 4 * E * np.abs(ref_lse), "lse")
