"""paged_tree_attention of requests of few rows (new tokens times the group) beside prompts: their weights are pairs of
16-bit numbers, whatever they are batched with (bounds: tree_cases.py, those of few rows)."""
import numpy as np
import pytest
import torch

import tree_cases
from block_cases import DTYPES, check
from tree_cases import Case, tree_mask

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt,fmt", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "int8"), ("f16", "int8")])
@pytest.mark.parametrize("H,KV,D", [(8, 2, 128), (8, 8, 64), (4, 1, 256), (5, 1, 80), (32, 1, 128)])
@pytest.mark.parametrize("tree", [False, True])
def test_few_rows_beside_a_prompt(gpu_lib, monkeypatch, tree, H, KV, D, xt, fmt):
    few = 32 // (H // KV)
    requests = [(700, 1), (600, 300), (2000, few), (90, max(1, few - 1)), (0, 0), (300, few + 1), (5000, 1)]
    rng = np.random.default_rng(D)
    c = Case(D + H, requests, H=H, KV=KV, D=D, xt=xt, fmt=fmt, masks=[tree_mask(rng, n) if n else np.zeros((0, 0), bool) for _, n in requests] if tree else None)
    out, lse = c.run(gpu_lib, return_lse=True)
    monkeypatch.setattr(tree_cases, "ONE", tree_cases.PAIR)
    want, want_lse, omag, lmag = c.reference()
    for b, (_, n) in enumerate(requests):
        if 0 < n * (H // KV) <= 32:
            rows = slice(c.starts64[b], c.starts64[b] + n)
            check(out[rows], want[rows], DTYPES[xt], omag[rows], "out of request %d" % b)
            check(lse[rows], want_lse[rows], torch.float32, lmag[rows], "lse of request %d" % b)
    monkeypatch.undo()
    c.check(gpu_lib)
