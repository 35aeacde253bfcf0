"""paged_tree_attention with a score scale of zero, or so small that it is none beside small queries: every token that is
seen weighs the same, and hidden ones stay hidden (bounds: tree_cases.py)."""
import numpy as np
import pytest

from tree_cases import Case, tree_mask

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt,fmt", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "int8"), ("f16", "int8")])
@pytest.mark.parametrize("scale,small", [(0.0, 0), (0.0, -10), (0.0, -40), (0.0, -100), (1e-30, -40), (-1e-30, -40), (1e-38, -24)])
@pytest.mark.parametrize("n,tree", [(3, False), (70, False), (9, True), (60, True)])
def test_scores_of_no_size(gpu_lib, n, tree, scale, small, xt, fmt):
    rng = np.random.default_rng(n)
    requests = [(300, n), (n, n), (77, 2)]
    c = Case(n, requests, H=4, KV=2, xt=xt, fmt=fmt, scale=scale, masks=[tree_mask(rng, m) for _, m in requests] if tree else None)
    c.q *= 2.0 ** small
    c.q64 = c.q.double().cpu().numpy()
    c.check(gpu_lib)
