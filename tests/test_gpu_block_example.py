"""The operators together: the AdaLN block of examples/ against its float64 form.

Bound on the error of what the block adds to its input (relative, in norm),
from the formats' steps alone.  An int8 code of a group of 128 nearly normal
values has step max|w| / 127 with max|w| about 2.7 to 3.2 sigma: rms error
3.2 / 127 / sqrt(12) = 0.73 %.  A 256-level codebook for the normal
distribution has rms error 0.65 %.  A bfloat16 or float16 rounding adds at most
2^-9 / sqrt(3) = 0.11 %.
  modulation 0.75, enters four times (scale, shift, gate of both branches);
  q, k, v: weights 0.73, roundings 0.2; k and v codes 0.8 each (a head of 128);
  logits: q and k off by 1.1 % each on logits of about unit spread: weights of
  the softmax off by 1.6 %, and o by as much of its spread;
  o: 0.73; up: 0.65 twice; down: 0.65 twice.
In quadrature, per branch: sqrt(0.75^2 * 3 + 1.1^2 * 3 + 1.6^2 + 0.73^2) =
2.9 % (attention), sqrt(0.75^2 * 3 + 0.65^2 * 4 + 2.9^2) = 3.4 % (MLP, with
the attention branch's error through the norm).  5 % leaves room for the
spread over draws and lies far below what a wrong page, group, adapter or
position gives (tens of per cent).
"""
import os
import sys

import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import adaln_block as ex  # noqa: E402

pytestmark = pytest.mark.gpu
BOUND = 0.05


@pytest.mark.parametrize("prompts,steps,adapters", [
    ([1], 3, [0]),
    ([17, 1, 33], 2, [-1, 2, 0]),
    ([70, 40, 5, 16, 31], 4, [1, -1, 0, 1, 2]),
])
def test_block_against_plain(gpu_lib, prompts, steps, adapters):
    cfg = ex.Config()
    weights = ex.draw_weights(cfg)
    far = ex.deviation(cfg, weights, *ex.serve(cfg, weights, prompts, steps, adapters), adapters)
    assert max(far) < BOUND, far


def test_decode_in_a_graph(gpu_lib):
    """Replays of a captured step follow its buffers and equal the eager step,
    with eager work in between."""
    cfg = ex.Config()
    weights = ex.draw_weights(cfg)
    prompts, adapters = [9, 30, 16, 1], [0, -1, 1, 2]
    n = len(prompts)
    block, pages = ex.Block(cfg, weights), ex.Pages(cfg, n, adapters)
    g = torch.Generator().manual_seed(3)
    mod = block.modulation(torch.randn(n, cfg.dim, generator=g).bfloat16().cuda())
    block.step(torch.randn(sum(prompts), cfg.dim, generator=g).bfloat16().cuda(), mod, pages.batch(prompts))
    x, batch = torch.empty(n, cfg.dim, device="cuda", dtype=torch.bfloat16), pages.batch([1] * n)
    x.copy_(torch.randn(n, cfg.dim, generator=g))
    graph, out = ex.captured(block, x, mod, batch)
    for _ in range(4):
        want = block.step(x, mod, batch)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        new = pages.batch([1] * n)  # the next token of every request
        for k, t in batch.items():
            t.copy_(new[k])
        x.copy_(torch.randn(n, cfg.dim, generator=g))


def test_pages_run_out():
    pages = ex.Pages(ex.Config(pages=1), 1, [-1], device="cpu")
    pages.batch([16])
    with pytest.raises(RuntimeError, match="no page"):
        pages.batch([1])
