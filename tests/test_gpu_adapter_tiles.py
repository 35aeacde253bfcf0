"""adapter_add above 256 tokens, where tiles of 16 or 64 tokens go through the
matrix cores (few adapters in a tile) or by rows (many): strides, in-place
outputs, odd places, every output type, every width and inner length, large
values, repeats and graphs, each with few and with many adapters in a tile.

Bounds as in test_gpu_adapter.py.
"""
import numpy as np
import pytest
import torch

import oracle
from block_cases import DTYPES, check, draw
from test_gpu_adapter import _mag, _run

pytestmark = pytest.mark.gpu

TOKENS = [257, 300, 1025]  # just past each limit of the token counts


def _ids(order, M, L):
    """Runs of 30 tokens, some without an adapter; or another adapter at every token."""
    return [m // 30 % (L + 1) - 1 for m in range(M)] if order == "few" else [m * 7 % (L + 1) - 1 for m in range(M)]


@pytest.mark.parametrize("order", ["few", "many"])
@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("pad,lead", [(8, 0), (16, 8), (8, 1), (8, 3), (8, 4), (3, 0)])
def test_strided_and_in_place(gpu_lib, order, M, pad, lead):
    ids = _ids(order, M, 20)
    for yt in DTYPES:
        for N in (248, 77):
            _run(gpu_lib, pad, M, 72, N, 16, 20, ids, xt="f16", yt=yt, inplace=True)
            if pad % 8 == 0:  # x's rows are strided alike
                _run(gpu_lib, pad, M, 72, N, 16, 20, ids, pad=pad, lead=lead, yt=yt)
                _run(gpu_lib, pad, M, 72, N, 16, 20, ids, pad=pad, lead=lead, yt=yt, inplace=True)


@pytest.mark.parametrize("order", ["few", "many"])
@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("N", [1, 3, 8, 12, 63, 64, 65, 255, 256, 257, 260, 1000])
@pytest.mark.parametrize("yt", list(DTYPES))
def test_every_width_and_output_type(gpu_lib, order, M, N, yt):
    _run(gpu_lib, N, M, 64, N, 8, 20, _ids(order, M, 20), yt=yt, ranks=[8 - a % 9 for a in range(20)])


@pytest.mark.parametrize("order", ["few", "many"])
@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("K", [8, 24, 120, 136, 520, 1000, 1032, 4096])
def test_every_inner_length(gpu_lib, order, M, K):
    _run(gpu_lib, K, M, K, 72, 16, 20, _ids(order, M, 20), xt="f16")


@pytest.mark.parametrize("order", ["few", "many"])
@pytest.mark.parametrize("M,R", [(257, 8), (300, 24), (300, 128), (1025, 40), (1025, 72), (1025, 104)])
def test_every_rank(gpu_lib, order, M, R):
    ranks = [(R, R - 3, 1, 0, R // 2)[a % 5] for a in range(20)]
    for xt, yt in (("bf16", "f16"), ("f16", "bf16"), ("bf16", "f32")):
        _run(gpu_lib, R, M, 136, 100, R, 20, _ids(order, M, 20), xt=xt, yt=yt, ranks=ranks)


@pytest.mark.parametrize("order", ["few", "many"])
@pytest.mark.parametrize("yt", list(DTYPES))
@pytest.mark.parametrize("M,N", [(1100, 14600), (4100, 4001)])  # 1024 blocks of 64 tokens and 256 columns
def test_tiles_of_64_tokens(gpu_lib, order, yt, M, N):
    _run(gpu_lib, M, M, 72, N, 24, 20, _ids(order, M, 20), xt="f16", yt=yt, inplace=True, ranks=[24 - a for a in range(20)])


@pytest.mark.parametrize("order", ["few", "many"])
@pytest.mark.parametrize("M", TOKENS)
def test_large_values_do_not_overflow_between_the_products(gpu_lib, order, M):
    # A x reaches 4e6, past float16's largest number; B brings it back
    rng = np.random.default_rng(4)
    x, x64 = draw(rng, (M, 512), torch.float16, 2000.0)
    A, A64 = draw(rng, (20, 8, 512), torch.float16, 100.0)
    B, B64 = draw(rng, (20, 64, 8), torch.float16, 1e-4)
    y, y64 = draw(rng, (M, 64), torch.float32)
    ids = _ids(order, M, 20)
    got = gpu_lib.adapter_add(y, x, A, B, torch.tensor(ids, dtype=torch.int32, device="cuda"))
    ref = oracle.adapter_add(y64, x64, A64, B64, ids)
    assert np.abs(ref).max() > 100
    check(got, ref, torch.float32, _mag(y64, x64, A64, B64, ids, None, None, torch.float16))


@pytest.mark.parametrize("M", TOKENS)
def test_repeats_are_identical_on_another_stream_and_in_a_graph(gpu_lib, M):
    rng = np.random.default_rng(6)
    x, _ = draw(rng, (M, 1024), torch.bfloat16)
    y, _ = draw(rng, (M, 136), torch.float32)
    A, _ = draw(rng, (20, 32, 1024), torch.bfloat16, 1 / 32)
    B, _ = draw(rng, (20, 136, 32), torch.bfloat16)
    ids = torch.tensor(_ids("few", M, 20), dtype=torch.int32, device="cuda")
    first = gpu_lib.adapter_add(y, x, A, B, ids)
    out = torch.empty_like(y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = gpu_lib.adapter_add(y, x, A, B, ids, out=out)
    side.synchronize()
    assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.adapter_add(y, x, A, B, ids, out=out)
    for order in ("many", "few", "many"):  # the tiles' forms change between replays
        ids.copy_(torch.tensor(_ids(order, M, 20), dtype=torch.int32))
        x.copy_(draw(rng, (M, 1024), torch.bfloat16)[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, gpu_lib.adapter_add(y, x, A, B, ids))


@pytest.mark.parametrize("M,N", [(300, 72), (1100, 72), (2100, 72), (1100, 14600)])
@pytest.mark.parametrize("height,per", [*((16, n) for n in (1, 7, 8, 9, 16)), *((64, n) for n in (9, 16, 23, 24, 25, 40, 64))])
def test_every_number_of_adapters_in_a_tile(gpu_lib, M, N, height, per):
    # `per` adapters in every `height` tokens, the last of them in runs
    L = 130
    ids = [(m // height * per + min(m % height, per - 1)) % L for m in range(M)]
    _run(gpu_lib, per, M, 72, N, 16, L, ids, xt="f16", yt="bf16", ranks=[16 - a % 4 for a in range(L)])
