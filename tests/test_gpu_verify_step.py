"""A layer's step over drafted tokens, its operators run after one another as a server would: rotated rows to 8 bits, their
product into queries, keys and values, these normed, turned and appended to the cache, the tree's attention over it, and
the product of the heads' codes back.  Each one is held to its bound in 64 bits from what the one before left; captured in
a graph the whole gives the same bits.
"""
import numpy as np
import pytest
import torch

import test_gpu_int8_qlinear as products
import test_gpu_int8_rows as rows
import test_gpu_qk_norm as norms
from block_cases import DTYPES, check, draw, f64
from tree_cases import Case, tree_mask

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, rbp, seed, requests, masks, fmt="bf16", xt="bf16", d=384, h=128, H=6, KV=2, D=64, **case):
        rng = np.random.default_rng(seed)
        self.rbp, self.dims, self.h, self.xt, self.fmt = rbp, (H, KV, D), h, xt, fmt
        self.c = c = Case(seed, requests, H=H, KV=KV, D=D, xt=xt, fmt=fmt, masks=masks, **case)
        self.rot, self.perm, self.signs = rows.rotation(rbp, d, h)
        self.x, _ = draw(rng, (c.tokens, d), DTYPES[xt])
        wqkv, _ = draw(rng, ((H + 2 * KV) * D, d), DTYPES[xt], d ** -0.5)
        wo, _ = draw(rng, (d, H * D), DTYPES[xt], (H * D) ** -0.5)
        self.wqkv, self.wo = rbp.int8_quant_rows(self.rot, wqkv), rbp.int8_quant_rows(None, wo)
        self.bias = torch.from_numpy(rng.standard_normal((H + 2 * KV) * D)).to(DTYPES[xt]).cuda()
        self.nq, self.nk = (draw(rng, (D,), torch.float32) for _ in "qk")
        places = np.concatenate([np.arange(length - n, length) for length, n in requests])
        pages = np.concatenate([c.table64[b][np.arange(length - n, length) // c.page] for b, (length, n) in enumerate(requests)])
        self.slots = torch.from_numpy((pages.astype(np.int64) * c.page + places % c.page)).cuda()
        depth = places if masks is None else np.concatenate([length - n + m.sum(1) - 1 for (length, n), m in zip(requests, masks)])
        self.at = depth
        self.positions, self.cos_sin = torch.from_numpy(depth.astype(np.int64)).cuda(), norms.table(max(n for n, _ in requests), D)

    def split(self, qkv):
        H, KV, D = self.dims
        heads = qkv.view(-1, H + 2 * KV, D)
        return heads[:, :H], heads[:, H:H + KV], heads[:, H + KV:]

    def append(self, qkv):
        q, k, v = self.split(qkv)
        return self.rbp.kv_append(k, v, self.c.k, self.c.v, self.slots, q=q, positions=self.positions, cos_sin=self.cos_sin, norm="rms",
                                  q_weight=self.nq[0], k_weight=self.nk[0], **self.c.kw)

    def attend(self, q):
        self.c.q = q
        return self.c.run(self.rbp)

    def step(self, out=None):
        qkv = self.rbp.int8_qlinear(*self.rbp.int8_quant_rows(self.rot, self.x), *self.wqkv, bias=self.bias, out_dtype=DTYPES[self.xt])
        o = self.attend(self.append(qkv))
        return self.rbp.int8_qlinear(*self.rbp.int8_quant_rows(None, o.flatten(1)), *self.wo, out_dtype=torch.float32, out=out)

    def check(self):
        H, KV, D = self.dims
        rbp, c, t = self.rbp, self.c, DTYPES[self.xt]
        qx, sx = rbp.int8_quant_rows(self.rot, self.x)
        rows.against(qx, sx, f64(self.x), self.perm, self.signs, self.h)
        qkv = rbp.int8_qlinear(qx, sx, *self.wqkv, bias=self.bias, out_dtype=t)
        want, mag = products.reference(qx, sx, *self.wqkv, self.bias, None)
        check(qkv, want, t, mag, "q, k, v")
        q = self.append(qkv)
        cs = f64(self.cos_sin)[self.at]
        raw_q, raw_k, raw_v = self.split(qkv)
        want, mag = norms.turned(*norms.normed(f64(raw_q), self.nq[1], "rms"), cs, D, False, False)
        check(q, want, t, mag, "q")
        page, off = self.slots // c.page, self.slots % c.page
        want, mag = norms.turned(*norms.normed(f64(raw_k), self.nk[1], "rms"), cs, D, False, False)
        if self.fmt == "int8":
            s = f64(c.kw["k_scale"][page, :, off])[..., None]
            top = np.abs(want).max(-1, keepdims=True) / 127
            wide = top * 2.0 ** -11 * (1 + 2.0 ** -9) + mag.max(-1, keepdims=True) / 127 + 2.0 ** -25
            assert (np.abs(s - top) <= wide).all()
            assert (np.abs(f64(c.k[page, :, off]) * s - want) <= s * 0.5 * (1 + 2.0 ** -10) + 127 * np.abs(s - top) + mag).all()
        else:
            check(c.k[page, :, off], want, DTYPES[self.fmt], mag, "k")
            assert torch.equal(c.v[page, :, off], raw_v.to(DTYPES[self.fmt]))
        c.q, c.q64 = q, f64(q)
        o = c.check(rbp)
        qo, so = rbp.int8_quant_rows(None, o.flatten(1))
        rows.against(qo, so, f64(o.flatten(1)), None, None, 0)
        y = rbp.int8_qlinear(qo, so, *self.wo, out_dtype=torch.float32)
        want, mag = products.reference(qo, so, *self.wo, None, None)
        check(y, want, torch.float32, mag, "y")
        assert torch.equal(self.step(), y)


@pytest.mark.parametrize("xt,fmt", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "int8")])
def test_trees(gpu_lib, xt, fmt):
    rng = np.random.default_rng(5)
    requests = [(90, 7), (400, 12), (5, 5)]
    Layer(gpu_lib, 1, requests, [tree_mask(rng, n) for _, n in requests], fmt, xt).check()


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_runs_behind_a_window_with_sinks(gpu_lib, fmt):
    Layer(gpu_lib, 2, [(300, 70), (33, 33), (129, 1)], None, fmt, window=50, sinks=4, D=128, H=4, KV=1, d=512).check()


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_graph_of_the_step(gpu_lib, fmt):
    rng = np.random.default_rng(6)
    requests = [(700, 9), (64, 4)]
    layer = Layer(gpu_lib, 3, requests, [tree_mask(rng, n) for _, n in requests], fmt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty(layer.c.tokens, layer.x.shape[1], device="cuda")
    with torch.cuda.stream(side):
        layer.step(out)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            layer.step(out)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(3):
        layer.x.copy_(draw(rng, tuple(layer.x.shape), DTYPES["bf16"])[0])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(layer.step(), got)


def test_two_steps_at_once(gpu_lib):
    """Each on a stream of its own, with workspaces of their own."""
    rng = np.random.default_rng(7)
    layers = [Layer(gpu_lib, 10 + i, [(3000, 6), (500 * i + 40, 3)], [tree_mask(rng, 6), tree_mask(rng, 3)]) for i in range(2)]
    want = [layer.step() for layer in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        got = []
        for layer, stream in zip(layers, streams):
            with torch.cuda.stream(stream):
                got.append(layer.step())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
