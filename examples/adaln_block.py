#!/usr/bin/env python3
"""A causal AdaLN transformer block served from rotated int8 weights.

Several requests, each with its own conditioning vector, its own low-rank
adapter (or none) and its own length, share one block.  A step takes any
number of new tokens of any of them: a prompt is a step with all its tokens, a
decode step one token per request.  Every operator is the library's:

    modulation     rotate, int8_linear          six chunks per request
    norm 1         block_norm                   layer norm, scale and shift
    q, k, v        rotate, int8_linear, adapter_add
    cache          kv_append                    position and Hadamard rotation, int8
    attention      paged_attention
    projection     rotate, int8_linear, adapter_add
    residual       block_norm                   gate, and norm 2 of the sum
    MLP            quant_act, qlinear           8-bit codes, GELU in the epilogue
    residual       block_norm                   gate alone

The rotated x' that int8_linear reads serves the adapters too: their A is
rotated once, beforehand, since A x = (A Pi^T)(Pi x).

    python examples/adaln_block.py              # compares with float64, times a decode step
"""
import argparse
import os
import sys
import time
from dataclasses import dataclass

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import synth  # noqa: E402


@dataclass
class Config:
    dim: int = 1024
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 128
    mlp: int = 4096
    adapters: int = 3
    rank: int = 16
    page_size: int = 16
    pages: int = 64
    max_pages: int = 16     # of one request
    eps: float = 1e-6

    @property
    def qkv(self):
        return (self.q_heads + 2 * self.kv_heads) * self.head_dim


def draw_weights(cfg, seed=0):
    """Random weights of the block's shapes, bfloat16 (adapters float16, the
    type of the rotated rows they read)."""
    g = torch.Generator().manual_seed(seed)

    def draw(*shape, std, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g) * std).to(dtype)

    D, A, R, F = cfg.dim, cfg.adapters, cfg.rank, cfg.q_heads * cfg.head_dim
    return dict(
        mod=draw(6 * D, D, std=0.5 * D ** -0.5), qkv=draw(cfg.qkv, D, std=D ** -0.5), o=draw(D, F, std=F ** -0.5),
        up=draw(cfg.mlp, D, std=D ** -0.5), down=draw(D, cfg.mlp, std=cfg.mlp ** -0.5),
        qkv_a=draw(A, R, D, std=D ** -0.5, dtype=torch.float16), qkv_b=draw(A, cfg.qkv, R, std=0.3 * R ** -0.5, dtype=torch.float16),
        o_a=draw(A, R, F, std=F ** -0.5, dtype=torch.float16), o_b=draw(A, D, R, std=0.3 * R ** -0.5, dtype=torch.float16))


def cos_sin(cfg):
    """float32 [positions, head_dim]: cosines, then sines."""
    n = cfg.page_size * cfg.max_pages
    f = 10000.0 ** (-torch.arange(0, cfg.head_dim, 2, dtype=torch.float64) / cfg.head_dim)
    angle = torch.arange(n, dtype=torch.float64)[:, None] * f
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


class Block:
    """The block on the device: packed weights, rotated adapters, the cache."""

    def __init__(self, cfg, weights, device="cuda"):
        import rotation_bit_ptq_amd as rbp
        self.rbp, self.cfg = rbp, cfg
        w = {k: t.to(device) for k, t in weights.items()}
        F = cfg.q_heads * cfg.head_dim
        self.rot = {d: rbp.Rotation(*synth.rotation_params(d, seed=d), 128, device=device) for d in {cfg.dim, F, cfg.mlp}}
        rot_x, rot_f = self.rot[cfg.dim], self.rot[F]
        self.mod, self.qkv = rbp.int8_pack_weights(rot_x, w["mod"]), rbp.int8_pack_weights(rot_x, w["qkv"])
        self.o = rbp.int8_pack_weights(rot_f, w["o"])
        self.cb_x, self.cb_m = rbp.fit_codebook(cfg.dim, 8), rbp.fit_codebook(cfg.mlp, 8)
        self.up = rbp.pack_weights(rot_x, self.cb_x, w["up"])
        self.down = rbp.pack_weights(self.rot[cfg.mlp], self.cb_m, w["down"])

        def absorbed(rot, a):
            return rbp.rotate(rot, a.view(-1, a.shape[2]).float()).view(a.shape)

        self.qkv_a, self.qkv_b = absorbed(rot_x, w["qkv_a"]), w["qkv_b"]
        self.o_a, self.o_b = absorbed(rot_f, w["o_a"]), w["o_b"]
        self.cos_sin = cos_sin(cfg).to(device)
        shape = (cfg.pages, cfg.kv_heads, cfg.page_size)
        self.k_cache, self.v_cache = (torch.zeros(*shape, cfg.head_dim, dtype=torch.int8, device=device) for _ in "kv")
        self.scales = {n: torch.zeros(shape, dtype=torch.float16, device=device) for n in ("k_scale", "v_scale")}

    def modulation(self, cond):
        """cond [requests, dim] -> six [requests, dim] chunks, views of one projection's output."""
        rbp = self.rbp
        y = rbp.int8_linear(rbp.rotate(self.rot[self.cfg.dim], torch.nn.functional.silu(cond)), *self.mod)
        return y.chunk(6, dim=1)

    def step(self, x, mod, batch):
        """x [tokens, dim] bfloat16, the new tokens; returns the block's output."""
        rbp, cfg, T = self.rbp, self.cfg, len(x)
        shift1, scale1, gate1, shift2, scale2, gate2 = mod
        request, adapter = batch["request"], batch["adapter"]
        rot_x, rot_f = self.rot[cfg.dim], self.rot[cfg.q_heads * cfg.head_dim]

        h = rbp.block_norm(x, norm="layer", scale=scale1, shift=shift1, groups=request, eps=cfg.eps)
        h = rbp.rotate(rot_x, h)
        qkv = rbp.int8_linear(h, *self.qkv)
        qkv = rbp.adapter_add(qkv, h, self.qkv_a, self.qkv_b, adapter, out=qkv)
        q, k, v = qkv.view(T, -1, cfg.head_dim).split([cfg.q_heads, cfg.kv_heads, cfg.kv_heads], dim=1)
        q = rbp.kv_append(k, v, self.k_cache, self.v_cache, batch["slots"], positions=batch["positions"],
                          cos_sin=self.cos_sin, q=q, hadamard=True, **self.scales)
        # every new token is a row of its own, with its request's pages and its own length
        o = rbp.paged_attention(q, self.k_cache, self.v_cache, batch["table"], batch["lengths"], **self.scales)
        o = rbp.rotate(rot_f, o.view(T, -1))
        b = rbp.int8_linear(o, *self.o)
        b = rbp.adapter_add(b, o, self.o_a, self.o_b, adapter, out=b)
        x, h = rbp.block_norm(x, b, norm="layer", gate=gate1, scale=scale2, shift=shift2, groups=request, eps=cfg.eps)

        codes = rbp.quant_act(rot_x, self.cb_x, h)
        u = rbp.qlinear(*codes, self.cb_x, *self.up, self.cb_x, cfg.dim, act="gelu")
        codes = rbp.quant_act(self.rot[cfg.mlp], self.cb_m, u)
        b = rbp.qlinear(*codes, self.cb_m, *self.down, self.cb_m, cfg.mlp)
        return rbp.block_norm(x, b, norm=None, gate=gate2, groups=request)


class Pages:
    """Which pages each request has; the arguments of a step."""

    def __init__(self, cfg, requests, adapters, device="cuda"):
        self.cfg, self.device, self.adapters = cfg, device, adapters
        self.free = list(range(cfg.pages))[::-1]
        self.table = torch.full((requests, cfg.max_pages), -1, dtype=torch.int32)
        self.length = [0] * requests

    def batch(self, tokens):
        """tokens: the number of new tokens of each request."""
        page, request, position = self.cfg.page_size, [], []
        for r, n in enumerate(tokens):
            for p in range(self.length[r], self.length[r] + n):
                if p // page >= self.cfg.max_pages or (self.table[r, p // page] < 0 and not self.free):
                    raise RuntimeError("no page is left for request %d" % r)
                if self.table[r, p // page] < 0:
                    self.table[r, p // page] = self.free.pop()
                request.append(r)
                position.append(p)
            self.length[r] += n
        request, position = torch.tensor(request), torch.tensor(position)
        slots = self.table[request, position // page].long() * page + position % page
        args = dict(request=request.int(), adapter=torch.tensor(self.adapters)[request].int(), slots=slots, positions=position,
                    lengths=(position + 1).int(), table=self.table[request])
        return {k: t.to(self.device) for k, t in args.items()}


def plain(cfg, weights, cond, rows, adapter):
    """One request's tokens `rows` [tokens, dim] through the block, float64 on
    the CPU, unquantized."""
    w = {k: t.double() for k, t in weights.items()}
    x, F = rows.double(), torch.nn.functional
    shift1, scale1, gate1, shift2, scale2, gate2 = (w["mod"] @ F.silu(cond.double())).chunk(6)

    def linear(h, name):
        y = h @ w[name].T
        return y if adapter < 0 else y + h @ w[name + "_a"][adapter].T @ w[name + "_b"][adapter].T

    def norm(v):
        return F.layer_norm(v, (cfg.dim,), eps=cfg.eps)

    T, half = len(x), cfg.head_dim // 2
    qkv = linear(norm(x) * (1 + scale1) + shift1, "qkv").view(T, -1, cfg.head_dim)
    cs = cos_sin(cfg).double()[:T, None]

    def turn(t):
        a, b = t[..., :half], t[..., half:]
        return torch.cat([a * cs[..., :half] - b * cs[..., half:], a * cs[..., half:] + b * cs[..., :half]], dim=-1)

    q, k, v = qkv.split([cfg.q_heads, cfg.kv_heads, cfg.kv_heads], dim=1)
    q, k = turn(q), turn(k)
    out = torch.empty_like(q)
    for h in range(cfg.q_heads):
        g = h * cfg.kv_heads // cfg.q_heads
        z = (q[:, h] @ k[:, g].T * cfg.head_dim ** -0.5).masked_fill(torch.ones(T, T).triu(1).bool(), float("-inf"))
        out[:, h] = z.softmax(-1) @ v[:, g]
    x = x + gate1 * linear(out.reshape(T, -1), "o")
    b = F.gelu((norm(x) * (1 + scale2) + shift2) @ w["up"].T) @ w["down"].T
    return x + gate2 * b


def serve(cfg, weights, prompts, steps, adapters, seed=1, device="cuda"):
    """Prompts of the given lengths in one step, then `steps` decode steps.
    Returns (tokens, outputs, cond): lists by request, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    n = len(prompts)
    cond = torch.randn(n, cfg.dim, generator=g).bfloat16()
    tokens = [torch.randn(p + steps, cfg.dim, generator=g).bfloat16() for p in prompts]
    block, pages = Block(cfg, weights, device), Pages(cfg, n, adapters, device)
    mod = block.modulation(cond.to(device))
    got = block.step(torch.cat([t[:p] for t, p in zip(tokens, prompts)]).to(device), mod, pages.batch(prompts))
    outputs = [[o] for o in got.cpu().split(prompts)]
    for s in range(steps):
        got = block.step(torch.stack([t[p + s] for t, p in zip(tokens, prompts)]).to(device), mod, pages.batch([1] * n))
        for r in range(n):
            outputs[r].append(got[r:r + 1].cpu())
    return tokens, [torch.cat(o) for o in outputs], cond


def deviation(cfg, weights, tokens, outputs, cond, adapters):
    """|output - plain| / |plain - tokens| (norms): the error of what the block
    adds to its input, by request."""
    far = []
    for t, o, c, a in zip(tokens, outputs, cond, adapters):
        want = plain(cfg, weights, c, t, a)
        far.append(float((o.double() - want).norm() / (want - t.double()).norm()))
    return far


def captured(block, x, mod, batch):
    """A decode step as a graph over the given buffers: replay() runs it on
    what they hold.  Returns (graph, output)."""
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):  # once outside the capture: first launches load their code
        block.step(x, mod, batch)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.step(x, mod, batch)
    return graph, out


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=40)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    cfg = Config(pages=16 * a.requests)
    weights = draw_weights(cfg)
    prompts = [max(1, a.prompt - 3 * r) for r in range(a.requests)]
    adapters = [r % (cfg.adapters + 1) - 1 for r in range(a.requests)]
    far = deviation(cfg, weights, *serve(cfg, weights, prompts, a.steps, adapters), adapters)
    print("error of what the block adds, against float64: %.2f %% at most" % (100 * max(far)))

    block, pages = Block(cfg, weights), Pages(cfg, a.requests, adapters)
    mod = block.modulation(torch.randn(a.requests, cfg.dim, device="cuda").bfloat16())
    block.step(torch.randn(sum(prompts), cfg.dim, device="cuda").bfloat16(), mod, pages.batch(prompts))
    x, batch = torch.randn(a.requests, cfg.dim, device="cuda").bfloat16(), pages.batch([1] * a.requests)
    graph, _ = captured(block, x, mod, batch)
    for name, run in (("eager", lambda: block.step(x, mod, batch)), ("graph", graph.replay)):
        for _ in range(5):
            run()
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(50):
            run()
        torch.cuda.synchronize()
        print("decode step of %d requests, %s: %.0f us" % (a.requests, name, (time.perf_counter() - t0) / 50 * 1e6))


if __name__ == "__main__":
    main()
