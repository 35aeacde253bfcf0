"""More operators of a served block, as cases.

Operators: `product` (the matrix product of 8-bit integers with a scale for each token and each channel, on codes that
are at hand, or as a `layer` that rotates and codes its tokens first), `heads` (norms of queries and keys for each head
with the position rotation in the same pass, alone or on the way into the paged cache), `attend` (attention over the
paged cache for a tree of drafted tokens, for a run of new tokens, and for single tokens; with a sliding window and a
few first tokens that stay visible).  `run` computes a case's operator in its plain form, or with this package's
kernels where `own` is set.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "int8": 1}


def listed():
    return [
        # the AdaLN projection of 16 conditioning vectors: the weights' bytes and the two launches count
        dict(name="layer_adaln", op="layer", tokens=16, k=3072, n=18432, x="bf16", y="bf16", h=128, bias=True, gelu=False),
        # the image layer: 4096 tokens of outlier channels, rotated and coded, then the product
        dict(name="layer_image", op="layer", tokens=4096, k=3072, n=3072, x="bf16", y="bf16", h=128, bias=True, gelu=False),
        # the weight-only layers' largest shape, on codes
        dict(name="product_prompt", op="product", tokens=16384, k=4096, n=4096, y="bf16", bias=False, gelu=False),
        # a continuous batch into an MLP's hidden layer: sizes that are no whole tiles
        dict(name="product_ragged", op="product", tokens=333, k=2064, n=8200, y="f32", bias=True, gelu=True),
        # one decode step of 64 requests into a 16-bit cache: latency counts
        dict(name="heads_decode", op="heads", tokens=64, q_heads=32, kv_heads=8, dim=128, rot=128, x="bf16", w="bf16", norm="rms",
             each=False, interleaved=False, fmt="bf16", page=16, mix="decode"),
        # the image layer's joint attention: queries and keys of 4096 tokens, no cache
        dict(name="heads_image", op="heads", tokens=4096, q_heads=24, kv_heads=24, dim=128, rot=128, x="bf16", w="f32", norm="rms",
             each=False, interleaved=True, fmt="none", page=16, mix="prompt"),
        # a tree of 8 drafted tokens of one request with a short history: latency counts
        dict(name="tree_short", op="attend", form="tree", batch=1, new=8, q_heads=32, kv_heads=8, dim=128, page=16, length=700,
             x="bf16", fmt="bf16", window=0, sinks=0, ragged=False),
        # a serving batch, up to 60 drafted tokens each, histories of very different lengths
        dict(name="tree_batch", op="attend", form="tree", batch=16, new=60, q_heads=32, kv_heads=8, dim=128, page=16, length=8192,
             x="bf16", fmt="bf16", window=0, sinks=0, ragged=True),
        # long histories in the int8 cache, small trees, six query heads to a key head
        dict(name="tree_long", op="attend", form="tree", batch=8, new=16, q_heads=24, kv_heads=4, dim=128, page=64, length=65000,
             x="f16", fmt="int8", window=0, sinks=0, ragged=True),
        # decoding behind a window with four sinks, histories far longer than the window
        dict(name="sinks_decode", op="attend", form="single", batch=64, new=1, q_heads=32, kv_heads=8, dim=128, page=16, length=16384,
             x="bf16", fmt="bf16", window=4096, sinks=4, ragged=True),
        # prompts behind a window with sinks
        dict(name="sinks_prompt", op="attend", form="run", batch=4, new=4096, q_heads=32, kv_heads=8, dim=128, page=16, length=8192,
             x="bf16", fmt="bf16", window=1024, sinks=16, ragged=True),
        # the last piece of one long prompt, all of it visible
        dict(name="run_prompt", op="attend", form="run", batch=1, new=4096, q_heads=32, kv_heads=8, dim=128, page=64, length=8192,
             x="bf16", fmt="bf16", window=0, sinks=0, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("layer", "product", "heads", "attend", "attend"))
    if op in ("layer", "product"):
        h = rng.choice((0, 64, 128, 128, 256))
        k = h * _log(rng, 4, 12288 // h) if op == "layer" and h else 16 * _log(rng, 16, 768)
        n = rng.choice((_log(rng, 16, 18432), 128 * _log(rng, 4, 144)))
        c = dict(op=op, tokens=max(1, min(_log(rng, 1, 16384), int(16384 * 4096 * 4096 / (k * n)))), k=k, n=n)
        if op == "layer":
            c.update(x=rng.choice(("bf16", "bf16", "f32", "f16")), h=h)
        return dict(c, y=rng.choice(("bf16", "bf16", "f32", "f16")), bias=rng.random() < 0.5, gelu=rng.random() < 0.3)
    dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    page = rng.choice((8, 16, 64, 256))
    if op == "heads":
        heads = kv_heads * rng.choice((1, 4, 5, 8))
        mix = rng.choice(("decode", "prompt"))
        most = max(300, min(16384, 4096 * 48 * 128 // (dim * (heads + 2 * kv_heads))))
        return dict(op="heads", tokens=_log(rng, 1, 256) if mix == "decode" else _log(rng, 100, most), q_heads=heads, kv_heads=kv_heads,
                    dim=dim, rot=rng.choice((dim, dim, dim // 2)), x=rng.choice(("bf16", "f16")), w=rng.choice(("f32", "bf16")),
                    norm=rng.choice(("rms", "rms", "layer")), each=rng.random() < 0.3, interleaved=rng.random() < 0.5,
                    fmt=rng.choice(("none", "x", "int8")), page=page, mix=mix)
    heads = kv_heads * rng.choice((1, 4, 5, 8, 16))
    x, fmt = rng.choice((("bf16", "bf16"), ("f16", "f16"), ("bf16", "int8"), ("f16", "int8")))
    form = rng.choice(("tree", "tree", "run", "single"))
    window = rng.choice((0, 0, 333, 2048)) if form != "single" else rng.choice((333, 2048))
    c = dict(op="attend", form=form, batch=_log(rng, 1, 32), q_heads=heads, kv_heads=kv_heads, dim=dim, page=page, x=x, fmt=fmt,
             window=window, sinks=rng.choice((0, 1, 4, 40)) if window else 0, ragged=rng.random() < 0.7)
    if form == "run":  # pairs of queries and keys as in the longest listed run at most
        c["batch"] = _log(rng, 1, 8)
        c["new"] = _log(rng, 20, max(40, min(4096, 4096 * 32 * 128 // (c["batch"] * heads * dim))))
        c["length"] = c["new"] + _log(rng, 1, max(2, 8192 - c["new"]))
    else:
        c["new"] = 1 if form == "single" else _log(rng, 2, 64)
        c["length"] = c["new"] + _log(rng, 50, max(100, min(65000, 16 * 8192 * 8 * 128 // (c["batch"] * kv_heads * dim))))
    return c


# ---- what a case fixes apart from its values ---------------------------------------------------------------------


def _requests(c):
    """(length, new tokens) of each request; in a ragged batch some with one new token, or with none."""
    B, out = c["batch"], []
    for i in range(B):
        part = (i * 37) % B + 1
        n, new = c["length"], c["new"]
        if c["ragged"]:
            new = max(1, new * (B - (part * 5) % B) // B)
            n = max(new, n * part // B)
            if i % 16 == 5:
                new = min(new, 1)
            if i % 16 == 9 and c["form"] != "single":
                new = 0
        out.append((n, new))
    return out


def _parents(n, i):
    """A tree of n drafted tokens, each one's parent before it: some long branches, some short ones."""
    return [-1] + [max(0, j - 1 - (j * (i + 3) + j // 7) % min(j, 5)) for j in range(1, n)]


def _seen(c, n, new, i):
    """[new, n]: what each new token of request i sees (numpy)."""
    t, j = np.arange(n)[None, :], np.arange(new)[:, None]
    if c["form"] == "tree":
        mask = np.zeros((new, new), bool)
        for a, p in enumerate(_parents(new, i)[:new]):
            mask[a] = mask[p] if p >= 0 else False
            mask[a, a] = True
        at = n - new + mask.sum(1)[:, None] - 1
        seen = np.concatenate([np.ones((new, n - new), bool), mask], 1)
    else:
        at = n - new + j
        seen = t <= at
        mask = None
    if c["window"]:
        inside = (t > at - c["window"]) | (t < c["sinks"])
        if mask is not None:
            inside |= t >= n - new
        seen = seen & inside
    return seen, mask


def work(case):
    c = case
    if c["op"] in ("layer", "product"):
        M, K, N = c["tokens"], c["k"], c["n"]
        read = M * K * SIZE[c["x"]] if c["op"] == "layer" else M * (K + 4)
        return {"bytes": read + N * (K + 4) + M * N * SIZE[c["y"]] + (4 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    H, KV, D = c["q_heads"], c["kv_heads"], c["dim"]
    if c["op"] == "heads":
        T, wide, fmt = c["tokens"], SIZE[c["x"]], c["x"] if c["fmt"] == "x" else c["fmt"]
        if fmt == "none":
            moved = 2 * T * D * (H + KV) * wide + T * (8 + 4 * c["rot"])
        else:
            moved = T * D * (2 * H + 2 * KV) * wide + T * (16 + 4 * c["rot"]) + T * KV * (2 * D * SIZE[fmt] + (4 if fmt == "int8" else 0))
            if fmt == "int8":  # read back
                moved += T * KV * (2 * D * (1 + wide) + 4)
        return {"bytes": moved, "flops": T * D * 12 * (H + KV)}
    kept = pairs = tokens = 0
    for i, (n, new) in enumerate(_requests(c)):
        seen, _ = _seen(c, n, new, i)
        kept += int(seen.any(0).sum()) if new else 0
        pairs += int(seen.sum())
        tokens += new
    row = KV * (2 * D * SIZE[c["fmt"]] + (4 if c["fmt"] == "int8" else 0))
    return {"bytes": kept * row + 2 * tokens * H * D * SIZE[c["x"]], "flops": 4 * pairs * H * D}


# ---- inputs ------------------------------------------------------------------------------------------------------


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _hadamard(n, dtype):
    h = torch.ones(1, 1, dtype=dtype, device="cuda")
    while h.shape[0] < n:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h * n ** -0.5


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    return dict(globals()["_prepare_" + c["op"]](c, g), case=c)


def _coded(x):
    """Rows in 8 bits: codes, and a float32 scale each."""
    s = x.abs().amax(-1) / 127.0
    q = torch.where(s[:, None] > 0, torch.round(x / s[:, None]), 0.0).clamp(-127, 127)
    return q.to(torch.int8), s


def _rotated(x, s, c):
    if not c["h"]:
        return x
    y = (x[:, s["perm"]] * s["signs"].to(x.dtype)).reshape(-1, c["h"]) @ _hadamard(c["h"], x.dtype)
    return y.reshape(x.shape)


def _prepare_layer(c, g):
    M, K, N = c["tokens"], c["k"], c["n"]
    s = dict(bias=_randn(g, N) if c["bias"] else None, rot=None, perm=None, signs=None)
    # a few channels far larger than the others, and tokens of different sizes
    chan = torch.where(torch.rand(K, generator=g, device="cuda") < 0.005, 50.0, 1.0)
    size = torch.exp(0.5 * torch.randn(M, 1, generator=g, device="cuda"))
    s["x"] = (_randn(g, M, K) * chan * size).to(DT[c["x"]])
    if c["h"]:
        s["perm"] = torch.randperm(K, generator=g, device="cuda")
        s["signs"] = 1.0 - 2.0 * torch.randint(0, 2, (K,), generator=g, device="cuda")
    s["qw"], s["sw"] = _coded(_rotated(_randn(g, N, K, std=K ** -0.5), s, c))  # packed once, before it is served
    if own and c["h"]:
        import rotation_bit_ptq_amd as rbp
        s["rot"] = rbp.Rotation(s["perm"].cpu().numpy(), s["signs"].cpu().numpy(), c["h"], s["x"].device)
    return s


def _prepare_product(c, g):
    M, K, N = c["tokens"], c["k"], c["n"]
    qx, sx = _coded(_randn(g, M, K))
    qw, sw = _coded(_randn(g, N, K, std=K ** -0.5))
    return dict(qx=qx, sx=sx, qw=qw, sw=sw, bias=_randn(g, N) if c["bias"] else None)


def _prepare_heads(c, g):
    T, H, KV, D, page, t = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"], c["page"], DT[c["x"]]
    chan = torch.ones(H + 2 * KV, D, device="cuda")
    chan[:, 3::32] = 8.0  # the outlier channels that queries and keys have
    qkv = (_randn(g, T, H + 2 * KV, D) * chan).to(t)  # one projection's output, split without a copy
    q, k, v = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
    most = 32768
    if c["mix"] == "decode":  # each token in a page of its own
        pages = T + 3
        slots = torch.randperm(pages, generator=g, device="cuda")[:T] * page + torch.randint(0, page, (T,), generator=g, device="cuda")
        positions = torch.randint(0, most, (T,), generator=g, device="cuda")
    else:  # prompts one after the other, their pages anywhere
        pages = -(-T // page)
        table = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(T, device="cuda")
        slots, positions = table[at // page] * page + at % page, at % max(1, -(-T // 3))
    angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
    wq, wk = ((1 + _randn(g, *((n, D) if c["each"] else (D,)), std=0.2)).to(DT[c["w"]]) for n in (H, KV))
    s = dict(q=q, k=k, v=v, wq=wq, wk=wk, slots=slots, positions=positions, cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(),
             k_scale=None, v_scale=None)
    if c["fmt"] != "none":
        ct = torch.int8 if c["fmt"] == "int8" else t
        s.update({n + "_cache": torch.zeros(pages, KV, page, D, dtype=ct, device="cuda") for n in "kv"})
    if c["fmt"] == "int8":
        s.update({n + "_scale": torch.zeros(pages, KV, page, dtype=torch.float16, device="cuda") for n in "kv"})
    return s


def _words(mask):
    """Rows of truth values as 64-bit words, bit j of word w for token 64 w + j."""
    pad = np.zeros((mask.shape[0], 64), np.uint64)
    pad[:, : mask.shape[1]] = mask
    return (pad << np.arange(64, dtype=np.uint64)).sum(1, dtype=np.uint64).view(np.int64)[:, None]


def _prepare_attend(c, g):
    B, H, KV, D, page, t = c["batch"], c["q_heads"], c["kv_heads"], c["dim"], c["page"], DT[c["x"]]
    requests = _requests(c)
    need = [-(-n // page) for n, _ in requests]
    width, pages = max(need), sum(need)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table, at = torch.zeros(B, width, dtype=torch.int32, device="cuda"), 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    new = [m for _, m in requests]
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    seen = [_seen(c, n, m, i) for i, (n, m) in enumerate(requests)]
    s = dict(q=_randn(g, int(starts[-1]), H, D, dtype=t, std=2.0), table=table, k_scale=None, v_scale=None, tree=None,
             lengths=torch.tensor([n for n, _ in requests], dtype=torch.int32, device="cuda"),
             starts=torch.from_numpy(starts).cuda())
    if c["form"] == "tree":
        s["tree"] = torch.from_numpy(np.concatenate([_words(m) for _, m in seen])).cuda()
    # the plain form's mask: made with the tree, before the layers that all use it
    s["seen"] = [torch.from_numpy(m).cuda() for m, _ in seen]
    if c["fmt"] == "int8":
        for n in "kv":
            s[n + "_cache"] = torch.randint(-127, 128, (pages, KV, page, D), generator=g, device="cuda", dtype=torch.int8)
            s[n + "_scale"] = ((0.5 + torch.rand(pages, KV, page, generator=g, device="cuda")) / 73).half()
    else:
        for n in "kv":
            s[n + "_cache"] = torch.empty(pages, KV, page, D, dtype=t, device="cuda").normal_(generator=g)
    return s


# ---- one pass ----------------------------------------------------------------------------------------------------


def run(state):
    s, c = state, state["case"]
    if not own:
        return globals()["_plain_" + c["op"]](s, c)
    import rotation_bit_ptq_amd as rbp
    if c["op"] in ("layer", "product"):
        q, scale = rbp.int8_quant_rows(s["rot"], s["x"]) if c["op"] == "layer" else (s["qx"], s["sx"])
        return rbp.int8_qlinear(q, scale, s["qw"], s["sw"], bias=s["bias"], out_dtype=DT[c["y"]], act="gelu" if c["gelu"] else None)
    if c["op"] == "heads":
        how = dict(norm=c["norm"], q_weight=s["wq"], k_weight=s["wk"], positions=s["positions"], cos_sin=s["cos_sin"],
                   interleaved=c["interleaved"])
        if c["fmt"] == "none":
            return rbp.qk_norm(s["q"], s["k"], **how)
        q = rbp.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], q=s["q"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                          hadamard=c["fmt"] == "int8", **how)
        if c["fmt"] != "int8":
            return q, s["k_cache"], s["v_cache"]
        k, v = rbp.kv_read(s["k_cache"], s["v_cache"], s["slots"], k_scale=s["k_scale"], v_scale=s["v_scale"], dtype=DT[c["x"]])
        return q, k, v, s["k_scale"], s["v_scale"]
    how = dict(window=c["window"], sinks=c["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=True)
    if c["form"] == "single":
        return rbp.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], **how)
    return rbp.paged_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["starts"], tree=s["tree"], **how)


EPS = 1e-6


def _plain_product(s, c):
    return _finished((s["qx"].float() @ s["qw"].float().t()) * s["sx"][:, None] * s["sw"], s, c)


def _plain_layer(s, c):
    # a code next to a half is decided in 64 bits, and without the rotation's factor, so that a tie stays one: in 32 bits
    # some 1e-6 of the codes fall to the other side, which moves a float32 output by 3e-5 of its norm
    x, h = s["x"].double(), c["h"] or 1
    if c["h"]:
        ones = (_hadamard(h, torch.float64) * h ** 0.5).round()
        x = ((x[:, s["perm"]] * s["signs"].double()).reshape(-1, h) @ ones).reshape(x.shape)
    top = x.abs().amax(-1, keepdim=True)
    qx = torch.where(top > 0, torch.round(127 * x / top), 0.0)
    sx = (top[:, 0] / (127 * h ** 0.5)).float()
    return _finished((qx.float() @ s["qw"].float().t()) * sx[:, None] * s["sw"], s, c)


def _finished(y, s, c):
    if c["bias"]:
        y = y + s["bias"]
    if c["gelu"]:
        y = 0.5 * y * (1 + torch.erf(y * 0.5 ** 0.5))
    return y.to(DT[c["y"]])


def _normed(x, w, c):
    if c["norm"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _turned(x, s, c):
    """The position rotation of the first `rot` coordinates of each head."""
    r = c["rot"]
    t = s["cos_sin"][s["positions"]][:, None, :]
    cos, sin = t[..., : r // 2], t[..., r // 2:]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        out = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2: r]
        out = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([out, x[..., r:]], -1)


def _plain_heads(s, c):
    page, t = c["page"], DT[c["x"]]
    q, k = (_turned(_normed(s[n].float(), s["w" + n], c), s, c) for n in "qk")
    if c["fmt"] == "none":
        return q.to(t), k.to(t)
    v, pg, at = s["v"].float(), s["slots"] // page, s["slots"] % page
    if c["fmt"] != "int8":
        s["k_cache"][pg, :, at] = k.to(t)
        s["v_cache"][pg, :, at] = v.to(t)
        return q.to(t), s["k_cache"], s["v_cache"]
    h = _hadamard(c["dim"], torch.float32)
    q, k = q @ h, k @ h
    back = []
    for n, x in (("k", k), ("v", v)):
        scale = (x.abs().amax(-1, keepdim=True) / 127.0).half()
        code = torch.where(scale > 0, torch.round(x / scale.float()), 0.0).clamp(-127, 127)
        s[n + "_cache"][pg, :, at], s[n + "_scale"][pg, :, at] = code.to(torch.int8), scale[..., 0]
        back.append((s[n + "_cache"][pg, :, at].float() * s[n + "_scale"][pg, :, at].float()[..., None]).to(t))
    return q.to(t), *back, s["k_scale"], s["v_scale"]


def _plain_attend(s, c):
    # one request after the other, as their sizes differ
    H, KV, D, page = c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    outs, lses, at = [], [], 0
    for i, (n, new) in enumerate(_requests(c)):
        if new == 0:
            continue
        pages = s["table"][i, : -(-n // page)].long()

        def rows(name):  # [KV, n, D]
            x = s[name + "_cache"][pages].float()
            if s[name + "_scale"] is not None:
                x = x * s[name + "_scale"][pages].float()[..., None]
            return x.transpose(0, 1).reshape(KV, -1, D)[:, :n]

        q = s["q"][at:at + new].float().reshape(new, KV, H // KV, D).permute(1, 2, 0, 3).reshape(KV, -1, D)
        z = (q @ rows("k").transpose(1, 2)).reshape(KV, H // KV, new, n) * D ** -0.5
        z = torch.where(s["seen"][i], z, float("-inf"))
        m = z.amax(-1, keepdim=True)
        p = torch.exp(z - torch.where(m > float("-inf"), m, 0.0))
        total = p.sum(-1, keepdim=True)
        o = (p.reshape(KV, -1, n) @ rows("v")).reshape(KV, H // KV, new, D) / torch.where(total > 0, total, 1.0)
        outs.append(o.permute(2, 0, 1, 3).reshape(new, H, D).to(DT[c["x"]]))
        lses.append((m + torch.log(total)).reshape(H, new).t())
        at += new
    return torch.cat(outs), torch.cat(lses)


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return globals()["_exact_" + case["op"]](s, case)


def _fwht(x, h):
    """Blocks of h of the last axis, a factor of two at a time; without the factor 1 / sqrt(h)."""
    shape, n = x.shape, 1
    while n < h:
        x = x.reshape(-1, 2, n)
        x = torch.stack([x[:, 0] + x[:, 1], x[:, 0] - x[:, 1]], 1)
        n *= 2
    return x.reshape(shape)


def _exact_product(s, c):
    if c["tokens"] * c["k"] * c["n"] > 1 << 40:
        return None
    y = torch.mm(s["qx"].double(), s["qw"].double().t().contiguous())
    y = torch.diag(s["sx"].double()) @ y if c["tokens"] <= 64 else y.mul_(s["sx"].double().unsqueeze(1))
    y = y.mul_(s["sw"].double().unsqueeze(0))
    if c["bias"]:
        y = y.add_(s["bias"].double())
    return y * torch.special.ndtr(y) if c["gelu"] else y


def _exact_layer(s, c):
    x = s["x"].double()
    if c["h"]:
        x = _fwht(x.index_select(1, s["perm"]).mul_(s["signs"].double()), c["h"])
    most = x.abs().max(1).values
    q = (x * 127 / most.clamp_min(1e-300).unsqueeze(1)).round_()
    return _exact_product(dict(s, qx=q, sx=most / 127 / math.sqrt(c["h"] or 1)), c)


def _exact_heads(s, c):
    D, r, page = c["dim"], c["rot"], c["page"]
    # cosines and sines are inputs, rounded to 32 bits: the pair's product with them as a complex number
    turn = torch.complex(*(s["cos_sin"][s["positions"]].double().reshape(-1, 1, 2, r // 2).unbind(2)))

    def done(x, w):
        x = x.double()
        mean = x.sum(2, keepdim=True) / D if c["norm"] == "layer" else 0.0
        x = (x - mean) / (((x - mean) ** 2).sum(2, keepdim=True) / D + EPS).sqrt() * w.double()
        first = slice(0, r, 2) if c["interleaved"] else slice(0, r // 2)
        second = slice(1, r, 2) if c["interleaved"] else slice(r // 2, r)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q, k, v = done(s["q"], s["wq"]), done(s["k"], s["wk"]), s["v"].double()
    if c["fmt"] == "none":
        return q, k
    pg, at = s["slots"] // page, s["slots"] % page
    if c["fmt"] != "int8":
        full = [torch.zeros(s["k_cache"].shape, dtype=torch.float64, device="cuda") for _ in "kv"]
        full[0][pg, :, at], full[1][pg, :, at] = k, v
        return q, *full
    q, k = _fwht(q, D) / math.sqrt(D), _fwht(k, D) / math.sqrt(D)
    values, scales = [], []
    for x in (k, v):
        sc = (x.abs().max(-1).values / 127).float().half()
        kept = torch.zeros(s["k_scale"].shape, dtype=torch.float64, device="cuda")
        kept[pg, :, at] = sc.double()
        step = sc.double()[..., None]
        values.append((x / step).round().clamp(-127, 127) * step)
        scales.append(kept)
    return q, *values, *scales


def _exact_attend(s, c):
    H, KV, D, G = c["q_heads"], c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((s["q"].shape[0], H), float("-inf"), dtype=torch.float64, device="cuda")
    row = 0
    for i, (n, new) in enumerate(_requests(c)):
        t = torch.arange(n, device="cuda")
        pg, off = s["table"][i].long()[t // c["page"]], t % c["page"]
        seen, _ = _seen(c, n, new, i)
        hidden = torch.from_numpy(~seen).cuda()
        here = slice(row, row + new)
        row += new
        for j in range(KV if new else 0):
            k, v = (s[x + "_cache"][pg, j, off].double() for x in "kv")  # [n, D]
            if c["fmt"] == "int8":
                k, v = k * s["k_scale"][pg, j, off].double()[:, None], v * s["v_scale"][pg, j, off].double()[:, None]
            for h in range(j * G, (j + 1) * G):
                z = (s["q"][here, h].double() @ k.t() / math.sqrt(D)).masked_fill_(hidden, float("-inf"))
                lse[here, h] = torch.logsumexp(z, 1)
                o[here, h] = torch.softmax(z, 1).nan_to_num(0.0) @ v
    return o, lse
