"""Attention of several new tokens over the paged cache in 64 bits, and inputs for it.

Bounds as for single tokens: a score is a sum of D <= 256 products (depth D / 32 + 32 on the matrix cores) and two scalings,
dz bounds its error; probabilities are within a relative 2 dz + 2^-20 of their values; sums over L tokens add (L / 128 +
60) E.  Above the products' denominator, which stays float32, a probability is a pair of 16-bit operands, within 2^-15
(bfloat16) or 2^-19 (float16, of the largest), where a request has at most 32 rows (tokens times the group) on average,
and one number, within half a step, where it has more: 2^-8 or 2^-11, in float16 and beside an int8 cache of the largest
at least 2^-39 steps down, inside the same 2^-11.  The output's error is the sum of these times sum p |v| / sum p.
"""
import numpy as np
import torch

from block_cases import DTYPES, E, check, draw, f64

PAIR = {"bf16": 2.0 ** -15, "f16": 2.0 ** -19, "int8": 2.0 ** -19}
ONE = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11 + 2.0 ** -19, "int8": 2.0 ** -11 + 2.0 ** -19}


def seen_by(length, n, window, sinks, mask=None):
    """[n, length] truth values: what each of the last n tokens of a request sees.  mask: [n, n], or None for a run."""
    base = length - n
    t, i = np.arange(length)[None, :], np.arange(n)[:, None]
    place = base + i if mask is None else base + mask.sum(1)[:, None] - 1
    near = (t > place - window) | (t < sinks) if window else np.ones((n, length), bool)
    if mask is None:
        return near & (t <= place)
    out = near & (t < base)
    for j in range(n):
        if 0 <= base + j < length:
            out[:, base + j] = mask[:, j]
    return out


class Case:
    """requests: (length, new tokens) each; masks: per request [n, n] truth values, or None for runs."""

    def __init__(self, seed, requests, H=8, KV=2, D=128, page=16, xt="bf16", fmt="bf16", window=0, sinks=0, masks=None, words=None,
                 std=1.0, lead=0, tail=0, width=None, scale=None):
        rng = np.random.default_rng(seed)
        self.requests, self.window, self.sinks, self.masks, self.xt, self.fmt, self.page = requests, window, sinks, masks, xt, fmt, page
        need = [max(0, -(-n // page)) for n, _ in requests]
        width = width or max(1, max(need, default=1))
        pages = sum(need) + 3
        order, table, at = rng.permutation(pages), rng.integers(0, pages, (len(requests), width)).astype(np.int32), 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n][:width]
            at += n
        starts = lead + np.concatenate([[0], np.cumsum([n for _, n in requests])]).astype(np.int32)
        self.tokens = int(starts[-1]) + tail
        self.q, self.q64 = draw(rng, (self.tokens, H, D), DTYPES[xt], 2.0)
        self.kw = {}
        if fmt == "int8":
            self.k, self.v = (torch.from_numpy(rng.integers(-127, 128, (pages, KV, page, D)).astype(np.int8)).cuda() for _ in "kv")
            ks, vs = (torch.from_numpy((std * rng.uniform(0.5, 1.5, (pages, KV, page)) / 73).astype(np.float16)).cuda() for _ in "kv")
            self.kw = dict(k_scale=ks, v_scale=vs)
        else:
            self.k, _ = draw(rng, (pages, KV, page, D), DTYPES[fmt], std)
            self.v, _ = draw(rng, (pages, KV, page, D), DTYPES[fmt], std)
        self.table64, self.starts64 = table, starts
        self.table, self.starts = torch.from_numpy(table).cuda(), torch.from_numpy(starts).cuda()
        self.lengths = torch.tensor([n for n, _ in requests], dtype=torch.int32, device="cuda")
        self.tree = None
        if masks is not None:
            words = words or max(1, -(-max(n for _, n in requests) // 64))
            bits = rng.integers(0, 2, (self.tokens, words * 64)).astype(bool)  # past a request's tokens: anything
            for (_, n), m, s in zip(requests, masks, starts):
                bits[s:s + n, :min(n, words * 64)] = m[:, :words * 64]
            self.tree = torch.from_numpy(pack(bits)).cuda()
        self.scale = D ** -0.5 if scale is None else scale

    def cache(self):
        k, v = f64(self.k), f64(self.v)
        if self.kw:
            k, v = (x * f64(s)[..., None] for x, s in zip((k, v), (self.kw["k_scale"], self.kw["v_scale"])))
        return k, v

    def run(self, rbp, **kw):
        return rbp.paged_tree_attention(self.q, self.k, self.v, self.table, self.lengths, self.starts, tree=self.tree, scale=self.scale,
                                        window=self.window, sinks=self.sinks, **self.kw, **kw)

    def reference(self):
        """out, lse, and their float32 errors' bounds; rows of no request: NaN."""
        k, v = self.cache()
        pages, KV, page, D = k.shape
        T, H, _ = self.q64.shape
        G, room = H // KV, self.table64.shape[1] * page
        few = -(-T // max(1, len(self.requests))) * G <= 32
        weight = (PAIR if few else ONE)[self.fmt]
        out, lse = np.full((T, H, D), np.nan), np.full((T, H), np.nan)
        omag, lmag = np.zeros((T, H, D)), np.zeros((T, H))
        for b, (length, n) in enumerate(self.requests):
            length = min(max(length, 0), room)
            seen = seen_by(length, n, self.window, self.sinks, None if self.masks is None else self.masks[b])
            t = np.arange(length)
            pg = self.table64[b][t // page]
            inside = (pg >= 0) & (pg < pages)
            seen = seen & inside[None, :]
            pg = np.where(inside, pg, 0)
            rows = slice(self.starts64[b], self.starts64[b] + n)
            for h in range(H):
                kk, vv = k[pg, h // G, t % page], v[pg, h // G, t % page]
                with np.errstate(all="ignore"):
                    z = np.where(seen, (self.q64[rows, h] @ np.where(np.isnan(kk), 0, kk).T) * self.scale, -np.inf)
                    top = z.max(1, initial=-np.inf)
                    p = np.where(seen, np.exp(z - np.where(np.isfinite(top), top, 0)[:, None]), 0)
                    total = p.sum(1)
                    fine = np.where(np.isfinite(vv), vv, 0)
                    o = (p @ fine) / np.where(total > 0, total, 1)[:, None]
                    for t_ in np.nonzero(~np.isfinite(vv).all(1))[0]:  # an infinite or NaN value with a weight
                        o = o + np.where((seen[:, t_] & (z[:, t_] > -np.inf))[:, None] & ~np.isfinite(vv[t_]), vv[t_], 0)
                    out[rows, h], lse[rows, h] = o, top + np.log(total)
                dz = (D / 32 + 36) * E * abs(self.scale) * np.abs(self.q64[rows, h]).sum(-1) * np.abs(np.where(np.isfinite(kk), kk, 0)).max(initial=0)
                rel = 2 * dz + (length / 128 + 60) * E
                omag[rows, h] = (rel + weight)[:, None] * (p @ np.abs(fine)) / np.where(total > 0, total, 1)[:, None]
                lmag[rows, h] = rel + 2.0 ** -20 + 4 * E * np.abs(np.where(np.isfinite(lse[rows, h]), lse[rows, h], 0))
        return out, lse, omag, lmag

    def check(self, rbp):
        want, want_lse, omag, lmag = self.reference()
        out, lse = self.run(rbp, return_lse=True)
        mine = slice(self.starts64[0], self.starts64[-1])
        check(out[mine], want[mine], DTYPES[self.xt], omag[mine], "out")
        check(lse[mine], want_lse[mine], torch.float32, lmag[mine], "lse")
        assert torch.equal(self.run(rbp)[mine].view(torch.int16), out[mine].view(torch.int16))  # the same bits, NaN too
        return out


def pack(bits):
    """[rows, 64 words] truth values as int64 words."""
    b = bits.reshape(bits.shape[0], -1, 64).astype(np.uint64)
    return (b << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64).view(np.int64)


def tree_mask(rng, n):
    """Ancestors and self of n tokens, each one's parent any before it (several roots)."""
    m = np.eye(n, dtype=bool)
    for i in range(1, n):
        p = int(rng.integers(-1, i))
        if p >= 0:
            m[i] |= m[p]
    return m
