"""What stands between the quantized projections of a block (fp64).

Direct definitions: the norms around a residual sum, low-rank adapters beside
a shared projection, keys and values in a paged cache (16-bit, or rotated and
coded to int8 as in OrbitQuant's Method: rotate, then quantize, with the int8
article's per-group scale), and the attention of one token over such a cache.
"""
import numpy as np

from .hadamard import sylvester
from .numfmt import f16_bits_to_f64, f64_to_f16_bits, f64_to_f32


def row_norm(v, kind, eps):
    """rms: v / sqrt(mean v^2 + eps); layer: centred first; None: v itself."""
    v = np.asarray(v, dtype=np.float64)
    if kind is None:
        return v
    if kind == "layer":
        v = v - v.mean(axis=-1, keepdims=True)
    elif kind != "rms":
        raise ValueError("kind must be 'rms', 'layer' or None")
    return v / np.sqrt((v * v).mean(axis=-1, keepdims=True) + eps)


def block_norm(x, branch=None, weight=None, norm="rms", post=None, post_weight=None, gate=None,
               scale=None, shift=None, groups=None, residual_scale=1.0, eps=1e-6):
    """(r, y) with r = rho x + gate post(branch) post_weight and y = norm(r)
    weight (1 + scale) + shift.  groups: each row's group; outside the
    parameters' rows: no modulation."""
    x = np.asarray(x, dtype=np.float64)
    M = len(x)
    G = next((len(t) for t in (gate, scale, shift) if t is not None), 1)
    g = np.arange(M) // max(1, -(-M // G)) if groups is None else np.asarray(groups)
    known = ((g >= 0) & (g < G))[:, None]
    row = np.clip(g, 0, G - 1)

    def of_group(t, neutral):
        return neutral if t is None else np.where(known, np.asarray(t, dtype=np.float64)[row], neutral)

    r = x
    if branch is not None:
        b = row_norm(branch, post, eps)
        if post_weight is not None:
            b = b * post_weight
        r = residual_scale * x + of_group(gate, 1.0) * b
    if norm is None:
        return r, None
    y = row_norm(r, norm, eps)
    if weight is not None:
        y = y * weight
    return r, y * (1.0 + of_group(scale, 0.0)) + of_group(shift, 0.0)


def adapter_add(y, x, A, B, ids, scale=None, ranks=None):
    """out[m] = y[m] + scale[a] B[a] (A[a] x[m]) over the first ranks[a] rows,
    a = ids[m]; y[m] where there is no such adapter."""
    out = np.array(y, dtype=np.float64)
    x = np.asarray(x, dtype=np.float64)
    for m, a in enumerate(np.asarray(ids)):
        if not 0 <= a < len(A):
            continue
        r = A.shape[1] if ranks is None else int(np.clip(ranks[a], 0, A.shape[1]))
        if r == 0:
            continue
        v = np.asarray(A[a][:r], dtype=np.float64) @ x[m]
        out[m] += (1.0 if scale is None else float(scale[a])) * (np.asarray(B[a][:, :r], dtype=np.float64) @ v)
    return out


def turn(x, cos, sin, interleaved):
    """Position rotation of the first 2 * cos.shape[-1] coordinates.  x:
    [tokens, heads, D]; cos, sin: [tokens, pairs]."""
    x = np.array(x, dtype=np.float64)
    n = cos.shape[-1]
    first = np.arange(n) * 2 if interleaved else np.arange(n)
    second = first + (1 if interleaved else n)
    c, s = np.asarray(cos, dtype=np.float64)[:, None, :], np.asarray(sin, dtype=np.float64)[:, None, :]
    a, b = x[..., first].copy(), x[..., second].copy()
    x[..., first], x[..., second] = a * c - b * s, a * s + b * c
    return x


def hadamard_heads(x):
    """H_D x / sqrt(D) on the last axis (the dense Sylvester matrix)."""
    D = x.shape[-1]
    return np.asarray(x, dtype=np.float64) @ sylvester(D).T / np.sqrt(D)


def kv_codes(x):
    """Rows [..., D] to (codes, fp16 scale bits [...]): scale = fp16(max|x| /
    127), code = round_half_even(x / scale), 0 where scale is 0; decided in
    float32."""
    g = f64_to_f32(np.asarray(x, dtype=np.float64))
    bits = f64_to_f16_bits((np.abs(g).max(axis=-1) / np.float32(127)).astype(np.float64))
    s = f16_bits_to_f64(bits).astype(np.float32)[..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where(s > 0, np.rint(g / s), 0.0)
    return np.clip(q, -127, 127).astype(np.int8), bits


def paged_attention(q, k, v, block_table, lengths, sm_scale, window=0):
    """q [batch, H, D] over caches [pages, heads, page, D] (values, not
    codes); returns (out, lse).  A table entry outside the cache hides its
    page; a request with nothing to see gives 0 and -inf."""
    q = np.asarray(q, dtype=np.float64)
    batch, H, D = q.shape
    pages, KV, page, _ = k.shape
    out, lse = np.zeros_like(q), np.full((batch, H), -np.inf)
    for b in range(batch):
        n = min(max(int(lengths[b]), 0), block_table.shape[1] * page)
        t = np.arange(max(0, n - window) if window else 0, n)
        at = np.asarray(block_table[b])[t // page] if n else np.zeros(0, dtype=int)
        ok = (at >= 0) & (at < pages)
        at, off = at[ok], t[ok] % page
        if not len(at):
            continue
        for h in range(H):
            g = h // (H // KV)
            z = np.asarray(k[at, g, off], dtype=np.float64) @ q[b, h] * sm_scale
            m = z.max()
            if m == -np.inf:
                continue
            p = np.exp(z - m)
            out[b, h] = p @ np.asarray(v[at, g, off], dtype=np.float64) / p.sum()
            lse[b, h] = m + np.log(p.sum())
    return out, lse
