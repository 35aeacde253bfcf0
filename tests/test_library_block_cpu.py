"""Argument checks of the operators between a block's projections: they run on
the host before any HIP call, so they need no GPU; every address below is
never dereferenced."""
import os
import re
import struct

import pytest

import rotation_bit_ptq_amd as rbp

OK, ARG, SHAPE, DTYPE = 0, 1, 2, 3
P = 0x10000   # 16-byte aligned
ODD = P + 8   # not
# the argument structs of include/orbit.h, field by field, in the C compiler's layout
NORM_ARGS = struct.Struct("@10P10q6i2f")
ADAPTER_ARGS = struct.Struct("@9P9q2i")
CACHE_ARGS = struct.Struct("@4Pq4i")
APPEND_ARGS = struct.Struct("@4Pq4i7P9q4i")
ATTENTION_ARGS = struct.Struct("@4Pq4i6P8qfi")
INF, NAN = float("inf"), float("nan")


def _norm(**kw):
    f = dict(x=P, branch=P, r=P, y=P, weight=0, post_weight=0, gate=0, scale=0, shift=0, ids=0, xs=64, bs=64, rs=64, ys=64,
             gs=64, cs=64, hs=64, rows=0, dim=64, groups=1, xt=1, bt=1, yt=1, pt=0, norm=1, post=0, rho=1.0, eps=1e-6)
    assert not set(kw) - set(f)
    f.update(kw)
    return rbp.lib.orbit_block_norm(NORM_ARGS.pack(*f.values()), None)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(rows=-1), SHAPE), (dict(rows=1 << 22), SHAPE), (dict(dim=0), SHAPE), (dict(dim=16385), SHAPE),
    (dict(norm=3), ARG), (dict(post=-1), ARG), (dict(xt=3), DTYPE), (dict(eps=-1.0), ARG), (dict(eps=INF), ARG),
    (dict(eps=NAN), ARG), (dict(branch=0, norm=0), ARG), (dict(branch=0, gate=P), ARG), (dict(branch=0, post=1), ARG),
    (dict(branch=0, post_weight=P), ARG), (dict(norm=0, weight=P), ARG), (dict(norm=0, scale=P), ARG), (dict(bt=2), DTYPE),
    (dict(xt=0, bt=2), OK), (dict(yt=0), DTYPE), (dict(xt=0, yt=2), OK), (dict(gate=P, pt=7), DTYPE),
    (dict(gate=P, groups=0), SHAPE), (dict(ids=P + 2), ARG), (dict(rows=4, x=0), ARG), (dict(rows=4, r=0), ARG),
    (dict(rows=4, y=0), ARG), (dict(rows=4, x=P + 1), ARG), (dict(rows=4, weight=P + 2), ARG), (dict(rows=4, xs=-64), SHAPE),
    (dict(rows=4, gate=P, gs=-1), SHAPE), (dict(rows=4, rs=63), SHAPE), (dict(rows=4, ys=0), SHAPE),
])
def test_block_norm(kw, want):
    assert _norm(**kw) == want


def _adapter(**kw):
    f = dict(x=P, A=P, B=P, y=P, out=P, ids=P, ranks=0, scale=0, ws=P, ws_bytes=1 << 40, xs=64, ys=64, os=64, M=0, K=64, N=64,
             adapters=2, rank=8, xt=1, yt=0)
    assert not set(kw) - set(f)
    f.update(kw)
    return rbp.lib.orbit_adapter_add(ADAPTER_ARGS.pack(*f.values()), None)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(M=4, N=0), OK), (dict(M=-1), SHAPE), (dict(M=1 << 22), SHAPE), (dict(K=60), SHAPE), (dict(K=0), SHAPE),
    (dict(K=65544), SHAPE), (dict(N=-1), SHAPE), (dict(N=(1 << 22) + 1), SHAPE), (dict(rank=4), SHAPE), (dict(rank=136), SHAPE),
    (dict(adapters=-1), SHAPE), (dict(xt=0), DTYPE), (dict(yt=3), DTYPE), (dict(xs=-64), SHAPE), (dict(M=4, x=0), ARG),
    (dict(M=4, x=ODD), ARG), (dict(M=4, xs=65), ARG), (dict(M=4, A=0), ARG), (dict(M=4, B=ODD), ARG), (dict(M=4, y=P + 2), ARG),
    (dict(M=4, out=0), ARG), (dict(M=4, ids=0), ARG), (dict(M=4, ranks=P + 1), ARG), (dict(M=4, scale=P + 2), ARG),
    (dict(M=4, os=63), SHAPE), (dict(M=4, ws=0), ARG), (dict(M=4, ws=ODD), ARG), (dict(M=4, ws_bytes=8), ARG),
])
def test_adapter_add(kw, want):
    assert _adapter(**kw) == want


def test_adapter_workspace():
    f = rbp.lib.orbit_adapter_workspace
    assert f(0, 64, 8) >= 0 and f(100, 4096, 16) >= 100 * 16 * 4
    for bad in ((-1, 64, 8), (1, 60, 8), (1, 64, 12), (1, 64, 0), (1, 64, 136), (1 << 22, 64, 8)):
        assert f(*bad) == -1


CACHE = dict(kc=P, vc=P, ks=0, vs=0, pages=4, page=16, kv=2, dim=64, fmt=1)
CACHE_CASES = [
    (dict(fmt=0), ARG), (dict(fmt=4), ARG), (dict(page=0), SHAPE), (dict(page=24), SHAPE), (dict(page=2048), SHAPE),
    (dict(kv=0), SHAPE), (dict(kv=1025), SHAPE), (dict(dim=0), SHAPE), (dict(dim=12), SHAPE), (dict(dim=264), SHAPE),
    (dict(pages=-1), SHAPE), (dict(pages=1 << 27), SHAPE), (dict(kc=0), ARG), (dict(vc=ODD), ARG), (dict(fmt=3), ARG),
    (dict(fmt=3, ks=P, vs=ODD), ARG), (dict(fmt=3, ks=P, vs=P, dim=8), SHAPE), (dict(fmt=3, ks=P, vs=P, page=2), SHAPE),
]


def _append(**kw):
    f = dict(CACHE, k=P, v=P, q=P, qo=P + 64, slots=P, pos=P, cs=P, kts=128, khs=64, vts=128, vhs=64, qts=256, qhs=64, tokens=0,
             q_heads=4, table=10, rot=64, xt=1, inter=0, had=0)
    assert not set(kw) - set(f)
    f.update(kw)
    return rbp.lib.orbit_kv_append(APPEND_ARGS.pack(*f.values()), None)


@pytest.mark.parametrize("kw,want", CACHE_CASES + [
    ({}, OK), (dict(fmt=3, ks=P, vs=P), OK), (dict(pages=0, kc=0, vc=0), OK), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 22), SHAPE),
    (dict(xt=3), DTYPE), (dict(q_heads=0), SHAPE), (dict(rot=63), SHAPE), (dict(rot=66), SHAPE), (dict(rot=-2), SHAPE),
    (dict(table=0), SHAPE), (dict(had=1, dim=48, rot=32), SHAPE), (dict(kts=-1), SHAPE), (dict(qhs=-1), SHAPE),
    (dict(tokens=3, k=0), ARG), (dict(tokens=3, v=P + 1), ARG), (dict(tokens=3, slots=0), ARG), (dict(tokens=3, slots=P + 4), ARG),
    (dict(tokens=3, pos=0), ARG), (dict(tokens=3, qo=0), ARG), (dict(tokens=3, qo=P), ARG), (dict(tokens=3, qo=P + 72), ARG),
])
def test_kv_append(kw, want):
    assert _append(**kw) == want


def _read(tokens=0, slots=P, k=P, v=P, dt=1, **kw):
    f = dict(CACHE)
    assert not set(kw) - set(f)
    f.update(kw)
    return rbp.lib.orbit_kv_read(CACHE_ARGS.pack(*f.values()), slots, tokens, k, v, dt, None)


@pytest.mark.parametrize("kw,want", CACHE_CASES + [
    ({}, OK), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 22), SHAPE), (dict(dt=3), DTYPE), (dict(tokens=2, slots=None), ARG),
    (dict(tokens=2, k=ODD), ARG), (dict(tokens=2, v=None), ARG),
    (dict(tokens=(1 << 22) - 1, kv=1024, dim=256), SHAPE),
])
def test_kv_read(kw, want):
    assert _read(**kw) == want


def _attend(**kw):
    f = dict(CACHE, q=P, out=P, lse=0, table=P, lengths=P, ws=0, ws_bytes=0, qbs=256, qhs=64, ts=4, batch=0, q_heads=4, width=4,
             window=0, scale=0.125, qt=1)
    assert not set(kw) - set(f)
    f.update(kw)
    return rbp.lib.orbit_paged_attention(ATTENTION_ARGS.pack(*f.values()), None)


@pytest.mark.parametrize("kw,want", CACHE_CASES + [
    ({}, OK), (dict(fmt=3, ks=P, vs=P, qt=2), OK), (dict(batch=-1), SHAPE), (dict(batch=65536), SHAPE), (dict(q_heads=3), SHAPE),
    (dict(q_heads=0), SHAPE), (dict(width=-1), SHAPE), (dict(width=(1 << 26) + 1), SHAPE), (dict(window=-1), SHAPE),
    (dict(window=(1 << 30) + 1), SHAPE), (dict(qt=0), DTYPE), (dict(qt=2), DTYPE), (dict(fmt=2), DTYPE), (dict(scale=INF), ARG),
    (dict(scale=NAN), ARG), (dict(qbs=-8), SHAPE), (dict(ts=-1), SHAPE), (dict(batch=2, q=0), ARG), (dict(batch=2, q=ODD), ARG),
    (dict(batch=2, qhs=68), ARG), (dict(batch=2, out=ODD), ARG), (dict(batch=2, lengths=0), ARG), (dict(batch=2, table=0), ARG),
    (dict(batch=2, lse=P + 2), ARG),
])
def test_paged_attention(kw, want):
    assert _attend(**kw) == want


def test_null_structs():
    for fn in ("orbit_block_norm", "orbit_adapter_add", "orbit_kv_append", "orbit_paged_attention"):
        assert getattr(rbp.lib, fn)(None, None) == ARG
    assert rbp.lib.orbit_kv_read(None, P, 1, P, P, 1, None) == ARG


def test_attention_workspace_of_invalid_sizes():
    f = rbp.lib.orbit_paged_attention_workspace
    assert f(0, 8, 2, 128, 16, 100, 0, 1) == 0 and f(1, 8, 2, 128, 16, 4096, 0, 3) > 0
    for bad in ((-1, 8, 2, 128, 16, 1, 0, 1), (1, 7, 2, 128, 16, 1, 0, 1), (1, 8, 2, 100, 16, 1, 0, 1), (1, 8, 2, 128, 0, 1, 0, 1),
                (1, 8, 2, 128, 16, -1, 0, 1), (1, 8, 2, 128, 16, 1, -1, 1), (1, 8, 2, 128, 16, 1, 0, 0)):
        assert f(*bad) == -1


def test_structs_hold_the_headers_fields():
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "orbit.h")).read()
    for fmt, name in ((CACHE_ARGS, "orbit_kv_cache"), (NORM_ARGS, "orbit_block_norm_args"), (ADAPTER_ARGS, "orbit_adapter_args"),
                      (APPEND_ARGS, "orbit_kv_append_args"), (ATTENTION_ARGS, "orbit_paged_attention_args")):
        end = header.index("} " + name + ";")
        body = re.sub(r"/\*.*?\*/", "", header[header.rindex("typedef struct {", 0, end) + 16:end], flags=re.S)
        got = "".join(("4Pq4i" if line.split()[0] == "orbit_kv_cache" else
                       {"void": "P", "int32_t": "i", "int64_t": "q", "float": "f"}[line.replace("const ", "").split()[0]]
                       if "*" not in line else "P") * len(line.split(","))
                      for line in body.replace("\n", " ").split(";") if line.strip())
        want = "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([Pqif])", fmt.format))
        assert "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([Pqif])", got)) == want, name


def test_the_binding_refuses_before_it_calls():
    import torch
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for f in (lambda: rbp.block_norm(x), lambda: rbp.block_norm(None), lambda: rbp.block_norm(x, norm="batch"),
              lambda: rbp.adapter_add(x, x, x, x, i), lambda: rbp.kv_append(x, x, x, x, i), lambda: rbp.kv_read(x, x, i),
              lambda: rbp.paged_attention(x, x, x, i, i), lambda: rbp.paged_attention(3, x, x, i, i)):
        with pytest.raises(rbp.OrbitError):
            f()
