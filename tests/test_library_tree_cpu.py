"""Argument checks of the attention of several new tokens: on the host, before any HIP call (no GPU; addresses are never read)."""
import os
import re
import struct

import pytest
import torch

import rotation_bit_ptq_amd as rbp

OK, ARG, SHAPE, DTYPE = 0, 1, 2, 3
P = 0x10000
ODD = P + 8
ARGS = struct.Struct("@4Pq4i8P11qfi")
INF, NAN = float("inf"), float("nan")


def _tree(**kw):
    f = dict(kc=P, vc=P, ks=0, vs=0, pages=4, page=16, kv=2, dim=64, fmt=1, q=P, out=P, lse=0, table=P, lengths=P, starts=P, tree=0, ws=P,
             ws_bytes=1 << 40, qts=256, qhs=64, ts=4, tokens=0, batch=2, q_heads=4, width=4, words=0, window=0, sinks=0, scale=0.125, qt=1)
    assert not set(kw) - set(f)
    f.update(kw)
    return rbp.lib.orbit_tree_attention(ARGS.pack(*f.values()), None)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(fmt=3, ks=P, vs=P, qt=2), OK), (dict(tokens=5, batch=0), OK), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 22), SHAPE),
    (dict(batch=-1), SHAPE), (dict(batch=65536), SHAPE), (dict(q_heads=3), SHAPE), (dict(q_heads=0), SHAPE), (dict(width=-1), SHAPE),
    (dict(width=(1 << 26) + 1), SHAPE), (dict(window=-1), SHAPE), (dict(window=(1 << 30) + 1), SHAPE), (dict(sinks=-1), SHAPE),
    (dict(sinks=(1 << 30) + 1), SHAPE), (dict(qt=0), DTYPE), (dict(qt=2), DTYPE), (dict(fmt=2), DTYPE), (dict(fmt=0), ARG), (dict(page=24), SHAPE),
    (dict(scale=INF), ARG), (dict(scale=NAN), ARG), (dict(qts=-8), SHAPE), (dict(ts=-1), SHAPE), (dict(tree=P, words=0), SHAPE),
    (dict(tree=P, words=1025), SHAPE), (dict(tree=P, words=1), OK), (dict(starts=0), SHAPE), (dict(starts=0, tokens=2, tree=P, words=1), SHAPE),
    (dict(tokens=3, q=0), ARG), (dict(tokens=3, q=ODD), ARG), (dict(tokens=3, qhs=68), ARG), (dict(tokens=3, out=ODD), ARG),
    (dict(tokens=3, lengths=0), ARG), (dict(tokens=3, lengths=P + 2), ARG), (dict(tokens=3, starts=P + 2), ARG),
    (dict(tokens=3, tree=P + 4, words=1), ARG), (dict(tokens=3, table=0), ARG), (dict(tokens=3, lse=P + 2), ARG),
    (dict(tokens=3, width=4000, ws=0), ARG), (dict(tokens=3, width=4000, ws=ODD), ARG), (dict(tokens=3, width=4000, ws_bytes=8), ARG),
    (dict(tokens=(1 << 22) - 1, kv=1, q_heads=1024), SHAPE),
])
def test_tree_attention(kw, want):
    assert _tree(**kw) == want


def test_null_struct_and_workspace():
    assert rbp.lib.orbit_tree_attention(None, None) == ARG
    f = rbp.lib.orbit_tree_attention_workspace
    assert f(0, 2, 8, 2, 128, 16, 100, 0, 0, 0) == 0 and f(3, 1, 8, 2, 128, 16, 4096, 0, 0, 0) > 0 and f(1, 1, 8, 2, 128, 16, 4096, 0, 0, 1) > 0
    for bad in ((-1, 1, 8, 2, 128, 16, 1, 0, 0, 0), (1, -1, 8, 2, 128, 16, 1, 0, 0, 0), (1, 1, 7, 2, 128, 16, 1, 0, 0, 0),
                (1, 1, 8, 2, 100, 16, 1, 0, 0, 0), (1, 1, 8, 2, 128, 0, 1, 0, 0, 0), (1, 1, 8, 2, 128, 16, -1, 0, 0, 0),
                (1, 1, 8, 2, 128, 16, 1, -1, 0, 0), (1, 1, 8, 2, 128, 16, 1, 0, -1, 0)):
        assert f(*bad) == -1


def test_struct_holds_the_headers_fields():
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "orbit.h")).read()
    end = header.index("} orbit_tree_attention_args;")
    body = re.sub(r"/\*.*?\*/", "", header[header.rindex("typedef struct {", 0, end) + 16:end], flags=re.S)
    names = re.findall(r"\w+(?=[,;])", body)
    assert names == ["cache", "q", "out", "lse", "block_table", "lengths", "starts", "tree", "workspace", "workspace_bytes", "q_token_stride",
                     "q_head_stride", "table_stride", "tokens", "batch", "q_heads", "table_width", "tree_words", "window", "sinks", "sm_scale",
                     "q_dtype"]


def test_the_binding_refuses_before_it_calls():
    x, i = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for f in (lambda: rbp.paged_tree_attention(x, x, x, i, i, i), lambda: rbp.paged_tree_attention(x, x, x, i, i, None),
              lambda: rbp.paged_attention(x, x, x, i, i, window=4, sinks=1), lambda: rbp.paged_attention(x, x, x, i, i, sinks=-1)):
        with pytest.raises(rbp.OrbitError):
            f()
