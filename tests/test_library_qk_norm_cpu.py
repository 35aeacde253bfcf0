"""Argument checks of the norms of queries and keys: on the host, before any HIP call (no GPU; addresses are never read)."""
import struct

import pytest
import torch

import rotation_bit_ptq_amd as rbp

OK, ARG, SHAPE, DTYPE = 0, 1, 2, 3
P = 0x10000
ODD = P + 8
NORM = struct.Struct("@2P2q2if4x")
QK = struct.Struct("@2P2q2if4x4P2P8q5q4i")
APPEND = struct.Struct("@4Pq4i7P9q4i")
NORM_FIELDS = dict(qw=P, kw=P, qws=0, kws=0, wt=0, norm=1, eps=1e-6)
NORM_CASES = [(dict(norm=0), ARG), (dict(norm=3), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
              (dict(wt=3), DTYPE), (dict(wt=3, qw=0, kw=0), OK), (dict(qws=-1), SHAPE), (dict(kws=-64), SHAPE), (dict(qw=P + 2), ARG),
              (dict(kw=P + 1, wt=1), ARG)]


def _qk(**kw):
    f = dict(NORM_FIELDS, q=P, k=P, qo=P, ko=P, pos=P, cs=P, qts=256, qhs=64, kts=128, khs=64, qots=256, qohs=64, kots=128, kohs=64, tokens=0,
             q_heads=4, k_heads=2, dim=64, table=10, rot=64, xt=1, inter=0, had=0)
    assert not set(kw) - set(f)
    f.update(kw)
    return rbp.lib.orbit_qk_norm(QK.pack(*f.values()), None)


@pytest.mark.parametrize("kw,want", NORM_CASES + [
    ({}, OK), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 22), SHAPE), (dict(xt=3), DTYPE), (dict(dim=0), SHAPE), (dict(dim=12), SHAPE),
    (dict(dim=264), SHAPE), (dict(q_heads=0), SHAPE), (dict(k_heads=-1), SHAPE), (dict(rot=63), SHAPE), (dict(rot=66), SHAPE),
    (dict(table=0), SHAPE), (dict(had=1, dim=48, rot=32), SHAPE), (dict(qts=-1), SHAPE), (dict(kohs=-1), SHAPE), (dict(tokens=2, q=0), ARG),
    (dict(tokens=2, q=P + 1), ARG), (dict(tokens=2, qo=0), ARG), (dict(tokens=2, k=0), ARG), (dict(tokens=2, ko=P + 1), ARG),
    (dict(tokens=2, pos=0), ARG), (dict(tokens=2, pos=P + 4), ARG), (dict(tokens=2, cs=P + 2), ARG),
])
def test_qk_norm(kw, want):
    assert _qk(**kw) == want


def _append(null=False, tokens=0, page=16, **kw):
    f = dict(NORM_FIELDS)
    assert not set(kw) - set(f)
    f.update(kw)
    args = APPEND.pack(P, P, 0, 0, 4, page, 2, 64, 1, P, P, P, P + 64, P, P, P, 128, 64, 128, 64, 256, 64, tokens, 4, 10, 64, 1, 0, 0)
    return rbp.lib.orbit_kv_append_normed(args, None if null else NORM.pack(*f.values()), None)


@pytest.mark.parametrize("kw,want", NORM_CASES + [({}, OK), (dict(null=True), ARG), (dict(page=24), SHAPE), (dict(tokens=-1), SHAPE)])
def test_kv_append_normed(kw, want):
    assert _append(**kw) == want


def test_null_structs():
    assert rbp.lib.orbit_qk_norm(None, None) == ARG
    assert rbp.lib.orbit_kv_append_normed(None, None, None) == ARG


def test_the_binding_refuses_before_it_calls():
    x = torch.zeros(2, 4, 64)
    for f in (lambda: rbp.qk_norm(x), lambda: rbp.qk_norm(x, x), lambda: rbp.qk_norm(None), lambda: rbp.qk_norm(x, norm=None),
              lambda: rbp.qk_norm(x, norm="batch"), lambda: rbp.kv_append(x, x, x, x, x, norm="batch")):
        with pytest.raises(rbp.OrbitError):
            f()
