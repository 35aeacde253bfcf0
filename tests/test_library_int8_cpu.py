"""Argument checks of the int8 layer with coded tokens: on the host, before any HIP call (no GPU; addresses are never read)."""
import os
import re
import struct

import pytest
import torch

import rotation_bit_ptq_amd as rbp

OK, ARG, SHAPE, DTYPE = 0, 1, 2, 3
P = 0x10000   # 16-byte aligned
ODD = P + 8   # not
RPBH = struct.Struct("@2i3Pi4x")
PRODUCT_ARGS = struct.Struct("@6P3q3i4x")


def _rows(rot=None, x=P, dt=1, M=0, K=256, stride=256, q=P, s=P):
    rot = RPBH.pack(*rot) if rot else None
    return rbp.lib.orbit_int8_quant_rows(rot, x, dt, M, K, stride, q, s, None)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(rot=(256, 128, P, P, 0, 0)), OK), (dict(rot=(128, 128, P, P, 0, 0)), SHAPE), (dict(rot=(256, 96, P, P, 0, 0)), SHAPE),
    (dict(rot=(256, 128, 0, P, 0, 0)), ARG), (dict(rot=(256, 128, P, P, ODD, 0)), ARG), (dict(M=-1), SHAPE), (dict(M=1 << 22), SHAPE),
    (dict(K=0), SHAPE), (dict(K=24), SHAPE), (dict(K=16400), SHAPE), (dict(stride=-1), SHAPE), (dict(dt=3), DTYPE), (dict(dt=-1), DTYPE),
    (dict(M=2, x=None), ARG), (dict(M=2, x=P + 1), ARG), (dict(M=2, dt=0, x=P + 2), ARG), (dict(M=2, q=None), ARG), (dict(M=2, q=ODD), ARG),
    (dict(M=2, s=None), ARG), (dict(M=2, s=P + 2), ARG),
])
def test_quant_rows(kw, want):
    assert _rows(**kw) == want


def _product(**kw):
    f = dict(qx=P, qw=P, sx=P, sw=P, bias=0, out=P, M=0, N=64, K=64, bt=0, ot=1, act=0)
    assert not set(kw) - set(f)
    f.update(kw)
    return rbp.lib.orbit_int8_qlinear(PRODUCT_ARGS.pack(*f.values()), None)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(M=4, N=0), OK), (dict(M=-1), SHAPE), (dict(M=1 << 22), SHAPE), (dict(N=-1), SHAPE), (dict(N=1 << 22), SHAPE),
    (dict(K=0), SHAPE), (dict(K=24), SHAPE), (dict(K=65552), SHAPE), (dict(ot=3), DTYPE), (dict(bias=P, bt=5), DTYPE), (dict(bt=5), OK),
    (dict(act=2), ARG), (dict(act=-1), ARG), (dict(M=4, qx=0), ARG), (dict(M=4, qx=ODD), ARG), (dict(M=4, qw=0), ARG), (dict(M=4, qw=ODD), ARG),
    (dict(M=4, sx=0), ARG), (dict(M=4, sx=P + 2), ARG), (dict(M=4, sw=0), ARG), (dict(M=4, out=0), ARG), (dict(M=4, out=P + 1), ARG),
    (dict(M=4, bias=P + 2), ARG), (dict(M=4, bias=P + 1, bt=1), ARG),
])
def test_product(kw, want):
    assert _product(**kw) == want


def test_null_struct():
    assert rbp.lib.orbit_int8_qlinear(None, None) == ARG


def test_struct_holds_the_headers_fields():
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "orbit.h")).read()
    end = header.index("} orbit_int8_qlinear_args;")
    body = re.sub(r"/\*.*?\*/", "", header[header.rindex("typedef struct {", 0, end) + 16:end], flags=re.S)
    names = re.findall(r"\w+(?=[,;])", body)
    assert names == ["qx", "qw", "sx", "sw", "bias", "out", "M", "N", "K", "bias_dtype", "out_dtype", "act"]


def test_the_binding_refuses_before_it_calls():
    x, q, s = torch.zeros(2, 64), torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2)
    for f in (lambda: rbp.int8_quant_rows(None, x), lambda: rbp.int8_quant_rows(None, None), lambda: rbp.int8_quant_rows(3, x),
              lambda: rbp.int8_qlinear(q, s, q, s), lambda: rbp.int8_qlinear(None, s, q, s), lambda: rbp.int8_qlinear(q, s, q, s, act="relu"),
              lambda: rbp.int8_qlinear(q, s, q, s, act=[])):
        with pytest.raises(rbp.OrbitError):
            f()
