"""Rotate-then-quantize linear layers on AMD MI355X (gfx950).

A thin ctypes binding of ``liborbit.so`` (C ABI in ``include/orbit.h``).
This module only marshals arguments: every step of the layer runs in the
library's HIP kernels on the caller's current torch stream.  Device buffers
are torch tensors; there is no CPU path, and importing fails if the library
has not been built (``__graft_entry__.build()`` or
``python rotation_bit_ptq_amd/build.py``).

Method (OrbitQuant paper page, Method): a randomized permuted block-Hadamard
rotation Pi = blkdiag(H_h D_i) P_pi is absorbed offline into the weights
(W' = W Pi^T, row norms in bf16, unit rows coded by a Lloyd-Max codebook) and
applied online to activations (x' = Pi x, split into ||x'|| and a coded unit
direction); the product of the two coded factors approximates W x with no
inverse rotation.  Also: the int8 per-group rotated weight-only path of the
int8 article (section 4) and its 4-bit sibling (int4 codes, two per byte).

Between those layers: norms around a branch with its gate and residual scale
(block_norm), low-rank adapters of many requests beside a shared projection
(adapter_add), and a paged key-value cache, 16-bit or rotate-then-quantize
int8 (kv_append, kv_read), with the attention of one new token that reads it
(paged_attention).
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np
import torch

__all__ = [
    "OrbitError", "Codebook", "Rotation", "fit_codebook", "pack_weights",
    "quant_act", "qlinear", "rotate", "int8_pack_weights", "int8_linear",
    "int4_pack_weights", "int4_linear",
    "block_norm", "adapter_add", "kv_append", "kv_read", "paged_attention",
    "packed_row_bytes", "LIB_PATH",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liborbit.so")

F32, BF16, F16 = 0, 1, 2
_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
MAX_LEVELS = 256


class OrbitError(RuntimeError):
    pass


class _Codebook(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("d", ctypes.c_int32),
                ("centroids", ctypes.c_float * MAX_LEVELS),
                ("thresholds", ctypes.c_float * (MAX_LEVELS - 1))]


class _RPBH(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("h", ctypes.c_int32),
                ("perm", ctypes.c_void_p), ("sign_bits", ctypes.c_void_p),
                ("gather", ctypes.c_void_p), ("flags", ctypes.c_int32)]

RPBH_IDENTITY = 1  # set by the library's plan builder when perm is the identity (Block-RHT)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, F, D = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                         ctypes.c_float, ctypes.c_double)
    sig = {
        "orbit_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "orbit_last_hip_error": ([ctypes.c_void_p], ctypes.c_int),
        "orbit_fit_codebook": ([I32, I32, I32, D, P, P, P, P], ctypes.c_int),
        "orbit_fit_codebook_sphere": ([I32, I32, I32, D, P, P, P, P], ctypes.c_int),
        "orbit_rpbh_gather_len": ([I32, I32], I64),
        "orbit_rpbh_build_gather": ([P, P, P], ctypes.c_int),
        "orbit_pack_weights": ([P, P, P, ctypes.c_int, I64, I64, P, P, P], ctypes.c_int),
        "orbit_quant_act": ([P, P, P, ctypes.c_int, I64, I64, F, P, P, P, P], ctypes.c_int),
        "orbit_qlinear": ([P, P, P, P, P, P, P, ctypes.c_int, I64, I64, I64, P,
                           ctypes.c_int, P], ctypes.c_int),
        "orbit_qlinear_act": ([P, P, P, P, P, P, P, ctypes.c_int, I64, I64, I64, P,
                               ctypes.c_int, ctypes.c_int, P], ctypes.c_int),
        "orbit_rotate": ([P, P, ctypes.c_int, I64, I64, P, ctypes.c_int, P], ctypes.c_int),
        "orbit_int8_pack_weights": ([P, P, ctypes.c_int, I64, I64, I32, P, P, P], ctypes.c_int),
        "orbit_int4_pack_weights": ([P, P, ctypes.c_int, I64, I64, I32, P, P, P], ctypes.c_int),
        "orbit_int8_linear": ([P, ctypes.c_int, I64, I64, P, P, I32, I64, P, ctypes.c_int,
                               P, ctypes.c_int, P], ctypes.c_int),
        "orbit_int4_linear": ([P, ctypes.c_int, I64, I64, P, P, I32, I64, P, ctypes.c_int,
                               P, ctypes.c_int, P], ctypes.c_int),
        "orbit_block_norm": ([P, P], ctypes.c_int),
        "orbit_adapter_add": ([P, P], ctypes.c_int),
        "orbit_adapter_workspace": ([I64, I64, I64], I64),
        "orbit_kv_append": ([P, P], ctypes.c_int),
        "orbit_kv_read": ([P, P, I64, P, P, ctypes.c_int, P], ctypes.c_int),
        "orbit_paged_attention": ([P, P], ctypes.c_int),
        "orbit_paged_attention_workspace": ([I64] * 7 + [I32], I64),
    }
    for name, (args, res) in sig.items():
        try:
            fn = getattr(lib, name)
        except AttributeError as e:  # a library built from older sources
            raise ImportError(f"{LIB_PATH} lacks {name}; rebuild it with "
                              "__graft_entry__.build()") from e
        fn.argtypes = args
        fn.restype = res
    return lib


lib = _load()


def _check(status: int, what: str):
    if status != 0:
        msg = lib.orbit_status_string(status).decode()
        hip = ctypes.c_int(0)
        if status == 5:
            lib.orbit_last_hip_error(ctypes.byref(hip))
        raise OrbitError(f"{what}: {msg} (status {status}, hip {hip.value})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise OrbitError(f"{name} must be a torch tensor on a GPU")
    if not t.is_contiguous():
        raise OrbitError(f"{name} must be contiguous")
    return t


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def packed_row_bytes(d: int, bits: int) -> int:
    """Bytes of one packed row of d indices of `bits` bits."""
    return d * bits // 8


class Codebook:
    """A Lloyd-Max codebook in N(0,1) units (host memory).

    marginal="gauss": fitted to N(0,1), the large-d form of the rotated
    coordinate's marginal; "sphere": fitted to the exact marginal of one
    coordinate of a uniform direction on S^{d-1} (d >= 3)."""

    def __init__(self, d: int, bits: int, max_iter: int = 0, tol: float = 0.0,
                 marginal: str = "gauss"):
        fitters = {"gauss": "orbit_fit_codebook", "sphere": "orbit_fit_codebook_sphere"}
        if marginal not in fitters:
            raise ValueError(f"marginal must be one of {sorted(fitters)}")
        levels = 1 << bits
        self.struct = _Codebook()
        self.centroids_f64 = np.zeros(levels)
        self.thresholds_f64 = np.zeros(levels - 1)
        mse = ctypes.c_double(0.0)
        _check(getattr(lib, fitters[marginal])(
            d, bits, max_iter, tol, ctypes.byref(self.struct),
            self.centroids_f64.ctypes.data_as(ctypes.c_void_p),
            self.thresholds_f64.ctypes.data_as(ctypes.c_void_p), ctypes.byref(mse)),
            fitters[marginal])
        self.mse = mse.value
        self.bits, self.d, self.levels, self.marginal = bits, d, levels, marginal

    @property
    def centroids(self) -> np.ndarray:
        return np.ctypeslib.as_array(self.struct.centroids)[: self.levels].copy()

    @property
    def thresholds(self) -> np.ndarray:
        return np.ctypeslib.as_array(self.struct.thresholds)[: self.levels - 1].copy()


def fit_codebook(d: int, bits: int, marginal: str = "gauss") -> Codebook:
    return Codebook(d, bits, marginal=marginal)


class Rotation:
    """RPBH rotation parameters on a device: perm (gather order), sign bits, h,
    and (unless plan=False) the gather plan the row kernels read instead of
    deriving their offsets from perm and the signs.  Building the plan also
    lets the library set the identity-permutation flag (struct.flags)."""

    def __init__(self, perm, signs, h: int, device="cuda", plan: bool = True):
        perm = np.ascontiguousarray(perm, dtype=np.int32)
        signs = np.asarray(signs)
        d = perm.shape[0]
        bits = np.zeros((d + 31) // 32, dtype=np.uint32)
        neg = np.nonzero(signs < 0)[0]
        np.bitwise_or.at(bits, neg // 32, (np.uint32(1) << (neg % 32).astype(np.uint32)))
        self.d, self.h = d, int(h)
        self.perm = torch.from_numpy(perm).to(device)
        self.sign_bits = torch.from_numpy(bits.view(np.int32)).to(device)
        self.struct = _RPBH(d, int(h), self.perm.data_ptr(), self.sign_bits.data_ptr(), None, 0)
        self.gather = None
        n = lib.orbit_rpbh_gather_len(d, int(h)) if plan else 0
        if n > 0:
            self.gather = torch.empty((n,), dtype=torch.int16, device=self.perm.device)
            _check(lib.orbit_rpbh_build_gather(ctypes.byref(self.struct), _ptr(self.gather),
                                               _stream(self.perm.device)), "orbit_rpbh_build_gather")
            self.struct.gather = self.gather.data_ptr()


def pack_weights(rot: Rotation, cw: Codebook, W: torch.Tensor):
    """Offline: (packed indices uint8 [N, K*bits/8], row norms bf16 [N])."""
    _dev(W, "W")
    N, K = W.shape
    idx = torch.empty((N, packed_row_bytes(K, cw.bits)), dtype=torch.uint8, device=W.device)
    r = torch.empty((N,), dtype=torch.bfloat16, device=W.device)
    _check(lib.orbit_pack_weights(ctypes.byref(rot.struct), ctypes.byref(cw.struct), _ptr(W),
                                  _DT[W.dtype], N, K, _ptr(idx), _ptr(r), _stream(W.device)),
           "orbit_pack_weights")
    return idx, r


def quant_act(rot: Rotation, ca: Codebook, X: torch.Tensor, eps: float = 1e-8,
              debug_xrot: bool = False):
    """Online: (packed indices uint8 [M, K*bits/8], s float32 [M][, x' float32])."""
    _dev(X, "X")
    M, K = X.shape
    idx = torch.empty((M, packed_row_bytes(K, ca.bits)), dtype=torch.uint8, device=X.device)
    s = torch.empty((M,), dtype=torch.float32, device=X.device)
    xr = torch.empty((M, K), dtype=torch.float32, device=X.device) if debug_xrot else None
    _check(lib.orbit_quant_act(ctypes.byref(rot.struct), ctypes.byref(ca.struct), _ptr(X),
                               _DT[X.dtype], M, K, float(eps), _ptr(idx), _ptr(s), _ptr(xr),
                               _stream(X.device)), "orbit_quant_act")
    return (idx, s, xr) if debug_xrot else (idx, s)


ACTS = {None: 0, "gelu": 1}


def qlinear(idx_a, s, ca: Codebook, idx_w, r, cw: Codebook, K: int, bias=None,
            out_dtype=torch.bfloat16, out=None, act=None):
    """out[m, n] = act(s_m r_n / K * sum_k ca[ia] cw[iw] (+ bias)); act None or "gelu"."""
    for t, n in ((idx_a, "idx_a"), (s, "s"), (idx_w, "idx_w"), (r, "r")):
        _dev(t, n)
    if act not in ACTS:
        raise OrbitError(f"unknown activation {act!r}")
    M, N = idx_a.shape[0], idx_w.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=idx_a.device)
    bias_dt = _DT[bias.dtype] if bias is not None else F32
    _check(lib.orbit_qlinear_act(_ptr(idx_a), _ptr(s), ctypes.byref(ca.struct), _ptr(idx_w),
                                 _ptr(r), ctypes.byref(cw.struct), _ptr(bias), bias_dt, M, N, K,
                                 _ptr(out), _DT[out.dtype], ACTS[act], _stream(idx_a.device)),
           "orbit_qlinear_act")
    return out


def rotate(rot: Rotation, X: torch.Tensor, out_dtype=torch.float16, out=None):
    """x' = Pi x per row."""
    _dev(X, "X")
    M, K = X.shape
    if out is None:
        out = torch.empty((M, K), dtype=out_dtype, device=X.device)
    _check(lib.orbit_rotate(ctypes.byref(rot.struct), _ptr(X), _DT[X.dtype], M, K, _ptr(out),
                            _DT[out.dtype], _stream(X.device)), "orbit_rotate")
    return out


def int8_pack_weights(rot: Rotation, W: torch.Tensor, group: int = 128):
    """Offline int8: (q int8 [N, K], scales fp16 [N, K/group])."""
    _dev(W, "W")
    N, K = W.shape
    q = torch.empty((N, K), dtype=torch.int8, device=W.device)
    sc = torch.empty((N, K // group), dtype=torch.float16, device=W.device)
    _check(lib.orbit_int8_pack_weights(ctypes.byref(rot.struct), _ptr(W), _DT[W.dtype], N, K,
                                       group, _ptr(q), _ptr(sc), _stream(W.device)),
           "orbit_int8_pack_weights")
    return q, sc


def int8_linear(xrot: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, group: int = 128,
                bias=None, out_dtype=torch.bfloat16, out=None):
    """out = x' (q * scale)^T (+ bias), x' = Pi x in fp16."""
    for t, n in ((xrot, "xrot"), (q, "q"), (scale, "scale")):
        _dev(t, n)
    M, K = xrot.shape
    N = q.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=xrot.device)
    bias_dt = _DT[bias.dtype] if bias is not None else F32
    _check(lib.orbit_int8_linear(_ptr(xrot), _DT[xrot.dtype], M, K, _ptr(q), _ptr(scale), group,
                                 N, _ptr(bias), bias_dt, _ptr(out), _DT[out.dtype],
                                 _stream(xrot.device)), "orbit_int8_linear")
    return out


def int4_pack_weights(rot: Rotation, W: torch.Tensor, group: int = 128):
    """Offline int4: (q uint8 [N, K/2] two codes per byte, scales fp16 [N, K/group])."""
    _dev(W, "W")
    N, K = W.shape
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
    sc = torch.empty((N, K // group), dtype=torch.float16, device=W.device)
    _check(lib.orbit_int4_pack_weights(ctypes.byref(rot.struct), _ptr(W), _DT[W.dtype], N, K,
                                       group, _ptr(q), _ptr(sc), _stream(W.device)),
           "orbit_int4_pack_weights")
    return q, sc


def int4_linear(xrot: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, group: int = 128,
                bias=None, out_dtype=torch.bfloat16, out=None):
    """out = x' (q * scale)^T (+ bias), x' = Pi x in fp16, q int4 two per byte."""
    for t, n in ((xrot, "xrot"), (q, "q"), (scale, "scale")):
        _dev(t, n)
    M, K = xrot.shape
    N = q.shape[0]
    if q.shape[1] * 2 != K:
        raise ValueError("q must be [N, K/2]")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=xrot.device)
    bias_dt = _DT[bias.dtype] if bias is not None else F32
    _check(lib.orbit_int4_linear(_ptr(xrot), _DT[xrot.dtype], M, K, _ptr(q), _ptr(scale), group,
                                 N, _ptr(bias), bias_dt, _ptr(out), _DT[out.dtype],
                                 _stream(xrot.device)), "orbit_int4_linear")
    return out


# ---- what stands between the quantized projections of a block ---------------
#
# Tensors of these functions may be strided rows or heads: only the innermost
# dimension has to be contiguous.  Argument structs of include/orbit.h are
# packed field by field ("@": the C compiler's own layout).

_NORMS = {None: 0, "rms": 1, "layer": 2}
_KV_FORMATS = {torch.bfloat16: 1, torch.float16: 2, torch.int8: 3}
_NORM_ARGS = struct.Struct("@10P10q6i2f")
_ADAPTER_ARGS = struct.Struct("@9P9q2i")
_CACHE = struct.Struct("@4Pq4i")
_APPEND_ARGS = struct.Struct("@4Pq4i7P9q4i")
_ATTENTION_ARGS = struct.Struct("@4Pq4i6P8qfi")


# These calls are made once per layer and decode step, so their checks are
# counted in tenths of microseconds: one test of everything per tensor, and
# the reason looked for only when it fails.

_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _tensor(t, name, dev, shape, dtype):
    """The strides of a tensor of this shape and dtype on GPU `dev` whose innermost
    dimension is contiguous."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev and t.shape == shape and t.dtype is dtype:
        strides = t.stride()
        if strides[-1] == 1 or t.shape[-1] <= 1 or t.numel() == 0:
            return strides
    raise OrbitError(_reason(t, name, dev, shape, dtype))


def _reason(t, name, dev, shape, dtype):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return f"{name} must be a torch tensor on a GPU"
    if t.get_device() != dev:
        return f"{name} must be on GPU {dev}, where the first argument is"
    if t.shape != shape:
        return f"{name} must be {list(shape)}, got {list(t.shape)}"
    if t.dtype is not dtype:
        return f"{name} must be {dtype}, got {t.dtype}"
    return f"{name}'s innermost dimension must be contiguous"


def _first(t, name, dims):
    """The GPU of a call's first tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise OrbitError(f"{name} must be a torch tensor on a GPU")
    if t.dim() != dims:
        raise OrbitError(f"{name} must have {dims} dimensions, got {t.dim()}")
    return t.get_device()


def _float(t, name):
    """A floating tensor's orbit_dtype."""
    try:
        return _DT[t.dtype]
    except (KeyError, AttributeError):
        raise OrbitError(f"{name} must be a float32, bfloat16 or float16 tensor") from None


def _launch(fn, what, dev, *args):
    """Calls the library on the current stream of GPU `dev`, with that device current."""
    if _current_device() == dev:
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        _check(status, what)


def block_norm(x, branch=None, *, weight=None, norm="rms", post=None, post_weight=None,
               gate=None, scale=None, shift=None, groups=None, residual_scale=1.0, eps=1e-6,
               out_dtype=None, r_out=None, out=None):
    """The norms around a residual sum, in one pass over the rows:

        b^ = post(branch) * post_weight                (post None: branch)
        r  = residual_scale * x + gate[g] * b^         (no branch: x)
        y  = norm(r) * weight * (1 + scale[g]) + shift[g]

    norm and post: "rms", "layer" or None.  Returns (r, y) with a branch, y
    without one, r where norm is None.  x, branch: [rows, dim] (branch of x's
    dtype, any where x is float32); weight, post_weight: [dim]; gate, scale,
    shift: [G, dim], rows of any stride (chunks of an AdaLN projection's
    output); all five of one dtype.  Row m belongs to group groups[m] (int32
    [rows]; an id outside 0 .. G - 1: no modulation), or, without groups, to
    m // ceil(rows / G).  r has x's dtype, y out_dtype (x's; any where x is
    float32).  r_out may be x; out may be x or branch.
    """
    dev = _first(x, "x", 2)
    shape = x.shape
    M, D = shape
    xt = _float(x, "x")
    dtype = x.dtype
    xs = _tensor(x, "x", dev, shape, dtype)[0]
    if norm not in _NORMS or post not in _NORMS:
        raise OrbitError(f"norm and post must be 'rms', 'layer' or None, got {norm!r}, {post!r}")
    bt = bp = bs = rp = rs = yt = yp = ys = 0
    r = y = None
    if branch is not None:
        bt = _float(branch, "branch")
        bs = _tensor(branch, "branch", dev, shape, branch.dtype)[0]
        bp = branch.data_ptr()
        r = x.new_empty(shape) if r_out is None else r_out
        rs = _tensor(r, "r_out", dev, shape, dtype)[0]
        rp = r.data_ptr()
    elif norm is None:
        raise OrbitError("block_norm needs a branch, a norm, or both")
    elif post is not None or post_weight is not None or gate is not None or r_out is not None:
        raise OrbitError("post, post_weight, gate and r_out need a branch")
    if norm is not None:
        if out is None:
            y = x.new_empty(shape) if out_dtype is None or out_dtype is dtype else x.new_empty(shape, dtype=out_dtype)
        else:
            y = out
        yt = _float(y, "out")
        ys = _tensor(y, "out", dev, shape, out_dtype or y.dtype)[0]
        yp = y.data_ptr()
    elif weight is not None or scale is not None or shift is not None or out is not None:
        raise OrbitError("weight, scale, shift and out need a norm")
    G, pt, wp, pwp, gp, cp, hp, gs, cs, hs, ip = 1, None, 0, 0, 0, 0, 0, 0, 0, 0, 0
    if weight is not None:
        pt = getattr(weight, "dtype", None)
        _tensor(weight, "weight", dev, (D,), pt)
        wp = weight.data_ptr()
    if post_weight is not None:
        pt = pt or getattr(post_weight, "dtype", None)
        _tensor(post_weight, "post_weight", dev, (D,), pt)
        pwp = post_weight.data_ptr()
    mod = gate if gate is not None else scale if scale is not None else shift
    if mod is not None:
        if not isinstance(mod, torch.Tensor) or mod.dim() != 2 or mod.shape[0] < 1:
            raise OrbitError(f"gate, scale and shift must be tensors [groups, {D}]")
        pt = pt or mod.dtype
        G = mod.shape[0]
        rows = (G, D)
        if gate is not None:
            gs = _tensor(gate, "gate", dev, rows, pt)[0]
            gp = gate.data_ptr()
        if scale is not None:
            cs = _tensor(scale, "scale", dev, rows, pt)[0]
            cp = scale.data_ptr()
        if shift is not None:
            hs = _tensor(shift, "shift", dev, rows, pt)[0]
            hp = shift.data_ptr()
    if pt is not None and pt not in _DT:
        raise OrbitError("weight, post_weight, gate, scale and shift must be float32, bfloat16 or float16")
    if groups is not None:
        _tensor(groups, "groups", dev, (M,), torch.int32)
        ip = groups.data_ptr()
    if M:  # an empty branch has no address to tell it from none
        _launch(lib.orbit_block_norm, "orbit_block_norm", dev, _NORM_ARGS.pack(
            x.data_ptr(), bp, rp, yp, wp, pwp, gp, cp, hp, ip, xs, bs, rs, ys, gs, cs, hs, M, D, G, xt,
            bt, yt, _DT[pt] if pt is not None else 0, _NORMS[norm], _NORMS[post], residual_scale, eps))
    return y if r is None else r if y is None else (r, y)


def adapter_add(y, x, A, B, ids, *, scale=None, ranks=None, out=None):
    """Low-rank adapters of many requests beside a shared projection:

        out[m] = y[m] + scale[a] * B[a] (A[a] x[m]),  a = ids[m]

    over the first ranks[a] rows of A[a]; out[m] = y[m] where a is outside
    0 .. adapters - 1 (-1 by convention).  y: [M, N], the shared projection's
    output; x: [M, K] bfloat16 or float16; A: [adapters, R, K] and B:
    [adapters, N, R] of x's dtype, R a multiple of 8 up to 128; ids: int32
    [M]; scale: float32 [adapters]; ranks: int32 [adapters].  Next to the
    weight-only layers x is the rotated x' they read, with A rotated once:
    rotate(rot, A.view(-1, K)).  out may be y.
    """
    dev = _first(x, "x", 2)
    M, K = x.shape
    dtype = x.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise OrbitError("x must be bfloat16 or float16")
    yt = _float(y, "y")
    if not isinstance(A, torch.Tensor) or A.dim() != 3 or y.dim() != 2:
        raise OrbitError("y must be [M, N] and A [adapters, R, K]")
    L, R, N = A.shape[0], A.shape[1], y.shape[1]
    xs = _tensor(x, "x", dev, x.shape, dtype)[0]
    ys = _tensor(y, "y", dev, (M, N), y.dtype)[0]
    _tensor(A, "A", dev, (L, R, K), dtype)
    _tensor(B, "B", dev, (L, N, R), dtype)
    if not A.is_contiguous() or not B.is_contiguous():
        raise OrbitError("A and B must be contiguous")
    _tensor(ids, "ids", dev, (M,), torch.int32)
    sp = rp = 0
    if scale is not None:
        _tensor(scale, "scale", dev, (L,), torch.float32)
        sp = scale.data_ptr()
    if ranks is not None:
        _tensor(ranks, "ranks", dev, (L,), torch.int32)
        rp = ranks.data_ptr()
    if out is None:
        out = y.new_empty((M, N))
    os_ = _tensor(out, "out", dev, (M, N), y.dtype)[0]
    ws = lib.orbit_adapter_workspace(M, K, R)
    if ws < 0:
        raise OrbitError(f"orbit_adapter_add: invalid shape (M {M}, K {K}, rank {R})")
    work = x.new_empty((ws,), dtype=torch.uint8)
    _launch(lib.orbit_adapter_add, "orbit_adapter_add", dev, _ADAPTER_ARGS.pack(
        x.data_ptr(), A.data_ptr(), B.data_ptr(), y.data_ptr(), out.data_ptr(), ids.data_ptr(), rp, sp,
        work.data_ptr(), ws, xs, ys, os_, M, K, N, L, R, _DT[dtype], yt))
    return out


def _cache_fields(k_cache, v_cache, k_scale, v_scale, dev):
    """The fields of orbit_kv_cache: caches [pages, heads, page size, head dim]."""
    fmt = _KV_FORMATS.get(getattr(k_cache, "dtype", None))
    if fmt is None:
        raise OrbitError("k_cache and v_cache must be bfloat16, float16 or int8 tensors")
    shape = k_cache.shape
    if len(shape) != 4:
        raise OrbitError("k_cache and v_cache must be [pages, kv_heads, page_size, dim]")
    _tensor(k_cache, "k_cache", dev, shape, k_cache.dtype)
    _tensor(v_cache, "v_cache", dev, shape, k_cache.dtype)
    if not k_cache.is_contiguous() or not v_cache.is_contiguous():
        raise OrbitError("k_cache and v_cache must be contiguous")
    ks = vs = 0
    if fmt == 3:
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _tensor(t, name, dev, shape[:3], torch.float16)
            if not t.is_contiguous():
                raise OrbitError(f"{name} must be contiguous")
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise OrbitError("k_scale and v_scale belong to an int8 cache")
    return (k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, shape[0], shape[2], shape[1], shape[3], fmt)


def kv_append(k, v, k_cache, v_cache, slots, *, positions=None, cos_sin=None, interleaved=False,
              q=None, q_out=None, k_scale=None, v_scale=None, hadamard=False):
    """Appends a key and a value per token and head to the paged cache, the
    position rotation (and, with hadamard, the orthonormal Hadamard rotation
    of each head) applied to keys on the way, and to the queries if given.

    k, v: [tokens, kv_heads, dim], q: [tokens, q_heads, dim], views of one
    projection's output for instance.  k_cache, v_cache: [pages, kv_heads,
    page_size, dim], bfloat16, float16, or int8 with k_scale, v_scale float16
    [pages, kv_heads, page_size].  slots: int64 [tokens], page * page_size +
    offset, all different; a slot outside the cache (-1) stores nothing.
    cos_sin: float32 [positions, rot_dim], cosines then sines; positions:
    int64 [tokens].  Returns the rotated queries (None without q).
    """
    dev = _first(k, "k", 3)
    kt = _float(k, "k")
    dtype = k.dtype
    cache = _cache_fields(k_cache, v_cache, k_scale, v_scale, dev)
    T, heads, dim = k.shape[0], cache[6], cache[7]
    ks = _tensor(k, "k", dev, (T, heads, dim), dtype)
    vs = _tensor(v, "v", dev, (T, heads, dim), dtype)
    _tensor(slots, "slots", dev, (T,), torch.int64)
    cp = pp = P = rot = 0
    if cos_sin is not None:
        if not isinstance(cos_sin, torch.Tensor) or cos_sin.dim() != 2 or not cos_sin.shape[0]:
            raise OrbitError("cos_sin must be a tensor [positions, rot_dim] of at least one row")
        P, rot = cos_sin.shape
        _tensor(cos_sin, "cos_sin", dev, cos_sin.shape, torch.float32)
        if not cos_sin.is_contiguous():
            raise OrbitError("cos_sin must be contiguous")
        if positions is None:
            raise OrbitError("cos_sin needs positions")
        _tensor(positions, "positions", dev, (T,), torch.int64)
        cp, pp = cos_sin.data_ptr(), positions.data_ptr()
    qp = qo = q0 = q1 = H = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise OrbitError("q must be a tensor [tokens, q_heads, dim]")
        H = q.shape[1]
        shape = (T, H, dim)
        q0, q1, _ = _tensor(q, "q", dev, shape, dtype)
        if q_out is None:
            q_out = q.new_empty(shape)
        else:
            _tensor(q_out, "q_out", dev, shape, dtype)
            if not q_out.is_contiguous():
                raise OrbitError("q_out must be contiguous")
        qp, qo = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise OrbitError("q_out needs q")
    _launch(lib.orbit_kv_append, "orbit_kv_append", dev, _APPEND_ARGS.pack(
        *cache, k.data_ptr(), v.data_ptr(), qp, qo, slots.data_ptr(), pp, cp, ks[0], ks[1], vs[0],
        vs[1], q0, q1, T, H, P, rot, kt, bool(interleaved), bool(hadamard)))
    return q_out


def kv_read(k_cache, v_cache, slots, *, k_scale=None, v_scale=None, dtype=None):
    """The keys and values of the tokens at `slots` (int64 [tokens]) as dense
    rows [tokens, kv_heads, dim] of `dtype` (default: the cache's; float16 for
    int8); zeros where a slot lies outside the cache."""
    dev = _first(k_cache, "k_cache", 4)
    cache = _cache_fields(k_cache, v_cache, k_scale, v_scale, dev)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise OrbitError("slots must be a tensor of one dimension")
    _tensor(slots, "slots", dev, slots.shape, torch.int64)
    if dtype is None:
        dtype = torch.float16 if cache[8] == 3 else k_cache.dtype
    if dtype not in _DT:
        raise OrbitError("dtype must be float32, bfloat16 or float16")
    shape = (slots.shape[0], cache[6], cache[7])
    k, v = k_cache.new_empty(shape, dtype=dtype), k_cache.new_empty(shape, dtype=dtype)
    _launch(lib.orbit_kv_read, "orbit_kv_read", dev, _CACHE.pack(*cache), slots.data_ptr(),
            shape[0], k.data_ptr(), v.data_ptr(), _DT[dtype])
    return k, v


def paged_attention(q, k_cache, v_cache, block_table, lengths, *, scale=None, window=0,
                    k_scale=None, v_scale=None, out=None, return_lse=False):
    """Attention of one new token per request over the paged cache.

    q: [batch, q_heads, dim] bfloat16 or float16 (the cache's dtype, either
    for int8); block_table: int32 [batch, width], the pages of each request;
    lengths: int32 [batch], the tokens each sees (0: the output is 0, its lse
    -inf).  Head h reads the keys of head h // (q_heads // kv_heads).  scale:
    1 / sqrt(dim) by default.  window > 0: the last `window` tokens alone.
    Returns out [batch, q_heads, dim], with return_lse also lse float32
    [batch, q_heads].
    """
    dev = _first(q, "q", 3)
    qt = _float(q, "q")
    cache = _cache_fields(k_cache, v_cache, k_scale, v_scale, dev)
    batch, H, dim = q.shape
    q0, q1, _ = _tensor(q, "q", dev, (batch, H, cache[7]), q.dtype)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise OrbitError("block_table must be a tensor [batch, pages]")
    width = block_table.shape[1]
    ts = _tensor(block_table, "block_table", dev, (batch, width), torch.int32)[0]
    _tensor(lengths, "lengths", dev, (batch,), torch.int32)
    if out is None:
        out = q.new_empty((batch, H, dim))
    else:
        _tensor(out, "out", dev, (batch, H, dim), q.dtype)
        if not out.is_contiguous():
            raise OrbitError("out must be contiguous")
    lse = q.new_empty((batch, H), dtype=torch.float32) if return_lse else None
    ws = lib.orbit_paged_attention_workspace(batch, H, cache[6], dim, cache[5], width, window, cache[8])
    if ws < 0:
        raise OrbitError(f"orbit_paged_attention: invalid shape (batch {batch}, {H} query heads on "
                         f"{cache[6]}, dim {dim}, window {window})")
    work = q.new_empty((ws,), dtype=torch.uint8) if ws else None
    _launch(lib.orbit_paged_attention, "orbit_paged_attention", dev, _ATTENTION_ARGS.pack(
        *cache, q.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(),
        block_table.data_ptr(), lengths.data_ptr(), 0 if work is None else work.data_ptr(), ws,
        q0, q1, ts, batch, H, width, window, dim ** -0.5 if scale is None else scale, qt))
    return (out, lse) if return_lse else out
