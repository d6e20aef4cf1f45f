"""The layer norm without a GPU: structs, refusals before any HIP call, workspace."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

import sparse_mixture_experts_49_amd as moe
from sparse_mixture_experts_49_amd import binding as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_mi355x.h")
X, ADD, W, XO, Y, M, R, WS = (0x1000000 * (i + 1) for i in range(8))


def test_header_structs_match_binding():
    text = open(HEADER).read()
    for struct, cls in (("moe_norm_desc", B.CNormDesc), ("moe_rows", B.CRows)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), text, re.S).group(1)
        fields = re.findall(r"\*?\s*(\w+)\s*;", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
        assert fields == [f for f, _ in cls._fields_], struct


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), B.MOE_ERR_INVALID), (dict(d=0), B.MOE_ERR_INVALID), (dict(d=32769), B.MOE_ERR_UNSUPPORTED),
    (dict(rows=1 << 40), B.MOE_ERR_UNSUPPORTED), (dict(dtype="f16"), B.MOE_ERR_INVALID),
    (dict(param_dtype="x"), B.MOE_ERR_INVALID), (dict(add_dtype="x"), B.MOE_ERR_INVALID),
    (dict(eps=float("nan")), B.MOE_ERR_INVALID), (dict(eps=-1e-5), B.MOE_ERR_INVALID),
])
def test_invalid_descriptors(kw, status):
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_norm_workspace_size(moe.NormDesc(**{**dict(rows=4, d=256), **kw}))
    assert ei.value.status == status


def _rows(p, stride=256):
    return None if p is None else ctypes.byref(B.CRows(p, stride))


def _forward(d=None, x=X, add=ADD, w=W, x_out=XO, y=Y, mean=M, rstd=R, strides=(256, 256, 256, 256)):
    lib = moe.load_library()
    d = d or moe.NormDesc(4, 256)
    st = lib.moe_layer_norm(d.ref(), _rows(x, strides[0]), _rows(add, strides[1]), w, None, _rows(x_out, strides[2]),
                            _rows(y, strides[3]), mean, rstd, None)
    return st, lib.moe_last_error().decode()


def test_forward_refusals():
    assert _forward(x=None)[0] == B.MOE_ERR_INVALID
    assert _forward(y=None)[0] == B.MOE_ERR_INVALID
    assert _forward(y=Y + 8)[0] == B.MOE_ERR_INVALID
    assert _forward(w=W + 4)[0] == B.MOE_ERR_INVALID
    assert _forward(mean=M + 4)[0] == B.MOE_ERR_INVALID
    assert _forward(strides=(255, 256, 256, 256))[0] == B.MOE_ERR_INVALID
    assert _forward(strides=(256, 256, 256, -256))[0] == B.MOE_ERR_INVALID
    assert _forward(strides=(256, 256, 256, 1 << 39))[0] == B.MOE_ERR_UNSUPPORTED
    st, msg = _forward(y=X)                                 # in place
    assert st == B.MOE_ERR_INVALID and "y overlaps x" in msg
    st, msg = _forward(x_out=Y + 1536)                      # the last row of y
    assert st == B.MOE_ERR_INVALID and "overlaps" in msg
    # columns of one buffer: 256 and 256 of 512 do not meet, 256 and 248 of 504 do
    assert "overlaps" in _forward(y=X + 496, strides=(512, 256, 256, 512))[1]
    assert "overlaps" in _forward(y=X + 512, strides=(504, 256, 256, 504))[1]


def _backward(dy=X, x=ADD, mean=M, rstd=R, res=None, dx=XO, dw=Y, db=None, ws=WS, n=None):
    lib = moe.load_library()
    d = moe.NormDesc(4, 256)
    n = moe.moe_norm_workspace_size(d) if n is None else n
    st = lib.moe_layer_norm_backward(d.ref(), _rows(dy), _rows(x), None, mean, rstd, _rows(res), _rows(dx), dw, db, ws,
                                     n, None)
    return st, lib.moe_last_error().decode()


def test_backward_refusals():
    n = moe.moe_norm_workspace_size(moe.NormDesc(4, 256))
    for kw in (dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None, dw=None),
               dict(dx=None, res=W), dict(dx=X), dict(dw=Y + 4), dict(db=Y + 512), dict(dx=M)):
        assert _backward(**kw)[0] == B.MOE_ERR_INVALID, kw
    for kw in (dict(ws=None), dict(ws=WS + 16), dict(n=n - 1)):
        assert _backward(**kw)[0] == B.MOE_ERR_WORKSPACE, kw


def test_binding_refusals():
    import torch
    with pytest.raises(moe.MoeError, match="expected a GPU"):
        moe.moe_layer_norm(moe.NormDesc(2, 8), torch.zeros(2, 8), torch.zeros(2, 8))
    with pytest.raises(moe.MoeError, match="must be a torch tensor"):
        moe.moe_layer_norm(moe.NormDesc(2, 8), None, None)
