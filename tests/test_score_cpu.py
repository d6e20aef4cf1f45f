"""The scored router without a GPU: its structs match the header, its descriptor and
pointers are checked before any HIP call, and its workspace grows with the shape."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

import sparse_mixture_experts_49_amd as moe
from sparse_mixture_experts_49_amd import binding as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_mi355x.h")
BASE = dict(tokens=64, d_model=256, n_experts=32, top_k=4, n_groups=4, top_groups=2, group_top=2)


def test_header_structs_match_binding():
    text = open(HEADER).read()
    for struct, cls in (("moe_score_desc", B.CScoreDesc), ("moe_score_out", B.CScoreOut),
                        ("moe_score_grads", B.CScoreGrads)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), text, re.S).group(1)
        fields = re.findall(r"\*?\s*(\w+)\s*;", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
        assert fields == [f for f, _ in cls._fields_], struct


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), B.MOE_ERR_INVALID),
    (dict(d_model=200), B.MOE_ERR_UNSUPPORTED),
    (dict(n_experts=257, n_groups=1, top_groups=1), B.MOE_ERR_UNSUPPORTED),
    (dict(n_experts=0), B.MOE_ERR_INVALID),
    (dict(top_k=0), B.MOE_ERR_INVALID),
    (dict(top_k=9), B.MOE_ERR_UNSUPPORTED),
    (dict(top_groups=1, top_k=9), B.MOE_ERR_INVALID),      # more than the groups' 8 experts
    (dict(n_groups=5), B.MOE_ERR_INVALID),
    (dict(n_groups=0), B.MOE_ERR_INVALID),
    (dict(top_groups=5), B.MOE_ERR_INVALID),
    (dict(group_top=3), B.MOE_ERR_INVALID),
    (dict(n_groups=32, group_top=2, top_groups=8), B.MOE_ERR_INVALID),   # groups of one expert
    (dict(n_experts=256, n_groups=128, top_groups=8), B.MOE_ERR_UNSUPPORTED),
    (dict(dtype="f16"), B.MOE_ERR_INVALID),
    (dict(score="tanh"), B.MOE_ERR_INVALID),
    (dict(scale=float("nan")), B.MOE_ERR_INVALID),
    (dict(scale=float("inf")), B.MOE_ERR_INVALID),
    (dict(tokens=1 << 26), B.MOE_ERR_UNSUPPORTED),
])
def test_invalid_descriptors(kw, status):
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_score_workspace_size(moe.ScoreDesc(**{**BASE, **kw}))
    assert ei.value.status == status


def test_workspace_grows_with_the_shape():
    size = moe.moe_score_workspace_size
    assert 0 < size(moe.ScoreDesc(1, 256, 8, 2)) < size(moe.ScoreDesc(4096, 4096, 256, 8))


def _route(desc, x=0x100000, w=0x200000, br=None, bs=None, idx=0x300000, tw=0x310000, load=None, ws=0x1000000,
           ws_bytes=None):
    lib = moe.load_library()
    out = B.CScoreOut(idx, tw, None, load, None, None, None)
    n = moe.moe_score_workspace_size(desc) if ws_bytes is None else ws_bytes
    st = lib.moe_score_route(ctypes.byref(desc.to_c()), x, w, br, bs, ctypes.byref(out), ws, n, None)
    return st, lib.moe_last_error().decode()


def test_route_refusals():
    d = moe.ScoreDesc(**BASE)
    n = moe.moe_score_workspace_size(d)
    assert _route(d, x=None)[0] == B.MOE_ERR_INVALID
    assert _route(d, w=0x200008)[0] == B.MOE_ERR_INVALID
    assert _route(d, bs=0x5004)[0] == B.MOE_ERR_INVALID
    assert _route(d, idx=None)[0] == B.MOE_ERR_INVALID
    assert _route(d, tw=None)[0] == B.MOE_ERR_INVALID
    assert _route(d, load=0x400004)[0] == B.MOE_ERR_INVALID
    assert _route(d, ws=None)[0] == B.MOE_ERR_WORKSPACE
    assert _route(d, ws=0x1000010)[0] == B.MOE_ERR_WORKSPACE
    assert _route(d, ws_bytes=n - 1)[0] == B.MOE_ERR_WORKSPACE
    st, msg = _route(d, tw=0x300000 + 512)                 # 64 * 4 indices are 1 KiB
    assert st == B.MOE_ERR_INVALID and "overlaps" in msg
    st, msg = _route(d, idx=0x100000 + 4096)
    assert st == B.MOE_ERR_INVALID and "overlaps x" in msg


def _backward(desc, grads, x=0x100000, w=0x200000, idx=0x300000, logits=0x400000, load=None, dw=0x500000,
              daux=None):
    lib = moe.load_library()
    fwd = B.CScoreOut(idx, None, logits, load, None, None, None)
    st = lib.moe_score_backward(ctypes.byref(desc.to_c()), x, w, ctypes.byref(fwd), dw, daux, None,
                                ctypes.byref(B.CScoreGrads(*grads)), 0x10000000,
                                moe.moe_score_workspace_size(desc), None)
    return st, lib.moe_last_error().decode()


def test_backward_refusals():
    d = moe.ScoreDesc(**BASE)
    dx = (0x600000, None, None, None)
    assert _backward(d, (None,) * 4)[0] == B.MOE_ERR_INVALID
    assert _backward(d, dx, w=None)[0] == B.MOE_ERR_INVALID
    assert _backward(d, (None, 0x600000, None, None), x=None)[0] == B.MOE_ERR_INVALID
    assert _backward(d, dx, logits=None)[0] == B.MOE_ERR_INVALID
    assert _backward(d, dx, idx=0x300004)[0] == B.MOE_ERR_INVALID
    assert _backward(d, dx, daux=0x700000)[0] == B.MOE_ERR_INVALID           # load is missing
    st, msg = _backward(d, (0x400000, None, None, None))
    assert st == B.MOE_ERR_INVALID and "d_x overlaps logits" in msg


def test_binding_refuses_host_tensors():
    import torch
    d = moe.ScoreDesc(4, 128, 8, 2, dtype="f32")
    with pytest.raises(moe.MoeError, match="expected a GPU"):
        moe.moe_score_route(d, torch.zeros(4, 128), torch.zeros(8, 128), moe.ScoreRouting.allocate(d, "cpu"))
    with pytest.raises(moe.MoeError, match="must be a torch tensor"):
        moe.moe_score_backward(d, None, None, moe.ScoreRouting(), None, moe.ScoreGrads())
