"""The whole sublayer without a GPU: its struct, descriptors that do not fit, refusals."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

import sparse_mixture_experts_49_amd as moe
from sparse_mixture_experts_49_amd import binding as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_mi355x.h")
T, D, F, E, K, S = 8, 256, 512, 16, 2, 384


def _block(norm={}, route={}, experts={}, up={}, down={}, shared=True):
    b = moe.MxBlock(moe.NormDesc(**{**dict(rows=T, d=D), **norm}), moe.ScoreDesc(**{**dict(tokens=T, d_model=D, n_experts=E, top_k=K), **route}),
                    moe.MxDesc(**{**dict(tokens=T, d_model=D, d_ff=F, n_experts=E, top_k=K), **experts}), None, None)
    if shared:
        b.up = moe.LoraDesc(**{**dict(tokens=T, d_in=D, d_out=S, rank=8, n_adapters=2, act="gelu"), **up})
        b.down = moe.LoraDesc(**{**dict(tokens=T, d_in=S, d_out=D, rank=8, n_adapters=2, out_dtype="f32"), **down})
    return b


def test_header_struct_matches_binding():
    body = re.search(r"typedef struct moe_mx_block \{(.*?)\} moe_mx_block;", open(HEADER).read(), re.S).group(1)
    fields = re.findall(r"\*?\s*(\w+)\s*;", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
    assert fields == [f for f, _ in B.CMxBlock._fields_]


def test_workspace_holds_the_parts():
    size = moe.moe_mx_block_workspace_size
    b = _block()
    assert size(b) >= moe.moe_mx_workspace_size(b.experts) + moe.moe_score_workspace_size(b.route) + \
        moe.moe_lora_shared_workspace_size(b.up, b.down) + T * D * 6
    assert size(_block(shared=False)) < size(b)


@pytest.mark.parametrize("kw,status", [
    (dict(norm=dict(rows=7)), B.MOE_ERR_INVALID), (dict(norm=dict(d=128)), B.MOE_ERR_INVALID),
    (dict(norm=dict(dtype="f32")), B.MOE_ERR_UNSUPPORTED), (dict(route=dict(tokens=9)), B.MOE_ERR_INVALID),
    (dict(route=dict(dtype="f32")), B.MOE_ERR_UNSUPPORTED), (dict(experts=dict(top_k=3)), B.MOE_ERR_INVALID),
    (dict(up=dict(tokens=9), down=dict(tokens=9)), B.MOE_ERR_INVALID),
    (dict(up=dict(d_in=128), down=dict(d_out=128)), B.MOE_ERR_INVALID),
    (dict(down=dict(out_dtype="bf16")), B.MOE_ERR_INVALID), (dict(experts=dict(d_ff=100)), B.MOE_ERR_UNSUPPORTED),
])
def test_descriptors_that_do_not_fit(kw, status):
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_mx_block_workspace_size(_block(**kw))
    assert ei.value.status == status
    one = _block()
    one.down = None
    with pytest.raises(moe.MoeError):
        moe.moe_mx_block_workspace_size(one)


P = {n: 0x10000000 * (i + 1) for i, n in enumerate(("x", "add", "x_out", "y", "w_router", "adapter", "ws", "mx", "lora"))}


def _forward(shared=True, n=None, **kw):
    lib = moe.load_library()
    p = {**P, **kw}
    s, keep = B._mx_block(_block(shared=shared), None, None)
    m = p["mx"]
    mx = B.CMxWeights(*((m + 0x1000000 * i if m else None) for i in range(6)))
    l = p["lora"]
    lw = B.CLoraWeights(*((l + 0x100000 * i if l and i < 4 else None) for i in range(5)))
    s.w_router, s.w = p["w_router"], ctypes.cast(ctypes.pointer(mx), ctypes.c_void_p)
    s.adapter = p["adapter"]
    s.w_up = s.w_down = ctypes.cast(ctypes.pointer(lw), ctypes.c_void_p)
    rows = lambda q: None if q is None else ctypes.byref(B.CRows(q, D))  # noqa: E731
    size = ctypes.c_size_t(0)
    assert lib.moe_mx_block_workspace_size(ctypes.byref(s), ctypes.byref(size)) == 0
    st = lib.moe_mx_block_forward(ctypes.byref(s), rows(p["x"]), rows(p["add"]), rows(p["x_out"]), p["y"], None,
                                  p["ws"], size.value if n is None else size.value + n, None)
    del keep
    return st, lib.moe_last_error().decode()


def test_refusals():
    for kw in (dict(x=None), dict(x=P["x"] + 8), dict(add=P["add"] + 8), dict(y=None), dict(w_router=None), dict(mx=None),
               dict(adapter=None), dict(lora=None), dict(x_out=P["x"]), dict(y=P["add"]), dict(y=P["ws"] + 4096),
               dict(ws=P["lora"])):
        assert _forward(**kw)[0] == B.MOE_ERR_INVALID, kw
    for kw in (dict(ws=None), dict(ws=P["ws"] + 16), dict(n=-1)):
        assert _forward(**kw)[0] == B.MOE_ERR_WORKSPACE, kw


def test_outputs_over_strided_rows_are_refused():
    """What lies between two rows counts as theirs, but for x, add and x_out among themselves."""
    lib = moe.load_library()
    wide = 1024
    assert _forward(y=P["x_out"])[0] == B.MOE_ERR_INVALID and _forward(x_out=P["w_router"])[0] == B.MOE_ERR_INVALID
    assert _forward(x_out=P["ws"])[0] == B.MOE_ERR_INVALID and _forward(x_out=P["add"] + 16)[0] == B.MOE_ERR_INVALID
    s, keep = B._mx_block(_block(shared=False), None, None)
    mx = B.CMxWeights(*(P["mx"] + 0x1000000 * i for i in range(6)))
    s.w_router, s.w = P["w_router"], ctypes.cast(ctypes.pointer(mx), ctypes.c_void_p)
    size = ctypes.c_size_t(0)
    assert lib.moe_mx_block_workspace_size(ctypes.byref(s), ctypes.byref(size)) == 0
    rows = lambda q: ctypes.byref(B.CRows(q, wide))  # noqa: E731
    for x_out, y in ((P["x"], P["y"]), (P["x"] + 2 * D - 16, P["y"]), (P["x"] + 2 * D, P["x"] + 4 * D),
                     (P["x_out"], P["x_out"] + 2 * D)):
        st = lib.moe_mx_block_forward(ctypes.byref(s), rows(P["x"]), None, rows(x_out), y, None, P["ws"], size, None)
        assert st == B.MOE_ERR_INVALID, (hex(x_out), hex(y))
    del keep
