"""The MXFP4 experts without a GPU: structs, descriptors and pointers are checked before
any HIP call; the 64-bit reference agrees with torch on what torch can say."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

import sparse_mixture_experts_49_amd as moe
from sparse_mixture_experts_49_amd import binding as B
from tests import _mx_ref as R

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_mi355x.h")
BASE = dict(tokens=64, d_model=256, d_ff=512, n_experts=8, top_k=2)


def test_header_structs_match_binding():
    text = open(HEADER).read()
    for struct, cls in (("moe_mx_desc", B.CMxDesc), ("moe_mx_weights", B.CMxWeights)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), text, re.S).group(1)
        fields = re.findall(r"\*?\s*(\w+)\s*;", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
        assert fields == [f for f, _ in cls._fields_], struct


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), B.MOE_ERR_INVALID), (dict(n_experts=0), B.MOE_ERR_INVALID),
    (dict(n_experts=257), B.MOE_ERR_UNSUPPORTED), (dict(top_k=0), B.MOE_ERR_INVALID),
    (dict(top_k=9, n_experts=16), B.MOE_ERR_UNSUPPORTED), (dict(top_k=9), B.MOE_ERR_INVALID),
    (dict(d_model=96), B.MOE_ERR_UNSUPPORTED), (dict(d_ff=160), B.MOE_ERR_UNSUPPORTED),
    (dict(act="fp8"), B.MOE_ERR_INVALID), (dict(tokens=1 << 20, d_ff=4096), B.MOE_ERR_UNSUPPORTED),
    (dict(tokens=1, top_k=1, d_model=65536, d_ff=65536), B.MOE_ERR_UNSUPPORTED),
])
def test_invalid_descriptors(kw, status):
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_mx_workspace_size(moe.MxDesc(**{**BASE, **kw}))
    assert ei.value.status == status


def _err(st):
    return st, moe.load_library().moe_last_error().decode()


@pytest.mark.parametrize("args,word", [
    ((0x1000, 1, 4, 48, 48, 0x8000, 0x9000), "cols"), ((0x1000, 1, 4, 0, 32, 0x8000, 0x9000), "cols"),
    ((0x1000, 1, -1, 64, 64, 0x8000, 0x9000), "rows"), ((0x1000, 1, 4, 64, 32, 0x8000, 0x9000), "row_stride"),
    ((0x1000, 1, 4, 64, 68, 0x8000, 0x9000), "row_stride"), ((0x1000, 2, 4, 64, 64, 0x8000, 0x9000), "dtype"),
    ((0x1008, 1, 4, 64, 64, 0x8000, 0x9000), "aligned"), ((None, 1, 4, 64, 64, 0x8000, 0x9000), "x must"),
    ((0x1000, 1, 4, 64, 64, 0x8000, None), "scales"), ((0x1000, 1, 4, 64, 64, 0x1000 + 256, 0x9000), "overlaps x"),
    ((0x1000, 1, 4, 64, 64, 0x8000, 0x8000 + 112), "overlaps"),
])
def test_quantize_refusals(args, word):
    st, msg = _err(moe.load_library().moe_mx_quantize(*args, None))
    assert st == B.MOE_ERR_INVALID and word in msg, msg


def test_no_rows_is_no_work():
    lib = moe.load_library()
    assert lib.moe_mx_quantize(None, 1, 0, 64, 64, None, None, None) == B.MOE_OK
    assert lib.moe_mx_dequantize(None, None, 0, 64, 1, None, 64, None) == B.MOE_OK


def _up(desc, x=0x10000000, src=None, off=0x100000, w=(0x20000000, 0x21000000, 0x22000000, None, None, None),
        h=0x30000000, ws=0x40000000, nb=None):
    lib = moe.load_library()
    nb = moe.moe_mx_workspace_size(desc) if nb is None else nb
    return _err(lib.moe_mx_ffn_up(ctypes.byref(desc.to_c()), x, src, off, ctypes.byref(B.CMxWeights(*w)), h, ws, nb, None))


def test_product_refusals():
    d = moe.MxDesc(**BASE)
    assert _up(d, x=None)[0] == B.MOE_ERR_INVALID
    assert _up(d, src=0x5004)[0] == B.MOE_ERR_INVALID
    assert _up(d, off=None)[0] == B.MOE_ERR_INVALID
    assert "b1" in _up(d, w=(0x20000000, 0x21000000, None, None, None, None))[1]
    assert "s1" in _up(d, w=(0x20000000, None, 0x22000000, None, None, None))[1]
    assert _up(d, ws=None)[0] == B.MOE_ERR_WORKSPACE
    assert _up(d, nb=moe.moe_mx_workspace_size(d) - 1)[0] == B.MOE_ERR_WORKSPACE
    assert "h overlaps w1" in _up(d, h=0x20000000 + 4096)[1]
    assert "h overlaps x" in _up(d, h=0x10000000 + 4096)[1]
    nob = moe.MxDesc(**BASE, has_expert_bias=False)
    assert "has_expert_bias" in _up(nob)[1]


def test_forward_refusals():
    lib = moe.load_library()
    d = moe.MxDesc(**BASE, has_expert_bias=False)
    w = B.CMxWeights(0x20000000, 0x21000000, None, 0x22000000, 0x23000000, None)

    def call(route, y=0x30000000, more=0):
        nb = moe.moe_mx_workspace_size(d) + moe.moe_score_workspace_size(route) + more
        return _err(lib.moe_mx_forward(ctypes.byref(route.to_c()), ctypes.byref(d.to_c()), 0x10000000, 0x11000000,
                                       None, None, ctypes.byref(w), y, None, 0x40000000, nb, None))

    assert "differ" in call(moe.ScoreDesc(64, 256, 8, 1))[1]
    assert "differ" in call(moe.ScoreDesc(32, 256, 8, 2))[1]
    assert call(moe.ScoreDesc(64, 256, 8, 2, dtype="f32"))[0] == B.MOE_ERR_UNSUPPORTED
    assert call(moe.ScoreDesc(64, 256, 8, 2), more=-1)[0] == B.MOE_ERR_WORKSPACE
    assert "y overlaps" in call(moe.ScoreDesc(64, 256, 8, 2), y=0x40000000 + 512)[1]
    assert "y overlaps w2" in call(moe.ScoreDesc(64, 256, 8, 2), y=0x22000000 + 256)[1]


def test_binding_refuses_what_it_cannot_read():
    codes, scales = moe.alloc_mx(4, 64, "cpu")
    with pytest.raises(moe.MoeError, match="expected a GPU"):
        moe.moe_mx_quantize(torch.zeros(4, 64), codes, scales)
    with pytest.raises(moe.MoeError, match="must be a torch tensor"):
        moe.moe_mx_ffn_up(moe.MxDesc(**BASE), None, None, moe.MxWeights(), None)


def test_reference_rounds_to_nearest_even():
    x = torch.tensor([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9] + [0.0] * 23 + [-4.0]])
    codes, scales = R.quantize(x)
    assert scales.tolist() == [[127]]
    assert R.values(codes, scales)[0, :8].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0]


@pytest.mark.parametrize("rows,cols", [(2 ** 29, 64), (2 ** 28 + 1, 64), (1, 2 ** 35)])
def test_more_values_than_a_launch_has_threads(rows, cols):
    lib = moe.load_library()
    for st in (lib.moe_mx_quantize(0x1000, 1, rows, cols, cols, 0x8000, 0x9000, None),
               lib.moe_mx_dequantize(0x8000, 0x9000, rows, cols, 1, 0x1000, cols, None)):
        assert st == B.MOE_ERR_UNSUPPORTED and "2^34" in lib.moe_last_error().decode()


def test_only_the_combine_takes_more_than_64_experts():
    """moe_combine takes the layers of moe_mx_dispatch, up to 256 experts; the others of its
    family keep to 64."""
    lib = moe.load_library()

    def combine(E, o=0x100000):
        d = moe.Desc(4, 128, 128, E, 2)
        return _err(lib.moe_combine(ctypes.byref(d.to_c()), o, 0x200000, 0x300000, None, 0x100100, None))

    for E in (64, 65, 256):
        st, msg = combine(E)
        assert st == B.MOE_ERR_INVALID and "y overlaps o" in msg, msg
        assert "o must not be NULL" in combine(E, o=None)[1]
    st, msg = combine(257)
    assert st == B.MOE_ERR_UNSUPPORTED and "256" in msg
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_workspace_size(moe.Desc(4, 128, 128, 65, 2))
    assert ei.value.status == B.MOE_ERR_UNSUPPORTED
