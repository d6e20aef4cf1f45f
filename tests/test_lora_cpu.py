"""The projection with low-rank adapters without a GPU: structs, refusals, workspace."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

import sparse_mixture_experts_49_amd as moe
from sparse_mixture_experts_49_amd import binding as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_mi355x.h")
BASE = dict(tokens=64, d_in=256, d_out=384, rank=16, n_adapters=4)
X, AD, W, A, BB, S, BIAS, Y, WS = (0x1000000 * (i + 1) for i in range(9))


def test_header_structs_match_binding():
    text = open(HEADER).read()
    for struct, cls in (("moe_lora_desc", B.CLoraDesc), ("moe_lora_weights", B.CLoraWeights)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), text, re.S).group(1)
        fields = re.findall(r"\*?\s*(\w+)\s*;", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
        assert fields == [f for f, _ in cls._fields_], struct


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), B.MOE_ERR_INVALID), (dict(d_in=0), B.MOE_ERR_INVALID), (dict(d_in=200), B.MOE_ERR_UNSUPPORTED),
    (dict(d_out=64), B.MOE_ERR_UNSUPPORTED), (dict(rank=0), B.MOE_ERR_INVALID), (dict(rank=12), B.MOE_ERR_UNSUPPORTED),
    (dict(rank=136), B.MOE_ERR_UNSUPPORTED), (dict(n_adapters=0), B.MOE_ERR_INVALID),
    (dict(n_adapters=4097), B.MOE_ERR_UNSUPPORTED), (dict(act="relu"), B.MOE_ERR_INVALID),
    (dict(out_dtype="f16"), B.MOE_ERR_INVALID), (dict(tokens=1 << 23, d_in=256), B.MOE_ERR_UNSUPPORTED),
    (dict(d_in=1 << 16, d_out=1 << 15), B.MOE_ERR_UNSUPPORTED),
])
def test_invalid_descriptors(kw, status):
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_lora_workspace_size(moe.LoraDesc(**{**BASE, **kw}))
    assert ei.value.status == status


def _linear(d=None, x=X, ad=AD, w=W, a=A, b=BB, s=S, bias=None, y=Y, ws=WS, n=None):
    lib, d = moe.load_library(), d or moe.LoraDesc(**BASE)
    n = moe.moe_lora_workspace_size(d) if n is None else n
    weights = B.CLoraWeights(w, a, b, s, bias)
    st = lib.moe_lora_linear(d.ref(), x, ad, ctypes.byref(weights), y, ws, n, None)
    return st, lib.moe_last_error().decode()


def test_linear_refusals():
    n = moe.moe_lora_workspace_size(moe.LoraDesc(**BASE))
    for kw in (dict(x=None), dict(ad=None), dict(w=None), dict(a=None), dict(b=None), dict(y=None), dict(x=X + 8),
               dict(ad=AD + 4), dict(s=S + 4), dict(bias=BIAS), dict(d=moe.LoraDesc(**BASE, has_bias=True)),
               dict(y=X + 64), dict(y=BB + 128), dict(y=WS)):
        assert _linear(**kw)[0] == B.MOE_ERR_INVALID, kw
    for kw in (dict(ws=None), dict(ws=WS + 16), dict(n=n - 1)):
        assert _linear(**kw)[0] == B.MOE_ERR_WORKSPACE, kw


def test_pairs_that_are_no_shared_expert():
    up = dict(BASE, act="gelu")
    down = dict(BASE, d_in=384, d_out=256, out_dtype="f32")
    size = moe.moe_lora_shared_workspace_size
    assert size(moe.LoraDesc(**up), moe.LoraDesc(**down)) >= 64 * 384 * 2
    for u, d in ((dict(up, tokens=63), down), (up, dict(down, d_in=512)), (dict(up, d_in=512), down),
                 (dict(up, act="none"), down), (dict(up, out_dtype="f32"), down), (up, dict(down, act="gelu")),
                 (up, dict(down, out_dtype="bf16"))):
        with pytest.raises(moe.MoeError) as ei:
            size(moe.LoraDesc(**u), moe.LoraDesc(**d))
        assert ei.value.status == B.MOE_ERR_INVALID


def test_binding_refuses_host_tensors():
    import torch
    z = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError, match="expected a GPU"):
        moe.moe_lora_linear(moe.LoraDesc(4, 128, 128, 8, 1), z, None, moe.LoraWeights(z, z, z), z)
