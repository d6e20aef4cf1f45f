"""ctypes binding of libmoe_mi355x.so: the C ABI's entry points under the same
names, taking torch tensors.  Argument marshalling only -- every step of the
layer runs in the library's HIP kernels.  There is no fallback: if the library
is missing the import of this module's functions raises."""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_mi355x.so")

MOE_DTYPE_F32, MOE_DTYPE_BF16 = 0, 1
MOE_OK, MOE_ERR_INVALID, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = 0, -1, -2, -3, -4
MOE_FFN_AUTO, MOE_FFN_TILED, MOE_FFN_STREAM = 0, 1, 2
MOE_H_AUTO, MOE_H_BF16, MOE_H_SPLIT = 0, 1, 2
MOE_CAPACITY_DROP, MOE_CAPACITY_REROUTE = 0, 1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
MOE_MX_ACT_BF16, MOE_MX_ACT_MXFP4 = 0, 1
_MX_ACTS = {"bf16": MOE_MX_ACT_BF16, "mxfp4": MOE_MX_ACT_MXFP4}
MOE_LORA_ACT_NONE, MOE_LORA_ACT_GELU = 0, 1
_LORA_ACTS = {"none": MOE_LORA_ACT_NONE, "gelu": MOE_LORA_ACT_GELU}
_DTYPES = {"bf16": MOE_DTYPE_BF16, "f32": MOE_DTYPE_F32}
_POLICIES = {"drop": MOE_CAPACITY_DROP, "reroute": MOE_CAPACITY_REROUTE}

ENTRY_POINTS = ("moe_status_string", "moe_last_error", "moe_workspace_size", "moe_query_plan",
                "moe_route", "moe_permute", "moe_ffn_up", "moe_ffn_up_gather", "moe_ffn_down", "moe_grouped_ffn",
                "moe_shared_ffn", "moe_combine", "moe_forward", "moe_forward_noalloc",
                "moe_read_probe", "moe_score_workspace_size", "moe_score_route",
                "moe_score_backward", "moe_mx_quantize", "moe_mx_dequantize", "moe_mx_workspace_size",
                "moe_mx_dispatch", "moe_mx_ffn_up", "moe_mx_ffn_down", "moe_mx_forward",
                "moe_score_backward_add", "moe_balance_workspace_size", "moe_balance_loss",
                "moe_balance_backward", "moe_norm_workspace_size", "moe_layer_norm",
                "moe_layer_norm_backward", "moe_lora_workspace_size", "moe_lora_linear",
                "moe_lora_shared_workspace_size", "moe_lora_shared_ffn", "moe_mx_block_workspace_size",
                "moe_mx_block_forward")


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


class CDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("tokens", "d_model", "d_ff", "n_experts", "top_k", "renormalize", "capacity",
                 "dtype", "has_expert_bias", "ffn_path", "h_mode", "d_ff_shared",
                 "capacity_policy")]


class CPlan(ctypes.Structure):
    _fields_ = [("ffn_path", ctypes.c_int32), ("h_mode", ctypes.c_int32),
                ("h_bytes", ctypes.c_size_t), ("workspace_bytes", ctypes.c_size_t)]


class CWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w_router", "b_router", "w1", "b1", "w2", "b2",
                                               "b_select", "w1_shared", "b1_shared", "w2_shared",
                                               "b2_shared")]


class CRouting(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("topk_idx", "topk_w", "counts", "offsets", "dest", "src", "top1_count",
                 "prob_mean", "z_loss", "reroute_rounds")]


class CScoreDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("tokens", "d_model", "n_experts", "top_k", "dtype", "score", "n_groups",
                 "top_groups", "group_top", "renormalize")] + [("scale", ctypes.c_float)]


class CScoreOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("topk_idx", "topk_w", "logits", "load", "prob_mean", "aux", "z_loss")]


class CScoreGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("d_x", "d_w_router", "d_b_router", "d_logits")]


class CMxDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("tokens", "d_model", "d_ff", "n_experts", "top_k", "act", "has_expert_bias")]


class CMxWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w1", "s1", "b1", "w2", "s2", "b2")]


class CBalanceDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tokens", "n_experts", "top_k", "n_seqs", "score")]


class CBalanceOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("load", "valid", "prob_mean", "seq_loss", "loss", "total_load")]


class CNormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("add_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class CLoraDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("tokens", "d_in", "d_out", "rank", "n_adapters", "act", "out_dtype", "has_bias")]


class CLoraWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w", "a", "b", "scale", "bias")]


class CMxBlock(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("norm", "weight", "bias", "route", "w_router", "b_router", "b_select", "experts", "w", "up", "down",
                 "w_up", "w_down", "adapter")]


class CRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64)]


_lib: Optional[ctypes.CDLL] = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m sparse_mixture_experts_49_amd.build`")
    lib = ctypes.CDLL(path)
    P, I, S, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
    pd, pw, pr = ctypes.POINTER(CDesc), ctypes.POINTER(CWeights), ctypes.POINTER(CRouting)
    sig = {
        "moe_status_string": (ctypes.c_char_p, [I]),
        "moe_last_error": (ctypes.c_char_p, []),
        "moe_workspace_size": (I, [pd, ctypes.POINTER(S)]),
        "moe_query_plan": (I, [pd, ctypes.POINTER(CPlan)]),
        "moe_route": (I, [pd, P, pw, pr, P, P, S, P]),
        "moe_permute": (I, [pd, P, pr, P, P, S, P]),
        "moe_ffn_up": (I, [pd, P, P, pw, P, P, S, P]),
        "moe_ffn_up_gather": (I, [pd, P, P, P, pw, P, P, S, P]),
        "moe_ffn_down": (I, [pd, P, P, pw, P, P, S, P]),
        "moe_grouped_ffn": (I, [pd, P, P, pw, P, P, P, S, P]),
        "moe_shared_ffn": (I, [pd, P, pw, P, P, S, P]),
        "moe_combine": (I, [pd, P, P, P, P, P, P]),
        "moe_forward": (I, [pd, P, pw, P, P, pr, P, S, P]),
        "moe_forward_noalloc": (I, [pd, P, pw, P, P, pr, P]),
        "moe_read_probe": (I, [P, S, P, P]),
        "moe_score_workspace_size": (I, [P, ctypes.POINTER(S)]),
        "moe_score_route": (I, [P, P, P, P, P, P, P, S, P]),
        "moe_score_backward": (I, [P, P, P, P, P, P, P, P, P, S, P]),
        "moe_score_backward_add": (I, [P, P, P, P, P, P, P, P, P, P, S, P]),
        "moe_balance_workspace_size": (I, [P, ctypes.POINTER(S)]),
        "moe_balance_loss": (I, [P, P, P, P, P, P, P, S, P]),
        "moe_balance_backward": (I, [P, P, P, P, P, P, P, P, P]),
        "moe_norm_workspace_size": (I, [P, ctypes.POINTER(S)]),
        "moe_layer_norm": (I, [P, P, P, P, P, P, P, P, P, P]),
        "moe_layer_norm_backward": (I, [P, P, P, P, P, P, P, P, P, P, P, S, P]),
        "moe_lora_workspace_size": (I, [P, ctypes.POINTER(S)]),
        "moe_lora_linear": (I, [P, P, P, P, P, P, S, P]),
        "moe_lora_shared_workspace_size": (I, [P, P, ctypes.POINTER(S)]),
        "moe_lora_shared_ffn": (I, [P, P, P, P, P, P, P, P, S, P]),
        "moe_mx_block_workspace_size": (I, [P, ctypes.POINTER(S)]),
        "moe_mx_block_forward": (I, [P, P, P, P, P, P, P, S, P]),
        "moe_mx_quantize": (I, [P, I, L, L, L, P, P, P]),
        "moe_mx_dequantize": (I, [P, P, L, L, I, P, L, P]),
        "moe_mx_workspace_size": (I, [P, ctypes.POINTER(S)]),
        "moe_mx_dispatch": (I, [P, pr, P, S, P]),
        "moe_mx_ffn_up": (I, [P, P, P, P, P, P, P, S, P]),
        "moe_mx_ffn_down": (I, [P, P, P, P, P, P, S, P]),
        "moe_mx_forward": (I, [P, P, P, P, P, P, P, P, P, P, S, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    _lib = lib
    return lib


@dataclasses.dataclass
class Desc:
    tokens: int
    d_model: int
    d_ff: int
    n_experts: int
    top_k: int
    renormalize: bool = True
    capacity: int = 0
    dtype: str = "bf16"          # "bf16" or "f32"
    has_expert_bias: bool = True
    ffn_path: int = MOE_FFN_AUTO
    h_mode: int = MOE_H_AUTO
    d_ff_shared: int = 0          # shared expert width, 0 = none
    capacity_policy: str = "drop"  # "drop" or "reroute": what happens past the capacity

    def to_c(self) -> CDesc:
        return CDesc(self.tokens, self.d_model, self.d_ff, self.n_experts, self.top_k,
                     int(bool(self.renormalize)), self.capacity,
                     MOE_DTYPE_BF16 if self.dtype == "bf16" else MOE_DTYPE_F32,
                     int(bool(self.has_expert_bias)), self.ffn_path, self.h_mode, self.d_ff_shared,
                     _POLICIES.get(self.capacity_policy, -1))

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype == "bf16" else torch.float32


@dataclasses.dataclass
class Weights:
    w_router: torch.Tensor
    w1: torch.Tensor
    w2: torch.Tensor
    b_router: Optional[torch.Tensor] = None
    b1: Optional[torch.Tensor] = None
    b2: Optional[torch.Tensor] = None
    b_select: Optional[torch.Tensor] = None
    w1_shared: Optional[torch.Tensor] = None
    b1_shared: Optional[torch.Tensor] = None
    w2_shared: Optional[torch.Tensor] = None
    b2_shared: Optional[torch.Tensor] = None

    def to_c(self) -> CWeights:
        return CWeights(*(_ptr(getattr(self, n)) for n, _ in CWeights._fields_))


@dataclasses.dataclass
class Routing:
    topk_idx: Optional[torch.Tensor] = None
    topk_w: Optional[torch.Tensor] = None
    counts: Optional[torch.Tensor] = None
    offsets: Optional[torch.Tensor] = None
    dest: Optional[torch.Tensor] = None
    src: Optional[torch.Tensor] = None
    top1_count: Optional[torch.Tensor] = None
    prob_mean: Optional[torch.Tensor] = None
    z_loss: Optional[torch.Tensor] = None
    reroute_rounds: Optional[torch.Tensor] = None

    @classmethod
    def allocate(cls, desc: Desc, device) -> "Routing":
        T, k, E = desc.tokens, desc.top_k, desc.n_experts
        i32 = dict(dtype=torch.int32, device=device)
        return cls(topk_idx=torch.empty(T, k, **i32),
                   topk_w=torch.empty(T, k, dtype=torch.float32, device=device),
                   counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                   dest=torch.empty(T, k, **i32), src=torch.empty(T * k, **i32),
                   top1_count=torch.empty(E, **i32),
                   prob_mean=torch.empty(E, dtype=torch.float32, device=device),
                   z_loss=torch.empty(1, dtype=torch.float32, device=device),
                   reroute_rounds=torch.empty(1, **i32))

    def to_c(self) -> CRouting:
        return CRouting(*(_ptr(getattr(self, f.name)) for f in dataclasses.fields(self)))


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE library must be contiguous")
    return t.data_ptr()


def _expected(desc: "Desc") -> dict:
    """(dtype, element count) of every array the C ABI sizes from the descriptor,
    by argument name (the same shapes the library's alias and bounds logic uses)."""
    T, d, F, E, k, Fs = (desc.tokens, desc.d_model, desc.d_ff, desc.n_experts, desc.top_k,
                         desc.d_ff_shared)
    dt, f32, i32 = desc.torch_dtype, torch.float32, torch.int32
    return {"x": (dt, T * d), "w_router": (dt, E * d), "b_router": (f32, E), "b_select": (f32, E),
            "w1": (dt, E * F * d), "b1": (dt, E * F), "w2": (dt, E * d * F), "b2": (dt, E * d),
            "w1_shared": (dt, Fs * d), "b1_shared": (dt, Fs), "w2_shared": (dt, d * Fs),
            "b2_shared": (dt, d),
            "topk_idx": (i32, T * k), "topk_w": (f32, T * k), "counts": (i32, E),
            "offsets": (i32, E + 1), "dest": (i32, T * k), "src": (i32, T * k),
            "top1_count": (i32, E), "prob_mean": (f32, E), "z_loss": (f32, 1),
            "reroute_rounds": (i32, 1),
            "x_perm": (dt, T * k * d), "o": (f32, T * k * d), "y": (f32, T * d),
            "o_shared": (f32, T * d), "aux": (f32, 1)}


def check_tensor(t, name: str, dtype, numel: int, device) -> None:
    """Refuse, before any call into the library, a tensor the library would read or
    write out of bounds or misinterpret: not on `device` (a GPU), wrong dtype, fewer
    than `numel` elements, or not contiguous.  Raw integer pointers are the
    caller's responsibility and pass unchecked."""
    if t is None or isinstance(t, int):
        return
    if not isinstance(t, torch.Tensor):
        raise MoeError(MOE_ERR_INVALID, f"{name} must be a torch tensor, an int pointer or None")
    if (t.device != device) if device is not None else (t.device.type != "cuda"):
        raise MoeError(MOE_ERR_INVALID, f"{name} is on {t.device}, expected {device or 'a GPU'}")
    if dtype is not None and t.dtype != dtype:
        raise MoeError(MOE_ERR_INVALID, f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.numel() < numel:
        raise MoeError(MOE_ERR_INVALID, f"{name} has {t.numel()} elements, needs {numel}")
    if not t.is_contiguous():
        raise MoeError(MOE_ERR_INVALID, f"{name} must be contiguous")


def _device_of(*ts):
    for t in ts:
        if isinstance(t, torch.Tensor):
            return t.device
    return None


class _Args:
    """Checks the tensors of one call against the descriptor (see check_tensor)."""

    def __init__(self, desc: "Desc", *anchor):
        self.desc = desc
        self.want = _expected(desc)
        self.device = _device_of(*anchor)
        if self.device is not None and self.device.type != "cuda":
            raise MoeError(MOE_ERR_INVALID, f"tensors are on {self.device}, expected a GPU")

    def t(self, t, name, key=None):
        dtype, n = self.want[key or name]
        check_tensor(t, name, dtype, n, self.device)
        return _ptr(t)

    def weights(self, w: "Weights", router: bool, experts: bool):
        names = (("w_router", "b_router", "b_select") if router else ()) + \
                (("w1", "b1", "w2", "b2", "w1_shared", "b1_shared", "w2_shared", "b2_shared")
                 if experts else ())
        for n in names:
            self.t(getattr(w, n), "weights." + n, n)
        return ctypes.byref(w.to_c())

    def routing(self, r: "Routing"):
        for f in dataclasses.fields(r):
            self.t(getattr(r, f.name), "routing." + f.name, f.name)
        return ctypes.byref(r.to_c())

    def h(self, t):
        if t is None or isinstance(t, int):
            return _ptr(t)
        plan = moe_query_plan(self.desc)
        check_tensor(t, "h", self.desc.torch_dtype, 0, self.device)
        if t.numel() * t.element_size() < plan["h_bytes"]:
            raise MoeError(MOE_ERR_INVALID, f"h has {t.numel() * t.element_size()} bytes, "
                                            f"needs {plan['h_bytes']}")
        return _ptr(t)

    def ws(self, t):
        """(pointer, bytes) of the workspace; None allocates one of the right size."""
        if t is None:
            t = alloc_workspace(self.desc, self.device)
        if isinstance(t, int):
            raise MoeError(MOE_ERR_INVALID, "pass the workspace as a tensor (its size is needed)")
        check_tensor(t, "workspace", None, 0, self.device)
        self._ws_keep = t
        return _ptr(t), t.numel() * t.element_size()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(status: int):
    if status != MOE_OK:
        lib = load_library()
        raise MoeError(status, lib.moe_last_error().decode() or lib.moe_status_string(status).decode())


def moe_workspace_size(desc: Desc) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_workspace_size(ctypes.byref(desc.to_c()), ctypes.byref(n)))
    return n.value


def moe_query_plan(desc: Desc) -> dict:
    """Resolved kernel path, h storage mode, h buffer bytes and workspace bytes."""
    p = CPlan()
    _check(load_library().moe_query_plan(ctypes.byref(desc.to_c()), ctypes.byref(p)))
    return {"ffn_path": p.ffn_path, "h_mode": p.h_mode, "h_bytes": p.h_bytes,
            "workspace_bytes": p.workspace_bytes}


def alloc_h(desc: Desc, device) -> torch.Tensor:
    """A buffer for the post-GELU activations as moe_ffn_up writes them."""
    plan = moe_query_plan(desc)
    rows = desc.tokens * desc.top_k
    if desc.dtype == "f32":
        return torch.empty(rows, desc.d_ff, dtype=torch.float32, device=device)
    if plan["h_mode"] == MOE_H_SPLIT:
        return torch.empty(2, rows, desc.d_ff, dtype=torch.bfloat16, device=device)
    return torch.empty(rows, desc.d_ff, dtype=torch.bfloat16, device=device)


def alloc_workspace(desc: Desc, device) -> torch.Tensor:
    return torch.empty(moe_workspace_size(desc), dtype=torch.uint8, device=device)


def moe_route(desc, x, weights, routing, aux=None, workspace=None, stream=None):
    a = _Args(desc, x)
    ws, nb = a.ws(workspace)
    _check(load_library().moe_route(ctypes.byref(desc.to_c()), a.t(x, "x"), a.weights(weights, True, False),
                                    a.routing(routing), a.t(aux, "aux"), ws, nb, _stream(stream)))


def moe_permute(desc, x, routing, x_perm, workspace=None, stream=None):
    a = _Args(desc, x)
    ws, nb = a.ws(workspace)
    _check(load_library().moe_permute(ctypes.byref(desc.to_c()), a.t(x, "x"), a.routing(routing),
                                      a.t(x_perm, "x_perm"), ws, nb, _stream(stream)))


def moe_ffn_up(desc, x_perm, offsets, weights, h, workspace=None, stream=None):
    a = _Args(desc, x_perm)
    ws, nb = a.ws(workspace)
    _check(load_library().moe_ffn_up(ctypes.byref(desc.to_c()), a.t(x_perm, "x_perm"),
                                     a.t(offsets, "offsets"), a.weights(weights, False, True), a.h(h),
                                     ws, nb, _stream(stream)))


def moe_ffn_up_gather(desc, x, src, offsets, weights, h, workspace=None, stream=None):
    a = _Args(desc, x)
    ws, nb = a.ws(workspace)
    _check(load_library().moe_ffn_up_gather(ctypes.byref(desc.to_c()), a.t(x, "x"), a.t(src, "src"),
                                            a.t(offsets, "offsets"), a.weights(weights, False, True),
                                            a.h(h), ws, nb, _stream(stream)))


def moe_ffn_down(desc, h, offsets, weights, o, workspace=None, stream=None):
    a = _Args(desc, h)
    ws, nb = a.ws(workspace)
    _check(load_library().moe_ffn_down(ctypes.byref(desc.to_c()), a.h(h), a.t(offsets, "offsets"),
                                       a.weights(weights, False, True), a.t(o, "o"), ws, nb,
                                       _stream(stream)))


def moe_grouped_ffn(desc, x_perm, offsets, weights, h, o, workspace=None, stream=None):
    a = _Args(desc, x_perm)
    ws, nb = a.ws(workspace)
    _check(load_library().moe_grouped_ffn(ctypes.byref(desc.to_c()), a.t(x_perm, "x_perm"),
                                          a.t(offsets, "offsets"), a.weights(weights, False, True),
                                          a.h(h), a.t(o, "o"), ws, nb, _stream(stream)))


def moe_shared_ffn(desc, x, weights, o_shared, workspace=None, stream=None):
    a = _Args(desc, x)
    ws, nb = a.ws(workspace)
    _check(load_library().moe_shared_ffn(ctypes.byref(desc.to_c()), a.t(x, "x"),
                                         a.weights(weights, False, True),
                                         a.t(o_shared, "o_shared"), ws, nb, _stream(stream)))


def moe_combine(desc, o, dest, topk_w, y, o_shared=None, stream=None):
    """Weighted sum of each token's expert rows; desc may have up to 256 experts here (the
    layouts of moe_mx_dispatch), of it only tokens, d_model and top_k enter."""
    a = _Args(desc, o)
    _check(load_library().moe_combine(ctypes.byref(desc.to_c()), a.t(o, "o"), a.t(dest, "dest"),
                                      a.t(topk_w, "topk_w"), a.t(o_shared, "o_shared"), a.t(y, "y"),
                                      _stream(stream)))


def moe_forward(desc, x, weights, y, aux=None, routing=None, workspace=None, stream=None):
    a = _Args(desc, x)
    ws, nb = a.ws(workspace)
    r = a.routing(routing) if routing is not None else None
    _check(load_library().moe_forward(ctypes.byref(desc.to_c()), a.t(x, "x"),
                                      a.weights(weights, True, True), a.t(y, "y"), a.t(aux, "aux"), r,
                                      ws, nb, _stream(stream)))


def moe_forward_noalloc(desc, x, weights, y, aux=None, routing=None, stream=None):
    """moe_forward on the library's own device scratch (no workspace, no allocation)."""
    a = _Args(desc, x)
    r = a.routing(routing) if routing is not None else None
    _check(load_library().moe_forward_noalloc(ctypes.byref(desc.to_c()), a.t(x, "x"),
                                              a.weights(weights, True, True), a.t(y, "y"),
                                              a.t(aux, "aux"), r, _stream(stream)))


def moe_read_probe(buf: torch.Tensor, sink: torch.Tensor, stream=None):
    """One plain streaming read of buf (a measurement aid, not part of the layer)."""
    check_tensor(buf, "buf", None, 0, None)
    check_tensor(sink, "sink", torch.int32, 1, buf.device)
    _check(load_library().moe_read_probe(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                                         _stream(stream)))


def forward(x: torch.Tensor, weights: Weights, desc: Desc, workspace=None, stream=None):
    """The layer's module-style call: returns (y [T, d] fp32, aux fp32 scalar tensor)."""
    y = torch.empty(desc.tokens, desc.d_model, dtype=torch.float32, device=x.device)
    aux = torch.empty((), dtype=torch.float32, device=x.device)
    moe_forward(desc, x, weights, y, aux, None, workspace, stream)
    return y, aux


# ---- scored routing --------------------------------------------------------------------

class _CDescOnce:
    """A descriptor whose C struct is made once and again after a field changes."""

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        self.__dict__.pop("_ref", None)

    def __getstate__(self):              # copies and pickles make their own
        return {k: v for k, v in self.__dict__.items() if k != "_ref"}

    def ref(self):
        """The C struct by reference, as the calls take it."""
        r = self.__dict__.get("_ref")
        if r is None:
            r = self.__dict__["_ref"] = ctypes.byref(self.to_c())
        return r


@dataclasses.dataclass
class ScoreDesc(_CDescOnce):
    """Options of the scored router (moe_score_desc)."""
    tokens: int
    d_model: int
    n_experts: int
    top_k: int
    dtype: str = "bf16"          # "bf16" or "f32"
    score: str = "softmax"       # "softmax" or "sigmoid"
    n_groups: int = 1
    top_groups: int = 1
    group_top: int = 1           # experts a group is valued by: its best, or its best two
    renormalize: bool = True
    scale: float = 1.0

    def to_c(self) -> CScoreDesc:
        return CScoreDesc(self.tokens, self.d_model, self.n_experts, self.top_k,
                          _DTYPES.get(self.dtype, -1), _SCORES.get(self.score, -1), self.n_groups,
                          self.top_groups, self.group_top, int(bool(self.renormalize)), self.scale)

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype == "bf16" else torch.float32


@dataclasses.dataclass
class ScoreRouting:
    """Results of moe_score_route; the backward reads topk_idx, logits and load."""
    topk_idx: Optional[torch.Tensor] = None
    topk_w: Optional[torch.Tensor] = None
    logits: Optional[torch.Tensor] = None
    load: Optional[torch.Tensor] = None
    prob_mean: Optional[torch.Tensor] = None
    aux: Optional[torch.Tensor] = None
    z_loss: Optional[torch.Tensor] = None

    @classmethod
    def allocate(cls, desc: ScoreDesc, device, train: bool = False) -> "ScoreRouting":
        """The indices and weights; with `train` also what the losses and the backward need."""
        T, k, E = desc.tokens, desc.top_k, desc.n_experts
        i32, f32 = dict(dtype=torch.int32, device=device), dict(dtype=torch.float32, device=device)
        r = cls(topk_idx=torch.empty(T, k, **i32), topk_w=torch.empty(T, k, **f32))
        if train:
            r.logits, r.load = torch.empty(T, E, **f32), torch.empty(E, **i32)
            r.prob_mean, r.aux, r.z_loss = (torch.empty(E, **f32), torch.empty((), **f32),
                                            torch.empty((), **f32))
        return r


@dataclasses.dataclass
class ScoreGrads:
    """What moe_score_backward writes; leave out (None) what is not wanted."""
    d_x: Optional[torch.Tensor] = None
    d_w_router: Optional[torch.Tensor] = None
    d_b_router: Optional[torch.Tensor] = None
    d_logits: Optional[torch.Tensor] = None

    @classmethod
    def allocate(cls, desc: ScoreDesc, device) -> "ScoreGrads":
        f32 = dict(dtype=torch.float32, device=device)
        return cls(d_x=torch.empty(desc.tokens, desc.d_model, dtype=desc.torch_dtype, device=device),
                   d_w_router=torch.empty(desc.n_experts, desc.d_model, **f32),
                   d_b_router=torch.empty(desc.n_experts, **f32))


try:                                   # the bare handle and index, without objects around them
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
except AttributeError:
    _current_device = torch.cuda.current_device

    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


class _Call:
    """One call of the operators below: checks its tensors, all on one GPU, and runs it
    there on the given stream, or on the current stream of that GPU."""

    def __init__(self, anchor, name):
        if not isinstance(anchor, torch.Tensor):
            raise MoeError(MOE_ERR_INVALID, f"{name} must be a torch tensor")
        self.anchor = anchor
        if not anchor.is_cuda:
            raise MoeError(MOE_ERR_INVALID, f"{name} is on {anchor.device}, expected a GPU")
        self.index = anchor.get_device()

    @property
    def device(self):
        return self.anchor.device

    def t(self, t, name, dtype, numel):
        """Pointer of a contiguous tensor with at least numel elements, or None."""
        if t is None:
            return None
        if not isinstance(t, torch.Tensor):
            raise MoeError(MOE_ERR_INVALID, f"{name} must be a torch tensor or None")
        if not (t.get_device() == self.index and t.dtype is dtype and t.numel() >= numel and t.is_contiguous()):
            check_tensor(t, name, dtype, numel, self.device)
        return t.data_ptr()

    def ws(self, t, size_of, stream):
        """(pointer, bytes) of the workspace; None allocates one, on the call's stream, so that
        its memory goes to nobody else before the call has run there."""
        if t is None:
            if stream is not None and not isinstance(stream, torch.cuda.Stream):
                handle = getattr(stream, "cuda_stream", stream)
                stream = (torch.cuda.ExternalStream(handle, device=self.device) if handle
                          else torch.cuda.default_stream(self.device))
            with torch.cuda.stream(stream):
                t = self._keep = torch.empty(size_of(), dtype=torch.uint8, device=self.device)
        elif not (isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == self.index and t.is_contiguous()):
            if not isinstance(t, torch.Tensor):
                raise MoeError(MOE_ERR_INVALID, "workspace must be a torch tensor or None")
            check_tensor(t, "workspace", None, 0, self.device)
        return t.data_ptr(), t.nbytes

    def run(self, fn, *args, stream=None):
        if stream is None:
            stream = _raw_stream(self.index)
        elif hasattr(stream, "cuda_stream"):
            stream = stream.cuda_stream
        if _current_device() != self.index:
            with torch.cuda.device(self.index):
                status = fn(*args, stream)
        else:
            status = fn(*args, stream)
        if status != MOE_OK:
            _check(status)


def moe_score_workspace_size(desc: ScoreDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_score_workspace_size(desc.ref(), ctypes.byref(n)))
    return n.value


def alloc_score_workspace(desc: ScoreDesc, device) -> torch.Tensor:
    return torch.empty(moe_score_workspace_size(desc), dtype=torch.uint8, device=device)


def _score_out(c: _Call, d: ScoreDesc, r: ScoreRouting) -> CScoreOut:
    T, k, E = d.tokens, d.top_k, d.n_experts
    i32, f32 = torch.int32, torch.float32
    return CScoreOut(c.t(r.topk_idx, "routing.topk_idx", i32, T * k),
                     c.t(r.topk_w, "routing.topk_w", f32, T * k),
                     c.t(r.logits, "routing.logits", f32, T * E), c.t(r.load, "routing.load", i32, E),
                     c.t(r.prob_mean, "routing.prob_mean", f32, E),
                     c.t(r.aux, "routing.aux", f32, 1), c.t(r.z_loss, "routing.z_loss", f32, 1))


def moe_score_route(desc: ScoreDesc, x, w_router, routing: ScoreRouting, b_router=None, b_select=None,
                    workspace=None, stream=None):
    """Scored routing: writes every field of `routing` that is not None (topk_idx and
    topk_w have to be there)."""
    c = _Call(x, "x")
    T, d, E, dt = desc.tokens, desc.d_model, desc.n_experts, desc.torch_dtype
    ws, nb = c.ws(workspace, lambda: moe_score_workspace_size(desc), stream)
    c.run(load_library().moe_score_route, desc.ref(), c.t(x, "x", dt, T * d),
          c.t(w_router, "w_router", dt, E * d), c.t(b_router, "b_router", torch.float32, E),
          c.t(b_select, "b_select", torch.float32, E), ctypes.byref(_score_out(c, desc, routing)), ws, nb,
          stream=stream)


def moe_score_backward(desc: ScoreDesc, x, w_router, routing: ScoreRouting, d_topk_w, grads: ScoreGrads,
                       d_aux=None, d_z_loss=None, workspace=None, stream=None):
    """Gradients of the scored router into the fields of `grads` that are not None; x may
    be None without d_w_router, w_router without d_x."""
    moe_score_backward_add(desc, x, w_router, routing, d_topk_w, grads, None, d_aux, d_z_loss, workspace, stream)


def moe_score_backward_add(desc: ScoreDesc, x, w_router, routing: ScoreRouting, d_topk_w, grads: ScoreGrads,
                           d_logits_in, d_aux=None, d_z_loss=None, workspace=None, stream=None):
    """The same with d_logits_in (fp32 [T, E] or None), which reaches the logits from elsewhere,
    added to their gradient."""
    c = _Call(routing.logits, "routing.logits")
    T, d, E, k, dt = desc.tokens, desc.d_model, desc.n_experts, desc.top_k, desc.torch_dtype
    f32 = torch.float32
    ws, nb = c.ws(workspace, lambda: moe_score_workspace_size(desc), stream)
    g = CScoreGrads(c.t(grads.d_x, "grads.d_x", dt, T * d), c.t(grads.d_w_router, "grads.d_w_router", f32, E * d),
                    c.t(grads.d_b_router, "grads.d_b_router", f32, E),
                    c.t(grads.d_logits, "grads.d_logits", f32, T * E))
    c.run(load_library().moe_score_backward_add, desc.ref(), c.t(x, "x", dt, T * d),
          c.t(w_router, "w_router", dt, E * d), ctypes.byref(_score_out(c, desc, routing)),
          c.t(d_topk_w, "d_topk_w", f32, T * k), c.t(d_aux, "d_aux", f32, 1),
          c.t(d_z_loss, "d_z_loss", f32, 1), c.t(d_logits_in, "d_logits_in", f32, T * E), ctypes.byref(g), ws, nb,
          stream=stream)


# ---- balance loss by sequence --------------------------------------------------------------

@dataclasses.dataclass
class BalanceDesc(_CDescOnce):
    """Options of the balance loss by sequence (moe_balance_desc)."""
    tokens: int
    n_experts: int
    top_k: int
    n_seqs: int
    score: str = "softmax"       # "softmax" or "sigmoid"

    def to_c(self) -> CBalanceDesc:
        return CBalanceDesc(self.tokens, self.n_experts, self.top_k, self.n_seqs, _SCORES.get(self.score, -1))


@dataclasses.dataclass
class BalanceOut:
    """Results of moe_balance_loss; the backward reads load and valid."""
    load: Optional[torch.Tensor] = None         # [S, E] int32
    valid: Optional[torch.Tensor] = None        # [S + 1] int32: tokens that count, then live sequences
    prob_mean: Optional[torch.Tensor] = None    # [S, E]
    seq_loss: Optional[torch.Tensor] = None     # [S]
    loss: Optional[torch.Tensor] = None         # scalar
    total_load: Optional[torch.Tensor] = None   # [E] int32

    @classmethod
    def allocate(cls, desc: BalanceDesc, device) -> "BalanceOut":
        S, E = desc.n_seqs, desc.n_experts
        i32, f32 = dict(dtype=torch.int32, device=device), dict(dtype=torch.float32, device=device)
        return cls(torch.empty(S, E, **i32), torch.empty(S + 1, **i32), torch.empty(S, E, **f32),
                   torch.empty(S, **f32), torch.empty((), **f32), torch.empty(E, **i32))


def moe_balance_workspace_size(desc: BalanceDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_balance_workspace_size(desc.ref(), ctypes.byref(n)))
    return n.value


def alloc_balance_workspace(desc: BalanceDesc, device) -> torch.Tensor:
    return torch.empty(moe_balance_workspace_size(desc), dtype=torch.uint8, device=device)


def _token_mask(c: _Call, mask, T):
    if isinstance(mask, torch.Tensor) and mask.dtype is torch.bool:
        mask = mask.view(torch.uint8)
    return c.t(mask, "token_mask", torch.uint8, T)


def _balance_out(c: _Call, d: BalanceDesc, r: BalanceOut) -> CBalanceOut:
    S, E, i32, f32 = d.n_seqs, d.n_experts, torch.int32, torch.float32
    return CBalanceOut(c.t(r.load, "out.load", i32, S * E), c.t(r.valid, "out.valid", i32, S + 1),
                       c.t(r.prob_mean, "out.prob_mean", f32, S * E), c.t(r.seq_loss, "out.seq_loss", f32, S),
                       c.t(r.loss, "out.loss", f32, 1), c.t(r.total_load, "out.total_load", i32, E))


def moe_balance_loss(desc: BalanceDesc, logits, topk_idx, seq_offsets, out: BalanceOut, token_mask=None,
                     workspace=None, stream=None):
    """Balance loss and expert counts of every sequence: writes every field of `out` that is not
    None (load and valid have to be there).  token_mask: bool or uint8 [T], 0 = padding."""
    c = _Call(logits, "logits")
    T, E, i32 = desc.tokens, desc.n_experts, torch.int32
    ws, nb = c.ws(workspace, lambda: moe_balance_workspace_size(desc), stream)
    c.run(load_library().moe_balance_loss, desc.ref(), c.t(logits, "logits", torch.float32, T * E),
          c.t(topk_idx, "topk_idx", i32, T * desc.top_k), c.t(seq_offsets, "seq_offsets", i32, desc.n_seqs + 1),
          _token_mask(c, token_mask, T), ctypes.byref(_balance_out(c, desc, out)), ws, nb, stream=stream)


def moe_balance_backward(desc: BalanceDesc, logits, seq_offsets, fwd: BalanceOut, d_logits, d_loss=None,
                         d_seq_loss=None, token_mask=None, stream=None):
    """Gradient of the logits into d_logits (fp32 [T, E], written whole)."""
    c = _Call(logits, "logits")
    T, E, S, f32 = desc.tokens, desc.n_experts, desc.n_seqs, torch.float32
    c.run(load_library().moe_balance_backward, desc.ref(), c.t(logits, "logits", f32, T * E),
          c.t(seq_offsets, "seq_offsets", torch.int32, S + 1), _token_mask(c, token_mask, T),
          ctypes.byref(_balance_out(c, desc, fwd)), c.t(d_loss, "d_loss", f32, 1),
          c.t(d_seq_loss, "d_seq_loss", f32, S), c.t(d_logits, "d_logits", f32, T * E), stream=stream)


# ---- layer norm ------------------------------------------------------------------------------

@dataclasses.dataclass
class NormDesc(_CDescOnce):
    """Options of the layer norm (moe_norm_desc)."""
    rows: int
    d: int
    dtype: str = "bf16"          # x, x_out, y and their gradients: "bf16" or "f32"
    param_dtype: str = "f32"     # weight and bias
    add_dtype: str = "f32"       # add
    eps: float = 1e-5

    def to_c(self) -> CNormDesc:
        return CNormDesc(self.rows, self.d, _DTYPES.get(self.dtype, -1), _DTYPES.get(self.param_dtype, -1),
                         _DTYPES.get(self.add_dtype, -1), self.eps)


def _torch_dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def moe_norm_workspace_size(desc: NormDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_norm_workspace_size(desc.ref(), ctypes.byref(n)))
    return n.value


def alloc_norm_workspace(desc: NormDesc, device) -> torch.Tensor:
    return torch.empty(moe_norm_workspace_size(desc), dtype=torch.uint8, device=device)


def _norm_rows(c: _Call, t, name, dtype, d: NormDesc):
    """A [rows, d] tensor with contiguous rows (any row stride), by reference, or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise MoeError(MOE_ERR_INVALID, f"{name} must be a torch tensor or None")
    if not (t.get_device() == c.index and t.dtype is dtype):
        check_tensor(t, name, dtype, 0, c.device)
    shape, strides = t.shape, t.stride()
    if len(shape) == 2 and shape[0] == d.rows and shape[1] == d.d and (strides[1] == 1 or d.d == 1):
        return ctypes.byref(CRows(t.data_ptr(), strides[0]))
    if t.dim() < 1 or t.shape[-1] != d.d or t.numel() != d.rows * d.d:
        raise MoeError(MOE_ERR_INVALID, f"{name} has shape {tuple(t.shape)}, expected [{d.rows}, {d.d}]")
    if not t.is_contiguous():
        raise MoeError(MOE_ERR_INVALID, f"{name} must be contiguous, or a matrix with contiguous rows")
    return ctypes.byref(CRows(t.data_ptr(), d.d))


def moe_layer_norm(desc: NormDesc, x, y, weight=None, bias=None, add=None, x_out=None, mean=None, rstd=None,
                   stream=None):
    """x_out = x + add and its layer norm y; tensors are [rows, d] with any row stride."""
    c = _Call(x, "x")
    dt, pt, at, f32 = _torch_dtype(desc.dtype), _torch_dtype(desc.param_dtype), _torch_dtype(desc.add_dtype), torch.float32
    c.run(load_library().moe_layer_norm, desc.ref(), _norm_rows(c, x, "x", dt, desc),
          _norm_rows(c, add, "add", at, desc), c.t(weight, "weight", pt, desc.d), c.t(bias, "bias", pt, desc.d),
          _norm_rows(c, x_out, "x_out", dt, desc), _norm_rows(c, y, "y", dt, desc),
          c.t(mean, "mean", f32, desc.rows), c.t(rstd, "rstd", f32, desc.rows), stream=stream)


def moe_layer_norm_backward(desc: NormDesc, dy, x, mean, rstd, weight=None, d_x_out=None, d_x=None, d_weight=None,
                            d_bias=None, workspace=None, stream=None):
    """Gradients into those of d_x, d_weight and d_bias that are not None; x is what was
    normalised (x_out, where there was an add), d_x_out the residual path's gradient."""
    c = _Call(x, "x")
    dt, f32 = _torch_dtype(desc.dtype), torch.float32
    ws, nb = (None, 0) if d_weight is None and d_bias is None else \
        c.ws(workspace, lambda: moe_norm_workspace_size(desc), stream)
    c.run(load_library().moe_layer_norm_backward, desc.ref(), _norm_rows(c, dy, "dy", dt, desc),
          _norm_rows(c, x, "x", dt, desc), c.t(weight, "weight", _torch_dtype(desc.param_dtype), desc.d),
          c.t(mean, "mean", f32, desc.rows), c.t(rstd, "rstd", f32, desc.rows),
          _norm_rows(c, d_x_out, "d_x_out", dt, desc), _norm_rows(c, d_x, "d_x", dt, desc),
          c.t(d_weight, "d_weight", f32, desc.d), c.t(d_bias, "d_bias", f32, desc.d), ws, nb, stream=stream)


# ---- a shared projection with low-rank adapters ----------------------------------------------

@dataclasses.dataclass
class LoraDesc(_CDescOnce):
    """Options of a projection with low-rank adapters (moe_lora_desc)."""
    tokens: int
    d_in: int
    d_out: int
    rank: int
    n_adapters: int
    act: str = "none"            # "none" or "gelu"
    out_dtype: str = "bf16"      # "bf16" or "f32"
    has_bias: bool = False

    def to_c(self) -> CLoraDesc:
        return CLoraDesc(self.tokens, self.d_in, self.d_out, self.rank, self.n_adapters,
                         _LORA_ACTS.get(self.act, -1), _DTYPES.get(self.out_dtype, -1), int(bool(self.has_bias)))


@dataclasses.dataclass
class LoraWeights:
    """The shared matrix w [d_out, d_in] and the adapters a [N, rank, d_in], b [N, d_out, rank]
    (bf16), their scales [N] (fp32, or None: 1) and the bias [d_out] (bf16)."""
    w: torch.Tensor
    a: torch.Tensor
    b: torch.Tensor
    scale: Optional[torch.Tensor] = None
    bias: Optional[torch.Tensor] = None


def moe_lora_workspace_size(desc: LoraDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_lora_workspace_size(desc.ref(), ctypes.byref(n)))
    return n.value


def alloc_lora_workspace(desc: LoraDesc, device) -> torch.Tensor:
    return torch.empty(moe_lora_workspace_size(desc), dtype=torch.uint8, device=device)


def _lora_weights(c: _Call, d: LoraDesc, w: LoraWeights) -> CLoraWeights:
    N, r, bf = d.n_adapters, d.rank, torch.bfloat16
    return CLoraWeights(c.t(w.w, "weights.w", bf, d.d_out * d.d_in), c.t(w.a, "weights.a", bf, N * r * d.d_in),
                        c.t(w.b, "weights.b", bf, N * d.d_out * r), c.t(w.scale, "weights.scale", torch.float32, N),
                        c.t(w.bias, "weights.bias", bf, d.d_out))


def moe_lora_linear(desc: LoraDesc, x, adapter, weights: LoraWeights, y, workspace=None, stream=None):
    """y = act(W x + bias + scale B A x) with each token's own A, B and scale (adapter: int32 [T],
    -1 for none)."""
    c = _Call(x, "x")
    T = desc.tokens
    ws, nb = c.ws(workspace, lambda: moe_lora_workspace_size(desc), stream)
    c.run(load_library().moe_lora_linear, desc.ref(), c.t(x, "x", torch.bfloat16, T * desc.d_in),
          c.t(adapter, "adapter", torch.int32, T), ctypes.byref(_lora_weights(c, desc, weights)),
          c.t(y, "y", _torch_dtype(desc.out_dtype), T * desc.d_out), ws, nb, stream=stream)


def moe_lora_shared_workspace_size(up: LoraDesc, down: LoraDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_lora_shared_workspace_size(up.ref(), down.ref(), ctypes.byref(n)))
    return n.value


def alloc_lora_shared_workspace(up: LoraDesc, down: LoraDesc, device) -> torch.Tensor:
    return torch.empty(moe_lora_shared_workspace_size(up, down), dtype=torch.uint8, device=device)


def moe_lora_shared_ffn(up: LoraDesc, down: LoraDesc, x, adapter, w_up: LoraWeights, w_down: LoraWeights, o_shared,
                        workspace=None, stream=None):
    """The shared expert with adapters on both products; o_shared fp32, as moe_combine takes it."""
    c = _Call(x, "x")
    T = up.tokens
    ws, nb = c.ws(workspace, lambda: moe_lora_shared_workspace_size(up, down), stream)
    c.run(load_library().moe_lora_shared_ffn, up.ref(), down.ref(), c.t(x, "x", torch.bfloat16, T * up.d_in),
          c.t(adapter, "adapter", torch.int32, T), ctypes.byref(_lora_weights(c, up, w_up)),
          ctypes.byref(_lora_weights(c, down, w_down)), c.t(o_shared, "o_shared", torch.float32, T * down.d_out), ws, nb,
          stream=stream)


# ---- experts in microscaled 4-bit floating point ------------------------------------------

@dataclasses.dataclass
class MxDesc(_CDescOnce):
    """Options of a layer with MXFP4 expert weights (moe_mx_desc)."""
    tokens: int
    d_model: int
    d_ff: int
    n_experts: int
    top_k: int
    act: str = "bf16"             # activations: "bf16", or "mxfp4" (quantised by the call)
    has_expert_bias: bool = True

    def to_c(self) -> CMxDesc:
        return CMxDesc(self.tokens, self.d_model, self.d_ff, self.n_experts, self.top_k,
                       _MX_ACTS.get(self.act, -1), int(bool(self.has_expert_bias)))


@dataclasses.dataclass
class MxWeights:
    """Codes [E, N, K/2] and scales [E, N, K/32] (uint8) of the expert matrices, biases bf16;
    a call needs only those of the products it runs."""
    w1: Optional[torch.Tensor] = None
    s1: Optional[torch.Tensor] = None
    b1: Optional[torch.Tensor] = None
    w2: Optional[torch.Tensor] = None
    s2: Optional[torch.Tensor] = None
    b2: Optional[torch.Tensor] = None

    @classmethod
    def quantize(cls, w1, w2, b1=None, b2=None) -> "MxWeights":
        """From bf16 or fp32 expert matrices w1 [E, F, d] and w2 [E, d, F]."""
        out = cls(b1=b1, b2=b2)
        for n, w in (("1", w1), ("2", w2)):
            codes, scales = alloc_mx(w.shape[0] * w.shape[1], w.shape[2], w.device)
            moe_mx_quantize(w.reshape(-1, w.shape[2]), codes, scales)
            setattr(out, "w" + n, codes.view(*w.shape[:2], -1))
            setattr(out, "s" + n, scales.view(*w.shape[:2], -1))
        return out


def alloc_mx(rows: int, cols: int, device):
    """(codes, scales) buffers of rows x cols values."""
    return (torch.empty(rows, cols // 2, dtype=torch.uint8, device=device),
            torch.empty(rows, cols // 32, dtype=torch.uint8, device=device))


def _mx_rows(t, name):
    """(pointer, dtype id, rows, cols, row stride) of a 2-D tensor whose rows are contiguous."""
    dt = MOE_DTYPE_BF16 if t.dtype is torch.bfloat16 else MOE_DTYPE_F32 if t.dtype is torch.float32 else -1
    shape, strides = t.shape, t.stride()
    if dt < 0 or len(shape) != 2 or (shape[1] > 1 and strides[1] != 1):
        raise MoeError(MOE_ERR_INVALID, f"{name} must be a bf16 or fp32 matrix with contiguous rows")
    rows, cols = shape
    return t.data_ptr(), dt, rows, cols, strides[0] if rows > 1 else -(-cols // 8) * 8


def moe_mx_quantize(x, codes, scales, stream=None):
    """Rows of x (bf16 or fp32 [rows, cols], any row stride) to MXFP4 codes and scales."""
    c = _Call(x, "x")
    p, dt, rows, cols, stride = _mx_rows(x, "x")
    c.run(load_library().moe_mx_quantize, p, dt, rows, cols, stride,
          c.t(codes, "codes", torch.uint8, rows * cols // 2),
          c.t(scales, "scales", torch.uint8, rows * cols // 32), stream=stream)


def moe_mx_dequantize(codes, scales, out, stream=None):
    """MXFP4 codes and scales to the rows of out (bf16 or fp32 [rows, cols])."""
    c = _Call(out, "out")
    p, dt, rows, cols, stride = _mx_rows(out, "out")
    c.run(load_library().moe_mx_dequantize, c.t(codes, "codes", torch.uint8, rows * cols // 2),
          c.t(scales, "scales", torch.uint8, rows * cols // 32), rows, cols, dt, p, stride, stream=stream)


def moe_mx_workspace_size(desc: MxDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_mx_workspace_size(desc.ref(), ctypes.byref(n)))
    return n.value


def alloc_mx_workspace(desc: MxDesc, device, route: Optional[ScoreDesc] = None) -> torch.Tensor:
    """The workspace of the calls below; with `route`, of moe_mx_forward."""
    n = moe_mx_workspace_size(desc) + (moe_score_workspace_size(route) if route is not None else 0)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _mx_weights(c: _Call, d: MxDesc, w: MxWeights, up: bool, down: bool) -> CMxWeights:
    E, D, F, u8, bf = d.n_experts, d.d_model, d.d_ff, torch.uint8, torch.bfloat16
    n = E * D * F
    return CMxWeights(c.t(w.w1, "weights.w1", u8, n // 2) if up else None,
                      c.t(w.s1, "weights.s1", u8, n // 32) if up else None,
                      c.t(w.b1, "weights.b1", bf, E * F) if up else None,
                      c.t(w.w2, "weights.w2", u8, n // 2) if down else None,
                      c.t(w.s2, "weights.s2", u8, n // 32) if down else None,
                      c.t(w.b2, "weights.b2", bf, E * D) if down else None)


def moe_mx_dispatch(desc: MxDesc, routing: Routing, workspace=None, stream=None):
    """counts, offsets, dest and src of `routing` from its topk_idx, for up to 256 experts."""
    c = _Call(routing.topk_idx, "routing.topk_idx")
    A, E, i32 = desc.tokens * desc.top_k, desc.n_experts, torch.int32
    r = CRouting(topk_idx=c.t(routing.topk_idx, "routing.topk_idx", i32, A),
                 counts=c.t(routing.counts, "routing.counts", i32, E),
                 offsets=c.t(routing.offsets, "routing.offsets", i32, E + 1),
                 dest=c.t(routing.dest, "routing.dest", i32, A), src=c.t(routing.src, "routing.src", i32, A))
    ws, nb = c.ws(workspace, lambda: moe_mx_workspace_size(desc), stream)
    c.run(load_library().moe_mx_dispatch, desc.ref(), ctypes.byref(r), ws, nb, stream=stream)


def moe_mx_ffn_up(desc: MxDesc, x, offsets, weights: MxWeights, h, src=None, workspace=None, stream=None):
    """First expert product with GELU; with src, x holds the tokens and row r reads token
    src[r] / top_k, else x holds the dispatched rows."""
    c = _Call(x, "x")
    R, bf = desc.tokens * desc.top_k, torch.bfloat16
    ws, nb = c.ws(workspace, lambda: moe_mx_workspace_size(desc), stream)
    c.run(load_library().moe_mx_ffn_up, desc.ref(),
          c.t(x, "x", bf, (desc.tokens if src is not None else R) * desc.d_model), c.t(src, "src", torch.int32, R),
          c.t(offsets, "offsets", torch.int32, desc.n_experts + 1),
          ctypes.byref(_mx_weights(c, desc, weights, True, False)), c.t(h, "h", bf, R * desc.d_ff), ws, nb,
          stream=stream)


def moe_mx_ffn_down(desc: MxDesc, h, offsets, weights: MxWeights, o, workspace=None, stream=None):
    """Second expert product, o fp32."""
    c = _Call(h, "h")
    R = desc.tokens * desc.top_k
    ws, nb = c.ws(workspace, lambda: moe_mx_workspace_size(desc), stream)
    c.run(load_library().moe_mx_ffn_down, desc.ref(), c.t(h, "h", torch.bfloat16, R * desc.d_ff),
          c.t(offsets, "offsets", torch.int32, desc.n_experts + 1),
          ctypes.byref(_mx_weights(c, desc, weights, False, True)),
          c.t(o, "o", torch.float32, R * desc.d_model), ws, nb, stream=stream)


def moe_mx_forward(route: ScoreDesc, desc: MxDesc, x, w_router, weights: MxWeights, y, routing=None,
                   b_router=None, b_select=None, workspace=None, stream=None):
    """The whole layer: scored routing, dispatch, both MXFP4 products, combine.  y fp32
    [T, d]; `routing` (a ScoreRouting, or None) receives the fields it has."""
    c = _Call(x, "x")
    T, D, E, bf, f32 = desc.tokens, desc.d_model, desc.n_experts, torch.bfloat16, torch.float32
    ws, nb = c.ws(workspace, lambda: moe_mx_workspace_size(desc) + moe_score_workspace_size(route), stream)
    out = ctypes.byref(_score_out(c, route, routing)) if routing is not None else None
    c.run(load_library().moe_mx_forward, route.ref(), desc.ref(),
          c.t(x, "x", bf, T * D), c.t(w_router, "w_router", bf, E * D), c.t(b_router, "b_router", f32, E),
          c.t(b_select, "b_select", f32, E), ctypes.byref(_mx_weights(c, desc, weights, True, True)),
          c.t(y, "y", f32, T * D), out, ws, nb, stream=stream)


@dataclasses.dataclass
class MxBlock:
    """One pre-norm sublayer (moe_mx_block): norm, router, MXFP4 experts, and the shared expert
    with its requests' adapters (up, down, w_up, w_down, adapter) or none."""
    norm: NormDesc
    route: ScoreDesc
    experts: MxDesc
    w_router: torch.Tensor
    weights: MxWeights
    weight: Optional[torch.Tensor] = None
    bias: Optional[torch.Tensor] = None
    b_router: Optional[torch.Tensor] = None
    b_select: Optional[torch.Tensor] = None
    up: Optional[LoraDesc] = None
    down: Optional[LoraDesc] = None
    w_up: Optional[LoraWeights] = None
    w_down: Optional[LoraWeights] = None


def _mx_block(block: MxBlock, c: Optional[_Call], adapter):
    """The C struct and what it points to; without a call only the descriptors."""
    def at(s):
        return None if s is None else ctypes.cast(ctypes.pointer(s), ctypes.c_void_p)

    b, f32, bf = block, torch.float32, torch.bfloat16
    up, down = (None if d is None else d.to_c() for d in (b.up, b.down))
    keep = [b.norm.to_c(), b.route.to_c(), b.experts.to_c(), up, down]
    s = CMxBlock(norm=at(keep[0]), route=at(keep[1]), experts=at(keep[2]), up=at(up), down=at(down))
    if c is not None:
        d, E, pt = b.norm.d, b.route.n_experts, _torch_dtype(b.norm.param_dtype)
        s.weight, s.bias = c.t(b.weight, "weight", pt, d), c.t(b.bias, "bias", pt, d)
        s.w_router = c.t(b.w_router, "w_router", bf, E * d)
        s.b_router, s.b_select = c.t(b.b_router, "b_router", f32, E), c.t(b.b_select, "b_select", f32, E)
        keep.append(_mx_weights(c, b.experts, b.weights, True, True))
        s.w = at(keep[-1])
        if b.up is not None and b.down is not None:
            if b.w_up is None or b.w_down is None:
                raise MoeError(MOE_ERR_INVALID, "w_up and w_down must not be None")
            keep += [_lora_weights(c, b.up, b.w_up), _lora_weights(c, b.down, b.w_down)]
            s.w_up, s.w_down = at(keep[-2]), at(keep[-1])
            s.adapter = c.t(adapter, "adapter", torch.int32, b.up.tokens)
    return s, keep


def moe_mx_block_workspace_size(block: MxBlock) -> int:
    n = ctypes.c_size_t(0)
    s, _keep = _mx_block(block, None, None)
    _check(load_library().moe_mx_block_workspace_size(ctypes.byref(s), ctypes.byref(n)))
    return n.value


def alloc_mx_block_workspace(block: MxBlock, device) -> torch.Tensor:
    return torch.empty(moe_mx_block_workspace_size(block), dtype=torch.uint8, device=device)


def moe_mx_block_forward(block: MxBlock, x, y, add=None, x_out=None, adapter=None, routing=None, workspace=None,
                         stream=None):
    """x_out = x + add, its norm, and y = the experts' and the shared expert's output on it (fp32
    [T, d], the next block's add)."""
    c = _Call(x, "x")
    n = block.norm
    ws, nb = c.ws(workspace, lambda: moe_mx_block_workspace_size(block), stream)
    s, _keep = _mx_block(block, c, adapter)
    out = ctypes.byref(_score_out(c, block.route, routing)) if routing is not None else None
    dt = _torch_dtype(n.dtype)
    c.run(load_library().moe_mx_block_forward, ctypes.byref(s), _norm_rows(c, x, "x", dt, n),
          _norm_rows(c, add, "add", _torch_dtype(n.add_dtype), n), _norm_rows(c, x_out, "x_out", dt, n),
          c.t(y, "y", torch.float32, n.rows * n.d), out, ws, nb, stream=stream)
