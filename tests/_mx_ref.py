"""MXFP4 and the expert products in 64 bits on the CPU, from their definition."""
from __future__ import annotations

import numpy as np
import torch

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x: torch.Tensor):
    """(codes [rows, cols/2], scales [rows, cols/32]) of rows of bf16 or fp32 values."""
    v = x.double().numpy()
    rows, cols = v.shape
    b = v.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(2)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(2)
    _, e = np.frexp(amax)                                   # amax in [2^(e-1), 2^e)
    s = np.where(amax > 0, np.maximum(e - 3, -127), -127)
    q = np.abs(b) / np.exp2(s.astype(np.float64))[..., None]
    d = np.abs(q[..., None] - LEVELS)                       # nearest, ties to the even code
    near = d == d.min(-1, keepdims=True)
    code = np.where(near[..., 0::2].any(-1), near[..., 0::2].argmax(-1) * 2, near[..., 1::2].argmax(-1) * 2 + 1)
    # a tie has one even and one odd neighbour; past 6 the nearest is 6 (code 7)
    code = code | (np.signbit(b).astype(np.int64) << 3)
    code[bad] = 0
    code = code.reshape(rows, cols)
    packed = (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)
    scale = np.where(bad, 255, s + 127).astype(np.uint8)
    return torch.from_numpy(packed), torch.from_numpy(scale)


def values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """fp64 values [..., K] of packed codes [..., K/2] and scales [..., K/32]."""
    c, s = codes.numpy(), scales.numpy().astype(np.float64)
    q = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)
    v = np.where(q & 8, -1.0, 1.0) * LEVELS[q & 7]
    f = np.where(s == 255, np.nan, np.exp2(s - 127))
    return torch.from_numpy(v * np.repeat(f, 32, -1))


def dispatch(idx: torch.Tensor, E: int):
    """(counts, offsets, dest, src) of assignments idx [T, k]; src has the kept rows only."""
    flat = idx.flatten().tolist()
    by = [[a for a, e in enumerate(flat) if e == x] for x in range(E)]
    counts = [len(b) for b in by]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    src = [a for b in by for a in b]
    dest = np.full(len(flat), -1)
    dest[src] = np.arange(len(src))
    return counts, offsets, dest.reshape(idx.shape), src


def product(a, offsets, w, bias):
    """(out, size): a [R, K] fp64 rows against w [E, N, K], and the sum of |terms|."""
    R, E, N = a.shape[0], w.shape[0], w.shape[1]
    out, size = torch.zeros(R, N, dtype=torch.float64), torch.zeros(R, N, dtype=torch.float64)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        out[lo:hi] = a[lo:hi] @ w[e].T
        size[lo:hi] = a[lo:hi].abs() @ w[e].abs().T
        if bias is not None:
            out[lo:hi] += bias[e].double()
            size[lo:hi] += bias[e].double().abs()
    return out, size


def gelu(z):
    return 0.5 * z * (1 + torch.erf(z * 2 ** -0.5))
