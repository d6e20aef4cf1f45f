"""The scored router and its gradients in 64 bits on the CPU, from their definition."""
from __future__ import annotations

import numpy as np
import torch


def scores(l, kind):
    if kind == "sigmoid":
        return torch.sigmoid(l)
    return torch.softmax(l, 1)


def select(s, b_select, E, k, G, top_groups, group_top):
    """Indices in rank order, by counting: a candidate's rank is the number of better ones
    (a NaN is worse than every number; equal values rank by index)."""
    v = s.numpy() + (b_select.numpy() if b_select is not None else 0.0)
    T = v.shape[0]
    out = np.empty((T, k), np.int64)

    def better(x):                       # matrix [i, j]: j ranks before i
        x = np.where(np.isnan(x), -np.inf, x), np.isnan(x)
        a, b = x[0][:, None], x[0][None, :]
        na, nb = x[1][:, None], x[1][None, :]
        i, j = np.arange(len(x[0]))[:, None], np.arange(len(x[0]))[None, :]
        higher = (b > a) | (na & ~nb)
        equal = (b == a) & (na == nb)
        return higher & ~(nb & ~na) | (equal & (j < i))

    for t in range(T):
        cand = np.arange(E)
        if G > 1:
            g = np.where(np.isnan(v[t]), -np.inf, v[t]).reshape(G, E // G)
            with np.errstate(invalid="ignore"):
                val = np.sort(g, 1)[:, ::-1][:, :group_top].sum(1)
            keep = better(val).sum(1) < top_groups
            cand = cand[np.repeat(keep, E // G)]
        order = np.argsort(better(v[t][cand]).sum(1), kind="stable")
        out[t] = cand[order[:k]]
    return torch.from_numpy(out)


def weights(s, idx, renorm, scale):
    r = torch.take_along_dim(s, idx, 1)
    return scale * (r / (r.sum(1, keepdim=True) + 1e-20) if renorm else r)


def forward(l, kind, b_select, k, G=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    """Everything from the [T, E] logits (fp64)."""
    T, E = l.shape
    s = scores(l, kind)
    idx = select(s, b_select, E, k, G, top_groups, group_top)
    load = torch.bincount(idx.flatten(), minlength=E)
    q = s / s.sum(1, keepdim=True)
    mean = q.mean(0)
    return {"idx": idx, "w": weights(s, idx, renorm, scale), "load": load, "prob_mean": mean,
            "aux": E * (load.double() / (T * k) * mean).sum(), "z": (torch.logsumexp(l, 1) ** 2).mean(), "s": s}


def loss(l, kind, idx, load, k, renorm, scale, d_w, d_aux, d_z):
    """The scalar whose gradient the backward gives; idx < 0 or >= E is a dropped slot."""
    T, E = l.shape
    s = scores(l, kind)
    ok = (idx >= 0) & (idx < E)
    r = torch.take_along_dim(s, idx.clamp(0, E - 1), 1) * ok
    w = scale * (r / (r.sum(1, keepdim=True) + 1e-20) if renorm else r)
    q = s / s.sum(1, keepdim=True)
    out = (w * d_w).sum()
    if d_aux is not None:
        out = out + d_aux * E * (load.double() / (T * k) * q.mean(0)).sum()
    if d_z is not None:
        out = out + d_z * (torch.logsumexp(l, 1) ** 2).mean()
    return out


def d_logits(l, *args):
    l = l.clone().requires_grad_(True)
    return torch.autograd.grad(loss(l, *args), l)[0]


def d_logits_size(l, kind, idx, load, k, renorm, scale, d_w, d_aux, d_z):
    """The same sum with every term's absolute value: what the rounding errors scale with."""
    T, E = l.shape
    s = scores(l, kind)
    ok = (idx >= 0) & (idx < E)
    r = torch.take_along_dim(s, idx.clamp(0, E - 1), 1) * ok
    g = (d_w * ok).abs()
    S = r.sum(1, keepdim=True) + 1e-20
    dr = scale * ((g + (g * r).sum(1, keepdim=True) / S) / S if renorm else g)
    ds = torch.zeros_like(l).scatter_add_(1, idx.clamp(0, E - 1), dr * ok)
    tot = s.sum(1, keepdim=True)
    if d_aux is not None:
        dq = abs(d_aux) * E * load.double() / (T * k) / T
        ds = ds + (dq + (dq * s).sum(1, keepdim=True) / tot) / tot
    out = ds * s if kind == "sigmoid" else s * (ds + (ds * s).sum(1, keepdim=True))
    if d_z is not None:
        out = out + abs(d_z) * 2 / T * torch.logsumexp(l, 1, keepdim=True).abs() * torch.softmax(l, 1)
    return out


def numeric(l, t, e, *args, h=1e-4):
    a, b = l.clone(), l.clone()
    a[t, e] += h
    b[t, e] -= h
    return float((loss(a, *args) - loss(b, *args)) / (2 * h))
