"""The balance loss by sequence and its gradient in 64 bits, from their definition."""
from __future__ import annotations

import torch


def shares(l, kind):
    s = torch.sigmoid(l) if kind == "sigmoid" else torch.softmax(l, 1)
    return s / s.sum(1, keepdim=True)


def forward(l, kind, idx, off, mask, k):
    T, E = l.shape
    S = len(off) - 1
    load, valid = torch.zeros(S, E, dtype=torch.long), torch.zeros(S + 1, dtype=torch.long)
    means, losses = [], []
    for b in range(S):
        rows = torch.arange(off[b], off[b + 1])
        rows = rows[mask[rows]] if mask is not None else rows
        n = valid[b] = len(rows)
        chosen = idx[rows].flatten()
        load[b] = torch.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E)
        means.append(shares(l[rows], kind).mean(0) if n else torch.zeros(E, dtype=l.dtype))
        losses.append(E * torch.dot(load[b].to(l.dtype) / (k * n), means[-1]) if n else torch.zeros((), dtype=l.dtype))
    valid[S] = (valid[:S] > 0).sum()
    seq = torch.stack(losses)
    return {"load": load, "valid": valid, "prob_mean": torch.stack(means), "seq_loss": seq,
            "loss": seq.sum() / max(1, int(valid[S])), "total_load": load.sum(0)}


def gradient(l, kind, idx, off, mask, k, d_loss, d_seq):
    l = l.clone().requires_grad_(True)
    r = forward(l, kind, idx, off, mask, k)
    loss = d_loss * r["loss"] + (torch.dot(d_seq, r["seq_loss"]) if d_seq is not None else 0.0)
    return torch.autograd.grad(loss, l)[0] if loss.requires_grad else torch.zeros_like(l)
