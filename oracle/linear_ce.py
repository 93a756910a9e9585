"""fp64 oracle of the linear cross entropy and of the balance loss.

Definitions of ``include/muon.h`` in torch fp64 (on any device); the operands
of the cross entropy are the bf16 values that its products take.
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch


class CrossEntropy(NamedTuple):
    loss: torch.Tensor
    dx: torch.Tensor
    dw: torch.Tensor
    logits: torch.Tensor
    dz: torch.Tensor


def cross_entropy(x, w, targets, g: Optional[torch.Tensor] = None) -> CrossEntropy:
    """Of [rows, hidden] and [vocab, hidden], each taken as bf16."""
    x, w = x.bfloat16().double(), w.bfloat16().double()
    live = targets >= 0
    g = torch.ones_like(targets, dtype=torch.float64) if g is None else g.double()
    takes = live & (g != 0)
    z = torch.where(live[:, None], x, torch.zeros_like(x)) @ w.t()
    logp = torch.log_softmax(z, dim=1)
    y = targets.clamp(min=0)
    loss = torch.where(live, -logp.gather(1, y[:, None])[:, 0], torch.zeros_like(g))
    dz = logp.exp()
    dz[torch.arange(len(y), device=y.device), y] -= 1.0
    dz = torch.where(takes[:, None], dz * g[:, None], torch.zeros_like(dz))
    return CrossEntropy(loss, dz @ w, dz.t() @ torch.where(takes[:, None], x, torch.zeros_like(x)), z, dz)


def balance(logits, index, weight: float = 1.0, g: float = 1.0):
    """(loss, counts, gradient) of [tokens, experts] and [tokens, top]."""
    z = logits.double()
    e = z.shape[1]
    live = (index >= 0).any(1)
    counts = torch.bincount(index[index >= 0], minlength=e)
    f = counts.double() * e / max(1, int(counts.sum()))
    n = max(1, int(live.sum()))
    p = torch.where(live[:, None], torch.softmax(z, dim=1), torch.zeros_like(z))
    return weight * (f * p.sum(0)).sum() / n, counts, weight * g / n * (p * (f - (p * f).sum(1, keepdim=True)))
