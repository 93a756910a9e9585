"""fp64 oracle of the token log probabilities and of the distillation loss.

Definitions of ``include/muon.h``, row by row, in numpy fp64.
"""

from __future__ import annotations

import numpy as np


def log_softmax(z: np.ndarray) -> np.ndarray:
    """Of one row; NaN throughout for a NaN, a +inf or only -inf."""
    m = np.max(z)
    if not np.isfinite(m):
        return np.full(z.shape, np.nan)
    with np.errstate(divide="ignore"):
        return (z - m) - np.log(np.sum(np.exp(z - m)))


def token_logprobs(logits, tokens, top: int, tau: float = 1.0):
    """(logprob, entropy, top_logprob, top_index) of fp64 logits [rows, vocab]."""
    rows, vocab = logits.shape
    lp, ent = np.zeros(rows), np.zeros(rows)
    tlp, tix = np.zeros((rows, top)), np.zeros((rows, top), np.int64)
    for r in range(rows):
        z = logits[r]
        with np.errstate(invalid="ignore"):
            l = log_softmax(z / tau)
            q = np.exp(l)
            ent[r] = -np.sum(np.where(q > 0, q * l, 0.0)) if not np.isnan(l).any() else np.nan
        t = int(tokens[r]) if tokens is not None else -1
        lp[r] = 0.0 if t < 0 else l[t] if t < vocab else np.nan
        key = np.where(np.isnan(z), np.inf, z)               # NaN first, then +inf
        order = np.lexsort((np.arange(vocab), -key, ~np.isnan(z)))[:top]
        tix[r], tlp[r] = order, l[order]
    return lp, ent, tlp, tix


def distill(logits, top_index, top_logit, tau: float = 1.0, g=None):
    """(loss [rows], gradient [rows, vocab]) in fp64."""
    rows, vocab = logits.shape
    loss, grad = np.zeros(rows), np.zeros((rows, vocab))
    for r in range(rows):
        gr = 1.0 if g is None else float(g[r])
        here = top_index[r] >= 0
        idx, t = top_index[r][here], top_logit[r][here].astype(np.float64) / tau
        if np.any(idx >= vocab) or np.any(np.isnan(t)) or np.any(t == np.inf):
            loss[r] = np.nan
            grad[r] = 0.0 if gr == 0.0 else np.nan
            continue
        if idx.size == 0 or np.all(t == -np.inf):
            continue
        logp = log_softmax(t)
        p = np.exp(logp)
        with np.errstate(invalid="ignore"):
            logq = log_softmax(logits[r] / tau)
        if np.isnan(logq).any():
            loss[r] = np.nan
            grad[r] = 0.0 if gr == 0.0 else np.nan
            continue
        with np.errstate(invalid="ignore"):
            terms = np.where(p > 0, p * (logp - logq[idx]), 0.0)
        loss[r] = tau * tau * np.sum(terms)
        d = np.exp(logq)
        np.add.at(d, idx, -p)
        grad[r] = gr * tau * d
    return loss, grad
