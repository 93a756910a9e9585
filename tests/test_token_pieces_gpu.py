"""Long rows of many sequences (cut into the large pieces) against the oracle,
and long rows in captured graphs, whose workspaces are their own.  Tolerances
are those of test_distill_gpu."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from oracle import distill as od
from test_distill_gpu import DTYPES, _check_distill, _check_logprobs, _logits, _teacher

pytestmark = pytest.mark.gpu

# 16 MiB of logits and more, in rows that neither operator holds whole
LONG = {torch.float32: (47, 100003), torch.bfloat16: (47, 190001)}


@pytest.mark.parametrize("dtype", DTYPES)
def test_logprobs_of_many_long_rows(dtype, monkeypatch):
    rows, vocab = LONG[dtype]
    z = _logits(rows, vocab, dtype, 31, pad=5, off=1)
    z[0, :50000] = -math.inf                  # whole pieces without a token
    z[1] = -math.inf
    z[2, vocab - 1] = math.nan
    z[3, 70000] = math.inf
    z[4, 60000:] = 9.0                        # a plateau over several pieces
    z[5] = torch.finfo(dtype).min
    z[5, 99999] = 1.0
    z[6] = -math.inf
    z[6, vocab - 3] = 0.5                     # one token left
    tok = torch.randint(0, vocab, (rows,), generator=torch.Generator().manual_seed(1))
    tok[7], tok[8] = -1, vocab
    tok[6] = vocab - 3
    _check_logprobs(z, tok.cuda(), 50, 1.0)
    # The lowest value over 0.5 is -6.8e38, beyond the largest fp32 3.4e38: the
    # nearest fp32 is -inf, so the oracle's values are held to that range.
    exact = od.token_logprobs

    def held(*a):
        lp, ent, tlp, tix = exact(*a)
        with np.errstate(over="ignore"):
            return lp, ent, np.where(np.isinf(tlp.astype(np.float32)), tlp.astype(np.float32), tlp), tix

    monkeypatch.setattr(od, "token_logprobs", held)
    _check_logprobs(z, None, 3, 0.5)


@pytest.mark.parametrize("dtype", DTYPES)
def test_distill_of_many_long_rows(dtype):
    rows, vocab = LONG[dtype]
    z = _logits(rows, vocab, dtype, 32, pad=3)
    idx, val = _teacher(rows, vocab, 17, 33)
    idx[0, 0], idx[0, 1] = 0, vocab - 1
    idx[1] = -1                               # skipped
    idx[2, 3:9] = -1
    idx[3, 4] = idx[3, 11]                    # a column named twice
    z[4, :50000] = -math.inf                  # whole pieces without a token, and a teacher elsewhere
    idx[4] = 50000 + torch.arange(17) * 2000
    z[5, 77] = math.nan
    z[6, int(idx[6, 0])] = -math.inf
    idx[7, 2] = vocab
    g = torch.rand(rows, generator=torch.Generator().manual_seed(2)) - 0.5
    g[8] = 0.0
    loss, _ = _check_distill(z, idx, val, 2.0, g)
    alone = mo.distill_loss(z, idx.cuda(), val.cuda(), temperature=2.0, grad=False)[0]
    assert torch.equal(torch.nan_to_num(alone), torch.nan_to_num(loss))


def test_long_rows_in_two_graphs():
    """Two graphs over long rows, replayed in turn, with eager calls of the
    same and of a larger size between them: every replay equals the eager
    result bit for bit."""
    gen = torch.Generator().manual_seed(34)

    def fresh(rows, vocab):
        idx = torch.randint(0, vocab, (rows, 8), generator=gen)
        return torch.randn(rows, vocab, generator=gen) * 3, idx, torch.randn(rows, 8, generator=gen)

    def step(z, idx, val):
        t = mo.token_logprobs(z, idx[:, 0].contiguous(), top=9, temperature=0.7)
        return [*t, *mo.distill_loss(z, idx, val, temperature=2.0)]

    graphs = []
    for rows in (2, 3):
        state = [t.cuda() for t in fresh(rows, 90001)]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step(*state)
        torch.cuda.current_stream().wait_stream(s)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step(*state)
        graphs.append((gr, state, out))
    large = [t.cuda() for t in fresh(5, 200001)]
    larger = [t.clone() for t in step(*large)]
    for rep in range(4):
        for gr, state, out in graphs:
            for t, new in zip(state, fresh(*state[0].shape)):
                t.copy_(new)
            gr.replay()
            again = step(*large)              # eager work behind the replay, on the stream's own workspace
            got = [t.clone() for t in out]
            want = step(*state)
            torch.cuda.synchronize()
            for a, b in zip(got + list(again), want + larger):
                assert torch.equal(a, b), rep
