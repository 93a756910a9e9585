"""The 8-bit layers, the balance loss and the LM head's cross entropy together,
as a training step of a mixture of experts uses them, and their behaviour on
streams, in threads and in captured graphs."""

from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from oracle import fp8 as of, linear_ce as oc

pytestmark = pytest.mark.gpu

T, H, F, E, K, V = 150, 96, 64, 6, 2, 500


def _model(seed):
    g = torch.Generator().manual_seed(seed)
    router = (torch.randn(E, H, generator=g) * 0.3).cuda()
    up = [(torch.randn(F, H, generator=g) * 0.1).cuda() for _ in range(E)]
    down = [(torch.randn(H, F, generator=g) * 0.1).cuda() for _ in range(E)]
    head = (torch.randn(V, H, generator=g) * 0.1).cuda()
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    y = torch.randint(-20, V, (T,), generator=g).cuda()
    return router, up, down, head, x, y


def _f64(t):
    return t.detach().cpu().double().numpy()


def _near(got, a, b, loose=0.0):
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    assert np.all(np.abs(_f64(got) - want) <= ((a.shape[1] + 1) * 2.0 ** -23 + loose) * size + half * 1.02 * np.abs(want) + 1e-40)


def test_step_against_the_formulas():
    """Each stage's output against the fp64 formula on the stage's own inputs
    (a stage's rounding to 8 or 16 bits is then the next one's input); the
    optimizer takes the gradients and keeps the images."""
    router, up, down, head, x, y = _model(1)
    opt = mo.MuonAdamW(up + down, [head], lr=1e-3, fp8="both")
    images = opt.refresh_fp8()
    z = (x.float() @ router.t()).contiguous()
    choice = torch.topk(z, K, dim=1)[1].contiguous()
    choice[:7] = -1                                               # padding
    bal = mo.balance_loss(z, choice, weight=0.01)
    wl, wc, wg = oc.balance(z, choice, 0.01)
    assert torch.equal(bal.counts, wc) and abs(float(bal.loss) - float(wl)) <= 2.0 ** -18 * float(wl)
    assert float((bal.grad.double() - wg).abs().max()) <= 2.0 ** -18 * float(wg.abs().max())

    h = x.float().clone()
    saved = []
    for e in range(E):
        (wu, wu_t), (wd, wd_t) = images[e], images[E + e]
        rows = (choice == e).any(1).nonzero()[:, 0]
        assert len(rows) == int(bal.counts[e])                    # nobody chose an expert twice here
        xe = x[rows]
        u, x_t = mo.fp8_linear(xe, wu, save=True)
        d, u_t = mo.fp8_linear(u, wd, out_dtype=torch.float32, save=True)
        _near(u, of.rounded(_f64(xe)), of.rounded(_f64(up[e]), True), 2.0 ** -11)
        _near(d, of.rounded(_f64(u)), of.rounded(_f64(down[e]), True))
        h.index_add_(0, rows, d)
        saved.append((rows, x_t, u_t, wu_t, wd_t, xe, u))
    n = int((y >= 0).sum())
    hb = h.to(torch.bfloat16)
    g = torch.full((T,), 1.0 / n, device="cuda")
    loss, dh, dhead = mo.linear_cross_entropy(hb, head, y, grad_loss=g)
    o = oc.cross_entropy(hb, head, y, g)
    assert float((loss.double() - o.loss).abs().max()) <= 2.0 ** -17      # logits near 10 of sums of 96 terms near 1
    for got, want in ((dh, o.dx), (dhead, o.dw)):
        # elements are sums of terms of many sizes: 2^-7 of the largest covers dz's and the result's rounding
        assert float((got.double() - want).abs().max()) <= 2.0 ** -7 * float(want.abs().max())
    for e, (rows, x_t, u_t, wu_t, wd_t, xe, u) in enumerate(saved):
        dd = dh[rows]
        du, dwd = mo.fp8_linear_backward(dd, u_t, wd_t)
        _, dwu = mo.fp8_linear_backward(du, x_t, wu_t)
        _near(du, of.rounded(_f64(dd)), of.rounded(_f64(down[e]).T.copy(), True), 2.0 ** -11)
        _near(dwd, of.rounded(_f64(dd).T.copy()), of.rounded(_f64(u).T.copy()))
        _near(dwu, of.rounded(_f64(du).T.copy()), of.rounded(_f64(xe).T.copy()))
        up[e].grad, down[e].grad = dwu, dwd
    head.grad = dhead
    opt.step()
    for w, (q, q_t) in zip(up + down, opt.fp8):
        assert np.array_equal(_f64(mo.fp8_dequantize(q, dtype=torch.float32)), of.rounded(_f64(w), True))
        assert np.array_equal(_f64(mo.fp8_dequantize(q_t, dtype=torch.float32)), of.rounded(_f64(w).T.copy(), True))


def _ops(x, w, head, z, idx, y, big):
    """One pass through every operator; outputs only."""
    q, q_t = mo.fp8_quantize(w, images="both", square=True)
    out, x_t = mo.fp8_linear(x, q, save=True)
    dx, dw = mo.fp8_linear_backward(out, x_t, q_t)
    b = mo.balance_loss(z, idx, weight=0.5)
    loss, dh, dhead = mo.linear_cross_entropy(out, head, y)
    l2, _, _ = mo.linear_cross_entropy(out, big, y, grad=False)
    return [out, dx, dw, b.loss, b.counts, b.grad, loss, dh, dhead, l2]


def _inputs(seed, t):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return [r(t, 200).to(torch.bfloat16), r(130, 200) * 0.1, r(300, 130) * 0.1, r(t, 40),
            torch.randint(-1, 40, (t, 3), generator=g, device="cuda"), torch.randint(-20, 300, (t,), generator=g, device="cuda"),
            (r(2000, 130) * 0.1).to(torch.bfloat16)]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_captured_graphs_replay_independently():
    """Two graphs of every operator, replayed in turn with fresh inputs, eager
    calls of other sizes and synchronizations between: each replay gives what
    the eager call gives."""
    sets = [_inputs(1, 90), _inputs(2, 700)]
    for s in sets:
        _ops(*s)                                                   # loads kernels, sizes the cached workspaces
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            graphs.append((gr, s, _ops(*s)))
        graphs[-1] = (gr, s, graphs[-1][2])
    for turn in range(4):
        for k, (gr, s, outs) in enumerate(graphs):
            fresh = _inputs(10 * turn + k, s[0].shape[0])
            for a, b in zip(s, fresh):
                a.copy_(b)
            want = [t.clone() for t in _ops(*s)]
            gr.replay()
            other = _ops(*_inputs(77, 333))                        # behind the replay, on the same workspaces as before
            torch.cuda.synchronize()
            assert _same(outs, want)
            del other


def test_other_streams_and_threads():
    """Calls on a stream of their own, their inputs and outputs of another; two
    threads on one stream and two on two: the same bits as alone."""
    sets = [_inputs(3, 80), _inputs(4, 260)]
    want = [[t.clone() for t in _ops(*s)] for s in sets]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    x, w, head, z, idx, y, big = sets[1]
    q = mo.fp8_quantize(w, square=True)
    side.wait_stream(torch.cuda.current_stream())
    got = [mo.fp8_linear(x, q, stream=side), mo.balance_loss(z, idx, weight=0.5, stream=side).grad,
           mo.linear_cross_entropy(want[1][0], head, y, stream=side)[2]]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[1][0]) and torch.equal(got[1], want[1][5]) and torch.equal(got[2], want[1][8])

    def work(k, stream, res):
        with torch.cuda.stream(stream):
            for _ in range(6):
                res[k] = _ops(*sets[k])
            stream.synchronize()

    for streams in ((side, side), (torch.cuda.Stream(), torch.cuda.Stream())):
        res = [None, None]
        ts = [threading.Thread(target=work, args=(k, streams[k], res)) for k in range(2)]
        for t in ts:
            t.start()
        for t in ts:
            t.join()
        torch.cuda.synchronize()
        assert _same(res[0], want[0]) and _same(res[1], want[1])


def test_timing_counters_see_the_operators():
    names = ["fp8_quant", "fp8_dequant", "fp8_matmul", "linear_ce", "balance"]
    s = _inputs(5, 50)
    mo.profile_reset()
    mo.profile_enable(names)
    try:
        _ops(*s)
        mo.fp8_dequantize(mo.fp8_quantize(s[1]))
        counts = {n: mo.profile_read(n) for n in names}
    finally:
        mo.profile_enable(())
        mo.profile_reset()
    assert counts["fp8_quant"][0] == 4 and counts["fp8_matmul"][0] == 3 and counts["linear_ce"][0] == 2 and counts["balance"][0] == 1
    assert all(c[1] > 0 and c[2] > 0 for c in counts.values())
