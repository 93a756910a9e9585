"""The 4-bit and distillation operators together, as a training step uses
them, and their behaviour on streams and in captured graphs."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from oracle import distill as od, mx4 as om

pytestmark = pytest.mark.gpu

T, H, V, K = 48, 96, 700, 12


def _f64(t):
    return t.detach().cpu().double().numpy()


def _student(seed):
    g = torch.Generator().manual_seed(seed)
    w1 = (torch.randn(H, H, generator=g) * 0.1).cuda()
    head = (torch.randn(V, H, generator=g) * 0.1).cuda()
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    return w1, head, x


def _step(x, w1, head, idx, val, g):
    """Gradients of one distillation step of a 4-bit two-matrix student."""
    (w1q, w1t), (hq, ht) = mo.mx4_quantize([w1, head], images="both")
    h, x_t = mo.mx4_linear(x, w1q, save=True)
    z, h_t = mo.mx4_linear(h, hq, out_dtype=torch.float32, save=True)
    loss, dz = mo.distill_loss(z, idx, val, grad_loss=g)
    dh, dhead = mo.mx4_linear_backward(dz, h_t, ht)
    _, dw1 = mo.mx4_linear_backward(dh, x_t, w1t)
    return loss, dw1, dhead


def test_step_against_the_formulas():
    """Each stage's output against the fp64 formula on the stage's own inputs
    (a stage's rounding to bf16 or 4 bits is then the next one's input)."""
    w1, head, x = _student(1)
    tl = (torch.randn(T, V, generator=torch.Generator().manual_seed(2)) * 2).cuda()
    teach = mo.token_logprobs(tl, top=K)
    (w1q, w1t), (hq, ht) = mo.mx4_quantize([w1, head], images="both")
    h, x_t = mo.mx4_linear(x, w1q, save=True)
    z, h_t = mo.mx4_linear(h, hq, out_dtype=torch.float32, save=True)
    g = torch.full((T,), 1.0 / T, device="cuda")
    loss, dz = mo.distill_loss(z, teach.top_index, teach.top_logprob, grad_loss=g)
    dh, dhead = mo.mx4_linear_backward(dz, h_t, ht)
    dx, dw1 = mo.mx4_linear_backward(dh, x_t, w1t)

    def near(got, a, b):
        want, size = a @ b.T, np.abs(a) @ np.abs(b).T
        half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
        assert np.all(np.abs(_f64(got) - want) <= (a.shape[1] + 1) * 2.0 ** -23 * size + half * 1.02 * np.abs(want))

    q = om.rounded
    near(h, q(_f64(x)), q(_f64(w1)))
    near(z, q(_f64(h)), q(_f64(head)))
    near(dh, q(_f64(dz)), q(_f64(head).T))
    near(dhead, q(_f64(dz).T), q(_f64(h).T))
    near(dx, q(_f64(dh)), q(_f64(w1).T))
    near(dw1, q(_f64(dh).T), q(_f64(x).T))
    wl, wg = od.distill(_f64(z), _f64(teach.top_index).astype(np.int64), _f64(teach.top_logprob), 1.0, _f64(g))
    assert np.max(np.abs(_f64(loss) - wl)) <= 2.0 ** -24 * 400        # about 40 roundings of logs below 10
    assert np.max(np.abs(_f64(dz) - wg)) <= 2.0 ** -24 * 100 / T
    # the step takes the gradients as they are
    opt = mo.MuonAdamW([w1], [head], lr=1e-3)
    w1.grad, head.grad = dw1, dhead
    before = (w1.clone(), head.clone())
    opt.step()
    assert not torch.equal(before[0], w1) and not torch.equal(before[1], head)
    assert bool(torch.isfinite(w1).all()) and bool(torch.isfinite(head).all())


def test_two_captured_steps_replay_independently():
    """Two graphs of the whole step, replayed in turn with fresh inputs, eager
    calls between them: every replay equals the eager step bit for bit."""
    gen = torch.Generator().manual_seed(3)
    graphs = []
    for i in range(2):
        w1, head, x = _student(10 + i)
        idx = torch.randint(0, V, (T, K), generator=gen).cuda()
        val = torch.randn(T, K, generator=gen).cuda()
        g = torch.full((T,), 1.0 / T, device="cuda")
        state = (x, w1, head, idx, val, g)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            _step(*state)
            mo.token_logprobs(head, top=5)
        torch.cuda.current_stream().wait_stream(s)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = _step(*state)
            lp = mo.token_logprobs(head, top=5)
        graphs.append((gr, state, out, lp))
    for rep in range(3):
        for gr, state, out, lp in graphs:
            x, w1, head, idx, val, g = state
            x.copy_(torch.randn(T, H, generator=gen))
            w1.mul_(1.25)
            idx.copy_(torch.randint(0, V, (T, K), generator=gen))
            gr.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out] + [t.clone() for t in lp if t is not None]
            want = list(_step(*state)) + [t for t in mo.token_logprobs(head, top=5) if t is not None]
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b), rep


def test_other_streams_and_long_rows():
    """Calls on their own streams at the same time give what they give alone
    (long rows of few sequences: the ones with a workspace)."""
    gen = torch.Generator().manual_seed(4)
    zs = [torch.randn(2, 150001, generator=gen).cuda() for _ in range(3)]
    idx = torch.randint(0, 150001, (2, 8), generator=gen).cuda()
    val = torch.randn(2, 8, generator=gen).cuda()
    w = mo.mx4_quantize(torch.randn(300, 500, generator=gen).cuda())
    x = torch.randn(3, 500, generator=gen).cuda()
    alone = [(mo.token_logprobs(z, top=9), mo.distill_loss(z, idx, val), mo.mx4_linear(x, w)) for z in zs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in zs]
    for _ in range(3):
        got = [(mo.token_logprobs(z, top=9, stream=s), mo.distill_loss(z, idx, val, stream=s),
                mo.mx4_linear(x, w, stream=s)) for z, s in zip(zs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            for u, v in zip([*a[0][1:], *a[1], a[2]], [*b[0][1:], *b[1], b[2]]):
                assert torch.equal(u, v)


@pytest.mark.parametrize("images", ["rows", "cols", "both"])
def test_optimizer_keeps_images_of_its_matrices(images):
    """The images behind a step are those of the weights it wrote, in the
    tensors that held the ones before."""
    gen = torch.Generator().manual_seed(5)
    shapes = [(96, 200), (200, 96), (64, 64)]
    ps = [(torch.randn(s, generator=gen) * 0.02).cuda() for s in shapes]
    plain = [p.clone() for p in ps]
    opt = mo.MuonAdamW(ps, lr=1e-2, mx4=images)
    other = mo.MuonAdamW(plain, lr=1e-2)
    first = opt.refresh_mx4()
    for step in range(3):
        for p, q in zip(ps, plain):
            p.grad = torch.randn(p.shape, generator=gen).cuda()
            q.grad = p.grad.clone()
        opt.step()
        other.step()
        want = mo.mx4_quantize(ps, images=images)
        for p, q, a, b, f in zip(ps, plain, opt.mx4, want, first):
            assert torch.equal(p, q)                 # the step itself is as it was
            for x, y, z in zip(*[t if images == "both" else (t,) for t in (a, b, f)]):
                assert x is z
                assert torch.equal(x.codes, y.codes) and torch.equal(x.scales, y.scales)
    with pytest.raises(RuntimeError, match="without mx4"):
        other.refresh_mx4()


def test_two_threads_on_one_stream():
    """Calls with a workspace from two threads of one stream, over and over:
    each gives what it gives alone."""
    import threading
    gen = torch.Generator().manual_seed(6)
    zs = [torch.randn(2, 90001, generator=gen).cuda() for _ in range(2)]
    idx = torch.randint(0, 90001, (2, 8), generator=gen).cuda()
    val = torch.randn(2, 8, generator=gen).cuda()
    alone = [(mo.token_logprobs(z, top=9), mo.distill_loss(z, idx, val)) for z in zs]
    got = [[], []]

    def work(i):
        for _ in range(20):
            got[i].append((mo.token_logprobs(zs[i], top=9), mo.distill_loss(zs[i], idx, val)))

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 20
        for a, b in got[i]:
            assert torch.equal(a.top_logprob, alone[i][0].top_logprob) and torch.equal(a.entropy, alone[i][0].entropy)
            assert torch.equal(b[0], alone[i][1][0]) and torch.equal(b[1], alone[i][1][1])


def test_small_and_large_temperatures():
    """Temperatures that make the softmax one-hot or flat."""
    z = torch.randn(3, 5000, generator=torch.Generator().manual_seed(7)).cuda()
    idx = torch.tensor([[1, 2], [3, 4], [5, 6]]).cuda()
    val = torch.tensor([[1.0, 0.5]] * 3).cuda()
    r = mo.token_logprobs(z, top=3, temperature=1e-30)
    best = z.argmax(1)
    assert torch.equal(r.top_index[:, 0], best)
    assert bool((r.entropy == 0).all()) and bool((r.top_logprob[:, 0] == 0).all())
    loss, g = mo.distill_loss(z, best[:, None].contiguous(), val[:, :1].contiguous(), temperature=1e-30)
    assert bool((loss == 0).all()) and bool((g == 0).all())
    r = mo.token_logprobs(z, top=3, temperature=1e18)
    flat = float(np.log(5000.0))
    assert bool(((r.entropy - flat).abs() <= 2.0 ** -24 * 60 * flat).all())
    loss, g = mo.distill_loss(z, idx, val, temperature=1e6)
    want = od.distill(_f64(z), _f64(idx).astype(np.int64), _f64(val), 1e6)[1]
    # g = tau (q - p): q and p are off by about 60 roundings
    assert np.max(np.abs(_f64(g) - want)) <= 1e6 * 60 * 2.0 ** -24
