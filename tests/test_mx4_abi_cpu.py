"""Host-side refusals of the MX4, log-probability and distillation entry
points: every bad argument is rejected before anything is enqueued, so these
run on a machine without a GPU (the addresses are never used)."""

from __future__ import annotations

import ctypes

import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from matrix_orthogonalizing_optimizer_amd import _lib as L

BASE = 0x10000000


def _item(**kw):
    it = L.MoMx4Item(BASE, BASE + 0x100000, BASE + 0x200000, BASE + 0x300000, BASE + 0x400000, 64, 96, 96)
    for k, v in kw.items():
        setattr(it, k, v)
    return it


def _quantize(*items, count=None, dtype=L.MO_BF16):
    arr = (L.MoMx4Item * max(1, len(items)))(*items)
    return L.lib().mo_mx4_quantize(arr if items else None, len(items) if count is None else count, dtype, None)


@pytest.mark.parametrize("kw,word", [
    (dict(rows=0), "rows and cols"), (dict(cols=0), "rows and cols"), (dict(rows=1 << 31), "rows and cols"),
    (dict(rows=1 << 21, cols=1 << 21, ld=1 << 21), "2^40"), (dict(ld=95), "ld"), (dict(ld=1 << 40), "ld"),
    (dict(src=None), "src"), (dict(src=BASE + 1), "aligned"), (dict(codes=None), "image"),
    (dict(scales_t=None), "image"), (dict(codes=None, scales=None, codes_t=None, scales_t=None), "image"),
    (dict(codes=BASE + 0x100008), "aligned"), (dict(scales=BASE + 0x200002), "aligned"),
    (dict(codes=BASE), "overlaps"), (dict(codes_t=BASE + 0x100010), "overlaps"),
    (dict(scales=BASE + 0x100400), "overlaps"),
])
def test_quantize_refuses(kw, word):
    assert _quantize(_item(**kw)) == L.MO_EINVAL
    assert word in L.last_error()


def test_quantize_refuses_the_list():
    assert _quantize(count=1) == L.MO_EINVAL and "NULL" in L.last_error()
    assert _quantize(_item(), count=-1) == L.MO_EINVAL
    assert _quantize(_item(), dtype=2) == L.MO_EINVAL
    # the second matrix writes where the first reads
    assert _quantize(_item(), _item(codes=BASE + 0x500000, scales=BASE + 0x600000, codes_t=BASE + 64)) == L.MO_EINVAL
    assert "overlaps" in L.last_error()
    assert _quantize(count=0) == L.MO_OK


def test_image_size():
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    for (r, k), want in {(1, 1): (16, 4), (3, 33): (96, 12), (7, 128): (448, 28), (2, 129): (160, 16)}.items():
        assert L.lib().mo_mx4_image_size(r, k, ctypes.byref(c), ctypes.byref(s)) == L.MO_OK
        assert (c.value, s.value) == want
    assert L.lib().mo_mx4_image_size(0, 4, ctypes.byref(c), ctypes.byref(s)) == L.MO_EINVAL
    assert L.lib().mo_mx4_image_size(4, 4, None, ctypes.byref(s)) == L.MO_EINVAL


def _image(rows=64, cols=96, at=BASE, **kw):
    x = L.MoMx4Image(at, at + 0x100000, rows, cols)
    for k, v in kw.items():
        setattr(x, k, v)
    return x


def _matmul(a, b, out=BASE + 0x800000, dt=L.MO_F32, ldo=64):
    return L.lib().mo_mx4_matmul(ctypes.byref(a) if a else None, ctypes.byref(b) if b else None, out, dt, ldo, 0, None)


def test_matmul_refuses():
    b = _image(at=BASE + 0x200000)
    for args, word in [
        ((None, b), "NULL"), ((_image(cols=95), b), "columns"), ((_image(codes=None), b), "non-NULL"),
        ((_image(codes=BASE + 4), b), "aligned"), ((_image(scales=BASE + 0x100001), b), "aligned"),
        ((_image(rows=0), b), "rows and cols"),
    ]:
        assert _matmul(*args) == L.MO_EINVAL
        assert word in L.last_error()
    a = _image()
    assert _matmul(a, b, out=None) == L.MO_EINVAL
    assert _matmul(a, b, out=BASE + 0x800002) == L.MO_EINVAL
    assert _matmul(a, b, ldo=63) == L.MO_EINVAL and "ldo" in L.last_error()
    assert _matmul(a, b, dt=7) == L.MO_EINVAL
    assert _matmul(a, b, out=BASE + 0x100000) == L.MO_EINVAL and "overlaps" in L.last_error()


def test_dequantize_refuses():
    dst = (ctypes.c_void_p * 1)(BASE + 0x800000)
    img = (L.MoMx4Image * 1)(_image())
    f = L.lib().mo_mx4_dequantize
    assert f(img, dst, 1, 5, None) == L.MO_EINVAL
    assert f(img, None, 1, L.MO_F32, None) == L.MO_EINVAL
    assert f(img, (ctypes.c_void_p * 1)(BASE + 0x800004), 1, L.MO_F32, None) == L.MO_EINVAL
    assert f(img, (ctypes.c_void_p * 1)(BASE + 16), 1, L.MO_F32, None) == L.MO_EINVAL
    assert f((L.MoMx4Image * 1)(_image(scales=None)), dst, 1, L.MO_F32, None) == L.MO_EINVAL


def _ws(rows, vocab, top, which):
    n = ctypes.c_size_t()
    assert getattr(L.lib(), which)(rows, vocab, top, ctypes.byref(n)) == L.MO_OK
    return n.value


_LP = dict(logits=BASE, dtype=L.MO_BF16, rows=8, vocab=100, ld=100, tokens=BASE + 0x10000, tau=1.0,
           logprob=BASE + 0x20000, entropy=BASE + 0x30000, top=4, top_index=BASE + 0x40000,
           top_logprob=BASE + 0x50000, ws=0x70000000, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=3), "dtype"), (dict(rows=-1), "rows"), (dict(rows=1 << 22), "rows"), (dict(vocab=0), "vocab"),
    (dict(vocab=1 << 31), "vocab"), (dict(ld=99), "stride"), (dict(logits=None), "logits"),
    (dict(logits=BASE + 1), "aligned"), (dict(tau=0.0), "temperature"), (dict(tau=-1.0), "temperature"),
    (dict(tau=float("nan")), "temperature"), (dict(tau=float("inf")), "temperature"), (dict(tau=1e-39), "temperature"), (dict(tau=1e20), "temperature"),
    (dict(tokens=None), "both"), (dict(logprob=None), "both"), (dict(top=-1), "top"), (dict(top=129), "top"),
    (dict(top=101, vocab=100), "exceeds"), (dict(top=0), "iff"), (dict(top_index=None), "iff"),
    (dict(top_index=BASE + 0x40004), "aligned"), (dict(entropy=BASE + 0x20004), "overlap"),
    (dict(logprob=BASE + 16), "overlap"), (dict(entropy=BASE + 0x30002), "aligned"),
])
def test_logprobs_refuses(kw, word):
    assert L.lib().mo_token_logprobs(*{**_LP, **kw}.values()) == L.MO_EINVAL
    assert word in L.last_error()


_DL = dict(logits=BASE, dtype=L.MO_F32, rows=8, vocab=100, ld=100, top_index=BASE + 0x10000, top_logit=BASE + 0x20000,
           top=4, tau=1.0, grad_loss=BASE + 0x30000, loss=BASE + 0x40000, grad=BASE + 0x50000, ld_grad=100,
           ws=0x70000000, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=-1), "dtype"), (dict(rows=-1), "rows"), (dict(vocab=0), "vocab"), (dict(ld=99), "stride"),
    (dict(ld_grad=99), "stride"), (dict(logits=None), "logits"), (dict(top=0), "top"), (dict(top=129), "top"),
    (dict(tau=0.0), "temperature"), (dict(loss=None, grad=None), "both NULL"), (dict(top_index=None), "non-NULL"),
    (dict(top_logit=None), "non-NULL"), (dict(top_index=BASE + 0x10004), "aligned"), (dict(grad=BASE), "overlap"),
    (dict(grad=BASE + 0x50002), "aligned"), (dict(loss=BASE + 0x30010), "overlap"),
    (dict(grad=BASE + 0x10000 - 64), "overlap"),
])
def test_distill_refuses(kw, word):
    assert L.lib().mo_distill_loss(*{**_DL, **kw}.values()) == L.MO_EINVAL
    assert word in L.last_error()


def test_no_rows_is_no_work():
    assert L.lib().mo_token_logprobs(*{**_LP, "rows": 0}.values()) == L.MO_OK
    assert L.lib().mo_distill_loss(*{**_DL, "rows": 0}.values()) == L.MO_OK


def test_workspace_must_hold_what_the_query_says():
    for rows, vocab in [(1, 32000), (1, 1 << 20), (2, 150001), (4096, 32000)]:
        need = _ws(rows, vocab, 8, "mo_token_logprobs_workspace_size")
        if need:
            a = {**_LP, "rows": rows, "vocab": vocab, "ld": vocab, "top": 8, "logits": BASE << 4, "ws_bytes": need - 1}
            assert L.lib().mo_token_logprobs(*a.values()) == L.MO_EWORKSPACE
            assert L.lib().mo_token_logprobs(*{**a, "ws": None}.values()) == L.MO_EWORKSPACE
        need = _ws(rows, vocab, 8, "mo_distill_loss_workspace_size")
        if need:
            a = {**_DL, "rows": rows, "vocab": vocab, "ld": vocab, "ld_grad": vocab, "top": 8, "logits": BASE << 4,
                 "grad": BASE << 5, "ws_bytes": need - 1}
            assert L.lib().mo_distill_loss(*a.values()) == L.MO_EWORKSPACE
    n = ctypes.c_size_t()
    for f in (L.lib().mo_token_logprobs_workspace_size, L.lib().mo_distill_loss_workspace_size):
        assert f(1, 0, 1, ctypes.byref(n)) == L.MO_EINVAL
        assert f(1, 10, 129, ctypes.byref(n)) == L.MO_EINVAL
        assert f(1, 10, 1, None) == L.MO_EINVAL


# ------------------------------------------------------------- the Python front
def test_front_refuses_cpu_tensors_and_shapes():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU"):
        mo.mx4_quantize(x)
    with pytest.raises(ValueError, match="GPU"):
        mo.token_logprobs(x)
    with pytest.raises(ValueError, match="GPU"):
        mo.distill_loss(x, torch.zeros(4, 1, dtype=torch.int64), torch.zeros(4, 1))
    with pytest.raises(ValueError, match="2-D"):
        mo.mx4_quantize(torch.zeros(4))
    with pytest.raises(TypeError):
        mo.mx4_quantize(x.double())
    with pytest.raises(TypeError):
        mo.mx4_quantize([x, x.bfloat16()])
    with pytest.raises(ValueError, match="strides"):
        mo.mx4_quantize(x.t())
    with pytest.raises(ValueError, match="strides"):
        mo.token_logprobs(torch.zeros(1, 64).expand(4, 64))
    with pytest.raises(ValueError, match="images"):
        mo.mx4_quantize(x, images="all")
    with pytest.raises(ValueError, match="at least one row"):
        mo.Mx4Matrix.empty(0, 32, "cpu")
    assert mo.mx4_quantize([]) == [] and mo.mx4_dequantize([]) == []


def test_front_checks_images():
    codes, scales = torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(3, 4, dtype=torch.uint8)
    q = mo.Mx4Matrix(codes, scales, 40)
    assert q.shape == (3, 40)
    for bad in [(codes, scales, 65), (codes, scales, 32), (codes.int(), scales, 40), (codes, scales[:2], 40),
                (codes[:, :16], scales, 32), (codes, scales, 0)]:
        with pytest.raises(ValueError):
            mo.Mx4Matrix(*bad)
    with pytest.raises(TypeError):
        mo.mx4_matmul(codes, q)
    with pytest.raises(ValueError, match="accumulate"):
        mo.mx4_matmul(q, q, accumulate=True)
    with pytest.raises(ValueError, match="features"):
        mo.mx4_linear(torch.zeros(2, 41), q)
    with pytest.raises(ValueError, match="want"):
        mo.mx4_linear_backward(torch.zeros(2, 41), q, q)


@pytest.mark.parametrize("kw", [dict(top_index=torch.zeros(4, 1)), dict(top_index=torch.zeros(4, dtype=torch.int64)),
                                dict(top_logit=torch.zeros(4, 2)), dict(grad_loss=torch.zeros(3)),
                                dict(out_grad=torch.zeros(4, 63)), dict(out_grad=torch.zeros(4, 64), grad=False)])
def test_front_checks_distill_arguments(kw):
    a = dict(top_index=torch.zeros(4, 1, dtype=torch.int64), top_logit=torch.zeros(4, 1))
    a.update(kw)
    with pytest.raises(ValueError):
        mo.distill_loss(torch.zeros(4, 64), a.pop("top_index"), a.pop("top_logit"), **a)


def test_front_checks_tokens():
    with pytest.raises(ValueError, match="tokens"):
        mo.token_logprobs(torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="tokens"):
        mo.token_logprobs(torch.zeros(4, 64), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(mo.MuonError, match="top"):
        mo.token_logprobs(torch.zeros(4, 64), top=200)


def test_optimizer_refuses_unknown_images():
    with pytest.raises(ValueError, match="mx4"):
        mo.MuonAdamW([torch.zeros(4, 4)], mx4="all")
    with pytest.raises(RuntimeError, match="without mx4"):
        mo.MuonAdamW([torch.zeros(4, 4)]).refresh_mx4()


def test_product_refuses_too_many_tiles_and_too_long_rows():
    a, b = _image(rows=1 << 18, cols=32), _image(rows=1 << 18, cols=32, at=BASE << 8)
    assert _matmul(a, b, out=BASE << 12, ldo=1 << 18) == L.MO_EINVAL and "tiles" in L.last_error()
    a, b = _image(rows=2, cols=(1 << 25) + 1), _image(rows=2, cols=(1 << 25) + 1, at=BASE << 8)
    a.scales, b.scales = BASE << 4, BASE << 9
    assert _matmul(a, b, out=BASE << 12, ldo=2) == L.MO_EINVAL and "2^25" in L.last_error()


def test_images_of_empty_matrices_are_refused():
    import torch
    import matrix_orthogonalizing_optimizer_amd as mo
    with pytest.raises(ValueError, match="at least one row"):
        mo.MuonAdamW([torch.empty(0, 8)], mx4="rows")
    mo.MuonAdamW([torch.empty(0, 8)])
