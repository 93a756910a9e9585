"""Host-side refusals of the 8-bit, cross-entropy and balance entry points:
every bad argument is rejected before anything is enqueued, so these run on a
machine without a GPU (the addresses are never used)."""

from __future__ import annotations

import ctypes

import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo
from matrix_orthogonalizing_optimizer_amd import _lib as L

BASE = 0x10000000


def _item(**kw):
    it = L.MoFp8Item(BASE, BASE + 0x100000, BASE + 0x200000, BASE + 0x300000, BASE + 0x400000, 64, 96, 96)
    for k, v in kw.items():
        setattr(it, k, v)
    return it


def _quantize(*items, count=None, dtype=L.MO_BF16, square=0):
    arr = (L.MoFp8Item * max(1, len(items)))(*items)
    return L.lib().mo_fp8_quantize(arr if items else None, len(items) if count is None else count, dtype, square, None)


@pytest.mark.parametrize("square", [0, 1])
@pytest.mark.parametrize("kw,word", [
    (dict(rows=-1), "rows and cols"), (dict(cols=-1), "rows and cols"), (dict(rows=1 << 31), "rows and cols"),
    (dict(rows=1 << 21, cols=1 << 21, ld=1 << 21), "2^40"), (dict(ld=95), "ld"), (dict(ld=1 << 40), "ld"),
    (dict(src=None), "src"), (dict(src=BASE + 1), "aligned"), (dict(codes=None), "image"),
    (dict(scales_t=None), "image"), (dict(codes=None, scales=None, codes_t=None, scales_t=None), "image"),
    (dict(codes=BASE + 0x100008), "aligned"), (dict(scales=BASE + 0x200008), "aligned"),
    (dict(codes=BASE), "overlaps"), (dict(codes_t=BASE + 0x100010), "overlaps"),
    (dict(scales=BASE + 0x100400), "overlaps"),
])
def test_quantize_refuses(kw, word, square):
    assert _quantize(_item(**kw), square=square) == L.MO_EINVAL
    assert word in L.last_error()


def test_quantize_refuses_the_list():
    assert _quantize(count=1) == L.MO_EINVAL and "NULL" in L.last_error()
    assert _quantize(_item(), count=-1) == L.MO_EINVAL
    assert _quantize(_item(), dtype=2) == L.MO_EINVAL
    assert _quantize(_item(), _item(codes=BASE + 0x500000, scales=BASE + 0x600000, codes_t=BASE + 64)) == L.MO_EINVAL
    assert "overlaps" in L.last_error()
    assert _quantize(count=0) == L.MO_OK
    # matrices without elements are no work, whatever their pointers
    assert _quantize(_item(rows=0, src=None), _item(cols=0, ld=0, codes=None, scales=None)) == L.MO_OK


def test_image_size():
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    for (r, k), want in {(1, 1): (128, 16), (3, 129): (768, 48), (7, 2048): (14336, 112), (2, 2049): (4352, 64),
                         (0, 5): (0, 0), (5, 0): (0, 0)}.items():
        assert L.lib().mo_fp8_image_size(r, k, ctypes.byref(c), ctypes.byref(s)) == L.MO_OK
        assert (c.value, s.value) == want
    assert L.lib().mo_fp8_image_size(-1, 4, ctypes.byref(c), ctypes.byref(s)) == L.MO_EINVAL
    assert L.lib().mo_fp8_image_size(4, 4, None, ctypes.byref(s)) == L.MO_EINVAL


def _image(rows=64, cols=96, at=BASE, **kw):
    x = L.MoFp8Image(at, at + 0x100000, rows, cols)
    for k, v in kw.items():
        setattr(x, k, v)
    return x


def _matmul(a, b, out=BASE + 0x800000, dt=L.MO_F32, ldo=64, accumulate=0):
    return L.lib().mo_fp8_matmul(ctypes.byref(a) if a else None, ctypes.byref(b) if b else None, out, dt, ldo,
                                 accumulate, None)


def test_matmul_refuses():
    b = _image(at=BASE + 0x200000)
    for args, word in [
        ((None, b), "NULL"), ((_image(cols=95), b), "columns"), ((_image(codes=None), b), "non-NULL"),
        ((_image(codes=BASE + 4), b), "aligned"), ((_image(scales=BASE + 0x100004), b), "aligned"),
        ((_image(rows=-1), b), "rows and cols"),
    ]:
        assert _matmul(*args) == L.MO_EINVAL
        assert word in L.last_error()
    a = _image()
    assert _matmul(a, b, out=None) == L.MO_EINVAL
    assert _matmul(a, b, out=BASE + 0x800002) == L.MO_EINVAL
    assert _matmul(a, b, ldo=63) == L.MO_EINVAL and "ldo" in L.last_error()
    assert _matmul(a, b, dt=7) == L.MO_EINVAL
    assert _matmul(a, b, out=BASE + 0x100000) == L.MO_EINVAL and "overlaps" in L.last_error()
    # nothing to write, and nothing to add
    assert _matmul(_image(rows=0, codes=None), b, out=None) == L.MO_OK
    assert _matmul(_image(cols=0), _image(cols=0, at=BASE + 0x200000), accumulate=1) == L.MO_OK


def test_product_refuses_too_many_tiles_and_too_long_rows():
    a, b = _image(rows=1 << 18, cols=32), _image(rows=1 << 18, cols=32, at=BASE << 8)
    assert _matmul(a, b, out=BASE << 12, ldo=1 << 18) == L.MO_EINVAL and "tiles" in L.last_error()
    a, b = _image(rows=2, cols=(1 << 23) + 1), _image(rows=2, cols=(1 << 23) + 1, at=BASE << 8)
    a.scales, b.scales = BASE << 4, BASE << 9
    assert _matmul(a, b, out=BASE << 12, ldo=2) == L.MO_EINVAL and "2^23" in L.last_error()


def test_dequantize_refuses():
    dst = (ctypes.c_void_p * 1)(BASE + 0x800000)
    img = (L.MoFp8Image * 1)(_image())
    f = L.lib().mo_fp8_dequantize
    assert f(img, dst, 1, 5, None) == L.MO_EINVAL
    assert f(img, None, 1, L.MO_F32, None) == L.MO_EINVAL
    assert f(img, (ctypes.c_void_p * 1)(BASE + 0x800004), 1, L.MO_F32, None) == L.MO_EINVAL
    assert f(img, (ctypes.c_void_p * 1)(BASE + 16), 1, L.MO_F32, None) == L.MO_EINVAL
    assert f((L.MoFp8Image * 1)(_image(scales=None)), dst, 1, L.MO_F32, None) == L.MO_EINVAL
    assert f((L.MoFp8Image * 1)(_image(cols=0)), dst, 1, L.MO_F32, None) == L.MO_OK


_CE = dict(x=BASE, x_dtype=L.MO_BF16, ldx=64, w=BASE + 0x10000, w_dtype=L.MO_BF16, ldw=64, rows=8, hidden=64, vocab=100,
           targets=BASE + 0x20000, grad_loss=BASE + 0x30000, loss=BASE + 0x40000, dx=BASE + 0x50000, ld_dx=64,
           dw=BASE + 0x60000, dw_dtype=L.MO_F32, ld_dw=64, accumulate=0, ws=0x70000000, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,word", [
    (dict(x_dtype=3), "x_dtype"), (dict(w_dtype=-1), "w_dtype"), (dict(dw_dtype=2), "dw_dtype"), (dict(rows=-1), "rows"),
    (dict(rows=(1 << 20) + 1), "rows"), (dict(hidden=0), "hidden"), (dict(hidden=(1 << 22) + 1), "hidden"),
    (dict(vocab=0), "vocab"), (dict(vocab=1 << 31), "vocab"), (dict(ldx=63), "stride of x"), (dict(ldw=63), "stride of w"),
    (dict(ld_dx=63), "stride of dx"), (dict(ld_dw=63), "stride of dw"), (dict(ldw=1 << 40), "2^40"), (dict(x=None), "x must"),
    (dict(w=None), "w must"), (dict(x=BASE + 1), "aligned"), (dict(dw=BASE + 0x60002), "aligned"),
    (dict(targets=None), "non-NULL"), (dict(loss=None), "non-NULL"), (dict(targets=BASE + 0x20004), "aligned"),
    (dict(grad_loss=BASE + 0x30002), "aligned"), (dict(accumulate=1, dw=None), "accumulate"),
    (dict(dx=BASE), "overlaps"), (dict(dw=BASE + 0x10000), "overlaps"), (dict(loss=BASE + 0x30010), "overlaps"),
    (dict(ws=BASE & ~0xfff), "overlaps"),
])
def test_cross_entropy_refuses(kw, word):
    assert L.lib().mo_linear_ce(*{**_CE, **kw}.values()) == L.MO_EINVAL
    assert word in L.last_error()


def _ce_need(rows, hidden, vocab, x_dt=L.MO_BF16, dw_dt=L.MO_BF16, dx=1, dw=1):
    n = ctypes.c_size_t()
    assert L.lib().mo_linear_ce_workspace_size(rows, hidden, vocab, x_dt, dw_dt, dx, dw, ctypes.byref(n)) == L.MO_OK
    return n.value


def test_cross_entropy_workspace():
    for kw in (dict(), dict(dx=None), dict(dw=None), dict(dx=None, dw=None)):
        a = {**_CE, **kw}
        need = _ce_need(8, 64, 100, dw_dt=L.MO_F32, dx=int(a["dx"] is not None), dw=int(a["dw"] is not None))
        assert L.lib().mo_linear_ce(*{**a, "ws_bytes": need - 1}.values()) == L.MO_EWORKSPACE
        assert L.lib().mo_linear_ce(*{**a, "ws": None}.values()) == L.MO_EWORKSPACE
    # no rows, and nothing to write: no work and no workspace
    assert L.lib().mo_linear_ce(*{**_CE, "rows": 0, "x": None, "dw": None, "ws": None, "ws_bytes": 0}.values()) == L.MO_OK
    assert L.lib().mo_linear_ce(*{**_CE, "rows": 0, "accumulate": 1, "ws": None, "ws_bytes": 0}.values()) == L.MO_OK
    n = ctypes.c_size_t()
    f = L.lib().mo_linear_ce_workspace_size
    assert f(1, 0, 10, 0, 0, 1, 1, ctypes.byref(n)) == L.MO_EINVAL
    assert f(1, 10, 10, 0, 5, 1, 1, ctypes.byref(n)) == L.MO_EINVAL
    assert f(1, 10, 10, 0, 0, 1, 1, None) == L.MO_EINVAL


def test_cross_entropy_workspace_does_not_grow_with_the_vocabulary():
    """Where 4 GiB do not hold the logits, the workspace holds pieces: those of
    16384 x 256000 in fp32 would be 16.8 GB."""
    some, more = _ce_need(16384, 4096, 66000), _ce_need(16384, 4096, 256000)
    assert more < 2 * some and more < 4e9
    for vocab in (32000, 64000, 65536, 66000, 1024000):
        assert _ce_need(16384, 4096, vocab) < (1 << 32) + 5e9
    assert _ce_need(16384, 4096, 256000, dx=0, dw=0) < 1e9


_BL = dict(logits=BASE, dtype=L.MO_F32, tokens=8, experts=16, ld=16, index=BASE + 0x10000, top=2, weight=0.01,
           grad_loss=BASE + 0x20000, loss=BASE + 0x30000, counts=BASE + 0x40000, grad=BASE + 0x50000, ld_grad=16,
           accumulate=0, ws=0x70000000, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=2), "dtype"), (dict(tokens=-1), "tokens"), (dict(tokens=1 << 31), "tokens"), (dict(experts=0), "experts"),
    (dict(experts=4097), "experts"), (dict(top=0), "top"), (dict(top=4097), "top"), (dict(ld=15), "stride of logits"),
    (dict(ld_grad=15), "stride of grad"), (dict(weight=float("nan")), "weight"), (dict(weight=float("inf")), "weight"),
    (dict(logits=None), "logits"), (dict(index=None), "index"), (dict(loss=None), "non-NULL"), (dict(counts=None), "non-NULL"),
    (dict(logits=BASE + 2), "aligned"), (dict(index=BASE + 0x10004), "aligned"), (dict(counts=BASE + 0x40004), "aligned"),
    (dict(accumulate=1, grad=None), "accumulate"), (dict(grad=BASE), "overlaps"), (dict(loss=BASE + 0x20000), "overlaps"),
    (dict(counts=BASE + 0x10008), "overlaps"),
])
def test_balance_refuses(kw, word):
    assert L.lib().mo_balance_loss(*{**_BL, **kw}.values()) == L.MO_EINVAL
    assert word in L.last_error()


def test_balance_workspace():
    n = ctypes.c_size_t()
    f = L.lib().mo_balance_loss_workspace_size
    assert f(8, 16, ctypes.byref(n)) == L.MO_OK and n.value == 0            # one workgroup, no workspace
    assert f(8000, 16, ctypes.byref(n)) == L.MO_OK and n.value > 0
    a = {**_BL, "tokens": 8000, "logits": BASE << 4, "index": BASE << 5, "grad": BASE << 6, "ws": BASE << 7}
    assert L.lib().mo_balance_loss(*{**a, "ws_bytes": n.value - 1}.values()) == L.MO_EWORKSPACE
    assert L.lib().mo_balance_loss(*{**a, "ws": None}.values()) == L.MO_EWORKSPACE
    assert f(-1, 16, ctypes.byref(n)) == L.MO_EINVAL and f(8, 4097, ctypes.byref(n)) == L.MO_EINVAL
    assert f(8, 16, None) == L.MO_EINVAL


# ------------------------------------------------------------- the Python front
@pytest.mark.parametrize("bad", [[[torch.zeros(2, 2)]], ["x"], [None], [torch.zeros(2, 2), "x"], [3]])
def test_front_refuses_lists_of_other_things(bad):
    with pytest.raises(TypeError, match="list"):
        mo.fp8_quantize(bad)
    with pytest.raises(TypeError, match="list"):
        mo.fp8_dequantize(bad)


def test_front_refuses_cpu_tensors_and_shapes():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU"):
        mo.fp8_quantize(x)
    with pytest.raises(ValueError, match="2-D"):
        mo.fp8_quantize(torch.zeros(4))
    with pytest.raises(TypeError):
        mo.fp8_quantize(x.double())
    with pytest.raises(TypeError):
        mo.fp8_quantize([x, x.bfloat16()])
    with pytest.raises(ValueError, match="strides"):
        mo.fp8_quantize(x.t())
    with pytest.raises(ValueError, match="images"):
        mo.fp8_quantize(x, images="all")
    with pytest.raises(ValueError, match="negative"):
        mo.Fp8Matrix.empty(-1, 32, "cpu")
    assert mo.fp8_quantize([]) == [] and mo.fp8_dequantize([]) == []
    assert mo.Fp8Matrix.empty(0, 300, "cpu").shape == (0, 300) and mo.Fp8Matrix.empty(3, 0, "cpu").codes.numel() == 0


def test_front_checks_images():
    codes, scales = torch.zeros(3, 128, dtype=torch.uint8), torch.zeros(3, 16, dtype=torch.uint8)
    q = mo.Fp8Matrix(codes, scales, 40)
    assert q.shape == (3, 40)
    for bad in [(codes, scales, 129), (codes.int(), scales, 40), (codes, scales[:2], 40), (codes[:, :64], scales, 40),
                (codes, scales, -1), (codes, scales, 0)]:
        with pytest.raises(ValueError):
            mo.Fp8Matrix(*bad)
    with pytest.raises(TypeError):
        mo.fp8_matmul(codes, q)
    with pytest.raises(TypeError):
        mo.fp8_matmul(q, mo.Mx4Matrix.empty(3, 40, "cpu"))
    with pytest.raises(ValueError, match="accumulate"):
        mo.fp8_matmul(q, q, accumulate=True)
    with pytest.raises(TypeError):
        mo.fp8_linear(torch.zeros(2, 40), codes)
    with pytest.raises(TypeError):
        mo.fp8_linear_backward(torch.zeros(2, 40), q, codes)
    with pytest.raises(ValueError, match="features"):
        mo.fp8_linear(torch.zeros(2, 41), q)
    with pytest.raises(ValueError, match="want"):
        mo.fp8_linear_backward(torch.zeros(2, 41), q, q)


def test_backward_refuses_before_any_work():
    dy, x_t, w_t = torch.zeros(5, 40), mo.Fp8Matrix.empty(64, 5, "cpu"), mo.Fp8Matrix.empty(64, 40, "cpu")
    with pytest.raises(ValueError, match="features"):
        mo.fp8_linear_backward(dy, mo.Fp8Matrix.empty(65, 5, "cpu"), w_t)
    with pytest.raises(ValueError, match="accumulate"):
        mo.fp8_linear_backward(dy, x_t, w_t, accumulate=True)
    with pytest.raises(ValueError, match="dw must be"):
        mo.fp8_linear_backward(dy, x_t, w_t, dw=torch.zeros(64, 40))
    with pytest.raises(ValueError, match="GPU"):
        mo.fp8_linear_backward(dy, x_t, w_t)


@pytest.mark.parametrize("kw,word", [
    (dict(weight=torch.zeros(9, 63)), "features"), (dict(targets=torch.zeros(4, dtype=torch.int32)), "targets"),
    (dict(targets=torch.zeros(3, dtype=torch.int64)), "targets"), (dict(grad_loss=torch.zeros(3)), "grad_loss"),
    (dict(grad="both"), "grad must"), (dict(dw=torch.zeros(9, 64), grad="x"), "dw given"), (dict(accumulate=True), "accumulate"),
    (dict(dw=torch.zeros(9, 65)), "dw must"), (dict(x=torch.zeros(4, 64).double()), "float64"), (dict(), "GPU"),
    (dict(weight=torch.zeros(64, 9).t()), "strides"), (dict(x=torch.zeros(4, 64, 2)[:, :, 0]), "strides"),
])
def test_front_checks_cross_entropy_arguments(kw, word):
    a = dict(x=torch.zeros(4, 64), weight=torch.zeros(9, 64), targets=torch.zeros(4, dtype=torch.int64))
    a.update(kw)
    with pytest.raises((ValueError, TypeError), match=word):
        mo.linear_cross_entropy(a.pop("x"), a.pop("weight"), a.pop("targets"), **a)


@pytest.mark.parametrize("kw,word", [
    (dict(index=torch.zeros(4, dtype=torch.int64)), "index"), (dict(index=torch.zeros(4, 2)), "index"),
    (dict(index=torch.zeros(3, 2, dtype=torch.int64)), "index"), (dict(grad_loss=torch.zeros(2)), "grad_loss"),
    (dict(out_grad=torch.zeros(4, 15)), "out_grad"), (dict(out_grad=torch.zeros(4, 16), grad=False), "out_grad"),
    (dict(accumulate=True), "accumulate"), (dict(), "GPU"),
])
def test_front_checks_balance_arguments(kw, word):
    a = dict(index=torch.zeros(4, 2, dtype=torch.int64))
    a.update(kw)
    with pytest.raises(ValueError, match=word):
        mo.balance_loss(torch.zeros(4, 16), a.pop("index"), **a)


def test_optimizer_refuses_unknown_images():
    with pytest.raises(ValueError, match="fp8"):
        mo.MuonAdamW([torch.zeros(4, 4)], fp8="all")
    with pytest.raises(RuntimeError, match="without fp8"):
        mo.MuonAdamW([torch.zeros(4, 4)]).refresh_fp8()
