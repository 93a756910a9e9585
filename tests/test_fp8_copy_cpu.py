"""Copies of 8-bit images: the addresses that the operators take are those of
the copy's own arrays.  No operator runs, so the arrays live on the CPU."""

from __future__ import annotations

import copy
import io
import pickle

import pytest
import torch

import matrix_orthogonalizing_optimizer_amd as mo


def _fill(q, seed):
    g = torch.Generator().manual_seed(seed)
    q.codes.copy_(torch.randint(0, 256, q.codes.shape, generator=g, dtype=torch.uint8))
    q.scales.copy_(torch.randint(0, 256, q.scales.shape, generator=g, dtype=torch.uint8))
    return q


def _made(seed=0):
    """As the operators make them: one allocation, cut up when asked for."""
    return _fill(mo.Fp8Matrix.empty(5, 300, "cpu"), seed)


def _given(seed=0):
    return _fill(mo.Fp8Matrix(torch.empty(5, 384, dtype=torch.uint8), torch.empty(5, 16, dtype=torch.uint8), 300), seed)


def _check(got, q, shares):
    assert type(got) is mo.Fp8Matrix and got is not q and got.shape == q.shape == (5, 300)
    assert torch.equal(got.codes, q.codes) and torch.equal(got.scales, q.scales)
    assert got._ptrs == (got.codes.data_ptr(), got.scales.data_ptr())
    assert list(got._struct()) == [*got._ptrs, 5, 300]
    assert (got._ptrs == q._ptrs) == shares
    # the memory is kept alive, and recorded on a stream, by the tensors that own it
    kept = {t.untyped_storage().data_ptr() for t in got._keep}
    assert {t.untyped_storage().data_ptr() for t in (got.codes, got.scales)} == kept
    got.codes[0, 0] ^= 1
    assert (int(got.codes[0, 0]) == int(q.codes[0, 0])) == shares
    got.codes[0, 0] ^= 1


def _torch_round_trip(q):
    f = io.BytesIO()
    torch.save(q, f)
    f.seek(0)
    return torch.load(f, weights_only=False)                    # written by this process


WAYS = {"deepcopy": copy.deepcopy, "pickle": lambda q: pickle.loads(pickle.dumps(q)), "torch": _torch_round_trip}


@pytest.mark.parametrize("used", [False, True])
@pytest.mark.parametrize("make", [_made, _given])
@pytest.mark.parametrize("way", sorted(WAYS))
def test_copies_own_their_addresses(way, make, used):
    q = make()
    if used:
        q._struct()                                             # the address list that calls keep
    _check(WAYS[way](q), q, False)


@pytest.mark.parametrize("make", [_made, _given])
def test_a_shallow_copy_shares_the_arrays(make):
    q = make()
    q._struct()
    _check(copy.copy(q), q, True)


def test_lists_and_pairs():
    """Images that share an allocation: their copies share one of their own, and
    one image is stored without the others."""
    qs = mo.Fp8Matrix._empty([(5, 300)] * 40, "cpu")
    for i, q in enumerate(qs):
        _fill(q, i)
    twice = copy.deepcopy([*qs, qs[0]])
    assert twice[-1] is twice[0]
    for got, q in zip(twice, qs):
        _check(got, q, False)
    assert len({t.untyped_storage().data_ptr() for q in twice for t in q._keep}) == 1
    assert len(pickle.dumps(qs[3])) < 2 * (qs[3].codes.numel() + qs[3].scales.numel()) + 4096
    for got, q in zip(pickle.loads(pickle.dumps(qs)), qs):
        _check(got, q, False)


def test_a_copy_keeps_what_shares_its_arrays():
    """A layer that registers an image's arrays as buffers, copied as a whole."""
    class Layer(torch.nn.Module):
        def __init__(self):
            super().__init__()
            q = _given()
            self.register_buffer("codes", q.codes)
            self.register_buffer("scales", q.scales)
            self.image = q

    a = Layer()
    b = copy.deepcopy(a)
    _check(b.image, a.image, False)
    assert b.image._ptrs == (b.codes.data_ptr(), b.scales.data_ptr())


def test_images_without_elements():
    for r, c in ((0, 5), (5, 0), (0, 0)):
        for got in (copy.deepcopy(mo.Fp8Matrix.empty(r, c, "cpu")), pickle.loads(pickle.dumps(mo.Fp8Matrix.empty(r, c, "cpu")))):
            assert got.shape == (r, c) and got._ptrs == (got.codes.data_ptr(), got.scales.data_ptr())


def test_an_optimizer_copied_before_its_first_step():
    """Its images are its own: rewriting them leaves the first one's alone."""
    p = torch.nn.Parameter(torch.zeros(5, 300))
    opt = mo.MuonAdamW([p], [], fp8="rows")
    opt.fp8 = [_made()]
    other = copy.deepcopy(opt)
    _check(other.fp8[0], opt.fp8[0], False)
