"""The workspace of the linear cross entropy: the logits in it are 4 GiB at most."""

from __future__ import annotations

import ctypes

import pytest

from matrix_orthogonalizing_optimizer_amd import _lib as L


def _need(rows, hidden, vocab):
    n = ctypes.c_size_t()
    assert L.lib().mo_linear_ce_workspace_size(rows, hidden, vocab, L.MO_BF16, L.MO_BF16, 1, 1, ctypes.byref(n)) == L.MO_OK
    return n.value


@pytest.mark.parametrize("rows,vocab", [(8192, 131072), (8192, 131000), (4096, 262144), (16384, 65536), (1 << 20, 1024),
                                        (1 << 20, 1000), (1 << 16, 16384), (1000, 1073700)])
def test_kept_logits_take_4_gib_at_most(rows, vocab):
    """Of 256 hidden columns on logits are kept, of 255 only small ones; the
    operands' copies are as large but for a row of each transpose."""
    logits = _need(rows, 256, vocab) - _need(rows, 255, vocab)
    more = 2 * (rows + vocab + 512) + 4096
    assert rows * vocab * 4 <= logits <= (4 << 30) + more
