"""MI355X-native Muon optimizer step (HIP, gfx950) behind a C ABI.

The method is that of "Muon is Scalable for LLM Training" (Moonshot AI /
UCLA, 2025): Nesterov momentum (section 2.1, Eq. 1), Frobenius
normalisation and quintic Newton-Schulz (Eq. 2), the 0.2 * sqrt(max(A, B))
shape scale with decoupled weight decay (section 2.2, Eq. 4), and AdamW with
the same learning rate and decay for non-matrix parameters.

Next to the step stand the operators that a 4-bit student of the trained
weights needs: microscaled 4-bit images of matrices and their products
(``mx4_*``), token log probabilities with the top alternatives, and the
distillation loss with its gradient.  For training in 8 bits: 8-bit floating
point images with a scale per block of 128 and their products (``fp8_*``), the
cross entropy of an LM head from its input and weights, which leaves no logits
behind, and a router's balance loss with its experts' counts.

No function here takes part in autograd: results carry no graph, also where
an argument requires a gradient.  The backward passes are calls of their own
(``mx4_linear_backward``, ``fp8_linear_backward``, the gradients that the
losses return).

This module only marshals torch tensors into the C ABI of ``libmuon.so``
(``include/muon.h``); PyTorch provides device memory and streams.  Every
arithmetic step runs in the HIP library, and there is no fallback.
"""

from __future__ import annotations

import contextlib
import copy
import ctypes
import functools
import threading
from typing import Iterable, List, NamedTuple, Optional, Sequence, Tuple, Union

import torch

from ._lib import (KERNEL_CLASS_NAMES, MO_BF16, MO_F32, MO_MAX_TOP, MoMatrix, MoMx4Image,  # noqa: F401
                   MoMx4Item, MoTensor, MuonError, check, last_error, lib)

__all__ = ["muon_step", "adamw_step", "newton_schulz", "muon_workspace_size",
           "newton_schulz_workspace_size", "svd_entropy", "svd_entropy_workspace_size",
           "Mx4Matrix", "mx4_quantize", "mx4_dequantize", "mx4_matmul", "mx4_linear",
           "mx4_linear_backward", "Fp8Matrix", "fp8_quantize", "fp8_dequantize", "fp8_matmul",
           "fp8_linear", "fp8_linear_backward", "linear_cross_entropy", "BalanceLoss", "balance_loss",
           "TokenLogprobs", "token_logprobs", "distill_loss",
           "MuonPlan", "MuonAdamW", "profile_enable", "profile_read", "profile_reset",
           "MuonError", "KERNEL_CLASS_NAMES"]

_DT = {torch.float32: MO_F32, torch.bfloat16: MO_BF16}


def _dtype_code(dt: torch.dtype, what: str) -> int:
    if dt not in _DT:
        raise TypeError(f"{what}: dtype {dt} is not float32 or bfloat16")
    return _DT[dt]


def _common_dtype(ts: Sequence[torch.Tensor], what: str) -> torch.dtype:
    dts = {t.dtype for t in ts}
    if len(dts) != 1:
        raise TypeError(f"{what}: all tensors must share one dtype, got {dts}")
    return next(iter(dts))


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream_handle(device: torch.device, stream=None) -> int:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _abc(abc) -> Optional[ctypes.Array]:
    if abc is None:
        return None
    a = (ctypes.c_float * 3)(*[float(x) for x in abc])
    return a


def _shape2(t: torch.Tensor) -> Tuple[int, int]:
    if t.dim() != 2:
        raise ValueError(f"Muon matrices must be 2-D, got shape {tuple(t.shape)}")
    return int(t.shape[0]), int(t.shape[1])


_WS: dict = {}


def _workspace(device: torch.device, nbytes: int, stream_handle: int, cache: Optional[dict] = None) -> torch.Tensor:
    """A cached byte buffer of at least ``nbytes`` for one (device, stream).
    Calls queued on different streams never share it, and it is allocated on
    that stream, so torch's allocator orders any reuse of its memory after
    the work queued there."""
    cache = _WS if cache is None else cache
    key = (device.type, device.index, int(stream_handle or 0))
    ws = cache.get(key)
    if ws is None or ws.numel() < nbytes:
        cache.pop(key, None)
        n = max(nbytes, 256)
        if stream_handle and stream_handle != torch.cuda.current_stream(device).cuda_stream:
            with torch.cuda.stream(torch.cuda.ExternalStream(stream_handle, device=device)):
                ws = torch.empty(n, dtype=torch.uint8, device=device)
        else:
            ws = torch.empty(n, dtype=torch.uint8, device=device)
        cache[key] = ws
    return ws


def _mk_tensors(params, grads, s0, s1=None):
    n = len(params)
    arr = (MoTensor * max(n, 1))()
    for i in range(n):
        r, c = (_shape2(params[i]) if params[i].dim() == 2
                else (1, params[i].numel()))
        arr[i].param = _ptr(params[i])
        arr[i].grad = _ptr(grads[i])
        arr[i].state0 = _ptr(s0[i])
        arr[i].state1 = _ptr(s1[i]) if s1 is not None else None
        arr[i].rows = r
        arr[i].cols = c
    return arr


def muon_workspace_size(shapes: Iterable[Tuple[int, int]],
                        ns_dtype: torch.dtype = torch.bfloat16) -> Tuple[int, int]:
    """(full, minimum) workspace bytes of ``mo_muon_step`` for these shapes."""
    shapes = list(shapes)
    arr = (MoTensor * max(len(shapes), 1))()
    for i, (r, c) in enumerate(shapes):
        arr[i].rows, arr[i].cols = int(r), int(c)
    full, mn = ctypes.c_size_t(), ctypes.c_size_t()
    check(lib().mo_muon_workspace_size(arr, len(shapes), _dtype_code(ns_dtype, "ns_dtype"),
                                       ctypes.byref(full), ctypes.byref(mn)))
    return full.value, mn.value


def muon_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
              moms: Sequence[torch.Tensor], *, lr: float, wd: float = 0.1,
              mu: float = 0.95, nesterov: bool = True, ns_steps: int = 5,
              abc=None, rms_scale: float = 0.2, eps: float = 1e-7,
              ns_dtype: torch.dtype = torch.bfloat16,
              update_rms: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """One Muon step over matrix parameters (``mo_muon_step``).

    ``params`` fp32 [A, B], ``grads`` fp32/bf16, ``moms`` fp32/bf16 (one
    dtype per list), all contiguous on one GPU.  ``update_rms``: optional
    fp32 tensor [len(params)] receiving sqrt(mean(X_N^2)) per matrix.
    """
    n = len(params)
    if not (len(grads) == len(moms) == n):
        raise ValueError("params, grads and moms must have the same length")
    if n == 0:
        return
    dev = params[0].device
    gdt = _dtype_code(_common_dtype(grads, "grads"), "grads")
    mdt = _dtype_code(_common_dtype(moms, "moms"), "moms")
    ndt = _dtype_code(ns_dtype, "ns_dtype")
    arr = _mk_tensors(params, grads, moms)
    full, mn = muon_workspace_size([_shape2(p) for p in params], ns_dtype)
    sh = _stream_handle(dev, stream)
    if workspace is None:
        workspace = _workspace(dev, full, sh)
    if update_rms is not None and (update_rms.dtype != torch.float32 or update_rms.numel() < n):
        raise ValueError("update_rms must be float32 with one slot per matrix")
    check(lib().mo_muon_step(arr, n, gdt, mdt, ndt, lr, wd, mu, int(nesterov), ns_steps,
                             _abc(abc), rms_scale, eps, _ptr(update_rms), _ptr(workspace),
                             workspace.numel() * workspace.element_size(),
                             sh))


_SCALINGS = {"shape": 0, "hidden": 1, "update_norm": 2}


class MuonPlan:
    """``mo_muon_plan_*``: binds one list of matrices for repeated steps."""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                 moms: Sequence[torch.Tensor], ns_dtype: torch.dtype = torch.bfloat16):
        n = len(params)
        if not (len(grads) == len(moms) == n):
            raise ValueError("params, grads and moms must have the same length")
        self.n = n
        self.device = params[0].device if n else torch.device("cuda")
        # the plan holds raw pointers: keep the tensors alive while it lives
        self._keep = (list(params), list(grads), list(moms))
        self._grad_meta = [(tuple(g.shape), g.dtype) for g in grads]
        self._grads_bound = True
        gdt = _dtype_code(_common_dtype(grads, "grads"), "grads") if n else MO_F32
        mdt = _dtype_code(_common_dtype(moms, "moms"), "moms") if n else MO_F32
        arr = _mk_tensors(params, grads, moms)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            check(lib().mo_muon_plan_create(arr, n, gdt, mdt, _dtype_code(ns_dtype, "ns_dtype"),
                                            ctypes.byref(h)))
        self._h = h
        full, mn = ctypes.c_size_t(), ctypes.c_size_t()
        check(lib().mo_muon_plan_workspace_size(self._h, ctypes.byref(full), ctypes.byref(mn)))
        self.workspace_bytes, self.min_workspace_bytes = full.value, mn.value

    def step(self, *, lr: float, wd: float = 0.1, mu: float = 0.95, nesterov: bool = True,
             ns_steps: int = 5, abc=None, rms_scale: float = 0.2, eps: float = 1e-7,
             update_rms: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, stream=None,
             scaling: str = "shape", hidden: Optional[float] = None) -> None:
        """scaling: "shape" (0.2 sqrt(max(A, B)), Eq. 4 / 7), "hidden"
        (0.2 sqrt(hidden), Eq. 5) or "update_norm" (0.2 / RMS(X_N), Eq. 6)."""
        if self._h is None:
            raise RuntimeError("plan was closed")
        if not self._grads_bound:
            raise RuntimeError("gradients were released: call set_grads() before step()")
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
        if scaling == "hidden" and hidden is None:
            raise ValueError('scaling="hidden" needs hidden=H')
        check(lib().mo_muon_plan_set_scaling(self._h, _SCALINGS[scaling],
                                             float(hidden) if hidden is not None else 0.0))
        sh = _stream_handle(self.device, stream)
        if workspace is None:
            workspace = _workspace(self.device, self.workspace_bytes, sh)
        check(lib().mo_muon_plan_step(self._h, lr, wd, mu, int(nesterov), ns_steps, _abc(abc),
                                      rms_scale, eps, _ptr(update_rms), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), sh))

    def set_grads(self, grads: Sequence[torch.Tensor], stream=None) -> None:
        """Rebind the plan's gradients (``mo_muon_plan_set_grads``): same
        shapes and dtype, new buffers.  Nothing is enqueued when the pointers
        are unchanged; otherwise one small kernel per 96 matrices updates the
        descriptor table on the stream, with no host synchronisation."""
        if self._h is None:
            raise RuntimeError("plan was closed")
        grads = list(grads)
        if len(grads) != self.n:
            raise ValueError(f"expected {self.n} gradients, got {len(grads)}")
        for i, (g, (shape, dt)) in enumerate(zip(grads, self._grad_meta)):
            if tuple(g.shape) != shape or g.dtype != dt:
                raise ValueError(f"grad {i}: expected {shape} {dt}, got {tuple(g.shape)} {g.dtype}")
        arr = (ctypes.c_void_p * max(self.n, 1))(*[_ptr(g) for g in grads])
        with torch.cuda.device(self.device):
            check(lib().mo_muon_plan_set_grads(self._h, arr, self.n,
                                               _stream_handle(self.device, stream)))
        self._keep = (self._keep[0], grads, self._keep[2])
        self._grads_bound = True

    def release_grads(self) -> None:
        """Drop the plan's references to its gradients once a step using
        them is queued (torch orders any reuse of their memory after the
        work already queued on the stream), so a framework that makes fresh
        gradients every step does not hold two sets.  The next step needs
        ``set_grads`` first."""
        self._keep = (self._keep[0], None, self._keep[2])
        self._grads_bound = False

    def close(self) -> None:
        if getattr(self, "_h", None) is not None:
            check(lib().mo_muon_plan_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
               exp_avg: Sequence[torch.Tensor], exp_avg_sq: Sequence[torch.Tensor], *,
               lr: float, step: int, wd: float = 0.1, beta1: float = 0.9,
               beta2: float = 0.999, eps: float = 1e-8, stream=None) -> None:
    """AdamW for non-matrix parameters (``mo_adamw_step``); fp32 params and
    moments, fp32/bf16 grads, ``step`` >= 1."""
    n = len(params)
    if not (len(grads) == len(exp_avg) == len(exp_avg_sq) == n):
        raise ValueError("all lists must have the same length")
    if n == 0:
        return
    gdt = _dtype_code(_common_dtype(grads, "grads"), "grads")
    arr = (MoTensor * n)()
    for i in range(n):
        arr[i].param = _ptr(params[i])
        arr[i].grad = _ptr(grads[i])
        arr[i].state0 = _ptr(exp_avg[i])
        arr[i].state1 = _ptr(exp_avg_sq[i])
        arr[i].rows, arr[i].cols = 1, params[i].numel()
    check(lib().mo_adamw_step(arr, n, gdt, lr, wd, beta1, beta2, eps, int(step),
                              _stream_handle(params[0].device, stream)))


def newton_schulz_workspace_size(batch: int, rows: int, cols: int,
                                 dtype: torch.dtype = torch.bfloat16) -> int:
    out = ctypes.c_size_t()
    check(lib().mo_newton_schulz_workspace_size(batch, rows, cols, _dtype_code(dtype, "dtype"),
                                                ctypes.byref(out)))
    return out.value


def newton_schulz(x: torch.Tensor, *, ns_steps: int = 5, abc=None, eps: float = 1e-7,
                  out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Normalise and iterate Eq. 2 (``mo_newton_schulz``) on ``x`` [rows, cols]
    or [batch, rows, cols] (fp32 or bf16); returns X_N in x's dtype."""
    squeeze = x.dim() == 2
    x3 = x.unsqueeze(0) if squeeze else x
    if x3.dim() != 3:
        raise ValueError("x must be 2-D or 3-D")
    b, r, c = (int(v) for v in x3.shape)
    dt = _dtype_code(x.dtype, "x")
    if out is None:
        out = torch.empty_like(x3)
    ws_need = newton_schulz_workspace_size(b, r, c, x.dtype)
    sh = _stream_handle(x.device, stream)
    if workspace is None:
        workspace = _workspace(x.device, ws_need, sh)
    check(lib().mo_newton_schulz(_ptr(x3), _ptr(out), b, r, c, dt, ns_steps, _abc(abc), eps,
                                 _ptr(workspace), workspace.numel() * workspace.element_size(), sh))
    return out[0] if squeeze else out


def _mk_matrices(shapes_ptrs):
    n = len(shapes_ptrs)
    arr = (MoMatrix * max(n, 1))()
    for i, (ptr, r, c) in enumerate(shapes_ptrs):
        arr[i].data = ptr
        arr[i].rows = r
        arr[i].cols = c
    return arr


def svd_entropy_workspace_size(shapes: Iterable[Tuple[int, int]]) -> Tuple[int, int]:
    """(full, minimum) workspace bytes of ``mo_svd_entropy`` for [rows, cols] shapes."""
    shapes = list(shapes)
    arr = _mk_matrices([(16, r, c) for r, c in shapes])   # placeholder aligned address
    full, mn = ctypes.c_size_t(), ctypes.c_size_t()
    check(lib().mo_svd_entropy_workspace_size(arr, len(shapes), ctypes.byref(full),
                                              ctypes.byref(mn)))
    return full.value, mn.value


def svd_entropy(mats: Sequence[torch.Tensor], *, sigma: bool = False,
                workspace: Optional[torch.Tensor] = None, stream=None):
    """SVD entropy (section 3.4) of each 2-D matrix (fp32 or bf16, one dtype),
    as an fp64 tensor [len(mats)]; with ``sigma=True`` also a list of each
    matrix's singular values, largest first (appendix F), fp64."""
    mats = list(mats)
    if not mats:
        return (torch.empty(0, dtype=torch.float64), []) if sigma else torch.empty(0, dtype=torch.float64)
    dt = _dtype_code(_common_dtype(mats, "mats"), "mats")
    dev = mats[0].device
    arr = _mk_matrices([(_ptr(m),) + _shape2(m) for m in mats])
    ent = torch.empty(len(mats), dtype=torch.float64, device=dev)
    counts = [min(_shape2(m)) for m in mats]
    sig = torch.empty(sum(counts), dtype=torch.float64, device=dev) if sigma else None
    sh = _stream_handle(dev, stream)
    if workspace is None:
        full, _ = svd_entropy_workspace_size(_shape2(m) for m in mats)
        workspace = _workspace(dev, full, sh)
    check(lib().mo_svd_entropy(arr, len(mats), dt, _ptr(ent), _ptr(sig), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), sh))
    if not sigma:
        return ent
    return ent, list(torch.split(sig, counts))


# ---------------------------------------------------------------- 4-bit matrices
def _raw_stream(index: int) -> int:
    """Handle of the current stream of a device (torch's quick form of
    ``torch.cuda.current_stream(index).cuda_stream`` where it has one)."""
    return torch.cuda.current_stream(index).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


class _launch_on:
    """Device and stream of one call: outputs made inside belong to that
    stream, and ``tensors`` used on another stream than the current one are
    recorded on it, so that the allocator keeps their memory until then.
    Gives the stream's handle.  A class, and nothing switched where nothing
    changes: small calls cost little more than their launch."""

    __slots__ = ("device", "stream", "tensors", "stack")

    def __init__(self, device: torch.device, stream, tensors: Sequence[Optional[torch.Tensor]]):
        if device.type != "cuda":
            raise ValueError("tensors must live on the GPU")
        for t in tensors:
            if t is not None and t.device != device:
                raise ValueError(f"tensors of one call must share a device, got {t.device} and {device}")
        self.device, self.stream, self.tensors, self.stack = device, stream, tensors, None

    def __enter__(self) -> int:
        dev = self.device
        handle = here = _raw_stream(dev.index)
        if self.stream is not None:
            handle = _stream_handle(dev, self.stream)
        if handle == here and torch.cuda.current_device() == dev.index:
            return handle
        self.stack = contextlib.ExitStack()
        self.stack.enter_context(torch.cuda.device(dev))
        if handle != here:
            other = torch.cuda.ExternalStream(handle, device=dev)
            self.stack.enter_context(torch.cuda.stream(other))
            for t in self.tensors:
                if t is not None:
                    t.record_stream(other)
        return handle

    def __exit__(self, *exc) -> None:
        if self.stack is not None:
            self.stack.close()


def _rows_of(t: torch.Tensor, what: str) -> Tuple[int, int, int, int]:
    """(pointer, rows, cols, row stride) of a 2-D tensor with unit column stride."""
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D, got shape {tuple(t.shape)}")
    r, c = t.shape
    ld, step = t.stride()
    if r < 2:
        ld = c or 1
    if (c > 1 and step != 1) or ld < c:
        raise ValueError(f"{what}: rows must be contiguous and must not overlap (strides {t.stride()})")
    return t.data_ptr(), r, c, ld


def _vector(t: Optional[torch.Tensor], dtype: torch.dtype, shape: Tuple[int, ...], what: str) -> Optional[int]:
    if t is None:
        return None
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


# Two threads on one stream share its cached workspace: a call's launches must
# not mix with another's (the binding releases the interpreter lock). Optimizer
# steps have workspaces of their own.
_TOKEN_WS: dict = {}
_SCRATCH_LOCK = threading.Lock()


@functools.lru_cache(maxsize=1024)
def _token_workspace(query: str, rows: int, vocab: int, top: int) -> int:
    need = ctypes.c_size_t()
    check(getattr(lib(), query)(rows, vocab, top, ctypes.byref(need)))
    return need.value


def _scratch(nbytes: int, handle: int, device: torch.device) -> Optional[torch.Tensor]:
    """Workspace of one call: the cached one of (device, stream), or, while a
    graph is being captured, memory of that graph alone."""
    if nbytes == 0:
        return None
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    return _workspace(device, nbytes, handle, _TOKEN_WS)


class Mx4Matrix:
    """The microscaled 4-bit image of a [rows, cols] matrix: ``codes`` uint8
    [rows, 16 nb] and ``scales`` uint8 [rows, 4 ceil(nb / 4)] with nb =
    ceil(cols / 32) blocks per row, as ``include/muon.h`` lays them out."""

    __slots__ = ("codes", "scales", "rows", "cols")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int):
        if codes.dim() != 2:
            raise ValueError("codes must be 2-D")
        rows, nb = int(codes.shape[0]), -(-int(cols) // 32)
        if cols < 1 or rows < 1:
            raise ValueError("an image has at least one row and one column")
        for t, w, what in ((codes, 16 * nb, "codes"), (scales, -(-nb // 4) * 4, "scales")):
            if t.dtype != torch.uint8 or tuple(t.shape) != (rows, w) or not t.is_contiguous():
                raise ValueError(f"{what} of a [{rows}, {cols}] image must be contiguous uint8 "
                                 f"[{rows}, {w}], got {t.dtype} {tuple(t.shape)}")
        if codes.device != scales.device:
            raise ValueError("codes and scales must share a device")
        self.codes, self.scales, self.rows, self.cols = codes, scales, rows, int(cols)

    @property
    def shape(self) -> Tuple[int, int]:
        return self.rows, self.cols

    @property
    def device(self) -> torch.device:
        return self.codes.device

    @classmethod
    def empty(cls, rows: int, cols: int, device) -> "Mx4Matrix":
        """An image whose contents are still to be written."""
        if rows < 1 or cols < 1:
            raise ValueError(f"an image has at least one row and one column, got [{rows}, {cols}]")
        nb = -(-cols // 32)
        q = object.__new__(cls)                 # right by construction: no checks
        q.codes = torch.empty((rows, 16 * nb), dtype=torch.uint8, device=device)
        q.scales = torch.empty((rows, -(-nb // 4) * 4), dtype=torch.uint8, device=device)
        q.rows, q.cols = rows, cols
        return q

    def _struct(self) -> MoMx4Image:
        return MoMx4Image(self.codes.data_ptr(), self.scales.data_ptr(), self.rows, self.cols)

    def __repr__(self) -> str:
        return f"Mx4Matrix([{self.rows}, {self.cols}], device={self.device})"


_IMAGES = ("rows", "cols", "both")


def mx4_quantize(x: Union[torch.Tensor, Sequence[torch.Tensor]], *, images: str = "rows",
                 out=None, stream=None):
    """4-bit images of a 2-D matrix or of a list of them (``mo_mx4_quantize``;
    fp32 or bf16, one dtype; rows may be strided).

    ``images``: "rows" -- the image of x (blocks along its rows); "cols" --
    the image of x^T (blocks along x's columns); "both" -- the pair of them,
    from one reading of x.  A list gives a list.  ``out``: images of an
    earlier call (same form) to overwrite.
    """
    if images not in _IMAGES:
        raise ValueError(f"images must be one of {_IMAGES}")
    single = isinstance(x, torch.Tensor)
    xs = [x] if single else list(x)
    if not xs:
        return []
    outs = None if out is None else ([out] if single else list(out))
    if outs is not None and len(outs) != len(xs):
        raise ValueError(f"out has {len(outs)} entries for {len(xs)} matrices")
    dt = _dtype_code(_common_dtype(xs, "x"), "x")
    dev = xs[0].device
    views = [_rows_of(t, "x") for t in xs]
    given = []                                   # (image, transposed image) of each matrix
    if outs is not None:
        for (_, r, c, _), o in zip(views, outs):
            pair = tuple(o) if images == "both" else (o, None) if images == "rows" else (None, o)
            if len(pair) != 2:
                raise ValueError('out must hold pairs for images="both"')
            for q, shape in zip(pair, ((r, c), (c, r))):
                if q is not None and not isinstance(q, Mx4Matrix):
                    raise TypeError("out must hold Mx4Matrix")
                if q is not None and q.shape != shape:
                    raise ValueError(f"out: expected an image of {shape}, got {q.shape}")
            if (images != "cols" and pair[0] is None) or (images != "rows" and pair[1] is None):
                raise ValueError("out lacks an image")
            given.append(pair)
    used = xs + [t for p in given for q in p if q is not None for t in (q.codes, q.scales)]
    with _launch_on(dev, stream, used) as handle:
        if outs is None:
            given = [(Mx4Matrix.empty(r, c, dev) if images != "cols" else None,
                      Mx4Matrix.empty(c, r, dev) if images != "rows" else None) for _, r, c, _ in views]
        arr = (MoMx4Item * len(xs))()
        for it, (ptr, r, c, ld), (q, qt) in zip(arr, views, given):
            it.src, it.rows, it.cols, it.ld = ptr, r, c, ld
            if q is not None:
                it.codes, it.scales = q.codes.data_ptr(), q.scales.data_ptr()
            if qt is not None:
                it.codes_t, it.scales_t = qt.codes.data_ptr(), qt.scales.data_ptr()
        check(lib().mo_mx4_quantize(arr, len(xs), dt, handle))
    res = [p if images == "both" else p[0] if images == "rows" else p[1] for p in given]
    return res[0] if single else res


def mx4_dequantize(q: Union[Mx4Matrix, Sequence[Mx4Matrix]], *, dtype: torch.dtype = torch.bfloat16,
                   stream=None):
    """The values that an image, or each of a list, stands for (``mo_mx4_dequantize``)."""
    single = isinstance(q, Mx4Matrix)
    qs = [q] if single else list(q)
    dt = _dtype_code(dtype, "dtype")
    if not qs:
        return []
    dev = qs[0].device
    with _launch_on(dev, stream, [t for i in qs for t in (i.codes, i.scales)]) as handle:
        res = [torch.empty(i.shape, dtype=dtype, device=dev) for i in qs]
        arr = (MoMx4Image * len(qs))(*[i._struct() for i in qs])
        ptrs = (ctypes.c_void_p * len(qs))(*[t.data_ptr() for t in res])
        check(lib().mo_mx4_dequantize(arr, ptrs, len(qs), dt, handle))
    return res[0] if single else res


def mx4_matmul(a: Mx4Matrix, b: Mx4Matrix, *, out_dtype: torch.dtype = torch.bfloat16,
               out: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """``a b^T`` over the values of two images with equal columns
    (``mo_mx4_matmul``): a [M, K], b [N, K] give [M, N], fp32 sums rounded
    once.  ``out``: written instead of a new tensor (its dtype counts, rows
    may be strided); with ``accumulate`` the product is added to it."""
    if not isinstance(a, Mx4Matrix) or not isinstance(b, Mx4Matrix):
        raise TypeError("a and b must be Mx4Matrix")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    dt = _dtype_code(out_dtype if out is None else out.dtype, "out")
    used = [a.codes, a.scales, b.codes, b.scales, out]
    with _launch_on(a.device, stream, used) as handle:
        if out is None:
            out = torch.empty(a.rows, b.rows, dtype=out_dtype, device=a.device)
        ptr, r, c, ld = _rows_of(out, "out")
        if (r, c) != (a.rows, b.rows):
            raise ValueError(f"out must be [{a.rows}, {b.rows}], got [{r}, {c}]")
        sa, sb = a._struct(), b._struct()
        check(lib().mo_mx4_matmul(ctypes.byref(sa), ctypes.byref(sb), ptr, dt, ld, int(accumulate), handle))
    return out


def _flat2(x: torch.Tensor) -> torch.Tensor:
    return x if x.dim() == 2 else x.view(x.shape[:-1].numel(), x.shape[-1])


def mx4_linear(x: torch.Tensor, w: Mx4Matrix, *, out_dtype: torch.dtype = torch.bfloat16,
               save: bool = False, stream=None):
    """``y = x W^T`` with W [N, K] held in 4 bits and x [..., K] (fp32 or
    bf16) quantised on the way.  ``save=True`` also returns the image of x^T
    that :func:`mx4_linear_backward` takes (and needs one token at least).
    Not seen by autograd."""
    x2 = _flat2(x)
    if x2.shape[1] != w.cols:
        raise ValueError(f"x has {x2.shape[1]} features, the weights {w.cols}")
    if x2.shape[0] == 0 and not save:
        return torch.empty(*x.shape[:-1], w.rows, dtype=out_dtype, device=x.device)
    if save:
        xq, x_t = mx4_quantize(x2, images="both", stream=stream)
    else:
        xq = mx4_quantize(x2, stream=stream)
    y = mx4_matmul(xq, w, out_dtype=out_dtype, stream=stream)
    y = y if x.dim() == 2 else y.view(*x.shape[:-1], w.rows)
    return (y, x_t) if save else y


def mx4_linear_backward(dy: torch.Tensor, x_t: Mx4Matrix, w_t: Mx4Matrix, *,
                        dx_dtype: torch.dtype = torch.bfloat16, dw: Optional[torch.Tensor] = None,
                        accumulate: bool = False, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dW) of ``y = x W^T`` from dy [..., N] (fp32 or bf16), the image of
    x^T [K, tokens] and the image of W^T [K, N]: dy is quantised along both of
    its axes, dx = dy W contracts over N and dW = dy^T x over the tokens.  The
    rounding of x and W passes gradients straight through.  dW is fp32 [N, K]
    unless ``dw`` gives it; ``accumulate`` adds to ``dw``."""
    d2 = _flat2(dy)
    if d2.shape[0] != x_t.cols or d2.shape[1] != w_t.cols:
        raise ValueError(f"dy is {tuple(d2.shape)}, the images want [{x_t.cols}, {w_t.cols}]")
    if x_t.rows != w_t.rows:
        raise ValueError(f"x has {x_t.rows} features, the weights {w_t.rows}")
    if accumulate and dw is None:
        raise ValueError("accumulate needs dw")
    if dw is not None and tuple(dw.shape) != (w_t.cols, x_t.rows):
        raise ValueError(f"dw must be [{w_t.cols}, {x_t.rows}], got {tuple(dw.shape)}")
    dq, dq_t = mx4_quantize(d2, images="both", stream=stream)
    dx = mx4_matmul(dq, w_t, out_dtype=dx_dtype, stream=stream)
    dw = mx4_matmul(dq_t, x_t, out_dtype=torch.float32, out=dw, accumulate=accumulate, stream=stream)
    return dx if dy.dim() == 2 else dx.view(*dy.shape[:-1], w_t.rows), dw


# ---------------------------------------------------------------- 8-bit matrices
_I64x1, _I64x4, _I64x8 = ctypes.c_int64 * 1, ctypes.c_int64 * 4, ctypes.c_int64 * 8


class Fp8Matrix:
    """The 8-bit image of a [rows, cols] matrix with a scale per block of 128:
    ``codes`` uint8 [rows, 128 nb] (e4m3) and ``scales`` uint8 [rows, 16 ceil(nb
    / 16)] with nb = ceil(cols / 128) blocks per row, as ``include/muon.h`` lays
    them out.  Rows or columns may be none.  Both arrays, and those of a list's
    images, may share one allocation, which lives as long as any of them."""

    __slots__ = ("rows", "cols", "_keep", "_at", "_codes", "_scales", "_ptrs", "_image")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int):
        if codes.dim() != 2:
            raise ValueError("codes must be 2-D")
        rows, nb = int(codes.shape[0]), -(-int(cols) // 128)
        if cols < 0:
            raise ValueError("cols must not be negative")
        for t, w, what in ((codes, 128 * nb, "codes"), (scales, -(-nb // 16) * 16, "scales")):
            if t.dtype != torch.uint8 or tuple(t.shape) != (rows, w) or not t.is_contiguous():
                raise ValueError(f"{what} of a [{rows}, {cols}] image must be contiguous uint8 "
                                 f"[{rows}, {w}], got {t.dtype} {tuple(t.shape)}")
        if codes.device != scales.device:
            raise ValueError("codes and scales must share a device")
        self.rows, self.cols = rows, int(cols)
        self._keep, self._at, self._codes, self._scales = (codes, scales), None, codes, scales
        self._ptrs, self._image = (codes.data_ptr(), scales.data_ptr()), None

    # The arrays of an image that was made here are cut out of their allocation
    # when they are asked for: the operators only need their addresses.
    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            at, w = self._at, -(-self.cols // 128) * 128
            self._codes = self._keep[0][at:at + self.rows * w].view(self.rows, w)
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            nb = -(-self.cols // 128)
            at, w = self._at + self.rows * 128 * nb, -(-nb // 16) * 16
            self._scales = self._keep[0][at:at + self.rows * w].view(self.rows, w)
        return self._scales

    @property
    def shape(self) -> Tuple[int, int]:
        return self.rows, self.cols

    @property
    def device(self) -> torch.device:
        return self._keep[0].device

    @classmethod
    def empty(cls, rows: int, cols: int, device) -> "Fp8Matrix":
        """An image whose contents are still to be written."""
        if rows < 0 or cols < 0:
            raise ValueError(f"rows and columns must not be negative, got [{rows}, {cols}]")
        return cls._empty([(rows, cols)], device)[0]

    @classmethod
    def _empty(cls, shapes, device) -> List["Fp8Matrix"]:
        total, ats, sizes = 0, [], []
        for rows, cols in shapes:
            nb = -(-cols // 128)
            codes = rows * 128 * nb
            ats.append(total)
            sizes.append(codes)
            total += (codes + rows * (-(-nb // 16) * 16) + 255) & ~255
        buf = torch.empty(total, dtype=torch.uint8, device=device)
        base, keep, made = buf.data_ptr(), (buf,), []
        for (rows, cols), at, codes in zip(shapes, ats, sizes):
            q = object.__new__(cls)             # right by construction: no checks
            q.rows, q.cols, q._keep, q._at, q._codes, q._scales = rows, cols, keep, at, None, None
            q._ptrs, q._image = (base + at, base + at + codes), None
            made.append(q)
        return made

    # A copy's addresses are its own arrays': they are found again, not copied.
    def __copy__(self) -> "Fp8Matrix":
        return Fp8Matrix(self.codes, self.scales, self.cols)

    def __deepcopy__(self, memo) -> "Fp8Matrix":
        return Fp8Matrix(copy.deepcopy(self.codes, memo), copy.deepcopy(self.scales, memo), self.cols)

    def __reduce__(self):
        codes, scales = self.codes, self.scales
        if self._at is not None:                # out of an allocation that would be stored whole
            codes, scales = codes.clone(), scales.clone()
        return Fp8Matrix, (codes, scales, self.cols)

    def _struct(self):                          # mo_fp8_image
        if self._image is None:
            self._image = _I64x4(*self._ptrs, self.rows, self.cols)
        return self._image

    def __repr__(self) -> str:
        return f"Fp8Matrix([{self.rows}, {self.cols}], device={self.device})"


_NO_IMAGE = (0, 0)


def fp8_quantize(x: Union[torch.Tensor, Sequence[torch.Tensor]], *, images: str = "rows",
                 square: bool = False, out=None, stream=None):
    """8-bit images of a 2-D matrix or of a list of them (``mo_fp8_quantize``;
    fp32 or bf16, one dtype; rows may be strided).

    ``images``: "rows" -- the image of x (blocks of 128 along its rows); "cols"
    -- the image of x^T (blocks along x's columns); "both" -- the pair of them,
    from one reading of x.  ``square``: one scale for 128 x 128 elements, so
    that both images hold the same values -- for weights.  A list gives a list.
    ``out``: images of an earlier call (same form) to overwrite.
    """
    if images not in _IMAGES:
        raise ValueError(f"images must be one of {_IMAGES}")
    single = isinstance(x, torch.Tensor)
    if single and out is None:                   # the common call, with little beside its launch
        dt, view, dev = _dtype_code(x.dtype, "x"), _rows_of(x, "x"), x.device
        with _launch_on(dev, stream, (x,)) as handle:
            made = _fp8_images(view, dt, images, dev, handle, int(square))
        return tuple(made) if images == "both" else made[0]
    xs = [x] if single else list(x)
    if not xs:
        return []
    if not all(isinstance(t, torch.Tensor) for t in xs):
        raise TypeError("x must be a tensor or a list of tensors")
    if len(xs) == 1 and out is None:
        return [fp8_quantize(xs[0], images=images, square=square, stream=stream)]
    outs = None if out is None else ([out] if single else list(out))
    if outs is not None and len(outs) != len(xs):
        raise ValueError(f"out has {len(outs)} entries for {len(xs)} matrices")
    dt = _dtype_code(_common_dtype(xs, "x"), "x")
    dev = xs[0].device
    views = [_rows_of(t, "x") for t in xs]
    given, used = [], xs                         # images in the matrices' order, each one's then its transpose's
    if outs is not None:
        for (_, r, c, _), o in zip(views, outs):
            pair = tuple(o) if images == "both" else (o, None) if images == "rows" else (None, o)
            if len(pair) != 2:
                raise ValueError('out must hold pairs for images="both"')
            for q, shape in zip(pair, ((r, c), (c, r))):
                if q is not None and not isinstance(q, Fp8Matrix):
                    raise TypeError("out must hold Fp8Matrix")
                if q is not None and q.shape != shape:
                    raise ValueError(f"out: expected an image of {shape}, got {q.shape}")
            if (images != "cols" and pair[0] is None) or (images != "rows" and pair[1] is None):
                raise ValueError("out lacks an image")
            given += [q for q in pair if q is not None]
        used = xs + [t for q in given for t in q._keep]
    with _launch_on(dev, stream, used) as handle:
        if outs is None:
            shapes = []
            for _, r, c, _ in views:
                if images != "cols":
                    shapes.append((r, c))
                if images != "rows":
                    shapes.append((c, r))
            given = Fp8Matrix._empty(shapes, dev)
        flat = []                                # mo_fp8_item: src, codes, scales, codes_t, scales_t, rows, cols, ld
        step = 2 if images == "both" else 1
        for i, (ptr, r, c, ld) in enumerate(views):
            q = given[i * step]._ptrs
            if images == "both":
                flat += (ptr, *q, *given[i * step + 1]._ptrs, r, c, ld)
            elif images == "rows":
                flat += (ptr, *q, *_NO_IMAGE, r, c, ld)
            else:
                flat += (ptr, *_NO_IMAGE, *q, r, c, ld)
        check(lib().mo_fp8_quantize((ctypes.c_int64 * len(flat))(*flat), len(xs), dt, int(square), handle))
    res = list(zip(given[::2], given[1::2])) if images == "both" else given
    return res[0] if single else res


def fp8_dequantize(q: Union[Fp8Matrix, Sequence[Fp8Matrix]], *, dtype: torch.dtype = torch.bfloat16,
                   stream=None):
    """The values that an image, or each of a list, stands for (``mo_fp8_dequantize``)."""
    dt = _dtype_code(dtype, "dtype")
    if isinstance(q, Fp8Matrix):
        dev = q.device
        with _launch_on(dev, stream, q._keep) as handle:
            res = torch.empty((q.rows, q.cols), dtype=dtype, device=dev)
            check(lib().mo_fp8_dequantize(q._struct(), _I64x1(res.data_ptr()), 1, dt, handle))
        return res
    qs = list(q)
    if not qs:
        return []
    if not all(isinstance(i, Fp8Matrix) for i in qs):
        raise TypeError("q must be an Fp8Matrix or a list of them")
    if len(qs) == 1:
        return [fp8_dequantize(qs[0], dtype=dtype, stream=stream)]
    dev = qs[0].device
    with _launch_on(dev, stream, [t for i in qs for t in i._keep]) as handle:
        res = [torch.empty((i.rows, i.cols), dtype=dtype, device=dev) for i in qs]
        flat = [v for i in qs for v in (*i._ptrs, i.rows, i.cols)]         # mo_fp8_image
        ptrs = (ctypes.c_int64 * len(qs))(*[t.data_ptr() for t in res])
        check(lib().mo_fp8_dequantize((ctypes.c_int64 * len(flat))(*flat), ptrs, len(qs), dt, handle))
    return res


def fp8_matmul(a: Fp8Matrix, b: Fp8Matrix, *, out_dtype: torch.dtype = torch.bfloat16,
               out: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """``a b^T`` over the values of two images with equal columns
    (``mo_fp8_matmul``): a [M, K], b [N, K] give [M, N], fp32 sums rounded
    once; fp32 results from exact products, bf16 ones from the 8-bit matrix
    instruction, which cuts small products beside large ones (``include/muon.h``
    says where).  ``out``: written instead of a new tensor (its dtype counts,
    rows may be strided); with ``accumulate`` the product is added to it."""
    if not isinstance(a, Fp8Matrix) or not isinstance(b, Fp8Matrix):
        raise TypeError("a and b must be Fp8Matrix")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    dt = _dtype_code(out_dtype if out is None else out.dtype, "out")
    dev = a.device
    used = [*a._keep, *b._keep, out]
    with _launch_on(dev, stream, used) as handle:
        if out is None:
            out = torch.empty((a.rows, b.rows), dtype=out_dtype, device=dev)
            ptr, ld = out.data_ptr(), max(b.rows, 1)
        else:
            ptr, r, c, ld = _rows_of(out, "out")
            if (r, c) != (a.rows, b.rows):
                raise ValueError(f"out must be [{a.rows}, {b.rows}], got [{r}, {c}]")
        check(lib().mo_fp8_matmul(a._struct(), b._struct(), ptr, dt, ld, int(accumulate), handle))
    return out


def _fp8_images(view, dt: int, images: str, dev: torch.device, handle: int, square: int = 0) -> List[Fp8Matrix]:
    """Images of one matrix, inside a launch context."""
    ptr, r, c, ld = view
    if images == "both":
        made = Fp8Matrix._empty(((r, c), (c, r)), dev)
        item = _I64x8(ptr, *made[0]._ptrs, *made[1]._ptrs, r, c, ld)
    elif images == "rows":
        made = Fp8Matrix._empty(((r, c),), dev)
        item = _I64x8(ptr, *made[0]._ptrs, 0, 0, r, c, ld)
    else:
        made = Fp8Matrix._empty(((c, r),), dev)
        item = _I64x8(ptr, 0, 0, *made[0]._ptrs, r, c, ld)
    check(lib().mo_fp8_quantize(item, 1, dt, square, handle))
    return made


def _fp8_product(a: Fp8Matrix, b: Fp8Matrix, dtype: torch.dtype, dt: int, dev: torch.device, handle: int) -> torch.Tensor:
    out = torch.empty((a.rows, b.rows), dtype=dtype, device=dev)
    check(lib().mo_fp8_matmul(a._struct(), b._struct(), out.data_ptr(), dt, max(b.rows, 1), 0, handle))
    return out


def fp8_linear(x: torch.Tensor, w: Fp8Matrix, *, out_dtype: torch.dtype = torch.bfloat16,
               save: bool = False, stream=None):
    """``y = x W^T`` with W [N, K] held in 8 bits and x [..., K] (fp32 or
    bf16) quantised on the way, a scale per 128 of a row.  ``save=True`` also
    returns the image of x^T that :func:`fp8_linear_backward` takes.  x may
    have no tokens.  Not seen by autograd."""
    if not isinstance(w, Fp8Matrix):
        raise TypeError("w must be an Fp8Matrix")
    x2 = _flat2(x)
    view = _rows_of(x2, "x")
    if view[2] != w.cols:
        raise ValueError(f"x has {view[2]} features, the weights {w.cols}")
    x_dt, out_dt, dev = _dtype_code(x.dtype, "x"), _dtype_code(out_dtype, "out_dtype"), x.device
    with _launch_on(dev, stream, (x2, *w._keep)) as handle:     # one context for both launches
        images = _fp8_images(view, x_dt, "both" if save else "rows", dev, handle)
        y = _fp8_product(images[0], w, out_dtype, out_dt, dev, handle)
    y = y if x.dim() == 2 else y.view(*x.shape[:-1], w.rows)
    return (y, images[1]) if save else y


def fp8_linear_backward(dy: torch.Tensor, x_t: Fp8Matrix, w_t: Fp8Matrix, *,
                        dx_dtype: torch.dtype = torch.bfloat16, dw: Optional[torch.Tensor] = None,
                        accumulate: bool = False, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dW) of ``y = x W^T`` from dy [..., N] (fp32 or bf16), the image of
    x^T [K, tokens] and the image of W^T [K, N]: dy is quantised along both of
    its axes, dx = dy W contracts over N and dW = dy^T x over the tokens.  The
    rounding of x and W passes gradients straight through.  dW is fp32 [N, K]
    unless ``dw`` gives it; ``accumulate`` adds to ``dw``.  Without tokens dW
    is zeros (or stays as it was)."""
    if not isinstance(x_t, Fp8Matrix) or not isinstance(w_t, Fp8Matrix):
        raise TypeError("x_t and w_t must be Fp8Matrix")
    d2 = _flat2(dy)
    view = _rows_of(d2, "dy")
    if view[1] != x_t.cols or view[2] != w_t.cols:
        raise ValueError(f"dy is {tuple(d2.shape)}, the images want [{x_t.cols}, {w_t.cols}]")
    if x_t.rows != w_t.rows:
        raise ValueError(f"x has {x_t.rows} features, the weights {w_t.rows}")
    if accumulate and dw is None:
        raise ValueError("accumulate needs dw")
    if dw is not None and tuple(dw.shape) != (w_t.cols, x_t.rows):
        raise ValueError(f"dw must be [{w_t.cols}, {x_t.rows}], got {tuple(dw.shape)}")
    dy_dt, dx_dt, dev = _dtype_code(dy.dtype, "dy"), _dtype_code(dx_dtype, "dx_dtype"), dy.device
    dw_dt = MO_F32 if dw is None else _dtype_code(dw.dtype, "dw")
    dw_view = None if dw is None else _rows_of(dw, "dw")
    with _launch_on(dev, stream, (d2, *x_t._keep, *w_t._keep, dw)) as handle:
        dq, dq_t = _fp8_images(view, dy_dt, "both", dev, handle)
        dx = _fp8_product(dq, w_t, dx_dtype, dx_dt, dev, handle)
        if dw is None:
            dw = _fp8_product(dq_t, x_t, torch.float32, dw_dt, dev, handle)
        else:
            check(lib().mo_fp8_matmul(dq_t._struct(), x_t._struct(), dw_view[0], dw_dt, dw_view[3], int(accumulate), handle))
    return dx if dy.dim() == 2 else dx.view(*dy.shape[:-1], w_t.rows), dw


# ------------------------------------------------- log probabilities, distillation
class TokenLogprobs(NamedTuple):
    logprob: Optional[torch.Tensor]       # fp32 [rows], None without tokens
    entropy: torch.Tensor                 # fp32 [rows], nats
    top_logprob: torch.Tensor             # fp32 [rows, top]
    top_index: torch.Tensor               # int64 [rows, top]


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, *, top: int = 0,
                   temperature: float = 1.0, stream=None) -> TokenLogprobs:
    """Log probability of ``tokens`` (int64 [rows], negative: not scored, 0),
    entropy and the ``top`` likeliest columns of softmax(logits /
    temperature), logits fp32 or bf16 [rows, vocab] (``mo_token_logprobs``;
    rows may be strided)."""
    ptr, rows, vocab, ld = _rows_of(logits, "logits")
    dt, dev = _dtype_code(logits.dtype, "logits"), logits.device
    tok = _vector(tokens, torch.int64, (rows,), "tokens")
    need = _token_workspace("mo_token_logprobs_workspace_size", rows, vocab, top)
    with _launch_on(dev, stream, [logits, tokens]) as handle:
        lp = torch.empty(rows, dtype=torch.float32, device=dev) if tokens is not None else None
        ent = torch.empty(rows, dtype=torch.float32, device=dev)
        tlp = torch.empty(rows, top, dtype=torch.float32, device=dev)
        tix = torch.empty(rows, top, dtype=torch.int64, device=dev)
        if rows:
            with _SCRATCH_LOCK:
                ws = _scratch(need, handle, dev)
                check(lib().mo_token_logprobs(ptr, dt, rows, vocab, ld, tok, temperature,
                                              lp.data_ptr() if lp is not None else None, ent.data_ptr(), top,
                                              tix.data_ptr() if top else None, tlp.data_ptr() if top else None,
                                              ws.data_ptr() if ws is not None else None,
                                              ws.numel() if ws is not None else 0, handle))
    return TokenLogprobs(lp, ent, tlp, tix)


def distill_loss(logits: torch.Tensor, top_index: torch.Tensor, top_logit: torch.Tensor, *,
                 temperature: float = 1.0, grad_loss: Optional[torch.Tensor] = None, grad: bool = True,
                 out_grad: Optional[torch.Tensor] = None, stream=None):
    """Distillation from a teacher's top logits (``mo_distill_loss``): loss
    fp32 [rows] = temperature^2 KL(teacher's softmax over its slots ||
    softmax(logits / temperature)), and the gradient for ``logits`` [rows,
    vocab] (fp32 or bf16) in its dtype, (loss, None) with ``grad=False``.

    ``top_index`` int64 [rows, k] (negative: absent slot; a row without slots
    is skipped) and ``top_logit`` fp32 [rows, k] -- ``top_index`` and
    ``top_logprob`` of :func:`token_logprobs` on the teacher serve as they
    are.  ``grad_loss`` fp32 [rows]: the gradient that reaches each row's
    loss (1 when None).  ``out_grad``: written instead of a new tensor.  Not
    seen by autograd: pass the gradient on yourself."""
    ptr, rows, vocab, ld = _rows_of(logits, "logits")
    dt, dev = _dtype_code(logits.dtype, "logits"), logits.device
    if top_index.dim() != 2:
        raise ValueError("top_index must be [rows, k]")
    k = int(top_index.shape[1])
    ti = _vector(top_index, torch.int64, (rows, k), "top_index")
    tl = _vector(top_logit, torch.float32, (rows, k), "top_logit")
    gl = _vector(grad_loss, torch.float32, (rows,), "grad_loss")
    if out_grad is not None:
        if not grad:
            raise ValueError("out_grad given with grad=False")
        if out_grad.dtype != logits.dtype or tuple(out_grad.shape) != (rows, vocab):
            raise ValueError(f"out_grad must be {logits.dtype} [{rows}, {vocab}]")
    need = _token_workspace("mo_distill_loss_workspace_size", rows, vocab, k)
    with _launch_on(dev, stream, [logits, top_index, top_logit, grad_loss, out_grad]) as handle:
        loss = torch.empty(rows, dtype=torch.float32, device=dev)
        g = out_grad
        if grad and g is None:
            g = torch.empty(rows, vocab, dtype=logits.dtype, device=dev)
        gp, _, _, ldg = _rows_of(g, "out_grad") if grad else (None, 0, 0, 0)
        if rows:
            with _SCRATCH_LOCK:
                ws = _scratch(need, handle, dev)
                check(lib().mo_distill_loss(ptr, dt, rows, vocab, ld, ti, tl, k, temperature, gl,
                                            loss.data_ptr(), gp, ldg, ws.data_ptr() if ws is not None else None,
                                            ws.numel() if ws is not None else 0, handle))
    return loss, g


# ------------------------------------------------- cross entropy, router balance
_GRADS = (True, False, "x", "weight")


def linear_cross_entropy(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, *,
                         grad_loss: Optional[torch.Tensor] = None, grad: Union[bool, str] = True,
                         dw: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None):
    """Cross entropy of the logits ``x weight^T``, which the call does not
    leave behind (``mo_linear_ce``): (loss fp32 [rows], dx, dW).  x [..., hidden] and weight
    [vocab, hidden] are fp32 or bf16 (rows may be strided) and are multiplied
    in bf16; ``targets`` int64, one per row of x (negative: the row is skipped).

    ``grad_loss`` fp32 [rows]: the gradient that reaches each row's loss (1
    when None).  ``grad``: True for both gradients, "x" or "weight" for one,
    False for the loss alone; what is not asked for is None.  dx has x's dtype
    and shape, dW the weights' dtype unless ``dw`` [vocab, hidden] gives it;
    ``accumulate`` adds to ``dw``.  Not seen by autograd: pass the gradients on
    yourself.  For the time of the call, gradients take a workspace: copies of
    the operands, up to 1 GiB of the logits' gradient, and the logits in fp32
    where 4 GiB hold them (computed twice where not): 2.5 GB for 8192 rows of
    2048 and a vocabulary of 32000, more than the logits alone in bf16 (0.5 GB).
    The gradients are formed relative to the largest ``|grad_loss|``."""
    if grad not in _GRADS:
        raise ValueError(f"grad must be one of {_GRADS}")
    x2 = _flat2(x)
    xp, rows, hidden, ldx = _rows_of(x2, "x")
    wp, vocab, wh, ldw = _rows_of(weight, "weight")
    if hidden != wh:
        raise ValueError(f"x has {hidden} features, the weights {wh}")
    x_dt, w_dt, dev = _dtype_code(x.dtype, "x"), _dtype_code(weight.dtype, "weight"), x.device
    tp = _vector(targets.view(-1) if targets.is_contiguous() else targets, torch.int64, (rows,), "targets")
    gp = _vector(grad_loss, torch.float32, (rows,), "grad_loss")
    want_dx, want_dw = grad in (True, "x"), grad in (True, "weight")
    if dw is not None and not want_dw:
        raise ValueError(f"dw given with grad={grad!r}")
    if accumulate and dw is None:
        raise ValueError("accumulate needs dw")
    if dw is not None and tuple(dw.shape) != (vocab, hidden):
        raise ValueError(f"dw must be [{vocab}, {hidden}], got {tuple(dw.shape)}")
    dw_dt = w_dt if dw is None else _dtype_code(dw.dtype, "dw")
    need = _linear_ce_workspace(rows, hidden, vocab, x_dt, dw_dt, want_dx, want_dw)
    with _launch_on(dev, stream, [x2, weight, targets, grad_loss, dw]) as handle:
        loss = torch.empty(rows, dtype=torch.float32, device=dev)
        dx = torch.empty(rows, hidden, dtype=x.dtype, device=dev) if want_dx else None
        if want_dw and dw is None:
            dw = torch.empty(vocab, hidden, dtype=weight.dtype, device=dev)
        wgp, _, _, ld_dw = _rows_of(dw, "dw") if want_dw else (None, 0, 0, 0)
        # gigabytes for long calls: of this call alone, not kept for the next one
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        check(lib().mo_linear_ce(xp, x_dt, ldx, wp, w_dt, ldw, rows, hidden, vocab, tp, gp, loss.data_ptr(),
                                 dx.data_ptr() if want_dx else None, hidden, wgp, dw_dt, ld_dw, int(accumulate),
                                 ws.data_ptr() if need else None, need, handle))
    return loss, dx if dx is None or x.dim() == 2 else dx.view(x.shape), dw


@functools.lru_cache(maxsize=1024)
def _linear_ce_workspace(rows: int, hidden: int, vocab: int, x_dt: int, dw_dt: int, dx: bool, dw: bool) -> int:
    need = ctypes.c_size_t()
    check(lib().mo_linear_ce_workspace_size(rows, hidden, vocab, x_dt, dw_dt, int(dx), int(dw), ctypes.byref(need)))
    return need.value


class BalanceLoss(NamedTuple):
    loss: torch.Tensor                    # fp32, no dimensions
    counts: torch.Tensor                  # int64 [experts]
    grad: Optional[torch.Tensor]          # [tokens, experts] in the logits' dtype, None with grad=False


@functools.lru_cache(maxsize=1024)
def _balance_workspace(tokens: int, experts: int) -> int:
    need = ctypes.c_size_t()
    check(lib().mo_balance_loss_workspace_size(tokens, experts, ctypes.byref(need)))
    return need.value


def balance_loss(logits: torch.Tensor, index: torch.Tensor, *, weight: float = 1.0,
                 grad_loss: Optional[torch.Tensor] = None, grad: bool = True,
                 out_grad: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None) -> BalanceLoss:
    """Balance loss of a router (``mo_balance_loss``): ``weight`` times the sum
    over experts of f_e, their share of the choices times their number, and
    P_e, the mean of softmax(logits)_e over the tokens that made a choice.
    logits fp32 or bf16 [tokens, experts] (rows may be strided), ``index``
    int64 [tokens, top]: the experts that each token chose (negative: none; a
    token without any is skipped).  ``counts`` are the choices of each expert:
    the rows that its layers will see.

    ``grad_loss``: one fp32 value, the gradient that reaches the loss (1 when
    None).  The gradient is for the logits, in their dtype; ``out_grad`` is
    written instead of a new tensor, and with ``accumulate`` added to.  Not
    seen by autograd: pass the gradient on yourself."""
    ptr, tokens, experts, ld = _rows_of(logits, "logits")
    dt, dev = _dtype_code(logits.dtype, "logits"), logits.device
    if index.dim() != 2:
        raise ValueError("index must be [tokens, top]")
    top = int(index.shape[1])
    ip = _vector(index, torch.int64, (tokens, top), "index")
    if grad_loss is not None and (grad_loss.dtype != torch.float32 or grad_loss.numel() != 1):
        raise ValueError("grad_loss must be one float32 value")
    if out_grad is not None:
        if not grad:
            raise ValueError("out_grad given with grad=False")
        if out_grad.dtype != logits.dtype or tuple(out_grad.shape) != (tokens, experts):
            raise ValueError(f"out_grad must be {logits.dtype} [{tokens}, {experts}]")
    if accumulate and out_grad is None:
        raise ValueError("accumulate needs out_grad")
    need = _balance_workspace(tokens, experts)
    with _launch_on(dev, stream, [logits, index, grad_loss, out_grad]) as handle:
        loss = torch.empty((), dtype=torch.float32, device=dev)
        counts = torch.empty(experts, dtype=torch.int64, device=dev)
        g = out_grad
        if grad and g is None:
            g = torch.empty(tokens, experts, dtype=logits.dtype, device=dev)
        gp, _, _, ldg = _rows_of(g, "out_grad") if grad else (None, 0, 0, 0)
        with _SCRATCH_LOCK:
            ws = _scratch(need, handle, dev)
            check(lib().mo_balance_loss(ptr, dt, tokens, experts, ld, ip, top, weight,
                                        grad_loss.data_ptr() if grad_loss is not None else None, loss.data_ptr(),
                                        counts.data_ptr(), gp, ldg, int(accumulate),
                                        ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
                                        handle))
    return BalanceLoss(loss, counts, g)


def profile_enable(classes: Iterable[str] = ()) -> None:
    """Time every later launch of the named kernel classes with HIP events."""
    mask = 0
    for c in classes:
        mask |= 1 << KERNEL_CLASS_NAMES.index(c)
    check(lib().mo_profile_enable(mask))


def profile_read(cls: str) -> Tuple[int, float, float]:
    """(launches, total GPU ms, total algorithmic work) of a kernel class."""
    n, ms, w = ctypes.c_int64(), ctypes.c_double(), ctypes.c_double()
    check(lib().mo_profile_read(KERNEL_CLASS_NAMES.index(cls), ctypes.byref(n),
                                ctypes.byref(ms), ctypes.byref(w)))
    return n.value, ms.value, w.value


def profile_reset() -> None:
    check(lib().mo_profile_reset())


class MuonAdamW:
    """Optimizer front: 2-D parameters take the Muon step, everything else
    (RMSNorm gains, embeddings and LM head passed in ``adamw_params``) takes
    AdamW, with one shared learning rate and weight decay (section 2.2).

    State lives in torch tensors owned here (momentum per Muon matrix; m, v
    per AdamW tensor), so checkpointing is saving ``state_dict()``.

    ``mx4`` ("rows", "cols" or "both"): keep 4-bit images of the Muon
    matrices in ``self.mx4`` (as :func:`mx4_quantize` gives them, in the
    matrices' order), rewritten in place behind every step, so that 4-bit
    layers always multiply the current weights.  ``refresh_mx4()`` makes them
    before the first step, or after weights were loaded.  ``fp8`` keeps 8-bit
    images in ``self.fp8`` in the same way, with square scales
    (``refresh_fp8()``).
    """

    def __init__(self, muon_params: Sequence[torch.Tensor],
                 adamw_params: Sequence[torch.Tensor] = (), *, lr: float = 1e-3,
                 wd: float = 0.1, mu: float = 0.95, nesterov: bool = True,
                 ns_steps: int = 5, mom_dtype: torch.dtype = torch.bfloat16,
                 ns_dtype: torch.dtype = torch.bfloat16, betas=(0.9, 0.999),
                 adam_eps: float = 1e-8, mx4: Optional[str] = None, fp8: Optional[str] = None):
        if mx4 is not None and mx4 not in _IMAGES:
            raise ValueError(f"mx4 must be None or one of {_IMAGES}")
        if fp8 is not None and fp8 not in _IMAGES:
            raise ValueError(f"fp8 must be None or one of {_IMAGES}")
        self.muon_params: List[torch.Tensor] = list(muon_params)
        self.adamw_params: List[torch.Tensor] = list(adamw_params)
        for p in self.muon_params:
            if 0 in _shape2(p) and mx4 is not None:
                raise ValueError(f"an image has at least one row and one column, got {list(p.shape)}")
        self.lr, self.wd, self.mu, self.nesterov = lr, wd, mu, nesterov
        self.ns_steps, self.ns_dtype, self.betas, self.adam_eps = ns_steps, ns_dtype, betas, adam_eps
        self.momentum = [torch.zeros_like(p, dtype=mom_dtype) for p in self.muon_params]
        self.exp_avg = [torch.zeros_like(p, dtype=torch.float32) for p in self.adamw_params]
        self.exp_avg_sq = [torch.zeros_like(p, dtype=torch.float32) for p in self.adamw_params]
        self.t = 0
        self._plan: Optional[MuonPlan] = None
        self.plans_created = 0
        self._mx4_images = mx4
        self.mx4: Optional[list] = None
        self._fp8_images = fp8
        self.fp8: Optional[list] = None

    def refresh_mx4(self) -> list:
        """Rewrite the 4-bit images from the matrices as they are now."""
        if self._mx4_images is None:
            raise RuntimeError('MuonAdamW was made without mx4="rows", "cols" or "both"')
        self.mx4 = mx4_quantize([p.detach() for p in self.muon_params], images=self._mx4_images, out=self.mx4)
        return self.mx4

    def refresh_fp8(self) -> list:
        """Rewrite the 8-bit images from the matrices as they are now."""
        if self._fp8_images is None:
            raise RuntimeError('MuonAdamW was made without fp8="rows", "cols" or "both"')
        self.fp8 = fp8_quantize([p.detach() for p in self.muon_params], images=self._fp8_images, square=True,
                                out=self.fp8)
        return self.fp8

    def _grads(self, ps):
        gs = [p.grad for p in ps]
        if any(g is None for g in gs):
            raise RuntimeError("every parameter needs a gradient before step()")
        return gs

    def zero_grad(self, set_to_none: bool = True) -> None:
        """As ``torch.optim.Optimizer.zero_grad``: drop (or zero) every
        parameter's gradient."""
        for p in self.muon_params + self.adamw_params:
            if p.grad is None:
                continue
            if set_to_none:
                p.grad = None
            else:
                p.grad.zero_()

    def step(self, lr: Optional[float] = None, update_rms: Optional[torch.Tensor] = None) -> None:
        lr = self.lr if lr is None else lr
        self.t += 1
        if self.muon_params:
            gs = self._grads(self.muon_params)
            if self._plan is None:
                # the plan binds params and momenta once; gradients that move
                # between steps (zero_grad(set_to_none=True)) are rebound
                self._plan = MuonPlan(self.muon_params, gs, self.momentum, self.ns_dtype)
                self.plans_created += 1
            else:
                self._plan.set_grads(gs)
            self._plan.step(lr=lr, wd=self.wd, mu=self.mu, nesterov=self.nesterov,
                            ns_steps=self.ns_steps, update_rms=update_rms)
            self._plan.release_grads()
            if self._mx4_images is not None:
                self.refresh_mx4()
            if self._fp8_images is not None:
                self.refresh_fp8()
        if self.adamw_params:
            adamw_step(self.adamw_params, self._grads(self.adamw_params), self.exp_avg,
                       self.exp_avg_sq, lr=lr, step=self.t, wd=self.wd, beta1=self.betas[0],
                       beta2=self.betas[1], eps=self.adam_eps)

    def state_dict(self) -> dict:
        return {"t": self.t, "momentum": [m.clone() for m in self.momentum],
                "exp_avg": [m.clone() for m in self.exp_avg],
                "exp_avg_sq": [v.clone() for v in self.exp_avg_sq]}

    def load_state_dict(self, sd: dict) -> None:
        # checked in full before anything is copied
        for name in ("momentum", "exp_avg", "exp_avg_sq"):
            dst, src = getattr(self, name), sd[name]
            if len(src) != len(dst):
                raise ValueError(f"state_dict[{name!r}] has {len(src)} tensors, the optimizer {len(dst)}")
            for i, (d, t) in enumerate(zip(dst, src)):
                if tuple(t.shape) != tuple(d.shape):
                    raise ValueError(f"state_dict[{name!r}][{i}] has shape {tuple(t.shape)}, "
                                     f"expected {tuple(d.shape)}")
        self.t = int(sd["t"])
        for name in ("momentum", "exp_avg", "exp_avg_sq"):
            for d, t in zip(getattr(self, name), sd[name]):
                d.copy_(t)
