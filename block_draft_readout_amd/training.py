"""Training operators of the drafter's readout: the row normalisation in front of the
LM head, the cross entropy over the full vocabulary and the distillation from the
target's top logits, each forward and backward (``include/bdr.h``, last section).

The losses never store the logits: they take the hidden states and the LM head (and
the Markov head with the previous tokens, as the drafter drafts with them) and return
fp32 values per row; their backward calls recompute the logits a piece of the
vocabulary at a time.  Gradients come back in the tensors' dtype.
"""
from __future__ import annotations

import contextlib
from typing import Dict, Optional, Sequence, Tuple

import torch

from . import _abi
from ._abi import BDR_BF16, BDR_F32

__all__ = ["dspark_norm", "dspark_norm_backward", "dspark_ce_loss", "dspark_ce_backward",
           "dspark_distill_loss", "dspark_distill_backward"]

_DT = {torch.bfloat16: BDR_BF16, torch.float32: BDR_F32}
_NO_GUARD = contextlib.nullcontext()


def _tensor(t, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")


def _dtype(t: torch.Tensor, name: str) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype} of {name} (bfloat16 or float32)") from None


def _on(device: torch.device):
    """Makes `device` current for the call where it is not: kernels are launched on the
    current device, and its default stream has no handle of its own."""
    return _NO_GUARD if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _need(t: torch.Tensor, name: str, shape, dtype, device) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device: torch.device) -> int:
    """Handle of the device's current stream (torch.cuda.current_stream without the object,
    whose construction costs as much as a small kernel's launch)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _space(nbytes: int, device, ws: Optional[torch.Tensor]):
    """(aligned pointer, bytes, tensor) of a workspace; these calls keep no state in it.  A
    tensor that ends before the first aligned byte has no bytes (the C ABI's size is unsigned
    and takes one that is too small for the refusal)."""
    if ws is None:
        if nbytes == 0:
            return None, 0, None
        ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    elif not ws.is_contiguous() or ws.device != device:
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    p = ws.data_ptr()
    al = (p + 255) & ~255
    return al, max(0, ws.numel() * ws.element_size() - (al - p)), ws


# ----------------------------------------------------------------------------- row norm
def _rows(t: torch.Tensor, name: str) -> Tuple[torch.Tensor, int, int, int]:
    """[..., H] as (tensor, rows, H, row stride): contiguous, or 2-D with a unit last stride."""
    _tensor(t, name)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() < 1:
        raise ValueError(f"{name} must be [..., H]")
    h = t.shape[-1]
    rows = t.numel() // h if h else 0
    if t.is_contiguous():
        return t, rows, h, h
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= h:
        return t, rows, h, t.stride(0)
    raise ValueError(f"{name} must be contiguous, or 2-D with unit stride along H and rows apart")


def dspark_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                eps: float = 1e-6, rms: bool = False, stats: bool = False,
                out: Optional[torch.Tensor] = None):
    """y[..., H] = (x - mean) * rstd * weight + bias over the last axis (rms: mean = 0).

    stats=True returns (y, mean, rstd), fp32 [rows] each (mean is None with rms=True), as
    dspark_norm_backward takes them."""
    L = _abi.load()
    x, rows, h, stride = _rows(x, "x")
    dt = _dtype(x, "x")
    dev = x.device
    _need(weight, "weight", (h,), x.dtype, dev)
    if bias is not None:
        _need(bias, "bias", (h,), x.dtype, dev)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        _need(out, "out", x.shape, x.dtype, dev)
    st = torch.empty((1 if rms else 2, rows), dtype=torch.float32, device=dev)
    at = st.data_ptr()   # rstd, then the means
    with _on(dev):
        _abi.check("dspark_norm", L.dspark_norm(
            x.data_ptr(), rows, h, stride, dt, weight.data_ptr(), _ptr(bias), eps, out.data_ptr(),
            None if rms else at + 4 * rows, at, _stream(dev)))
    return (out, None if rms else st[1], st[0]) if stats else out


def dspark_norm_backward(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                         mean: Optional[torch.Tensor], rstd: torch.Tensor, *,
                         bias: bool = True, want_x: bool = True, want_weight: bool = True,
                         workspace: Optional[torch.Tensor] = None):
    """(dx, dweight, dbias) of dspark_norm for the gradient `grad` of its output; mean is
    None for the root-mean-square form.  bias=False: no bias gradient (None);
    want_x / want_weight=False likewise."""
    L = _abi.load()
    _tensor(grad, "grad")
    x, rows, h, xs = _rows(x, "x")
    dt = _dtype(x, "x")
    dev = x.device
    if grad.shape != x.shape or grad.dtype != x.dtype or grad.device != dev:
        raise ValueError("grad must have x's shape, dtype and device")
    grad, _, _, gs = _rows(grad, "grad")
    _need(weight, "weight", (h,), x.dtype, dev)
    _need(rstd, "rstd", (rows,), torch.float32, dev)
    if mean is not None:
        _need(mean, "mean", (rows,), torch.float32, dev)
    dx = torch.empty_like(x, memory_format=torch.contiguous_format) if want_x else None
    dw = torch.empty(h, dtype=x.dtype, device=dev) if want_weight else None
    db = torch.empty(h, dtype=x.dtype, device=dev) if bias else None
    need = L.dspark_norm_backward_workspace_bytes(rows, h) if want_weight or bias else 0
    wp, wn, _keep = _space(need, dev, workspace)
    with _on(dev):
        _abi.check("dspark_norm_backward", L.dspark_norm_backward(
            grad.data_ptr(), gs, x.data_ptr(), xs, rows, h, dt, weight.data_ptr(), _ptr(mean),
            rstd.data_ptr(), _ptr(dx), _ptr(dw), _ptr(db), wp, wn, _stream(dev)))
    return dx, dw, db


# ----------------------------------------------------------------------------- losses
class _Readout:
    """Checked arguments that every loss call shares."""

    def __init__(self, hidden, lm_head_w, markov_w1, markov_w2, prev_token, teacher=()):
        _tensor(hidden, "hidden")
        _tensor(lm_head_w, "lm_head_w")   # (a PackedWeight is none)
        if markov_w1 is not None:
            _tensor(markov_w1, "markov_w1")
        for name, t in zip(("teacher_ids", "teacher_logits"), teacher):
            _tensor(t, name)
        if not hidden.is_cuda:
            raise ValueError("hidden must be a device tensor")
        if hidden.dim() < 1 or lm_head_w.dim() != 2:
            raise ValueError("hidden must be [..., H] and lm_head_w [V, H]")
        if not hidden.is_contiguous():
            raise ValueError("hidden must be contiguous")
        self.device = dev = hidden.device
        self.dt = _dtype(hidden, "hidden")
        self.vocab, self.h = lm_head_w.shape
        _need(lm_head_w, "lm_head_w", (self.vocab, self.h), hidden.dtype, dev)
        if hidden.shape[-1] != self.h:
            raise ValueError(f"hidden must be [..., {self.h}]")
        self.lead = tuple(hidden.shape[:-1])
        self.rows = hidden.numel() // self.h if self.h else 0
        self.rank = 0
        if (markov_w1 is None) != (markov_w2 is None):
            raise ValueError("markov_w1 and markov_w2 must both be given or both be None")
        if markov_w1 is not None:
            if markov_w1.dim() != 2:
                raise ValueError("markov_w1 must be [V, r]")
            self.rank = markov_w1.shape[1]
            for name, w in (("markov_w1", markov_w1), ("markov_w2", markov_w2)):
                _need(w, name, (self.vocab, self.rank), hidden.dtype, dev)
            if prev_token is None:
                raise ValueError("prev_token is needed with a Markov head")
            _need(prev_token, "prev_token", self.lead, torch.int32, dev)
        self.args = (hidden.data_ptr(), self.rows, self.h, self.vocab, self.dt,
                     lm_head_w.data_ptr(), _ptr(markov_w1), _ptr(markov_w2), self.rank,
                     _ptr(prev_token) if self.rank else None)
        self.dtype = hidden.dtype

    def per_row(self, t, name, dtype, tail=()):
        return _need(t, name, self.lead + tail, dtype, self.device)

    def new_rows(self, *tail):
        return torch.empty(self.lead + tail, dtype=torch.float32, device=self.device)

    def stream(self):
        return _stream(self.device)

    def gradients(self, names: Optional[Sequence[str]]) -> Dict[str, torch.Tensor]:
        shapes = {"hidden": self.lead + (self.h,), "lm_head_w": (self.vocab, self.h)}
        if self.rank:
            shapes["markov_w1"] = shapes["markov_w2"] = (self.vocab, self.rank)
        if names is None:
            names = tuple(shapes)
        for n in names:
            if n not in shapes:
                raise ValueError(f"unknown gradient {n!r}: one of {', '.join(shapes)}")
        return {n: torch.empty(shapes[n], dtype=self.dtype, device=self.device) for n in names}


def _grad_ptrs(grads):
    return tuple(_ptr(grads.get(n)) for n in ("hidden", "lm_head_w", "markov_w1", "markov_w2"))


def dspark_ce_loss(hidden: torch.Tensor, lm_head_w: torch.Tensor, labels: torch.Tensor,
                   markov_w1: Optional[torch.Tensor] = None,
                   markov_w2: Optional[torch.Tensor] = None,
                   prev_token: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """(loss [...], lse [...]) fp32: cross entropy of hidden[..., H] @ lm_head_w[V, H]^T (plus
    the Markov bias of prev_token [...] int32) against labels [...] int32.  A label outside
    [0, V) leaves its row out (loss and lse 0)."""
    L = _abi.load()
    r = _Readout(hidden, lm_head_w, markov_w1, markov_w2, prev_token)
    r.per_row(labels, "labels", torch.int32)
    loss, lse = r.new_rows(), r.new_rows()
    wp, wn, _keep = _space(L.dspark_ce_workspace_bytes(r.rows, r.h, r.vocab, r.rank, r.dt, 0),
                           r.device, workspace)
    with _on(r.device):
        _abi.check("dspark_ce_loss", L.dspark_ce_loss(
            *r.args, labels.data_ptr(), loss.data_ptr(), lse.data_ptr(), wp, wn, r.stream()))
    return loss, lse


def dspark_ce_backward(hidden: torch.Tensor, lm_head_w: torch.Tensor, labels: torch.Tensor,
                       lse: torch.Tensor, loss_grad: torch.Tensor,
                       markov_w1: Optional[torch.Tensor] = None,
                       markov_w2: Optional[torch.Tensor] = None,
                       prev_token: Optional[torch.Tensor] = None,
                       grads: Optional[Sequence[str]] = None,
                       workspace: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Gradients of sum(loss_grad * loss) for the loss and lse of dspark_ce_loss on the same
    inputs: a dict with the wanted ones of hidden, lm_head_w, markov_w1, markov_w2 (default:
    all), each in the tensors' dtype."""
    L = _abi.load()
    r = _Readout(hidden, lm_head_w, markov_w1, markov_w2, prev_token)
    r.per_row(labels, "labels", torch.int32)
    r.per_row(lse, "lse", torch.float32)
    r.per_row(loss_grad, "loss_grad", torch.float32)
    out = r.gradients(grads)
    wp, wn, _keep = _space(L.dspark_ce_workspace_bytes(r.rows, r.h, r.vocab, r.rank, r.dt, 1),
                           r.device, workspace)
    with _on(r.device):
        _abi.check("dspark_ce_backward", L.dspark_ce_backward(
            *r.args, labels.data_ptr(), lse.data_ptr(), loss_grad.data_ptr(), *_grad_ptrs(out), wp,
            wn, r.stream()))
    return out


def _teacher(r: _Readout, ids: torch.Tensor, logits: torch.Tensor):
    if ids.dim() != len(r.lead) + 1:
        raise ValueError("teacher_ids must be [..., top]")
    top = ids.shape[-1]
    r.per_row(ids, "teacher_ids", torch.int32, (top,))
    tdt = _dtype(logits, "teacher_logits")
    r.per_row(logits, "teacher_logits", logits.dtype, (top,))
    return top, (ids.data_ptr(), logits.data_ptr(), top, tdt)


def dspark_distill_loss(hidden: torch.Tensor, lm_head_w: torch.Tensor, teacher_ids: torch.Tensor,
                        teacher_logits: torch.Tensor, markov_w1: Optional[torch.Tensor] = None,
                        markov_w2: Optional[torch.Tensor] = None,
                        prev_token: Optional[torch.Tensor] = None, temperature: float = 1.0,
                        workspace: Optional[torch.Tensor] = None):
    """(loss [...], lse [...], picked [..., top]) fp32: T^2 times the divergence of the drafter's
    softmax over the vocabulary from the target's over its listed entries, teacher_ids
    [..., top] int32 and teacher_logits [..., top] fp32 or bf16, at temperature T.  An id
    outside [0, V) is not listed; a row without listed mass is left out (loss and lse 0)."""
    L = _abi.load()
    r = _Readout(hidden, lm_head_w, markov_w1, markov_w2, prev_token, (teacher_ids, teacher_logits))
    top, targs = _teacher(r, teacher_ids, teacher_logits)
    loss, lse, picked = r.new_rows(), r.new_rows(), r.new_rows(top)
    wp, wn, _keep = _space(
        L.dspark_distill_workspace_bytes(r.rows, r.h, r.vocab, r.rank, top, r.dt, 0), r.device,
        workspace)
    with _on(r.device):
        _abi.check("dspark_distill_loss", L.dspark_distill_loss(
            *r.args, *targs, temperature, loss.data_ptr(), lse.data_ptr(), picked.data_ptr(), wp, wn,
            r.stream()))
    return loss, lse, picked


def dspark_distill_backward(hidden: torch.Tensor, lm_head_w: torch.Tensor,
                            teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                            lse: torch.Tensor, picked: torch.Tensor, loss_grad: torch.Tensor,
                            markov_w1: Optional[torch.Tensor] = None,
                            markov_w2: Optional[torch.Tensor] = None,
                            prev_token: Optional[torch.Tensor] = None, temperature: float = 1.0,
                            grads: Optional[Sequence[str]] = None,
                            workspace: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Gradients of sum(loss_grad * loss) for the loss, lse and picked of dspark_distill_loss on
    the same inputs, as dspark_ce_backward returns them."""
    L = _abi.load()
    r = _Readout(hidden, lm_head_w, markov_w1, markov_w2, prev_token, (teacher_ids, teacher_logits))
    top, targs = _teacher(r, teacher_ids, teacher_logits)
    r.per_row(lse, "lse", torch.float32)
    r.per_row(picked, "picked", torch.float32, (top,))
    r.per_row(loss_grad, "loss_grad", torch.float32)
    out = r.gradients(grads)
    wp, wn, _keep = _space(
        L.dspark_distill_workspace_bytes(r.rows, r.h, r.vocab, r.rank, top, r.dt, 1), r.device,
        workspace)
    with _on(r.device):
        _abi.check("dspark_distill_backward", L.dspark_distill_backward(
            *r.args, *targs, temperature, lse.data_ptr(), picked.data_ptr(), loss_grad.data_ptr(),
            *_grad_ptrs(out), wp, wn, r.stream()))
    return out
