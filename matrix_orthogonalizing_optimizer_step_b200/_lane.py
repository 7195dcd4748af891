"""Binding of the AdamW lane's layers: token embedding, LayerNorm and output
head with its loss, and the gradients that the lane's step reads.

Like the rest of the binding these functions check and marshal arguments; the
arithmetic runs in the library's kernels.  Outputs and workspaces are torch
allocations on the current stream, so the calls can be captured into a CUDA
graph (each graph then has workspaces of its own) and several streams may use
them at once.  All tensors of a call must be on one device, which need not be
the current one; tensors made on another stream need that stream's work
ordered before the call, as for any torch operator.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import MuonError, _check, lib
from ._lib import MUON_DTYPE_BF16, MUON_DTYPE_F32, MUON_INDEX_I32, MUON_INDEX_I64

_DTYPE = {torch.bfloat16: MUON_DTYPE_BF16, torch.float32: MUON_DTYPE_F32}
_INDEX = {torch.int32: MUON_INDEX_I32, torch.int64: MUON_INDEX_I64}

# The bound stream is the library's; autograd runs backward passes of several
# devices on threads of their own, so binding and call are one step.
_lock = threading.RLock()


def _call(fn, device, *args):
    """fn(*args) on the current stream of `device`, with `device` current."""
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _call(fn, device, *args)
    L = lib()
    with _lock:
        L.muon_set_stream(torch.cuda.current_stream(index).cuda_stream)
        rc = getattr(L, fn)(*args)
        if rc:
            _check(rc)


def _workspace(fn, device, *args):
    """Scratch of the bytes that the library's query `fn` asks for."""
    n = getattr(lib(), fn)(*args)
    if n < 0:
        raise MuonError(n, lib().muon_last_error().decode(errors="replace"))
    return torch.empty(n, dtype=torch.uint8, device=device), n


def _dtype(t, name):
    if t.dtype not in _DTYPE:
        raise ValueError(f"{name} must be bfloat16 or float32")
    return _DTYPE[t.dtype]


def _same_device(first, *rest):
    if not first.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    for t in rest:
        if t is not None and t.device != first.device:
            raise ValueError("tensors must be on one device")


def _index(t, name):
    if t.dtype not in _INDEX:
        raise ValueError(f"{name} must be int32 or int64")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _INDEX[t.dtype]


def _rows(t, name):
    """(tensor, rows, dim, row stride) of t seen as rows of its last dimension."""
    if t.dim() == 0:
        raise ValueError(f"{name} must have at least one dimension")
    dim = t.shape[-1]
    if dim == 0:
        raise ValueError(f"{name} must not have an empty last dimension")
    if t.is_contiguous():
        return t, t.numel() // dim, dim, dim
    if t.dim() != 2:
        try:
            t = t.view(-1, dim)
        except RuntimeError:
            raise ValueError(f"{name} must be viewable as rows of one stride") from None
    rows = t.shape[0]
    if t.stride(1) != 1 and dim > 1 or rows > 1 and t.stride(0) < dim:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t, rows, dim, t.stride(0) if rows > 1 else dim


def _contiguous_2d(t, name):
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D tensor")
    if t.numel() == 0:
        raise ValueError(f"{name} must not be empty")


def _vector(t, name, n, dtype=None):
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} elements")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")


def muon_embedding(tokens, table, scale=1.0, out_dtype=None):
    """scale * table[tokens]: tokens int32 or int64 of any shape, table (vocab,
    dim) bf16 or fp32; the result has tokens' shape with dim appended, in
    out_dtype (default: the table's).  Rows of tokens outside the vocabulary
    are NaN (muon_device_status reports them)."""
    _contiguous_2d(table, "table")
    it = _index(tokens, "tokens")
    td = _dtype(table, "table")
    _same_device(table, tokens)
    out = torch.empty(*tokens.shape, table.shape[1], dtype=out_dtype or table.dtype, device=table.device)
    od = _dtype(out, "out_dtype")
    n = tokens.numel()
    if n:
        _call("muon_embedding", table.device, tokens.data_ptr(), it, n, table.data_ptr(), td, table.shape[0],
              table.shape[1], float(scale), out.data_ptr(), od)
    return out


def muon_embedding_backward(tokens, grad_out, num_embeddings, scale=1.0, padding_idx=None, grad_dtype=None, out=None):
    """Gradient of the table of muon_embedding: (num_embeddings, dim) in
    grad_dtype (default: grad_out's), dense, rows of unused tokens and of
    padding_idx zero.  grad_out: tokens.numel() rows.  out: the contiguous
    tensor to write instead of a new one."""
    it = _index(tokens, "tokens")
    gd = _dtype(grad_out, "grad_out")
    grad_out, rows, dim, ld = _rows(grad_out, "grad_out")
    n, vocab = tokens.numel(), int(num_embeddings)
    if rows != n:
        raise ValueError("grad_out must have one row per token")
    if vocab < 1:
        raise ValueError("num_embeddings must be >= 1")
    if padding_idx is not None and not 0 <= padding_idx < vocab:
        raise ValueError("padding_idx must be a token")
    if out is None:
        out = torch.empty(vocab, dim, dtype=grad_dtype or grad_out.dtype, device=grad_out.device)
    else:
        _contiguous_2d(out, "out")
        if tuple(out.shape) != (vocab, dim) or grad_dtype not in (None, out.dtype):
            raise ValueError("out must have shape (num_embeddings, dim) and grad_dtype")
    od = _dtype(out, "grad_dtype")
    _same_device(grad_out, tokens, out)
    ws, nb = _workspace("muon_embedding_backward_workspace", grad_out.device, n, vocab, dim)
    _call("muon_embedding_backward", grad_out.device, tokens.data_ptr(), it, n, grad_out.data_ptr(), gd, ld, vocab, dim,
          float(scale), -1 if padding_idx is None else int(padding_idx), out.data_ptr(), od, ws.data_ptr(), nb)
    return out


def _norm_params(x, dim, weight, bias):
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _vector(t, name, dim)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias must have one dtype")
    _same_device(x, weight, bias)
    p = weight if weight is not None else bias
    return MUON_DTYPE_F32 if p is None else _dtype(p, "weight and bias")


def _ptr(t):
    return None if t is None else t.data_ptr()


def muon_layer_norm(x, weight=None, bias=None, eps=1e-5):
    """LayerNorm over x's last dimension: (y, mean, rstd).  x bf16 or fp32 with
    contiguous rows; weight and bias bf16 or fp32.  y is contiguous in x's
    dtype; mean and rstd are fp32, one per row, for the backward pass."""
    xd = _dtype(x, "x")
    shape = x.shape
    x, rows, dim, ld = _rows(x, "x")
    pd = _norm_params(x, dim, weight, bias)
    y = torch.empty(shape, dtype=x.dtype, device=x.device)
    mean, rstd = torch.empty(2, *shape[:-1], dtype=torch.float32, device=x.device).unbind(0)
    if rows:
        _call("muon_layer_norm", x.device, x.data_ptr(), xd, ld, rows, dim, _ptr(weight), _ptr(bias), pd, float(eps),
              y.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    return y, mean, rstd


def muon_layer_norm_backward(grad_out, x, mean, rstd, weight=None, bias=True, param_dtype=None):
    """Gradients of muon_layer_norm: (dx, dweight, dbias) in x's dtype and in
    the weight's (without a weight: param_dtype, default fp32).  dweight is
    None without a weight, dbias None with bias=False."""
    xd = _dtype(x, "x")
    shape = x.shape
    if grad_out.shape != shape or grad_out.dtype != x.dtype:
        raise ValueError("grad_out must have x's shape and dtype")
    x, rows, dim, ldx = _rows(x, "x")
    grad_out, _, _, ldg = _rows(grad_out, "grad_out")
    _vector(mean, "mean", rows, torch.float32)
    _vector(rstd, "rstd", rows, torch.float32)
    pd = _norm_params(x, dim, weight, None)
    _same_device(x, grad_out, mean, rstd)
    if weight is not None:
        pt = weight.dtype
        if param_dtype not in (None, pt):
            raise ValueError("param_dtype must be the weight's dtype")
    else:
        pt = param_dtype or torch.float32
        if pt not in _DTYPE:
            raise ValueError("param_dtype must be bfloat16 or float32")
        pd = _DTYPE[pt]
    dx = torch.empty(shape, dtype=x.dtype, device=x.device)
    dw = torch.empty(dim, dtype=pt, device=x.device) if weight is not None else None
    db = torch.empty(dim, dtype=pt, device=x.device) if bias else None
    ws, nb = _workspace("muon_layer_norm_backward_workspace", x.device, rows, dim)
    _call("muon_layer_norm_backward", x.device, grad_out.data_ptr(), ldg, x.data_ptr(), xd, ldx, rows, dim,
          mean.data_ptr(), rstd.data_ptr(), _ptr(weight), pd, dx.data_ptr(), _ptr(dw), _ptr(db), ws.data_ptr(), nb)
    return dx, dw, db


def _head(hidden, weight, targets):
    _contiguous_2d(weight, "weight")
    if hidden.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise ValueError("hidden and weight must be bfloat16")
    it = _index(targets, "targets")
    hidden, rows, dim, ld = _rows(hidden, "hidden")
    if dim != weight.shape[1]:
        raise ValueError("hidden and weight must have one width")
    if dim % 8 or ld % 8:
        raise ValueError("the width and hidden's row stride must be multiples of 8")
    if targets.numel() != rows:
        raise ValueError("targets must have one entry per row of hidden")
    _same_device(weight, hidden, targets)
    for t, name in ((hidden, "hidden"), (weight, "weight")):
        if t.data_ptr() % 16:
            raise ValueError(f"{name} must be 16-byte aligned")
    return hidden, rows, dim, ld, it


def muon_head_loss(hidden, weight, targets, ignore_index=-100):
    """(loss, lse) per token of the softmax cross entropy of hidden . weight^T:
    hidden (..., dim) and weight (vocab, dim) bf16 with dim a multiple of 8,
    targets int32 or int64.  Both results are fp32 in targets' shape, 0 for
    tokens whose target is ignore_index; the logits are not kept."""
    hidden, rows, dim, ld, it = _head(hidden, weight, targets)
    loss, lse = torch.empty(2, *targets.shape, dtype=torch.float32, device=weight.device).unbind(0)
    if rows:
        vocab = weight.shape[0]
        ws, nb = _workspace("muon_head_loss_workspace", weight.device, rows, vocab, dim, 0)
        _call("muon_head_loss", weight.device, hidden.data_ptr(), ld, weight.data_ptr(), targets.data_ptr(), it, rows,
              vocab, dim, int(ignore_index), loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), nb)
    return loss, lse


def muon_head_loss_backward(hidden, weight, targets, lse, grad_loss, ignore_index=-100, hidden_grad=True,
                            weight_grad=True):
    """(dhidden, dweight), bf16, from the lse of muon_head_loss and the fp32
    gradient of its per-token loss.  Either can be left out (None)."""
    shape = hidden.shape
    hidden, rows, dim, ld, it = _head(hidden, weight, targets)
    _vector(lse, "lse", rows, torch.float32)
    _vector(grad_loss, "grad_loss", rows, torch.float32)
    _same_device(weight, lse, grad_loss)
    if not (hidden_grad or weight_grad):
        raise ValueError("one gradient at least")
    vocab = weight.shape[0]
    dh = torch.empty(shape, dtype=torch.bfloat16, device=weight.device) if hidden_grad else None
    dw = torch.empty_like(weight) if weight_grad else None
    ws, nb = _workspace("muon_head_loss_workspace", weight.device, rows, vocab, dim, 1)
    if rows or weight_grad:
        _call("muon_head_loss_backward", weight.device, hidden.data_ptr(), ld, weight.data_ptr(), targets.data_ptr(), it,
              rows, vocab, dim, int(ignore_index), lse.data_ptr(), grad_loss.data_ptr(), _ptr(dh), _ptr(dw),
              ws.data_ptr(), nb)
    return dh, dw
