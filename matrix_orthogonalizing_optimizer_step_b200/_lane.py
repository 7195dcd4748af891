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

import functools
import threading

import torch

from . import MuonError, _check, lib
from ._lib import MUON_DTYPE_BF16, MUON_DTYPE_F32, MUON_INDEX_I32, MUON_INDEX_I64

_DTYPE = {torch.bfloat16: MUON_DTYPE_BF16, torch.float32: MUON_DTYPE_F32}
_INDEX = {torch.int32: MUON_INDEX_I32, torch.int64: MUON_INDEX_I64}

# The bound stream is the library's; autograd runs backward passes of several
# devices on threads of their own, so binding and call are one step.
_lock = threading.Lock()
_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without a Stream object


def _call(name, index, *args):
    """One call of the library on the current stream of device `index`, with
    that device current."""
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _call(name, index, *args)
    L = lib()
    with _lock:
        L.muon_set_stream(_raw_stream(index))
        rc = getattr(L, name)(*args)
        if rc:
            _check(rc)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name, *sizes):
    n = getattr(lib(), name)(*sizes)
    if n < 0:
        raise MuonError(n, lib().muon_last_error().decode(errors="replace"))
    return n


def _workspace(name, device, *sizes):
    """Scratch of the bytes that the library's query `name` asks for."""
    n = _workspace_bytes(name, *sizes)
    return torch.empty(n, dtype=torch.uint8, device=device), n


def _dtype(dtype, name):
    code = _DTYPE.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float32")
    return code


def _same_device(first, *rest):
    """The device index that all tensors share."""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must be CUDA tensors")
    for t in rest:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must be on one device")
    return index


def _index(t, name):
    code = _INDEX.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be int32 or int64")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return code


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
    vocab, dim = table.shape
    td = _dtype(table.dtype, "table")
    od = td if out_dtype is None else _dtype(out_dtype, "out_dtype")
    index = _same_device(table, tokens)
    n = tokens.numel()
    out = table.new_empty((*tokens.shape, dim), dtype=out_dtype)
    if n:
        _call("muon_embedding", index, tokens.data_ptr(), it, n, table.data_ptr(), td, vocab, dim, scale,
              out.data_ptr(), od)
    return out


def muon_embedding_backward(tokens, grad_out, num_embeddings, scale=1.0, padding_idx=None, grad_dtype=None, out=None):
    """Gradient of the table of muon_embedding: (num_embeddings, dim) in
    grad_dtype (default: grad_out's), dense, rows of unused tokens and of
    padding_idx zero.  grad_out: tokens.numel() rows.  out: the contiguous
    tensor to write instead of a new one."""
    it = _index(tokens, "tokens")
    gd = _dtype(grad_out.dtype, "grad_out")
    grad_out, rows, dim, ld = _rows(grad_out, "grad_out")
    n, vocab = tokens.numel(), int(num_embeddings)
    if rows != n:
        raise ValueError("grad_out must have one row per token")
    if vocab < 1:
        raise ValueError("num_embeddings must be >= 1")
    if padding_idx is not None and not 0 <= padding_idx < vocab:
        raise ValueError("padding_idx must be a token")
    index = _same_device(grad_out, tokens, out)
    if out is None:
        od = gd if grad_dtype is None else _dtype(grad_dtype, "grad_dtype")
        out = grad_out.new_empty((vocab, dim), dtype=grad_dtype)
    else:
        od = _dtype(out.dtype, "out")
        _contiguous_2d(out, "out")
        if out.shape != (vocab, dim) or grad_dtype not in (None, out.dtype):
            raise ValueError("out must have shape (num_embeddings, dim) and grad_dtype")
    ws, nb = _workspace("muon_embedding_backward_workspace", grad_out.device, n, vocab, dim)
    _call("muon_embedding_backward", index, tokens.data_ptr(), it, n, grad_out.data_ptr(), gd, ld, vocab, dim, scale,
          -1 if padding_idx is None else padding_idx, out.data_ptr(), od, ws.data_ptr(), nb)
    return out


def _norm_params(x, dim, weight, bias):
    """(device index, type code of the parameters)."""
    if weight is not None:
        _vector(weight, "weight", dim)
    if bias is not None:
        _vector(bias, "bias", dim)
        if weight is not None and weight.dtype != bias.dtype:
            raise ValueError("weight and bias must have one dtype")
    p = weight if weight is not None else bias
    return _same_device(x, weight, bias), MUON_DTYPE_F32 if p is None else _dtype(p.dtype, "weight and bias")


def _ptr(t):
    return None if t is None else t.data_ptr()


def muon_layer_norm(x, weight=None, bias=None, eps=1e-5):
    """LayerNorm over x's last dimension: (y, mean, rstd).  x bf16 or fp32 with
    contiguous rows; weight and bias bf16 or fp32.  y is contiguous in x's
    dtype; mean and rstd are fp32, one per row, for the backward pass."""
    xd = _dtype(x.dtype, "x")
    shape = x.shape
    x, rows, dim, ld = _rows(x, "x")
    index, pd = _norm_params(x, dim, weight, bias)
    y = x.new_empty(shape)
    mean = x.new_empty(shape[:-1], dtype=torch.float32)
    rstd = torch.empty_like(mean)
    if rows:
        _call("muon_layer_norm", index, x.data_ptr(), xd, ld, rows, dim, _ptr(weight), _ptr(bias), pd, eps,
              y.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    return y, mean, rstd


def muon_layer_norm_backward(grad_out, x, mean, rstd, weight=None, bias=True, param_dtype=None):
    """Gradients of muon_layer_norm: (dx, dweight, dbias) in x's dtype and in
    the weight's (without a weight: param_dtype, default fp32).  dweight is
    None without a weight, dbias None with bias=False."""
    xd = _dtype(x.dtype, "x")
    shape = x.shape
    if grad_out.shape != shape or grad_out.dtype != x.dtype:
        raise ValueError("grad_out must have x's shape and dtype")
    x, rows, dim, ldx = _rows(x, "x")
    grad_out, _, _, ldg = _rows(grad_out, "grad_out")
    _vector(mean, "mean", rows, torch.float32)
    _vector(rstd, "rstd", rows, torch.float32)
    _, pd = _norm_params(x, dim, weight, None)
    index = _same_device(x, grad_out, mean, rstd)
    if weight is not None:
        pt = weight.dtype
        if param_dtype not in (None, pt):
            raise ValueError("param_dtype must be the weight's dtype")
    else:
        pt = torch.float32 if param_dtype is None else param_dtype
        pd = _dtype(pt, "param_dtype")
    dx = x.new_empty(shape)
    dw = torch.empty_like(weight) if weight is not None else None
    db = x.new_empty((dim,), dtype=pt) if bias else None
    ws, nb = _workspace("muon_layer_norm_backward_workspace", x.device, rows, dim)
    _call("muon_layer_norm_backward", index, grad_out.data_ptr(), ldg, x.data_ptr(), xd, ldx, rows, dim,
          mean.data_ptr(), rstd.data_ptr(), _ptr(weight), pd, dx.data_ptr(), _ptr(dw), _ptr(db), ws.data_ptr(), nb)
    return dx, dw, db


def _head(hidden, weight, targets):
    """(hidden as rows, rows, dim, row stride, type code of targets, device index)."""
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
    index = _same_device(weight, hidden, targets)
    if hidden.data_ptr() % 16 or weight.data_ptr() % 16:
        raise ValueError("hidden and weight must be 16-byte aligned")
    return hidden, rows, dim, ld, it, index


def muon_head_loss(hidden, weight, targets, ignore_index=-100):
    """(loss, lse) per token of the softmax cross entropy of hidden . weight^T:
    hidden (..., dim) and weight (vocab, dim) bf16 with dim a multiple of 8,
    targets int32 or int64.  Both results are fp32 in targets' shape, 0 for
    tokens whose target is ignore_index; the logits are not kept."""
    hidden, rows, dim, ld, it, index = _head(hidden, weight, targets)
    loss = torch.empty_like(targets, dtype=torch.float32)
    lse = torch.empty_like(loss)
    if rows:
        vocab = weight.shape[0]
        ws, nb = _workspace("muon_head_loss_workspace", weight.device, rows, vocab, dim, 0)
        _call("muon_head_loss", index, hidden.data_ptr(), ld, weight.data_ptr(), targets.data_ptr(), it, rows, vocab,
              dim, ignore_index, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), nb)
    return loss, lse


def muon_head_loss_backward(hidden, weight, targets, lse, grad_loss, ignore_index=-100, hidden_grad=True,
                            weight_grad=True):
    """(dhidden, dweight), bf16, from the lse of muon_head_loss and the fp32
    gradient of its per-token loss.  Either can be left out (None)."""
    shape = hidden.shape
    hidden, rows, dim, ld, it, index = _head(hidden, weight, targets)
    _vector(lse, "lse", rows, torch.float32)
    _vector(grad_loss, "grad_loss", rows, torch.float32)
    _same_device(weight, lse, grad_loss)
    if not (hidden_grad or weight_grad):
        raise ValueError("one gradient at least")
    vocab = weight.shape[0]
    dh = weight.new_empty(shape) if hidden_grad else None
    dw = torch.empty_like(weight) if weight_grad else None
    if rows or weight_grad:
        ws, nb = _workspace("muon_head_loss_workspace", weight.device, rows, vocab, dim, 1)
        _call("muon_head_loss_backward", index, hidden.data_ptr(), ld, weight.data_ptr(), targets.data_ptr(), it, rows,
              vocab, dim, ignore_index, lse.data_ptr(), grad_loss.data_ptr(), _ptr(dh), _ptr(dw), ws.data_ptr(), nb)
    return dh, dw
