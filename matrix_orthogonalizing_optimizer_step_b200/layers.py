"""The layers whose parameters the hybrid optimizer's AdamW lane steps, as
torch modules: token embedding, LayerNorm and the output head with its loss.

[NanoGPT-Muon] "从 SGD 到 Muon" keeps the embedding, the output head and the
1-D parameters out of Muon.  Modules of this file held under the names that
`split_params` knows (embed, wte, wpe, head, lm_head, ...) land in the AdamW
lane; their backward passes write the gradients that MuonHybrid.step reads.
All arithmetic runs in the library's kernels; the classes only keep
parameters and pass tensors.

Backward passes are not differentiable again.  As for any torch module, a
backward pass that is captured into a CUDA graph needs its forward pass in the
same capture and no eager graph of the same parameters alive at that time.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

import matrix_orthogonalizing_optimizer_step_b200 as _mo


def _rows(g):
    """g with rows that the kernels can read (autograd may hand over expanded
    or transposed gradients)."""
    if g.is_contiguous():
        return g
    if g.dim() == 2 and g.stride(1) == 1 and g.stride(0) >= g.shape[1]:
        return g
    return g.contiguous()


def _check_padding(padding_idx, vocab):
    if padding_idx is not None and not 0 <= padding_idx < vocab:
        raise ValueError("padding_idx must be a token of the vocabulary (0 or more)")


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale, padding_idx, out_dtype):
        ctx.save_for_backward(tokens)
        ctx.args = (weight.shape[0], scale, padding_idx, weight.dtype)
        return _mo.muon_embedding(tokens, weight, scale=scale, out_dtype=out_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        tokens, = ctx.saved_tensors
        vocab, scale, padding_idx, dtype = ctx.args
        dw = _mo.muon_embedding_backward(tokens, _rows(grad), vocab, scale=scale, padding_idx=padding_idx,
                                         grad_dtype=dtype)
        return None, dw, None, None, None


def embedding(tokens, weight, scale=1.0, padding_idx=None, out_dtype=None):
    """scale * weight[tokens] in out_dtype (default: the weight's).  The
    weight's gradient is dense, in the weight's dtype; padding_idx gets none."""
    _check_padding(padding_idx, weight.shape[0])
    tokens = tokens.contiguous()
    return _Embedding.apply(tokens, weight, scale, padding_idx, out_dtype)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = _mo.muon_layer_norm(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = _mo.muon_layer_norm_backward(_rows(grad), x, mean, rstd, weight, bias=ctx.needs_input_grad[2],
                                                  param_dtype=ctx.bias_dtype if weight is None else None,
                                                  weight_grad=ctx.needs_input_grad[1])
        return dx, dw, db, None


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """LayerNorm over the last dimension, in x's dtype (bf16 or fp32); weight
    and bias bf16 or fp32."""
    return _LayerNorm.apply(_rows(x), weight, bias, eps)


class _HeadLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, targets, ignore_index):
        loss, lse = _mo.muon_head_loss(hidden, weight, targets, ignore_index=ignore_index)
        ctx.save_for_backward(hidden, weight, targets, lse)
        ctx.ignore_index = ignore_index
        ctx.mark_non_differentiable(lse)
        return loss, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, grad, _):
        hidden, weight, targets, lse = ctx.saved_tensors
        dh, dw = _mo.muon_head_loss_backward(hidden, weight, targets, lse, grad.contiguous(),
                                             ignore_index=ctx.ignore_index, hidden_grad=ctx.needs_input_grad[0],
                                             weight_grad=ctx.needs_input_grad[1])
        return dh, dw, None, None


def head_loss(hidden, weight, targets, ignore_index=-100, reduction="mean"):
    """Softmax cross entropy of hidden . weight^T against targets, without the
    logits.  The products take bf16: an fp32 hidden or weight is rounded to it
    first, and its gradient comes back in fp32.  reduction "none" gives the
    per-token loss (0 for ignored targets), "sum" its sum, "mean" the mean over
    the tokens that count (0 if there are none)."""
    if reduction not in ("none", "sum", "mean"):
        raise ValueError("reduction must be none, sum or mean")
    targets = targets.contiguous()
    hidden = _rows(hidden.to(torch.bfloat16))
    if hidden.data_ptr() % 16 or (hidden.dim() == 2 and hidden.stride(0) % 8):
        hidden = hidden.clone(memory_format=torch.contiguous_format)
    loss, _ = _HeadLoss.apply(hidden, weight.to(torch.bfloat16), targets, ignore_index)
    if reduction == "none":
        return loss
    if reduction == "sum":
        return loss.sum()
    return loss.sum() / (targets != ignore_index).sum().clamp(min=1)


class Embedding(torch.nn.Module):
    """Token embedding with scaling; N(0, 0.02^2) at the start."""

    def __init__(self, num_embeddings, dim, scale=1.0, padding_idx=None, out_dtype=None, device=None, dtype=None):
        super().__init__()
        _check_padding(padding_idx, num_embeddings)
        self.scale, self.padding_idx, self.out_dtype = scale, padding_idx, out_dtype
        self.weight = torch.nn.Parameter(torch.empty(num_embeddings, dim, device=device, dtype=dtype))
        torch.nn.init.normal_(self.weight, std=0.02)

    def forward(self, tokens):
        return embedding(tokens, self.weight, self.scale, self.padding_idx, self.out_dtype)


class LayerNorm(torch.nn.Module):
    def __init__(self, dim, eps=1e-5, bias=True, device=None, dtype=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(dim, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(dim, device=device, dtype=dtype)) if bias else None

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias, self.eps)


class HeadLoss(torch.nn.Module):
    """Output head (vocab x dim, no bias) with its loss; N(0, 1 / dim) at the
    start.  `weight` may be another module's parameter (a tied embedding)."""

    def __init__(self, dim, vocab, ignore_index=-100, reduction="mean", weight=None, device=None, dtype=None):
        super().__init__()
        self.ignore_index, self.reduction = ignore_index, reduction
        if weight is None:
            weight = torch.nn.Parameter(torch.empty(vocab, dim, device=device, dtype=dtype))
            torch.nn.init.normal_(weight, std=1 / math.sqrt(dim))
        if tuple(weight.shape) != (vocab, dim):
            raise ValueError("weight must have shape (vocab, dim)")
        self.weight = weight

    def forward(self, hidden, targets):
        return head_loss(hidden, self.weight, targets, self.ignore_index, self.reduction)
