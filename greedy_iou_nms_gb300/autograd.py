"""The detection-head operators for torch's autograd.

Functions of the names and arguments of greedy_iou_nms_gb300 whose results
carry gradients, each by the library's own gradient kernels; nothing but what
the gradient reads is saved (a dropout mask is drawn again from its numbers).
First derivatives only.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import head


class _GroupNormAct(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, groups, eps, act, p, seed, offset):
        y, mean, rstd = head.group_norm_act(x, groups, weight, bias, eps=eps, act=act, p=p, seed=seed, offset=offset,
                                            return_stats=True)
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        ctx.numbers = (groups, act, p, seed, offset)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, mean, rstd = ctx.saved_tensors
        groups, act, p, seed, offset = ctx.numbers
        dx, dweight, dbias = head.group_norm_act_grad(dy, x, mean, rstd, groups, weight, bias, act=act, p=p, seed=seed,
                                                      offset=offset)
        return (dx, None if weight is None else dweight.to(weight.dtype), None if bias is None else dbias.to(bias.dtype),
                None, None, None, None, None, None)


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset):
        ctx.numbers = (p, seed, offset)
        return head.dropout(x, p, seed, offset, residual=residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        dx = head.dropout_grad(dy, *ctx.numbers) if ctx.needs_input_grad[0] else None
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None


class _RelationSoftmax(torch.autograd.Function):
    @staticmethod
    def forward(ctx, scores, table, buckets, scale, key_mask):
        probs = head.relation_softmax(scores, table, buckets, scale=scale, key_mask=key_mask)
        ctx.save_for_backward(probs, buckets, key_mask)
        ctx.scale, ctx.rows, ctx.table_type = scale, table.shape[0], table.dtype
        return probs

    @staticmethod
    @once_differentiable
    def backward(ctx, dprobs):
        probs, buckets, key_mask = ctx.saved_tensors
        dscores, dtable = head.relation_softmax_grad(dprobs, probs, buckets, ctx.rows, scale=ctx.scale,
                                                     key_mask=key_mask)
        return dscores, dtable.to(ctx.table_type), None, None, None


def group_norm_act(x, groups: int, weight=None, bias=None, *, eps: float = 1e-5, act: str = "none", p: float = 0.0,
                   seed: int = 0, offset: int = 0):
    """`greedy_iou_nms_gb300.group_norm_act` with gradients to x, weight and bias."""
    return _GroupNormAct.apply(x, weight, bias, groups, eps, act, p, seed, offset)


def dropout(x, p: float, seed: int, offset: int = 0, *, residual=None):
    """`greedy_iou_nms_gb300.dropout` with gradients to x and the residual."""
    return _Dropout.apply(x, residual, p, seed, offset)


def relation_softmax(scores, table, buckets, *, scale: float = 1.0, key_mask=None):
    """`greedy_iou_nms_gb300.relation_softmax` with gradients to the scores and the table."""
    return _RelationSoftmax.apply(scores, table, buckets, scale, key_mask)
