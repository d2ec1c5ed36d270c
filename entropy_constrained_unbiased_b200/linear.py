"""Linear layers on 8-bit data: the integer product for serving, and training
with 8-bit activation checkpoints.

`int8_linear` quantises its tokens and multiplies them by 8-bit weights.
`checkpoint_linear` is F.linear for training: the forward product is the plain
one, but what it keeps of its input for the backward pass is the unbiased 8-bit
checkpoint, about half the bytes of bfloat16. The weight gradient is linear in
the input, so its mean over the rounding is the exact gradient; the input's and
the bias's gradients do not use the checkpoint.

The operators are the library's kernels (ecasq.py); there is no CPU path.
"""
from __future__ import annotations

import torch
import torch.nn.functional as F

from . import ecasq as E


def _rows(x):
    """x [..., k] as a matrix with adjacent columns and distinct rows: a view, or a copy of a transposed or expanded x."""
    rows = x if x.dim() == 2 else x.reshape(-1, x.shape[-1])
    n, k = rows.shape
    ld, one = rows.stride()
    return rows.contiguous() if (k > 1 and one != 1) or (n > 1 and ld < k) else rows


def _whole_rows(weight):
    """8-bit weights in rows of whole 16 bytes: as they are, or a copy of dense rows of another length."""
    if weight.dim() != 2 or weight.dtype != torch.int8:
        return weight
    n, k = weight.shape
    if (k if n == 1 else weight.stride(0)) % 16 == 0:  # the pitch of a single row says nothing
        return weight
    return F.pad(weight, (0, -k % 16))[:, :k]


def int8_linear(x: torch.Tensor, weight: torch.Tensor, weight_scale: torch.Tensor, bias=None) -> torch.Tensor:
    """x [..., k] (float32, bfloat16 or float16) times 8-bit weights: quantises each
    token and multiplies, Y [..., n] in x's type. weight int8 [n, k] and
    weight_scale float32 [n] are ecasq.int8_quantize's of the layer's weight
    matrix; bias float32 [n]. For serving: it has no gradient, and refuses an x,
    a scale or a bias that asks for one.

    int8_quantize lays rows out in whole 32 bytes. Weights that lost this (a dense
    copy, a loaded state, of a k that is no multiple of 16) are copied in every
    call; F.pad(weight, (0, -k % 16))[:, :k], kept, saves that."""
    if torch.is_grad_enabled() and (x.requires_grad or weight_scale.requires_grad
                                    or (bias is not None and bias.requires_grad)):
        raise E.EcasqError("int8_linear has no gradient; use checkpoint_linear for training, or torch.no_grad()")
    if x.dim() == 0:
        raise E.EcasqError("x must have at least one dimension")
    y = E.int8_linear(_rows(x), _whole_rows(weight), weight_scale, bias)
    return y if x.dim() == 2 else y.reshape(*x.shape[:-1], y.shape[1])


class _CheckpointLinear(torch.autograd.Function):
    @staticmethod
    @torch.amp.custom_fwd(device_type="cuda")
    def forward(ctx, x, weight, bias, seed):
        if ctx.needs_input_grad[1]:
            # whole rows: a hook may copy what is saved, and a part's copy would lose their pitch
            q, scale = E._checkpoint8(_rows(x), seed)
        else:
            q = scale = None
        ctx.save_for_backward(q, scale, weight if ctx.needs_input_grad[0] else None)
        ctx.columns = x.shape[-1]
        ctx.dtypes = x.dtype, weight.dtype, None if bias is None else bias.dtype
        return F.linear(x, weight, bias)

    @staticmethod
    @torch.autograd.function.once_differentiable
    @torch.amp.custom_bwd(device_type="cuda")
    def backward(ctx, dy):
        q, scale, weight = ctx.saved_tensors
        x_type, w_type, b_type = ctx.dtypes
        dx = dw = db = None
        if ctx.needs_input_grad[0]:
            dx = torch.matmul(dy, weight).to(x_type)
        rows = _rows(dy)
        if ctx.needs_input_grad[1]:
            q, scale = E._part8(q, scale, ctx.columns)
            dw = E.checkpoint8_wgrad(rows, q, scale, w_type)
        if ctx.needs_input_grad[2]:
            db = rows.sum(0, dtype=torch.float32).to(b_type)
        return dx, dw, db, None


def checkpoint_linear(x: torch.Tensor, weight: torch.Tensor, bias=None, *, seed) -> torch.Tensor:
    """x [..., k] W^T + bias, keeping x for the backward pass in 8 bits (unbiased,
    keyed by `seed`: another value for each layer and step, so that roundings are
    independent; an integer, or a CUDA int64 tensor of one entry for graphs).
    weight [n, k] and bias [n] in x's type, or in any under autocast.

    Gradients are of first order, by backward or autograd.grad; torch.func transforms
    and forward mode are not supported (torch refuses them).

    A backward pass may be captured into a graph, as with F.linear: warm up on the
    capturing stream, and keep no eager autograd graph of the same leaves alive."""
    if x.device.type != "cuda" or weight.device != x.device:
        raise E.EcasqError("checkpoint_linear needs x and weight on one CUDA device; there is no CPU path")
    if weight.dim() != 2 or 0 in weight.shape or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise E.EcasqError(f"x [..., k] and weight [n, k] do not match: {list(x.shape)}, {list(weight.shape)}")
    if not torch.is_grad_enabled():
        return F.linear(x, weight, bias)  # nothing is kept
    return _CheckpointLinear.apply(x, weight, bias, seed)
