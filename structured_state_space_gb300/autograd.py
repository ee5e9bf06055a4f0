"""The selective block's operators as differentiable functions: torch.autograd nodes whose forward and
backward are the library's calls (block.py).  Nothing beside the inputs is kept for the backward
pass.  Activations and parameters as in block.py; sequences start from a state of zeros.  There are
no second derivatives: gradients taken with create_graph=True raise where they are differentiated.

    short_conv(x, w, bias, lengths)                               -> y
    selective_scan(x, dt, A, B, C, D, z, dt_bias, lengths)        -> y
    block_norm(o, gate, h, w_post, scale, w_pre, eps)             -> h_out, y
"""
from __future__ import annotations

import torch

from . import block

__all__ = ["short_conv", "selective_scan", "block_norm"]


class _Final(torch.autograd.Function):
    """Gradients, as functions of `inputs` that cannot be differentiated."""
    @staticmethod
    def forward(ctx, count, *values):
        return tuple(v.detach() for v in values[:count])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the selective block's operators have no second derivatives")


def _final(grads, inputs):
    """The gradients as they are; with create_graph=True, linked to the inputs so that differentiating them
    raises.  (Without the link they would be constants there, and a loss that uses them would silently lose a term.)"""
    if not torch.is_grad_enabled():
        return grads
    given = [g for g in grads if g is not None]
    linked = iter(_Final.apply(len(given), *given, *inputs))
    return tuple(None if g is None else next(linked) for g in grads)


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, lengths):
        ctx.save_for_backward(x, w, bias, lengths)
        return block.s4_short_conv_fwd(x, w, bias, lengths=lengths)

    @staticmethod
    def backward(ctx, dy):
        x, w, bias, lengths = ctx.saved_tensors
        g = block.s4_short_conv_bwd(x, w, bias, dy.contiguous(), lengths=lengths)
        return _final((g["dx"], g["dw"], g.get("dbias"), None), (x, w, bias, dy))


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, lengths):
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, lengths)
        return block.s4_selective_scan_fwd(x, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, lengths=lengths)

    @staticmethod
    def backward(ctx, dy):
        x, dt, A, B, C, D, z, dt_bias, lengths = ctx.saved_tensors
        g = block.s4_selective_scan_bwd(x, dt, A, B, C, dy.contiguous(), D=D, z=z, dt_bias=dt_bias, lengths=lengths)
        return _final((g["dx"], g["ddt"], g["dA"], g["dB"], g["dC"], g.get("dD"), g.get("dz"), g.get("ddt_bias"), None),
                      (x, dt, A, B, C, D, z, dt_bias, dy))


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, o, gate, h, w_post, scale, w_pre, eps):
        ctx.save_for_backward(o, gate, h, w_post, scale, w_pre)
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        return block.s4_block_norm_fwd(o, gate=gate, h=h, w_post=w_post, scale=scale, w_pre=w_pre, eps=eps)

    @staticmethod
    def backward(ctx, dh_out, dy):
        if dh_out is None and dy is None:
            return (None,) * 7
        o, gate, h, w_post, scale, w_pre = ctx.saved_tensors
        g = block.s4_block_norm_bwd(o, None if dy is None else dy.contiguous(),
                                    dh_out=None if dh_out is None else dh_out.contiguous(), gate=gate, h=h, w_post=w_post,
                                    scale=scale, w_pre=w_pre, eps=ctx.eps)
        return _final((g["do"], g.get("dgate"), g.get("dh"), g.get("dw_post"), g.get("dscale"), g.get("dw_pre"), None),
                      (o, gate, h, w_post, scale, w_pre, dh_out, dy))


def short_conv(x, w, bias=None, lengths=None):
    return _ShortConv.apply(x, w, bias, lengths)


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, lengths=None):
    return _SelectiveScan.apply(x, dt, A, B, C, D, z, dt_bias, lengths)


def block_norm(o, gate=None, h=None, w_post=None, scale=None, w_pre=None, eps=1e-5):
    """(h_out, y); y is None without w_pre."""
    return _BlockNorm.apply(o, gate, h, w_post, scale, w_pre, eps)
