"""The library's block operators as differentiable functions: torch.autograd nodes whose forward and
backward are the library's calls (block.py, sequence.py).  Nothing beside the inputs is kept for the backward
pass (the vocabulary loss keeps its lse).  Activations and parameters as there; sequences start from a state of zeros.
There are no second derivatives: gradients taken with create_graph=True raise where they are differentiated.
What is a constant of an operator and requires a gradient all the same is refused.
A backward pass that is captured into a CUDA graph needs leaves of its own: torch accumulates a leaf's gradient on the stream of
the first graph that still holds it, which may not be captured.

    short_conv(x, w, bias, lengths)                               -> y
    selective_scan(x, dt, A, B, C, D, z, dt_bias, lengths)        -> y
    block_norm(o, gate, h, w_post, scale, w_pre, eps)             -> h_out, y
    linear_attention(q, k, v, log_decay, scale, lengths, ws)      -> o          (log_decay is a constant)
    rotary(q, k, freqs, positions, pairs, amplitude)              -> q, k       (k may be None; freqs are constants)
    layer_norm(x, w, b, eps)                                      -> y
    vocab_loss(h, w, targets, ws)                                 -> losses     (one per row)
"""
from __future__ import annotations

import torch

from . import block, sequence

__all__ = ["short_conv", "selective_scan", "block_norm", "linear_attention", "rotary", "layer_norm", "vocab_loss"]


class _Final(torch.autograd.Function):
    """Gradients, as functions of `inputs` that cannot be differentiated."""
    @staticmethod
    def forward(ctx, count, *values):
        return tuple(v.detach() for v in values[:count])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the library's block operators have no second derivatives")


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


class _LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, scale, lengths, ws):
        ctx.save_for_backward(q, k, v, log_decay, lengths)
        ctx.scale = scale
        return sequence.s4_linear_attention_fwd(q, k, v, log_decay, scale=scale, lengths=lengths, ws=ws)

    @staticmethod
    def backward(ctx, do):
        q, k, v, log_decay, lengths = ctx.saved_tensors
        g = sequence.s4_linear_attention_bwd(q, k, v, log_decay, do.contiguous(), scale=ctx.scale, lengths=lengths)
        return _final((g["dq"], g["dk"], g["dv"], None, None, None, None), (q, k, v, do))


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, freqs, positions, pairs, amplitude):
        ctx.save_for_backward(freqs, positions)
        ctx.how = pairs, amplitude
        ctx.set_materialize_grads(False)
        return sequence.s4_rotary_fwd(q, k, freqs, positions=positions, pairs=pairs, amplitude=amplitude)

    @staticmethod
    def backward(ctx, dq, dk):
        freqs, positions = ctx.saved_tensors
        pairs, amplitude = ctx.how
        given = [g.contiguous() for g in (dq, dk) if g is not None]
        if not given:
            return (None,) * 6
        # each alone where one is missing: they may have different numbers of heads
        back = sequence.s4_rotary_bwd(given[0], given[1] if len(given) == 2 else None, freqs, positions=positions,
                                      pairs=pairs, amplitude=amplitude)
        got = iter(back)
        return _final((None if dq is None else next(got), None if dk is None else next(got), None, None, None, None),
                      (dq, dk))


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, eps):
        ctx.save_for_backward(x, w, b)
        ctx.eps = eps
        return sequence.s4_layer_norm_fwd(x, w, b, eps=eps)

    @staticmethod
    def backward(ctx, dy):
        x, w, b = ctx.saved_tensors
        g = sequence.s4_layer_norm_bwd(x, dy.contiguous(), w, b, eps=ctx.eps)
        return _final((g["dx"], g.get("dw"), g.get("db"), None), (x, w, dy))


class _VocabLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, targets, ws):
        loss, lse = sequence.s4_vocab_loss_fwd(h, w, targets, ws=ws)
        ctx.save_for_backward(h, w, targets, lse)
        return loss

    @staticmethod
    def backward(ctx, dloss):
        h, w, targets, lse = ctx.saved_tensors
        g = sequence.s4_vocab_loss_bwd(h, w, targets, lse, dloss.contiguous())
        return _final((g["dh"], g["dw"], None, None), (h, w, dloss))


def _constant(t, name):
    """Raises where a gradient is wanted of what has none: a parameter would silently stay as it is."""
    if isinstance(t, torch.Tensor) and t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} has no gradient here: pass {name}.detach()")


def linear_attention(q, k, v, log_decay, scale=None, lengths=None, ws=None):
    """o.  A length out of range is recorded in ws, the forward call's workspace (see s4_get_status)."""
    _constant(log_decay, "log_decay")
    return _LinearAttention.apply(q, k, v, log_decay, scale, lengths, ws)


def rotary(q, k, freqs, positions=None, pairs=False, amplitude=1.0):
    """(q, k), turned; k may be None."""
    _constant(freqs, "freqs")
    return _Rotary.apply(q, k, freqs, positions, pairs, amplitude)


def layer_norm(x, w=None, b=None, eps=1e-5):
    return _LayerNorm.apply(x, w, b, eps)


def vocab_loss(h, w, targets, ws=None):
    """One loss per row of h (0 where the target is negative).  A target beyond the vocabulary counts as a negative one and is
    recorded in ws, the forward call's workspace (see s4_get_status)."""
    return _VocabLoss.apply(h, w, targets, ws)
