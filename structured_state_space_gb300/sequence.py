"""Linear attention with a decay for each head, rotary positions, layer norm and the vocabulary loss over the C ABI,
each with its backward pass.

Arrays of heads are [batch, L, heads, width] tensors, or [batch, heads, width] for one token per sequence (float32,
bfloat16 or float16), whose last dimension is contiguous; any other strides are taken as they are, so slices of a
projection's output need no copy.  Parameters, states and losses are float32.  As in block.py a tensor that does not fit
raises, a call runs on the GPU of its first tensor, whichever is current, and with ``stream`` given (one of that
GPU's) results and workspaces are allocated for that stream, which the caller orders after the work that fills
the inputs.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import S4Error, load
from .block import _away, _bad, _code, _dense, _flat, _on, _raw_stream, _scratch, _slots

__all__ = ["s4_linear_attention_fwd", "s4_linear_attention_step", "s4_linear_attention_bwd", "s4_rotary_freqs",
           "s4_rotary_fwd", "s4_rotary_bwd", "s4_layer_norm_fwd", "s4_layer_norm_bwd", "s4_vocab_loss_fwd",
           "s4_vocab_loss_bwd"]

_F32, _F64, _I32, _I64 = torch.float32, torch.float64, torch.int32, torch.int64
_empty = torch.empty

# The argument structs of include/s4.h, packed as C lays them out.
_ATTENTION = struct.Struct("@16q6PNf8i0q")
_ATTENTION_BWD = struct.Struct("@28q6PNf7i0q")
_ROTARY = struct.Struct("@16q2Pqf9i0q")
_LAYER_NORM = struct.Struct("@4P3qf2i0q")
_LAYER_NORM_BWD = struct.Struct("@7PN4qf2i0q")
_LOSS = struct.Struct("@6PN3q4i0q")
_LOSS_BWD = struct.Struct("@8PN3q4i0q")

_fn = {}


def _lib():
    """The library's entry points by name, with their argument types set once."""
    lib = load()
    vp, i32, sz, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong
    for name in ("s4_linear_attention_fwd", "s4_linear_attention_bwd", "s4_rotary", "s4_layer_norm_fwd", "s4_layer_norm_bwd",
                 "s4_vocab_loss_fwd", "s4_vocab_loss_bwd"):
        f = getattr(lib, name)
        f.argtypes, f.restype = [ctypes.c_char_p, vp], i32
        _fn[name] = f
    for name, args in (("s4_linear_attention_workspace_bytes", [i32] * 6),
                       ("s4_linear_attention_bwd_workspace_bytes", [i32] * 6),
                       ("s4_layer_norm_bwd_workspace_bytes", [ll, i32]), ("s4_vocab_loss_workspace_bytes", [ctypes.c_char_p]),
                       ("s4_vocab_loss_bwd_workspace_bytes", [ctypes.c_char_p])):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, sz
        _fn[name] = f
    return _fn


def _call(name, args, dev):
    code = (_fn.get(name) or _lib()[name])(args, _raw_stream(dev))
    if code:
        raise S4Error(code, name)


def _bytes(name, *sizes):
    n = (_fn.get(name) or _lib()[name])(*sizes)
    if n == 0:
        raise S4Error(1, name)
    return n


def _heads(t, dtype, shape, dev, name):
    """(address, batch, row and head strides) of [batch, L, heads, width], or of one token's [batch, heads, width]."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != dev:
        _bad(t, name, dtype, shape, dev)
    s = t.stride()
    if s[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name}: its last dimension must be contiguous")
    return t.data_ptr(), s[0], s[-3], s[-2]


def _of_heads(t, dims, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected {dims}")
    return t.shape


def _widths(q, k, v, dims):
    """(batch, L, heads, groups, key width, value width)."""
    s, c, d = _of_heads(q, dims, "q"), _of_heads(k, dims, "k"), _of_heads(v, dims, "v")
    if c[-2] < 1 or s[-2] % c[-2]:
        raise ValueError(f"k: {c[-2]} heads do not divide q's {s[-2]}")
    return s[0], (s[1] if dims == 4 else 1), s[-2], c[-2], s[-1], d[-1]


def _attention(q, k, v, log_decay, scale, lengths, state, state_out, index, o, ws, dims):
    (code, dev), ty = _code(q), q.dtype
    batch, L, H, G, K, V = _widths(q, k, v, dims)
    lead = q.shape[:dims - 2]
    if o is None:
        o = _empty((*lead, H, V), dtype=ty, device=q.device)
    slots = _slots(state, state_out, batch, index)
    if ws is None and L > 1:
        need = _bytes("s4_linear_attention_workspace_bytes", batch, L, H, G, K, V)
        ws, wp, wn = _scratch(None, dev, need if need > 256 else 0, q)
    else:
        ws, wp, wn = _scratch(ws, dev)
    past = (slots, H, K, V)
    args = _ATTENTION.pack(*_heads(q, ty, (*lead, H, K), dev, "q"), *_heads(k, ty, (*lead, G, K), dev, "k"),
                           *_heads(v, ty, (*lead, G, V), dev, "v"), *_heads(o, ty, (*lead, H, V), dev, "o"),
                           _dense(log_decay, _F32, (H,), dev, "log_decay"), _dense(lengths, _I32, (batch,), dev, "lengths"),
                           _dense(index, _I32, (batch,), dev, "index"), _dense(state, _F32, past, dev, "state"),
                           _dense(state_out, _F32, past, dev, "state_out"), wp, wn,
                           K ** -0.5 if scale is None else scale, batch, L, H, G, K, V, slots, code)
    _call("s4_linear_attention_fwd", args, dev)
    return o


def s4_linear_attention_fwd(q, k, v, log_decay, *, scale=None, lengths=None, state=None, state_out=None, index=None, o=None,
                            ws=None, stream=None):
    """Linear attention with a decay for each head: S = exp(log_decay) S + k v^T, o = scale S^T q, along L.

    q [batch, L, H, K]; k [batch, L, G, K], v [batch, L, G, V] (H/G heads to each); log_decay [H] (0 or less);
    scale: K^-0.5 when None.  lengths, index as for s4_short_conv_fwd; state, state_out [slots, H, K, V] float32 (the
    same tensor for in place).  ws: s4_linear_attention_workspace_bytes (allocated per call when None)."""
    if stream is not None or _away(q):
        return _on(stream, s4_linear_attention_fwd, q, k, v, log_decay, scale=scale, lengths=lengths, state=state,
                   state_out=state_out, index=index, o=o, ws=ws)
    return _attention(q, k, v, log_decay, scale, lengths, state, state_out, index, o, ws, 4)


def s4_linear_attention_step(q, k, v, log_decay, state, *, scale=None, state_out=None, index=None, o=None, ws=None,
                             stream=None):
    """One token per sequence: q [batch, H, K], k [batch, G, K], v [batch, G, V] -> o [batch, H, V].  The state is
    updated in place, or written to state_out (the old one then stays, as for tokens that may be rejected)."""
    if stream is not None or _away(q):
        return _on(stream, s4_linear_attention_step, q, k, v, log_decay, state, scale=scale, state_out=state_out,
                   index=index, o=o, ws=ws)
    return _attention(q, k, v, log_decay, scale, None, state, state if state_out is None else state_out, index, o, ws, 3)


def s4_linear_attention_bwd(q, k, v, log_decay, do, *, scale=None, lengths=None, state=None, dstate=None,
                            want_dstate0=False, ws=None, stream=None):
    """Gradients of s4_linear_attention_fwd from do: a dict of dq, dk, dv, and dstate0, the gradient of the state on
    entry, where asked for (the decay is a constant).  state, dstate [batch, H, K, V]: the state on entry and the
    gradient of the state on return (None: zeros).  Nothing is kept from the forward call.  ws:
    s4_linear_attention_bwd_workspace_bytes."""
    if stream is not None or _away(q):
        return _on(stream, s4_linear_attention_bwd, q, k, v, log_decay, do, scale=scale, lengths=lengths, state=state,
                   dstate=dstate, want_dstate0=want_dstate0, ws=ws)
    (code, dev), ty, on = _code(q), q.dtype, q.device
    batch, L, H, G, K, V = _widths(q, k, v, 4)
    ws, wp, wn = _scratch(ws, dev, _bytes("s4_linear_attention_bwd_workspace_bytes", batch, L, H, G, K, V), q)
    shapes = {"dq": (batch, L, H, K), "dk": (batch, L, G, K), "dv": (batch, L, G, V)}
    out = {n: _empty(s, dtype=ty, device=on) for n, s in shapes.items()}
    past = (batch, H, K, V)
    if want_dstate0:
        out["dstate0"] = _empty(past, dtype=_F32, device=on)
    args = _ATTENTION_BWD.pack(
        *_heads(q, ty, shapes["dq"], dev, "q"), *_heads(k, ty, shapes["dk"], dev, "k"), *_heads(v, ty, shapes["dv"], dev, "v"),
        *_heads(do, ty, (batch, L, H, V), dev, "do"), *(x for n, s in shapes.items() for x in _heads(out[n], ty, s, dev, n)),
        _dense(log_decay, _F32, (H,), dev, "log_decay"), _dense(lengths, _I32, (batch,), dev, "lengths"),
        _dense(state, _F32, past, dev, "state"), _dense(dstate, _F32, past, dev, "dstate"),
        _dense(out.get("dstate0"), _F32, past, dev, "dstate0"), wp, wn, K ** -0.5 if scale is None else scale,
        batch, L, H, G, K, V, code)
    _call("s4_linear_attention_bwd", args, dev)
    return out


def s4_rotary_freqs(width, base=10000.0, *, scaling=None, factor=1.0, length=None, turns=(1.0, 32.0), device=None):
    """The angles per position of a rotated part of `width` channels, [width / 2] float64, and the amplitude that goes
    with them: base^(-2i / width), scaled for contexts `factor` times those of training.

    scaling: None; "linear": all angles over factor (positions interpolated); "base": a larger base, so that the
    slowest pair is slowed by factor and the fastest not at all; "parts": pairs that turn less than turns[0] times in
    `length` positions (the length of training) are slowed by factor, those that turn more than turns[1] times
    stay, a linear mixture between; the amplitude is then 1 + 0.1 log(factor), else 1."""
    if width < 2 or width % 2:
        raise ValueError(f"width: {width}, expected a positive even number")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    if scaling == "base" and width > 2:
        base = base * factor ** (width / (width - 2))
    f = torch.pow(torch.tensor(float(base), dtype=_F64), -torch.arange(0, width, 2, dtype=_F64) / width)
    amplitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if length is None or not turns[1] > turns[0]:
            raise ValueError("scaling by parts needs the length of training and turns[1] > turns[0]")
        kept = ((f * length / (2 * math.pi) - turns[0]) / (turns[1] - turns[0])).clamp(0, 1)
        f = f / factor * (1 - kept) + f * kept
        amplitude = 1 + 0.1 * math.log(factor) if factor > 1 else 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"scaling: {scaling!r}, expected None, 'linear', 'base' or 'parts'")
    return f.to(device) if device is not None else f, amplitude


def _rotary(q, k, freqs, positions, pairs, amplitude, q_out, k_out, inverse):
    (code, dev), ty, shape = _code(q), q.dtype, q.shape
    if len(shape) not in (3, 4):
        raise ValueError(f"q: {len(shape)} dimensions, expected 3 or 4")
    lead = shape[:-2]
    batch, L = lead[0], (lead[1] if len(lead) == 2 else 1)
    H, D = shape[-2:]
    heads = None if k is None else (*lead, _of_heads(k, len(shape), "k")[-2], D)
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
        raise TypeError("freqs must be a torch.Tensor of one dimension")
    R = freqs.shape[0]
    if q_out is None:
        q_out = _empty(shape, dtype=ty, device=q.device)
    if k is not None and k_out is None:
        k_out = _empty(heads, dtype=ty, device=q.device)
    pp = pb = 0
    if positions is None:
        if len(lead) == 1:
            raise ValueError("single tokens need their positions")
    elif isinstance(positions, torch.Tensor) and positions.dim() == 1 and len(lead) == 2:
        pp = _dense(positions, _I32, (L,), dev, "positions")  # of every sequence
    else:
        pp, pb = _dense(positions, _I32, lead, dev, "positions"), L
    none = (0, 0, 0, 0)
    args = _ROTARY.pack(*_heads(q, ty, shape, dev, "q"), *(none if k is None else _heads(k, ty, heads, dev, "k")),
                        *_heads(q_out, ty, shape, dev, "q_out"),
                        *(none if k is None else _heads(k_out, ty, heads, dev, "k_out")),
                        _dense(freqs, _F64, (R,), dev, "freqs"), pp, pb, amplitude, batch, L, H, 0 if k is None else heads[-2],
                        D, R, 1 if pairs else 0, inverse, code)
    _call("s4_rotary", args, dev)
    return q_out, k_out


def s4_rotary_fwd(q, k, freqs, *, positions=None, pairs=False, amplitude=1.0, q_out=None, k_out=None, stream=None):
    """Queries and keys turned by their tokens' positions -> (q_out, k_out).

    q [batch, L, H, D], k [batch, L, G, D] or None (or [batch, heads, D] each, one token per sequence); freqs [R]
    float64 on their GPU (s4_rotary_freqs): the first 2 R channels of a head are turned, the others copied.
    positions int32 [batch, L], [L] for every sequence, or [batch] for single tokens (None: 0 .. L-1).  Pair i is
    channels (i, R + i), or (2i, 2i + 1) with pairs=True.  q_out may be q and k_out may be k (in place)."""
    if stream is not None or _away(q):
        return _on(stream, s4_rotary_fwd, q, k, freqs, positions=positions, pairs=pairs, amplitude=amplitude, q_out=q_out,
                   k_out=k_out)
    return _rotary(q, k, freqs, positions, pairs, amplitude, q_out, k_out, 0)


def s4_rotary_bwd(dq, dk, freqs, *, positions=None, pairs=False, amplitude=1.0, q_out=None, k_out=None, stream=None):
    """The gradients of s4_rotary_fwd's inputs from those of its outputs: turned back, times the same amplitude."""
    if stream is not None or _away(dq):
        return _on(stream, s4_rotary_bwd, dq, dk, freqs, positions=positions, pairs=pairs, amplitude=amplitude, q_out=q_out,
                   k_out=k_out)
    return _rotary(dq, dk, freqs, positions, pairs, amplitude, q_out, k_out, 1)


def s4_layer_norm_fwd(x, w=None, b=None, *, eps=1e-5, y=None, stream=None):
    """y = (x - mean) / sqrt(mean((x - mean)^2) + eps) * w + b over the last dimension of x [..., H]; w, b [H] (None:
    ones, zeros).  y may be x."""
    if stream is not None or _away(x):
        return _on(stream, s4_layer_norm_fwd, x, w, b, eps=eps, y=y)
    (code, dev), dt, shape = _code(x), x.dtype, x.shape
    H = shape[-1]
    if y is None:
        y = _empty(shape, dtype=dt, device=x.device)
    px, sx = _flat(x, dt, shape, dev, "x")
    py, sy = _flat(y, dt, shape, dev, "y")
    args = _LAYER_NORM.pack(px, py, _dense(w, _F32, (H,), dev, "w"), _dense(b, _F32, (H,), dev, "b"), sx, sy,
                            x.numel() // H if H else 0, eps, H, code)
    _call("s4_layer_norm_fwd", args, dev)
    return y


def s4_layer_norm_bwd(x, dy, w=None, b=None, *, eps=1e-5, ws=None, stream=None):
    """Gradients of s4_layer_norm_fwd from dy: a dict of dx and, for what was given, dw and db."""
    if stream is not None or _away(x):
        return _on(stream, s4_layer_norm_bwd, x, dy, w, b, eps=eps, ws=ws)
    (code, dev), dt, shape, on = _code(x), x.dtype, x.shape, x.device
    H = shape[-1]
    rows = x.numel() // H if H else 0
    ws, wp, wn = _scratch(ws, dev, _bytes("s4_layer_norm_bwd_workspace_bytes", rows, H), x)
    out = {"dx": _empty(shape, dtype=dt, device=on)}
    for k, v in (("dw", w), ("db", b)):
        if v is not None:
            out[k] = _empty((H,), dtype=_F32, device=on)
    _dense(b, _F32, (H,), dev, "b")
    px, sx = _flat(x, dt, shape, dev, "x")
    py, sy = _flat(dy, dt, shape, dev, "dy")
    args = _LAYER_NORM_BWD.pack(px, py, out["dx"].data_ptr(), _dense(w, _F32, (H,), dev, "w"),
                                _dense(out.get("dw"), _F32, (H,), dev, "dw"), _dense(out.get("db"), _F32, (H,), dev, "db"),
                                wp, wn, sx, sy, H, rows, eps, H, code)
    _call("s4_layer_norm_bwd", args, dev)
    return out


def _targets(targets, lead, dev):
    """(address, whether they have 64 bits)."""
    wide = isinstance(targets, torch.Tensor) and targets.dtype == _I64
    return _dense(targets, _I64 if wide else _I32, lead, dev, "targets"), 1 if wide else 0


def _vocab(h, w, dev):
    """(rows, H, V, h's address and row stride, w's)."""
    H = h.shape[-1]
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise TypeError("w must be a torch.Tensor of two dimensions")
    V = w.shape[0]
    return (h.numel() // H if H else 0, H, V, *_flat(h, h.dtype, h.shape, dev, "h"), *_flat(w, h.dtype, (V, H), dev, "w"))


def s4_vocab_loss_fwd(h, w, targets, *, loss=None, lse=None, ws=None, stream=None):
    """Softmax cross entropy of hidden states h [..., H] against a vocabulary's weights w [V, H] (of one type), without
    keeping the logits -> (loss, lse), float32 of h's leading dimensions: lse = log sum exp(w h), loss =
    lse - w[target] . h, and 0 where the target is negative.  targets: int64 or int32.  ws (see s4_get_status)
    records a target of V or more, which counts as a negative one; its size is that of
    s4_vocab_loss_workspace_bytes (allocated per call when None)."""
    if stream is not None or _away(h):
        return _on(stream, s4_vocab_loss_fwd, h, w, targets, loss=loss, lse=lse, ws=ws)
    (code, dev), lead, on = _code(h), h.shape[:-1], h.device
    rows, H, V, hp, hs, wp, wr = _vocab(h, w, dev)
    if loss is None:
        loss = _empty(lead, dtype=_F32, device=on)
    if lse is None:
        lse = _empty(lead, dtype=_F32, device=on)
    tp, wide = _targets(targets, lead, dev)
    head = hp, wp, tp, _dense(loss, _F32, lead, dev, "loss"), _dense(lse, _F32, lead, dev, "lse")
    tail = hs, wr, rows, H, V, wide, code
    need = _bytes("s4_vocab_loss_workspace_bytes", _LOSS.pack(*head, 0, 0, *tail)) if ws is None else 0
    ws, sp, sn = _scratch(ws, dev, need, h)
    _call("s4_vocab_loss_fwd", _LOSS.pack(*head, sp, sn, *tail), dev)
    return loss, lse


def s4_vocab_loss_bwd(h, w, targets, lse, dloss, *, ws=None, stream=None):
    """Gradients of s4_vocab_loss_fwd from dloss (of the losses' shape) and the forward call's lse: a dict of dh and dw,
    of the inputs' type.  The logits are formed again, a piece of the vocabulary at a time.  ws:
    s4_vocab_loss_bwd_workspace_bytes."""
    if stream is not None or _away(h):
        return _on(stream, s4_vocab_loss_bwd, h, w, targets, lse, dloss, ws=ws)
    (code, dev), lead, on, ty = _code(h), h.shape[:-1], h.device, h.dtype
    rows, H, V, hp, hs, wp, wr = _vocab(h, w, dev)
    out = {"dh": _empty(h.shape, dtype=ty, device=on), "dw": _empty((V, H), dtype=ty, device=on)}
    tp, wide = _targets(targets, lead, dev)
    head = (hp, wp, tp, _dense(lse, _F32, lead, dev, "lse"), _dense(dloss, _F32, lead, dev, "dloss"), out["dh"].data_ptr(),
            out["dw"].data_ptr())
    tail = hs, wr, rows, H, V, wide, code
    need = _bytes("s4_vocab_loss_bwd_workspace_bytes", _LOSS_BWD.pack(*head, 0, 0, *tail)) if ws is None else 0
    ws, sp, sn = _scratch(ws, dev, need, h)
    _call("s4_vocab_loss_bwd", _LOSS_BWD.pack(*head, sp, sn, *tail), dev)
    return out
