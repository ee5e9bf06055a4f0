"""The selective block's operators over the C ABI: the short causal convolution, the selective
scan and the norms around a block, each with its backward pass.

Activations are [batch, L, channels] tensors (float32, bfloat16 or float16) whose channels are
contiguous; any batch and row strides are taken as they are, so slices of a projection's
output need no copy.  Parameters are float32.  As in the rest of the binding there is no
fallback: a tensor that does not fit raises, and the library's kernels do all the work.

A call runs on the GPU of its activations, whichever is current; all its tensors lie on that one.
With ``stream`` given (one of that GPU's), results and workspaces are allocated for that stream; the caller
orders it after the work that fills the inputs.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import S4Error, load

__all__ = ["s4_short_conv_fwd", "s4_short_conv_step", "s4_short_conv_bwd", "s4_selective_scan_fwd", "s4_selective_step",
           "s4_selective_scan_bwd", "s4_block_norm_fwd", "s4_block_norm_bwd"]

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_F32, _I32 = torch.float32, torch.int32
_empty = torch.empty
_raw_stream = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice

# The argument structs of include/s4.h, packed as C lays them out.
_CONV = struct.Struct("@6q7PN7i0q")
_CONV_BWD = struct.Struct("@9q9PN6i0q")
_SCAN = struct.Struct("@18q8PN2q8i")
_SCAN_BWD = struct.Struct("@27q13PN2q7i0q")
_NORM = struct.Struct("@8P6qf3i0q")
_NORM_BWD = struct.Struct("@15PN9qf3i0q")

_fn = {}


def _lib():
    """The library's entry points by name, with their argument types set once."""
    lib = load()
    vp, i32, sz, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong
    for name in ("s4_short_conv_fwd", "s4_short_conv_bwd", "s4_selective_scan_fwd", "s4_selective_scan_bwd",
                 "s4_block_norm_fwd", "s4_block_norm_bwd"):
        f = getattr(lib, name)
        f.argtypes, f.restype = [ctypes.c_char_p, vp], i32
        _fn[name] = f
    for name, args in (("s4_short_conv_bwd_workspace_bytes", [i32] * 4),
                       ("s4_selective_scan_workspace_bytes", [i32] * 5),
                       ("s4_selective_scan_bwd_workspace_bytes", [i32] * 5), ("s4_block_norm_bwd_workspace_bytes", [ll, i32])):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, sz
        _fn[name] = f
    return _fn


def _call(name, args, dev):
    f = _fn.get(name) or _lib()[name]
    code = f(args, _raw_stream(dev))
    if code:
        raise S4Error(code, name)


def _bytes(name, *sizes):
    n = (_fn.get(name) or _lib()[name])(*sizes)
    if n == 0:
        raise S4Error(1, name)
    return n


def _scratch(ws, dev, need=0, x=None):
    """(tensor, address, bytes) of a workspace; `need` bytes on x's GPU where there is none (0: none at all)."""
    if ws is None:
        if need == 0:
            return None, 0, 0
        ws = _empty(need, dtype=torch.uint8, device=x.device)
    elif not isinstance(ws, torch.Tensor):
        raise TypeError("ws must be a torch.Tensor")
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous on cuda:{dev}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _bad(t, name, dtype, shape, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{dev}")
    raise ValueError(f"{name}: its last dimension must be contiguous" if t.dim() > 1 and not t.is_contiguous()
                     else f"{name} must be contiguous")


def _dense(t, dtype, shape, dev, name):
    """Address of a contiguous tensor of this type and shape; 0 for None."""
    if t is None:
        return 0
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        _bad(t, name, dtype, shape, dev)
    return t.data_ptr()


def _rows(t, dtype, shape, dev, name):
    """(address, batch stride, row stride) of [batch, L, channels]; zeros for None."""
    if t is None:
        return 0, 0, 0
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != dev:
        _bad(t, name, dtype, shape, dev)
    sb, sr, sc = t.stride()
    if sc != 1 and shape[2] != 1:
        raise ValueError(f"{name}: its channels must be contiguous")
    return t.data_ptr(), sb, sr


def _tokens(t, dtype, shape, dev, name):
    """The same of one token per sequence, [batch, channels]."""
    if t is None:
        return 0, 0, 0
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != dev:
        _bad(t, name, dtype, shape, dev)
    sb, sc = t.stride()
    if sc != 1 and shape[1] != 1:
        raise ValueError(f"{name}: its channels must be contiguous")
    return t.data_ptr(), sb, sb


def _code(x):
    """The code of the activations' type and their GPU."""
    c = _DTYPES.get(x.dtype) if isinstance(x, torch.Tensor) else None
    if c is None:
        raise TypeError("activations must be float32, bfloat16 or float16 tensors")
    dev = x.get_device()
    if dev < 0:
        raise ValueError("activations must be CUDA tensors")
    return c, dev


def _away(x):
    """Whether the activations lie on another GPU than the current one."""
    dev = x.get_device() if isinstance(x, torch.Tensor) else -1
    return dev >= 0 and dev != _current()


def _on(stream, f, x, *args, **kw):
    """f on `stream`, or with x's GPU current."""
    if stream is None:
        with torch.cuda.device(x.get_device()):
            return f(x, *args, **kw)
    if isinstance(x, torch.Tensor) and x.get_device() >= 0 and stream.device != x.device:
        raise ValueError(f"the stream is {stream.device}'s, the activations are on {x.device}")
    with torch.cuda.stream(stream):
        return f(x, *args, **kw)


def _slots(state, state_out, batch, index):
    n = state.shape[0] if state is not None else state_out.shape[0] if state_out is not None else 0
    if n < batch and index is None and (state is not None or state_out is not None):
        raise ValueError(f"state: {n} slots for {batch} sequences and no index")
    return n


def s4_short_conv_fwd(x, w, bias=None, *, silu=True, lengths=None, state=None, state_out=None, index=None, y=None,
                      ws=None, stream=None):
    """y = silu(causal convolution of x [batch, L, H] with w [H, W] along L, plus bias).

    lengths [batch] int32: real tokens of each sequence.  state, state_out [slots, W-1, H] (x's type):
    the inputs before the first token and where the last ones go (the same tensor for in place;
    neither is needed); index [batch] int32: each sequence's slot, negative for none.  ws (256 bytes, see
    s4_get_status) records a length or slot out of range."""
    if stream is not None or _away(x):
        return _on(stream, s4_short_conv_fwd, x, w, bias, silu=silu, lengths=lengths, state=state, state_out=state_out,
                   index=index, y=y, ws=ws)
    (code, dev), dt, shape = _code(x), x.dtype, x.shape
    batch, L, H = shape
    W = w.shape[1]
    if y is None:
        y = _empty(shape, dtype=dt, device=x.device)
    slots = _slots(state, state_out, batch, index)
    _, wp, wn = _scratch(ws, dev)
    args = _CONV.pack(*_rows(x, dt, shape, dev, "x"), *_rows(y, dt, shape, dev, "y"), _dense(w, _F32, (H, W), dev, "w"),
                      _dense(bias, _F32, (H,), dev, "bias"), _dense(lengths, _I32, (batch,), dev, "lengths"),
                      _dense(index, _I32, (batch,), dev, "index"), _dense(state, dt, (slots, W - 1, H), dev, "state"),
                      _dense(state_out, dt, (slots, W - 1, H), dev, "state_out"),
                      wp, wn, batch, L, H, W, slots, code, 1 if silu else 0)
    _call("s4_short_conv_fwd", args, dev)
    return y


def s4_short_conv_step(x, w, bias, state, *, silu=True, state_out=None, index=None, y=None, ws=None, stream=None):
    """One token per sequence: x [batch, H] -> y [batch, H] (y may be x).  The state is updated in place, or
    written to state_out (the old one then stays, as for tokens that may be rejected)."""
    if stream is not None or _away(x):
        return _on(stream, s4_short_conv_step, x, w, bias, state, silu=silu, state_out=state_out, index=index, y=y, ws=ws)
    (code, dev), dt, shape = _code(x), x.dtype, x.shape
    batch, H = shape
    W = w.shape[1]
    if y is None:
        y = _empty(shape, dtype=dt, device=x.device)
    slots = _slots(state, state, batch, index)
    old = _dense(state, dt, (slots, W - 1, H), dev, "state")
    _, wp, wn = _scratch(ws, dev)
    args = _CONV.pack(*_tokens(x, dt, shape, dev, "x"), *_tokens(y, dt, shape, dev, "y"), _dense(w, _F32, (H, W), dev, "w"),
                      _dense(bias, _F32, (H,), dev, "bias"), 0, _dense(index, _I32, (batch,), dev, "index"), old,
                      old if state_out is None else _dense(state_out, dt, (slots, W - 1, H), dev, "state_out"),
                      wp, wn, batch, 1, H, W, slots, code, 1 if silu else 0)
    _call("s4_short_conv_fwd", args, dev)
    return y


def s4_short_conv_bwd(x, w, bias, dy, *, silu=True, lengths=None, state=None, dstate=None, want_dstate0=False, ws=None,
                      stream=None):
    """Gradients of s4_short_conv_fwd from dy: a dict of dx, dw, dbias (with a bias), and dstate0, the
    gradient of the state on entry, where asked for.  state, dstate [batch, W-1, H]: the state on
    entry and the gradient of the state on return (None: zeros)."""
    if stream is not None or _away(x):
        return _on(stream, s4_short_conv_bwd, x, w, bias, dy, silu=silu, lengths=lengths, state=state, dstate=dstate,
                   want_dstate0=want_dstate0, ws=ws)
    (code, dev), dt, shape, on = _code(x), x.dtype, x.shape, x.device
    batch, L, H = shape
    W = w.shape[1]
    ws, wp, wn = _scratch(ws, dev, _bytes("s4_short_conv_bwd_workspace_bytes", batch, L, H, W), x)
    out = {"dx": _empty(shape, dtype=dt, device=on), "dw": _empty((H, W), dtype=_F32, device=on)}
    if bias is not None:
        out["dbias"] = _empty((H,), dtype=_F32, device=on)
    if want_dstate0:
        out["dstate0"] = _empty((batch, W - 1, H), dtype=dt, device=on)
    past = (batch, W - 1, H)
    args = _CONV_BWD.pack(*_rows(x, dt, shape, dev, "x"), *_rows(dy, dt, shape, dev, "dy"),
                          *_rows(out["dx"], dt, shape, dev, "dx"),
                          _dense(w, _F32, (H, W), dev, "w"), _dense(bias, _F32, (H,), dev, "bias"),
                          _dense(lengths, _I32, (batch,), dev, "lengths"), _dense(state, dt, past, dev, "state"),
                          _dense(dstate, dt, past, dev, "dstate"), _dense(out.get("dstate0"), dt, past, dev, "dstate0"),
                          out["dw"].data_ptr(), _dense(out.get("dbias"), _F32, (H,), dev, "dbias"),
                          wp, wn, batch, L, H, W, code, 1 if silu else 0)
    _call("s4_short_conv_bwd", args, dev)
    return out


def _groups(t, dtype, shape, dev, name):
    """(address, batch, row and group strides) of [batch, L, G, N], or of one token's [batch, G, N]."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != dev:
        _bad(t, name, dtype, shape, dev)
    s = t.stride()
    if s[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name}: its states must be contiguous")
    return t.data_ptr(), s[0], s[-3], s[-2]


def s4_selective_scan_fwd(x, dt, A, B, C, *, D=None, z=None, dt_bias=None, softplus=True, lengths=None, state=None,
                          state_out=None, index=None, y=None, ws=None, stream=None):
    """The selective state-space scan: s = exp(d A) s + d x B, y = (C.s + D x) silu(z) with
    d = softplus(dt + dt_bias), along L.

    x, dt, z [batch, L, H]; A [H, N]; B, C [batch, L, G, N] (channels in G equal groups);
    D, dt_bias [H].  lengths, index as for s4_short_conv_fwd; state, state_out [slots, H, N]
    float32.  ws: s4_selective_scan_workspace_bytes (allocated per call when None)."""
    if stream is not None or _away(x):
        return _on(stream, s4_selective_scan_fwd, x, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, softplus=softplus,
                   lengths=lengths, state=state, state_out=state_out, index=index, y=y, ws=ws)
    (code, dev), ty, shape = _code(x), x.dtype, x.shape
    batch, L, H = shape
    G, N = B.shape[2:]
    if y is None:
        y = _empty(shape, dtype=ty, device=x.device)
    slots = _slots(state, state_out, batch, index)
    need = _bytes("s4_selective_scan_workspace_bytes", batch, L, H, N, G) if ws is None else 0
    ws, wp, wn = _scratch(ws, dev, need if need > 256 else 0, x)
    bp, bb, br, bg = _groups(B, ty, (batch, L, G, N), dev, "B")
    cp, cb, cr, cg = _groups(C, ty, (batch, L, G, N), dev, "C")
    args = _SCAN.pack(*_rows(x, ty, shape, dev, "x"), *_rows(dt, ty, shape, dev, "dt"), *_rows(z, ty, shape, dev, "z"),
                      bp, bb, br, cp, cb, cr, *_rows(y, ty, shape, dev, "y"), _dense(A, _F32, (H, N), dev, "A"),
                      _dense(D, _F32, (H,), dev, "D"), _dense(dt_bias, _F32, (H,), dev, "dt_bias"),
                      _dense(lengths, _I32, (batch,), dev, "lengths"), _dense(index, _I32, (batch,), dev, "index"),
                      _dense(state, _F32, (slots, H, N), dev, "state"),
                      _dense(state_out, _F32, (slots, H, N), dev, "state_out"),
                      wp, wn, bg, cg,
                      batch, L, H, N, G, slots, code, 1 if softplus else 0)
    _call("s4_selective_scan_fwd", args, dev)
    return y


def s4_selective_step(x, dt, A, B, C, state, *, D=None, z=None, dt_bias=None, softplus=True, state_out=None, index=None,
                      y=None, ws=None, stream=None):
    """One token per sequence: x, dt, z [batch, H], B, C [batch, G, N] -> y [batch, H].  The state is
    updated in place, or written to state_out."""
    if stream is not None or _away(x):
        return _on(stream, s4_selective_step, x, dt, A, B, C, state, D=D, z=z, dt_bias=dt_bias, softplus=softplus,
                   state_out=state_out, index=index, y=y, ws=ws)
    (code, dev), ty, shape = _code(x), x.dtype, x.shape
    batch, H = shape
    G, N = B.shape[1:]
    if y is None:
        y = _empty(shape, dtype=ty, device=x.device)
    slots = _slots(state, state, batch, index)
    old = _dense(state, _F32, (slots, H, N), dev, "state")
    _, wp, wn = _scratch(ws, dev)
    bp, bb, br, bg = _groups(B, ty, (batch, G, N), dev, "B")
    cp, cb, cr, cg = _groups(C, ty, (batch, G, N), dev, "C")
    args = _SCAN.pack(*_tokens(x, ty, shape, dev, "x"), *_tokens(dt, ty, shape, dev, "dt"), *_tokens(z, ty, shape, dev, "z"),
                      bp, bb, br, cp, cb, cr, *_tokens(y, ty, shape, dev, "y"), _dense(A, _F32, (H, N), dev, "A"),
                      _dense(D, _F32, (H,), dev, "D"), _dense(dt_bias, _F32, (H,), dev, "dt_bias"), 0,
                      _dense(index, _I32, (batch,), dev, "index"), old,
                      old if state_out is None else _dense(state_out, _F32, (slots, H, N), dev, "state_out"),
                      wp, wn, bg, cg,
                      batch, 1, H, N, G, slots, code, 1 if softplus else 0)
    _call("s4_selective_scan_fwd", args, dev)
    return y


def s4_selective_scan_bwd(x, dt, A, B, C, dy, *, D=None, z=None, dt_bias=None, softplus=True, lengths=None, state=None,
                          dstate=None, want_dstate0=False, ws=None, stream=None):
    """Gradients of s4_selective_scan_fwd from dy: a dict of dx, ddt, dA, dB, dC and, for what was given, dD, dz,
    ddt_bias; dstate0, the gradient of the state on entry, where asked for.  state, dstate [batch, H, N]: the
    state on entry and the gradient of the state on return (None: zeros).  Nothing is kept from the
    forward call: its states are formed again.  ws: s4_selective_scan_bwd_workspace_bytes."""
    if stream is not None or _away(x):
        return _on(stream, s4_selective_scan_bwd, x, dt, A, B, C, dy, D=D, z=z, dt_bias=dt_bias, softplus=softplus,
                   lengths=lengths, state=state, dstate=dstate, want_dstate0=want_dstate0, ws=ws)
    (code, dev), ty, shape, on = _code(x), x.dtype, x.shape, x.device
    batch, L, H = shape
    vec = B.shape
    G, N = vec[2:]
    ws, wp, wn = _scratch(ws, dev, _bytes("s4_selective_scan_bwd_workspace_bytes", batch, L, H, N, G), x)
    out = {"dx": _empty(shape, dtype=ty, device=on), "ddt": _empty(shape, dtype=ty, device=on),
           "dA": _empty((H, N), dtype=_F32, device=on), "dB": _empty(vec, dtype=ty, device=on),
           "dC": _empty(vec, dtype=ty, device=on)}
    if D is not None:
        out["dD"] = _empty((H,), dtype=_F32, device=on)
    if z is not None:
        out["dz"] = _empty(shape, dtype=ty, device=on)
    if dt_bias is not None:
        out["ddt_bias"] = _empty((H,), dtype=_F32, device=on)
    if want_dstate0:
        out["dstate0"] = _empty((batch, H, N), dtype=_F32, device=on)
    get = out.get
    bp, bb, br, bg = _groups(B, ty, (batch, L, G, N), dev, "B")
    cp, cb, cr, cg = _groups(C, ty, (batch, L, G, N), dev, "C")
    past = (batch, H, N)
    args = _SCAN_BWD.pack(
        *_rows(x, ty, shape, dev, "x"), *_rows(dt, ty, shape, dev, "dt"), *_rows(z, ty, shape, dev, "z"),
        bp, bb, br, cp, cb, cr, *_rows(dy, ty, shape, dev, "dy"), *_rows(out["dx"], ty, shape, dev, "dx"),
        *_rows(out["ddt"], ty, shape, dev, "ddt"), *_rows(get("dz"), ty, shape, dev, "dz"), out["dB"].data_ptr(),
        out["dC"].data_ptr(), _dense(A, _F32, (H, N), dev, "A"), _dense(D, _F32, (H,), dev, "D"),
        _dense(dt_bias, _F32, (H,), dev, "dt_bias"), _dense(lengths, _I32, (batch,), dev, "lengths"),
        _dense(state, _F32, past, dev, "state"), _dense(dstate, _F32, past, dev, "dstate"),
        _dense(get("dstate0"), _F32, past, dev, "dstate0"), out["dA"].data_ptr(), _dense(get("dD"), _F32, (H,), dev, "dD"),
        _dense(get("ddt_bias"), _F32, (H,), dev, "ddt_bias"), wp, wn, bg, cg,
        batch, L, H, N, G, code, 1 if softplus else 0)
    _call("s4_selective_scan_bwd", args, dev)
    return out


def _flat(t, dtype, shape, dev, name):
    """(address, row stride) of [rows, H], or of leading dimensions that make rows of one stride."""
    if t is None:
        return 0, 0
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != dev:
        _bad(t, name, dtype, shape, dev)
    if len(shape) != 2:
        t = t.view(-1, shape[-1])
    sr, sc = t.stride()
    if sc != 1 and shape[-1] != 1:
        raise ValueError(f"{name}: its channels must be contiguous")
    return t.data_ptr(), sr


def _residual(h, dtype):
    if h is not None and h.dtype != dtype and h.dtype != _F32:
        raise TypeError(f"h: dtype {h.dtype}, expected {dtype} or float32")
    return dtype if h is None else h.dtype


def s4_block_norm_fwd(o, *, w_post=None, gate=None, scale=None, h=None, w_pre=None, eps=1e-5, h_out=None, y=None,
                      stream=None):
    """What joins two blocks: h_out = h + scale * norm(o * silu(gate)) * w_post and
    y = norm(h_out) * w_pre, norm(v) = v / sqrt(mean(v^2) + eps) over the last dimension.

    o, gate [..., H] of one type; h [..., H] of that type or float32, and h_out of h's (h_out may be h);
    w_post, scale, w_pre [H].  What is None is left out: without gate no gating, without w_post no
    first norm, without h nothing is added.  Returns (h_out, y), y None without w_pre."""
    if stream is not None or _away(o):
        return _on(stream, s4_block_norm_fwd, o, w_post=w_post, gate=gate, scale=scale, h=h, w_pre=w_pre, eps=eps,
                   h_out=h_out, y=y)
    (code, dev), dt, shape, on = _code(o), o.dtype, o.shape, o.device
    H = shape[-1]
    res = _residual(h if h is not None else h_out, dt)
    if h_out is None:
        h_out = _empty(shape, dtype=res, device=on)
    if y is None and w_pre is not None:
        y = _empty(shape, dtype=dt, device=on)
    po, so = _flat(o, dt, shape, dev, "o")
    pg, sg = _flat(gate, dt, shape, dev, "gate")
    ph, sh = _flat(h, res, shape, dev, "h")
    pq, sq = _flat(h_out, res, shape, dev, "h_out")
    py, sy = _flat(y, dt, shape, dev, "y")
    args = _NORM.pack(po, pg, ph, pq, py, _dense(w_post, _F32, (H,), dev, "w_post"), _dense(scale, _F32, (H,), dev, "scale"),
                      _dense(w_pre, _F32, (H,), dev, "w_pre"), so, sg, sh, sq, sy, o.numel() // H if H else 0, eps, H, code,
                      1 if res is _F32 else 0)
    _call("s4_block_norm_fwd", args, dev)
    return h_out, y


def s4_block_norm_bwd(o, dy=None, *, dh_out=None, w_post=None, gate=None, scale=None, h=None, w_pre=None, eps=1e-5,
                      ws=None, stream=None):
    """Gradients of s4_block_norm_fwd from dy and dh_out (None: zeros; not both): a dict of do and, for
    what was given, dgate, dh, dw_post, dscale and dw_pre."""
    if stream is not None or _away(o):
        return _on(stream, s4_block_norm_bwd, o, dy, dh_out=dh_out, w_post=w_post, gate=gate, scale=scale, h=h,
                   w_pre=w_pre, eps=eps, ws=ws)
    (code, dev), dt, shape, on = _code(o), o.dtype, o.shape, o.device
    H = shape[-1]
    rows = o.numel() // H if H else 0
    res = _residual(h if h is not None else dh_out, dt)
    ws, wp, wn = _scratch(ws, dev, _bytes("s4_block_norm_bwd_workspace_bytes", rows, H), o)
    out = {"do": _empty(shape, dtype=dt, device=on)}
    if gate is not None:
        out["dgate"] = _empty(shape, dtype=dt, device=on)
    if h is not None:
        out["dh"] = _empty(shape, dtype=res, device=on)
    for k, v in (("dw_post", w_post), ("dscale", scale), ("dw_pre", w_pre)):
        if v is not None:
            out[k] = _empty((H,), dtype=_F32, device=on)
    po, so = _flat(o, dt, shape, dev, "o")
    pg, sg = _flat(gate, dt, shape, dev, "gate")
    ph, sh = _flat(h, res, shape, dev, "h")
    py, sy = _flat(dy, dt, shape, dev, "dy")
    pq, sq = _flat(dh_out, res, shape, dev, "dh_out")
    get = out.get
    args = _NORM_BWD.pack(po, pg, ph, py, pq, out["do"].data_ptr(), _dense(get("dgate"), dt, shape, dev, "dgate"),
                          _dense(get("dh"), res, shape, dev, "dh"), _dense(w_post, _F32, (H,), dev, "w_post"),
                          _dense(scale, _F32, (H,), dev, "scale"), _dense(w_pre, _F32, (H,), dev, "w_pre"),
                          _dense(get("dw_post"), _F32, (H,), dev, "dw_post"),
                          _dense(get("dscale"), _F32, (H,), dev, "dscale"),
                          _dense(get("dw_pre"), _F32, (H,), dev, "dw_pre"), wp, wn,
                          so, sg, sh, sy, sq, H, H, H, rows, eps, H, code, 1 if res is _F32 else 0)
    _call("s4_block_norm_bwd", args, dev)
    return out
