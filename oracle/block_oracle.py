"""Float64 CPU definitions of the selective block's operators and of their gradients (test
infrastructure): the short causal convolution, the selective scan and the norms around a block.

Plain numpy, one token after the other, written from the formulas; the gradients are
written out by hand and pinned against central differences of the forward definitions
by tests/test_block_oracle.py."""
import numpy as np


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def silu(v):
    return v * sigmoid(v)


def silu_grad(v):
    s = sigmoid(v)
    return s * (1 + v * (1 - s))


def softplus(v):
    return np.logaddexp(v, 0.0)


def _lens(lengths, batch, L):
    return [L] * batch if lengths is None else [int(n) for n in lengths]


# ---- short causal convolution -----------------------------------------------------------------------

def short_conv(x, w, bias=None, act=True, lengths=None, state=None):
    """x [B][L][H], w [H][W], state [B][W-1][H] -> y, state after the last real token."""
    B, L, H = x.shape
    W = w.shape[1]
    y = np.zeros((B, L, H))
    new = np.zeros((B, W - 1, H))
    for b, n in enumerate(_lens(lengths, B, L)):
        past = np.zeros((W - 1, H)) if state is None else state[b]
        seen = np.concatenate([past, x[b, :n]])
        for t in range(n):
            v = sum(w[:, k] * seen[t + k] for k in range(W)) + (0.0 if bias is None else bias)
            y[b, t] = silu(v) if act else v
        new[b] = seen[n:]
    return y, new


def short_conv_grad(x, w, bias, dy, act=True, lengths=None, state=None, dstate=None):
    """Gradients of sum(y dy) + sum(new state dstate): dict of dx, dw, dbias, dstate0."""
    B, L, H = x.shape
    W = w.shape[1]
    dx, dw, db = np.zeros((B, L, H)), np.zeros((H, W)), np.zeros(H)
    d0 = np.zeros((B, W - 1, H))
    for b, n in enumerate(_lens(lengths, B, L)):
        past = np.zeros((W - 1, H)) if state is None else state[b]
        seen = np.concatenate([past, x[b, :n]])
        dseen = np.zeros_like(seen)
        if dstate is not None:
            dseen[n:] += dstate[b]
        for t in range(n):
            v = sum(w[:, k] * seen[t + k] for k in range(W)) + (0.0 if bias is None else bias)
            dv = dy[b, t] * silu_grad(v) if act else dy[b, t]
            db += dv
            for k in range(W):
                dw[:, k] += dv * seen[t + k]
                dseen[t + k] += dv * w[:, k]
        d0[b] = dseen[:W - 1]
        dx[b, :n] = dseen[W - 1:]
    return {"dx": dx, "dw": dw, "dbias": db, "dstate0": d0}


# ---- selective scan ---------------------------------------------------------------------------------

def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, soft=True, lengths=None, state=None):
    """x, dt, z [b][L][H]; A [H][N]; B, C [b][L][G][N]; state [b][H][N] -> y, state after the last real token."""
    nb, L, H = x.shape
    G, N = B.shape[2:]
    y = np.zeros((nb, L, H))
    new = np.zeros((nb, H, N))
    of = np.arange(H) // (H // G)
    for b, n in enumerate(_lens(lengths, nb, L)):
        s = np.zeros((H, N)) if state is None else state[b].astype(float).copy()
        for t in range(n):
            d = dt[b, t] + (0.0 if dt_bias is None else dt_bias)
            d = softplus(d) if soft else d
            s = np.exp(d[:, None] * A) * s + (d * x[b, t])[:, None] * B[b, t][of]
            v = (s * C[b, t][of]).sum(1) + (0.0 if D is None else D * x[b, t])
            y[b, t] = v if z is None else v * silu(z[b, t])
        new[b] = s
    return y, new


def selective_scan_grad(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, soft=True, lengths=None, state=None,
                        dstate=None):
    """Gradients of sum(y dy) + sum(new state dstate) with respect to every input."""
    nb, L, H = x.shape
    G, N = B.shape[2:]
    of = np.arange(H) // (H // G)
    out = {"dx": np.zeros((nb, L, H)), "ddt": np.zeros((nb, L, H)), "dA": np.zeros((H, N)),
           "dB": np.zeros((nb, L, G, N)), "dC": np.zeros((nb, L, G, N)), "dD": np.zeros(H),
           "dz": np.zeros((nb, L, H)), "ddt_bias": np.zeros(H), "dstate0": np.zeros((nb, H, N))}
    for b, n in enumerate(_lens(lengths, nb, L)):
        s = np.zeros((n + 1, H, N))
        if state is not None:
            s[0] = state[b]
        raw = dt[b, :n] + (0.0 if dt_bias is None else dt_bias)
        d = softplus(raw) if soft else raw
        for t in range(n):
            s[t + 1] = np.exp(d[t][:, None] * A) * s[t] + (d[t] * x[b, t])[:, None] * B[b, t][of]
        carry = np.zeros((H, N)) if dstate is None else dstate[b].astype(float).copy()
        for t in range(n - 1, -1, -1):
            g_out = dy[b, t]
            if z is not None:
                v = (s[t + 1] * C[b, t][of]).sum(1) + (0.0 if D is None else D * x[b, t])
                out["dz"][b, t] = g_out * v * silu_grad(z[b, t])
                g_out = g_out * silu(z[b, t])
            a = np.exp(d[t][:, None] * A)
            g = C[b, t][of] * g_out[:, None] + carry
            u = (g * B[b, t][of]).sum(1)
            q = g * a * s[t]
            out["dC"][b, t] = (g_out[:, None] * s[t + 1]).reshape(G, -1, N).sum(1)
            out["dB"][b, t] = (g * (d[t] * x[b, t])[:, None]).reshape(G, -1, N).sum(1)
            out["dx"][b, t] = d[t] * u + (0.0 if D is None else D * g_out)
            out["dD"] += g_out * x[b, t]
            out["dA"] += d[t][:, None] * q
            dd = x[b, t] * u + (q * A).sum(1)
            out["ddt"][b, t] = dd * sigmoid(raw[t]) if soft else dd
            out["ddt_bias"] += out["ddt"][b, t]
            carry = a * g
        out["dstate0"][b] = carry
    return out


# ---- norms around a block ---------------------------------------------------------------------------

def block_norm(o, gate=None, h=None, w_post=None, scale=None, w_pre=None, eps=1e-5):
    """o, gate, h [R][H] -> h_out, y (None without w_pre)."""
    v = o if gate is None else o * silu(gate)
    p = v if w_post is None else v / np.sqrt((v * v).mean(1, keepdims=True) + eps) * w_post
    h2 = (0.0 if h is None else h) + (p if scale is None else scale * p)
    y = None if w_pre is None else h2 / np.sqrt((h2 * h2).mean(1, keepdims=True) + eps) * w_pre
    return h2, y


def block_norm_grad(o, dy=None, dh_out=None, gate=None, h=None, w_post=None, scale=None, w_pre=None, eps=1e-5):
    """Gradients of sum(y dy) + sum(h_out dh_out)."""
    v = o if gate is None else o * silu(gate)
    r1 = 1.0 if w_post is None else 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    unit = v * r1
    p = unit if w_post is None else unit * w_post
    h2 = (0.0 if h is None else h) + (p if scale is None else scale * p)
    out = {}
    dh = np.zeros_like(v) if dh_out is None else dh_out.astype(float)
    if dy is not None:
        r2 = 1 / np.sqrt((h2 * h2).mean(1, keepdims=True) + eps)
        unit2 = h2 * r2
        out["dw_pre"] = (dy * unit2).sum(0)
        d = dy * w_pre
        dh = dh + r2 * (d - unit2 * (d * unit2).mean(1, keepdims=True))
    out["dh"] = dh
    if scale is not None:
        out["dscale"] = (dh * p).sum(0)
    dp = dh if scale is None else dh * scale
    dv = dp
    if w_post is not None:
        out["dw_post"] = (dp * unit).sum(0)
        d = dp * w_post
        dv = r1 * (d - unit * (d * unit).mean(1, keepdims=True))
    if gate is None:
        out["do"] = dv
    else:
        out["do"] = dv * silu(gate)
        out["dgate"] = dv * o * silu_grad(gate)
    return out
