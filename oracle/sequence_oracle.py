"""Linear attention with a decay for each head, rotary positions, layer norm and the vocabulary loss in float64 numpy,
token by token or row by row from their definitions: test infrastructure only."""
import numpy as np


def linear_attention(q, k, v, g, scale, lengths=None, state=None):
    """q [B, L, H, K], k [B, L, G, K], v [B, L, G, V] -> o [B, L, H, V] and the states [B, H, K, V] after the last
    real tokens."""
    B, L, H, K = q.shape
    each, V = H // k.shape[2], v.shape[3]
    k, v = np.repeat(k, each, 2), np.repeat(v, each, 2)
    lengths = [L] * B if lengths is None else lengths
    o, s = np.zeros((B, L, H, V)), np.zeros((B, H, K, V)) if state is None else np.array(state, dtype=np.float64)
    f = np.exp(g)[:, None, None]
    for b in range(B):
        for t in range(int(lengths[b])):
            s[b] = f * s[b] + k[b, t][:, :, None] * v[b, t][:, None, :]
            o[b, t] = scale * np.einsum("hk,hkv->hv", q[b, t], s[b])
    return o, s


def linear_attention_grad(q, k, v, g, do, scale, lengths=None, state=None, dstate=None):
    """dq, dk, dv and dstate0."""
    B, L, H, K = q.shape
    G, V = k.shape[2], v.shape[3]
    kk, vv = np.repeat(k, H // G, 2), np.repeat(v, H // G, 2)
    lengths = [L] * B if lengths is None else lengths
    dq, dk, dv = np.zeros(q.shape), np.zeros(kk.shape), np.zeros(vv.shape)
    s = np.zeros((B, H, K, V)) if state is None else np.array(state, dtype=np.float64)
    r = np.zeros((B, H, K, V)) if dstate is None else np.array(dstate, dtype=np.float64)
    f = np.exp(g)[:, None, None]
    for b in range(B):
        for t in range(int(lengths[b])):
            s[b] = f * s[b] + kk[b, t][:, :, None] * vv[b, t][:, None, :]
            dq[b, t] = scale * np.einsum("hkv,hv->hk", s[b], do[b, t])
        for t in reversed(range(int(lengths[b]))):
            r[b] = r[b] + scale * q[b, t][:, :, None] * do[b, t][:, None, :]
            dk[b, t] = np.einsum("hkv,hv->hk", r[b], vv[b, t])
            dv[b, t] = np.einsum("hkv,hk->hv", r[b], kk[b, t])
            r[b] = f * r[b]
    dk, dv = (x.reshape(B, L, G, H // G, -1).sum(3) for x in (dk, dv))
    return {"dq": dq, "dk": dk, "dv": dv, "dstate0": r}


def rotary(x, freqs, positions, pairs, amplitude=1.0, sign=1.0):
    """x [B, L, H, D], positions [B, L]."""
    y, R = np.array(x, dtype=np.float64), len(freqs)
    t = np.asarray(positions, dtype=np.float64)[:, :, None, None] * freqs
    c, s = amplitude * np.cos(t), sign * amplitude * np.sin(t)
    i = np.arange(R)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, R + i)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def layer_norm(x, w=None, b=None, eps=1e-5):
    u = x - x.mean(-1, keepdims=True)
    u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    return u * (1.0 if w is None else w) + (0.0 if b is None else b)


def layer_norm_grad(x, dy, w=None, eps=1e-5):
    u = x - x.mean(-1, keepdims=True)
    r = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    u = u * r
    d = dy * (1.0 if w is None else w)
    lead = tuple(range(x.ndim - 1))
    return {"dx": r * (d - d.mean(-1, keepdims=True) - u * (d * u).mean(-1, keepdims=True)), "dw": (dy * u).sum(lead),
            "db": dy.sum(lead)}


def vocab_loss(h, w, targets):
    """Losses [rows] and lse of h [rows, H] against w [V, H]."""
    x = h @ w.T
    m = x.max(-1)
    lse = m + np.log(np.exp(x - m[:, None]).sum(-1))
    rows = np.arange(len(h))
    return np.where(targets >= 0, lse - x[rows, np.maximum(targets, 0)], 0.0), lse


def vocab_loss_grad(h, w, targets, dloss):
    x = h @ w.T
    _, lse = vocab_loss(h, w, targets)
    g = np.exp(x - lse[:, None])
    g[np.arange(len(h)), np.maximum(targets, 0)] -= 1
    g *= np.where(targets >= 0, dloss, 0.0)[:, None]
    return {"dh": g @ w, "dw": g.T @ h}
