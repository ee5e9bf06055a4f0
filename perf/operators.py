"""Cases of the selective state-space block's operators, their plain forms and their definitions in 64 bits.

Three operators, each with the forms a model needs:

* ``conv``: the short causal convolution along time, one filter of a few taps per channel, with SiLU
  (``step``: one token per sequence; ``prompt``: whole prompts of ragged lengths; ``grad``: the backward pass);
* ``scan``: the selective state-space scan, whose step size, input and output vectors change with every token
  (the same three forms);
* ``norm``: the norms after and before a block, fused with the block's gate, its residual scale and the residual sum
  (``forward`` and ``grad``).

``prepare`` makes a case's inputs, ``run`` is one pass over them: through the library's entry points where ``own`` is
true, in elementary torch operations in 32 bits where it is false.
"""
import math
import random

import torch

own = False

DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
EPS = 1e-5


# ---- cases ------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token each for a few sequences: a call that is all latency
        dict(name="conv-step-8x1024", op="conv", form="step", batch=8, L=1, H=1024, W=4, slots=16, dtype="bfloat16"),
        # a ragged batch of prompts, one of them empty, the last inputs of each kept for decoding
        dict(name="conv-prompt-8x1023x1024", op="conv", form="prompt", batch=8, L=1023, H=1024, W=4, slots=8,
             dtype="float16"),
        # a training batch's backward pass
        dict(name="conv-grad-8x4096x2048", op="conv", form="grad", batch=8, L=4096, H=2048, W=4, slots=0,
             dtype="bfloat16"),
        # decoding for one user
        dict(name="scan-step-1x1024", op="scan", form="step", batch=1, L=1, H=1024, N=16, G=1, slots=1,
             dtype="bfloat16"),
        # decoding for many users at once: the states of a large cache, some rows of the batch not in use
        dict(name="scan-step-256x2048", op="scan", form="step", batch=256, L=1, H=2048, N=16, G=1, slots=320,
             dtype="bfloat16"),
        # a ragged batch of prompts into the cache
        dict(name="scan-prompt-4x1500x2048", op="scan", form="prompt", batch=4, L=1500, H=2048, N=16, G=1, slots=4,
             dtype="bfloat16"),
        # one document of the greatest length, channels and length those of the library's largest workload
        dict(name="scan-prompt-1x65536x1024", op="scan", form="prompt", batch=1, L=65536, H=1024, N=16, G=1, slots=1,
             dtype="bfloat16"),
        # a training batch's backward pass
        dict(name="scan-grad-4x4096x2048", op="scan", form="grad", batch=4, L=4096, H=2048, N=16, G=1, slots=0,
             dtype="bfloat16"),
        # an odd length in 32 bits with a wider state and two groups of input and output vectors
        dict(name="scan-grad-2x333x256", op="scan", form="grad", batch=2, L=333, H=256, N=64, G=2, slots=0,
             dtype="float32"),
        # the norms around a block while decoding
        dict(name="norm-forward-8x1024", op="norm", form="forward", rows=8, H=1024, dtype="bfloat16"),
        # a long prompt's rows, an odd number of them
        dict(name="norm-forward-16001x2560", op="norm", form="forward", rows=16001, H=2560, dtype="float16"),
        # a training batch's backward pass
        dict(name="norm-grad-16384x2048", op="norm", form="grad", rows=16384, H=2048, dtype="bfloat16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _width(rng, lo, hi):
    """A number of channels: a usual one twice of three times, else any."""
    usual = [n for n in (64, 128, 192, 256, 384, 512, 768, 1024, 1280, 2048, 2560, 4096, 5120, 8192) if n <= hi]
    return rng.choice(usual) if rng.random() < 0.67 else _log(rng, lo, hi) // 2 * 2 + 1


def draw(rng):
    op, form = rng.choice([("conv", "step"), ("conv", "prompt"), ("conv", "grad"), ("scan", "step"),
                           ("scan", "prompt"), ("scan", "grad"), ("norm", "forward"), ("norm", "grad")])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    if op == "norm":
        H = _width(rng, 64, 8192)
        rows = _log(rng, 1, max(1, min(32768, (1 << 25) // H)))
        return dict(op=op, form=form, rows=rows, H=H, dtype=dtype)
    G = rng.choice([1, 1, 1, 2, 4]) if op == "scan" else 1
    H = max(1, _width(rng, 32, 4096) // G) * G
    c = dict(op=op, form=form, H=H, dtype=dtype)
    if op == "conv":
        c["W"] = rng.choice([2, 3, 4, 4, 4, 5, 8])
        most, cells = 1 << 26, H
    else:
        c["N"] = rng.choice([16, 16, 16, 8, 64, 128, rng.randint(1, 256)])
        c["G"] = G
        most, cells = (1 << 29) if form != "step" else (1 << 23), H * c["N"]
    if form == "step":
        c["batch"], c["L"] = _log(rng, 1, max(1, min(512, most // cells))), 1
    else:
        c["L"] = _log(rng, 1, max(1, min(65536, most // cells)))
        c["batch"] = _log(rng, 1, max(1, min(16, most // cells // c["L"])))
    c["slots"] = 0 if form == "grad" else c["batch"] + rng.choice([0, 0, 1, c["batch"] // 4 + 1])
    return c


def _lengths(case):
    """How many tokens of each sequence are real: the first has them all, one of three or more none, the others any."""
    n, L, rng = case["batch"], case["L"], random.Random("lengths %(batch)d %(L)d %(H)d" % case)
    got = [L] + [rng.randint(1, L) for _ in range(n - 1)]
    return got[:2] + [0] + got[3:] if n > 2 else got


def _slots(case):
    """The cache slot of each sequence; while decoding, some rows of a batch of 8 or more have none (-1)."""
    rng = random.Random("slots %(batch)d %(slots)d %(H)d" % case)
    got = rng.sample(range(case["slots"]), case["batch"])
    if case["form"] == "step" and case["batch"] >= 8:
        for i in rng.sample(range(case["batch"]), case["batch"] // 8):
            got[i] = -1
    return got


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    def uniform(*shape, lo, hi):
        return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo

    H = case["H"]
    s = {"op": case["op"], "form": case["form"]}
    if case["op"] == "norm":
        rows = case["rows"]
        # a projection writes the block's output; the gate is one half of another projection's output
        s["o"] = normal(rows, H, dtype=dtype)
        s["gate"] = normal(rows, 2 * H, dtype=dtype)[:, H:]
        s["h"] = normal(rows, H, scale=2.0)  # the residual stream is kept in 32 bits
        s["w_post"] = 1 + normal(H, scale=0.1)
        s["w_pre"] = 1 + normal(H, scale=0.1)
        s["scale"] = uniform(H, lo=0.1, hi=1.0)
        if case["form"] == "grad":
            s["dy"] = normal(rows, H, dtype=dtype)
            s["dh_out"] = normal(rows, H)
        return s

    batch, L, form = case["batch"], case["L"], case["form"]
    shape = (batch,) if form == "step" else (batch, L)
    if form != "grad":
        index = _slots(case)
        s["index"] = torch.tensor(index, dtype=torch.int32, device="cuda")
        s["rows"] = torch.tensor([b for b in range(batch) if index[b] >= 0], device="cuda")
        s["at"] = torch.tensor([i for i in index if i >= 0], device="cuda")
    if form == "prompt":
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    # the block's input projection writes x and z side by side
    xz = normal(*shape, 2 * H, dtype=dtype)
    s["x"], s["z"] = xz[..., :H], xz[..., H:]
    if case["op"] == "conv":
        del s["z"]
        W = case["W"]
        s["w"], s["bias"] = normal(H, W, scale=W ** -0.5), normal(H, scale=0.1)
        if form == "grad":
            s["dy"] = normal(*shape, H, dtype=dtype)
        else:
            s["state"] = normal(case["slots"], W - 1, H, dtype=dtype)
            s["state_out"] = s["state"].clone()
        return s
    N, G = case["N"], case["G"]
    # B and C are slices of one projection's output, behind the low-rank part of dt
    rank = (H + 15) // 16
    bc = normal(*shape, rank + 2 * G * N, dtype=dtype)[..., rank:]
    s["B"] = bc[..., :G * N].unflatten(-1, (G, N))
    s["C"] = bc[..., G * N:].unflatten(-1, (G, N))
    # steps of 1e-3 to 1e-1 after the softplus, spread by the token
    step = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["dt"] = normal(*shape, H, scale=0.5, dtype=dtype)
    s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(normal(H, N, scale=0.1))
    s["D"] = 1 + normal(H, scale=0.1)
    if form == "grad":
        s["dy"] = normal(*shape, H, dtype=dtype)
    else:
        s["state"] = normal(case["slots"], H, N, scale=0.1)
        s["state_out"] = s["state"].clone()
    return s


def run(s):
    return (_own if own else _plain)[s["op"] + "-" + s["form"]](s)


# ---- through the library ----------------------------------------------------------------------------------

def _own_conv_step(s):
    import structured_state_space_gb300 as s4
    y = s4.s4_short_conv_step(s["x"], s["w"], s["bias"], s["state"], state_out=s["state_out"], index=s["index"])
    return {"y": y, "state": s["state_out"]}


def _own_conv_prompt(s):
    import structured_state_space_gb300 as s4
    y = s4.s4_short_conv_fwd(s["x"], s["w"], s["bias"], lengths=s["lengths"], state=s["state"],
                             state_out=s["state_out"], index=s["index"])
    return {"y": y, "state": s["state_out"]}


def _own_conv_grad(s):
    import structured_state_space_gb300 as s4
    return s4.s4_short_conv_bwd(s["x"], s["w"], s["bias"], s["dy"])


def _own_scan_step(s):
    import structured_state_space_gb300 as s4
    y = s4.s4_selective_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"],
                             dt_bias=s["dt_bias"], state_out=s["state_out"], index=s["index"])
    return {"y": y, "state": s["state_out"]}


def _own_scan_prompt(s):
    import structured_state_space_gb300 as s4
    y = s4.s4_selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                                 lengths=s["lengths"], state=s["state"], state_out=s["state_out"], index=s["index"])
    return {"y": y, "state": s["state_out"]}


def _own_scan_grad(s):
    import structured_state_space_gb300 as s4
    return s4.s4_selective_scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["dy"], D=s["D"], z=s["z"],
                                    dt_bias=s["dt_bias"])


def _own_norm_forward(s):
    import structured_state_space_gb300 as s4
    h, y = s4.s4_block_norm_fwd(s["o"], w_post=s["w_post"], gate=s["gate"], scale=s["scale"], h=s["h"],
                                w_pre=s["w_pre"], eps=EPS)
    return {"h": h, "y": y}


def _own_norm_grad(s):
    import structured_state_space_gb300 as s4
    return s4.s4_block_norm_bwd(s["o"], s["dy"], dh_out=s["dh_out"], w_post=s["w_post"], gate=s["gate"],
                                scale=s["scale"], h=s["h"], w_pre=s["w_pre"], eps=EPS)


# ---- the plain forms --------------------------------------------------------------------------------------

def _silu_grad(v):
    sig = torch.sigmoid(v)
    return sig * (1 + v * (1 - sig))


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _put(s, new):
    """The new states at their slots; slots that no sequence has keep what they hold."""
    return s["state_out"].index_copy(0, s["at"], new.index_select(0, s["rows"]).to(s["state_out"].dtype))


def _plain_conv_step(s):
    dtype, slot = s["x"].dtype, s["index"].clamp(min=0).long()
    past = torch.cat([s["state"][slot], s["x"][:, None]], 1)
    v = (past.float() * s["w"].t()).sum(1) + s["bias"]
    y = torch.where(s["index"][:, None] >= 0, v * torch.sigmoid(v), 0.0)
    return {"y": y.to(dtype), "state": _put(s, past[:, 1:])}


def _plain_conv_prompt(s):
    dtype, W, L = s["x"].dtype, s["w"].shape[1], s["x"].shape[1]
    past = torch.cat([s["state"][s["index"].long()], s["x"]], 1)
    v = (past.float().unfold(1, W, 1) * s["w"]).sum(-1) + s["bias"]
    live = torch.arange(L, device="cuda") < s["lengths"][:, None]
    y = torch.where(live[..., None], v * torch.sigmoid(v), 0.0)
    last = s["lengths"][:, None] + torch.arange(W - 1, device="cuda")  # row len is x[len - (W - 1)]
    new = past.gather(1, last[..., None].expand(-1, -1, past.shape[2]))
    return {"y": y.to(dtype), "state": _put(s, new)}


def _plain_conv_grad(s):
    dtype, W = s["x"].dtype, s["w"].shape[1]
    x = torch.nn.functional.pad(s["x"].float(), (0, 0, W - 1, 0)).unfold(1, W, 1)
    dv = s["dy"].float() * _silu_grad((x * s["w"]).sum(-1) + s["bias"])
    dw = (dv[..., None] * x).sum((0, 1))
    dx = (torch.nn.functional.pad(dv, (0, 0, 0, W - 1)).unfold(1, W, 1) * s["w"].flip(1)).sum(-1)
    return {"dx": dx.to(dtype), "dw": dw, "dbias": dv.sum((0, 1))}


def _recur(a, b):
    """s_t = a_t s_{t-1} + b_t along dimension 1, from s_{-1} = 0, by doubling the span that each entry covers."""
    span, L = 1, a.shape[1]
    while span < L:
        b = torch.cat([b[:, :span], torch.addcmul(b[:, span:], a[:, span:], b[:, :-span])], 1)
        a = torch.cat([a[:, :span], a[:, span:] * a[:, :-span]], 1) if 2 * span < L else a
        span *= 2
    return b


def _grouped(v, G):
    """[..., H] as [..., G, H/G, 1], to go with B and C as [..., G, 1, N]."""
    return v.unflatten(-1, (G, -1))[..., None]


def _plain_scan_step(s):
    dtype, G = s["x"].dtype, s["B"].shape[1]
    x, dt = s["x"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    A, B, C = s["A"].unflatten(0, (G, -1)), s["B"].float()[:, :, None], s["C"].float()[:, :, None]
    old = s["state"][s["index"].clamp(min=0).long()].unflatten(1, (G, -1))
    new = torch.exp(_grouped(dt, G) * A) * old + _grouped(dt * x, G) * B
    z = s["z"].float()
    y = ((new * C).sum(-1).flatten(1) + s["D"] * x) * (z * torch.sigmoid(z))
    y = torch.where(s["index"][:, None] >= 0, y, 0.0)
    return {"y": y.to(dtype), "state": _put(s, new.flatten(1, 2))}


def _plain_scan_prompt(s):
    dtype, G, L = s["x"].dtype, s["B"].shape[2], s["x"].shape[1]
    live = (torch.arange(L, device="cuda") < s["lengths"][:, None])[..., None]
    x = s["x"].float()
    dt = torch.where(live, _softplus(s["dt"].float() + s["dt_bias"]), 0.0)
    a = torch.exp(_grouped(dt, G) * s["A"].unflatten(0, (G, -1)))
    b = _grouped(dt * x, G) * s["B"].float()[:, :, :, None]
    b[:, 0] += a[:, 0] * s["state"][s["index"].long()].unflatten(1, (G, -1))
    states = _recur(a, b)
    del a, b
    z = s["z"].float()
    y = ((states * s["C"].float()[:, :, :, None]).sum(-1).flatten(2) + s["D"] * x) * (z * torch.sigmoid(z))
    return {"y": torch.where(live, y, 0.0).to(dtype), "state": _put(s, states[:, -1].flatten(1, 2))}


def _plain_scan_grad(s):
    dtype, G = s["x"].dtype, s["B"].shape[2]
    x, z, dout = s["x"].float(), s["z"].float(), s["dy"].float()
    raw = s["dt"].float() + s["dt_bias"]
    dt = _softplus(raw)
    A, B, C = s["A"].unflatten(0, (G, -1)), s["B"].float()[:, :, :, None], s["C"].float()[:, :, :, None]
    a = torch.exp(_grouped(dt, G) * A)
    states = _recur(a, _grouped(dt * x, G) * B)
    y = (states * C).sum(-1).flatten(2) + s["D"] * x
    dz = dout * y * _silu_grad(z)
    dy = dout * z * torch.sigmoid(z)
    dC = (_grouped(dy, G) * states).sum(3)
    # g_t = C_t dy_t + a_{t+1} g_{t+1}: the same recurrence from the end
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1).flip(1)
    g = _recur(later, (_grouped(dy, G) * C).flip(1)).flip(1)
    del later
    dB = (g * _grouped(dt * x, G)).sum(3)
    u = (g * B).sum(-1).flatten(2)
    prev = torch.cat([torch.zeros_like(states[:, :1]), states[:, :-1]], 1)
    q = g * a * prev
    del a, g, states, prev
    dA = (q * _grouped(dt, G)).sum((0, 1)).flatten(0, 1)
    draw_ = ((q * A).sum(-1).flatten(2) + u * x) * torch.sigmoid(raw)
    return {"dx": (dt * u + s["D"] * dy).to(dtype), "ddt": draw_.to(dtype), "dA": dA, "dB": dB.to(dtype),
            "dC": dC.to(dtype), "dD": (dy * x).sum((0, 1)), "dz": dz.to(dtype), "ddt_bias": draw_.sum((0, 1))}


def _unit(v):
    """v over its root mean square along the last dimension, and that factor."""
    r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    return v * r, r


def _plain_norm_forward(s):
    g = s["gate"].float()
    unit, _ = _unit(s["o"].float() * g * torch.sigmoid(g))
    h = s["h"] + s["scale"] * (unit * s["w_post"])
    return {"h": h, "y": (_unit(h)[0] * s["w_pre"]).to(s["o"].dtype)}


def _plain_norm_grad(s):
    o, g, dy, dtype = s["o"].float(), s["gate"].float(), s["dy"].float(), s["o"].dtype
    act = g * torch.sigmoid(g)
    unit, r = _unit(o * act)
    p = unit * s["w_post"]
    unit2, r2 = _unit(s["h"] + s["scale"] * p)
    d = dy * s["w_pre"]
    dh = s["dh_out"] + r2 * (d - unit2 * (d * unit2).mean(-1, keepdim=True))
    dp = dh * s["scale"]
    d = dp * s["w_post"]
    dv = r * (d - unit * (d * unit).mean(-1, keepdim=True))
    return {"do": (dv * act).to(dtype), "dgate": (dv * o * _silu_grad(g)).to(dtype), "dh": dh,
            "dw_post": (dp * unit).sum(0), "dscale": (dh * p).sum(0), "dw_pre": (dy * unit2).sum(0)}


_own = {"conv-step": _own_conv_step, "conv-prompt": _own_conv_prompt, "conv-grad": _own_conv_grad,
        "scan-step": _own_scan_step, "scan-prompt": _own_scan_prompt, "scan-grad": _own_scan_grad,
        "norm-forward": _own_norm_forward, "norm-grad": _own_norm_grad}
_plain = {"conv-step": _plain_conv_step, "conv-prompt": _plain_conv_prompt, "conv-grad": _plain_conv_grad,
          "scan-step": _plain_scan_step, "scan-prompt": _plain_scan_prompt, "scan-grad": _plain_scan_grad,
          "norm-forward": _plain_norm_forward, "norm-grad": _plain_norm_grad}


# ---- what a pass cannot do without ------------------------------------------------------------------------

def work(case):
    e = 4 if case["dtype"] == "float32" else 2
    H, form = case["H"], case["form"]
    if case["op"] == "norm":
        cells = case["rows"] * H
        if form == "forward":  # o, gate, y in the type; the residual in and out in 32 bits
            return {"bytes": cells * (3 * e + 8) + 12 * H, "flops": 16 * cells}
        return {"bytes": cells * (5 * e + 12) + 24 * H, "flops": 50 * cells}
    batch, L = case["batch"], case["L"]
    live = sum(_lengths(case)) if form == "prompt" else batch * L
    rows = sum(i >= 0 for i in _slots(case)) if form != "grad" else batch
    if form == "step":
        live = rows
    if case["op"] == "conv":
        W = case["W"]
        if form == "grad":
            return {"bytes": batch * L * H * 3 * e + 8 * H * (W + 1), "flops": (6 * W + 8) * batch * L * H}
        past = 2 * rows * (W - 1) * H * e
        return {"bytes": (live + batch * L) * H * e + past + 4 * H * (W + 1), "flops": (2 * W + 5) * live * H}
    N, G = case["N"], case["G"]
    if form == "grad":
        data = batch * L * (7 * H + 4 * G * N) * e
        return {"bytes": data + 8 * H * (N + 2), "flops": batch * L * H * (22 * N + 40)}
    data = live * (3 * H + 2 * G * N) * e + batch * L * H * e
    return {"bytes": data + 8 * rows * H * N + 4 * H * (N + 2), "flops": live * H * (7 * N + 20)}


# ---- the definitions in 64 bits ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    grad = case["form"] == "grad"
    if case["op"] == "scan" and grad and case["L"] > 16384:
        return None  # the tape of so many steps takes too long
    names = {"conv": ["x", "w", "bias"], "scan": ["x", "dt", "A", "B", "C", "D", "z", "dt_bias"],
             "norm": ["o", "gate", "h", "w_post", "scale", "w_pre"]}[case["op"]]
    if grad:
        for k in names:
            wide[k] = wide[k].detach().requires_grad_(True)
    with torch.set_grad_enabled(grad):
        out = {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](wide, case)
        if not grad:
            return out
        if case["op"] == "norm":
            total = (out["y"] * wide["dy"]).sum() + (out["h"] * wide["dh_out"]).sum()
        else:
            total = (out["y"] * wide["dy"]).sum()
        got = torch.autograd.grad(total, [wide[k] for k in names])
    return {"d" + k: v for k, v in zip(names, got)}


def _silu64(v):
    return v / (1 + torch.exp(-v))


def _exact_live(s, case):
    if case["form"] == "prompt":
        return s["lengths"].tolist()
    if case["form"] == "step":
        return [int(i >= 0) for i in s["index"].tolist()]
    return [case["L"]] * case["batch"]


def _exact_conv(s, case):
    W, H, L, batch = case["W"], case["H"], case["L"], case["batch"]
    x = s["x"].reshape(batch, L, H)
    ys, state = [], None if case["form"] == "grad" else s["state_out"].clone()
    for b, n in enumerate(_exact_live(s, case)):
        slot = None if state is None else int(s["index"][b])
        before = x.new_zeros(W - 1, H) if slot is None else s["state"][max(slot, 0)]
        seen = torch.cat([before, x[b, :n]])
        v = s["bias"].expand(n, H)
        for k in range(W):
            v = v + seen[k:k + n] * s["w"][:, k]
        ys.append(torch.cat([_silu64(v), x.new_zeros(L - n, H)]))
        if slot is not None and slot >= 0:
            state[slot] = seen[n:]
    y = torch.stack(ys).reshape(s["x"].shape)
    return {"y": y} if state is None else {"y": y, "state": state}


def _exact_scan(s, case):
    H, L, batch, N, G = case["H"], case["L"], case["batch"], case["N"], case["G"]
    x, z = s["x"].reshape(batch, L, H), s["z"].reshape(batch, L, H)
    step = torch.logaddexp(s["dt"].reshape(batch, L, H) + s["dt_bias"], x.new_zeros(()))
    B, C = s["B"].reshape(batch, L, G, N).unbind(1), s["C"].reshape(batch, L, G, N).unbind(1)
    xs, steps = x.unbind(1), step.unbind(1)
    live = torch.tensor(_exact_live(s, case), device=x.device)
    grad = case["form"] == "grad"
    now = x.new_zeros(batch, H, N) if grad else s["state"][s["index"].clamp(min=0).long()]
    ys = []
    for t in range(L):
        b = B[t].repeat_interleave(H // G, 1)
        c = C[t].repeat_interleave(H // G, 1)
        d = steps[t][..., None]
        new = torch.exp(d * s["A"]) * now + d * xs[t][..., None] * b
        now = new if grad else torch.where((live > t)[:, None, None], new, now)
        ys.append((now * c).sum(-1) + s["D"] * xs[t])
    y = torch.stack(ys, 1) * _silu64(z)
    y = torch.where((torch.arange(L, device=x.device) < live[:, None])[..., None], y, 0.0).reshape(s["x"].shape)
    if grad:
        return {"y": y}
    state = s["state_out"].clone()
    for b, slot in enumerate(s["index"].tolist()):
        if slot >= 0:
            state[slot] = now[b]
    return {"y": y, "state": state}


def _exact_norm(s, case):
    v = s["o"] * _silu64(s["gate"])
    p = v / torch.sqrt((v * v).sum(-1, keepdim=True) / case["H"] + EPS) * s["w_post"]
    h = s["h"] + s["scale"] * p
    return {"h": h, "y": h / torch.sqrt((h * h).sum(-1, keepdim=True) / case["H"] + EPS) * s["w_pre"]}
