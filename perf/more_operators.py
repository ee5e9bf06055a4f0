"""Cases of the linear-attention block's operators and of the vocabulary loss, their plain forms and their definitions
in 64 bits.

Four operators, each with the forms a model needs:

* ``attention``: linear attention with a decay for each head (``step``: one token per sequence on states in slots;
  ``prompt``: whole prompts of ragged lengths; ``grad``: the backward pass);
* ``rotary``: rotary positions of queries and keys, halves or interleaved pairs, the whole head or its first part,
  frequencies as they are or scaled for long contexts (``forward`` and ``grad``);
* ``layernorm``: layer norm (``forward``; ``grad``: with the weight's and the bias's gradients);
* ``loss``: softmax cross entropy of hidden states against a vocabulary's weights (``forward``: the losses alone;
  ``grad``: a training step's losses and gradients).

``prepare`` makes a case's inputs, ``run`` is one pass over them: through the library's entry points where ``own`` is
true, in elementary torch operations in 32 bits where it is false.
"""
import math
import random

import torch

own = False

DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
EPS = 1e-5
CHUNK = 64


# ---- cases ------------------------------------------------------------------------------------------------

def listed():
    return [
        # decoding for one user: a call that is all latency
        dict(name="attention-step-1x16x64", op="attention", form="step", batch=1, L=1, heads=16, groups=16, dk=64, dv=64,
             slots=1, dtype="bfloat16"),
        # decoding for many users at once: the states of a large cache, some rows of the batch not in use
        dict(name="attention-step-128x32x128", op="attention", form="step", batch=128, L=1, heads=32, groups=32, dk=128,
             dv=128, slots=160, dtype="bfloat16"),
        # a ragged batch of prompts into the cache, one of them empty, 4 heads to each key and value
        dict(name="attention-prompt-4x1500x16x128", op="attention", form="prompt", batch=4, L=1500, heads=16, groups=4,
             dk=128, dv=128, slots=4, dtype="bfloat16"),
        # one document of the greatest length, the channels and length those of the library's largest workload
        dict(name="attention-prompt-1x65536x16x64", op="attention", form="prompt", batch=1, L=65536, heads=16, groups=16,
             dk=64, dv=64, slots=1, dtype="bfloat16"),
        # a training batch's backward pass
        dict(name="attention-grad-4x4096x16x128", op="attention", form="grad", batch=4, L=4096, heads=16, groups=16, dk=128,
             dv=128, slots=0, dtype="bfloat16"),
        # odd lengths and widths in 32 bits, 3 heads to each key and value
        dict(name="attention-grad-2x333x6x48", op="attention", form="grad", batch=2, L=333, heads=6, groups=2, dk=48, dv=80,
             slots=0, dtype="float32"),
        # decoding at far positions, interleaved pairs of a part of each head, fewer key heads than query heads
        dict(name="rotary-forward-64x1x16x128", op="rotary", form="forward", batch=64, L=1, heads=16, groups=4, d=128, rot=64,
             pairs=True, scaling="parts", far=1 << 20, dtype="float16"),
        # a training batch or a batch of prompts, halves of whole heads
        dict(name="rotary-forward-4x4096x16x128", op="rotary", form="forward", batch=4, L=4096, heads=16, groups=16, d=128,
             rot=128, pairs=False, scaling="none", far=4096, dtype="bfloat16"),
        # a long prompt's rows, an odd number of them
        dict(name="layernorm-forward-16001x2560", op="layernorm", form="forward", rows=16001, H=2560, dtype="float16"),
        # a training batch's backward pass
        dict(name="layernorm-grad-16384x2048", op="layernorm", form="grad", rows=16384, H=2048, dtype="bfloat16"),
        # evaluation of one sequence: the losses alone
        dict(name="loss-forward-1001x1024x32000", op="loss", form="forward", rows=1001, H=1024, vocab=32000,
             dtype="bfloat16"),
        # a training step's loss, its vocabulary an odd number of words
        dict(name="loss-grad-8192x2048x50257", op="loss", form="grad", rows=8192, H=2048, vocab=50257, dtype="bfloat16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _width(rng, lo, hi):
    """A number of channels: a usual one twice of three times, else any."""
    usual = [n for n in (32, 64, 128, 192, 256, 384, 512, 768, 1024, 1280, 2048, 2560, 4096, 5120, 8192) if lo <= n <= hi]
    return rng.choice(usual) if rng.random() < 0.67 else _log(rng, lo, hi) // 2 * 2 + 1


def _heads(rng, most):
    groups = rng.choice([1, 2, 4, 5, 8, 16, 32])
    return groups, groups * rng.choice([n for n in (1, 1, 1, 2, 3, 4, 8) if groups * n <= most])


def draw(rng):
    op, form = rng.choice([("attention", "step"), ("attention", "prompt"), ("attention", "grad"), ("rotary", "forward"),
                           ("rotary", "grad"), ("layernorm", "forward"), ("layernorm", "grad"), ("loss", "forward"),
                           ("loss", "grad")])
    c = dict(op=op, form=form, dtype=rng.choice(["bfloat16", "bfloat16", "float16", "float32"]))
    if op == "layernorm":
        c["H"] = _width(rng, 32, 8192)
        c["rows"] = _log(rng, 1, max(1, min(262144, (1 << 25) // c["H"])))
        return c
    if op == "loss":
        c["H"] = rng.choice([64, 128, 256, 512, 768, 1024, 2048, 4096]) if rng.random() < 0.8 else _log(rng, 32, 2048)
        c["vocab"] = rng.choice([256, 1000, 32000, 50257, 65536]) if rng.random() < 0.67 else _log(rng, 30, 131072)
        c["rows"] = _log(rng, 1, max(1, min(16384, (1 << 38) // (c["H"] * c["vocab"]))))
        return c
    c["groups"], c["heads"] = _heads(rng, 32)
    if op == "rotary":
        c["d"] = rng.choice([32, 64, 64, 128, 128, 128, 256, 80, 2 * rng.randint(1, 128)])
        c["rot"] = c["d"] if rng.random() < 0.67 else 2 * rng.randint(1, c["d"] // 2)
        c["pairs"], c["scaling"] = rng.random() < 0.5, rng.choice(["none", "none", "linear", "parts"])
        c["far"] = _log(rng, 4096, 1 << 24)
        most = (1 << 26) // (c["d"] * (c["heads"] + c["groups"]))
        c["L"] = rng.choice([1, _log(rng, 1, max(1, min(65536, most)))])
        c["batch"] = _log(rng, 1, max(1, min(512, most // c["L"])))
        return c
    usual = [16, 32, 64, 64, 64, 128, 128, 128, 256]
    c["dk"], c["dv"] = (rng.choice(usual) if rng.random() < 0.75 else rng.randint(4, 160) for _ in range(2))
    if rng.random() < 0.5:
        c["dv"] = c["dk"]
    most = (1 << 26 if form == "step" else 1 << 31) // (c["heads"] * c["dk"] * c["dv"])
    if form == "step":
        c["batch"], c["L"] = _log(rng, 1, max(1, min(512, most))), 1
    else:
        c["L"] = _log(rng, 1, max(1, min(65536, most)))
        c["batch"] = _log(rng, 1, max(1, min(16, most // c["L"])))
    c["slots"] = 0 if form == "grad" else c["batch"] + rng.choice([0, 0, 1, c["batch"] // 4 + 1])
    return c


def _lengths(case):
    """How many tokens of each sequence are real: the first has them all, one of three or more none, the others any."""
    n, L, rng = case["batch"], case["L"], random.Random("lengths %(batch)d %(L)d %(heads)d" % case)
    got = [L] + [rng.randint(1, L) for _ in range(n - 1)]
    return got[:2] + [0] + got[3:] if n > 2 else got


def _slots(case):
    """The cache slot of each sequence; while decoding, some rows of a batch of 8 or more have none (-1)."""
    rng = random.Random("slots %(batch)d %(slots)d %(heads)d" % case)
    got = rng.sample(range(case["slots"]), case["batch"])
    if case["form"] == "step" and case["batch"] >= 8:
        for i in rng.sample(range(case["batch"]), case["batch"] // 8):
            got[i] = -1
    return got


def _freqs(case):
    """Angles per position of the pairs of a rotated part, in 64 bits: 10000^(-2i/rot); "linear": a fourth of them;
    "parts": a fourth of those that turn less than once in 4096 positions, all of those that turn more than 32 times,
    and in between a mixture that goes with the number of turns."""
    f = torch.pow(10000.0, -torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
    if case["scaling"] == "none":
        return f
    if case["scaling"] == "linear":
        return f / 4
    kept = ((f * 4096 / (2 * math.pi) - 1) / 31).clamp(0, 1)
    return f / 4 * (1 - kept) + f * kept


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    op, form = case["op"], case["form"]
    s = {"op": op, "form": form}
    if op == "layernorm":
        rows, H = case["rows"], case["H"]
        # a residual stream: channels of different sizes, rows that are not centred
        s["x"] = (normal(rows, H) * (0.5 + torch.rand(H, generator=gen, device="cuda")) + normal(rows, 1)).to(dtype)
        s["w"], s["b"] = 1 + normal(H, scale=0.1), normal(H, scale=0.1)
        if form == "grad":
            s["dy"] = normal(rows, H, dtype=dtype)
        return s
    if op == "loss":
        rows, H, V = case["rows"], case["H"], case["vocab"]
        s["h"] = normal(rows, H, dtype=dtype)
        s["w"] = normal(V, H, scale=2 * H ** -0.5, dtype=dtype)  # logits of about 2
        s["targets"] = torch.randint(0, V, (rows,), generator=gen, device="cuda")
        if rows > 1:  # one of eight tokens or so is padding, or a prompt's
            s["targets"][torch.rand(rows, generator=gen, device="cuda") < 0.125] = -1
        if form == "grad":  # the mean over the tokens that count, times a loss scale
            s["dloss"] = torch.full((rows,), 1024.0 / rows, device="cuda")
        return s
    batch, L, heads, groups = case["batch"], case["L"], case["heads"], case["groups"]
    if op == "rotary":
        d = case["d"]
        # queries, keys and values lie side by side in a projection's output
        qkv = normal(batch, L, (heads + 2 * groups) * d, dtype=dtype)
        s["q"] = qkv[..., :heads * d].unflatten(-1, (heads, d))
        s["k"] = qkv[..., heads * d:(heads + groups) * d].unflatten(-1, (groups, d))
        first = torch.randint(0, max(1, case["far"] - L + 1), (batch, 1), generator=gen, device="cuda")
        s["positions"] = (first + torch.arange(L, device="cuda")).to(torch.int32)
        s["freqs"], s["pairs"] = _freqs(case).cuda(), case["pairs"]
        s["amplitude"] = 1 + 0.1 * math.log(4) if case["scaling"] == "parts" else 1.0
        return s
    dk, dv = case["dk"], case["dv"]
    shape = (batch,) if form == "step" else (batch, L)
    qkv = normal(*shape, heads * dk + groups * (dk + dv), dtype=dtype)
    s["q"] = qkv[..., :heads * dk].unflatten(-1, (heads, dk))
    s["k"] = qkv[..., heads * dk:heads * dk + groups * dk].unflatten(-1, (groups, dk))
    s["v"] = qkv[..., heads * dk + groups * dk:].unflatten(-1, (groups, dv))
    # half-lives from some 20 tokens to some thousands, spread over the heads
    s["log_decay"] = torch.log1p(-torch.exp2(-5 - 7 * torch.rand(heads, generator=gen, device="cuda")))
    if form == "grad":
        s["do"] = normal(*shape, heads, dv, dtype=dtype)
        return s
    index = _slots(case)
    s["index"] = torch.tensor(index, dtype=torch.int32, device="cuda")
    s["rows"] = torch.tensor([b for b in range(batch) if index[b] >= 0], device="cuda")
    s["at"] = torch.tensor([i for i in index if i >= 0], device="cuda")
    if form == "prompt":
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    s["state"] = normal(case["slots"], heads, dk, dv)
    s["state_out"] = s["state"].clone()
    return s


def run(s):
    return (_own if own else _plain)[s["op"] + "-" + s["form"]](s)


# ---- through the library ----------------------------------------------------------------------------------

def _own_attention_step(s):
    import structured_state_space_gb300 as s4
    o = s4.s4_linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], state_out=s["state_out"],
                                    index=s["index"])
    return {"o": o, "state": s["state_out"]}


def _own_attention_prompt(s):
    import structured_state_space_gb300 as s4
    o = s4.s4_linear_attention_fwd(s["q"], s["k"], s["v"], s["log_decay"], lengths=s["lengths"], state=s["state"],
                                   state_out=s["state_out"], index=s["index"])
    return {"o": o, "state": s["state_out"]}


def _own_attention_grad(s):
    import structured_state_space_gb300 as s4
    return s4.s4_linear_attention_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"])


def _own_rotary_forward(s):
    import structured_state_space_gb300 as s4
    q, k = s4.s4_rotary_fwd(s["q"], s["k"], s["freqs"], positions=s["positions"], pairs=s["pairs"],
                            amplitude=s["amplitude"])
    return {"q": q, "k": k}


def _own_rotary_grad(s):
    import structured_state_space_gb300 as s4
    q, k = s4.s4_rotary_bwd(s["q"], s["k"], s["freqs"], positions=s["positions"], pairs=s["pairs"],
                            amplitude=s["amplitude"])
    return {"dq": q, "dk": k}


def _own_layernorm_forward(s):
    import structured_state_space_gb300 as s4
    return s4.s4_layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS)


def _own_layernorm_grad(s):
    import structured_state_space_gb300 as s4
    return s4.s4_layer_norm_bwd(s["x"], s["dy"], s["w"], s["b"], eps=EPS)


def _own_loss_forward(s):
    import structured_state_space_gb300 as s4
    loss, lse = s4.s4_vocab_loss_fwd(s["h"], s["w"], s["targets"])
    return {"loss": loss, "lse": lse}


def _own_loss_grad(s):
    import structured_state_space_gb300 as s4
    loss, lse = s4.s4_vocab_loss_fwd(s["h"], s["w"], s["targets"])
    g = s4.s4_vocab_loss_bwd(s["h"], s["w"], s["targets"], lse, s["dloss"])
    return {"loss": loss, "dh": g["dh"], "dw": g["dw"]}


# ---- the plain forms --------------------------------------------------------------------------------------

def _per_head(t, heads):
    """[batch, L, groups, d] as [batch, heads, L, d] in 32 bits, each group's row for every head of the group."""
    t = t.float().repeat_interleave(heads // t.shape[2], 2) if t.shape[2] != heads else t.float()
    return t.transpose(1, 2)


def _recur(a, b):
    """s_n = a s_{n-1} + b_n along dimension 2, from s_{-1} = 0, by doubling the span that each entry covers; a [heads]."""
    span, n = 1, b.shape[2]
    a = a[:, None, None, None]
    while span < n:
        b = torch.cat([b[:, :, :span], torch.addcmul(b[:, :, span:], b[:, :, :-span], a.expand_as(b[0, :, span:]))], 2)
        a, span = a * a, 2 * span
    return b


def _decays(g, exponents):
    """exp(g n) for each head and exponent, [heads, ...], formed in 64 bits."""
    return torch.exp(g.double().view(-1, *[1] * exponents.dim()) * exponents).float()


def _attend(a, b, c, g, state=None):
    """out_i = sum_{j<=i} exp(g (i-j)) (a_i . b_j) c_j + exp(g (i+1)) a_i state, in chunks; all [batch, heads, L, d]."""
    L = a.shape[2]
    n = -(-L // CHUNK)
    a, b, c = (torch.nn.functional.pad(t, (0, 0, 0, n * CHUNK - L)).unflatten(2, (n, CHUNK)) for t in (a, b, c))
    i = torch.arange(CHUNK, device="cuda")
    lag = i[:, None] - i
    mask = torch.where(lag >= 0, _decays(g, lag.clamp(min=0)), 0.0)
    add = (b * _decays(g, CHUNK - 1 - i)[:, None, :, None]).transpose(-1, -2) @ c
    carry = _decays(g, torch.tensor(CHUNK, device="cuda"))
    first = torch.zeros_like(add[:, :, :1]) if state is None else state[:, :, None]
    add[:, :, 0] += carry[:, None, None] * first[:, :, 0]
    before = torch.cat([first, _recur(carry, add)[:, :, :-1]], 2)
    out = ((a @ b.transpose(-1, -2)) * mask[:, None]) @ c + (a * _decays(g, i + 1)[:, None, :, None]) @ before
    return out.flatten(2, 3)[:, :, :L]


def _put(s, new):
    """The new states at their slots; slots that no sequence has keep what they hold."""
    return s["state_out"].index_copy(0, s["at"], new.index_select(0, s["rows"]))


def _plain_attention_step(s):
    heads, dtype = s["q"].shape[1], s["q"].dtype
    q, k, v = (_per_head(s[n][:, None], heads)[:, :, 0] for n in "qkv")
    old = s["state"][s["index"].clamp(min=0).long()]
    new = torch.exp(s["log_decay"])[:, None, None] * old + k[..., None] * v[..., None, :]
    o = (q[..., None] * new).sum(2) * q.shape[-1] ** -0.5
    o = torch.where(s["index"][:, None, None] >= 0, o, 0.0)
    return {"o": o.to(dtype), "state": _put(s, new)}


def _plain_attention_prompt(s):
    heads, dtype, L, g = s["q"].shape[2], s["q"].dtype, s["q"].shape[1], s["log_decay"]
    t = torch.arange(L, device="cuda")
    live = (t < s["lengths"][:, None])[:, None, :, None]
    q, k, v = (_per_head(s[n], heads) for n in "qkv")
    k = torch.where(live, k, 0.0)
    v = torch.where(live, v, 0.0)
    old = s["state"][s["index"].long()]
    o = torch.where(live, _attend(q, k, v, g, old) * q.shape[-1] ** -0.5, 0.0)
    behind = (s["lengths"][:, None] - 1 - t).clamp(min=0)  # how many tokens follow each
    weight = _decays(g, behind).transpose(0, 1)[..., None]
    new = (k * weight).transpose(-1, -2) @ v + _decays(g, s["lengths"]).t()[..., None, None] * old
    return {"o": o.transpose(1, 2).to(dtype), "state": _put(s, new)}


def _plain_attention_grad(s):
    heads, groups, dtype, g = s["q"].shape[2], s["k"].shape[2], s["q"].dtype, s["log_decay"]
    q, k, v, do = (_per_head(s[n], heads) for n in ("q", "k", "v", "do"))
    scale = q.shape[-1] ** -0.5
    dq = _attend(do, v, k, g) * scale
    # the others are the same sums from the end
    dk = _attend(v.flip(2), do.flip(2), q.flip(2), g).flip(2) * scale
    dv = _attend(k.flip(2), q.flip(2), do.flip(2), g).flip(2) * scale
    shared = [t.unflatten(1, (groups, -1)).sum(2) for t in (dk, dv)]
    return {n: t.transpose(1, 2).to(dtype) for n, t in zip(("dq", "dk", "dv"), [dq] + shared)}


def _rotate(s, t, sign):
    angle = s["positions"][..., None].double() * s["freqs"]
    cos = (torch.cos(angle) * s["amplitude"]).float()[:, :, None]
    sin = (torch.sin(angle) * (sign * s["amplitude"])).float()[:, :, None]
    n = cos.shape[-1]
    x = t.float()
    part, rest = x[..., :2 * n], x[..., 2 * n:]
    a, b = (part[..., 0::2], part[..., 1::2]) if s["pairs"] else (part[..., :n], part[..., n:])
    a, b = a * cos - b * sin, a * sin + b * cos
    part = torch.stack([a, b], -1).flatten(-2) if s["pairs"] else torch.cat([a, b], -1)
    return torch.cat([part, rest], -1).to(t.dtype)


def _plain_rotary_forward(s):
    return {"q": _rotate(s, s["q"], 1), "k": _rotate(s, s["k"], 1)}


def _plain_rotary_grad(s):
    return {"dq": _rotate(s, s["q"], -1), "dk": _rotate(s, s["k"], -1)}


def _unit(x):
    """x less its mean along the last dimension, over its standard deviation, and that factor."""
    x = x.float()
    x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _plain_layernorm_forward(s):
    return (_unit(s["x"])[0] * s["w"] + s["b"]).to(s["x"].dtype)


def _plain_layernorm_grad(s):
    unit, r = _unit(s["x"])
    dy = s["dy"].float()
    d = dy * s["w"]
    dx = r * (d - d.mean(-1, keepdim=True) - unit * (d * unit).mean(-1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * unit).sum(0), "db": dy.sum(0)}


def _plain_losses(s):
    logits = s["h"].float() @ s["w"].float().t()
    most = logits.amax(-1, keepdim=True)
    lse = (torch.log(torch.exp(logits - most).sum(-1, keepdim=True)) + most)[:, 0]
    at = logits.gather(1, s["targets"].clamp(min=0)[:, None])[:, 0]
    return logits, lse, torch.where(s["targets"] >= 0, lse - at, 0.0)


def _plain_loss_forward(s):
    _, lse, loss = _plain_losses(s)
    return {"loss": loss, "lse": lse}


def _plain_loss_grad(s):
    logits, lse, loss = _plain_losses(s)
    weight = torch.where(s["targets"] >= 0, s["dloss"], 0.0)[:, None]
    d = torch.exp(logits - lse[:, None]) * weight
    del logits
    d.scatter_add_(1, s["targets"].clamp(min=0)[:, None], -weight)
    dtype = s["h"].dtype
    return {"loss": loss, "dh": (d @ s["w"].float()).to(dtype), "dw": (d.t() @ s["h"].float()).to(dtype)}


_own = {"attention-step": _own_attention_step, "attention-prompt": _own_attention_prompt,
        "attention-grad": _own_attention_grad, "rotary-forward": _own_rotary_forward, "rotary-grad": _own_rotary_grad,
        "layernorm-forward": _own_layernorm_forward, "layernorm-grad": _own_layernorm_grad,
        "loss-forward": _own_loss_forward, "loss-grad": _own_loss_grad}
_plain = {"attention-step": _plain_attention_step, "attention-prompt": _plain_attention_prompt,
          "attention-grad": _plain_attention_grad, "rotary-forward": _plain_rotary_forward,
          "rotary-grad": _plain_rotary_grad, "layernorm-forward": _plain_layernorm_forward,
          "layernorm-grad": _plain_layernorm_grad, "loss-forward": _plain_loss_forward, "loss-grad": _plain_loss_grad}


# ---- what a pass cannot do without ------------------------------------------------------------------------

def work(case):
    e, op, form = 4 if case["dtype"] == "float32" else 2, case["op"], case["form"]
    if op == "layernorm":
        cells = case["rows"] * case["H"]
        if form == "forward":
            return {"bytes": 2 * e * cells + 8 * case["H"], "flops": 8 * cells}
        return {"bytes": 3 * e * cells + 12 * case["H"], "flops": 18 * cells}
    if op == "loss":
        rows, H, V = case["rows"], case["H"], case["vocab"]
        if form == "forward":
            return {"bytes": (rows + V) * H * e + 16 * rows, "flops": 2 * rows * V * H + 3 * rows * V}
        # the logits are formed again for the gradients: they are not kept
        return {"bytes": 2 * (rows + V) * H * e + 16 * rows, "flops": 8 * rows * V * H + 6 * rows * V}
    tokens, heads, groups = case["batch"] * case["L"], case["heads"], case["groups"]
    if op == "rotary":
        cells = tokens * (heads + groups) * case["d"]
        return {"bytes": 2 * e * cells + 4 * tokens, "flops": 3 * tokens * (heads + groups) * case["rot"]}
    dk, dv = case["dk"], case["dv"]
    live = sum(_lengths(case)) if form == "prompt" else tokens
    rows = sum(i >= 0 for i in _slots(case)) if form != "grad" else case["batch"]
    if form == "step":
        live = rows
    read = live * (heads * dk + groups * (dk + dv)) * e
    if form == "grad":
        return {"bytes": 2 * read + tokens * heads * dv * e, "flops": 10 * tokens * heads * dk * dv}
    return {"bytes": read + tokens * heads * dv * e + 8 * rows * heads * dk * dv, "flops": 4 * live * heads * dk * dv}


# ---- the definitions in 64 bits ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    with torch.no_grad():
        if case["op"] == "attention":
            return (_exact_attention_grad if case["form"] == "grad" else _exact_attention)(wide, case)
        return {"rotary": _exact_rotary, "layernorm": _exact_layernorm, "loss": _exact_loss}[case["op"]](wide, case)


def _exact_attention(s, case):
    """Token by token: the state decays, takes the token's key times its value, and is read by its query."""
    batch, L, heads, dk = case["batch"], case["L"], case["heads"], case["dk"]
    each = heads // case["groups"]
    q, k, v = (s[n].reshape(batch, L, -1, s[n].shape[-1]).unbind(1) for n in "qkv")
    factor = torch.exp(s["log_decay"])[:, None, None]
    live = s["lengths"] if case["form"] == "prompt" else (s["index"] >= 0).long()
    now = s["state"][s["index"].clamp(min=0).long()].clone()
    outs = []
    for t in range(L):
        kk, vv = k[t].repeat_interleave(each, 1), v[t].repeat_interleave(each, 1)
        new = torch.baddbmm((now * factor).flatten(0, 1), kk.flatten(0, 1)[:, :, None], vv.flatten(0, 1)[:, None]).view_as(now)
        now = torch.where((live > t)[:, None, None, None], new, now)
        outs.append((q[t].unsqueeze(-2) @ now)[..., 0, :] / math.sqrt(dk))
    o = torch.stack(outs, 1)
    o = torch.where((torch.arange(L, device=o.device) < live[:, None])[..., None, None], o, 0.0)
    state = s["state_out"].clone()
    for b, slot in enumerate(s["index"].tolist()):
        if slot >= 0:
            state[slot] = now[b]
    return {"o": o.reshape(s["q"].shape[:-1] + (case["dv"],)), "state": state}


def _exact_attention_grad(s, case):
    """Token by token forward for the queries' gradients, and back for the keys' and the values'."""
    batch, L, heads, groups, dk, dv = (case[n] for n in ("batch", "L", "heads", "groups", "dk", "dv"))
    each = heads // groups
    q, k, v, do = (s[n].unbind(1) for n in ("q", "k", "v", "do"))
    factor = torch.exp(s["log_decay"])[:, None, None]
    now = s["q"].new_zeros(batch, heads, dk, dv)
    dq, dkey, dval = [], [None] * L, [None] * L
    for t in range(L):
        kk, vv = k[t].repeat_interleave(each, 1), v[t].repeat_interleave(each, 1)
        now = torch.baddbmm((now * factor).flatten(0, 1), kk.flatten(0, 1)[:, :, None], vv.flatten(0, 1)[:, None]).view_as(now)
        dq.append((now @ do[t].unsqueeze(-1))[..., 0])
    now.zero_()
    for t in reversed(range(L)):
        kk, vv = k[t].repeat_interleave(each, 1), v[t].repeat_interleave(each, 1)
        now = torch.baddbmm((now * factor).flatten(0, 1), q[t].flatten(0, 1)[:, :, None], do[t].flatten(0, 1)[:, None]).view_as(now)
        dkey[t] = (now @ vv.unsqueeze(-1))[..., 0].unflatten(1, (groups, each)).sum(2)
        dval[t] = (kk.unsqueeze(-2) @ now)[..., 0, :].unflatten(1, (groups, each)).sum(2)
    return {n: torch.stack(t, 1) / math.sqrt(dk) for n, t in (("dq", dq), ("dk", dkey), ("dv", dval))}


def _exact_rotary(s, case):
    """Each pair as a complex number, turned by its position's angle (back, for the gradients)."""
    sign = -1.0 if case["form"] == "grad" else 1.0
    angle = sign * s["positions"].double()[:, :, None] * s["freqs"]
    turn = torch.polar(torch.full_like(angle, s["amplitude"]), angle)[:, :, None]
    n, got = case["rot"] // 2, {}
    for name in "qk":
        x = s[name].clone()
        even, odd = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if case["pairs"] else (slice(0, n), slice(n, 2 * n))
        z = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * turn
        x[..., even], x[..., odd] = z.real, z.imag
        got[("d" if case["form"] == "grad" else "") + name] = x
    return got


def _exact_layernorm(s, case):
    x, H = s["x"], case["H"]
    centred = x - x.sum(-1, keepdim=True) / H
    deviation = torch.sqrt((centred * centred).sum(-1, keepdim=True) / H + EPS)
    if case["form"] == "forward":
        return centred / deviation * s["w"] + s["b"]
    d, unit = s["dy"] * s["w"], centred / deviation
    dx = (d - d.sum(-1, keepdim=True) / H - unit * (d * unit).sum(-1, keepdim=True) / H) / deviation
    return {"dx": dx, "dw": torch.einsum("rh,rh->h", s["dy"], unit), "db": s["dy"].sum(0)}


def _exact_loss(s, case):
    grad, step = case["form"] == "grad", 1024
    loss, lses, dh, dw = [], [], [], torch.zeros_like(s["w"])
    for at in range(0, case["rows"], step):
        h, targets = s["h"][at:at + step], s["targets"][at:at + step]
        logits = torch.einsum("rd,vd->rv", h, s["w"])
        lse = torch.logsumexp(logits, -1)
        counts = (targets >= 0).double()
        rows = torch.arange(len(targets), device=h.device)
        lses.append(lse)
        loss.append((lse - logits[rows, targets.clamp(min=0)]) * counts)
        if grad:
            d = torch.exp(logits - lse[:, None])
            d[rows, targets.clamp(min=0)] -= 1
            d *= (s["dloss"][at:at + step] * counts)[:, None]
            dh.append(torch.einsum("rv,vd->rd", d, s["w"]))
            dw += torch.einsum("rv,rd->vd", d, h)
    return {"loss": torch.cat(loss), "dh": torch.cat(dh), "dw": dw} if grad else {"loss": torch.cat(loss), "lse": torch.cat(lses)}
