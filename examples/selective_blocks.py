"""A small language model of selective state-space blocks, trained, prompted and decoded.

    python examples/selective_blocks.py [--steps N]

Each block is: projection -> short causal convolution -> step sizes and input and output vectors from the
convolved channels -> selective scan, gated -> projection; the norms before and after the blocks, their
gates, residual scales and the residual sum are one call between two blocks.  The model learns to
repeat a random sequence after a separator (the second half of each sequence is predictable from the
first).  Then a ragged batch of prompts fills a cache of states, one call per layer and operator,
and decoding continues token by token, on states in slots; its logits are compared with those of
the whole sequences.  Needs the GPU library (build it with __graft_entry__.build())."""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import structured_state_space_gb300 as s4  # noqa: E402
from structured_state_space_gb300 import autograd as ops  # noqa: E402

VOCAB, MODEL, INNER, STATES, RANK, TAPS, LAYERS = 32, 128, 256, 16, 8, 4, 2


class Block(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.inp = torch.nn.Linear(MODEL, 2 * INNER + MODEL, bias=False)  # x, z, and the gate of the block's output
        self.conv = torch.nn.Parameter(torch.randn(INNER, TAPS) * TAPS ** -0.5)
        self.conv_bias = torch.nn.Parameter(torch.zeros(INNER))
        self.vectors = torch.nn.Linear(INNER, RANK + 2 * STATES, bias=False)
        self.step = torch.nn.Linear(RANK, INNER, bias=False)
        step = torch.exp(torch.empty(INNER).uniform_(-6.9, -2.3))  # 1e-3 .. 1e-1
        self.dt_bias = torch.nn.Parameter(step + torch.log(-torch.expm1(-step)))
        self.log_A = torch.nn.Parameter(torch.log(torch.arange(1.0, STATES + 1).repeat(INNER, 1)))
        self.D = torch.nn.Parameter(torch.ones(INNER))
        self.out = torch.nn.Linear(INNER, MODEL, bias=False)
        self.w_pre = torch.nn.Parameter(torch.ones(MODEL))
        self.w_post = torch.nn.Parameter(torch.ones(MODEL))
        self.scale = torch.nn.Parameter(torch.full((MODEL,), 0.5))

    def project(self, y):
        x, z, gate = self.inp(y).split([INNER, INNER, MODEL], -1)
        return x, z, gate

    def select(self, u):
        """dt, B, C of the convolved channels."""
        low, B, C = self.vectors(u).split([RANK, STATES, STATES], -1)
        return self.step(low), B.unsqueeze(-2), C.unsqueeze(-2)


class Model(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.embed = torch.nn.Embedding(VOCAB, MODEL)
        torch.nn.init.normal_(self.embed.weight, std=MODEL ** -0.5)  # also the output's: logits of size 1
        self.blocks = torch.nn.ModuleList(Block() for _ in range(LAYERS))
        self.w_last = torch.nn.Parameter(torch.ones(MODEL))

    def join(self, i):
        """The norm that follows block i's: the next block's, or the last."""
        return self.blocks[i + 1].w_pre if i + 1 < LAYERS else self.w_last

    def hidden(self, tokens):
        """What the output's weights are multiplied by, for whole sequences, differentiable."""
        h = self.embed(tokens).float()
        h, y = ops.block_norm(h, w_pre=self.blocks[0].w_pre)
        for i, b in enumerate(self.blocks):
            x, z, gate = b.project(y)
            u = ops.short_conv(x, b.conv, b.conv_bias)
            dt, B, C = b.select(u)
            o = b.out(ops.selective_scan(u, dt, -torch.exp(b.log_A), B, C, b.D, z, b.dt_bias))
            h, y = ops.block_norm(o, gate, h, b.w_post, b.scale, self.join(i))
        return y

    def forward(self, tokens):
        """Logits of whole sequences, differentiable."""
        return F.linear(self.hidden(tokens), self.embed.weight)

    def cache(self, slots, device):
        """Per layer: the convolution's last inputs and the scan's states, one slot per sequence."""
        return [(torch.zeros(slots, TAPS - 1, INNER, device=device), torch.zeros(slots, INNER, STATES, device=device))
                for _ in range(LAYERS)]

    @torch.no_grad()
    def serve(self, tokens, cache, index, lengths=None):
        """Logits of prompts [batch, L] of the given lengths, or of one token each [batch]; the states in
        `cache` at the slots `index` are advanced in place."""
        one = tokens.dim() == 1
        h = self.embed(tokens).float()
        h, y = s4.s4_block_norm_fwd(h, w_pre=self.blocks[0].w_pre)
        for i, b in enumerate(self.blocks):
            past, state = cache[i]
            x, z, gate = b.project(y)
            A = -torch.exp(b.log_A)
            if one:
                u = s4.s4_short_conv_step(x, b.conv, b.conv_bias, past, index=index)
                dt, B, C = b.select(u)
                v = s4.s4_selective_step(u, dt, A, B, C, state, D=b.D, z=z, dt_bias=b.dt_bias, index=index)
            else:
                u = s4.s4_short_conv_fwd(x, b.conv, b.conv_bias, lengths=lengths, state=past, state_out=past, index=index)
                dt, B, C = b.select(u)
                v = s4.s4_selective_scan_fwd(u, dt, A, B, C, D=b.D, z=z, dt_bias=b.dt_bias, lengths=lengths, state=state,
                                             state_out=state, index=index)
            h, y = s4.s4_block_norm_fwd(b.out(v), gate=gate, h=h, w_post=b.w_post, scale=b.scale, w_pre=self.join(i))
        return F.linear(y, self.embed.weight)


def batch(n, half, device, generator):
    """Sequences r, separator, r: the second r can be predicted."""
    r = torch.randint(1, VOCAB, (n, half), device=device, generator=generator)
    return torch.cat([r, torch.zeros(n, 1, dtype=r.dtype, device=device), r], 1)


def train(model, steps, half=4, n=64, lr=3e-3, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        seq = batch(n, half, "cuda", g)
        # the loss of the second half, without the logits
        y = model.hidden(seq[:, :-1])[:, half:].flatten(0, 1)
        loss = ops.vocab_loss(y, model.embed.weight, seq[:, half + 1:].flatten()).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def decode(model, lengths=(9, 14, 1, 25), more=6, seed=2):
    """Largest difference between the logits of prompts continued token by token and those of the whole
    sequences, over their size."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, longest = len(lengths), max(lengths)
    seq = torch.randint(1, VOCAB, (n, longest + more), device="cuda", generator=g)
    cache = model.cache(n + 2, "cuda")
    index = torch.tensor([n + 1 - i for i in range(n)], dtype=torch.int32, device="cuda")
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    got = model.serve(seq[:, :longest], cache, index, lens)
    with torch.no_grad():
        want = model(seq)
    off = max((got[i, :k] - want[i, :k]).abs().max().item() for i, k in enumerate(lengths))
    rows = torch.arange(n, device="cuda")
    for t in range(more):
        at = lens.long() + t
        got = model.serve(seq[rows, at], cache, index)
        off = max(off, (got - want[rows, at]).abs().max().item())
    return off / want.abs().max().item()


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=300)
    a = p.parse_args()
    torch.manual_seed(0)
    model = Model().cuda()
    losses = train(model, a.steps)
    every = max(1, a.steps // 6)
    print("loss", " ".join(f"{v:.3f}" for v in losses[::every]), f"... {losses[-1]:.3f}")
    print(f"decoded token by token against whole sequences: {decode(model):.1e} of the largest logit")


if __name__ == "__main__":
    main()
