"""A small language model of linear-attention blocks, trained, prompted and decoded.

    python examples/linear_attention_blocks.py [--steps N]

Each block is: layer norm -> projection -> rotary positions of queries and keys -> linear attention with a decay
for each head -> a norm of each head's output -> gate -> projection, on a residual stream; half as many keys and
values as queries.  The model learns to repeat a random sequence after a separator; its loss is formed without
the logits.  Then a ragged batch of prompts fills a cache of states, and decoding continues token by token, on
states in slots; its logits are compared with those of the whole sequences.  Needs the GPU library (build
it with __graft_entry__.build())."""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import structured_state_space_gb300 as s4  # noqa: E402
from structured_state_space_gb300 import autograd as ops  # noqa: E402
from selective_blocks import batch  # noqa: E402

VOCAB, MODEL, HEADS, GROUPS, KEY, VALUE, LAYERS = 32, 128, 4, 2, 32, 48, 2


class Block(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.sizes = [HEADS * KEY, GROUPS * KEY, GROUPS * VALUE, HEADS * VALUE]  # q, k, v, gate
        self.inp = torch.nn.Linear(MODEL, sum(self.sizes), bias=False)
        self.out = torch.nn.Linear(HEADS * VALUE, MODEL, bias=False)
        self.w, self.b = torch.nn.Parameter(torch.ones(MODEL)), torch.nn.Parameter(torch.zeros(MODEL))
        self.w_head = torch.nn.Parameter(torch.ones(VALUE))
        # half-lives of some 2 to some 100 tokens
        self.register_buffer("log_decay", torch.log1p(-torch.exp2(-2 - 5 * torch.arange(HEADS) / max(1, HEADS - 1))))

    def project(self, y):
        q, k, v, gate = self.inp(y).split(self.sizes, -1)
        return q.unflatten(-1, (HEADS, KEY)), k.unflatten(-1, (GROUPS, KEY)), v.unflatten(-1, (GROUPS, VALUE)), gate

    def finish(self, o, gate, norm):
        return self.out(norm(o, self.w_head).flatten(-2) * F.silu(gate))


class Model(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.embed = torch.nn.Embedding(VOCAB, MODEL)
        torch.nn.init.normal_(self.embed.weight, std=MODEL ** -0.5)  # also the output's: logits of size 1
        self.blocks = torch.nn.ModuleList(Block() for _ in range(LAYERS))
        self.w, self.b = torch.nn.Parameter(torch.ones(MODEL)), torch.nn.Parameter(torch.zeros(MODEL))
        self.register_buffer("freqs", s4.s4_rotary_freqs(KEY)[0])

    def hidden(self, tokens):
        """What the output's weights are multiplied by, for whole sequences, differentiable."""
        h = self.embed(tokens)
        for b in self.blocks:
            q, k, v, gate = b.project(ops.layer_norm(h, b.w, b.b))
            q, k = ops.rotary(q, k, self.freqs)
            h = h + b.finish(ops.linear_attention(q, k, v, b.log_decay), gate, ops.layer_norm)
        return ops.layer_norm(h, self.w, self.b)

    def forward(self, tokens):
        return F.linear(self.hidden(tokens), self.embed.weight)

    def cache(self, slots, device):
        """The states of each layer, one slot per sequence."""
        return [torch.zeros(slots, HEADS, KEY, VALUE, device=device) for _ in range(LAYERS)]

    @torch.no_grad()
    def serve(self, tokens, cache, index, lengths=None, positions=None):
        """Logits of prompts [batch, L] of the given lengths, or of one token each [batch] at `positions`; the
        states in `cache` at the slots `index` are advanced in place."""
        h = self.embed(tokens)
        for b, state in zip(self.blocks, cache):
            q, k, v, gate = b.project(s4.s4_layer_norm_fwd(h, b.w, b.b))
            q, k = s4.s4_rotary_fwd(q, k, self.freqs, positions=positions)
            if tokens.dim() == 1:
                o = s4.s4_linear_attention_step(q, k, v, b.log_decay, state, index=index)
            else:
                o = s4.s4_linear_attention_fwd(q, k, v, b.log_decay, lengths=lengths, state=state, state_out=state,
                                               index=index)
            h = h + b.finish(o, gate, s4.s4_layer_norm_fwd)
        return F.linear(s4.s4_layer_norm_fwd(h, self.w, self.b), self.embed.weight)


def train(model, steps, half=4, n=64, lr=3e-3, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        seq = batch(n, half, "cuda", g)
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
        at = lens + t
        got = model.serve(seq[rows, at.long()], cache, index, positions=at)
        off = max(off, (got - want[rows, at.long()]).abs().max().item())
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
