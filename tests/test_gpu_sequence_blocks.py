"""The linear-attention block's operators together: the example model runs, decodes what it computes on whole sequences, and
its gradients are those of the same model in elementary float64 operations; the differentiable functions; the
framework's other example with its loss formed without the logits."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")

from block_util import need_gpu  # noqa: E402

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    need_gpu()
    torch.backends.cuda.matmul.allow_tf32 = False
    import linear_attention_blocks
    return linear_attention_blocks


def test_training_runs(example):
    torch.manual_seed(0)
    losses = example.train(example.Model().cuda(), 5)
    assert len(losses) == 5 and all(math.isfinite(v) for v in losses)


def test_decoding_follows_the_whole_sequences(example):
    torch.manual_seed(1)
    # float32 throughout: two orders of the same sums over 2 layers, a few 1e-6 of the largest logit
    assert example.decode(example.Model().cuda()) < 2e-5


def _plain(m, tokens, e):
    """The example's forward in elementary operations, for any dtype."""
    def norm(v, w, b=0.0):
        v = v - v.mean(-1, keepdim=True)
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * w + b

    def turn(x):
        t = torch.arange(x.shape[1], device=x.device, dtype=torch.float64)[:, None] * m.freqs
        c, s = torch.cos(t).to(x.dtype)[:, None], torch.sin(t).to(x.dtype)[:, None]
        a, b = x.chunk(2, -1)
        return torch.cat([a * c - b * s, a * s + b * c], -1)
    h = m.embed(tokens)
    L = tokens.shape[1]
    for blk in m.blocks:
        q, k, v, gate = blk.project(norm(h, blk.w, blk.b))
        q, k = turn(q), turn(k)
        k, v = (x.repeat_interleave(e.HEADS // e.GROUPS, 2) for x in (k, v))
        lag = torch.arange(L, device=h.device)[:, None] - torch.arange(L, device=h.device)
        w = torch.where(lag >= 0, torch.exp(blk.log_decay.to(h.dtype)[:, None, None] * lag.clamp(min=0)), 0.0)
        o = torch.einsum("bihk,bjhk,hij,bjhv->bihv", q, k, w, v) * e.KEY ** -0.5
        h = h + blk.finish(o, gate, norm)
    return norm(h, m.w, m.b)


def test_gradients_of_the_whole_model(example):
    torch.manual_seed(2)
    m = example.Model().cuda()
    wide = example.Model().cuda().double()
    wide.load_state_dict({k: v.double() for k, v in m.state_dict().items()})
    for a, b in zip(wide.blocks, m.blocks):
        a.log_decay = b.log_decay.double()
    tokens = torch.randint(0, example.VOCAB, (3, 21), device="cuda")
    targets = torch.randint(-1, example.VOCAB, (3, 21), device="cuda")
    weight = torch.rand(3, 21, device="cuda")
    (example.ops.vocab_loss(m.hidden(tokens), m.embed.weight, targets) * weight).sum().backward()
    x = torch.log_softmax(_plain(wide, tokens, example) @ wide.embed.weight.t(), -1)
    loss = torch.where(targets >= 0, -x.gather(-1, targets.clamp(min=0)[..., None])[..., 0], 0.0)
    (loss * weight.double()).sum().backward()
    for (k, p), q in zip(m.named_parameters(), wide.named_parameters()):
        # float32 through 2 layers forward and back: some 1e-6, a decade of room
        off = (p.grad.double() - q[1].grad).norm() / q[1].grad.norm()
        assert off < 5e-5, (k, off.item())


def test_second_derivatives_raise(example):
    ops = example.ops
    q = torch.randn(1, 5, 2, 8, device="cuda", requires_grad=True)
    g = torch.tensor([-0.1, -0.2], device="cuda")
    freqs = example.s4.s4_rotary_freqs(8, device="cuda")[0]
    x = torch.randn(4, 16, device="cuda", requires_grad=True)
    w = torch.randn(9, 16, device="cuda", requires_grad=True)
    t = torch.tensor([1, 2, -1, 8], device="cuda")
    for y, v in ((ops.linear_attention(q, q, q, g), q), (ops.rotary(q, q, freqs)[0], q), (ops.layer_norm(x), x),
                 (ops.vocab_loss(x, w, t), x)):
        d, = torch.autograd.grad((y * y).sum(), v, create_graph=True)
        with pytest.raises(RuntimeError, match="second derivatives"):
            d.sum().backward()


def test_gradients_that_are_not_asked_for(example):
    ops = example.ops
    q, k = torch.randn(2, 5, 4, 8, device="cuda", requires_grad=True), torch.randn(2, 5, 2, 8, device="cuda", requires_grad=True)
    freqs = example.s4.s4_rotary_freqs(8, device="cuda")[0]
    # one output of the two, and each alone
    (ops.rotary(q, k, freqs)[1] ** 2).sum().backward()
    assert q.grad is None and torch.allclose(k.grad, 2 * k, atol=1e-5)
    k.grad = None
    (ops.rotary(q, None, freqs)[0] ** 2).sum().backward()
    assert torch.allclose(q.grad, 2 * q, atol=1e-5) and k.grad is None
    # an expanded gradient, and one value shared by all heads
    v = torch.randn(2, 5, 1, 8, device="cuda", requires_grad=True)
    ops.linear_attention(q.detach(), k.detach(), v.expand(2, 5, 2, 8), torch.full((4,), -0.1, device="cuda")).sum().backward()
    assert v.grad.shape == v.shape and torch.isfinite(v.grad).all() and v.grad.any()
    x = torch.randn(3, 16, device="cuda", requires_grad=True)
    ops.layer_norm(x).sum().backward()
    assert x.grad.abs().max() < 1e-5  # the sum of a row's unit is 0 whatever the row is


def test_a_backward_pass_in_a_graph_beside_an_eager_one(example):
    ops = example.ops
    x = torch.randn(70, 64, device="cuda", requires_grad=True)
    w = torch.randn(300, 64, device="cuda", requires_grad=True)
    t = torch.randint(0, 300, (70,), device="cuda")
    want = torch.autograd.grad(ops.vocab_loss(ops.layer_norm(x), w, t).sum(), (x, w))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = (v.detach().clone().requires_grad_(True) for v in (x, w))  # leaves of the graph's own
    with torch.cuda.stream(s):
        torch.autograd.grad(ops.vocab_loss(ops.layer_norm(a), b, t).sum(), (a, b))
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = torch.autograd.grad(ops.vocab_loss(ops.layer_norm(a), b, t).sum(), (a, b))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_the_selective_model_trains_without_logits(example):
    import selective_blocks
    torch.manual_seed(3)
    m = selective_blocks.Model().cuda()
    seq = selective_blocks.batch(8, 4, "cuda", torch.Generator(device="cuda").manual_seed(4))
    y = m.hidden(seq[:, :-1])[:, 4:].flatten(0, 1)
    loss = example.ops.vocab_loss(y, m.embed.weight, seq[:, 5:].flatten()).mean()
    want = torch.nn.functional.cross_entropy(m(seq[:, :-1])[:, 4:].flatten(0, 1), seq[:, 5:].flatten())
    assert abs(loss.item() - want.item()) < 1e-5 * abs(want.item())
    params = list(m.parameters())
    for p, q in zip(torch.autograd.grad(loss, params), torch.autograd.grad(want, params)):
        assert (p - q).norm() <= 5e-5 * q.norm()
