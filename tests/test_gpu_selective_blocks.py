"""The selective block's operators together: the example model learns, decodes what it computes on whole
sequences, and its gradients are those of the same model in elementary float64 operations."""
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
    import selective_blocks
    return selective_blocks


def test_the_model_learns(example):
    torch.manual_seed(0)
    losses = example.train(example.Model().cuda(), 150)
    assert all(math.isfinite(v) for v in losses)
    # a uniform guess costs log 31 = 3.43; what the recalled half leaves to learn is all of it
    assert abs(losses[0] - math.log(31)) < 1.5 and sum(losses[-10:]) / 10 < 0.7 * losses[0], losses[::15]


def test_decoding_follows_the_whole_sequences(example):
    torch.manual_seed(1)
    # float32 throughout: two orders of the same sums over 2 layers, a few 1e-6 of the largest logit
    assert example.decode(example.Model().cuda()) < 2e-5


def _plain(m, tokens):
    """The example's forward in elementary operations, for any dtype."""
    def norm(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * w

    def silu(v):
        return v * torch.sigmoid(v)
    h = m.embed(tokens)
    y = norm(h, m.blocks[0].w_pre)
    for i, b in enumerate(m.blocks):
        x, z, gate = b.project(y)
        taps = b.conv.shape[1]
        seen = torch.nn.functional.pad(x, (0, 0, taps - 1, 0))
        u = silu(sum(seen[:, k:k + x.shape[1]] * b.conv[:, k] for k in range(taps)) + b.conv_bias)
        dt, B, C = b.select(u)
        d = torch.logaddexp(dt + b.dt_bias, torch.zeros_like(dt))
        s, ys = torch.zeros(*x.shape[::2], b.log_A.shape[1], dtype=x.dtype, device=x.device), []
        for t in range(x.shape[1]):
            s = torch.exp(d[:, t, :, None] * -torch.exp(b.log_A)) * s + (d * u)[:, t, :, None] * B[:, t]
            ys.append((s * C[:, t]).sum(-1) + b.D * u[:, t])
        v = b.out(torch.stack(ys, 1) * silu(z))
        h = h + b.scale * norm(v * silu(gate), b.w_post)
        y = norm(h, m.join(i))
    return torch.nn.functional.linear(y, m.embed.weight)


def test_gradients_of_the_whole_model(example):
    torch.manual_seed(2)
    m = example.Model().cuda()
    wide = example.Model().cuda().double()
    wide.load_state_dict({k: v.double() for k, v in m.state_dict().items()})
    tokens = torch.randint(0, example.VOCAB, (3, 21), device="cuda")
    weight = torch.randn(3, 21, example.VOCAB, device="cuda")
    (m(tokens) * weight).sum().backward()
    (_plain(wide, tokens) * weight.double()).sum().backward()
    for (k, p), q in zip(m.named_parameters(), wide.parameters()):
        # float32 through 2 layers forward and back: some 1e-6, a decade of room
        off = (p.grad.double() - q.grad).norm() / q.grad.norm()
        assert off < 5e-5, (k, off.item())


def test_shapes_without_a_gradient(example):
    from structured_state_space_gb300 import autograd as ops
    o = torch.randn(4, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    h, y = ops.block_norm(o, w_pre=w)
    y.sum().backward()
    assert o.grad is not None and w.grad is not None and torch.equal(h, o)
    h, y = ops.block_norm(o, w_post=w)
    assert y is None
    h.sum().backward()
