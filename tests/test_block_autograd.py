"""The selective block's differentiable functions with create_graph=True (no GPU: the library's calls are
stand-ins).  Their gradients have no gradients of their own: a second derivative has to raise, never to
be left out."""
import pytest

torch = pytest.importorskip("torch")

from structured_state_space_gb300 import autograd as ops  # noqa: E402
from structured_state_space_gb300 import block  # noqa: E402


def _zeros_of(**named):
    return {k: torch.zeros_like(v) for k, v in named.items() if v is not None}


@pytest.fixture()
def calls(monkeypatch):
    """Each operator as a function of its inputs' shapes: outputs of ones, gradients of zeros."""
    def conv_bwd(x, w, bias, dy, *, lengths=None):
        return _zeros_of(dx=x, dw=w, dbias=bias)

    def scan_bwd(x, dt, A, B, C, dy, *, D=None, z=None, dt_bias=None, lengths=None):
        return _zeros_of(dx=x, ddt=dt, dA=A, dB=B, dC=C, dD=D, dz=z, ddt_bias=dt_bias)

    def norm(o, *, gate=None, h=None, w_post=None, scale=None, w_pre=None, eps=0.0):
        return torch.ones_like(o), None if w_pre is None else torch.ones_like(o)

    def norm_bwd(o, dy=None, *, dh_out=None, gate=None, h=None, w_post=None, scale=None, w_pre=None, eps=0.0):
        return {"do": torch.zeros_like(o)} | _zeros_of(dgate=gate, dh=h, dw_post=w_post, dscale=scale, dw_pre=w_pre)
    monkeypatch.setattr(block, "s4_short_conv_fwd", lambda x, *a, **kw: torch.ones_like(x))
    monkeypatch.setattr(block, "s4_short_conv_bwd", conv_bwd)
    monkeypatch.setattr(block, "s4_selective_scan_fwd", lambda x, *a, **kw: torch.ones_like(x))
    monkeypatch.setattr(block, "s4_selective_scan_bwd", scan_bwd)
    monkeypatch.setattr(block, "s4_block_norm_fwd", norm)
    monkeypatch.setattr(block, "s4_block_norm_bwd", norm_bwd)


def leaf(*shape):
    return torch.ones(shape, requires_grad=True)


def conv():
    x, w = leaf(2, 5, 4), leaf(4, 3)
    return [x, w], ops.short_conv(x, w)


def scan():
    x, dt, A, B, C = leaf(2, 5, 4), leaf(2, 5, 4), leaf(4, 6), leaf(2, 5, 1, 6), leaf(2, 5, 1, 6)
    return [x, dt, A, B, C], ops.selective_scan(x, dt, A, B, C)


def norms():
    o, w = leaf(3, 4), leaf(4)
    return [o, w], ops.block_norm(o, w_pre=w)[1]


def norm_alone():
    o, w = leaf(3, 4), leaf(4)
    return [o, w], ops.block_norm(o, w_post=w)[0]


@pytest.mark.parametrize("make", [conv, scan, norms, norm_alone])
@pytest.mark.parametrize("weighted", [False, True])
def test_a_second_derivative_raises(calls, make, weighted):
    leaves, y = make()
    # the gradient of the output itself may or may not depend on what is differentiated
    loss = (y * y).sum() if weighted else y.sum()
    g = torch.autograd.grad(loss, leaves, create_graph=True)
    with pytest.raises(RuntimeError):
        (loss + sum((v ** 2).sum() for v in g)).backward()


@pytest.mark.parametrize("make", [conv, scan, norms, norm_alone])
def test_one_of_the_gradients_is_enough(calls, make):
    leaves, y = make()
    g = torch.autograd.grad(y.sum(), leaves[:1], create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad((g[0] ** 2).sum(), leaves[-1])


@pytest.mark.parametrize("make", [conv, scan, norms, norm_alone])
def test_first_derivatives_are_as_before(calls, make):
    leaves, y = make()
    y.sum().backward()
    assert all((v.grad == 0).all() for v in leaves)
    leaves, y = make()
    g = torch.autograd.grad(y.sum(), leaves, create_graph=True)  # a graph that is not used costs nothing
    assert all((v.detach() == 0).all() and v.shape == t.shape for v, t in zip(g, leaves))
