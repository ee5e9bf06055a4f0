"""The differentiable functions of linear attention and rotary positions: what has no gradient may not ask for one (no GPU)."""
import pytest

torch = pytest.importorskip("torch")

from structured_state_space_gb300 import autograd as ops  # noqa: E402


def test_constants_that_require_gradients_are_refused():
    q = torch.zeros(1, 4, 2, 8, requires_grad=True)
    g, freqs = torch.zeros(2, requires_grad=True), torch.ones(4, dtype=torch.float64, requires_grad=True)
    with pytest.raises(ValueError, match="log_decay has no gradient"):
        ops.linear_attention(q, q, q, g)
    with pytest.raises(ValueError, match="freqs has no gradient"):
        ops.rotary(q, None, freqs)
    # without gradients, and detached, they go on to the library (which wants the GPU)
    with pytest.raises(ValueError, match="CUDA"):
        ops.linear_attention(q, q, q, g.detach())
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        ops.linear_attention(q, q, q, g)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        ops.rotary(q, None, freqs)
