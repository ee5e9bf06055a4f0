"""Lengths and targets out of range in the differentiable functions: recorded in the workspace that the caller gives."""
import pytest

torch = pytest.importorskip("torch")

import structured_state_space_gb300 as s4  # noqa: E402
from block_util import need_gpu  # noqa: E402
from structured_state_space_gb300 import autograd as ops  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_what_is_out_of_range_is_recorded(dtype):
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    h = torch.randn(9, 64, device="cuda").to(dtype).requires_grad_(True)
    w = torch.randn(50, 64, device="cuda").to(dtype).requires_grad_(True)
    t = torch.tensor([0, 49, 50, -1, 3, 3, 1 << 40, 5, 6], device="cuda")
    loss = ops.vocab_loss(h, w, t, ws=ws)
    assert s4.STATUS[s4.s4_get_status(ws)] == "S4_ERR_INVALID_INDEX"
    loss.sum().backward()
    assert not loss[[2, 3, 6]].any() and not h.grad[[2, 3, 6]].any() and w.grad.any()
    ok = ops.vocab_loss(h, w, torch.where(t < 50, t, -1), ws=ws)
    assert s4.s4_get_status(ws) == 0 and torch.equal(ok, loss)

    q = torch.randn(2, 70, 2, 32, device="cuda").to(dtype).requires_grad_(True)
    g = torch.tensor([-0.1, -0.2], device="cuda")
    o = ops.linear_attention(q, q, q, g, lengths=torch.tensor([70, 71], dtype=torch.int32, device="cuda"), ws=ws)
    assert s4.STATUS[s4.s4_get_status(ws)] == "S4_ERR_INVALID_INDEX" and not o[1].any() and o[0].any()
    o.sum().backward()
    assert not q.grad[1].any() and q.grad[0].any()
    ops.linear_attention(q, q, q, g, lengths=torch.tensor([70, 69], dtype=torch.int32, device="cuda"), ws=ws)
    assert s4.s4_get_status(ws) == 0


def test_a_workspace_used_again_has_the_last_calls_status():
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    h, w = torch.randn(9, 64, device="cuda"), torch.randn(50, 64, device="cuda")
    for _ in range(2):
        s4.s4_vocab_loss_fwd(h, w, torch.full((9,), 50, device="cuda"), ws=ws)
        assert s4.STATUS[s4.s4_get_status(ws)] == "S4_ERR_INVALID_INDEX"
        s4.s4_layer_norm_bwd(h, h, w[0], w[1], ws=ws)
        assert s4.s4_get_status(ws) == 0
