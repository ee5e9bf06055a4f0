"""Rows without a target in the vocabulary loss: what padding holds reaches nothing but its own lse."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.sequence_oracle as O  # noqa: E402
import structured_state_space_gb300 as s4  # noqa: E402
from block_util import DTYPES, Inputs, close, need_gpu, to64  # noqa: E402
from test_gpu_vocab_loss import GRAD  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


# rows, channels (tiles of 64, 128 and 256 columns), words; the third has more rows than one fp32 accumulator takes
@pytest.mark.parametrize("size", [(200, 64, 600), (65, 128, 1000), (5000, 40, 300), (333, 264, 257), (64, 100, 70), (1, 64, 30)])
@pytest.mark.parametrize("dt", DTYPES)
def test_rows_without_a_target_hold_anything(size, dt):
    rows, H, V = size
    r = Inputs(1)
    h, w, dl = r.normal(rows, H, dtype=DTYPES[dt]), r.normal(V, H, dtype=DTYPES[dt], scale=2 * H ** -0.5), r.normal(rows)
    t = torch.from_numpy(r.rng.integers(0, V, rows)).cuda()
    out = torch.from_numpy(r.rng.random(rows) < 0.4).cuda()
    out[-1] = True
    if rows > 128:
        out[64:128] = True  # a whole tile of them
    t[out] = torch.from_numpy(r.rng.choice([-1, -100, V, V + 7], rows)).cuda()[out]
    clean, dirty = h.clone(), h.clone()
    clean[out] = 0
    n = int(out.sum())
    dirty[out] = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda", dtype=h.dtype)[torch.arange(n * H, device="cuda") % 3].view(n, H)
    dl2 = dl.clone()
    dl2[out] = float("nan")
    for targets in (t, t.int()):
        loss, lse = s4.s4_vocab_loss_fwd(clean, w, targets)
        want = s4.s4_vocab_loss_bwd(clean, w, targets, lse, dl)
        loss2, lse2 = s4.s4_vocab_loss_fwd(dirty, w, targets)
        assert torch.equal(loss, loss2) and not loss[out].any() and torch.equal(lse[~out], lse2[~out])
        got = s4.s4_vocab_loss_bwd(dirty, w, targets, lse2, dl2)
        assert torch.equal(got["dw"], want["dw"]) and torch.equal(got["dh"], want["dh"]) and not got["dh"][out].any()
    ref = O.vocab_loss_grad(to64(clean), to64(w), np.where(out.cpu().numpy(), -1, t.cpu().numpy()), to64(dl))
    if not out.all():
        close(got["dw"], ref["dw"], "dw", GRAD[h.dtype])
