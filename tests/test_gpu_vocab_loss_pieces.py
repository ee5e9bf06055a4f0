"""Gradients of the vocabulary loss over several pieces of the vocabulary (512 MB of logits' gradients each) in every type: 4096 rows
and 66000 words are 2 pieces in bfloat16, 3 in float16 (two terms) and 4 in float32 (three), 140000 words 3 in bfloat16."""
import pytest

torch = pytest.importorskip("torch")

import structured_state_space_gb300 as s4  # noqa: E402
from block_util import DTYPES, close, need_gpu, to64  # noqa: E402
from test_gpu_vocab_loss import GRAD  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,V", [("f32", 66000), ("f16", 66000), ("bf16", 140000)])
def test_pieces_of_every_type(dt, V):
    need_gpu()
    rows, H, dtype = 4096, 72, DTYPES[dt]
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(rows, H, device="cuda", generator=gen).to(dtype)
    w = (torch.randn(V, H, device="cuda", generator=gen) * 0.2).to(dtype)
    t = torch.randint(0, V, (rows,), device="cuda", generator=gen)
    t[:3] = torch.tensor([0, V - 1, -1], device="cuda")
    dl = torch.rand(rows, device="cuda", generator=gen)
    clean = h.clone()
    h[2] = float("nan")
    clean[2] = 0
    loss, lse = s4.s4_vocab_loss_fwd(h, w, t)
    g = s4.s4_vocab_loss_bwd(h, w, t, lse, dl)
    x = clean.double() @ w.double().t()
    l64 = torch.logsumexp(x, -1)
    at, live = torch.arange(rows, device="cuda"), t >= 0
    close(lse[live], to64(l64[live]), "lse")
    close(loss[live], to64((l64 - x[at, t.clamp(min=0)])[live]), "loss")
    d = torch.exp(x - l64[:, None])
    d[at, t.clamp(min=0)] -= 1
    d *= torch.where(live, dl.double(), 0.0)[:, None]
    close(g["dh"], to64(d @ w.double()), "dh", GRAD[dtype])
    close(g["dw"], to64(d.t() @ clean.double()), "dw", GRAD[dtype])
