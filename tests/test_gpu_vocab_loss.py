"""The vocabulary loss against its definition in float64.

Tolerances, relative in the 2-norm: losses and lse are float32 sums of exact products (1e-5).  With bfloat16 inputs
the logits' gradients are rounded to bfloat16 before the products that make dh and dw (2^-8 of each at most), which
are rounded once more: 2 x 2^-8.  With float16 inputs they go as two bfloat16 terms, with float32 as three."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.sequence_oracle as O  # noqa: E402
import structured_state_space_gb300 as s4  # noqa: E402
from block_util import DTYPES, F32_TOL, TOL, Inputs, close, need_gpu, to64  # noqa: E402

pytestmark = pytest.mark.gpu
GRAD = {torch.float32: F32_TOL, torch.bfloat16: 2 * 2.0 ** -8, torch.float16: TOL[torch.float16] + 2.0 ** -15}
SIZES = [(1, 8, 1), (1, 64, 1000), (3, 40, 257), (128, 64, 256), (129, 72, 300), (200, 33, 5000), (257, 256, 513), (40, 1000, 999),
         (1000, 128, 70), (2, 1, 3)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def make(seed, rows, H, V, dtype, scale=2.0):
    r = Inputs(seed)
    h, w = r.normal(rows, H, dtype=dtype), r.normal(V, H, dtype=dtype, scale=scale * H ** -0.5)
    t = torch.from_numpy(r.rng.integers(0, V, rows)).cuda()
    if rows > 2:
        t[1] = -100
        t[2] = V - 1
    return r, h, w, t


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dt", DTYPES)
def test_losses(size, dt):
    r, h, w, t = make(1, *size, DTYPES[dt])
    for targets in (t, t.int()):
        loss, lse = s4.s4_vocab_loss_fwd(h, w, targets)
        want, l64 = O.vocab_loss(to64(h), to64(w), t.cpu().numpy())
        close(lse, l64, "lse")
        # a loss is a difference of two sums of the logits' size
        assert np.linalg.norm(to64(loss) - want) <= 1e-5 * (np.linalg.norm(want) + np.linalg.norm(l64))
        assert (loss[t < 0] == 0).all()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dt", DTYPES)
def test_gradients(size, dt):
    r, h, w, t = make(2, *size, DTYPES[dt])
    dloss = r.normal(size[0], scale=3.0)
    loss, lse = s4.s4_vocab_loss_fwd(h, w, t)
    got = s4.s4_vocab_loss_bwd(h, w, t, lse, dloss)
    ref = O.vocab_loss_grad(to64(h), to64(w), t.cpu().numpy(), to64(dloss))
    if size[2] == 1:  # one word: the loss is 0 whatever h is, to what exp(x - lse) - 1 leaves
        assert got["dh"].abs().max() < 1e-4 and got["dw"].abs().max() < 1e-4
        return
    for n in ("dh", "dw"):
        close(got[n], ref[n], n, GRAD[got[n].dtype])


@pytest.mark.parametrize("dt", DTYPES)
def test_slices_and_leading_dimensions(dt):
    r = Inputs(3)
    dtype = DTYPES[dt]
    t = torch.from_numpy(r.rng.integers(0, 301, 60)).cuda()
    dl = r.normal(60)
    for left, H in ((0, 64), (3, 64), (8, 50)):
        h, w = r.wide(60, H, dtype=dtype, left=left, right=8), r.wide(301, H, dtype=dtype, left=left, right=8)
        a = s4.s4_vocab_loss_fwd(h, w, t)
        b = s4.s4_vocab_loss_fwd(h.contiguous().view(4, 15, H), w.contiguous(), t.view(4, 15))
        assert b[0].shape == (4, 15) and torch.equal(a[0], b[0].view(-1)) and torch.equal(a[1], b[1].view(-1))
        x = s4.s4_vocab_loss_bwd(h, w, t, a[1], dl)
        y = s4.s4_vocab_loss_bwd(h.contiguous().view(4, 15, H), w.contiguous(), t.view(4, 15), b[1], dl.view(4, 15))
        assert torch.equal(x["dh"], y["dh"].view(60, H)) and torch.equal(x["dw"], y["dw"])
    # every row the same one
    one = r.normal(1, 64, dtype=dtype)
    w = r.normal(301, 64, dtype=dtype)
    a, b = s4.s4_vocab_loss_fwd(one.expand(60, 64), w, t), s4.s4_vocab_loss_fwd(one.expand(60, 64).contiguous(), w, t)
    assert torch.equal(a[0], b[0])


def test_targets_out_of_range():
    r, h, w, t = make(4, 10, 16, 50, torch.float32)
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    t[5] = 50
    loss, lse = s4.s4_vocab_loss_fwd(h, w, t, ws=ws)
    assert s4.STATUS[s4.s4_get_status(ws)] == "S4_ERR_INVALID_INDEX" and loss[5] == 0 and torch.isfinite(lse).all()
    ws2 = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    g = s4.s4_vocab_loss_bwd(h, w, t, lse, torch.ones(10, device="cuda"), ws=ws2)
    assert s4.STATUS[s4.s4_get_status(ws2)] == "S4_ERR_INVALID_INDEX" and not g["dh"][5].any()
    t[5] = 49
    s4.s4_vocab_loss_fwd(h, w, t, ws=ws)
    assert s4.s4_get_status(ws) == 0


def test_rows_that_do_not_count_may_hold_anything():
    r, h, w, t = make(5, 200, 64, 600, torch.bfloat16)
    dl = r.normal(200)
    loss, lse = s4.s4_vocab_loss_fwd(h, w, t)
    g = s4.s4_vocab_loss_bwd(h, w, t, lse, dl)
    assert not g["dh"][1].any()
    # large logits, and rows with one certain word
    h2 = h * 200
    loss, lse = s4.s4_vocab_loss_fwd(h2, w, t)
    want, l64 = O.vocab_loss(to64(h2), to64(w), t.cpu().numpy())
    close(lse, l64, "lse")


def test_pieces_of_the_vocabulary():
    # rows x words beyond one piece of 256 MB of gradients of logits: 3 pieces
    rows, H, V = 4096, 64, 66000
    r = Inputs(6)
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(rows, H, device="cuda", generator=gen).bfloat16()
    w = (torch.randn(V, H, device="cuda", generator=gen) * 0.2).bfloat16()
    t = torch.randint(0, V, (rows,), device="cuda", generator=gen)
    dl = torch.rand(rows, device="cuda", generator=gen)
    loss, lse = s4.s4_vocab_loss_fwd(h, w, t)
    g = s4.s4_vocab_loss_bwd(h, w, t, lse, dl)
    x = h.double() @ w.double().t()
    l64 = torch.logsumexp(x, -1)
    at = torch.arange(rows, device="cuda")
    close(lse, to64(l64), "lse")
    close(loss, to64(l64 - x[at, t]), "loss")
    d = torch.exp(x - l64[:, None])
    d[at, t] -= 1
    d *= dl.double()[:, None]
    close(g["dh"], to64(d @ w.double()), "dh", 2 * 2.0 ** -8)
    close(g["dw"], to64(d.t() @ h.double()), "dw", 2 * 2.0 ** -8)


@pytest.mark.parametrize("rows,H,V", [(16384, 48, 300), (40, 64, 40000), (6000, 130, 700), (300, 1500, 9000)])
def test_long_sums_in_float32(rows, H, V):
    """Sums over many rows and many words: the tensor cores cut what they shift out of an accumulator towards zero, so an
    accumulator that takes up too many products drifts (6e-5 for 16384 rows in one)."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    h = torch.randn(rows, H, device="cuda", generator=gen)
    w = torch.randn(V, H, device="cuda", generator=gen) * 2 * H ** -0.5
    t = torch.randint(-1, V, (rows,), device="cuda", generator=gen)
    dl = torch.rand(rows, device="cuda", generator=gen)
    loss, lse = s4.s4_vocab_loss_fwd(h, w, t)
    g = s4.s4_vocab_loss_bwd(h, w, t, lse, dl)
    x = h.double() @ w.double().t()
    l64 = torch.logsumexp(x, -1)
    close(lse, to64(l64), "lse")
    d = torch.exp(x - l64[:, None])
    at = torch.arange(rows, device="cuda")
    d[at, t.clamp(min=0)] -= 1
    d *= torch.where(t >= 0, dl.double(), 0.0)[:, None]
    close(g["dh"], to64(d @ w.double()), "dh")
    close(g["dw"], to64(d.t() @ h.double()), "dw")
