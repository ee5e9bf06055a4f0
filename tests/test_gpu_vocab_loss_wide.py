"""The vocabulary loss of many channels: logits that one accumulator of the tensor cores, which cuts off what its additions shift
out, would let drift (16384 channels in float32 1.2e-5 in lse, all of one sign).

Tolerances, relative in the 2-norm, as in test_gpu_vocab_loss.py: an accumulator that takes up 8192 products (logits of 16-bit inputs)
is off by 6e-6 at most, within the 1e-5 of float32 results; in float32 they go in parts of 1024, so below 1e-6."""
import pytest

torch = pytest.importorskip("torch")

import structured_state_space_gb300 as s4  # noqa: E402
from block_util import DTYPES, close, need_gpu, to64  # noqa: E402
from test_gpu_vocab_loss import GRAD  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


# rows, channels, words: two parts (the second of one channel, or one of eight), four; more tiles than SMs
@pytest.mark.parametrize("size", [(100, 4097, 700), (200, 8200, 300), (300, 16384, 2000), (2500, 9000, 2600)])
@pytest.mark.parametrize("shift", [0.0, 0.3])
@pytest.mark.parametrize("dt", DTYPES)
def test_many_channels(size, shift, dt):
    rows, H, V = size
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = (torch.randn(rows, H, device="cuda", generator=gen) + shift).to(DTYPES[dt])
    w = ((torch.randn(V, H, device="cuda", generator=gen) * 2 + shift) * H ** -0.5).to(DTYPES[dt])
    t = torch.randint(-1, V, (rows,), device="cuda", generator=gen)
    dl = torch.rand(rows, device="cuda", generator=gen)
    loss, lse = s4.s4_vocab_loss_fwd(h, w, t)
    got = s4.s4_vocab_loss_bwd(h, w, t, lse, dl)
    x = h.double() @ w.double().t()
    l64 = torch.logsumexp(x, -1)
    close(lse, to64(l64), "lse", 1e-6 if dt == "f32" else None)
    at = torch.arange(rows, device="cuda")
    want = torch.where(t >= 0, l64 - x[at, t.clamp(min=0)], 0.0)
    assert (loss.double() - want).norm() <= 1e-5 * (want.norm() + l64.norm())
    d = torch.exp(x - l64[:, None])
    d[at, t.clamp(min=0)] -= 1
    d *= torch.where(t >= 0, dl.double(), 0.0)[:, None]
    close(got["dh"], to64(d @ w.double()), "dh", GRAD[h.dtype])
    close(got["dw"], to64(d.t() @ h.double()), "dw", GRAD[h.dtype])


def test_many_rows_in_16_bits():
    """dw over 2^18 rows in one accumulator was short by 1.3e-4 of itself; in parts of 65536 rows it is by 4096 additions of
    1e-8 at most (the roundings to float16 are as often up as down: 2^-12 over the root of their number).  The logits,
    H / 16 additions, are short by 2.6e-6 of themselves as well: of 12 at most (6 times their deviation of 2) 3.1e-5, their lse
    by no more, and the relative error of exp(x - lse) is the difference of the two, 6.2e-5 at most."""
    rows, H, V, some = 1 << 18, 4096, 1024, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    h = torch.randn(rows, H, device="cuda", generator=gen, dtype=torch.float16)
    w = (torch.randn(V, H, device="cuda", generator=gen) * 2 * H ** -0.5).half()
    t = torch.randint(-1, V, (rows,), device="cuda", generator=gen)
    dl = torch.rand(rows, device="cuda", generator=gen) + 1
    loss, lse = s4.s4_vocab_loss_fwd(h, w, t)
    got = s4.s4_vocab_loss_bwd(h, w, t, lse, dl)["dw"][:, :some].double()
    want = torch.zeros_like(got)
    step = 1 << 14
    at = torch.arange(step, device="cuda")
    for a in range(0, rows, step):
        x, targets = h[a:a + step].double() @ w.double().t(), t[a:a + step]
        d = torch.exp(x - torch.logsumexp(x, -1, keepdim=True))
        d[at, targets.clamp(min=0)] -= 1
        d *= torch.where(targets >= 0, dl[a:a + step].double(), 0.0)[:, None]
        want += d.t() @ h[a:a + step, :some].double()
    close(got, to64(want), "dw", GRAD[torch.float16])
    short = ((got * want).sum() / (want * want).sum() - 1).abs().item()
    assert short <= 4096 * 1e-8 + 2.0 ** -12 * (V * some) ** -0.5 + 2 * 12 * (H / 16) * 1e-8, short


@pytest.mark.parametrize("rows,H,V", [(16384, 48, 300), (40, 64, 40000), (6000, 130, 700), (300, 1500, 9000), (4096, 64, 66000)])
def test_gradients_in_float32_keep_their_digits(rows, H, V):
    """Sums over many rows and words in parts of 1024: 64 additions of 1e-8, and as much from the logits (|x - lse| below 16, whose 3e-7
    are 5e-6 of the smallest gradients, 1e-6 of those that count): 2e-6 in the 2-norm."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    h = torch.randn(rows, H, device="cuda", generator=gen)
    w = torch.randn(V, H, device="cuda", generator=gen) * 2 * H ** -0.5
    t = torch.randint(-1, V, (rows,), device="cuda", generator=gen)
    dl = torch.rand(rows, device="cuda", generator=gen)
    loss, lse = s4.s4_vocab_loss_fwd(h, w, t)
    got = s4.s4_vocab_loss_bwd(h, w, t, lse, dl)
    x = h.double() @ w.double().t()
    d = torch.exp(x - torch.logsumexp(x, -1, keepdim=True))
    at = torch.arange(rows, device="cuda")
    d[at, t.clamp(min=0)] -= 1
    d *= torch.where(t >= 0, dl.double(), 0.0)[:, None]
    close(got["dh"], to64(d @ w.double()), "dh", 2e-6)
    close(got["dw"], to64(d.t() @ h.double()), "dw", 2e-6)
