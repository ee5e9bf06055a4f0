"""The short causal convolution at every filter length, with whole packs of channels and with single ones, forward and
backward, against the float64 definition."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.block_oracle as O  # noqa: E402
import structured_state_space_gb300 as s4  # noqa: E402
from block_util import DTYPES, Inputs, close, need_gpu, to64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def lens(t):
    return torch.tensor(t, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("W", range(2, 9))
@pytest.mark.parametrize("L,H,left", [(37, 64, 8), (70, 33, 3), (530, 36, -1)])
def test_forward_and_gradients(dtype, W, L, H, left):
    dt, r = DTYPES[dtype], Inputs(100 * W + H)

    def rows():
        return r.normal(3, L, H, dtype=dt) if left < 0 else r.wide(3, L, H, dtype=dt, left=left, right=left)
    x, dy, w, b = rows(), rows(), r.normal(H, W), r.normal(H)
    st, ds = r.normal(3, W - 1, H, dtype=dt), r.normal(3, W - 1, H, dtype=dt)
    n = [L, W // 2, L - 3]
    out = torch.empty_like(st)
    y = s4.s4_short_conv_fwd(x, w, b, lengths=lens(n), state=st, state_out=out)
    ry, rs = O.short_conv(to64(x), to64(w), to64(b), lengths=n, state=to64(st))
    close(y, ry, "y")
    assert np.array_equal(to64(out), rs)
    g = s4.s4_short_conv_bwd(x, w, b, dy, lengths=lens(n), state=st, dstate=ds, want_dstate0=True)
    ref = O.short_conv_grad(to64(x), to64(w), to64(b), to64(dy), True, n, to64(st), to64(ds))
    for k in ref:
        close(g[k], ref[k], k)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("W", range(2, 9))
@pytest.mark.parametrize("H", [64, 33])
def test_single_tokens(dtype, W, H):
    dt, r = DTYPES[dtype], Inputs(W + H)
    x, w, b, st = r.normal(2, H, dtype=dt), r.normal(H, W), r.normal(H), r.normal(2, W - 1, H, dtype=dt)
    ry, rs = O.short_conv(to64(x)[:, None], to64(w), to64(b), state=to64(st))
    close(s4.s4_short_conv_step(x, w, b, st), ry[:, 0], "y")
    assert np.array_equal(to64(st), rs)
