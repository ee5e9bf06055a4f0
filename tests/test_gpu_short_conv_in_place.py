"""The short causal convolution of single tokens whose output replaces the input."""
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


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("batch,H,W,left", [(1, 8, 4, 8), (3, 64, 4, 8), (2, 33, 2, 3), (5, 130, 8, 1)])
def test_a_token_in_place_leaves_its_input_in_the_state(dtype, batch, H, W, left):
    r, dt = Inputs(H + W), DTYPES[dtype]
    x, w, b = r.wide(batch, H, dtype=dt, left=left, right=8), r.normal(H, W), r.normal(H)
    state = r.normal(batch + 1, W - 1, H, dtype=dt)
    index = torch.arange(batch, 0, -1, dtype=torch.int32, device="cuda")
    want = to64(state)
    ry, rs = O.short_conv(to64(x)[:, None], to64(w), to64(b), state=want[index.cpu().numpy()])
    want[index.cpu().numpy()] = rs
    y = s4.s4_short_conv_step(x, w, b, state, index=index, y=x)
    assert y.data_ptr() == x.data_ptr()
    close(y, ry[:, 0], "y")
    assert np.array_equal(to64(state), want)


def test_a_row_of_no_real_token_keeps_its_state_in_place():
    r = Inputs(4)
    x, w, state = r.normal(2, 1, 16), r.normal(16, 4), r.normal(2, 3, 16)
    kept, n = state.clone(), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    first = x.clone()
    s4.s4_short_conv_fwd(x, w, lengths=n, state=state, state_out=state, y=x)
    assert torch.equal(state[0], kept[0]) and (x[0] == 0).all()
    assert torch.equal(state[1], torch.cat([kept[1, 1:], first[1]]))


def test_in_place_needs_the_same_addresses():
    r = Inputs(5)
    wide, w = r.normal(4, 16), r.normal(16, 4)
    state = r.normal(2, 3, 16)
    with pytest.raises(s4.S4Error):  # the second output would be the second input of another row
        s4.s4_short_conv_step(wide[::2], w, None, state, y=wide[:2])
