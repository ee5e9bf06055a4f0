"""The selective scan's gradients where a sequence ends in an infinite state: what padding holds back stays
finite, and padding's own gradients are zeros."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.block_oracle as O  # noqa: E402
import structured_state_space_gb300 as s4  # noqa: E402
from block_util import need_gpu, to64  # noqa: E402
from test_gpu_selective import GRAD_TOL, lens, scan_inputs, split  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


# Lengths that end inside a tile of 16 tokens and inside and at the end of a block of four; channels that
# fill a block (64 channels of 16 states, 256 of 4) and others.
@pytest.mark.parametrize("H,N,G", [(64, 16, 1), (40, 16, 2), (256, 4, 1), (10, 100, 1)])
@pytest.mark.parametrize("L,n", [(21, [21, 13, 4]), (30, [29, 7, 18])])
def test_an_infinite_last_input(H, N, G, L, n):
    a, r = scan_inputs(H + N + L, 3, L, H, N, G, torch.float32)
    dy = r.normal(3, L, H)
    for b in range(3):
        for k in ("x", "dt", "z", "B", "C"):
            a[k][b, n[b]:] = 0
        dy[b, n[b]:] = 0
        a["x"][b, n[b] - 1, 1 + 2 * b] = float("inf")
    pos, named = split(a)
    got = s4.s4_selective_scan_bwd(*pos, dy, **named, lengths=lens(n))
    pos, named = split({k: to64(v) for k, v in a.items()})
    with np.errstate(invalid="ignore"):
        ref = O.selective_scan_grad(*pos, to64(dy), **named, lengths=n)
    assert np.isfinite(ref["dA"]).all() and np.isfinite(ref["dx"]).all()
    for k, v in got.items():
        v, finite = to64(v), np.isfinite(ref[k])
        assert np.isfinite(v[finite]).all(), k
        off = np.linalg.norm(v[finite] - ref[k][finite])
        assert off <= GRAD_TOL * np.linalg.norm(ref[k][finite]), (k, off)
        if k in ("dx", "ddt", "dz", "dB", "dC"):
            assert all((v[b, n[b]:] == 0).all() for b in range(3)), k
