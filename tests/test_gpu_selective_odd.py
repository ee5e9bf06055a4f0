"""The selective scan's gradients where an odd number of channels meets whole words of states: rows of
partial sums of several sequences and segments, in every type."""
import pytest

torch = pytest.importorskip("torch")

from block_util import DTYPES, need_gpu  # noqa: E402
from test_gpu_selective import check_gradients, scan_inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


# H (N + 2) is 2 modulo 4 here: without padding, every second row of the sums over (sequence, segment)
# starts in the middle of a word of 16 bytes.  Two sequences; one sequence of several segments.
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("N", [4, 8, 16, 64])
@pytest.mark.parametrize("batch,L,H,G", [(2, 9, 5, 1), (3, 33, 33, 3), (1, 70, 7, 1), (2, 40, 333, 1)])
def test_gradients_with_odd_channels(dtype, N, batch, L, H, G):
    dt = DTYPES[dtype]
    a, r = scan_inputs(L * N + H + 2, batch, L, H, N, G, dt)
    dy = r.normal(batch, L, H, dtype=dt)
    check_gradients(a, dy, state=r.normal(batch, H, N), dstate=r.normal(batch, H, N), want_dstate0=True)
