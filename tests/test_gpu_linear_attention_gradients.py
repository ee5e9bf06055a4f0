"""Gradients of linear attention where a batch's sequences end in different segments, at the ends of the range of decays, and in
one launch or two.  Tolerances as in test_gpu_linear_attention.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.sequence_oracle as O  # noqa: E402
import structured_state_space_gb300 as s4  # noqa: E402
from block_util import DTYPES, F32_TOL, close, need_gpu, to64  # noqa: E402
from test_gpu_linear_attention import OUT, SIZES, make, wide  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


# several segments, which the sequences end in or leave unused, and the shared heads of one kernel's sizes
@pytest.mark.parametrize("size", [(4, 1100, 2, 2, 64, 64), (3, 1500, 4, 2, 128, 64), (3, 1300, 2, 2, 128, 128), (2, 1100, 2, 1, 64, 128),
                                  (4, 900, 2, 1, 33, 7), (2, 700, 2, 1, 48, 200), SIZES[11]])
@pytest.mark.parametrize("dt", DTYPES)
def test_sequences_that_end_in_different_segments(size, dt):
    batch, L, H, G, K, V = size
    r, q, k, v, g = make(1, *size, DTYPES[dt])
    do = r.normal(batch, L, H, V, dtype=DTYPES[dt])
    lens = ([L - 1, 129, 0, L] if L > 129 else [L - 1, L])[:batch]
    s0, ds = r.normal(batch, H, K, V), r.normal(batch, H, K, V)
    for b, n in enumerate(lens):
        for t in (q, k, v, do):
            t[b, n:] = float("nan")
    got = s4.s4_linear_attention_bwd(q, k, v, g, do, lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"), state=s0,
                                     dstate=ds, want_dstate0=True)
    clean = [torch.nan_to_num(t, 0.0) for t in (q, k, v, do)]
    ref = O.linear_attention_grad(*wide(*clean[:3], g, clean[3]), K ** -0.5, lens, to64(s0), to64(ds))
    for n, want in ref.items():
        close(got[n], want, n, F32_TOL if n == "dstate0" else OUT[got[n].dtype])
        for b, length in enumerate(lens):
            assert n == "dstate0" or not got[n][b, length:].any(), n


@pytest.mark.parametrize("dt", DTYPES)
def test_decays_of_one_of_none_and_in_between(dt):
    size = (2, 300, 4, 2, 64, 96)
    r, q, k, v, _ = make(2, *size, DTYPES[dt])
    do, s0 = r.normal(2, 300, 4, 96, dtype=DTYPES[dt]), r.normal(2, 4, 64, 96)
    g = torch.tensor([0.0, float("-inf"), -80.0, -1e-7], device="cuda")
    w = np.array([0.0, -1e30, -80.0, -1e-7])
    out = torch.empty_like(s0)
    o = s4.s4_linear_attention_fwd(q, k, v, g, state=s0, state_out=out)
    ref, s = O.linear_attention(*wide(q, k, v), w, 64 ** -0.5, None, to64(s0))
    got = s4.s4_linear_attention_bwd(q, k, v, g, do, state=s0)
    want = O.linear_attention_grad(*wide(q, k, v), w, to64(do), 64 ** -0.5, None, to64(s0))
    for h in range(4):
        close(o[:, :, h], ref[:, :, h], f"o of head {h}", OUT[o.dtype])
        close(out[:, h], s[:, h], f"state of head {h}", F32_TOL)
        close(got["dq"][:, :, h], want["dq"][:, :, h], f"dq of head {h}", OUT[o.dtype])
    for n in ("dk", "dv"):
        close(got[n], want[n], n, OUT[o.dtype])


@pytest.mark.parametrize("size", [(2, 1500, 4, 4, 128, 128), (2, 1500, 4, 4, 64, 64), (1, 700, 4, 4, 256, 128)])
def test_bfloat16_loses_no_more_than_its_two_roundings(size):
    """Many elements, rounded twice: the weights (or the state) and the output.  A rounding is off by half a step at most, evenly
    spread: 2^-8 / sqrt(3) of the element in the mean square at most, and the two are independent.  2 % of room for chance
    (10^5 elements and more)."""
    batch, L, H, G, K, V = size
    r, q, k, v, g = make(3, *size, torch.bfloat16)
    do = r.normal(batch, L, H, V, dtype=torch.bfloat16)
    most = 1.02 * (2 / 3) ** 0.5 * 2.0 ** -8
    close(s4.s4_linear_attention_fwd(q, k, v, g), O.linear_attention(*wide(q, k, v, g), K ** -0.5)[0], "o", most)
    got = s4.s4_linear_attention_bwd(q, k, v, g, do)
    want = O.linear_attention_grad(*wide(q, k, v, g), to64(do), K ** -0.5)
    for n in ("dq", "dk", "dv"):
        close(got[n], want[n], n, most)


@pytest.mark.parametrize("heads,L,launches", [(8, 64, 1), (152, 64, 2), (4, 333, 3), (8, 333, 3), (16, 333, 6), (2, 16000, 6)])
def test_one_launch_where_all_walks_fit_the_gpu(heads, L, launches):
    """Walks of 48 and 80 channels: one launch while 4 CTAs for each 64 tokens of a head are two for each SM at most, else one for
    each width (with segments three kernels each)."""
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("counted for 152 SMs")
    r, q, k, v, g = make(4, 1, L, heads, heads, 48, 80, torch.float32)
    do = r.normal(1, L, heads, 80)
    s4.timing.enable()
    s4.timing.reset()
    try:
        got = s4.s4_linear_attention_bwd(q, k, v, g, do)
        assert s4.timing.read("linear_attention")[0] == launches
    finally:
        s4.timing.enable(False)
    if L < 1000:
        want = O.linear_attention_grad(*wide(q, k, v, g), to64(do), 48 ** -0.5)
        for n in ("dq", "dk", "dv"):
            close(got[n], want[n], n)


@pytest.mark.parametrize("size", [(2, 333, 2, 2, 48, 80), (1, 400, 2, 1, 64, 64), (1, 400, 2, 2, 128, 128), (1, 300, 1, 1, 256, 256)])
def test_float32_keeps_its_digits(size):
    """Relative in the 2-norm: weights off by the exponential's 2^-22, and what the tensor cores cut off their accumulators: 2e-8 for each of the
    additions of 16 products, K / 16 and V / 16 of them in a row and 4 for a chunk's tokens."""
    batch, L, H, G, K, V = size
    r, q, k, v, _ = make(5, *size, torch.float32)
    g = torch.tensor([-0.03, -0.0005], device="cuda")[:H]
    do = r.normal(batch, L, H, V)
    most = 2.0 ** -22 + 2e-8 * (K / 16 + V / 16 + 4)
    close(s4.s4_linear_attention_fwd(q, k, v, g), O.linear_attention(*wide(q, k, v, g), K ** -0.5)[0], "o", most)
    got = s4.s4_linear_attention_bwd(q, k, v, g, do)
    want = O.linear_attention_grad(*wide(q, k, v, g), to64(do), K ** -0.5)
    for n in ("dq", "dk", "dv"):
        close(got[n], want[n], n, most)
