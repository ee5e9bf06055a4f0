"""The selective scan's compiled instances that take whole packs and whole tiles (channels that fill the warps' and CTAs'
blocks, 8, 16 or 32 states, aligned arrays), against the float64 definition: prompts, ragged and chunked, gradients,
single tokens; and the step sizes to their relative precision."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.block_oracle as O  # noqa: E402
import structured_state_space_gb300 as s4  # noqa: E402
from block_util import DTYPES, Inputs, close, need_gpu, to64  # noqa: E402
from test_gpu_selective import GRAD_TOL, STATE_TOL, check_gradients, lens, reference, scan_inputs, split  # noqa: E402

pytestmark = pytest.mark.gpu

# (channels, states, groups): per group a multiple of the gradients' CTA block (128, 64, 32 channels with 8, 16, 32
# states), which the forward's warp blocks (64, 32, 16) divide
WHOLE = [(128, 8, 1), (256, 8, 2), (64, 16, 1), (128, 16, 2), (32, 32, 1), (96, 32, 3)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,N,G", WHOLE)
@pytest.mark.parametrize("L", [2, 32, 45])
def test_prompts(dtype, H, N, G, L):
    a, r = scan_inputs(H + N + L, 2, L, H, N, G, DTYPES[dtype])
    state = r.normal(2, H, N)
    out = torch.empty_like(state)
    pos, named = split(a)
    y = s4.s4_selective_scan_fwd(*pos, **named, state=state, state_out=out)
    ry, rs = reference(a, state=to64(state))
    close(y, ry, "y", None if dtype != "f32" else STATE_TOL)
    close(out, rs, "state", STATE_TOL)


def ragged(seed, L, H, N, G, dtype):
    """Inputs of six sequences, some short or empty; the same with infinities and NaN in the padding."""
    n = [L, 0, 1, L // 2, 16, L - 1]
    a, r = scan_inputs(seed, 6, L, H, N, G, dtype)
    dy = r.normal(6, L, H, dtype=dtype)
    for b in range(6):
        for v in [dy] + [a[k] for k in ("x", "dt", "z", "B", "C")]:
            v[b, n[b]:] = 0
    dirty, ddy = {k: v.clone() for k, v in a.items()}, dy.clone()
    for b in range(6):
        for v in [ddy] + [dirty[k] for k in ("x", "dt", "z", "B", "C")]:
            v[b, n[b]:] = float("nan") if b % 2 else float("inf")
    return n, a, dy, dirty, ddy, r


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,N,G", WHOLE)
@pytest.mark.parametrize("L", [75, 700])  # in one piece, and in chunks where there are few channels
def test_ragged_prompts(dtype, H, N, G, L):
    n, a, _, dirty, _, r = ragged(H + N + L, L, H, N, G, DTYPES[dtype])
    cache, index = r.normal(9, H, N), [4, 8, 0, 2, -1, 7]
    want = to64(cache)
    pos, named = split(dirty)
    y = s4.s4_selective_scan_fwd(*pos, **named, lengths=lens(n), state=cache, state_out=cache, index=lens(index))
    ry, rs = reference(a, lengths=n, state=want[np.maximum(index, 0)])
    ry[4] = 0
    close(y, ry, "y", None if dtype != "f32" else STATE_TOL)
    for b in range(6):
        assert (to64(y)[b, n[b]:] == 0).all()
        if index[b] >= 0:
            want[index[b]] = rs[b]
    close(cache, want, "cache", STATE_TOL)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,N,G", WHOLE)
@pytest.mark.parametrize("L", [3, 32, 45])
def test_gradients(dtype, H, N, G, L):
    dt = DTYPES[dtype]
    a, r = scan_inputs(H + N + L + 1, 2, L, H, N, G, dt)
    check_gradients(a, r.normal(2, L, H, dtype=dt), state=r.normal(2, H, N), dstate=r.normal(2, H, N), want_dstate0=True)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,N,G", WHOLE)
def test_ragged_gradients(dtype, H, N, G):
    n, a, dy, dirty, ddy, r = ragged(H + N, 75, H, N, G, DTYPES[dtype])
    kw = dict(lengths=n, state=r.normal(6, H, N), dstate=r.normal(6, H, N), want_dstate0=True)
    g = check_gradients(a, dy, **kw)
    pos, named = split(dirty)
    again = s4.s4_selective_scan_bwd(*pos, ddy, **named, **{**kw, "lengths": lens(n)})
    for k in g:
        assert torch.equal(g[k], again[k]), k
        if k in ("dx", "ddt", "dz", "dB", "dC"):
            assert all((again[k][b, n[b]:] == 0).all() for b in range(6)), k


@pytest.mark.parametrize("H,N", [(128, 8), (64, 16), (32, 32)])
def test_gradients_over_segments(H, N):
    a, r = scan_inputs(H + N, 1, 1501, H, N, 1, torch.float32)
    check_gradients(a, r.normal(1, 1501, H), state=r.normal(1, H, N), dstate=r.normal(1, H, N), want_dstate0=True)


# A thread takes 8 states of one channel, a CTA 1024 of them: (channels, states, groups) that fill it
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,N,G", [(128, 8, 1), (256, 8, 2), (64, 16, 1), (192, 16, 3), (32, 32, 1), (16, 64, 1), (32, 64, 2),
                                   (8, 128, 1), (4, 256, 1), (12, 256, 3)])
def test_single_tokens(dtype, H, N, G):
    batch = 5
    a, r = scan_inputs(H + N + 3, batch, 1, H, N, G, DTYPES[dtype])
    cache = r.normal(batch + 3, H, N)
    index = np.array([6, 0, -1, 3, 7])
    old = to64(cache)
    ry, rs = reference(a, state=old[np.maximum(index, 0)])
    pos, named = split({k: v[:, 0] if v.dim() > 2 else v for k, v in a.items()})
    out = cache.clone()
    y = s4.s4_selective_step(*pos, cache, **named, state_out=out, index=lens(index.tolist()))
    want = old.copy()
    ry[2] = 0
    for b in (0, 1, 3, 4):
        want[index[b]] = rs[b]
    close(y, ry[:, 0], "y")
    close(out, want, "state")
    assert torch.equal(y, s4.s4_selective_step(*pos, cache, **named, index=lens(index.tolist()))) and torch.equal(cache, out)


# log(1 + e^v) is formed as max(v, 0) + log1p(u), u = 2^(-|v| log2 e).  The exponent is rounded once and its constant is off
# by 2^-26: |v| 1.25 2^-24 relative in u.  Powers of two and reciprocals are approximate to 2^-22 and 2^-23; the products,
# the polynomial (8e-9) and the last sum add about four roundings of 2^-24: 10 + 1.25 |v|, here 16 + 2 |v|, units of 2^-24.
# Results below the smallest normal number (2^-126) may be zeros.
def steps_of(v, seed):
    r = Inputs(seed)
    bias = r.normal(v.shape[-1], scale=0.25)
    raw = (torch.tensor(v, dtype=torch.float32, device="cuda") - bias).contiguous()
    return raw, bias, to64(raw) + to64(bias)


VALUES = np.concatenate([-np.geomspace(1e-6, 86.0, 500), [0.0], np.geomspace(1e-6, 86.0, 523)])


@pytest.mark.parametrize("L", [1, 2])  # single tokens, and prompts
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_are_precise_relative_to_their_size(L, dtype):
    # with x = B = 1 the state after the first token is the step itself
    H, dt = len(VALUES), DTYPES[dtype]
    if dtype == "f32":
        raw, bias, _ = steps_of(VALUES, 1)
    else:
        raw, bias = torch.tensor(VALUES, device="cuda").to(dt), None
    exact_raw = to64(raw.float() if bias is None else raw + bias)  # the sum is rounded once before the softplus
    ones = torch.ones(1, L, 1, 1, dtype=dt, device="cuda")
    out = torch.empty(1, H, 1, device="cuda")
    s4.s4_selective_scan_fwd(torch.ones(1, L, H, dtype=dt, device="cuda"), raw.expand(1, L, H), -torch.ones(H, 1, device="cuda"),
                             ones, ones, dt_bias=bias, lengths=lens([1]), state_out=out)
    want = np.logaddexp(exact_raw, 0.0)
    bound = (16 + 2 * np.abs(exact_raw)) * 2.0 ** -24 * want + 2.0 ** -126
    off = np.abs(to64(out).ravel() - want)
    assert (off <= bound).all(), (exact_raw[np.argmax(off / bound)], (off / bound).max())


def test_the_steps_derivative_is_precise_relative_to_its_size():
    # with everything else 1 and no state on entry, ddt is the softplus' derivative sigmoid(v), formed of the step d as
    # 1 - e^-d: the step's bound, 2^-23 for the polynomial below d = 1/2 and some roundings, and above it 2^-22 and the
    # exponent's rounding of e^-d < 0.61 against results above 0.39
    raw, bias, _ = steps_of(VALUES, 2)
    H = len(VALUES)
    exact_raw = to64(raw + bias)
    one = torch.ones(1, 1, H, device="cuda")
    unit = torch.ones(1, 1, 1, 1, device="cuda")
    g = s4.s4_selective_scan_bwd(one, raw.expand(1, 1, H), -torch.ones(H, 1, device="cuda"), unit, unit, one, dt_bias=bias)
    want = O.sigmoid(exact_raw)
    small = exact_raw < -20  # where tanh has lost the digits
    want[small] = np.exp(exact_raw[small] - np.log1p(np.exp(exact_raw[small])))
    bound = (32 + 2 * np.abs(exact_raw)) * 2.0 ** -24 * want + 2.0 ** -126
    off = np.abs(to64(g["ddt"]).ravel() - want)
    assert (off <= bound).all(), (exact_raw[np.argmax(off / bound)], (off / bound).max())
    assert GRAD_TOL > bound[np.abs(exact_raw) < 4].max()
