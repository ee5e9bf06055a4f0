"""The selective scan on the GPU against its float64 definition: types, numbers of states, groups,
odd and strided sizes, chunked long sequences, ragged and empty sequences, states in slots
and in place, single tokens."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.block_oracle as O  # noqa: E402
import structured_state_space_gb300 as s4  # noqa: E402
from block_util import DTYPES, Inputs, close, need_gpu, to64  # noqa: E402

pytestmark = pytest.mark.gpu

# The state's tolerance, relative in the 2-norm: each step's factor 2^(d A) is off by 2^-22 and its
# exponent's rounding, |d A| 2^-23, and a state remembers 1 / (1 - factor) of them: at most 10^3 steps
# at d A = 1e-3, where errors of either sign add to about 30 and of one sign to 10^3 times 2^-22.
# Inputs here have d A >= 5e-3 for most states: 2e-5.
STATE_TOL = 2e-5


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def lens(t):
    return torch.tensor(t, dtype=torch.int32, device="cuda")


def scan_inputs(seed, batch, L, H, N, G, dt, wide=False):
    r = Inputs(seed)
    act = (lambda: r.wide(batch, L, H, dtype=dt, left=8, right=3)) if wide else (lambda: r.normal(batch, L, H, dtype=dt))
    a = {"x": act(), "dt": act(), "z": act()}
    bc = r.normal(batch, L, 5 + 2 * G * N, dtype=dt)[..., 5:] if wide else r.normal(batch, L, 2 * G * N, dtype=dt)
    a["B"], a["C"] = bc[..., :G * N].unflatten(-1, (G, N)), bc[..., G * N:].unflatten(-1, (G, N))
    a["A"] = -torch.exp(r.normal(H, N, scale=0.5))
    a["D"], a["dt_bias"] = r.normal(H), r.normal(H, shift=-3.0)
    return a, r


def split(a):
    return [a[k] for k in ("x", "dt", "A", "B", "C")], {k: a[k] for k in ("D", "z", "dt_bias") if k in a}


def reference(a, **kw):
    pos, named = split({k: to64(v) for k, v in a.items()})
    return O.selective_scan(*pos, **named, **kw)


SIZES = [(1, 1, 1, 1, 1), (1, 2, 3, 16, 1), (2, 33, 40, 16, 1), (2, 40, 70, 16, 2), (3, 31, 9, 5, 3), (1, 64, 130, 4, 1),
         (2, 17, 20, 8, 4), (1, 50, 24, 30, 1), (2, 35, 12, 64, 2), (1, 20, 10, 128, 1), (1, 37, 6, 256, 2), (1, 9, 5, 200, 1),
         (1, 700, 64, 16, 1)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("batch,L,H,N,G", SIZES)
def test_forward(dtype, batch, L, H, N, G):
    a, r = scan_inputs(L * N + H, batch, L, H, N, G, DTYPES[dtype])
    state = r.normal(batch, H, N)
    out = torch.empty_like(state)
    pos, named = split(a)
    y = s4.s4_selective_scan_fwd(*pos, **named, state=state, state_out=out)
    ry, rs = reference(a, state=to64(state))
    close(y, ry, "y", None if dtype != "f32" else STATE_TOL)
    close(out, rs, "state", STATE_TOL)


@pytest.mark.parametrize("parts", [(), ("D",), ("z",), ("dt_bias",)])
def test_absent_parts(parts):
    a, _ = scan_inputs(7, 2, 45, 36, 16, 1, torch.float32)
    for k in ("D", "z", "dt_bias"):
        if k not in parts:
            del a[k]
    a["dt"] = a["dt"].abs() * 0.1  # steps as they are: positive ones
    if "dt_bias" in a:
        a["dt_bias"] = a["dt_bias"].abs() * 0.1
    pos, named = split(a)
    close(s4.s4_selective_scan_fwd(*pos, **named, softplus=False), reference(a, soft=False)[0], "y", STATE_TOL)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("L,H,N,G", [(75, 48, 16, 1), (75, 36, 16, 2), (40, 20, 64, 2), (1500, 32, 16, 1)])
def test_ragged_slots_in_place_and_strides(dtype, L, H, N, G):
    n = [L, 0, 1, L // 2, 20, L - 1]
    batch = len(n)
    a, r = scan_inputs(L + H + N, batch, L, H, N, G, DTYPES[dtype], wide=True)
    clean = {k: v.clone() for k, v in a.items()}
    for b in range(batch):  # padding holds what may not be used
        for k in ("x", "dt", "z", "B", "C"):
            clean[k][b, n[b]:] = 0
            a[k][b, n[b]:] = float("nan") if b % 2 else float("inf")
    cache = r.normal(9, H, N)
    index = [4, 8, 0, 2, -1, 7]
    want = to64(cache)
    need = int(s4.load().s4_selective_scan_workspace_bytes(batch, L, H, N, G))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    pos, named = split(a)
    y = s4.s4_selective_scan_fwd(*pos, **named, lengths=lens(n), state=cache, state_out=cache, index=lens(index), ws=ws)
    assert s4.s4_get_status(ws) == 0
    ry, rs = reference(clean, lengths=n, state=want[np.maximum(index, 0)])
    ry[4] = 0
    close(y, ry, "y", None if dtype != "f32" else STATE_TOL)
    for b in range(batch):
        assert (to64(y)[b, n[b]:] == 0).all()
        if index[b] >= 0:
            want[index[b]] = rs[b]
    close(cache, want, "cache", STATE_TOL)
    untouched = [i for i in range(9) if i not in index]
    assert np.array_equal(to64(cache)[untouched], want[untouched])
    assert np.array_equal(to64(cache)[8], want[8])  # of length 0: as it was


def test_long_sequences_in_chunks_equal_short_ones():
    # one sequence of few channels is split into chunks; the same tokens in short calls are not
    L, H = 4000, 32
    a, _ = scan_inputs(3, 1, L, H, 16, 1, torch.float32)
    pos, named = split(a)
    assert s4.load().s4_selective_scan_workspace_bytes(1, L, H, 16, 1) > 256
    state = torch.zeros(1, H, 16, device="cuda")
    y = s4.s4_selective_scan_fwd(*pos, **named, state_out=state)
    s2, ys = torch.zeros_like(state), []
    for t in range(0, L, 200):
        part = {k: v[:, t:t + 200] if v.dim() > 2 else v for k, v in a.items()}
        pos, named = split(part)
        ys.append(s4.s4_selective_scan_fwd(*pos, **named, state=s2, state_out=s2))
    close(y, to64(torch.cat(ys, 1)), "y", 2 * STATE_TOL)
    close(state, to64(s2), "state", 2 * STATE_TOL)
    ry, rs = reference(a)
    close(y, ry, "y", STATE_TOL)
    close(state, rs, "state", STATE_TOL)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("batch,H,N,G", [(1, 1, 1, 1), (3, 70, 16, 1), (5, 24, 16, 2), (2, 9, 5, 3), (2, 20, 64, 1),
                                         (2, 6, 200, 2), (9, 33, 128, 1)])
def test_single_tokens(dtype, batch, H, N, G):
    dt = DTYPES[dtype]
    a, r = scan_inputs(batch + H + N, batch, 2, H, N, G, dt, wide=True)
    cache = r.normal(batch + 3, H, N)
    index = np.random.default_rng(1).permutation(batch + 3)[:batch]
    if batch > 2:
        index[1] = -1
    old = to64(cache)
    one = {k: v[:, :1] if v.dim() > 2 else v for k, v in a.items()}
    ry, rs = reference(one, state=old[np.maximum(index, 0)])
    tok = {k: v[:, 0] if v.dim() > 2 else v for k, v in a.items()}
    pos, named = split(tok)
    out = cache.clone()
    y = s4.s4_selective_step(*pos, cache, **named, state_out=out, index=lens(index.tolist()))
    assert np.array_equal(to64(cache), old)
    want = old.copy()
    for b in range(batch):
        if index[b] < 0:
            ry[b] = 0
        else:
            want[index[b]] = rs[b]
    close(y, ry[:, 0], "y")
    close(out, want, "state")
    y2 = s4.s4_selective_step(*pos, cache, **named, index=lens(index.tolist()))
    assert torch.equal(y, y2) and torch.equal(cache, out)


def test_tokens_one_by_one_follow_the_prompt():
    a, _ = scan_inputs(11, 2, 20, 40, 16, 1, torch.float32)
    pos, named = split(a)
    s1 = torch.zeros(2, 40, 16, device="cuda")
    y = s4.s4_selective_scan_fwd(*pos, **named, state=s1, state_out=s1)
    s2, ys = torch.zeros_like(s1), []
    for t in range(20):
        pos, named = split({k: v[:, t] if v.dim() > 2 else v for k, v in a.items()})
        ys.append(s4.s4_selective_step(*pos, s2, **named))
    close(torch.stack(ys, 1), to64(y), "y", 1e-5)
    close(s2, to64(s1), "state", 1e-5)


def test_extreme_steps_and_decays():
    # steps of 0 (the softplus of -inf and of very negative values) keep the state; very large ones
    # forget it; A = 0 sums; all without NaN
    a, r = scan_inputs(12, 1, 6, 8, 16, 1, torch.float32)
    a["dt"][0, 0] = -float("inf")
    a["dt"][0, 1] = -200.0
    a["dt"][0, 2] = 90.0
    a["A"][0] = 0
    state = r.normal(1, 8, 16)
    pos, named = split(a)
    out = torch.empty_like(state)
    y = s4.s4_selective_scan_fwd(*pos, **named, state=state, state_out=out)
    ry, rs = reference(a, state=to64(state))
    close(y, ry, "y", STATE_TOL)
    close(out, rs, "state", STATE_TOL)


def test_bad_lengths_and_slots_are_recorded():
    a, r = scan_inputs(13, 3, 5, 16, 16, 1, torch.float32)
    pos, named = split(a)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    cache = r.normal(3, 16, 16)
    kept = cache.clone()
    for n, index in (([5, 6, -1], [0, 1, 2]), ([5, 5, 5], [0, 3, 1 << 30])):
        y = s4.s4_selective_scan_fwd(*pos, **named, lengths=lens(n), state=cache, state_out=cache, index=lens(index), ws=ws)
        assert s4.STATUS[s4.s4_get_status(ws)] == "S4_ERR_INVALID_INDEX"
        assert (y[1:] == 0).all() and (y[0] != 0).any() and torch.equal(cache[1:], kept[1:])
    s4.s4_selective_scan_fwd(*pos, **named, ws=ws)
    assert s4.s4_get_status(ws) == 0


def test_other_stream_graph_and_determinism():
    a, _ = scan_inputs(14, 2, 1200, 64, 16, 1, torch.bfloat16)
    pos, named = split(a)
    y = s4.s4_selective_scan_fwd(*pos, **named)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = s4.s4_selective_scan_fwd(*pos, **named, stream=side)
    side.synchronize()
    assert torch.equal(y, y2)
    ws = torch.empty(int(s4.load().s4_selective_scan_workspace_bytes(2, 1200, 64, 16, 1)), dtype=torch.uint8, device="cuda")
    y3, graph = torch.empty_like(y), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s4.s4_selective_scan_fwd(*pos, **named, y=y3, ws=ws)
    a["x"].neg_()
    graph.replay()
    assert torch.equal(y3, s4.s4_selective_scan_fwd(*pos, **named)) and s4.s4_get_status(ws) == 0


# Gradients: as the state, and dA, ddt sum products of two of them over up to 10^3 remembered steps; the
# sums over channels and tokens have up to 10^4 terms of either sign: 4e-5.
GRAD_TOL = 4e-5


def check_gradients(a, dy, tol=GRAD_TOL, **kw):
    pos, named = split(a)
    t = {k: (lens(v) if k == "lengths" else v) for k, v in kw.items()}
    g = s4.s4_selective_scan_bwd(*pos, dy, **named, **t)
    pos, named = split({k: to64(v) for k, v in a.items()})
    r = {k: (to64(v) if torch.is_tensor(v) else v) for k, v in kw.items() if k != "want_dstate0"}
    ref = O.selective_scan_grad(*pos, to64(dy), **named, **r)
    for k in g:
        close(g[k], ref[k], k, tol if g[k].dtype == torch.float32 else None)
    return g


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("batch,L,H,N,G", SIZES)
def test_gradients(dtype, batch, L, H, N, G):
    dt = DTYPES[dtype]
    a, r = scan_inputs(L * N + H + 1, batch, L, H, N, G, dt)
    dy = r.normal(batch, L, H, dtype=dt)
    g = check_gradients(a, dy, state=r.normal(batch, H, N), dstate=r.normal(batch, H, N), want_dstate0=True)
    assert set(g) == {"dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate0"}


@pytest.mark.parametrize("parts", [(), ("D",), ("z",), ("dt_bias",)])
@pytest.mark.parametrize("soft", [True, False])
def test_gradients_with_absent_parts(parts, soft):
    a, r = scan_inputs(8, 2, 45, 36, 16, 1, torch.float32)
    for k in ("D", "z", "dt_bias"):
        if k not in parts:
            del a[k]
    a["dt"] = a["dt"].abs() * 0.1
    if "dt_bias" in a:
        a["dt_bias"] = a["dt_bias"].abs() * 0.1
    pos, named = split(a)
    dy = r.normal(2, 45, 36)
    g = s4.s4_selective_scan_bwd(*pos, dy, **named, softplus=soft)
    pos, named = split({k: to64(v) for k, v in a.items()})
    ref = O.selective_scan_grad(*pos, to64(dy), **named, soft=soft)
    for k in g:
        close(g[k], ref[k], k, GRAD_TOL)
    assert set(g) == {"dx", "ddt", "dA", "dB", "dC"} | {{"z": "dz", "D": "dD", "dt_bias": "ddt_bias"}[k] for k in parts}


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("L,H,N,G", [(75, 48, 16, 1), (75, 36, 16, 2), (40, 20, 64, 2), (500, 32, 16, 1)])
def test_ragged_gradients_and_strides(dtype, L, H, N, G):
    n = [L, 0, 1, L // 2, 20, L - 1]
    a, r = scan_inputs(L + H + N + 1, 6, L, H, N, G, DTYPES[dtype], wide=True)
    dy = r.wide(6, L, H, dtype=DTYPES[dtype], left=8, right=0)
    for b in range(6):
        for k in ("x", "dt", "z", "B", "C"):
            a[k][b, n[b]:] = 0
        dy[b, n[b]:] = 0
    kw = dict(lengths=n, state=r.normal(6, H, N), dstate=r.normal(6, H, N), want_dstate0=True)
    g = check_gradients(a, dy, **kw)
    for b in range(6):  # padding holds what may not be used
        for k in ("x", "dt", "z", "B", "C"):
            a[k][b, n[b]:] = float("nan") if b % 2 else float("inf")
        dy[b, n[b]:] = float("nan")
    pos, named = split(a)
    again = s4.s4_selective_scan_bwd(*pos, dy, **named, **{**kw, "lengths": lens(n)})
    for k in g:
        assert torch.equal(g[k], again[k]), k
        if k in ("dx", "ddt", "dz", "dB", "dC"):
            assert all((again[k][b, n[b]:] == 0).all() for b in range(6)), k


def test_gradients_over_segments():
    # few channels and many tokens: the first kernel runs in several segments, joined by the second
    a, r = scan_inputs(21, 1, 3001, 24, 16, 1, torch.float32)
    check_gradients(a, r.normal(1, 3001, 24), state=r.normal(1, 24, 16), dstate=r.normal(1, 24, 16), want_dstate0=True)


def test_gradient_against_differences_of_the_forward_definition():
    # float64 central differences along random directions (error ~1e-9); float32 gradients are off by ~1e-5 at most
    a, r = scan_inputs(22, 2, 30, 12, 16, 2, torch.float32)
    dy = r.normal(2, 30, 12)
    pos, named = split(a)
    g = s4.s4_selective_scan_bwd(*pos, dy, **named)
    for k in a:
        v = r.rng.standard_normal(a[k].shape)
        val = []
        for sign in (1, -1):
            p = {n: to64(t) for n, t in a.items()}
            p[k] = p[k] + sign * 1e-5 * v
            pos, named = split(p)
            val.append((O.selective_scan(*pos, **named)[0] * to64(dy)).sum())
        gk = to64(g["d" + k])
        assert abs((val[0] - val[1]) / 2e-5 - (gk * v).sum()) <= 1e-4 * np.linalg.norm(gk) * np.linalg.norm(v), k


def test_gradients_on_another_stream_and_deterministic():
    a, r = scan_inputs(23, 2, 300, 96, 16, 1, torch.bfloat16)
    dy = r.normal(2, 300, 96, dtype=torch.bfloat16)
    pos, named = split(a)
    g = s4.s4_selective_scan_bwd(*pos, dy, **named)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g2 = s4.s4_selective_scan_bwd(*pos, dy, **named, stream=side)
    side.synchronize()
    assert all(torch.equal(g[k], g2[k]) for k in g)
    with pytest.raises(s4.S4Error):
        s4.s4_selective_scan_bwd(*pos, dy, **named, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_refusals():
    a, r = scan_inputs(15, 2, 8, 16, 16, 2, torch.float32)
    pos, named = split(a)
    x, dt, A, B, C = pos
    with pytest.raises(TypeError):
        s4.s4_selective_scan_fwd(x, dt.half(), A, B, C)
    with pytest.raises(ValueError):
        s4.s4_selective_scan_fwd(x, dt[:, :4], A, B, C)
    with pytest.raises(ValueError):
        s4.s4_selective_scan_fwd(x, dt, A[:, :8], B, C)
    with pytest.raises(ValueError):
        s4.s4_selective_scan_fwd(x.transpose(1, 2).contiguous().transpose(1, 2), dt, A, B, C)
    with pytest.raises(ValueError):
        s4.s4_selective_scan_fwd(*pos, state=r.normal(1, 16, 16))
    with pytest.raises(TypeError):
        s4.s4_selective_scan_fwd(*pos, state=r.normal(2, 16, 16, dtype=torch.bfloat16))
    with pytest.raises(s4.S4Error):  # channels do not divide into groups
        s4.s4_selective_scan_fwd(x, dt, A, r.normal(2, 8, 3, 16), r.normal(2, 8, 3, 16))
    with pytest.raises(s4.S4Error):  # more than 256 states
        s4.s4_selective_scan_fwd(x, dt, r.normal(16, 257), r.normal(2, 8, 1, 257), r.normal(2, 8, 1, 257))
    big, named = split(scan_inputs(16, 1, 2000, 32, 16, 1, torch.float32)[0])
    with pytest.raises(s4.S4Error):
        s4.s4_selective_scan_fwd(*big, **named, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
