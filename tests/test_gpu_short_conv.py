"""The short causal convolution on the GPU against its float64 definition: types, widths, odd and
strided sizes, ragged and empty sequences, states in slots and in place, single tokens,
gradients, streams, graphs."""
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
@pytest.mark.parametrize("batch,L,H,W", [(1, 1, 1, 2), (2, 3, 64, 4), (3, 17, 72, 4), (2, 50, 33, 3), (1, 65, 7, 8),
                                         (2, 33, 130, 5), (1, 16, 8, 2), (1, 200, 256, 4)])
def test_forward(dtype, batch, L, H, W):
    dt, r = DTYPES[dtype], Inputs(L + H + W)
    x, w, b = r.normal(batch, L, H, dtype=dt), r.normal(H, W), r.normal(H)
    st = r.normal(batch, W - 1, H, dtype=dt)
    out = torch.empty_like(st)
    y = s4.s4_short_conv_fwd(x, w, b, state=st, state_out=out)
    ry, rs = O.short_conv(to64(x), to64(w), to64(b), state=to64(st))
    close(y, ry, "y")
    assert np.array_equal(to64(out), rs)
    y = s4.s4_short_conv_fwd(x, w, silu=False)
    close(y, O.short_conv(to64(x), to64(w), act=False)[0], "y without bias, state and activation")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,left", [(48, 3), (48, 8), (41, 1)])
def test_ragged_slots_in_place_and_strides(dtype, H, left):
    dt, r, W, L = DTYPES[dtype], Inputs(H + left), 4, 37
    n = [37, 0, 1, 2, 20, 36]
    B = len(n)
    x = r.wide(B, L, H, dtype=dt, left=left, right=8)
    for b in range(B):  # padding holds what may not be used
        x[b, n[b]:] = float("nan") if b % 2 else float("inf")
    w, bias = r.normal(H, W), r.normal(H)
    cache = r.normal(9, W - 1, H, dtype=dt)
    index = [4, 8, 0, 2, -1, 7]
    want = to64(cache)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    y = s4.s4_short_conv_fwd(x, w, bias, lengths=lens(n), state=cache, state_out=cache, index=lens(index), ws=ws)
    assert s4.s4_get_status(ws) == 0
    xs = to64(x)
    for b in range(B):
        xs[b, n[b]:] = 0
    ry, rs = O.short_conv(xs, to64(w), to64(bias), lengths=n, state=want[np.maximum(index, 0)])
    ry[4] = 0  # a row without a slot is not in use
    close(y, ry, "y")
    for b in range(B):
        assert (to64(y)[b, n[b]:] == 0).all()
        if index[b] >= 0:
            want[index[b]] = rs[b]
    assert np.array_equal(to64(cache), want)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_tokens_one_by_one_equal_the_prompt(dtype):
    dt, r, B, L, H, W = DTYPES[dtype], Inputs(5), 3, 11, 40, 4
    x, w, bias = r.normal(B, L, H, dtype=dt), r.normal(H, W), r.normal(H)
    s1 = torch.zeros(B, W - 1, H, dtype=dt, device="cuda")
    y = s4.s4_short_conv_fwd(x, w, bias, state=s1, state_out=s1)
    s2 = torch.zeros(B + 2, W - 1, H, dtype=dt, device="cuda")
    index = lens([3, 0, 4])
    for t in range(L):
        yt = s4.s4_short_conv_step(x[:, t], w, bias, s2, index=index)
        assert torch.equal(yt, y[:, t]), t
    assert torch.equal(s2[index.long()], s1)
    # a token tried without touching the state
    kept = s2.clone()
    other = torch.empty_like(s2)
    s4.s4_short_conv_step(x[:, 0], w, bias, s2, state_out=other, index=index)
    assert torch.equal(s2, kept) and not torch.equal(other[3], kept[3])


def test_bad_lengths_and_slots_are_recorded():
    r, ws = Inputs(6), torch.empty(256, dtype=torch.uint8, device="cuda")
    x, w = r.normal(3, 5, 16), r.normal(16, 4)
    cache = r.normal(3, 3, 16)
    kept = cache.clone()
    for n, index in (([5, 6, -1], [0, 1, 2]), ([5, 5, 5], [0, 3, 1000])):
        y = s4.s4_short_conv_fwd(x, w, lengths=lens(n), state=cache, state_out=cache, index=lens(index), ws=ws)
        assert s4.STATUS[s4.s4_get_status(ws)] == "S4_ERR_INVALID_INDEX"
        assert (y[1:] == 0).all() and (y[0] != 0).any()
        assert torch.equal(cache[1:], kept[1:])
    s4.s4_short_conv_fwd(x, w, ws=ws)
    assert s4.s4_get_status(ws) == 0  # the last call's status only


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("batch,L,H,W,act", [(1, 1, 1, 2, True), (2, 3, 64, 4, True), (3, 70, 36, 4, True),
                                             (2, 65, 33, 3, False), (1, 130, 9, 8, True), (2, 600, 132, 4, True)])
def test_gradients(dtype, batch, L, H, W, act):
    dt, r = DTYPES[dtype], Inputs(L * W + H)
    x, dy = r.wide(batch, L, H, dtype=dt, left=4, right=4), r.normal(batch, L, H, dtype=dt)
    w, b = r.normal(H, W), r.normal(H)
    st, ds = r.normal(batch, W - 1, H, dtype=dt), r.normal(batch, W - 1, H, dtype=dt)
    n = [L] + [max(0, L - 3 * (i + 1)) for i in range(batch - 1)]
    g = s4.s4_short_conv_bwd(x, w, b, dy, silu=act, lengths=lens(n), state=st, dstate=ds, want_dstate0=True)
    ref = O.short_conv_grad(to64(x), to64(w), to64(b), to64(dy), act, n, to64(st), to64(ds))
    assert set(g) == set(ref)
    for k in g:
        close(g[k], ref[k], k)
    g = s4.s4_short_conv_bwd(x, w, None, dy, silu=act)
    ref = O.short_conv_grad(to64(x), to64(w), None, to64(dy), act)
    assert set(g) == {"dx", "dw"}
    for k in g:
        close(g[k], ref[k], k)


def test_gradient_against_differences_of_the_forward_definition():
    # central differences in float64 (step 1e-5: error ~1e-9) along a random direction; the kernel's
    # float32 gradient is off by ~1e-6 of its norm, the product with the direction by as much
    r = Inputs(8)
    a = {"x": r.normal(2, 40, 24), "w": r.normal(24, 4), "bias": r.normal(24)}
    dy = r.normal(2, 40, 24)
    g = s4.s4_short_conv_bwd(a["x"], a["w"], a["bias"], dy)
    for k in a:
        v = r.rng.standard_normal(a[k].shape)
        val = []
        for sign in (1, -1):
            p = {n: to64(t) for n, t in a.items()}
            p[k] = p[k] + sign * 1e-5 * v
            val.append((O.short_conv(p["x"], p["w"], p["bias"])[0] * to64(dy)).sum())
        num = (val[0] - val[1]) / 2e-5
        gk = to64(g["d" + k])
        assert abs(num - (gk * v).sum()) <= 1e-5 * np.linalg.norm(gk) * np.linalg.norm(v), k


def test_padding_does_not_reach_the_gradients():
    r, n = Inputs(9), [20, 0, 7]
    x, dy, w, b = r.normal(3, 20, 16), r.normal(3, 20, 16), r.normal(16, 4), r.normal(16)
    clean = s4.s4_short_conv_bwd(x, w, b, dy, lengths=lens(n))
    for i in range(3):
        x[i, n[i]:], dy[i, n[i]:] = float("nan"), float("inf")
    again = s4.s4_short_conv_bwd(x, w, b, dy, lengths=lens(n))
    for k in clean:
        assert torch.equal(clean[k], again[k]), k
    assert (again["dx"][1] == 0).all() and (again["dx"][2, 7:] == 0).all()


@pytest.mark.parametrize("W", [2, 3, 4, 5, 7])
def test_an_infinity_reaches_only_its_taps(W):
    r = Inputs(W)
    x, w, dy = r.normal(1, 40, 8), r.normal(8, W), r.normal(1, 40, 8)
    x[0, 11] = float("inf")
    y = s4.s4_short_conv_fwd(x, w, silu=False)
    bad = ~torch.isfinite(y[0]).any(1)
    assert torch.nonzero(bad).flatten().tolist() == list(range(11, 11 + W))
    dy[0, 20] = float("inf")
    x[0, 11] = 0
    g = s4.s4_short_conv_bwd(x, w, None, dy, silu=False)
    bad = ~torch.isfinite(g["dx"][0]).any(1)
    assert torch.nonzero(bad).flatten().tolist() == list(range(20 - W + 1, 21))


def test_other_stream_and_graph_and_determinism():
    r = Inputs(10)
    x, w, b, dy = r.normal(2, 300, 64, dtype=torch.bfloat16), r.normal(64, 4), r.normal(64), \
        r.normal(2, 300, 64, dtype=torch.bfloat16)
    y, g = s4.s4_short_conv_fwd(x, w, b), s4.s4_short_conv_bwd(x, w, b, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, g2 = s4.s4_short_conv_fwd(x, w, b, stream=side), s4.s4_short_conv_bwd(x, w, b, dy, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in g)
    graph = torch.cuda.CUDAGraph()
    y3, ws = torch.empty_like(y), torch.empty(256, dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(graph):
        s4.s4_short_conv_fwd(x, w, b, y=y3, ws=ws)
    x.neg_()
    graph.replay()
    assert torch.equal(y3, s4.s4_short_conv_fwd(x, w, b)) and s4.s4_get_status(ws) == 0


def test_refusals():
    r = Inputs(11)
    x, w, b = r.normal(2, 8, 16), r.normal(16, 4), r.normal(16)
    with pytest.raises(TypeError):
        s4.s4_short_conv_fwd(x.double(), w, b)
    with pytest.raises(TypeError):
        s4.s4_short_conv_fwd(x, w.half(), b)
    with pytest.raises(ValueError):
        s4.s4_short_conv_fwd(x, w, b[:8])
    with pytest.raises(ValueError):
        s4.s4_short_conv_fwd(x.transpose(1, 2).contiguous().transpose(1, 2), w, b)  # channels not contiguous
    with pytest.raises(ValueError):
        s4.s4_short_conv_fwd(x, w, b, state=r.normal(1, 3, 16))  # fewer slots than sequences
    with pytest.raises(ValueError):
        s4.s4_short_conv_fwd(x.cpu(), w, b)
    with pytest.raises(s4.S4Error):
        s4.s4_short_conv_fwd(x, r.normal(16, 9), b)
    with pytest.raises(s4.S4Error):
        s4.s4_short_conv_bwd(x, w, b, x, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
