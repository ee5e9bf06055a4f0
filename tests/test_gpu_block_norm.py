"""The norms around a block, with gate, residual scale and sum, on the GPU against their float64
definition: types, sizes in every row layout, absent parts, strides, gradients."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.block_oracle as O  # noqa: E402
import structured_state_space_gb300 as s4  # noqa: E402
from block_util import DTYPES, TOL, Inputs, close, need_gpu, to64  # noqa: E402

pytestmark = pytest.mark.gpu
ALL = ("gate", "h", "w_post", "scale", "w_pre")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def inputs(seed, rows, H, dt, res, parts=ALL, wide=False):
    r = Inputs(seed)
    act = (lambda t: r.wide(rows, H, dtype=t, left=5, right=6)) if wide else (lambda t: r.normal(rows, H, dtype=t))
    a = {"o": act(dt), "gate": act(dt), "h": act(res), "w_post": r.normal(H, scale=0.2, shift=1),
         "scale": r.normal(H, scale=0.3, shift=0.5), "w_pre": r.normal(H, scale=0.2, shift=1)}
    a = {k: v for k, v in a.items() if k == "o" or k in parts}
    d = {"dy": act(dt), "dh_out": act(res)}
    return a, d


def check(a, d, eps=1e-5):
    a64 = {k: to64(v) for k, v in a.items()}
    h_out, y = s4.s4_block_norm_fwd(**a, eps=eps, h_out=torch.empty_like(d["dh_out"], memory_format=torch.contiguous_format))
    rh, ry = O.block_norm(**a64, eps=eps)
    close(h_out, rh, "h_out")
    assert (y is None) == ("w_pre" not in a)
    if y is not None:
        close(y, ry, "y")
    dy = d["dy"] if "w_pre" in a else None
    g = s4.s4_block_norm_bwd(**a, dy=dy, dh_out=d["dh_out"], eps=eps)
    ref = O.block_norm_grad(**a64, dy=to64(dy), dh_out=to64(d["dh_out"]), eps=eps)
    assert set(g) == {"d" + k for k in a}
    for k in g:
        close(g[k], ref[k], k)


# rows of one warp (one and two packs a lane), of one CTA (1, 2, 4 and 8 packs a thread)
@pytest.mark.parametrize("dtype,rows,H", [
    ("f32", 1, 1), ("f32", 3, 5), ("bf16", 5, 64), ("f16", 7, 100), ("bf16", 9, 256), ("f32", 4, 130), ("bf16", 6, 500),
    ("f16", 3, 777), ("bf16", 10, 1024), ("f32", 5, 2048), ("bf16", 3, 4096), ("f32", 3, 4000), ("f16", 2, 8192),
    ("bf16", 2, 16384), ("f32", 2, 16383), ("bf16", 700, 2560), ("f32", 1300, 96)])
def test_forward_and_gradients(dtype, rows, H):
    dt = DTYPES[dtype]
    for res in {dt, torch.float32}:
        check(*inputs(rows + H, rows, H, dt, res))


@pytest.mark.parametrize("parts", [(), ("w_post",), ("w_pre",), ("gate", "w_post"), ("h", "w_pre"), ("h", "scale"),
                                   ("gate", "h", "scale"), ("h", "w_post", "w_pre")])
@pytest.mark.parametrize("H", [96, 1000])
def test_absent_parts(parts, H):
    check(*inputs(H, 6, H, torch.bfloat16, torch.bfloat16, parts))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H", [64, 1024])
def test_strided_rows(dtype, H):
    dt = DTYPES[dtype]
    check(*inputs(H, 11, H, dt, torch.float32, wide=True))


def test_in_place_and_leading_dimensions():
    a, _ = inputs(3, 24, 320, torch.bfloat16, torch.float32)
    want_h, want_y = s4.s4_block_norm_fwd(**a)
    b = {k: v.view(2, 12, 320) if v.dim() == 2 else v for k, v in a.items()}
    h2, y2 = s4.s4_block_norm_fwd(**b)
    assert torch.equal(h2.view(24, 320), want_h) and torch.equal(y2.view(24, 320), want_y)
    h, y = s4.s4_block_norm_fwd(**a, h_out=a["h"])
    assert h is a["h"] and torch.equal(h, want_h) and torch.equal(y, want_y)


def test_rows_of_zeros_and_extremes():
    # a row of zeros has unit 0 (the eps keeps it finite); gates at the ends of the type's range
    a, d = inputs(4, 4, 128, torch.bfloat16, torch.float32)
    a["o"][0], a["h"][0] = 0, 0
    a["gate"][1], a["gate"][2] = -3e38, 80.0
    h, y = s4.s4_block_norm_fwd(**a)
    assert torch.isfinite(h).all() and torch.isfinite(y).all() and (y[0] == 0).all()
    g = s4.s4_block_norm_bwd(**a, dy=d["dy"])
    assert all(torch.isfinite(v).all() for v in g.values())
    ref = O.block_norm(**{k: to64(v) for k, v in a.items()})
    close(h, ref[0], "h")


@pytest.mark.parametrize("which", ["dy", "dh_out"])
def test_one_incoming_gradient(which):
    a, d = inputs(5, 33, 192, torch.float32, torch.float32)
    g = s4.s4_block_norm_bwd(**a, **{which: d[which]})
    ref = O.block_norm_grad(**{k: to64(v) for k, v in a.items()}, **{which: to64(d[which])})
    for k in g:
        close(g[k], ref.get(k, np.zeros(a[k[1:]].shape)), k)


def test_gradient_against_differences_of_the_forward_definition():
    # float64 central differences (error ~1e-9) along random directions; float32 gradients are off by ~1e-6
    a, d = inputs(6, 8, 160, torch.float32, torch.float32)
    g = s4.s4_block_norm_bwd(**a, **d)
    rng = np.random.default_rng(7)
    for k in a:
        v = rng.standard_normal(a[k].shape)
        val = []
        for sign in (1, -1):
            p = {n: to64(t) for n, t in a.items()}
            p[k] = p[k] + sign * 1e-5 * v
            h, y = O.block_norm(**p)
            val.append((h * to64(d["dh_out"])).sum() + (y * to64(d["dy"])).sum())
        num = (val[0] - val[1]) / 2e-5
        gk = to64(g["d" + k])
        assert abs(num - (gk * v).sum()) <= 1e-5 * np.linalg.norm(gk) * np.linalg.norm(v), k


def test_other_stream_and_determinism():
    a, d = inputs(8, 500, 1024, torch.bfloat16, torch.float32)
    h, y = s4.s4_block_norm_fwd(**a)
    g = s4.s4_block_norm_bwd(**a, **d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h2, y2 = s4.s4_block_norm_fwd(**a, stream=side)
    g2 = s4.s4_block_norm_bwd(**a, **d, stream=side)
    side.synchronize()
    assert torch.equal(h, h2) and torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in g)


def test_refusals():
    a, d = inputs(9, 4, 64, torch.bfloat16, torch.float32)
    with pytest.raises(TypeError):
        s4.s4_block_norm_fwd(a["o"].double())
    with pytest.raises(TypeError):
        s4.s4_block_norm_fwd(a["o"], gate=a["gate"].float())
    with pytest.raises(TypeError):
        s4.s4_block_norm_fwd(a["o"], h=a["h"].half())
    with pytest.raises(ValueError):
        s4.s4_block_norm_fwd(a["o"], w_post=a["w_post"][:32])
    with pytest.raises(ValueError):
        s4.s4_block_norm_fwd(a["o"].t().contiguous().t())
    with pytest.raises(s4.S4Error):
        s4.s4_block_norm_fwd(torch.zeros(2, 16385, device="cuda"))
    with pytest.raises(s4.S4Error):
        s4.s4_block_norm_fwd(a["o"], eps=-1.0)
    with pytest.raises(s4.S4Error):
        s4.s4_block_norm_bwd(a["o"])  # no incoming gradient
    with pytest.raises(s4.S4Error):
        s4.s4_block_norm_bwd(a["o"], d["dy"])  # dy without w_pre
    assert TOL[torch.bfloat16] < 0.01
