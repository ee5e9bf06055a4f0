"""Rotary positions and layer norm against their definitions in float64.

Tolerances, relative in the 2-norm: one rounding to the output's type (block_util.TOL); rotary in float32 adds sines
and cosines of 2^-23 or so and an angle of 2^-25 half turns."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.sequence_oracle as O  # noqa: E402
import structured_state_space_gb300 as s4  # noqa: E402
from block_util import DTYPES, Inputs, close, need_gpu, to64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


# batch, L, H, G, D, rot
SIZES = [(1, 1, 1, 1, 2, 2), (2, 37, 4, 2, 64, 64), (3, 5, 16, 4, 128, 64), (1, 130, 3, 3, 80, 48), (2, 9, 2, 1, 256, 256),
         (1, 7, 5, 5, 33, 30), (1, 3, 1, 1, 256, 2), (64, 1, 16, 4, 128, 64), (2, 300, 32, 8, 64, 32)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("pairs", [False, True])
def test_rotary(size, dt, pairs):
    batch, L, H, G, D, rot = size
    r, dtype = Inputs(1), DTYPES[dt]
    q, k = r.normal(batch, L, H, D, dtype=dtype), r.normal(batch, L, G, D, dtype=dtype)
    freqs, _ = s4.s4_rotary_freqs(rot, device="cuda")
    pos = torch.from_numpy(r.rng.integers(-2 ** 31, 2 ** 31, (batch, L)).astype(np.int32)).cuda()
    pos[0, 0] = 2 ** 31 - 1
    p64 = pos.cpu().numpy()
    # float64 forms angles of 2^31 radians to 2^-22: compare the definition with the exact reduction
    turns = [[int(p) * int(round(float(f) / (2 * np.pi) * 2 ** 64)) % 2 ** 64 / 2 ** 64 for f in freqs.cpu()] for p in p64.ravel()]
    c = np.exp(2j * np.pi * np.array(turns)).reshape(batch, L, 1, rot // 2)
    for sign, f in ((1, s4.s4_rotary_fwd), (-1, s4.s4_rotary_bwd)):
        got = f(q, k, freqs, positions=pos, pairs=pairs, amplitude=1.25)
        for g, x in zip(got, (q, k)):
            want = to64(x)
            a, b = (want[..., 0:rot:2], want[..., 1:rot:2]) if pairs else (want[..., :rot // 2], want[..., rot // 2:rot])
            z = 1.25 * (a + 1j * b) * (c if sign > 0 else c.conj())
            if pairs:
                want[..., 0:rot:2], want[..., 1:rot:2] = z.real, z.imag
            else:
                want[..., :rot // 2], want[..., rot // 2:rot] = z.real.copy(), z.imag.copy()
            # (the fractions above come from a double: 2^-53 of a turn per position, 2^-22 at the farthest)
            close(g, want, f.__name__, {torch.float32: 2e-6, torch.bfloat16: 2.0 ** -8 + 2e-6, torch.float16: 2.0 ** -11 + 2e-6}[dtype])
            assert torch.equal(g[..., rot:], x[..., rot:])
    # in place, and alone
    q2, k2 = q.clone(), k.clone()
    s4.s4_rotary_fwd(q2, k2, freqs, positions=pos, pairs=pairs, q_out=q2, k_out=k2)
    one, none = s4.s4_rotary_fwd(q, None, freqs, positions=pos, pairs=pairs)
    assert none is None and torch.equal(one, q2)
    assert torch.equal(k2, s4.s4_rotary_fwd(k, None, freqs, positions=pos, pairs=pairs)[0])
    if L == 1:
        q3, k3 = s4.s4_rotary_fwd(q[:, 0], k[:, 0], freqs, positions=pos[:, 0], pairs=pairs)
        assert torch.equal(q3, q2[:, 0]) and torch.equal(k3, k2[:, 0])


@pytest.mark.parametrize("dt", DTYPES)
def test_rotary_of_slices_and_plain_positions(dt):
    r = Inputs(2)
    for left in (0, 1):
        qkv = r.normal(2, 40, left + 5 * 32, dtype=DTYPES[dt])[..., left:]
        q, k = qkv[..., :64].unflatten(-1, (2, 32)), qkv[..., 64:96].unflatten(-1, (1, 32))
        freqs, _ = s4.s4_rotary_freqs(32, device="cuda")
        got = s4.s4_rotary_fwd(q, k, freqs)
        pos = np.broadcast_to(np.arange(40), (2, 40))
        for g, x in zip(got, (q, k)):
            close(g, O.rotary(to64(x), to64(freqs), pos, False), "by place")
        p1 = torch.arange(40, dtype=torch.int32, device="cuda")
        for other in (s4.s4_rotary_fwd(q, k, freqs, positions=p1),
                      s4.s4_rotary_fwd(q, k, freqs, positions=p1.expand(2, 40).contiguous()),
                      s4.s4_rotary_fwd(q.contiguous(), k.contiguous(), freqs)):
            assert all(torch.equal(x, y) for x, y in zip(got, other))


def test_rotary_turned_back_is_the_input():
    r = Inputs(3)
    q = r.normal(2, 50, 4, 64)
    freqs, a = s4.s4_rotary_freqs(64, scaling="parts", factor=8.0, length=1024, device="cuda")
    y, _ = s4.s4_rotary_fwd(q, None, freqs, amplitude=a)
    x, _ = s4.s4_rotary_bwd(y, None, freqs, amplitude=1 / a)
    close(x, to64(q), "x", 1e-6)


# ---- layer norm -----------------------------------------------------------------------------------------
ROWS = [(1, 1), (3, 2), (1, 16384), (5, 33), (700, 64), (37, 128), (1001, 40), (64, 256), (130, 512), (33, 1000), (17, 2048),
        (9, 2561), (300, 5120), (7, 8200), (2000, 8)]


@pytest.mark.parametrize("rows,H", ROWS)
@pytest.mark.parametrize("dt", DTYPES)
def test_layer_norm(rows, H, dt):
    r, dtype = Inputs(4), DTYPES[dt]
    x, dy = r.normal(rows, H, dtype=dtype, shift=3.0), r.normal(rows, H, dtype=dtype)
    w, b = r.normal(H, shift=1.0), r.normal(H)
    # eps of the size of the variance: rows of one and two channels have a gradient too
    for ww, bb in ((w, b), (None, None), (w, None), (None, b)):
        y = s4.s4_layer_norm_fwd(x, ww, bb, eps=0.5)
        close(y, O.layer_norm(to64(x), to64(ww), to64(bb), 0.5), "y")
        got = s4.s4_layer_norm_bwd(x, dy, ww, bb, eps=0.5)
        ref = O.layer_norm_grad(to64(x), to64(dy), to64(ww), 0.5)
        assert set(got) == {"dx"} | ({"dw"} if ww is not None else set()) | ({"db"} if bb is not None else set())
        if H == 1:
            # 0 but for one rounding: mean d is the product dy w rounded (off by 2^-24 of it at most), from which the
            # unrounded product is taken in one operation; r is 1 / sqrt(0.5); one more 2^-8 of that in 16 bits
            most = to64(dy) * (1.0 if ww is None else to64(ww)) * 2.0 ** -24 * 2 ** 0.5 * (1 + 2.0 ** -8)
            assert (np.abs(to64(got["dx"])) <= np.abs(most)).all() and (ww is None or not got["dw"].any())
            continue
        for n in got:
            close(got[n], ref[n], n)
    same = x.clone()
    s4.s4_layer_norm_fwd(same, w, b, eps=0.5, y=same)
    assert torch.equal(same, s4.s4_layer_norm_fwd(x, w, b, eps=0.5))


@pytest.mark.parametrize("dt", DTYPES)
def test_layer_norm_of_slices(dt):
    r, dtype = Inputs(5), DTYPES[dt]
    for H in (24, 256, 1030):
        x, dy = r.wide(11, H, dtype=dtype), r.wide(11, H, dtype=dtype, left=8, right=8)
        w, b = r.normal(H), r.normal(H)
        assert torch.equal(s4.s4_layer_norm_fwd(x, w, b), s4.s4_layer_norm_fwd(x.contiguous(), w, b))
        got, want = s4.s4_layer_norm_bwd(x, dy, w, b), s4.s4_layer_norm_bwd(x.contiguous(), dy.contiguous(), w, b)
        for n in got:
            assert torch.allclose(got[n].float(), want[n].float(), rtol=2.0 ** -7 if n == "dx" else 1e-5, atol=1e-4), n


def test_layer_norm_keeps_its_digits_far_from_zero():
    r = Inputs(6)
    x = r.normal(50, 512, shift=1000.0)  # (in float32 the inputs themselves have steps of 6e-5)
    close(s4.s4_layer_norm_fwd(x), O.layer_norm(to64(x)), "y", 1e-4)


def test_layer_norm_of_equal_channels():
    x = torch.full((4, 96), 7.5, device="cuda", dtype=torch.bfloat16)
    b = torch.arange(96.0, device="cuda")
    assert torch.equal(s4.s4_layer_norm_fwd(x, None, b), b.bfloat16().expand(4, 96))
    got = s4.s4_layer_norm_bwd(x, x, b, b)
    assert torch.isfinite(got["dx"]).all() and not got["dw"].any()


def test_rows_that_are_infinite_stay_alone():
    x = torch.randn(70, 64, device="cuda")
    ok = s4.s4_layer_norm_fwd(x)
    x[3, 5], x[33] = float("inf"), float("nan")
    y = s4.s4_layer_norm_fwd(x)
    keep = [i for i in range(70) if i not in (3, 33)]
    assert torch.equal(y[keep], ok[keep]) and torch.isnan(y[3]).any() and torch.isnan(y[33]).all()
