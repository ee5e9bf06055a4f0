"""Pins of oracle/block_oracle.py: every gradient against central differences of the forward
definition, the carried states against one long call, closed forms, and planted mistakes."""
import numpy as np
import pytest

import oracle.block_oracle as O

# A central difference with step 1e-5 of a smooth float64 function of size ~1 is off by its third
# derivative times 1e-10 / 6 and by rounding 1e-16 * (terms ~1e2) / 1e-5 = 1e-9.
STEP, TOL = 1e-5, 2e-8


def _directional(f, args, grads, rng):
    """Difference quotient of f along a random direction in each argument, against the gradient."""
    for k, g in grads.items():
        v = rng.standard_normal(args[k].shape)
        up, dn = dict(args), dict(args)
        up[k], dn[k] = args[k] + STEP * v, args[k] - STEP * v
        num = (f(up) - f(dn)) / (2 * STEP)
        assert abs(num - (g * v).sum()) <= TOL * max(1.0, np.linalg.norm(g) * np.linalg.norm(v)), k


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("lengths", [None, [5, 0, 2]])
def test_short_conv_gradient(act, lengths):
    rng = np.random.default_rng(1)
    a = {"x": rng.standard_normal((3, 5, 4)), "w": rng.standard_normal((4, 3)), "bias": rng.standard_normal(4),
         "state": rng.standard_normal((3, 2, 4))}
    dy, ds = rng.standard_normal((3, 5, 4)), rng.standard_normal((3, 2, 4))

    def f(a):
        y, s = O.short_conv(a["x"], a["w"], a["bias"], act, lengths, a["state"])
        return (y * dy).sum() + (s * ds).sum()
    g = O.short_conv_grad(a["x"], a["w"], a["bias"], dy, act, lengths, a["state"], ds)
    _directional(f, a, {"x": g["dx"], "w": g["dw"], "bias": g["dbias"], "state": g["dstate0"]}, rng)


@pytest.mark.parametrize("lengths", [None, [6, 0, 3]])
@pytest.mark.parametrize("gated", [True, False])
def test_selective_scan_gradient(lengths, gated):
    rng = np.random.default_rng(2)
    nb, L, H, N, G = 3, 6, 4, 3, 2
    a = {"x": rng.standard_normal((nb, L, H)), "dt": rng.standard_normal((nb, L, H)),
         "A": -np.exp(rng.standard_normal((H, N))), "B": rng.standard_normal((nb, L, G, N)),
         "C": rng.standard_normal((nb, L, G, N)), "D": rng.standard_normal(H), "dt_bias": rng.standard_normal(H),
         "state": rng.standard_normal((nb, H, N))}
    if gated:
        a["z"] = rng.standard_normal((nb, L, H))
    dy, ds = rng.standard_normal((nb, L, H)), rng.standard_normal((nb, H, N))

    def f(a):
        y, s = O.selective_scan(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a.get("z"), a["dt_bias"], True,
                                lengths, a["state"])
        return (y * dy).sum() + (s * ds).sum()
    g = O.selective_scan_grad(a["x"], a["dt"], a["A"], a["B"], a["C"], dy, a["D"], a.get("z"), a["dt_bias"], True,
                              lengths, a["state"], ds)
    names = {k: g["d" + k] for k in a if k != "state"}
    _directional(f, a, {**names, "state": g["dstate0"]}, rng)


@pytest.mark.parametrize("absent", [(), ("gate",), ("w_post",), ("scale",), ("h",), ("gate", "w_post", "scale", "h")])
def test_block_norm_gradient(absent):
    rng = np.random.default_rng(3)
    a = {k: rng.standard_normal((3, 7)) for k in ("o", "gate", "h")}
    a |= {k: 1 + 0.2 * rng.standard_normal(7) for k in ("w_post", "scale", "w_pre")}
    for k in absent:
        del a[k]
    dy, dh = rng.standard_normal((3, 7)), rng.standard_normal((3, 7))

    def f(a):
        h2, y = O.block_norm(**a)
        return (y * dy).sum() + (h2 * dh).sum()
    g = O.block_norm_grad(dy=dy, dh_out=dh, **a)
    _directional(f, a, {k: g["d" + k] for k in a}, rng)


def test_states_carry():
    rng = np.random.default_rng(4)
    x, w = rng.standard_normal((2, 9, 3)), rng.standard_normal((3, 4))
    y, s = O.short_conv(x, w)
    y1, s1 = O.short_conv(x[:, :2], w)
    y2, s2 = O.short_conv(x[:, 2:], w, state=s1)
    assert np.allclose(np.concatenate([y1, y2], 1), y, atol=1e-14) and np.array_equal(s2, s)
    dt, A = rng.standard_normal((2, 9, 3)), -np.exp(rng.standard_normal((3, 5)))
    B, C = rng.standard_normal((2, 2, 9, 1, 5))
    y, s = O.selective_scan(x, dt, A, B, C)
    y1, s1 = O.selective_scan(x[:, :4], dt[:, :4], A, B[:, :4], C[:, :4])
    y2, s2 = O.selective_scan(x[:, 4:], dt[:, 4:], A, B[:, 4:], C[:, 4:], state=s1)
    assert np.allclose(np.concatenate([y1, y2], 1), y, atol=1e-14) and np.allclose(s2, s, atol=1e-14)


def test_closed_forms():
    # A = 0, B = C = 1, unit steps: the scan is a running sum
    x = np.arange(1.0, 6.0).reshape(1, 5, 1)
    one = np.ones((1, 5, 1, 1))
    y, s = O.selective_scan(x, np.ones((1, 5, 1)), np.zeros((1, 1)), one, one, soft=False)
    assert np.allclose(y[0, :, 0], np.cumsum(x[0, :, 0])) and s[0, 0, 0] == 15
    # a filter that only has its last tap passes x through
    w = np.array([[0.0, 0.0, 1.0]])
    assert np.array_equal(O.short_conv(x, w, act=False)[0], x)
    # the norm of a row of equal entries is 1 (eps aside)
    h2, y = O.block_norm(np.full((1, 8), 3.0), w_post=np.ones(8), w_pre=np.ones(8), eps=0.0)
    assert np.allclose(h2, 1.0) and np.allclose(y, 1.0)
    assert np.isclose(O.silu_grad(0.3), (O.silu(0.3 + 1e-6) - O.silu(0.3 - 1e-6)) / 2e-6)


def test_planted_mistakes_are_caught():
    # a gradient without the term through the norm's denominator does not pass the difference test
    rng = np.random.default_rng(5)
    a = {"o": rng.standard_normal((2, 6)), "w_post": np.ones(6), "w_pre": np.ones(6)}
    dy = rng.standard_normal((2, 6))
    wrong = dy * 1.0

    def f(a):
        return (O.block_norm(**a)[1] * dy).sum()
    with pytest.raises(AssertionError):
        _directional(f, a, {"o": wrong}, rng)
