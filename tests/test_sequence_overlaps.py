"""Arrays that may not be one another: the host refuses calls of linear attention, rotary positions and layer norm that
would read what another part of the same call writes (no GPU: validation rejects before any use)."""
import ctypes

import pytest

import structured_state_space_gb300 as s4
from structured_state_space_gb300 import build as s4build

torch = pytest.importorskip("torch")
from structured_state_space_gb300 import sequence  # noqa: E402

A = 0x10000  # aligned stand-in addresses


@pytest.fixture(scope="module")
def lib():
    s4build.build()
    return s4.load()


def call(lib, name, fmt, values):
    f = getattr(lib, name)
    f.argtypes, f.restype = [ctypes.c_char_p, ctypes.c_void_p], ctypes.c_int
    return f(fmt.pack(*values), None)


# q, k, v, dout, dq, dk, dv; log_decay, lengths, state0, dstate, dstate0; ws, its bytes (too few: what is not refused
# for its arrays is refused for that, with 2); scale; batch L H G K V dtype
GRADIENTS = [x for i in range(7) for x in (A * (i + 1), 64, 16, 8)] + [A, 0, 8 * A, 9 * A, 10 * A, A, 100, 1.0, 2, 4, 2, 2, 8, 8, 1]


def gradients(lib, **changes):
    at = {"dq": 16, "dk": 20, "dv": 24, "state0": 30, "dstate": 31, "dstate0": 32}
    v = list(GRADIENTS)
    for n, x in changes.items():
        v[at[n]] = x
    return call(lib, "s4_linear_attention_bwd", sequence._ATTENTION_BWD, v)


def test_a_states_gradient_is_neither_state(lib):
    # one launch reads state0 for dq and writes dstate0 with dv, in no order
    assert gradients(lib) == 2
    assert gradients(lib, dstate0=0) == 2 and gradients(lib, state0=0, dstate=0) == 2
    assert gradients(lib, dstate=8 * A) == 2  # (both are only read)
    assert gradients(lib, dstate0=9 * A) == 1
    assert gradients(lib, dstate0=8 * A) == 1
    assert gradients(lib, dstate0=8 * A, dstate=0) == 1


def test_outputs_of_one_address_for_many_elements_are_refused(lib):
    """A stride of 0 in a dimension of more than one: an output's elements would replace one another, and in place a
    broadcast head would be turned once for each head that shares it."""
    # attention: q, k, v, o; ...; ws, its bytes (too few); scale; batch L H G K V slots dtype
    ok = [x for i in range(4) for x in (A * (i + 1), 64, 16, 8)] + [A, 0, 0, 0, 0, A, 100, 1.0, 2, 4, 2, 2, 8, 8, 0, 1]
    assert call(lib, "s4_linear_attention_fwd", sequence._ATTENTION, ok) == 2
    for at in (13, 14, 15):
        v = list(ok)
        v[at] = 0
        assert call(lib, "s4_linear_attention_fwd", sequence._ATTENTION, v) == 1, at
        v[at - 12] = 0
        v[at] = ok[at]
        assert call(lib, "s4_linear_attention_fwd", sequence._ATTENTION, v) == 2, at  # inputs may be broadcast
        v[at], v[{13: 24, 14: 25, 15: 26}[at]] = 0, 1  # one element has any stride
        v[27] = 1
        if at != 14:  # (a token is another form, which takes this workspace)
            assert call(lib, "s4_linear_attention_fwd", sequence._ATTENTION, v) == 2, at
    for first in (16, 20, 24):
        for at in range(first + 1, first + 4):
            v = list(GRADIENTS)
            v[at] = 0
            assert call(lib, "s4_linear_attention_bwd", sequence._ATTENTION_BWD, v) == 1, at
    # rotary, in place: q, k, q_out, k_out; freqs, positions, batch stride; amplitude; batch L H G D R pairs inverse dtype
    ok = [A, 64, 16, 8, 2 * A, 64, 16, 8, A, 64, 16, 8, 2 * A, 64, 16, 8, A, 0, 0, 1.0, 2, 4, 2, 2, 8, 4, 0, 0, 1]
    for at in (1, 2, 3, 5, 6, 7):
        v = list(ok)
        v[at] = v[at + 8] = 0
        assert call(lib, "s4_rotary", sequence._ROTARY, v) == 1, at
    # layer norm: x, y, w, b; x_row, y_row, rows; eps; H dtype
    assert call(lib, "s4_layer_norm_fwd", sequence._LAYER_NORM, [A, 2 * A, 0, 0, 8, 0, 4, 1e-5, 8, 1]) == 1
    assert call(lib, "s4_layer_norm_fwd", sequence._LAYER_NORM, [A, A, 0, 0, 0, 0, 4, 1e-5, 8, 1]) == 1
    ok = [A, 2 * A, 3 * A, 0, 4 * A, 5 * A, A, 100, 8, 8, 8, 4, 1e-5, 8, 1]
    assert call(lib, "s4_layer_norm_bwd", sequence._LAYER_NORM_BWD, ok) == 2
    assert call(lib, "s4_layer_norm_bwd", sequence._LAYER_NORM_BWD, ok[:10] + [0] + ok[11:]) == 1


def test_a_gradients_scale_has_an_inverse(lib):
    """The state's gradient goes through the walks in units of the scale; 1 / 2e-39 is an infinity in 32 bits."""
    at = 35
    for scale, code in ((1.0, 2), (-0.3, 2), (3e-39, 2), (0.0, 1), (2e-39, 1), (-1e-45, 1), (float("nan"), 1), (float("inf"), 1)):
        assert call(lib, "s4_linear_attention_bwd", sequence._ATTENTION_BWD, GRADIENTS[:at] + [scale] + GRADIENTS[at + 1:]) == code, scale
