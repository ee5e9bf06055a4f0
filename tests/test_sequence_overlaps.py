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
