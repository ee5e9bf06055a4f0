"""Argument structs of linear attention, rotary positions, layer norm and the vocabulary loss, as the Python binding packs
them, against the C compiler's layout; the host's refusals; frequencies of rotary positions (no GPU)."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import structured_state_space_gb300 as s4
from structured_state_space_gb300 import build as s4build

torch = pytest.importorskip("torch")
from structured_state_space_gb300 import sequence  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"s4_linear_attention_args": sequence._ATTENTION, "s4_linear_attention_bwd_args": sequence._ATTENTION_BWD,
           "s4_rotary_args": sequence._ROTARY, "s4_layer_norm_args": sequence._LAYER_NORM,
           "s4_layer_norm_bwd_args": sequence._LAYER_NORM_BWD, "s4_vocab_loss_args": sequence._LOSS,
           "s4_vocab_loss_bwd_args": sequence._LOSS_BWD}
A = 0x10000  # an aligned stand-in address; validation rejects before any use


@pytest.fixture(scope="module")
def lib():
    s4build.build()
    return s4.load()


def test_struct_sizes(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "s4.h"\nint main(void) {\n'
                   + "".join(f'  printf("%zu\\n", sizeof({n}));\n' for n in STRUCTS) + "  return 0;\n}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [s.size for s in STRUCTS.values()]


def call(lib, name, fmt, *values):
    f = getattr(lib, name)
    f.argtypes, f.restype = [ctypes.c_char_p, ctypes.c_void_p], ctypes.c_int
    return f(fmt.pack(*values), None)


def refused(lib, name, fmt, ok, changes, code=1):
    for at, bad in changes:
        v = list(ok)
        v[at] = bad
        assert call(lib, name, fmt, *v) == code, (name, at, bad)


def test_linear_attention_refuses(lib):
    # q, k, v, o; log_decay, lengths, index, state, state_out, ws, bytes; scale; batch L H G K V slots dtype
    ok = [A, 8, 8, 8, A, 8, 8, 8, A, 8, 8, 8, 2 * A, 8, 8, 8, A, 0, 0, A, A, A, 256, 1.0, 1, 1, 2, 1, 8, 8, 1, 1]
    refused(lib, "s4_linear_attention_fwd", sequence._ATTENTION, ok,
            [(0, 0), (0, A + 1), (4, 0), (8, 0), (12, 0), (12, A), (1, -1), (3, -8), (16, 0), (16, A + 2), (17, A + 1), (18, A + 2),
             (19, A + 1), (20, A + 2), (24, 0), (24, 65536), (25, 0), (25, (1 << 24) + 1), (26, 0), (26, 4097), (27, 0), (27, 3), (28, 0),
             (28, 257), (29, 0), (29, 257), (30, 0), (31, 3), (31, -1)])
    refused(lib, "s4_linear_attention_fwd", sequence._ATTENTION, ok, [(22, 255), (21, A + 64)], 2)
    long = list(ok)
    long[25] = 100000  # needs more than the status block
    refused(lib, "s4_linear_attention_fwd", sequence._ATTENTION, long, [(21, 0), (22, 256)], 2)
    two = list(ok)
    two[24], two[21], two[22] = 2, A, 256  # two sequences, one slot, no index
    assert call(lib, "s4_linear_attention_fwd", sequence._ATTENTION, *two) == 1
    assert call(lib, "s4_linear_attention_bwd", sequence._ATTENTION_BWD,
                *[A, 8, 8, 8] * 4, *[2 * A, 8, 8, 8] * 3, A, 0, 0, 0, 0, A, 100, 1.0, 1, 4, 1, 1, 8, 8, 1) == 2
    ok = [A, 8, 8, 8] * 4 + [2 * A, 8, 8, 8] * 3 + [A, 0, A, A, 2 * A, A, 1 << 30, 1.0, 1, 4, 2, 1, 8, 8, 1]
    refused(lib, "s4_linear_attention_bwd", sequence._ATTENTION_BWD, ok,
            [(0, 0), (12, 0), (16, 0), (20, A), (24, A + 1), (5, -1), (28, 0), (30, A + 1), (32, A), (35, 0.0), (36, 0), (38, 0), (39, 3),
             (40, 300), (42, 9)])


def test_rotary_refuses(lib):
    # q, k, q_out, k_out; freqs, positions, batch stride; amplitude; batch L H G D R pairs inverse dtype
    ok = [A, 8, 8, 8, 3 * A, 8, 8, 8, 2 * A, 8, 8, 8, 4 * A, 8, 8, 8, A, A, 1, 1.0, 1, 1, 2, 1, 8, 4, 0, 0, 1]
    refused(lib, "s4_rotary", sequence._ROTARY, ok,
            [(0, 0), (0, A + 1), (4, A + 1), (8, 0), (12, 0), (2, -1), (16, 0), (16, A + 4), (17, A + 2), (18, -1), (20, 0), (21, 0),
             (22, 0), (22, 4097), (23, 0), (24, 0), (24, 257), (25, 0), (25, 5), (28, 4), (12, 2 * A), (12, A), (8, 3 * A)])
    same = list(ok)
    same[8], same[11] = A, 16  # in place at another stride of the heads
    assert call(lib, "s4_rotary", sequence._ROTARY, *same) == 1
    alone = list(ok)
    alone[4] = 0  # an output without its input
    assert call(lib, "s4_rotary", sequence._ROTARY, *alone) == 1


def test_layer_norm_refuses(lib):
    ok = [A, 2 * A, A, A, 8, 8, 4, 1e-5, 8, 1]
    refused(lib, "s4_layer_norm_fwd", sequence._LAYER_NORM, ok,
            [(0, 0), (1, 0), (0, A + 1), (2, A + 2), (3, A + 1), (4, -1), (6, 0), (7, -1.0), (7, float("nan")), (8, 0), (8, 16385), (9, 3)])
    same = list(ok)
    same[1], same[5] = A, 16
    assert call(lib, "s4_layer_norm_fwd", sequence._LAYER_NORM, *same) == 1
    ok = [A, A, 2 * A, A, A, A, A, 1 << 30, 8, 8, 8, 4, 1e-5, 8, 1]
    refused(lib, "s4_layer_norm_bwd", sequence._LAYER_NORM_BWD, ok,
            [(0, 0), (1, 0), (2, 0), (2, A), (3, A + 1), (4, A + 2), (8, -1), (11, 0), (12, -1.0), (13, 0), (14, 5)])
    refused(lib, "s4_layer_norm_bwd", sequence._LAYER_NORM_BWD, ok, [(6, 0), (6, A + 8), (7, 256)], 2)
    f = lib.s4_layer_norm_bwd_workspace_bytes
    f.argtypes, f.restype = [ctypes.c_longlong, ctypes.c_int], ctypes.c_size_t
    assert f(0, 8) == 0 and f(1, 16385) == 0 and f(1, 8) >= 256


def test_vocab_loss_refuses(lib):
    ok = [A, A, A, A, 2 * A, A, 1 << 30, 8, 8, 4, 8, 100, 1, 1]
    refused(lib, "s4_vocab_loss_fwd", sequence._LOSS, ok,
            [(0, 0), (1, 0), (2, 0), (3, 0), (4, 0), (4, A), (0, A + 1), (2, A + 4), (3, A + 1), (7, -1), (8, -1), (9, 0), (9, (1 << 22) + 1),
             (10, 0), (10, 16385), (11, 0), (11, (1 << 22) + 1), (13, 3)])
    refused(lib, "s4_vocab_loss_fwd", sequence._LOSS, ok, [(5, 0), (5, A + 8), (6, 256)], 2)
    ok = [A, A, A, A, A, 2 * A, 3 * A, A, 1 << 30, 8, 8, 4, 8, 100, 1, 1]
    refused(lib, "s4_vocab_loss_bwd", sequence._LOSS_BWD, ok,
            [(0, 0), (1, 0), (2, 0), (3, 0), (4, 0), (5, 0), (6, 0), (5, A), (6, A), (6, 2 * A), (4, A + 2), (5, 2 * A + 1), (12, 0), (13, 0),
             (15, 7)])
    refused(lib, "s4_vocab_loss_bwd", sequence._LOSS_BWD, ok, [(7, 0), (8, 256)], 2)


def test_workspace_sizes_grow_with_what_they_hold(lib):
    n = sequence._bytes
    assert n("s4_linear_attention_workspace_bytes", 1, 1, 4, 4, 64, 64) == 256
    assert n("s4_linear_attention_workspace_bytes", 1, 100, 4096, 1, 64, 64) == 256  # enough sequences: one segment
    shared = n("s4_linear_attention_bwd_workspace_bytes", 2, 100, 4, 2, 64, 32)
    own = n("s4_linear_attention_bwd_workspace_bytes", 2, 100, 4, 4, 64, 32)
    assert shared - own == 2 * 100 * 4 * (64 + 32) * 4
    for bad in [(0, 1, 1, 1, 1, 1), (1, 1, 3, 2, 1, 1), (1, 1, 1, 1, 257, 1), (1, 0, 1, 1, 1, 1)]:
        with pytest.raises(s4.S4Error):
            n("s4_linear_attention_workspace_bytes", *bad)


def test_tensors_that_do_not_fit():
    q = torch.zeros(1, 4, 2, 8)
    g = torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        s4.s4_linear_attention_fwd(q, q, q, g)
    with pytest.raises(TypeError):
        s4.s4_linear_attention_fwd(q.double(), q, q, g)
    with pytest.raises(TypeError):
        s4.s4_layer_norm_fwd([1.0])
    with pytest.raises(ValueError, match="CUDA"):
        s4.s4_vocab_loss_fwd(torch.zeros(2, 8), torch.zeros(5, 8), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        s4.s4_rotary_fwd(q, None, s4.s4_rotary_freqs(8)[0])


def test_rotary_frequencies():
    f, a = s4.s4_rotary_freqs(8)
    assert a == 1.0 and f.dtype == torch.float64
    np.testing.assert_allclose(f, [1, 0.1, 0.01, 0.001], rtol=1e-14)
    np.testing.assert_allclose(s4.s4_rotary_freqs(8, scaling="linear", factor=4.0)[0], f / 4, rtol=1e-15)
    # a larger base: the slowest pair is slowed by the factor, the fastest not at all
    b, _ = s4.s4_rotary_freqs(8, scaling="base", factor=4.0)
    np.testing.assert_allclose([b[0], b[-1]], [1, 0.001 / 4], rtol=1e-13)
    # by parts: at a length of 1000, turns are 159, 16, 1.6, 0.16
    p, a = s4.s4_rotary_freqs(8, scaling="parts", factor=4.0, length=1000)
    kept = [(f[i].item() * 1000 / (2 * math.pi) - 1) / 31 for i in (1, 2)]
    want = [1.0] + [f[i].item() * (k + (1 - k) / 4) for i, k in zip((1, 2), kept)] + [0.001 / 4]
    np.testing.assert_allclose(p, want, rtol=1e-14)
    assert abs(a - (1 + 0.1 * math.log(4))) < 1e-15
    assert s4.s4_rotary_freqs(8, scaling="parts", factor=1.0, length=1000)[1] == 1.0
    for bad in (dict(width=7), dict(width=0), dict(width=8, scaling="other"), dict(width=8, scaling="parts"),
                dict(width=8, base=-1.0), dict(width=8, factor=0.0), dict(width=8, scaling="parts", length=9, turns=(2, 2))):
        with pytest.raises(ValueError):
            s4.s4_rotary_freqs(**bad)


def test_oracle_against_itself():
    """The oracle's gradients against differences of its forward passes, in float64."""
    import oracle.sequence_oracle as O
    r = np.random.default_rng(0)
    q, k, v, do = r.standard_normal((2, 9, 4, 5)), r.standard_normal((2, 9, 2, 5)), r.standard_normal((2, 9, 2, 3)), r.standard_normal((2, 9, 4, 3))
    s0, ds, g, lens = r.standard_normal((2, 4, 5, 3)), r.standard_normal((2, 4, 5, 3)), -r.random(4), [9, 4]

    def loss(q, k, v, s0):
        o, s = O.linear_attention(q, k, v, g, 0.7, lens, s0)
        return (o * do).sum() + (s * ds).sum()
    grads = O.linear_attention_grad(q, k, v, g, do, 0.7, lens, s0, ds)
    for n, at in (("dq", 0), ("dk", 1), ("dv", 2), ("dstate0", 3)):
        args = [q, k, v, s0]
        way = r.standard_normal(args[at].shape)
        up, down = ([x + e * way if i == at else x for i, x in enumerate(args)] for e in (0.5, -0.5))
        assert abs(loss(*up) - loss(*down) - (grads[n] * way).sum()) < 1e-9, n  # (linear in each)
    h, w, t, dl = r.standard_normal((6, 4)), r.standard_normal((7, 4)), np.array([1, -1, 0, 6, 3, 2]), r.standard_normal(6)
    gl = O.vocab_loss_grad(h, w, t, dl)
    for n, at in (("dh", 0), ("dw", 1)):
        way = r.standard_normal((h, w)[at].shape)
        f = [(O.vocab_loss(*(x + e * way if i == at else x for i, x in enumerate((h, w))), t)[0] * dl).sum() for e in (1e-5, -1e-5)]
        assert abs((f[0] - f[1]) / 2e-5 - (gl[n] * way).sum()) < 1e-7, n
    x, dy, w = r.standard_normal((3, 8)), r.standard_normal((3, 8)), r.standard_normal(8)
    way = r.standard_normal(x.shape)
    f = [(O.layer_norm(x + e * way, w) * dy).sum() for e in (1e-5, -1e-5)]
    assert abs((f[0] - f[1]) / 2e-5 - (O.layer_norm_grad(x, dy, w)["dx"] * way).sum()) < 1e-8
