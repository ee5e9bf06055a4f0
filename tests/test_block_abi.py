"""The selective block's argument structs, as the Python binding packs them, against the C
compiler's layout of include/s4.h, and the host's refusal of bad arguments (no GPU)."""
import ctypes
import os
import struct
import subprocess

import pytest

import structured_state_space_gb300 as s4
from structured_state_space_gb300 import block
from structured_state_space_gb300 import build as s4build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"s4_short_conv_args": block._CONV, "s4_short_conv_bwd_args": block._CONV_BWD,
           "s4_selective_args": block._SCAN, "s4_selective_bwd_args": block._SCAN_BWD,
           "s4_block_norm_args": block._NORM, "s4_block_norm_bwd_args": block._NORM_BWD}
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


def conv(**kw):
    v = dict(x=(A, 8, 8), y=(2 * A, 8, 8), w=A, bias=A, lengths=0, index=0, state=A, out=A, ws=A, nws=256, batch=1, L=1, H=8,
             W=4, slots=1, dtype=1, silu=1) | kw
    return *v["x"], *v["y"], *(v[k] for k in ("w", "bias", "lengths", "index", "state", "out", "ws", "nws", "batch", "L",
                                              "H", "W", "slots", "dtype", "silu"))


@pytest.mark.parametrize("kw,code", [
    ({"x": (0, 8, 8)}, 1), ({"y": (0, 8, 8)}, 1), ({"x": (A + 1, 8, 8)}, 1), ({"x": (A, -8, 8)}, 1), ({"w": 0}, 1),
    ({"w": A + 2}, 1), ({"batch": 0}, 1), ({"batch": 65536}, 1), ({"L": 0}, 1), ({"L": (1 << 24) + 1}, 1), ({"H": 0}, 1),
    ({"H": 65537}, 1), ({"W": 1}, 1), ({"W": 9}, 1), ({"dtype": 3}, 1), ({"slots": 0}, 1), ({"batch": 2}, 1),
    ({"state": A + 1}, 1), ({"index": A + 2}, 1), ({"L": 2, "y": (A, 8, 8)}, 1), ({"nws": 255}, 2), ({"ws": A + 64}, 2)])
def test_short_conv_refuses(lib, kw, code):
    assert call(lib, "s4_short_conv_fwd", block._CONV, *conv(**kw)) == code


def scan(**kw):
    v = dict(x=(A, 8, 8), dt=(A, 8, 8), z=(0, 0, 0), B=(A, 8, 8), C=(A, 8, 8), y=(A, 8, 8), A=A, D=A, bias=A, lengths=0,
             index=0, state=A, out=A, ws=A, nws=256, bg=4, cg=4, batch=1, L=1, H=8, N=4, G=1, slots=1, dtype=1,
             softplus=1) | kw
    return (*v["x"], *v["dt"], *v["z"], *v["B"], *v["C"], *v["y"], *(v[k] for k in (
        "A", "D", "bias", "lengths", "index", "state", "out", "ws", "nws", "bg", "cg", "batch", "L", "H", "N", "G", "slots",
        "dtype", "softplus")))


@pytest.mark.parametrize("kw,code", [
    ({"x": (0, 8, 8)}, 1), ({"dt": (A + 1, 8, 8)}, 1), ({"z": (A + 1, 8, 8)}, 1), ({"B": (0, 8, 8)}, 1), ({"C": (A, 8, -1)}, 1),
    ({"y": (0, 8, 8)}, 1), ({"A": 0}, 1), ({"D": A + 1}, 1), ({"state": A + 2}, 1), ({"N": 0}, 1), ({"N": 257}, 1), ({"G": 0}, 1),
    ({"G": 3}, 1), ({"batch": 2}, 1), ({"slots": 0}, 1), ({"dtype": -1}, 1), ({"bg": -1}, 1), ({"nws": 100}, 2),
    ({"ws": A + 8}, 2), ({"L": 100000, "ws": 0}, 2), ({"L": 100000, "nws": 256}, 2)])
def test_selective_scan_refuses(lib, kw, code):
    assert call(lib, "s4_selective_scan_fwd", block._SCAN, *scan(**kw)) == code


def test_selective_scan_bwd_refuses(lib):
    # nine strided arrays; dB, dC, A, D, dt_bias, lengths, state0, dstate, dstate0, dA, dD, ddt_bias, ws
    ok = [A, 8, 8] * 9 + [A] * 8 + [A + 256] + [A] * 4 + [256, 4, 4, 1, 1, 8, 4, 1, 1, 1]
    assert call(lib, "s4_selective_scan_bwd", block._SCAN_BWD, *ok) == 2  # workspace too small
    # x, dz without z, z without dz, dB, D without dD, dstate0 = dstate, dA, batch, N, G, a stride
    for at, bad in [(0, 0), (6, 0), (24, 0), (27, 0), (37, 0), (35, A), (36, 0), (43, 0), (46, 257), (47, 3), (1, -1)]:
        v = list(ok)
        v[at] = bad
        assert call(lib, "s4_selective_scan_bwd", block._SCAN_BWD, *v) == 1, (at, bad)


def test_null_structs_and_workspace_sizes(lib):
    for n in ("s4_short_conv_fwd", "s4_short_conv_bwd", "s4_block_norm_fwd", "s4_block_norm_bwd"):
        f = getattr(lib, n)
        f.argtypes, f.restype = [ctypes.c_char_p, ctypes.c_void_p], ctypes.c_int
        assert f(None, None) == 1
    f = lib.s4_short_conv_bwd_workspace_bytes
    f.restype = ctypes.c_size_t
    assert f(1, 1, 8, 4) >= 256 and f(0, 1, 8, 4) == 0 and f(1, 1, 8, 9) == 0
    f = lib.s4_block_norm_bwd_workspace_bytes
    f.argtypes, f.restype = [ctypes.c_longlong, ctypes.c_int], ctypes.c_size_t
    assert f(0, 8) == 0 and f(1, 16385) == 0


def test_block_norm_refuses(lib):
    ok = [A] * 8 + [8] * 5 + [4, 1e-5, 8, 1, 1]
    for at, bad in [(0, 0), (3, 0), (4, 0), (0, A + 1), (2, A + 2), (13, 0), (14, -1.0), (14, float("nan")), (15, 0),
                    (15, 16385), (16, 3), (8, -1)]:
        v = list(ok)
        v[at] = bad
        assert call(lib, "s4_block_norm_fwd", block._NORM, *v) == 1, (at, bad)
    ok = [A] * 15 + [256] + [8] * 8 + [4, 1e-5, 8, 1, 1]
    assert call(lib, "s4_block_norm_bwd", block._NORM_BWD, *ok) == 2  # workspace too small
    for at, bad in [(0, 0), (5, 0), (6, 0), (7, 0), (11, 0), (10, 0)]:
        v = list(ok)
        v[at] = bad
        assert call(lib, "s4_block_norm_bwd", block._NORM_BWD, *v) == 1, (at, bad)


def test_status_string():
    assert s4.s4_status_str(10) == "length or state slot out of range"
    assert s4.STATUS[10] == "S4_ERR_INVALID_INDEX"
    assert struct.calcsize("@P") == 8
