"""The bounds-checked build keeps the sections of linear attention's and the vocabulary loss's workspaces apart, so that an access beyond
one's end is not within the next, and finds none."""
import ctypes
import json
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import structured_state_space_gb300 as s4  # noqa: E402
from block_util import need_gpu  # noqa: E402
from structured_state_space_gb300 import build as s4build, sequence  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GAP = 4096
A = 0x10000  # an aligned address: sizes alone count


@pytest.fixture(scope="module")
def checked():
    need_gpu()
    return s4build.build(bounds_check=True)


def test_sections_lie_apart(checked):
    libs = [s4.load(), ctypes.CDLL(checked)]

    def more(name, *args):
        got = []
        for lib in libs:
            f = getattr(lib, name)
            f.argtypes = [ctypes.c_char_p] if isinstance(args[0], bytes) else [ctypes.c_int] * len(args)
            f.restype = ctypes.c_size_t
            got.append(f(*args))
        return got[1] - got[0]
    assert more("s4_linear_attention_workspace_bytes", 1, 2000, 2, 1, 64, 64) == GAP
    assert more("s4_linear_attention_bwd_workspace_bytes", 1, 2000, 2, 2, 64, 64) == 3 * GAP
    assert more("s4_linear_attention_bwd_workspace_bytes", 1, 2000, 2, 1, 64, 64) == 5 * GAP
    # partial sums, targets' logits, copies of h and w; logits' gradients, partial dw, padding, copies
    for dtype, copies in ((0, 2), (1, 0)):
        assert more("s4_vocab_loss_workspace_bytes", sequence._LOSS.pack(A, A, A, A, A, 0, 0, 64, 64, 3000, 64, 300, 1, dtype)) == (2 + copies) * GAP
        assert more("s4_vocab_loss_bwd_workspace_bytes",
                    sequence._LOSS_BWD.pack(A, A, A, A, A, A, A, 0, 0, 64, 64, 3000, 64, 300, 1, dtype)) == (3 + copies) * GAP


def test_no_index_leaves_its_section(checked):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "sequence_bounds_more_cases.py")],
                       env=dict(os.environ, S4_LIB=checked), capture_output=True, text=True, timeout=900, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["calls"] >= 90 and out["violations"] == 0, out
