"""The selective block's operators in the bounds-checked build: every access to global memory lies inside an array of its
call, or a section of its workspace, that may be accessed so, and is aligned to its width.  What the check finds is
tested on the CPU (test_block_extents.py)."""
import json
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from block_util import need_gpu  # noqa: E402
from structured_state_space_gb300 import build as s4build  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def test_every_access_fits():
    lib = s4build.build(bounds_check=True)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "block_extents_cases.py")],
                       env=dict(os.environ, S4_LIB=lib), capture_output=True, text=True, timeout=900, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["calls"] >= 900 and out["violations"] == 0, out
