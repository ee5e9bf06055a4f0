"""The package without torch: importing it, and all its names, does not load torch; the selective block's operators load it
when they are first called."""
import subprocess
import sys
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]


def test_all_names_without_torch():
    run("import sys\nsys.modules['torch'] = None\n"
        "from structured_state_space_gb300 import *\n"
        "assert s4_workspace_bytes and callable(s4_short_conv_fwd) and callable(s4_block_norm_bwd)\n"
        "try:\n    s4_selective_step(None, None, None, None, None, None)\n"
        "except ImportError:\n    pass\nelse:\n    raise AssertionError('ran without torch')\n")


def test_names_become_the_operators():
    run("import structured_state_space_gb300 as s4\nfrom structured_state_space_gb300 import s4_short_conv_fwd as early\n"
        "for f in (early, s4.s4_short_conv_fwd, s4.s4_short_conv_fwd):\n"
        "    try:\n        f(1, 2)\n    except (TypeError, AttributeError):\n        pass\n"
        "from structured_state_space_gb300 import block\n"
        "assert all(getattr(s4, n) is getattr(block, n) for n in block.__all__)\n"
        "assert set(block.__all__) <= set(s4.__all__)\n")
