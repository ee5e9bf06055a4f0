"""The selective block's operators in the bounds-checked build (no index may leave its buffer), and
with offsets beyond 32 bits: long caches and far rows."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.block_oracle as O  # noqa: E402
import structured_state_space_gb300 as s4  # noqa: E402
from block_util import Inputs, close, need_gpu, to64  # noqa: E402
from structured_state_space_gb300 import build as s4build  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def test_no_index_leaves_its_buffer():
    lib = s4build.build(bounds_check=True)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "block_bounds_cases.py")],
                       env=dict(os.environ, S4_LIB=lib), capture_output=True, text=True, timeout=900, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["calls"] >= 100 and out["violations"] == 0, out


def test_slots_beyond_32_bits():
    # 2^31 / (2048 * 256) = 4096 slots of 2 MiB; the last ones are written, read back and left alone
    r, H, N = Inputs(1), 2048, 256
    cache = torch.empty(4100, H, N, device="cuda")
    index = torch.tensor([4099, 4097], dtype=torch.int32, device="cuda")
    old = r.normal(2, H, N)
    cache[4099], cache[4097] = old[0], old[1]
    cache[4098] = 7.0
    x, dt, z = (r.normal(2, 1, H) for _ in range(3))
    A, B, C = -torch.exp(r.normal(H, N, scale=0.5)), r.normal(2, 1, 1, N), r.normal(2, 1, 1, N)
    ry, rs = O.selective_scan(*(to64(v) for v in (x, dt, A, B, C)), z=to64(z), state=to64(old))
    y = s4.s4_selective_step(x[:, 0], dt[:, 0], A, B[:, 0], C[:, 0], cache, z=z[:, 0], index=index)
    close(y, ry[:, 0], "y")
    close(cache[4099], rs[0], "slot 4099")
    close(cache[4097], rs[1], "slot 4097")
    assert (cache[4098] == 7.0).all()
    # and as prompts of one token more
    cache[4099], cache[4097] = old[0], old[1]
    two = [torch.cat([v, v], 1) for v in (x, dt, z, B, C)]
    y = s4.s4_selective_scan_fwd(two[0], two[1], A, two[3], two[4], z=two[2], state=cache, state_out=cache, index=index)
    ry, rs = O.selective_scan(*(to64(v) for v in (two[0], two[1], A, two[3], two[4])), z=to64(two[2]), state=to64(old))
    close(y, ry, "y of two tokens", 2e-5)
    close(cache[4097], rs[1], "slot 4097 after two tokens", 2e-5)


def test_rows_beyond_32_bits():
    # two sequences 2^31 elements apart in one buffer (4 GiB of bfloat16 and a little)
    L, H, W = 40, 64, 4
    far = 2 ** 31 + 8
    r = Inputs(2)
    buf = torch.zeros(far + L * H, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, L, H), (far, H, 1))
    x.copy_(r.normal(2, L, H, dtype=torch.bfloat16))
    w, b = r.normal(H, W), r.normal(H)
    close(s4.s4_short_conv_fwd(x, w, b), O.short_conv(to64(x), to64(w), to64(b))[0], "convolution")
    g = s4.s4_short_conv_bwd(x, w, b, x)
    ref = O.short_conv_grad(to64(x), to64(w), to64(b), to64(x))
    for k in g:
        close(g[k], ref[k], k)
    dt, A, B = r.normal(2, L, H, dtype=torch.bfloat16), -torch.exp(r.normal(H, 16)), r.normal(2, L, 1, 16, dtype=torch.bfloat16)
    close(s4.s4_selective_scan_fwd(x, dt, A, B, B), O.selective_scan(*(to64(v) for v in (x, dt, A, B, B)))[0], "scan")
    g = s4.s4_selective_scan_bwd(x, dt, A, B, B, x)
    ref = O.selective_scan_grad(*(to64(v) for v in (x, dt, A, B, B)), to64(x))
    close(g["dx"], ref["dx"], "scan's dx")
    rows = buf.as_strided((2, H), (far, 1))
    h, _ = s4.s4_block_norm_fwd(rows, w_post=b)
    close(h, O.block_norm(to64(rows), w_post=to64(b))[0], "norm")


def test_outputs_may_not_be_inputs():
    r = Inputs(3)
    x, w = r.normal(2, 8, 16), r.normal(16, 4)
    with pytest.raises(s4.S4Error):
        s4.s4_short_conv_fwd(x, w, y=x)
    y = s4.s4_short_conv_fwd(x, w)
    assert np.isfinite(to64(y)).all()
