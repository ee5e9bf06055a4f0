"""The angle of rotary positions: off by 2^-30 turns at most, at any position of 32 bits and any frequency below 2^10."""
import random
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import structured_state_space_gb300 as s4  # noqa: E402
from block_util import need_gpu  # noqa: E402

pytestmark = pytest.mark.gpu
PI = Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899, 10 ** 80)


@pytest.mark.parametrize("freq", [1023.9, 700.3, 1.0, 0.37, 1e-5, -513.7])
def test_angles_near_whole_turns(freq):
    need_gpu()
    r = random.Random(1)
    one = Fraction(freq) / (2 * PI)
    unit = round(one * 2 ** 200)  # turns of a position, in units of 2^-200
    # positions that end within 2^-8 of a whole turn, where a sine shows the angle's last bits, and the farthest ones
    near = []
    for p in [2 ** 31 - 1, -2 ** 31] + [r.randrange(-2 ** 31, 2 ** 31) for _ in range(200000)]:
        turn = (p * unit) % 2 ** 200
        turn -= 2 ** 200 if turn >= 2 ** 199 else 0
        if abs(turn) < 2 ** 192 or abs(p) >= 2 ** 31 - 1:
            near.append((p, turn / 2 ** 200))
    assert len(near) > 500
    pos = torch.tensor([p for p, _ in near], dtype=torch.int32, device="cuda")
    x = torch.zeros(len(near), 1, 2, device="cuda")
    x[..., 0] = 1
    y, _ = s4.s4_rotary_fwd(x, None, torch.tensor([freq], dtype=torch.float64, device="cuda"), positions=pos)
    t = 2 * np.pi * np.array([t for _, t in near])
    off = np.abs(y[:, 0].double().cpu().numpy() - np.stack([np.cos(t), np.sin(t)], -1))
    # the angle, and a few roundings of the results: 2^-22 of each
    assert (off[:, 1] <= 2 * np.pi * 2.0 ** -30 + 2.0 ** -22 * np.abs(np.sin(t))).all(), off[:, 1].max()
    assert (off[:, 0] <= 2 * np.pi * 2.0 ** -30 + 2.0 ** -22).all()
