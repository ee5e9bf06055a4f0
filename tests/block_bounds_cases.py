"""Small calls of the selective block's operators, for the bounds-checked build.

Run as a child process with S4_LIB pointing at libs4_checked.so (see tests/test_gpu_block_bounds.py): it makes the
calls at odd, ragged and aligned sizes, checks that the outputs are finite, and prints one JSON line with the
number of out-of-extent indices that the kernels counted."""
import json
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import structured_state_space_gb300 as s4  # noqa: E402


def finite(v):
    if isinstance(v, dict):
        return all(finite(x) for x in v.values())
    if isinstance(v, tuple):
        return all(finite(x) for x in v if x is not None)
    return bool(torch.isfinite(v).all())


def main():
    s4.load()
    assert s4.s4_bounds_violations() >= 0, "not a bounds-checked build"
    torch.manual_seed(0)
    calls = 0

    def n(*shape, dtype=torch.float32):
        return torch.randn(shape, device="cuda").to(dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        for batch, L, H, W in [(1, 1, 1, 2), (3, 37, 33, 3), (2, 130, 256, 4), (2, 70, 136, 8)]:
            x, w, b, st = n(batch, L, H, dtype=dtype), n(H, W), n(H), n(batch + 1, W - 1, H, dtype=dtype)
            lens, index = ints([L, 0, L // 2][:batch]), ints([1, -1, 0][:batch])
            assert finite(s4.s4_short_conv_fwd(x, w, b, lengths=lens, state=st, state_out=st, index=index))
            assert finite(s4.s4_short_conv_step(x[:, 0], w, b, st, index=index))
            assert finite(s4.s4_short_conv_bwd(x, w, b, x, lengths=lens, state=n(batch, W - 1, H, dtype=dtype),
                                               dstate=n(batch, W - 1, H, dtype=dtype), want_dstate0=True))
            calls += 3
        for batch, L, H, N, G in [(1, 1, 1, 1, 1), (3, 37, 34, 16, 2), (2, 64, 256, 16, 1), (1, 700, 64, 16, 1),
                                  (2, 50, 32, 64, 1), (1, 40, 12, 200, 3)]:
            x, dt, z = n(batch, L, H, dtype=dtype), n(batch, L, H, dtype=dtype), n(batch, L, H, dtype=dtype)
            A, B, C = -torch.exp(n(H, N)), n(batch, L, G, N, dtype=dtype), n(batch, L, G, N, dtype=dtype)
            kw = dict(D=n(H), z=z, dt_bias=n(H))
            lens, index, st = ints([L, 0, L // 2][:batch]), ints([1, -1, 0][:batch]), n(batch + 1, H, N)
            assert finite(s4.s4_selective_scan_fwd(x, dt, A, B, C, **kw, lengths=lens, state=st, state_out=st, index=index))
            assert finite(s4.s4_selective_step(x[:, 0], dt[:, 0], A, B[:, 0], C[:, 0], st, D=kw["D"], z=z[:, 0],
                                               dt_bias=kw["dt_bias"], index=index))
            assert finite(s4.s4_selective_scan_bwd(x, dt, A, B, C, x, **kw, lengths=lens, state=n(batch, H, N),
                                                   dstate=n(batch, H, N), want_dstate0=True))
            calls += 3
        for rows, H in [(1, 1), (5, 33), (9, 256), (7, 1000), (300, 2048), (3, 6000)]:
            o = n(rows, H, dtype=dtype)
            kw = dict(gate=n(rows, H, dtype=dtype), h=n(rows, H), w_post=n(H), scale=n(H), w_pre=n(H))
            assert finite(s4.s4_block_norm_fwd(o, **kw))
            assert finite(s4.s4_block_norm_bwd(o, o, dh_out=n(rows, H), **kw))
            calls += 2
    print(json.dumps({"calls": calls, "violations": s4.s4_bounds_violations()}))


if __name__ == "__main__":
    main()
