"""Calls of the selective block's operators for the bounds-checked build, at the sizes, strides and alignments that
take different accesses: whole packs and single elements, whole tiles and partial ones, chunks and segments,
slices of wider arrays, odd numbers of channels with whole words of states.

Run as a child process with S4_LIB pointing at libs4_checked.so (tests/test_gpu_block_extents.py): prints one JSON line
with the number of calls and of accesses that fitted no array of their call or were misaligned."""
import json
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import structured_state_space_gb300 as s4  # noqa: E402

DTYPES = (torch.float32, torch.bfloat16, torch.float16)


def n(*shape, dtype=torch.float32):
    return torch.randn(shape, device="cuda").to(dtype)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rows(batch, L, C, dtype, left):
    """Dense for left < 0, else a slice of wider rows that starts at channel `left`."""
    return n(batch, L, C, dtype=dtype) if left < 0 else n(batch, L, left + C + 5, dtype=dtype)[..., left:left + C]


def conv(dtype):
    for W in range(2, 9):
        for batch, L, H, left in [(1, 1, 5, -1), (3, 21, 64, -1), (2, 530, 36, 8), (2, 70, 33, 3), (2, 40, 130, 4)]:
            x, dy, w, b = rows(batch, L, H, dtype, left), rows(batch, L, H, dtype, left), n(H, W), n(H)
            st, lens = n(batch + 2, W - 1, H, dtype=dtype), ints([L, 0, min(L, 3)][:batch])
            index = ints([batch + 1, -1, 0][:batch])
            s4.s4_short_conv_fwd(x, w, b, lengths=lens, state=st, state_out=st, index=index)
            s4.s4_short_conv_fwd(x, w, silu=False)
            s4.s4_short_conv_step(x[:, 0], w, b, st, index=index)
            s4.s4_short_conv_bwd(x, w, b, dy, lengths=lens, state=st[:batch], dstate=st[1:batch + 1], want_dstate0=True)
            s4.s4_short_conv_bwd(x, w, None, dy)
            yield 5


def scan(dtype):
    for batch, L, H, N, G, left in [
            (1, 1, 1, 1, 1, -1), (2, 24, 64, 4, 1, -1), (2, 37, 256, 4, 1, 8), (2, 37, 256, 8, 2, -1), (2, 40, 128, 16, 1, -1),
            (2, 41, 128, 16, 2, 8), (2, 33, 64, 32, 1, -1), (2, 20, 64, 64, 1, -1), (1, 20, 32, 128, 1, 8), (1, 21, 8, 256, 1, -1),
            (3, 35, 33, 16, 1, -1), (3, 35, 33, 4, 3, 1), (2, 40, 333, 16, 1, 3), (2, 19, 7, 64, 1, -1), (1, 90, 5, 8, 1, -1),
            (2, 30, 10, 30, 2, 2), (1, 40, 9, 200, 3, -1), (1, 1500, 64, 16, 1, -1), (2, 1100, 33, 16, 1, 1),
            (1, 700, 12, 100, 2, -1), (1, 600, 6, 256, 2, -1)]:
        x, dt, z, dy = (rows(batch, L, H, dtype, left) for _ in range(4))
        A, B, C = -torch.exp(n(H, N)), *(rows(batch, L, G * N, dtype, left).unflatten(-1, (G, N)) for _ in range(2))
        kw = dict(D=n(H), z=z, dt_bias=n(H))
        st, lens = n(batch + 2, H, N), ints([L, 0, L // 2][:batch])
        index = ints([batch + 1, -1, 0][:batch])
        s4.s4_selective_scan_fwd(x, dt, A, B, C, **kw, lengths=lens, state=st, state_out=st, index=index)
        s4.s4_selective_scan_fwd(x, dt, A, B, C)
        tok = dict(kw, z=z[:, 0])
        s4.s4_selective_step(x[:, 0], dt[:, 0], A, B[:, 0], C[:, 0], st, **tok, index=index)
        s4.s4_selective_scan_bwd(x, dt, A, B, C, dy, **kw, lengths=lens, state=st[:batch], dstate=st[1:batch + 1],
                                 want_dstate0=True)
        s4.s4_selective_scan_bwd(x, dt, A, B, C, dy)
        yield 5


def norm(dtype):
    for R, H, left in [(1, 1, -1), (5, 33, 3), (9, 256, -1), (37, 512, 8), (7, 1000, -1), (300, 2048, 16), (3, 2052, -1),
                       (3, 6000, 1), (2, 16384, -1), (2, 16383, -1)]:
        for res in {torch.float32, dtype}:
            o, gate, dy = (rows(1, R, H, dtype, left)[0] for _ in range(3))
            h, dh = rows(1, R, H, res, left)[0], rows(1, R, H, res, left)[0]
            kw = dict(gate=gate, h=h, w_post=n(H), scale=n(H), w_pre=n(H))
            s4.s4_block_norm_fwd(o, **kw)
            s4.s4_block_norm_fwd(o, w_pre=kw["w_pre"])
            s4.s4_block_norm_bwd(o, dy, dh_out=dh, **kw)
            s4.s4_block_norm_bwd(o, dh_out=dh, h=h, w_post=kw["w_post"])
            yield 4


def main():
    s4.load()
    assert s4.s4_bounds_violations() >= 0, "not a bounds-checked build"
    torch.manual_seed(0)
    calls, per = 0, {}
    for dtype in DTYPES:
        for op in (conv, scan, norm):
            before = s4.s4_bounds_violations()
            calls += sum(op(dtype))
            per[f"{op.__name__} {dtype}"] = s4.s4_bounds_violations() - before
    print(json.dumps({"calls": calls, "violations": s4.s4_bounds_violations(), "where": per}))


if __name__ == "__main__":
    main()
