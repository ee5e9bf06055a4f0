"""Small calls of linear attention, rotary positions, layer norm and the vocabulary loss, for the bounds-checked build
(run as tests/block_bounds_cases.py is, by tests/test_gpu_sequence_bounds.py)."""
import json
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import structured_state_space_gb300 as s4  # noqa: E402
from block_bounds_cases import finite  # noqa: E402


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
        for batch, L, H, G, K, V in [(1, 1, 1, 1, 1, 1), (3, 37, 4, 2, 33, 7), (2, 130, 2, 2, 64, 64), (2, 300, 2, 1, 128, 72),
                                     (1, 900, 1, 1, 40, 128), (1, 70, 1, 1, 256, 256), (3, 129, 2, 1, 16, 128)]:
            for left in (0, 1):
                q, k, v = (n(batch, L, h, left + d, dtype=dtype)[..., left:] for h, d in ((H, K), (G, K), (G, V)))
                do, g, cache = n(batch, L, H, V, dtype=dtype), -torch.rand(H, device="cuda"), n(batch + 1, H, K, V)
                lens, index = ints([L, 0, L // 2][:batch]), ints([1, -1, 0][:batch])
                assert finite(s4.s4_linear_attention_fwd(q, k, v, g, lengths=lens, state=cache, state_out=cache, index=index))
                assert finite(s4.s4_linear_attention_fwd(q, k, v, g))
                assert finite(s4.s4_linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g, cache, index=index))
                assert finite(s4.s4_linear_attention_bwd(q, k, v, g, do, lengths=lens, state=cache[:batch],
                                                         dstate=cache[:batch].clone(), want_dstate0=True))
                calls += 4
        for batch, L, H, G, D, rot in [(1, 1, 1, 1, 2, 2), (2, 37, 4, 2, 64, 64), (3, 5, 8, 2, 33, 30), (2, 9, 2, 1, 256, 128)]:
            freqs, _ = s4.s4_rotary_freqs(rot, device="cuda")
            for pairs in (False, True):
                q, k = n(batch, L, H, D, dtype=dtype), n(batch, L, G, D, dtype=dtype)
                assert finite(s4.s4_rotary_fwd(q, k, freqs, pairs=pairs))
                assert finite(s4.s4_rotary_bwd(q, k, freqs, pairs=pairs, positions=ints(list(range(L))), q_out=q, k_out=k))
                calls += 2
        for rows, H in [(1, 1), (5, 33), (70, 64), (37, 128), (100, 1000), (33, 2048), (9, 8200), (300, 512)]:
            x, dy, w, b = n(rows, H, dtype=dtype), n(rows, H, dtype=dtype), n(H), n(H)
            assert finite(s4.s4_layer_norm_fwd(x, w, b)) and finite(s4.s4_layer_norm_bwd(x, dy, w, b))
            calls += 2
        for rows, H, V in [(1, 1, 1), (3, 40, 257), (130, 33, 300), (129, 64, 1000), (40, 264, 70)]:
            h, w = n(rows, H, dtype=dtype), n(V, H, dtype=dtype)
            t = torch.randint(-1, V, (rows,), device="cuda")
            loss, lse = s4.s4_vocab_loss_fwd(h, w, t)
            assert finite(loss) and finite(s4.s4_vocab_loss_bwd(h, w, t.int(), lse, torch.ones_like(loss)))
            calls += 2
    torch.cuda.synchronize()
    print(json.dumps({"calls": calls, "violations": s4.s4_bounds_violations()}))


if __name__ == "__main__":
    main()
