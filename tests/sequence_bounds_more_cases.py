"""More calls for the bounds-checked build (run as tests/block_bounds_cases.py is, by tests/test_gpu_sequence_sections.py): linear
attention over several segments of ragged batches, walks made again token by token, losses with padding, many channels
and partial sums."""
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
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        for batch, L, H, G, K, V in [(4, 700, 2, 1, 64, 64), (3, 600, 2, 2, 128, 40), (2, 500, 1, 1, 33, 128), (2, 300, 2, 1, 200, 64)]:
            q, k, v, do = n(batch, L, H, K, dtype=dtype), n(batch, L, G, K, dtype=dtype), n(batch, L, G, V, dtype=dtype), n(batch, L, H, V, dtype=dtype)
            g, s0 = -torch.rand(H, device="cuda"), n(batch, H, K, V)
            lens = torch.tensor([L - 1, 129, 0, L][:batch], dtype=torch.int32, device="cuda")
            assert finite(s4.s4_linear_attention_fwd(q, k, v, g, lengths=lens, state=s0, state_out=s0.clone()))
            assert finite(s4.s4_linear_attention_bwd(q, k, v, g, do, lengths=lens, state=s0, dstate=s0.clone(), want_dstate0=True))
            # walks made again: states kept in place, and none
            v[0, L // 2, 0, 1] = float("nan")
            do[1, 3, 0, 0] = float("inf")
            both = s0.clone()
            s4.s4_linear_attention_fwd(q, k, v, g, lengths=lens, state=both, state_out=both)
            s4.s4_linear_attention_fwd(q, k, v, g)
            s4.s4_linear_attention_bwd(q, k, v, g, do, lengths=lens, state=s0, dstate=s0.clone(), want_dstate0=True)
            calls += 5
        for rows, H, V in [(300, 64, 600), (5000, 40, 300), (130, 300, 513), (70, 4100, 300), (20, 8200, 70)]:
            h, w = n(rows, H, dtype=dtype), n(V, H, dtype=dtype)
            t = torch.randint(-1, V, (rows,), device="cuda")
            h[t < 0] = float("nan")
            loss, lse = s4.s4_vocab_loss_fwd(h, w, t)
            assert finite(loss) and finite(s4.s4_vocab_loss_bwd(h, w, t.int(), lse, torch.ones_like(loss)))
            calls += 2
    torch.cuda.synchronize()
    print(json.dumps({"calls": calls, "violations": s4.s4_bounds_violations()}))


if __name__ == "__main__":
    main()
