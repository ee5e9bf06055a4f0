"""Linear attention, rotary positions, layer norm and the vocabulary loss: the bounds-checked build, offsets beyond
32 bits, other streams, captured graphs, and waits that give up."""
import json
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import oracle.sequence_oracle as O  # noqa: E402
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
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "sequence_bounds_cases.py")],
                       env=dict(os.environ, S4_LIB=lib), capture_output=True, text=True, timeout=900, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["calls"] >= 200 and out["violations"] == 0, out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_and_slots_beyond_32_bits(dtype):
    # two sequences 2^31 elements apart in one buffer; states at slots beyond 2^31 elements
    L, H, D = 140, 2, 64
    far = 2 ** 31 + 8
    r = Inputs(1)
    buf = torch.zeros(far + L * H * D, dtype=dtype, device="cuda")
    q = buf.as_strided((2, L, H, D), (far, H * D, D, 1))
    q.copy_(r.normal(2, L, H, D, dtype=dtype))
    g = torch.tensor([-0.01, -0.3], device="cuda")
    slots = 2 ** 31 // (H * D * D) + 3
    cache = torch.empty(slots, H, D, D, device="cuda")
    index = torch.tensor([slots - 1, slots - 3], dtype=torch.int32, device="cuda")
    old = r.normal(2, H, D, D)
    cache[slots - 1], cache[slots - 3] = old[0], old[1]
    cache[slots - 2] = 7.0
    tol = 1e-5 if dtype == torch.float32 else 2 * 2.0 ** -8
    o = s4.s4_linear_attention_fwd(q, q, q, g, state=cache, state_out=cache, index=index)
    ref, s = O.linear_attention(to64(q), to64(q), to64(q), to64(g), D ** -0.5, state=to64(old))
    close(o, ref, "o", tol)
    close(cache[slots - 1], s[0], "the last slot")
    close(cache[slots - 3], s[1], "another")
    assert (cache[slots - 2] == 7.0).all()
    o = s4.s4_linear_attention_step(q[:, 0], q[:, 0], q[:, 0], g, cache, index=index)
    ref, s = O.linear_attention(to64(q[:, :1]), to64(q[:, :1]), to64(q[:, :1]), to64(g), D ** -0.5, state=s)
    close(o, ref[:, 0], "a token's o", tol)
    close(cache[slots - 1], s[0], "the last slot after a token", 2e-5)
    del cache
    got = s4.s4_linear_attention_bwd(q, q, q, g, q)
    want = O.linear_attention_grad(to64(q), to64(q), to64(q), to64(g), to64(q), D ** -0.5)
    for n in ("dq", "dk", "dv"):
        close(got[n], want[n], n, tol)
    freqs, _ = s4.s4_rotary_freqs(D, device="cuda")
    y, _ = s4.s4_rotary_fwd(q, None, freqs)
    close(y, O.rotary(to64(q), to64(freqs), [list(range(L))] * 2, False), "rotary")
    rows = buf.as_strided((2, H * D), (far, 1))
    close(s4.s4_layer_norm_fwd(rows), O.layer_norm(to64(rows)), "layer norm")
    t = torch.tensor([1, 0], device="cuda")
    w = r.normal(5, H * D, dtype=dtype)
    close(s4.s4_vocab_loss_fwd(rows, w, t)[1], O.vocab_loss(to64(rows), to64(w), to64(t).astype(int))[1], "lse")


def calls(seed, dtype=torch.bfloat16):
    """Every operator once: a function, and its tensors."""
    r = Inputs(seed)
    q, k, v, do = (r.normal(2, 300, 2, 64, dtype=dtype) for _ in range(4))
    g = torch.tensor([-0.01, -0.2], device="cuda")
    freqs, _ = s4.s4_rotary_freqs(64, device="cuda")
    x, w, b = r.normal(50, 256, dtype=dtype), r.normal(256), r.normal(256)
    words = r.normal(700, 256, dtype=dtype)
    t = torch.from_numpy(r.rng.integers(-1, 700, 50)).cuda()
    cache, dl = r.normal(2, 2, 64, 64), r.normal(50)

    def run(ws=None, stream=None):
        out = [s4.s4_linear_attention_fwd(q, k, v, g, state=cache, stream=stream),
               s4.s4_linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g, cache, state_out=torch.empty_like(cache),
                                           stream=stream),
               *s4.s4_linear_attention_bwd(q, k, v, g, do, stream=stream).values(),
               *s4.s4_rotary_fwd(q, k, freqs, stream=stream), s4.s4_layer_norm_fwd(x, w, b, stream=stream),
               *s4.s4_layer_norm_bwd(x, x, w, b, stream=stream).values()]
        loss, lse = s4.s4_vocab_loss_fwd(x, words, t, stream=stream)
        return out + [loss, lse, *s4.s4_vocab_loss_bwd(x, words, t, lse, dl, stream=stream).values()]
    return run, (q, k, v, do, x, words, cache)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_another_stream_and_twice_the_same(dtype):
    run, _ = calls(2, dtype)
    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = run(stream=s)
    s.synchronize()
    for a, b, c in zip(want, got, run()):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_captured_graphs():
    run, tensors = calls(3)
    run2, _ = calls(4)
    want2 = run2()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run(), run2()
    s.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one, stream=s):
        got = run()
    with torch.cuda.graph(two, stream=s, pool=one.pool()):
        got2 = run2()
    # other inputs at the same places, replayed in turn, twice
    other, filled = calls(5)
    for a, b in zip(tensors, filled):
        a.copy_(b)
    for _ in range(2):
        one.replay()
        torch.cuda.synchronize()
        saved = [v.clone() for v in got]
        two.replay()
        torch.cuda.synchronize()
        # (decays, weights and targets are those of the first inputs)
        for a, b in zip(saved, run()):
            assert torch.equal(a, b)
        for a, b in zip(got2, want2):
            assert torch.equal(a, b)


def test_two_calls_at_once_on_two_streams():
    run, _ = calls(6)
    run2, _ = calls(7)
    want, want2 = run(), run2()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got, got2 = run(stream=a), run2(stream=b)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got + got2, want + want2))


def test_waits_that_give_up_are_recorded():
    r = Inputs(8)
    q = r.normal(1, 300, 2, 64, dtype=torch.bfloat16)
    g = torch.tensor([-0.1, -0.1], device="cuda")
    h, w, t = r.normal(20, 64, dtype=torch.bfloat16), r.normal(300, 64, dtype=torch.bfloat16), torch.arange(20, device="cuda")
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    want = s4.s4_linear_attention_fwd(q, q, q, g), *s4.s4_vocab_loss_fwd(h, w, t)
    try:
        s4.s4_set_wait_limit(0)
        s4.s4_linear_attention_fwd(q, q, q, g, ws=ws)
        assert s4.STATUS[s4.s4_get_status(ws)] == "S4_ERR_TIMEOUT"
        s4.s4_vocab_loss_fwd(h, w, t, ws=ws)
        assert s4.STATUS[s4.s4_get_status(ws)] == "S4_ERR_TIMEOUT"
    finally:
        s4.s4_set_wait_limit(-1)
    got = s4.s4_linear_attention_fwd(q, q, q, g, ws=ws), *s4.s4_vocab_loss_fwd(h, w, t)
    assert s4.s4_get_status(ws) == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
