"""Linear attention with a decay for each head against the token-by-token definition in float64.

Tolerances, relative in the 2-norm.  An output rounded to bfloat16 or float16 is off by half a step of each element
(2^-8, 2^-11) at most.  With bfloat16 inputs the weights of a chunk, and the state where it is multiplied, are rounded to
bfloat16 before the second product: each of the two parts of a sum is off by up to 2^-8 of it, and as the two
parts are independent so is their sum; with the output's rounding 2 x 2^-8.  With float16 inputs those are sums of two
bfloat16 terms (off by 2^-16 or so), with float32 of three (2^-24).  States are fp32; with bfloat16 and float16
inputs the keys enter them as two bfloat16 terms: 2^-17 of each, within 1e-5."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.sequence_oracle as O  # noqa: E402
import structured_state_space_gb300 as s4  # noqa: E402
from block_util import DTYPES, F32_TOL, TOL, Inputs, close, need_gpu, to64  # noqa: E402

pytestmark = pytest.mark.gpu
OUT = {torch.float32: F32_TOL, torch.bfloat16: 2 * 2.0 ** -8, torch.float16: TOL[torch.float16] + 2.0 ** -15}
# batch, L, H, G, K, V
SIZES = [(1, 2, 1, 1, 1, 1), (1, 63, 2, 1, 16, 16), (2, 64, 2, 2, 64, 64), (1, 65, 3, 3, 40, 72), (2, 200, 4, 2, 128, 128),
         (1, 1030, 2, 1, 48, 80), (3, 300, 2, 2, 33, 7), (1, 600, 1, 1, 64, 256), (1, 100, 2, 1, 256, 64), (1, 130, 1, 1, 256, 256),
         (1, 4099, 2, 2, 64, 128), (2, 33, 8, 1, 128, 64)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def make(seed, batch, L, H, G, K, V, dtype):
    r = Inputs(seed)
    q, k, v = r.normal(batch, L, H, K, dtype=dtype), r.normal(batch, L, G, K, dtype=dtype), r.normal(batch, L, G, V, dtype=dtype)
    g = torch.from_numpy(np.log1p(-np.exp2(-1 - 9 * r.rng.random(H))).astype(np.float32)).cuda()
    return r, q, k, v, g


def wide(*ts):
    return [to64(t) for t in ts]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dt", DTYPES)
def test_prompt(size, dt):
    batch, L, H, G, K, V = size
    r, q, k, v, g = make(1, *size, DTYPES[dt])
    o = s4.s4_linear_attention_fwd(q, k, v, g)
    ref, _ = O.linear_attention(*wide(q, k, v, g), K ** -0.5)
    close(o, ref, "o", OUT[o.dtype])


@pytest.mark.parametrize("size", [(3, 130, 2, 1, 64, 64), (4, 1100, 2, 2, 64, 64), (3, 257, 2, 2, 128, 40), (5, 65, 4, 2, 20, 130)])
@pytest.mark.parametrize("dt", DTYPES)
def test_ragged_with_states_in_slots(size, dt):
    batch, L, H, G, K, V = size
    r, q, k, v, g = make(2, *size, DTYPES[dt])
    lens = ([L, 0, 1, L // 2, L - 1])[:batch]
    index = [batch + 1 - i for i in range(batch)]
    index[-1] = -1
    old = r.normal(batch + 2, H, K, V)
    out = old.clone()
    # padding holds anything, NaN and infinities too
    for b, n in enumerate(lens):
        for t in (q, k, v):
            t[b, n:] = float("nan") if b % 2 else float("inf")
    lt, it = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, index))
    o = s4.s4_linear_attention_fwd(q, k, v, g, scale=0.3, lengths=lt, state=old, state_out=out, index=it)
    real = [0 if i < 0 else n for n, i in zip(lens, index)]
    clean = [torch.nan_to_num(t, 0.0, 0.0, 0.0) for t in (q, k, v)]
    ref, s = O.linear_attention(*wide(*clean, g), 0.3, real, to64(old)[[max(i, 0) for i in index]])
    close(o, ref, "o", OUT[o.dtype])
    want = to64(old)
    for b, i in enumerate(index):
        if i >= 0:
            want[i] = s[b]
    close(out, want, "states", F32_TOL)
    untouched = [i for i in range(batch + 2) if i not in index]
    assert torch.equal(out[untouched], old[untouched])
    # in place gives the same bits
    both = old.clone()
    again = s4.s4_linear_attention_fwd(q, k, v, g, scale=0.3, lengths=lt, state=both, state_out=both, index=it)
    assert torch.equal(again, o) and torch.equal(both, out)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("H,G,K,V", [(2, 2, 64, 64), (4, 1, 16, 48), (3, 3, 7, 5), (16, 4, 128, 128), (1, 1, 256, 256)])
def test_step(dt, H, G, K, V):
    batch = 9
    r, q, k, v, g = make(3, batch, 1, H, G, K, V, DTYPES[dt])
    index = torch.tensor([3, -1, 0, 11, 5, 4, -7, 8, 10], dtype=torch.int32, device="cuda")
    old = r.normal(12, H, K, V)
    at = index.clamp(min=0).tolist()
    live = [int(i >= 0) for i in index.tolist()]
    ref, s = O.linear_attention(*wide(q, k, v, g), K ** -0.5, live, to64(old)[at])
    want = to64(old)
    for b, i in enumerate(index.tolist()):
        if i >= 0:
            want[i] = s[b]
    apart = old.clone()
    o = s4.s4_linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g, old, state_out=apart, index=index)
    close(o, ref[:, 0], "o", TOL[o.dtype])
    close(apart, want, "states apart", F32_TOL)
    o2 = s4.s4_linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g, old, index=index)
    assert torch.equal(o, o2) and torch.equal(old, apart)


@pytest.mark.parametrize("size", SIZES[:1] + SIZES[1:11])
@pytest.mark.parametrize("dt", DTYPES)
def test_gradients(size, dt):
    batch, L, H, G, K, V = size
    if L > 2000:
        L = 1500
    r, q, k, v, g = make(4, batch, L, H, G, K, V, DTYPES[dt])
    do = r.normal(batch, L, H, V, dtype=DTYPES[dt])
    lens = [L, L // 2, 0][:batch]
    for b, n in enumerate(lens):
        for t in (q, k, v, do):
            t[b, n:] = float("nan")
    s0, ds = r.normal(batch, H, K, V), r.normal(batch, H, K, V)
    got = s4.s4_linear_attention_bwd(q, k, v, g, do, lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"), state=s0,
                                     dstate=ds, want_dstate0=True)
    clean = [torch.nan_to_num(t, 0.0) for t in (q, k, v, do)]
    ref = O.linear_attention_grad(*wide(*clean[:3], g, clean[3]), K ** -0.5, lens, to64(s0), to64(ds))
    for n, want in ref.items():
        close(got[n], want, n, F32_TOL if n == "dstate0" else OUT[got[n].dtype])


def test_gradients_against_differences():
    r, q, k, v, g = make(5, 1, 70, 2, 1, 12, 20, torch.float32)
    do = r.normal(1, 70, 2, 20)
    got = s4.s4_linear_attention_bwd(q, k, v, g, do)
    w = wide(q, k, v, g)
    for i, n in enumerate(("dq", "dk", "dv")):
        way = r.rng.standard_normal(w[i].shape)
        f = [np.sum(to64(do) * O.linear_attention(*[x + s * 1e-5 * way if j == i else x for j, x in enumerate(w)], 12 ** -0.5)[0])
             for s in (1, -1)]
        want = (f[0] - f[1]) / 2e-5  # (the loss is linear in each: rounding alone, some 1e-10)
        have = np.sum(to64(got[n]) * way)
        assert abs(have - want) <= 1e-5 * np.linalg.norm(to64(got[n])) * np.linalg.norm(way), n


@pytest.mark.parametrize("dt", DTYPES)
def test_slices_of_a_projection(dt):
    H, G, K, V, L = 4, 2, 64, 32, 150
    r = Inputs(6)
    g = torch.full((H,), -0.05, device="cuda")
    for left in (0, 3):  # aligned rows, and rows that are not
        wide_ = r.normal(2, L, left + H * K + G * (K + V), dtype=DTYPES[dt])
        q, k, v = wide_[..., left:].split([H * K, G * K, G * V], -1)
        q, k, v = q.unflatten(-1, (H, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (G, V))
        got = s4.s4_linear_attention_fwd(q, k, v, g)
        # rows that are not aligned to 16 bytes may go through another kernel: both are off from the definition by OUT at
        # most, so from each other by twice that
        far = 2 * OUT[got.dtype] if left else 0.0
        close(got, to64(s4.s4_linear_attention_fwd(q.contiguous(), k.contiguous(), v.contiguous(), g)), "rows apart", far)
        # heads outermost
        t = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v)]
        close(got, to64(s4.s4_linear_attention_fwd(*t, g)), "heads outermost", far)
        # a broadcast key
        one = k[:, :, :1].expand(-1, -1, G, -1)
        assert torch.equal(s4.s4_linear_attention_fwd(q, one, v, g), s4.s4_linear_attention_fwd(q, one.contiguous(), v, g))


def test_decays_of_one_and_none():
    r, q, k, v, _ = make(7, 1, 300, 2, 2, 32, 32, torch.float32)
    g = torch.tensor([0.0, float("-inf")], device="cuda")
    o = s4.s4_linear_attention_fwd(q, k, v, g)
    ref, _ = O.linear_attention(*wide(q, k, v), np.array([0.0, -1e30]), 32 ** -0.5)
    close(o, ref, "o")
    got = s4.s4_linear_attention_bwd(q, k, v, g, v)
    for n, want in O.linear_attention_grad(*wide(q, k, v), np.array([0.0, -1e30]), to64(v), 32 ** -0.5).items():
        if n in got:
            close(got[n], want, n)


def test_prompts_go_on_as_tokens():
    size = (2, 100, 4, 2, 64, 64)
    r, q, k, v, g = make(8, *size, torch.bfloat16)
    lens = torch.tensor([60, 99], dtype=torch.int32, device="cuda")
    cache = torch.zeros(2, 4, 64, 64, device="cuda")
    s4.s4_linear_attention_fwd(q, k, v, g, lengths=lens, state_out=cache)
    rows = torch.arange(2, device="cuda")
    at = lens.long()
    o = s4.s4_linear_attention_step(q[rows, at], k[rows, at], v[rows, at], g, cache)
    ref, s = O.linear_attention(*wide(q, k, v, g), 64 ** -0.5, (lens + 1).tolist())
    close(o, ref[[0, 1], [60, 99]], "o", TOL[o.dtype])
    close(cache, s, "states")


def test_a_length_or_slot_out_of_range():
    r, q, k, v, g = make(9, 3, 40, 2, 2, 16, 16, torch.float32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    cache = r.normal(3, 2, 16, 16)
    keep = cache.clone()
    o = s4.s4_linear_attention_fwd(q, k, v, g, lengths=torch.tensor([40, 41, -1], dtype=torch.int32, device="cuda"),
                                   state=cache, state_out=cache, ws=ws)
    assert s4.STATUS[s4.s4_get_status(ws)] == "S4_ERR_INVALID_INDEX"
    assert not o[1:].any() and o[0].any() and torch.equal(cache[1:], keep[1:])
    s4.s4_linear_attention_fwd(q, k, v, g, ws=ws)
    assert s4.s4_get_status(ws) == 0
    o = s4.s4_linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g, cache, index=torch.tensor([0, 3, 1], dtype=torch.int32, device="cuda"),
                                    ws=ws)
    assert s4.STATUS[s4.s4_get_status(ws)] == "S4_ERR_INVALID_INDEX"
    assert not o[1].any() and o[0].any() and o[2].any()


def test_long_sums_in_float32():
    """A long sequence of slow decay: the state of 40000 tokens, and their gradients, against float64 sums on the GPU."""
    L, K, V = 40000, 100, 34
    r, q, k, v, g = make(10, 1, L, 1, 1, K, V, torch.float32)
    g = torch.tensor([-1e-4], device="cuda")
    do, out = r.normal(1, L, 1, V), torch.zeros(1, 1, K, V, device="cuda")
    o = s4.s4_linear_attention_fwd(q, k, v, g, state_out=out)
    got = s4.s4_linear_attention_bwd(q, k, v, g, do)
    q, k, v, do = (t[0, :, 0].double() for t in (q, k, v, do))
    i = torch.arange(L, device="cuda")
    g64 = g.double().item()
    close(out[0, 0], to64((k * torch.exp(g64 * (L - 1 - i))[:, None]).t() @ v), "state")
    # (blocks of rows of the whole matrix of weights)
    want = {n: torch.zeros_like(t) for n, t in (("dq", q), ("dk", k), ("dv", v), ("o", v))}
    for a in range(0, L, 4000):
        rows = slice(a, a + 4000)
        lag = i[rows, None] - i
        w = torch.where(lag >= 0, torch.exp(g64 * lag.clamp(min=0)), 0.0) * K ** -0.5
        want["o"][rows] = ((q[rows] @ k.t()) * w) @ v
        want["dq"][rows] = ((do[rows] @ v.t()) * w) @ k
        want["dk"] += ((do[rows] @ v.t()) * w).t() @ q[rows]
        want["dv"] += ((q[rows] @ k.t()) * w).t() @ do[rows]
    close(o[0, :, 0], to64(want["o"]), "o")
    for n in ("dq", "dk", "dv"):
        close(got[n][0, :, 0], to64(want[n]), n)
