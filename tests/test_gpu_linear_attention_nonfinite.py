"""What an infinite or NaN value of a real token reaches in linear attention: the outputs that the token-by-token definition
makes infinite or NaN, and no others: tokens before it stay as they are (their tolerances are those of finite inputs)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.sequence_oracle as O  # noqa: E402
import structured_state_space_gb300 as s4  # noqa: E402
from block_util import DTYPES, Inputs, need_gpu, to64  # noqa: E402
from test_gpu_linear_attention import OUT  # noqa: E402

pytestmark = pytest.mark.gpu
# batch, L, H, G, K, V: one chunk and several, several segments, widths of each kernel
SIZES = [(1, 128, 2, 1, 64, 64), (2, 300, 2, 2, 128, 128), (1, 1500, 2, 2, 64, 128), (1, 200, 2, 1, 128, 40), (1, 140, 1, 1, 256, 70),
         (1, 70, 2, 1, 33, 7)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def same(got, ref, name):
    """The finite ones are those of the reference, and as near to it as finite inputs' are."""
    g, fine = to64(got), np.isfinite(ref)
    assert np.array_equal(np.isfinite(g), fine), (name, np.argwhere(np.isfinite(g) != fine)[:4])
    off, size = np.linalg.norm(g[fine] - ref[fine]), np.linalg.norm(ref[fine])
    assert off <= OUT[got.dtype] * size + 2.0 ** -25 * np.sqrt(ref.size) * (got.dtype == torch.float16), (name, off / size)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("which,value", [("v", float("nan")), ("v", float("inf")), ("k", float("nan")), ("q", float("inf")),
                                         ("do", float("nan"))])
def test_reaches_no_other_token(size, dt, which, value):
    batch, L, H, G, K, V = size
    r, dtype = Inputs(1), DTYPES[dt]
    x = {"q": r.normal(batch, L, H, K, dtype=dtype), "k": r.normal(batch, L, G, K, dtype=dtype),
         "v": r.normal(batch, L, G, V, dtype=dtype), "do": r.normal(batch, L, H, V, dtype=dtype)}
    g = torch.tensor([-0.02, -0.3], device="cuda")[:H]
    lens = [L - 9, L][:batch]
    # one channel of two tokens (the second in another head), and one of the first token of the last chunk
    for t, head, c in ((L // 2, 0, 3), (L // 2 + 5, -1, 5), ((L - 10) // 128 * 128, 0, 1)):
        x[which][0, t, head, c] = value
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    with np.errstate(invalid="ignore", over="ignore"):
        w = [to64(x[i]) for i in ("q", "k", "v")] + [to64(g)]
        o, _ = O.linear_attention(*w, K ** -0.5, lens)
        ref = O.linear_attention_grad(*w, to64(x["do"]), K ** -0.5, lens)
    if which != "do":
        same(s4.s4_linear_attention_fwd(x["q"], x["k"], x["v"], g, lengths=n), o, "o")
    got = s4.s4_linear_attention_bwd(x["q"], x["k"], x["v"], g, x["do"], lengths=n)
    for name in ("dq", "dk", "dv"):
        same(got[name], ref[name], name)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("where", ["v", "state"])
def test_states_on_return(size, dt, where):
    """The state after an infinity, in place and apart, and after one on entry."""
    batch, L, H, G, K, V = size
    r, dtype = Inputs(2), DTYPES[dt]
    q, k, v = r.normal(batch, L, H, K, dtype=dtype), r.normal(batch, L, G, K, dtype=dtype), r.normal(batch, L, G, V, dtype=dtype)
    g = torch.tensor([-0.02, -0.3], device="cuda")[:H]
    old = r.normal(batch, H, K, V)
    if where == "v":
        v[0, L // 3, 0, 2] = float("inf")
        v[-1, L - 1, -1, 4] = float("nan")
    else:
        old[0, 0, 1, 3], old[-1, -1, 2, 1] = float("nan"), float("inf")
    with np.errstate(invalid="ignore"):
        ref, s = O.linear_attention(to64(q), to64(k), to64(v), to64(g), K ** -0.5, None, to64(old))
    apart, both = torch.empty_like(old), old.clone()
    o = s4.s4_linear_attention_fwd(q, k, v, g, state=old, state_out=apart)
    same(o, ref, "o")
    same(apart, s, "state")
    again = s4.s4_linear_attention_fwd(q, k, v, g, state=both, state_out=both)
    assert torch.equal(torch.nan_to_num(again), torch.nan_to_num(o)) and torch.equal(torch.nan_to_num(both), torch.nan_to_num(apart))
