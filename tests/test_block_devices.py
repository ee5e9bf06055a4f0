"""Which GPU the selective block's operators run on (no GPU: tensors, streams and the library's calls are
stand-ins).  Every query and launch of a call has the GPU of its activations current, tensors of one call lie on
one GPU, and workspaces are checked like the other arrays."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from structured_state_space_gb300 import block  # noqa: E402

F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


class On(torch.Tensor):
    """A tensor that says it lies on GPU `dev` (-1: none)."""
    @staticmethod
    def __new__(cls, dev, shape, dtype=F32):
        t = torch.Tensor._make_subclass(cls, torch.empty(shape, dtype=dtype))
        t.dev = dev
        return t

    is_cuda = property(lambda self: self.dev >= 0)
    device = property(lambda self: torch.device("cuda", self.dev) if self.dev >= 0 else torch.device("cpu"))

    def get_device(self):
        return self.dev


class Side:
    """A stream of GPU `dev`."""
    def __init__(self, dev):
        self.dev, self.device = dev, torch.device("cuda", dev)


@pytest.fixture()
def gpus(monkeypatch):
    """The current GPU (0 at first) and the library's calls with the GPU that was current in each."""
    class State:
        current, calls = 0, []
    State.calls = []

    @contextlib.contextmanager
    def use(dev):
        before, State.current = State.current, dev
        yield
        State.current = before

    def entry(name):
        return lambda *a: State.calls.append((name, State.current)) or (1024 if name.endswith("bytes") else 0)
    names = ["s4_short_conv_fwd", "s4_short_conv_bwd", "s4_selective_scan_fwd", "s4_selective_scan_bwd", "s4_block_norm_fwd",
             "s4_block_norm_bwd", "s4_short_conv_bwd_workspace_bytes", "s4_selective_scan_workspace_bytes",
             "s4_selective_scan_bwd_workspace_bytes", "s4_block_norm_bwd_workspace_bytes"]
    monkeypatch.setattr(block, "_fn", {n: entry(n) for n in names})
    monkeypatch.setattr(block, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(block, "_current", lambda: State.current, raising=False)
    monkeypatch.setattr(block, "_empty", lambda shape, dtype, device: On(device.index, shape, dtype))
    monkeypatch.setattr(torch.cuda, "device", use)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: use(s.dev))
    return State


def calls_on(dev):
    """Each operator's function and arguments, all of them on GPU `dev`."""
    def t(*shape, dtype=F32):
        return On(dev, shape, dtype)
    conv = dict(x=t(2, 5, 8), w=t(8, 4), bias=t(8), state=t(2, 3, 8))
    scan = dict(x=t(2, 5, 8), dt=t(2, 5, 8), A=t(8, 4), B=t(2, 5, 2, 4), C=t(2, 5, 2, 4), D=t(8), z=t(2, 5, 8), dt_bias=t(8),
                state=t(2, 8, 4))
    norm = dict(o=t(6, 8), gate=t(6, 8), h=t(6, 8), w_post=t(8), scale=t(8), w_pre=t(8))
    ints, ws = dict(lengths=t(2, dtype=I32), index=t(2, dtype=I32)), dict(ws=t(1024, dtype=U8))
    tokens = {k: t(*v.shape[:1], *v.shape[2:]) if k in ("x", "dt", "z", "B", "C") else v for k, v in scan.items()}
    grads = dict(lengths=ints["lengths"])
    return {
        "conv": (block.s4_short_conv_fwd, conv | ints | ws | dict(y=t(2, 5, 8), state_out=t(2, 3, 8))),
        "conv_step": (block.s4_short_conv_step, conv | ws | dict(x=t(2, 8), index=ints["index"], state_out=t(2, 3, 8))),
        "conv_bwd": (block.s4_short_conv_bwd, conv | grads | ws | dict(dy=t(2, 5, 8), dstate=t(2, 3, 8))),
        "scan": (block.s4_selective_scan_fwd, scan | ints | ws | dict(y=t(2, 5, 8), state_out=t(2, 8, 4))),
        "scan_step": (block.s4_selective_step, tokens | ws | dict(index=ints["index"], state_out=t(2, 8, 4))),
        "scan_bwd": (block.s4_selective_scan_bwd, scan | grads | ws | dict(dy=t(2, 5, 8), dstate=t(2, 8, 4))),
        "norm": (block.s4_block_norm_fwd, norm | dict(h_out=t(6, 8), y=t(6, 8))),
        "norm_bwd": (block.s4_block_norm_bwd, norm | ws | dict(dy=t(6, 8), dh_out=t(6, 8))),
    }


OPS = list(calls_on(0))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("given_ws", [True, False])
def test_the_activations_gpu_is_current_in_every_call(gpus, op, given_ws):
    for dev in (0, 1):
        f, kw = calls_on(dev)[op]
        if not given_ws:
            kw.pop("ws", None)
        gpus.calls.clear()
        out = f(**kw)
        assert gpus.calls and all(current == dev for _, current in gpus.calls), gpus.calls
        assert gpus.current == 0
        for v in out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else [out]:
            assert v.get_device() == dev


@pytest.mark.parametrize("op", OPS)
def test_tensors_of_another_gpu_or_none_are_refused(gpus, op):
    f, kw = calls_on(0)[op]
    for k, v in kw.items():
        for dev in (1, -1):
            gpus.calls.clear()
            with pytest.raises(ValueError):
                f(**(kw | {k: On(dev, tuple(v.shape), v.dtype)}))
            assert not any(not n.endswith("bytes") for n, _ in gpus.calls), k


@pytest.mark.parametrize("op", [op for op in OPS if op != "norm"])
def test_workspaces_are_checked(gpus, op):
    f, kw = calls_on(0)[op]
    sent = []
    for n in list(block._fn):
        if not n.endswith("bytes"):
            block._fn[n] = lambda args, stream: sent.append(args) or 0
    for bad, error in ((torch.zeros(1), ValueError), (b"0" * 1024, TypeError), (On(0, (2048,), U8)[::2], ValueError)):
        if isinstance(bad, On):
            bad.dev = 0
        with pytest.raises(error):
            f(**(kw | dict(ws=bad)))
    assert not sent
    f(**kw)
    f(**(kw | dict(ws=On(0, (256,), F32))))  # the size passed on is in bytes
    assert len(sent) == 2 and len(set(map(len, sent))) == 1
    n = (1024).to_bytes(8, "little")
    assert n in sent[0] and n in sent[1]


@pytest.mark.parametrize("op", OPS)
def test_a_stream_of_another_gpu_is_refused(gpus, op):
    f, kw = calls_on(1)[op]
    with pytest.raises(ValueError):
        f(**kw, stream=Side(0))
    assert not gpus.calls and gpus.current == 0
    f(**kw, stream=Side(1))
    assert gpus.calls and all(current == 1 for _, current in gpus.calls) and gpus.current == 0
