"""Workspaces that the binding allocates belong to the stream that the call runs on: a block of the
current stream's pool may still be in use by what that stream has queued. Which pool is asked is
tested without a GPU; the GPU tests queue such work and run the call beside it."""
import types

import pytest
import torch

from diffusion_drafted_lossless_b200 import _lib
from tests import layers_ref as R

BF, F32 = torch.bfloat16, torch.float32


class _Pools:
    """Stands in for torch.cuda.stream: remembers the stream whose pool allocations come from."""

    def __init__(self, monkeypatch):
        self.active, self.asked = "current", []

        def stream(s):
            pools = self

            class Context:
                def __enter__(self):
                    self.before, pools.active = pools.active, s

                def __exit__(self, *_):
                    pools.active = self.before

            return Context()

        monkeypatch.setattr(torch.cuda, "stream", stream)

    def allocate(self, n):
        self.asked.append(self.active)
        return types.SimpleNamespace(numel=lambda: n, element_size=lambda: 2, record_stream=lambda s: None,
                                     data_ptr=lambda: 0, shape=(n,))


@pytest.mark.parametrize("stream", [None, "side"])
def test_fp8_linear_workspace_is_the_streams_own(monkeypatch, stream):
    pools = _Pools(monkeypatch)
    t = lambda *s: types.SimpleNamespace(shape=torch.Size(s), dtype=BF, get_device=lambda: 0,  # noqa: E731
                                         new_empty=pools.allocate)
    monkeypatch.setattr(_lib, "load", lambda: types.SimpleNamespace(uno_fp8_gated_lora_linear=None))
    monkeypatch.setattr(_lib, "uno_fp8_gated_lora_linear_workspace_size", lambda *a: 512)
    monkeypatch.setattr(_lib, "_lead", lambda name, x, dtypes: (x.shape, 0))
    monkeypatch.setattr(_lib, "_arg", lambda *a: 0)
    monkeypatch.setattr(_lib, "_ptr", lambda x: 0)
    ran = []
    monkeypatch.setattr(_lib, "_call", lambda fn, index, s, *a: ran.append(s))
    _lib.uno_fp8_gated_lora_linear(t(16, 128), t(16, 1), t(256, 128), t(2, 1), t(16, 256), x=t(16, 128),
                                   lora_a=t(8, 128), lora_b=t(256, 8), row_gate=t(16), stream=stream)
    assert pools.asked == ["side" if stream else "current"] and ran == [stream] and pools.active == "current"


@pytest.mark.parametrize("stream", [None, "side"])
@pytest.mark.parametrize("op", ["uno_gated_lora_linear", "uno_block_verify", "uno_tv_loss"])
def test_other_workspaces_are_the_streams_own(monkeypatch, op, stream):
    pools = _Pools(monkeypatch)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: pools.allocate(n))
    monkeypatch.setattr(_lib, "load", lambda: types.SimpleNamespace(**{op: lambda *a: 0}))
    monkeypatch.setattr(_lib, op + "_workspace_size", lambda *a: 512)
    monkeypatch.setattr(_lib, "_ptr", lambda x: None)
    monkeypatch.setattr(_lib, "_stream", lambda s: s)
    t = lambda *s: types.SimpleNamespace(shape=torch.Size(s), dtype=BF, device="cuda:0")  # noqa: E731
    args = {"uno_gated_lora_linear": (t(16, 64), t(64, 64), t(8, 64), t(64, 8), None, 1.0, t(16, 64)),
            "uno_block_verify": (t(2, 4, 100), t(2, 4, 100), 1.0, 5, 0.9, t(2, 4, 3), t(2, 4), t(2)),
            "uno_tv_loss": (t(4, 100), t(4, 100), t(4), t(1))}[op]
    getattr(_lib, op)(*args, stream=stream)
    assert pools.asked == ["side" if stream else "current"] and pools.active == "current"


def _operands(M, d_in, d_out, rank):
    g = torch.Generator().manual_seed(M + d_out)
    o = {"xq": (60 * torch.randn((M, d_in), generator=g)).clamp(-448, 448).to(R.F8),
         "xs": torch.rand((M, -(-d_in // 128)), generator=g) * 0.02,
         "wq": (60 * torch.randn((d_out, d_in), generator=g)).clamp(-448, 448).to(R.F8),
         "ws": torch.rand((-(-d_out // 128), -(-d_in // 128)), generator=g) * 0.02,
         "x": torch.randn((M, d_in), generator=g).to(BF), "a": (0.1 * torch.randn((rank, d_in), generator=g)).to(BF),
         "b": torch.randn((d_out, rank), generator=g).to(BF), "gate": torch.ones(M)}
    return {k: v.cuda() for k, v in o.items()}


def _run(c, y, stream=None):
    return _lib.uno_fp8_gated_lora_linear(c["xq"], c["xs"], c["wq"], c["ws"], y, x=c["x"], lora_a=c["a"],
                                          lora_b=c["b"], row_gate=c["gate"], scale=2.0, stream=stream)


def _busy(a):
    """Some milliseconds of work on the current stream."""
    for _ in range(12):
        a = a @ a
    return a


@pytest.mark.gpu
def test_a_block_the_current_stream_still_uses_is_not_taken():
    """The current stream has work queued that reads a freed block of the workspace's size; a call on
    another stream, which waits for nothing, leaves that block alone."""
    M, d_in, d_out, rank = 512, 256, 512, 64
    c, side = _operands(M, d_in, d_out, rank), torch.cuda.Stream()
    alone = _run(c, torch.empty((M, d_out), dtype=BF, device="cuda"))
    y = torch.zeros_like(alone)
    big = torch.zeros((8192, 8192), dtype=BF, device="cuda")
    n = _lib.uno_fp8_gated_lora_linear_workspace_size(M, d_in, d_out, rank)
    for _ in range(5):
        block = torch.full((n,), 7, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        _busy(big)
        copy = block.clone()
        del block
        _run(c, y, stream=side)
        torch.cuda.synchronize()
        assert (copy == 7).all() and torch.equal(y, alone)


@pytest.mark.gpu
def test_calls_on_two_streams_at_once_without_a_workspace():
    """One call on the current stream behind queued work, one on another stream that waits for
    nothing, with workspaces of one size."""
    M, d_in, d_out, rank = 512, 256, 512, 64
    one, two, side = _operands(M, d_in, d_out, rank), _operands(M, d_in, d_out + 8, rank), torch.cuda.Stream()
    outs = [torch.empty((M, n), dtype=BF, device="cuda") for n in (d_out, d_out + 8)]
    alone = [_run(c, torch.empty_like(y)) for c, y in zip((one, two), outs)]
    big = torch.zeros((4096, 4096), dtype=BF, device="cuda")
    for _ in range(20):
        torch.cuda.synchronize()
        _busy(big)
        _run(one, outs[0])
        _run(two, outs[1], stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))
    assert _lib.uno_read_device_status() == _lib.UNO_OK


@pytest.mark.gpu
@pytest.mark.parametrize("rank", [0, 64])
def test_launches_that_start_early_on_two_streams_at_once(rank):
    """Calls of two and three launches, each started beside the one before it on its stream, on two streams
    with nothing waited for between them: the bits that each has alone."""
    shapes = ((40, 4096, 19200), (642, 4096, 12584), (16, 4096, 4096))
    streams = (torch.cuda.Stream(), torch.cuda.Stream())
    sets = []
    for M, d_in, d_out in shapes:
        c = _operands(M, d_in, d_out, max(rank, 8))
        if not rank:
            c["a"] = c["b"] = c["x"] = c["gate"] = None
        ys = [torch.empty((M, d_out), dtype=BF, device="cuda") for _ in range(3)]
        sets.append((c, _run(c, ys[0]), ys[1:]))
    torch.cuda.synchronize()
    for _ in range(30):
        for i in range(len(sets)):
            for k, st in enumerate(streams):
                c, _, ys = sets[(i + k) % len(sets)]
                _run(c, ys[k], stream=st)
        torch.cuda.synchronize()
        for _, alone, ys in sets:
            assert all(torch.equal(alone, y) for y in ys)
            for y in ys:
                y.zero_()
        torch.cuda.synchronize()
    assert _lib.uno_read_device_status() == _lib.UNO_OK
