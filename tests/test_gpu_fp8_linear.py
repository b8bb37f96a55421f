"""uno_fp8_gated_lora_linear against its plain 64-bit form, within the bound that
tests/layers_ref.py derives; gates, ragged sizes, untouched rows, streams and graphs."""
import math

import pytest
import torch

from diffusion_drafted_lossless_b200 import _lib
from tests import layers_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _operands(M, d_in, d_out, rank, seed=0):
    """Seeded operands on the CPU: e4m3 values over the whole range, scales of mixed sizes."""
    g = torch.Generator().manual_seed(seed + M + 7 * d_in + 13 * d_out)
    o = {"xq": (torch.randn((M, d_in), generator=g) * 60).clamp(-448, 448).to(R.F8),
         "xs": torch.rand((M, -(-d_in // 128)), generator=g) * 0.02 + 1e-3,
         "wq": (torch.randn((d_out, d_in), generator=g) * 60).clamp(-448, 448).to(R.F8),
         "ws": torch.rand((-(-d_out // 128), -(-d_in // 128)), generator=g) * 0.02 + 1e-3}
    if rank:
        o["x"] = torch.randn((M, d_in), generator=g).to(BF)
        o["a"] = (torch.randn((rank, d_in), generator=g) * 0.1).to(BF)
        o["b"] = torch.randn((d_out, rank), generator=g).to(BF)
        o["gate"] = (torch.arange(M) % 4 != 0).float() * (0.5 + torch.rand(M, generator=g))
    return o


def _cuda(o):
    return {k: v.cuda() for k, v in o.items()}


def _run(c, y, scale=2.0, **kw):
    _lib.uno_fp8_gated_lora_linear(c["xq"], c["xs"], c["wq"], c["ws"], y, x=c.get("x"), lora_a=c.get("a"),
                                   lora_b=c.get("b"), row_gate=c.get("gate"), scale=scale, **kw)
    return y


def _check(o, y, scale=2.0):
    rank = o["a"].shape[0] if "a" in o else 0
    ref, size, low, tb = R.linear(o["xq"], o["xs"], o["wq"], o["ws"], o.get("x"), o.get("a"), o.get("b"),
                                  o.get("gate"), scale)
    bound = R.linear_bound(size, low, tb, ref, o["xq"].shape[1], rank, y.dtype == BF)
    err = (y.cpu().double() - ref).abs()
    assert torch.isfinite(y).all()
    assert (err <= bound).all(), (float((err / bound).max()), int((err > bound).sum()))


@pytest.mark.parametrize("M,d_in,d_out,rank,dtype", [
    (1, 16, 1, 0, F32), (1, 128, 128, 0, BF), (1, 4096, 1024, 128, BF), (3, 144, 130, 0, F32), (7, 272, 257, 0, BF),
    (16, 4096, 640, 64, BF), (16, 2560, 4096, 0, F32), (33, 1040, 200, 8, BF), (64, 512, 5000, 0, BF),
    (127, 640, 384, 16, BF), (128, 128, 128, 8, BF), (129, 2576, 1001, 0, F32), (257, 1024, 384, 128, BF),
    (300, 9728, 264, 200, BF), (1024, 512, 1536, 256, BF), (2, 65536, 72, 0, F32), (513, 400, 2056, 24, BF),
    (1000, 4096, 136, 0, BF), (40, 128, 20000, 0, F32), (256, 256, 4096, 128, BF), (260, 2560, 9728, 64, BF),
])
def test_linear(M, d_in, d_out, rank, dtype):
    o = _operands(M, d_in, d_out, rank)
    y = torch.full((M, d_out), math.nan, dtype=dtype, device="cuda")
    _check(o, _run(_cuda(o), y))


def test_large_products_on_sampled_rows():
    """The draft step's widest projection and a long prompt: every tile form that large sizes
    select, checked on spread rows (all columns)."""
    for M, d_in, d_out, rank in ((1024, 4096, 12288, 128), (4096, 2560, 9728, 0), (1100, 2560, 9728, 64)):
        o = _operands(M, d_in, d_out, rank)
        y = _run(_cuda(o), torch.full((M, d_out), math.nan, dtype=BF, device="cuda"))
        assert torch.isfinite(y).all()
        rows = torch.unique(torch.cat([torch.arange(0, M, max(1, M // 61)), torch.tensor([1, 127, 128, 255, M - 1])]))
        part = {k: (v if k in ("wq", "ws", "a", "b") else v[rows]) for k, v in o.items()}
        _check(part, y[rows.cuda()])


@pytest.mark.parametrize("M,d_in,d_out,rank,dtype", [
    (9, 640, 40001, 0, BF), (16, 1152, 39000, 0, F32), (24, 512, 40000, 64, BF), (33, 384, 39168, 16, BF),
    (64, 768, 38400, 0, BF), (31, 256, 300, 8, BF), (32, 2048, 129, 0, F32), (17, 4096, 2056, 200, BF),
    (8, 16, 128, 0, F32), (25, 144, 64, 0, BF),
])
def test_few_rows_and_last_turns(M, d_in, d_out, rank, dtype):
    """Calls of at most 64 rows, and widths of more than two tiles of 128 columns an SM, a few
    over: the last turn of the persistent CTAs is mostly empty."""
    o = _operands(M, d_in, d_out, rank)
    y = torch.full((M, d_out), math.nan, dtype=dtype, device="cuda")
    _check(o, _run(_cuda(o), y))


def test_rows_without_gate_are_the_base_product():
    o = _operands(70, 512, 384, 32)
    c = _cuda(o)
    base = {k: c[k] for k in ("xq", "xs", "wq", "ws")}
    y0 = _run(base, torch.empty((70, 384), dtype=BF, device="cuda"))
    y = _run(c, torch.empty((70, 384), dtype=BF, device="cuda"))
    off = o["gate"] == 0
    assert off.any() and torch.equal(y[off.cuda()], y0[off.cuda()])
    assert (y[~off.cuda()] != y0[~off.cuda()]).any()
    # no gate at all, and a scale of 0: the base everywhere, whatever the adapter reads
    c["x"] = c["x"].clone()
    c["x"][:] = math.inf
    for kw in ({"gate": None}, {"scale": 0.0}):
        y1 = _run({**c, **({"gate": None} if "gate" in kw else {})}, torch.empty_like(y), scale=kw.get("scale", 2.0))
        assert torch.equal(y1, y0)


def test_nan_and_inf_stay_in_their_rows():
    o = _operands(130, 256, 256, 0)
    c = _cuda(o)
    y0 = _run(c, torch.empty((130, 256), dtype=BF, device="cuda")).clone()
    c["xq"].view(torch.uint8)[5, 9] = 0x7F    # an e4m3 NaN
    c["xs"][129, 1] = math.inf
    y = _run(c, torch.empty((130, 256), dtype=BF, device="cuda"))
    keep = torch.ones(130, dtype=torch.bool, device="cuda")
    keep[5] = keep[129] = False
    assert torch.equal(y[keep], y0[keep]) and torch.isnan(y[5]).all() and not torch.isfinite(y[129]).any()


def test_rows_behind_the_last_and_columns_stay():
    """Only [M, d_out] is written, also where d_out is odd and M ends inside a tile."""
    o = _operands(5, 256, 77, 0)
    c = _cuda(o)
    big = torch.full((9, 77), 3.0, dtype=BF, device="cuda")
    _run(c, big[:5])
    assert (big[5:] == 3).all()
    _check(o, big[:5])
    _lib.uno_fp8_gated_lora_linear(c["xq"][:0], c["xs"][:0], c["wq"], c["ws"], big[:0])
    assert (big[5:] == 3).all()


def test_two_streams_dirty_workspaces_and_graphs():
    shapes = ((40, 1024, 512, 64), (300, 512, 1032, 128))
    sets = []
    for sh in shapes:
        o = _operands(*sh)
        c = _cuda(o)
        ws = torch.full((_lib.uno_fp8_gated_lora_linear_workspace_size(*sh),), 255, dtype=torch.uint8, device="cuda")
        sets.append((o, c, ws, torch.empty((sh[0], sh[2]), dtype=BF, device="cuda")))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for st, (_, c, ws, y) in zip(streams, sets):
            _run(c, y, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for o, _, _, y in sets:
        _check(o, y)
    # without a workspace of their own the calls on another stream keep theirs until it is done
    for st, (_, c, _, y) in zip(streams, sets):
        y.zero_()
        st.wait_stream(torch.cuda.current_stream())
        _run(c, y, stream=st)
    torch.cuda.synchronize()
    for o, _, _, y in sets:
        _check(o, y)
    # two captured graphs that share a workspace, replayed in turn on changed inputs
    o, c, ws, y = sets[0]
    graphs, ys = [], [torch.empty_like(y), torch.empty_like(y)]
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _run(c, ys[k], workspace=ws)
        graphs.append(g)
    for seed in (1, 2):
        o = _operands(*shapes[0], seed=seed)
        for k, v in o.items():
            c[k].copy_(v.cuda())
        for k in range(2):
            ys[k].zero_()
            graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            _check(o, ys[k])


@pytest.mark.parametrize("M,d_in,d_out,rank", [(24, 512, 4000, 64), (16, 4096, 4096, 128), (40, 1024, 20000, 64),
                                               (200, 512, 9728, 64), (700, 1024, 9728, 128)])
def test_the_adapter_reads_what_this_call_made(M, d_in, d_out, rank):
    """The projection reads the T that its own call made: with the workspace overwritten between
    calls, every call gives the first one's bits."""
    c = _cuda(_operands(M, d_in, d_out, rank))
    ws = torch.empty(_lib.uno_fp8_gated_lora_linear_workspace_size(M, d_in, d_out, rank), dtype=torch.uint8,
                     device="cuda")
    first = _run(c, torch.empty((M, d_out), dtype=BF, device="cuda"), workspace=ws)
    y = torch.empty_like(first)
    for _ in range(60):
        ws.fill_(0x45)
        assert torch.equal(_run(c, y, workspace=ws), first)


@pytest.mark.parametrize("M,d_in,d_out,rank,dtype", [(16, 4096, 19067, 0, F32), (40, 4112, 19200, 64, BF),
                                                     (1, 4096, 37900, 0, BF), (200, 4096, 19184, 8, BF),
                                                     (642, 4096, 12584, 16, BF), (514, 4096, 15139, 0, F32)])
def test_last_columns_in_a_launch_of_their_own(M, d_in, d_out, rank, dtype):
    """Tiles for a few turns of the SMs and a little more: every element is written, by the launch of
    the last columns or the one beside it, and nothing on the stream runs before both have ended."""
    o = _operands(M, d_in, d_out, rank)
    c = _cuda(o)
    y = torch.full((M, d_out), math.nan, dtype=dtype, device="cuda")
    first = _run(c, y).clone()
    assert torch.isfinite(first).all()
    rows = torch.unique(torch.cat([torch.arange(min(M, 8)), torch.arange(max(0, M - 8), M)]))
    _check({k: (v[rows] if k in ("xq", "xs", "x", "gate") else v) for k, v in o.items()}, first[rows.cuda()])
    for _ in range(20):
        y.fill_(math.nan)
        assert torch.equal(_run(c, y), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y.fill_(math.nan)
        _run(c, y)
        copy = y.clone()
    for _ in range(5):
        graph.replay()
        assert torch.equal(copy, first)
    assert _lib.uno_read_device_status() == _lib.UNO_OK


@pytest.mark.parametrize("M,d_in,d_out,rank", [(210, 1632, 4448, 64), (4696, 1200, 432, 128), (7877, 1056, 1472, 8),
                                               (195, 816, 584, 8)])
def test_call_after_call(M, d_in, d_out, rank):
    """Hundreds of calls on an idle GPU, each with the sums of its few K blocks joined by clusters or
    its last row tile partly empty: the first one's bits every time, and no wait gives up."""
    o = _operands(M, d_in, d_out, rank)
    c = _cuda(o)
    first = _run(c, torch.empty((M, d_out), dtype=BF, device="cuda"))
    y = torch.empty_like(first)
    for _ in range(400):
        torch.cuda.synchronize()
        assert torch.equal(_run(c, y), first)
    assert _lib.uno_read_device_status() == _lib.UNO_OK
    rows = torch.cat([torch.arange(8), torch.arange(M - 8, M)])
    _check({k: (v[rows] if k in ("xq", "xs", "x", "gate") else v) for k, v in o.items()}, first[rows.cuda()])


def test_same_bits_every_time():
    o = _cuda(_operands(16, 4096, 1024, 128))
    y = [_run(o, torch.empty((16, 1024), dtype=BF, device="cuda")) for _ in range(5)]
    assert all(torch.equal(y[0], v) for v in y[1:])


def test_offsets_past_32_bits():
    """An output of more than 2^31 elements: its last rows and columns are where they belong."""
    M, d_in, d_out = 16400, 16, 131080
    o = _operands(M, d_in, 256, 0)
    c = _cuda(o)
    c["wq"] = c["wq"].view(torch.uint8).repeat(513, 1)[:d_out].view(R.F8)
    c["ws"] = c["ws"].repeat(513, 1)[: -(-d_out // 128)].contiguous()
    y = _run(c, torch.empty((M, d_out), dtype=BF, device="cuda"))
    small = _run({**c, "wq": c["wq"][:256].contiguous(), "ws": c["ws"][:2].contiguous()},
                 torch.empty((M, 256), dtype=BF, device="cuda"))
    for lo in (0, 256, 131072 - 256):
        assert torch.equal(y[:, lo:lo + 256], small)
    assert torch.equal(y[:, 131072:], small[:, :8])
    _check({k: (v[-4:] if k in ("xq", "xs") else v) for k, v in o.items()}, small[-4:])


def test_binding_refuses_wrong_operands():
    c = _cuda(_operands(16, 256, 256, 8))
    y = torch.empty((16, 256), dtype=BF, device="cuda")
    for k, bad in (("xs", c["xs"][:, :1].contiguous()), ("ws", c["ws"][:1].contiguous()),
                   ("x", c["x"].float()), ("b", c["b"][:128].contiguous()), ("gate", c["gate"][:8])):
        with pytest.raises(ValueError):
            _run({**c, k: bad}, y)
    with pytest.raises(TypeError):
        _run({**c, "xq": c["xq"].view(torch.uint8)}, y)
    with pytest.raises(_lib.UnoError, match="float32 output"):
        _run(c, torch.empty((16, 256), device="cuda"))
    with pytest.raises(_lib.UnoError, match="workspace"):
        _run(c, y, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert _lib.uno_read_device_status() == _lib.UNO_OK
