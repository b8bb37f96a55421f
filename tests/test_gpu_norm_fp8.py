"""uno_rms_norm_fp8 and uno_fp8_quantize against their plain 64-bit forms: e4m3 values equal
(ties included), scales and the unquantised output within the roundings counted below."""
import math

import pytest
import torch

from diffusion_drafted_lossless_b200 import _lib
from tests import layers_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def _x(M, d, dtype, seed, wide=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, d), generator=g)
    if wide and d > 3:
        x[:, 3] *= 40.0
    return x.to(dtype)


def _norm(x, w, res=None, y=True, q=True, inplace=False, eps=EPS):
    M, d = x.shape
    xd, wd = x.cuda(), w.cuda()
    rd = None if res is None else res.cuda()
    oq = torch.full((M, d), 1.5, device="cuda").to(R.F8) if q else None
    os = torch.full((M, -(-d // 128)), -1.0, device="cuda") if q else None
    ores = None if rd is None else (rd if inplace else torch.empty_like(rd))
    oy = torch.empty_like(xd) if y else None
    _lib.uno_rms_norm_fp8(xd, wd, eps, oq, os, residual=rd, out_residual=ores, out_y=oy)
    torch.cuda.synchronize()
    c = lambda t: None if t is None else t.cpu()  # noqa: E731
    return c(oq), c(os), c(ores), c(oy)


def _same(q, ref):
    """Equal e4m3 values (NaN in the same places)."""
    q = q.double()
    assert torch.equal(torch.isnan(q), torch.isnan(ref))
    assert torch.equal(q.nan_to_num(0.0), ref.nan_to_num(0.0))


def _stat_bound(d, dtype):
    """Relative error of rstd (and then of a scale or y). The sum of squares: one rounding of
    each square's multiply-add, at most d / 512 + 8 of them in a thread, then 10 across it; a
    square root halves it; 4 roundings for the mean, eps, the root and its inverse; 2 for the
    product and the quotient."""
    return ((d / 512 + 18) / 2 + 6) * R.F32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,d,res", [(1, 16, True), (3, 128, False), (5, 144, True), (2, 4096, True), (7, 2576, False),
                                     (300, 2560, True), (2, 5120, True), (2, 32768, True), (1, 12304, True)])
def test_norm(M, d, res, dtype):
    x, w = _x(M, d, dtype, d), (1 + 0.2 * _x(1, d, F32, 1, False)[0]).to(dtype)
    r = _x(M, d, dtype, 2) if res else None
    h, y, q, s = R.rms_norm(x, w, EPS, r)
    gq, gs, gres, gy = _norm(x, w, r)
    if res:
        assert torch.equal(gres, h)
    _same(gq, q)
    tol = _stat_bound(d, dtype)
    assert ((gs.double() - s).abs() <= tol * s).all()
    half = R.HALF_BF16 if dtype == BF else R.F32
    assert ((gy.double() - y).abs() <= (half + tol) * y.abs() * 1.01).all()


@pytest.mark.parametrize("q,y", [(True, False), (False, True)])
def test_norm_one_output_and_in_place_residual(q, y):
    x, r, w = _x(9, 272, BF, 1), _x(9, 272, BF, 2), _x(1, 272, BF, 3)[0]
    full = _norm(x, w, r)
    part = _norm(x, w, r, q=q, y=y, inplace=True)
    for a, b in zip(full, part):
        assert b is None or torch.equal(a.float(), b.float())


def test_norm_zero_rows_and_smallest_scales():
    """A row of zeros, a block of zeros, and rows so small that their scales sit at 2^-126."""
    x = torch.zeros((4, 256))
    x[1, 128:] = _x(1, 128, F32, 5)[0]
    x[2] = 1e-38 * _x(1, 256, F32, 6, False)[0]
    x[3] = 2.0 ** -120
    w = torch.ones(256)
    for dtype in (F32, BF):
        for eps in (1e-6, 1.0):
            xd, wd = x.to(dtype), w.to(dtype)
            _, y, q, s = R.rms_norm(xd, wd, eps)
            gq, gs, _, gy = _norm(xd, wd, eps=eps)
            tol = _stat_bound(256, dtype)
            # where the smallest scale is used the row's factor is in the values: a border may
            # be met from either side
            small = s <= R.MIN_SCALE * (1 + 1e-6)
            wide = small.repeat_interleave(128, 1)
            assert torch.equal(gq.double()[~wide], q[~wide])
            assert ((gq.double() - q).abs()[wide] <= 0.126 * q.abs()[wide] + 2.0 ** -9).all()
            assert ((gs.double() - s).abs() <= tol * s).all()
            assert (gq.double()[0] == 0).all() and (gs[0] == R.MIN_SCALE).all()
            assert (gy[0] == 0).all()


def test_norm_nan_and_inf_stay_in_their_row():
    x, w = _x(5, 384, BF, 8), torch.ones(384, dtype=BF)
    clean = _norm(x, w)
    x[1, 7], x[3, 200] = math.nan, math.inf
    gq, gs, _, gy = _norm(x, w)
    for row in (0, 2, 4):
        assert torch.equal(gq[row].float(), clean[0][row].float()) and torch.equal(gs[row], clean[1][row])
        assert torch.equal(gy[row], clean[3][row])
    assert torch.isnan(gs[1]).all() and torch.isnan(gy[1]).all()
    assert torch.isnan((gq[3].float() * gs[3].repeat_interleave(128))[200])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,d", [(1, 16), (1, 128), (127, 144), (128, 256), (129, 4112), (300, 2576), (2049, 48)])
def test_quantize(M, d, block_rows, dtype):
    x = _x(M, d, dtype, M + d)
    if M > 2:
        x[2] = 0
        x[1, : min(128, d)] *= 1e-30
    q, s = R.quantize(x.double(), block_rows)
    oq = torch.full((M, d), 1.5, device="cuda").to(R.F8)
    os = torch.full(s.shape, -1.0, device="cuda")
    _lib.uno_fp8_quantize(x.cuda(), oq, os, block_rows)
    _same(oq.cpu(), q)
    assert torch.equal(os.cpu(), s.float())  # a float32 quotient, rounded once


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_ties_and_extremes(dtype):
    """Every border between e4m3 values (in a block whose largest size is 448, and scaled by
    powers of two), float32's neighbours of each, the smallest and largest blocks."""
    mid = (R.CODES[1:] + R.CODES[:-1]) / 2
    rows = []
    for f in (1.0, 2.0 ** -20, 2.0 ** 30, 2.0 ** -100, 2.0 ** 100, 2.0 ** -130):
        rows.append(torch.cat([mid, torch.tensor([448.0, -448.0], dtype=torch.float64)]) * f)
    x = torch.stack(rows).float()
    if dtype == F32:
        x = torch.cat([x, torch.nextafter(x, torch.zeros_like(x)), torch.nextafter(x, x * 2)])
        x[:, 127] = x[:, 127].sign() * x.abs().amax(1)
    x = torch.cat([x, torch.full((1, 128), torch.finfo(dtype).max), torch.full((1, 128), torch.finfo(dtype).tiny)])
    x = x.to(dtype)
    q, s = R.quantize(x.double(), 1)
    oq, os = torch.empty(x.shape, dtype=R.F8, device="cuda"), torch.empty(s.shape, device="cuda")
    _lib.uno_fp8_quantize(x.cuda(), oq, os)
    _same(oq.cpu(), q)
    assert torch.equal(os.cpu(), s.float())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_nan_and_inf(block_rows):
    x = _x(256, 256, BF, 3)
    x[5, 7], x[200, 130] = math.nan, math.inf
    oq = torch.empty((256, 256), dtype=R.F8, device="cuda")
    os = torch.empty((256 if block_rows == 1 else 2, 2), device="cuda")
    _lib.uno_fp8_quantize(x.cuda(), oq, os, block_rows)
    v = oq.cpu().double() * R.expand_scales(os.cpu(), block_rows, 256, 256)
    assert math.isnan(v[5, 7]) and torch.isnan(v[200, 130])
    bad = torch.zeros(256, 256, dtype=torch.bool)
    bad[5, 7] = True
    bad[200 if block_rows == 1 else slice(128, 256), 128:] = True
    assert torch.isfinite(v[~bad]).all()
    q, s = R.quantize(x.double(), block_rows)
    assert torch.equal(oq.cpu().double()[~bad], q[~bad])


def test_rows_behind_the_last_are_left():
    big_q = torch.full((8, 256), 2.0, device="cuda").to(R.F8)
    big_s = torch.full((8, 2), 7.0, device="cuda")
    x = _x(5, 256, BF, 4).cuda()
    _lib.uno_rms_norm_fp8(x, torch.ones(256, dtype=BF, device="cuda"), EPS, big_q[:5], big_s[:5])
    assert (big_q[5:].float() == 2).all() and (big_s[5:] == 7).all()
    _lib.uno_fp8_quantize(x, big_q[:5], big_s[:5])
    assert (big_q[5:].float() == 2).all() and (big_s[5:] == 7).all()
    e = torch.empty((0, 256), dtype=BF, device="cuda")
    _lib.uno_fp8_quantize(e, big_q[:0], big_s[:0])
    _lib.uno_rms_norm_fp8(e, torch.ones(256, dtype=BF, device="cuda"), EPS, big_q[:0], big_s[:0])


def test_other_stream_and_graph_replay():
    w = torch.ones(512, dtype=BF, device="cuda")
    x = _x(40, 512, BF, 9).cuda()
    q, s = torch.empty((40, 512), dtype=R.F8, device="cuda"), torch.empty((40, 4), device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    _lib.uno_rms_norm_fp8(x, w, EPS, q, s, stream=st)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    with torch.cuda.graph(g):
        _lib.uno_rms_norm_fp8(x, w, EPS, q2, s2)
    g.replay()
    assert torch.equal(q.float(), q2.float()) and torch.equal(s, s2)
    x.copy_(_x(40, 512, BF, 10).cuda())
    g.replay()
    _lib.uno_rms_norm_fp8(x, w, EPS, q, s)
    assert torch.equal(q.float(), q2.float()) and torch.equal(s, s2)


def test_binding_refuses_wrong_shapes():
    x = _x(4, 256, BF, 1).cuda()
    w, q, s = torch.ones(256, dtype=BF, device="cuda"), torch.empty((4, 256), dtype=R.F8, device="cuda"), \
        torch.empty((4, 2), device="cuda")
    with pytest.raises(ValueError, match="weight"):
        _lib.uno_rms_norm_fp8(x, w[:128], EPS, q, s)
    with pytest.raises(ValueError, match="out_scale"):
        _lib.uno_rms_norm_fp8(x, w, EPS, q, s[:, :1].contiguous())
    with pytest.raises(ValueError, match="out_q"):
        _lib.uno_fp8_quantize(x, q.view(torch.uint8), s)
    with pytest.raises(TypeError):
        _lib.uno_fp8_quantize(x.half(), q, s)
    with pytest.raises(ValueError, match="contiguous"):
        _lib.uno_fp8_quantize(x.t(), q, s)
    with pytest.raises(_lib.UnoError, match="out_q or out_y"):
        _lib.uno_rms_norm_fp8(x, w, EPS)
