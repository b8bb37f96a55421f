"""The operators of include/uno_layers.h at the far ends of the sizes they state, a few GB each:
many rows, wide outputs, long rows, and the adapter's product when it takes several turns itself."""
import math

import pytest
import torch

from diffusion_drafted_lossless_b200 import _lib
from tests import layers_ref as R
from tests.test_gpu_fp8_linear import _check, _cuda, _operands, _run

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _rows_of(o, rows):
    return {k: (v[rows] if k in ("xq", "xs", "x", "gate") else v) for k, v in o.items()}


@pytest.mark.parametrize("M,d_in,d_out,rank", [
    (19300, 2048, 264, 128),      # X A^T in one turn and three tiles over, those in a launch of their own
    (38000, 2064, 136, 256),      # and in two turns
    (1 << 20, 128, 24, 8), (3, 128, 1 << 20, 8), (5, 65536, 24, 256),
])
def test_linear(M, d_in, d_out, rank):
    g = torch.Generator().manual_seed(M + d_out)
    o = _operands(M, d_in, d_out, rank) if M * d_in < 5e7 else None
    if o is None:  # (rows repeated: the generator would take minutes)
        o = _operands(1009, d_in, d_out, rank)
        take = torch.randint(0, 1009, (M,), generator=g)
        o = _rows_of(o, take)
    c = _cuda(o)
    y = _run(c, torch.full((M, d_out), math.nan, dtype=BF, device="cuda"))
    assert torch.isfinite(y).all()
    rows = torch.unique(torch.cat([torch.arange(min(M, 40)), torch.randint(0, M, (60,), generator=g),
                                   torch.arange(max(0, M - 400), M, 7), torch.tensor([M - 1])]))
    _check(_rows_of(o, rows), y[rows.cuda()])
    for _ in range(3):
        assert torch.equal(_run(c, torch.empty_like(y)), y)
    assert _lib.uno_read_device_status() == _lib.UNO_OK


@pytest.mark.parametrize("dtype", [BF, F32])
def test_logprobs_many_short_rows(dtype):
    N, V = 2_000_003, 11
    x = (3 * torch.randn((N, V), device="cuda")).to(dtype)
    tok = torch.randint(-1, V, (N,), device="cuda", dtype=torch.int32)
    lp, ent = torch.full((N,), math.nan, device="cuda"), torch.full((N,), math.nan, device="cuda")
    st, ids, tl = torch.empty((N, 2), device="cuda"), torch.empty((N, 2), dtype=torch.int32, device="cuda"), \
        torch.empty((N, 2), device="cuda")
    _lib.uno_token_logprobs(x, tok, lp, 1.0, ent, st, ids, tl)
    ref = torch.log_softmax(x.double(), 1)
    keep = tok >= 0
    at = torch.where(keep, ref.gather(1, tok.clamp(min=0).long()[:, None])[:, 0], 0.0)
    bound = R.logs_bound(V)
    assert ((lp.double() - at).abs() <= 4 * R.F32 * at.abs() + 1.1 * bound).all()
    h = torch.where(keep, -(ref.exp() * ref).sum(1), 0.0)
    assert ((ent.double() - h).abs() <= 1.1 * bound + 2 * bound * (h.abs() + math.log(V))).all()
    best = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(ids.long(), torch.where(keep[:, None], best, torch.full_like(best, -1)))
    g = torch.empty_like(x)
    _lib.uno_token_logprobs_grad(x, tok, st, g, grad_logprob=torch.ones(N, device="cuda"))
    one = torch.zeros_like(ref).scatter_(1, tok.clamp(min=0).long()[:, None], 1.0)
    exact = torch.where(keep[:, None], one - ref.exp(), 0.0)
    # (p is off by its argument's and its own roundings, 1e-6 of it at most here; then the type's)
    half = R.HALF_BF16 if dtype == BF else R.F32
    assert ((g.double() - exact).abs() <= 1.01 * half * exact.abs() + 3e-6).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_logprobs_long_rows(dtype):
    """300 million tokens a row: ids past 2^28, the best of them at both ends and in the middle."""
    N, V, k = 2, 300_000_007, 8
    x = torch.empty((N, V), dtype=dtype, device="cuda")
    for n in range(N):
        x[n].normal_().mul_(0.5)
    far = [0, 1, V // 3, V // 2, V - 9, V - 2, V - 1]
    for i, v in enumerate(far):
        x[0, v] = 20.0 + i
    x[1] = x[1].clamp_(max=8.0)
    tok = torch.tensor([V - 1, V // 2], dtype=torch.int32, device="cuda")
    lp, ent, ids, tl = (torch.empty(2, device="cuda"), torch.empty(2, device="cuda"),
                        torch.empty((2, k), dtype=torch.int32, device="cuda"), torch.empty((2, k), device="cuda"))
    _lib.uno_token_logprobs(x, tok, lp, 1.0, ent, None, ids, tl)
    assert ids[0, :7].tolist() == far[::-1]
    for n in range(N):
        mx = x[n].max().double()
        s = sum(torch.exp(part.double() - mx).sum() for part in x[n].split(1 << 25))
        z = x[n, tok[n].long()].double() - mx
        # a thread adds some 18300 weights of 2^-24 relative rounding each
        tol = (V / 8 / 256 / (16 // x.element_size()) * 2 + 80) * R.F32
        assert abs(float(lp[n]) - float(z - s.log())) <= tol
        top = torch.topk(x[n].float(), k).values
        assert torch.equal(x[n, ids[n].long()].float(), top)
        assert ((tl[n].double() - (top.double() - mx - s.log())).abs() <= tol + 4 * R.F32 * 30).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_and_quantize_many_rows_and_long_ones(dtype):
    M, d = 1_500_001, 272
    x = torch.randn((M, d), device="cuda").to(dtype)
    w = torch.ones(d, dtype=dtype, device="cuda")
    q, s = torch.empty((M, d), dtype=R.F8, device="cuda"), torch.empty((M, 3), device="cuda")
    _lib.uno_rms_norm_fp8(x, w, 1e-6, q, s)
    rows = torch.cat([torch.arange(50), torch.randint(0, M, (100,)), torch.arange(M - 50, M)])
    _, _, rq, _ = R.rms_norm(x[rows.cuda()].cpu(), w.cpu(), 1e-6)
    assert torch.equal(q[rows.cuda()].cpu().double(), rq)
    _lib.uno_fp8_quantize(x, q, s)
    rq, rs = R.quantize(x[rows.cuda()].cpu().double(), 1)
    assert torch.equal(q[rows.cuda()].cpu().double(), rq) and torch.equal(s[rows.cuda()].cpu(), rs.float())
    del x, q, s
    rows, cols = 3, (1 << 28) + 16
    x = torch.randn((rows, cols), device="cuda").to(dtype)
    for block in (1, 128):
        q = torch.empty((rows, cols), dtype=R.F8, device="cuda")
        s = torch.empty((rows if block == 1 else 1, -(-cols // 128)), device="cuda")
        _lib.uno_fp8_quantize(x, q, s, block)
        for lo, hi in ((0, 4096), (1 << 27, (1 << 27) + 4096), (cols - 4112, cols)):
            rq, rs = R.quantize(x[:, lo:hi].cpu().double(), block)
            assert torch.equal(q[:, lo:hi].cpu().double(), rq)
            assert torch.equal(s[:, lo // 128:-(-hi // 128)].cpu(), rs.float())
        del q, s
