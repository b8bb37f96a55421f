"""uno_token_logprobs and its gradient against their plain 64-bit forms: log probabilities,
entropies and gradients within the roundings counted below, alternatives' ids equal."""
import math

import pytest
import torch

from diffusion_drafted_lossless_b200 import _lib
from tests import layers_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NINF = -math.inf


def _logits(N, V, dtype, seed, sigma=3.0):
    g = torch.Generator().manual_seed(seed + N + 3 * V)
    x = (sigma * torch.randn((N, V), generator=g)).to(dtype)
    tok = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    return x, tok


def _run(x, tok, k=5, T=1.0, **kw):
    N = x.shape[0]
    o = {"logprob": torch.full((N,), 9.0, device="cuda"), "entropy": torch.full((N,), 9.0, device="cuda"),
         "stats": torch.full((N, 2), 9.0, device="cuda"),
         "ids": torch.full((N, k), 9, dtype=torch.int32, device="cuda") if k else None,
         "lps": torch.full((N, k), 9.0, device="cuda") if k else None}
    xd = x if x.is_cuda else x.cuda()
    _lib.uno_token_logprobs(xd, None if tok is None else tok.cuda(), None if tok is None else o["logprob"], T,
                            o["entropy"], o["stats"], o["ids"], o["lps"], **kw)
    torch.cuda.synchronize()
    return {k2: None if v is None else v.cpu() for k2, v in o.items()}


def _near(got, ref, tol):
    """Within tol where ref is finite, equal to it elsewhere."""
    got = got.double()
    fine = torch.isfinite(ref)
    assert torch.equal(got[~fine], ref[~fine])
    err = (got - ref).abs()[fine]
    tol = tol.expand_as(ref)[fine] if isinstance(tol, torch.Tensor) else tol
    assert (err <= tol).all(), float((err / tol).max())


def _check(x, tok, o, k, T=1.0):
    """z = (x - max) / T: three roundings of it; then log s's own error and a rounding."""
    N, V = x.shape
    r = R.logprobs(x, tok, T)
    lb = R.logs_bound(V)
    if tok is not None:
        _near(o["logprob"], r["logprob"], 4 * R.F32 * r["logprob"].abs() + 1.1 * lb)
    # a / s: the errors of two such sums, relative, on a mean of octaves of at most H + log V
    _near(o["entropy"], r["entropy"], 1.1 * lb + 2 * lb * (r["entropy"].abs() + math.log(V)) + 1e-30)
    live = r["keep"] & ~r["empty"]
    assert torch.equal(o["stats"][live, 0].double(), r["max"][live])
    _near(o["stats"][live, 1], r["logs"][live], 1.1 * lb + R.F32 * r["logs"][live].abs())
    assert (o["stats"][~r["keep"]] == 0).all()
    gone = r["keep"] & r["empty"]
    assert (o["stats"][gone, 0] == NINF).all() and (o["stats"][gone, 1] == 0).all()
    if k:
        ids, lps = R.top(x, r, k)
        assert torch.equal(o["ids"].long(), ids)
        _near(o["lps"], lps, 4 * R.F32 * lps.abs().nan_to_num(posinf=0.0) + 1.1 * lb)
    return r


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,V,k,T", [
    (1, 1, 1, 1.0), (2, 2, 5, 0.5), (3, 7, 32, 1.0), (5, 8, 3, 2.0), (4, 9, 0, 1.0), (40, 31, 20, 0.7), (3, 513, 32, 1.0),
    (700, 65, 4, 1.0), (6, 4097, 20, 1.3), (5, 16384, 1, 1.0), (3, 20003, 32, 0.9), (33, 32000, 5, 1.0),
    (150, 20001, 20, 1.0), (310, 8200, 7, 1.0), (2, 151936, 20, 1.0), (17, 166144, 32, 0.8), (1, 151935, 20, 1.0),
])
def test_logprobs(N, V, k, T, dtype):
    x, tok = _logits(N, V, dtype, 1)
    tok[1::5] = -1
    if N > 2:
        tok[2] = V  # not a token either
    _check(x, tok, _run(x, tok, k, T), k, float(torch.tensor(T)))


@pytest.mark.parametrize("V", [1000, 20008, 151936])
def test_masked_rows(V):
    """-inf in places, everywhere but one token, everywhere; the type's lowest value everywhere
    and beside ordinary values; very large values; more alternatives than tokens."""
    for dtype in (BF, F32):
        x, tok = _logits(10, V, dtype, 2)
        low = torch.finfo(dtype).min
        x[0, V // 3:] = NINF
        x[1] = NINF
        x[1, 5] = 2.0
        x[2] = NINF
        x[3] = low
        x[4, ::2] = low
        x[5] = 1e4 * x[5]
        x[6, :V // 2] = NINF
        x[7] = NINF
        x[7, V - 1] = low
        x[8, :17] = NINF
        tok[0], tok[1], tok[4], tok[7] = V - 1, 5, 0, V - 1
        _check(x, tok, _run(x, tok, 20), 20)


@pytest.mark.parametrize("V", [3000, 40000, 151936])
def test_rows_in_order_and_ties(V):
    """Rows whose candidates arrive best last, rows of few distinct values, rows of one value:
    the list of candidates overflows and the alternatives are still the exact ones."""
    up = torch.linspace(-8, 8, V)
    for dtype in (BF, F32):
        x = torch.stack([up, up.flip(0), torch.zeros(V), (torch.arange(V) % 3).float(),
                         torch.where(torch.arange(V) < V - 5, 1.0, 0.0), -up.abs(), up.abs()]).to(dtype)
        tok = torch.arange(7, dtype=torch.int32)
        for k in (1, 20, 32):
            _check(x, tok, _run(x, tok, k), k)
        many = x.repeat(60, 1)  # one CTA per row
        _check(many, tok.repeat(60), _run(many, tok.repeat(60), 7), 7)


def test_large_steps_within_a_row():
    """References move: values that rise by hundreds along the row, with and without a
    temperature, and a single late value far above the rest."""
    V = 50000
    x = torch.stack([torch.linspace(-3000, 3000, V), torch.linspace(3000, -3000, V),
                     torch.where(torch.arange(V) == V - 3, 500.0, -1.0)])
    tok = torch.tensor([V - 1, 0, V - 3], dtype=torch.int32)
    for T in (0.25, 1.0, 4.0):
        _check(x, tok, _run(x, tok, 5, T), 5, T)


def test_nan_and_inf_stay_in_their_rows():
    x, tok = _logits(6, 30001, BF, 4)
    clean = _run(x, tok, 5)
    x[1, 9], x[4, 77] = math.nan, math.inf
    o = _run(x, tok, 5)
    for n in (0, 2, 3, 5):
        for key in ("logprob", "entropy", "stats", "ids", "lps"):
            assert torch.equal(o[key][n], clean[key][n])
    assert math.isnan(o["logprob"][1]) and math.isnan(o["logprob"][4])
    assert (o["ids"] >= -1).all() and (o["ids"] < 30001).all()


def test_without_tokens_and_single_outputs():
    x, tok = _logits(9, 5000, BF, 5)
    _check(x, None, _run(x, None, 3), 3)
    full = _run(x, tok, 3)
    xd, td = x.cuda(), tok.cuda()
    lp, ent = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
    _lib.uno_token_logprobs(xd, td, lp)
    _lib.uno_token_logprobs(xd, td, None, out_entropy=ent)
    assert torch.equal(lp.cpu(), full["logprob"]) and torch.equal(ent.cpu(), full["entropy"])
    _lib.uno_token_logprobs(xd[:0], td[:0], lp[:0])


def _grad(x, tok, gl, ge, T=1.0, inplace=False):
    xd, td = x.cuda(), None if tok is None else tok.cuda()
    N = x.shape[0]
    ent, st = torch.empty(N, device="cuda"), torch.empty((N, 2), device="cuda")
    _lib.uno_token_logprobs(xd, td, None, T, ent, st)
    g = xd if inplace else torch.full_like(xd, 7.0)
    dv = lambda t: None if t is None else t.cuda()  # noqa: E731
    _lib.uno_token_logprobs_grad(xd, td, st, g, dv(gl), ent if ge is not None else None, dv(ge), T)
    torch.cuda.synchronize()
    return g.cpu()


def _check_grad(x, tok, gl, ge, g, T=1.0):
    """p = exp2 of an argument: its own 2^-22, the argument's roundings (of itself and of its
    two terms) and log s's error; the entropy's factor carries the entropy's error; then the
    sum with the token's own term and the rounding to the type."""
    ref, r = R.logprobs_grad(x, tok, T, gl, ge)
    V = x.shape[1]
    lb = R.logs_bound(V)
    a = torch.zeros(len(x)) if gl is None else gl.abs()
    b = torch.zeros(len(x)) if ge is None else ge.abs()
    z = r["lp"].abs().nan_to_num(posinf=0.0)
    rel = 4 * R.F32 + 4 * R.F32 * (z + r["logs"].abs()[:, None] + 1) * 1.5 + lb
    size = r["p"] * (a[:, None] + b[:, None] * (z + r["h"].abs()[:, None] + 1)) / T
    h_err = r["p"] * (b[:, None] * 3 * lb * (r["h"].abs()[:, None] + math.log(V) + 1)) / T
    own = (a / T)[:, None] * (r["p"] > 2).double()
    if gl is not None:
        own = own.scatter(1, tok.clamp(0, V - 1).long()[:, None], (4 * R.F32 * a / T).double()[:, None])
    half = R.HALF_BF16 if x.dtype == BF else R.F32
    tol = (rel * size + h_err + own) * 1.1 + half * ref.abs() * 1.01 + 1e-37
    err = (g.double() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,V,T", [(1, 1, 1.0), (3, 2, 1.0), (7, 9, 0.5), (40, 65, 1.0), (5, 4097, 1.3), (3, 8192, 1.0),
                                   (33, 20003, 0.8), (2, 151936, 1.0)])
def test_grad(N, V, T, dtype):
    x, tok = _logits(N, V, dtype, 6)
    tok[1::4] = -1
    if V > 8:
        x[0, V // 2:] = NINF
        tok[0] = V - 1  # a token that cannot be produced: its own gradient is still 1
    if N > 2:
        x[2] = NINF
    g = torch.Generator().manual_seed(9)
    gl, ge = torch.randn(N, generator=g), 0.3 * torch.randn(N, generator=g)
    T = float(torch.tensor(T))
    for a, b in ((gl, ge), (gl, None), (None, ge)):
        _check_grad(x, tok, a, b, _grad(x, tok, a, b, T), T)
    assert torch.equal(_grad(x, tok, gl, ge, T), _grad(x, tok, gl, ge, T, inplace=True))
    _check_grad(x, None, None, ge, _grad(x, None, None, ge, T), T)


def test_grad_against_differences():
    """Central differences of the forward call on float32 logits. A step of 2^-6: the third
    derivative of log p and of H is at most about 3 here (h^2 / 6 of it: 1.3e-4), and the
    forward error of 2e-6 over the step's width is 6e-5."""
    V, T, h = 50, 0.9, 2.0 ** -6
    x, _ = _logits(1, V, F32, 8, sigma=1.0)
    tok = torch.tensor([3], dtype=torch.int32)
    both = torch.cat([x + h * torch.eye(V), x - h * torch.eye(V)])
    o = _run(both, tok.repeat(2 * V), 0, T)
    d_lp = (o["logprob"][:V] - o["logprob"][V:]) / (2 * h)
    d_h = (o["entropy"][:V] - o["entropy"][V:]) / (2 * h)
    one = torch.ones(1)
    assert (_grad(x, tok, one, None, T)[0] - d_lp).abs().max() <= 3e-4
    assert (_grad(x, tok, None, one, T)[0] - d_h).abs().max() <= 3e-4


def test_rows_behind_the_last_are_left():
    x, tok = _logits(5, 1001, BF, 3)
    xd = torch.full((8, 1001), 5.0, dtype=BF, device="cuda")
    xd[:5] = x.cuda()
    lp, st = torch.full((8,), 5.0, device="cuda"), torch.full((8, 2), 5.0, device="cuda")
    ent = torch.full((8,), 5.0, device="cuda")
    ids, tl = torch.full((8, 3), 5, dtype=torch.int32, device="cuda"), torch.full((8, 3), 5.0, device="cuda")
    _lib.uno_token_logprobs(xd[:5], tok.cuda(), lp[:5], 1.0, ent[:5], st[:5], ids[:5], tl[:5])
    _lib.uno_token_logprobs_grad(xd[:5], tok.cuda(), st[:5], xd[:5], torch.ones(5, device="cuda"))
    for t in (xd, lp, st, ent, ids, tl):
        assert (t[5:] == 5).all()


def test_streams_and_graph_replay():
    x, tok = _logits(24, 30000, BF, 11)
    xd, td = x.cuda(), tok.cuda()
    outs = [(torch.empty(24, device="cuda"), torch.empty((24, 2), device="cuda"),
             torch.empty((24, 4), dtype=torch.int32, device="cuda"), torch.empty((24, 4), device="cuda"))
            for _ in range(3)]

    def call(o, stream=None):
        _lib.uno_token_logprobs(xd, td, o[0], out_stats=o[1], out_top_ids=o[2], out_top_logprobs=o[3], stream=stream)

    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st, o in zip(streams, outs):
        call(o, st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    grad = torch.empty_like(xd)
    gl = torch.ones(24, device="cuda")
    with torch.cuda.graph(g):
        call(outs[2])
        _lib.uno_token_logprobs_grad(xd, td, outs[2][1], grad, gl)
    for seed in (11, 12):
        x, tok = _logits(24, 30000, BF, seed)
        xd.copy_(x.cuda())
        td.copy_(tok.cuda())
        g.replay()
        call(outs[0])
        torch.cuda.synchronize()
        for a, b in zip(outs[0], outs[2]):
            assert torch.equal(a, b)
        _check_grad(x, tok, torch.ones(24), None, grad.cpu())


def test_offsets_past_32_bits():
    """More than 2^31 logits: the last rows are the ones that were asked for."""
    N, V = 16400, 131080
    xd = torch.zeros((N, V), dtype=BF, device="cuda")
    x, tok = _logits(3, V, BF, 21)
    xd[-3:] = x.cuda()
    td = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    td[-3:] = tok.cuda()
    o = _run(xd, td, 4)
    _check(x, tok, {k: v[-3:] for k, v in o.items()}, 4)
    st, gl = o["stats"].cuda(), torch.ones(N, device="cuda")
    _lib.uno_token_logprobs_grad(xd, td, st, xd, gl)
    _check_grad(x, tok, torch.ones(3), None, xd[-3:].cpu())
    assert (xd[:-3] == 0).all()


def test_binding_refuses_wrong_shapes():
    x, tok = _logits(4, 100, BF, 1)
    xd, td = x.cuda(), tok.cuda()
    lp = torch.empty(4, device="cuda")
    with pytest.raises(ValueError, match="tokens"):
        _lib.uno_token_logprobs(xd, td.long(), lp)
    with pytest.raises(ValueError, match="out_logprob"):
        _lib.uno_token_logprobs(xd, td, lp[:3])
    with pytest.raises(_lib.UnoError, match="top_n"):
        _lib.uno_token_logprobs(xd, td, lp, out_top_ids=torch.empty((4, 3), dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        _lib.uno_token_logprobs(xd.half(), td, lp)
    with pytest.raises(ValueError, match="stats"):
        _lib.uno_token_logprobs_grad(xd, td, lp, xd, lp)
