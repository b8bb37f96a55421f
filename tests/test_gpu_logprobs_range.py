"""uno_token_logprobs and its gradient over the whole range they state: finite logits of any size,
temperatures from 1e-30 to the largest float32, references that cross from one kind of sums to
the other within a row. Held to the plain 64-bit forms within test_gpu_logprobs's bounds, which
count roundings relative to the results and hold at every size and temperature (the gradient's,
with what an exponential below float32's normal numbers loses)."""
import math

import pytest
import torch

from tests import layers_ref as R
from tests.test_gpu_logprobs import _check, _grad, _logits, _near, _run

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NINF = -math.inf
FLUSHED = 2.0 ** -126  # an exponential below float32's least normal number is 0


def _rows(V, dtype):
    """Rows of one value of every size, of a maximum of every size, with masked places, and
    rows whose values pass 2^20 octaves at temperature 1 (726817 nats) on the way up or down."""
    x, tok = _logits(17, V, F32, 31)
    for n, v in enumerate((-1e9, -1e10, -1e12, -1e15, -1e20, 1e15, -1e31)):
        x[n] = v
    x[7, V // 3] = 1e10
    x[8, V - 2] = 1e15
    x[9, V // 2:] = NINF
    x[10] += 50.0
    x[10, ::2] = NINF
    x[11] = torch.linspace(726700, 726900, V)
    x[12] = torch.linspace(726900, 726700, V)
    x[13] = torch.where(torch.arange(V) % 2 == 0, 726817.0, 726817.5)
    x[14] = NINF
    x[15] = x[15] * 1e-6
    x = x.to(dtype)
    tok[7], tok[8], tok[11], tok[14] = V // 3, V - 2, V - 1, 0
    return x, tok


def _check_grad(x, tok, gl, ge, g, T):
    """p = exp2 of an argument: its own error, the argument's roundings (of itself and of its two
    terms) and log s's error, all relative; and 2^-126 where it is flushed, which a factor over a
    small temperature brings back into sight. The entropy's factor carries the entropy's error;
    then the token's own term and the rounding to the type."""
    ref, r = R.logprobs_grad(x, tok, T, gl, ge)
    lb, zero = R.logs_bound(x.shape[1]), torch.zeros(len(x))
    a, b = ((zero if t is None else t.abs()).double()[:, None] for t in (gl, ge))
    z, h = r["lp"].abs().nan_to_num(posinf=0.0), r["h"].abs()[:, None]
    rel = 4 * R.F32 * (1 + 1.5 * (z + r["logs"].abs()[:, None] + 1)) + lb
    factor = (a + b * (z + h + 1)) / T
    lost = (r["p"] > 0) & (r["p"] < 1.01 * FLUSHED)
    tol = (rel * r["p"] + torch.where(lost, FLUSHED, 0.0)) * factor
    tol += r["p"] * b * 3 * lb * (h + math.log(x.shape[1]) + 1) / T
    tol.scatter_add_(1, tok.clamp(0, x.shape[1] - 1).long()[:, None], 4 * R.F32 * a / T)
    half = R.HALF_BF16 if x.dtype == BF else R.F32
    _near(g, ref, tol * 1.1 + half * ref.abs() * 1.01 + 1e-37)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1.0, 0.3, 1e-3, 1e-6, 1e-8, 1.4426e-8, 1.4428e-8, 3e-9, 1e-9, 1e-12, 1e-20, 1e-24, 1e10,
                               1e19, 1e20, 1e21, 1e30])
def test_values_of_any_size_and_any_temperature(T, dtype):
    T = float(torch.tensor(T))
    for V in (700, 20003, 151936):
        x, tok = _rows(V, dtype)
        if T < 1e-20:  # (differences over T that float32 cannot hold)
            x[7], x[8] = x[16], x[16]
        _check(x, tok, _run(x, tok, 20, T), 20, T)
    many = _rows(20003, dtype)  # one CTA per row
    x, tok = many[0].repeat(18, 1), many[1].repeat(18)
    if T < 1e-20:
        x[7::17], x[8::17] = x[16], x[16]
    _check(x, tok, _run(x, tok, 3, T), 3, T)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_smallest_temperature(dtype):
    """1e-30: rows of ordinary values, masked places, rows of one value."""
    x, tok = _rows(20003, dtype)
    x[7], x[8] = x[16], x[16]
    for n in range(11, 14):
        x[n] = x[16]
    _check(x, tok, _run(x, tok, 5, 1.001e-30), 5, float(torch.tensor(1.001e-30)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1e35, 1e38, 3.4e38])
def test_the_largest_values_and_temperatures(T, dtype):
    """Differences of logits beyond float32's largest number, which a large temperature brings
    back into it."""
    T = float(torch.tensor(T))
    V = 20003
    x, tok = _logits(6, V, F32, 41)
    big = torch.finfo(dtype).max
    x[0] = torch.where(torch.arange(V) % 2 == 0, big, -big)
    x[1] = torch.linspace(-1, 1, V) * big
    x[2] = -big
    x[2, V - 1] = big
    x[3] = (x[3] / 12).clamp(-1, 1) * big
    x[3, ::3] = NINF
    x[4] = big
    x = x.clamp(-math.inf, big).to(dtype)
    tok[0], tok[2] = 1, 0
    _check(x, tok, _run(x, tok, 5, T), 5, T)
    gl = 1e38 * torch.ones(6)
    _check_grad(x, tok, gl, None, _grad(x, tok, gl, None, T), T)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [0.3, 1e-3, 1e-7, 1e-9, 1e-12, 1e-24])
def test_grad_of_any_size_and_small_temperatures(T, dtype):
    T = float(torch.tensor(T))
    x, tok = _rows(20003, dtype)
    if T < 1e-20:
        x[7], x[8] = x[16], x[16]
    g = torch.Generator().manual_seed(9)
    gl, ge = torch.randn(17, generator=g), 0.3 * torch.randn(17, generator=g)
    for a, b in ((gl, None), (None, ge), (gl, ge)):
        _check_grad(x, tok, a, b, _grad(x, tok, a, b, T), T)


def test_entropy_gradient_where_a_weight_vanishes_beside_a_large_factor():
    """A factor whose product with a far octave passes float32: a token without weight still has
    the gradient 0."""
    x = torch.tensor([[0.0, 0.0, -5.0, NINF]])
    T = float(torch.tensor(1e-30))
    ge = torch.tensor([1e6])
    g = _grad(x, None, None, ge, T)
    assert (g[0, 2:] == 0).all() and torch.isfinite(g).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_log_probabilities_and_entropies_keep_their_signs(dtype):
    """One late token far above the sample holds all the weight: its probability is not above 1,
    its alternatives' neither, and no entropy is negative."""
    N, V = 300, 40000
    g = torch.Generator().manual_seed(3)
    x = torch.full((N, V), -1.0)
    x[torch.arange(N), V - 3] = 20 + 20 * torch.rand(N, generator=g)
    x = x.to(dtype)
    tok = torch.full((N,), V - 3, dtype=torch.int32)
    for T in (0.7, 1.0, 1e-9):
        o = _run(x, tok, 2, T)
        assert (o["logprob"] <= 0).all() and (o["lps"] <= 0).all() and (o["stats"][:, 1] >= 0).all()
        assert (o["entropy"] >= 0).all()
        _check(x, tok, o, 2, float(torch.tensor(T)))
