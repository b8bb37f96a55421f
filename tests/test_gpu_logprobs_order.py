"""Alternatives of rows whose best tokens lie in the middle of a slope: far more candidates than a
list holds arrive before and after them. The ids are the exact ones, and the time does not grow
with the slope's length."""
import pytest
import torch

from diffusion_drafted_lossless_b200 import _lib
from tests.test_gpu_logprobs import _check, _run

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _hump(V, at):
    """Up to position `at`, then down: float32 values that all differ on a side."""
    i = torch.arange(V, dtype=torch.float64)
    return (-(i - at * V).abs() / V * 16).float()


@pytest.mark.parametrize("V", [40000, 151936, 600011])
@pytest.mark.parametrize("k", [1, 20, 32])
def test_humps(V, k):
    for dtype in (BF, F32):
        x = torch.stack([_hump(V, at) for at in (0.1, 0.5, 0.6, 0.97)] + [-_hump(V, 0.4)]).to(dtype)
        tok = torch.arange(len(x), dtype=torch.int32)
        _check(x, tok, _run(x, tok, k), k)
        many = x[:4].repeat(50, 1)  # one CTA per row
        ids = torch.empty((200, k), dtype=torch.int32, device="cuda")
        lps = torch.empty((200, k), device="cuda")
        for _ in range(3):
            _lib.uno_token_logprobs(many.cuda(), None, out_top_ids=ids, out_top_logprobs=lps)
            few = _run(x[:4], None, k)
            assert torch.equal(ids.view(50, 4, k).cpu(), few["ids"].expand(50, 4, k))


def _us(x, k):
    ids, lps = torch.empty((len(x), k), dtype=torch.int32, device="cuda"), torch.empty((len(x), k), device="cuda")
    times = []
    for _ in range(7):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        _lib.uno_token_logprobs(x, None, out_top_ids=ids, out_top_logprobs=lps)
        e[1].record()
        torch.cuda.synchronize()
        times.append(1e3 * e[0].elapsed_time(e[1]))
    return sorted(times)[3]


def test_a_hump_is_read_a_few_times_at_most():
    """A few readings more than a row in no order needs, each of them slower for the candidates that
    are counted one by one: below thirty times its time (seventy to a hundred where each reading
    got no further than a list's length)."""
    for dtype in (BF, F32):
        x = _hump(151936, 0.5).to(dtype).repeat(600, 1).cuda()
        plain = (3 * torch.randn((600, 151936), device="cuda")).to(dtype)
        assert _us(x, 20) <= 30 * _us(plain, 20)
