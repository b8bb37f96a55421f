"""The entry points of include/uno_layers.h without a GPU: every declared symbol is exported
and bound, and arguments they cannot take are refused before any device work."""
import re
from pathlib import Path

import pytest
import torch

from diffusion_drafted_lossless_b200 import _lib
from diffusion_drafted_lossless_b200.build import build

ROOT = Path(__file__).resolve().parents[1]
FAKE = 0x7F0000000000  # a 256-byte aligned address that is never dereferenced
OK, ARG, UNSUP, WS = _lib.UNO_OK, _lib.UNO_ERR_INVALID_ARG, _lib.UNO_ERR_UNSUPPORTED, _lib.UNO_ERR_WORKSPACE
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", (ROOT / "include" / "uno_layers.h").read_text(), flags=re.S)
    names = set(re.findall(r"\b(uno_[a-z0-9_]+)\s*\(", text))
    assert names == set(_lib.EXPORTED_LAYERS)
    for n in names:
        assert hasattr(lib, n) and hasattr(_lib, n), n


def test_norm_refusals(lib):
    def call(x=FAKE, res=None, w=FAKE, dt=0, M=4, d=256, eps=1e-6, ores=None, q=FAKE, s=FAKE, y=None):
        return lib.uno_rms_norm_fp8(x, res, w, dt, M, d, eps, ores, q, s, y, None)

    assert call(dt=7) == ARG and call(M=-1) == ARG and call(d=0) == ARG
    for eps in (0.0, -1.0, INF, NAN):
        assert call(eps=eps) == ARG
    assert call(d=24) == UNSUP and call(d=32768 + 16) == UNSUP and call(M=1 << 31) == UNSUP
    assert call(x=None) == ARG and call(w=None) == ARG
    assert call(q=None) == ARG and call(s=None) == ARG and call(q=None, s=None) == ARG
    assert call(ores=FAKE) == ARG  # without a residual there is no sum to store
    for k in ("x", "w", "q", "s", "y", "res"):
        assert call(**{k: FAKE + 8}) == UNSUP, k
    assert b"16-byte" in lib.uno_last_error_string()
    assert call(M=0, x=None, w=None, q=None, s=None) == OK


def test_quantize_refusals(lib):
    def call(x=FAKE, dt=0, M=4, d=256, rows=1, q=FAKE, s=FAKE):
        return lib.uno_fp8_quantize(x, dt, M, d, rows, q, s, None)

    assert call(dt=2) == ARG and call(M=-1) == ARG and call(d=0) == ARG
    assert call(rows=0) == ARG and call(rows=64) == ARG and call(rows=-128) == ARG
    assert call(d=8) == UNSUP and call(M=1 << 31) == UNSUP and call(d=1 << 31) == UNSUP
    assert call(x=None) == ARG and call(q=None) == ARG and call(s=None) == ARG
    assert call(x=FAKE + 4) == UNSUP and call(q=FAKE + 4) == UNSUP and call(s=FAKE + 4) == UNSUP
    assert call(M=0, x=None, q=None, s=None) == OK


def test_linear_refusals(lib):
    def call(xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, x=FAKE, a=FAKE, b=FAKE, gate=FAKE, scale=2.0, M=16, i=256, o=256,
             r=8, y=FAKE, dt=0, wsp=FAKE, wsb=1 << 30):
        return lib.uno_fp8_gated_lora_linear(xq, xs, wq, ws, x, a, b, gate, scale, M, i, o, r, y, dt, wsp, wsb, None)

    assert call(dt=3) == ARG and call(M=-1) == ARG and call(i=0) == ARG and call(o=0) == ARG and call(r=-8) == ARG
    assert call(i=264) == UNSUP and call(i=65536 + 16) == UNSUP and call(o=(1 << 20) + 1) == UNSUP
    assert call(M=(1 << 20) + 1) == UNSUP and call(r=12) == UNSUP and call(r=264) == UNSUP
    assert call(M=1 << 20, i=65536, o=1 << 20) == UNSUP  # 8192 * 4096 tiles * 513 K blocks
    assert call(dt=1) == UNSUP  # float32 output with an adapter
    for k in ("xq", "xs", "wq", "ws", "y", "x", "a", "b"):
        assert call(**{k: None}) == ARG, k
    for k in ("xq", "xs", "wq", "ws", "y", "x", "a", "b", "gate"):
        assert call(**{k: FAKE + 8}) == UNSUP, k
    for s in (INF, NAN):
        assert call(scale=s) == ARG
    assert call(wsp=None) == WS and call(wsp=FAKE + 16) == WS and call(wsb=255) == WS
    assert call(M=0, xq=None, wq=None, y=None, wsp=None) == OK
    size = lib.uno_fp8_gated_lora_linear_workspace_size
    assert size(16, 256, 256, 8) == 256 and size(1024, 4096, 4096, 128) == 1024 * 128 * 2
    assert size(16, 256, 256, 0) == 0 and size(0, 256, 256, 8) == 0


def test_logprobs_refusals(lib):
    def call(x=FAKE, dt=0, N=4, V=100, T=1.0, tok=FAKE, k=5, lp=FAKE, ent=None, st=None, ids=FAKE, tlp=FAKE):
        return lib.uno_token_logprobs(x, dt, N, V, T, tok, k, lp, ent, st, ids, tlp, None)

    assert call(dt=9) == ARG and call(N=-1) == ARG and call(V=0) == ARG and call(k=-1) == ARG
    for T in (0.0, -1.0, INF, NAN):
        assert call(T=T) == ARG
    assert call(T=1e-31) == UNSUP and call(k=33) == UNSUP
    assert call(V=0x7FFFF001) == UNSUP and call(N=1 << 31) == UNSUP and call(N=1 << 20, V=1 << 20) == UNSUP
    assert call(x=None) == ARG
    assert call(tok=None) == ARG  # a log probability of which token?
    assert call(ids=None) == ARG and call(tlp=None) == ARG and call(k=0) == ARG
    assert call(k=0, ids=None, tlp=None, lp=None) == ARG  # nothing to write
    for n in ("x", "tok", "lp", "ids", "tlp"):
        assert call(**{n: FAKE + 4}) == UNSUP, n
    assert call(N=0, x=None) == OK


def test_logprobs_grad_refusals(lib):
    def call(x=FAKE, dt=0, N=4, V=100, T=1.0, tok=FAKE, st=FAKE, ent=FAKE, gl=FAKE, ge=FAKE, g=FAKE):
        return lib.uno_token_logprobs_grad(x, dt, N, V, T, tok, st, ent, gl, ge, g, None)

    assert call(dt=9) == ARG and call(N=-1) == ARG and call(V=0) == ARG and call(T=0.0) == ARG
    assert call(x=None) == ARG and call(st=None) == ARG and call(g=None) == ARG
    assert call(gl=None, ge=None) == ARG and call(tok=None) == ARG and call(ent=None) == ARG
    for n in ("x", "tok", "st", "ent", "gl", "ge", "g"):
        assert call(**{n: FAKE + 4}) == UNSUP, n
    assert call(N=1 << 20, V=1 << 20) == UNSUP
    assert call(N=0, x=None) == OK


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 256), dtype=torch.float8_e4m3fn), torch.zeros((4, 2))
    tok = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        _lib.uno_rms_norm_fp8(x, x[0], 1e-6, q, s)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        _lib.uno_fp8_quantize(x, q, s)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        _lib.uno_fp8_gated_lora_linear(q, s, q, s, x)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        _lib.uno_token_logprobs(x, tok, torch.zeros(4))
    with pytest.raises(ValueError, match="contiguous CUDA"):
        _lib.uno_token_logprobs_grad(x, tok, torch.zeros(4, 2), x, torch.zeros(4))


def test_reference_values_of_e4m3():
    """The plain form's rounding agrees with torch's own conversion away from ties and above
    float32's reach, and takes ties to the even code."""
    from tests.layers_ref import CODES, nearest_e4m3
    x = torch.linspace(-448, 448, 4001, dtype=torch.float32)
    assert torch.equal(nearest_e4m3(x.double()), x.to(torch.float8_e4m3fn).double())
    mid = (CODES[1:] + CODES[:-1]) / 2
    got = nearest_e4m3(mid)
    even = torch.where(torch.arange(126) % 2 == 0, CODES[:-1], CODES[1:])
    assert torch.equal(got, even)
