"""The operators of include/uno_layers.h as they are used together: norm, projection on the
8-bit base, head, verify, report of the emitted tokens and the gradient of their log
probabilities, each stage held to its plain 64-bit form on the stage's own inputs; and the
step driver on the 8-bit base, eager and as a graph."""
import threading

import numpy as np
import pytest
import torch

from diffusion_drafted_lossless_b200 import _lib
from diffusion_drafted_lossless_b200 import workloads as W
from diffusion_drafted_lossless_b200.driver import DraftVerifyDriver
from tests import layers_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _check_logprobs(logits, tokens, T, lp, ent, ids, tlp):
    r = R.logprobs(logits, tokens, T)
    lb, V = R.logs_bound(logits.shape[1]), logits.shape[1]
    assert ((lp.double() - r["logprob"]).abs() <= 4 * R.F32 * r["logprob"].abs() + 1.1 * lb).all()
    assert ((ent.double() - r["entropy"]).abs() <= 1.1 * lb + 2 * lb * (r["entropy"].abs() + np.log(V))).all()
    if ids is not None:
        ref_ids, ref_lp = R.top(logits, r, ids.shape[1])
        assert torch.equal(ids.long(), ref_ids)
        fine = torch.isfinite(ref_lp)
        assert ((tlp.double() - ref_lp).abs()[fine] <= (4 * R.F32 * ref_lp.abs() + 1.1 * lb)[fine]).all()


def test_a_step_of_a_model_with_an_8bit_base():
    """Hidden states -> norm -> gated projection -> residual and norm -> head -> logits, which
    the verify takes as the verifier's; the emitted tokens are reported and trained on."""
    B, K, d, V, r = 3, 8, 512, 5003, 16
    M = B * K
    g = torch.Generator().manual_seed(77)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, res = rnd(M, d).to(BF), rnd(M, d).to(BF)
    w1, w2 = (1 + 0.1 * rnd(d)).to(BF), (1 + 0.1 * rnd(d)).to(BF)
    wo, head = (0.05 * rnd(d, d)).to(BF), (0.2 * rnd(V, d)).to(BF)
    a, b = (0.05 * rnd(r, d)).to(BF), (0.05 * rnd(d, r)).to(BF)
    gate = (torch.arange(M) % K != 0).float()
    dev = lambda t: t.cuda()  # noqa: E731

    def q8(rows, cols, block):
        return torch.empty((rows, cols), dtype=R.F8, device="cuda"), \
            torch.empty((rows if block == 1 else -(-rows // 128), -(-cols // 128)), device="cuda")

    wo8, wos = q8(d, d, 128)
    h8, hs = q8(V, d, 128)
    _lib.uno_fp8_quantize(dev(wo), wo8, wos, 128)
    _lib.uno_fp8_quantize(dev(head), h8, hs, 128)
    xq, xs = q8(M, d, 1)
    h1, y1, o, h2 = (torch.empty((M, d), dtype=BF, device="cuda") for _ in range(4))
    _lib.uno_rms_norm_fp8(dev(x), dev(w1), 1e-6, xq, xs, residual=dev(res), out_residual=h1, out_y=y1)
    _lib.uno_fp8_gated_lora_linear(xq, xs, wo8, wos, o, x=y1, lora_a=dev(a), lora_b=dev(b), row_gate=dev(gate), scale=2.0)
    oq, os = q8(M, d, 1)
    _lib.uno_rms_norm_fp8(o, dev(w2), 1e-6, oq, os, residual=h1, out_residual=h2)
    logits = torch.empty((M, V), dtype=BF, device="cuda")
    _lib.uno_fp8_gated_lora_linear(oq, os, h8, hs, logits)

    # each stage against its plain form on what it was given
    c = lambda t: t.cpu()  # noqa: E731
    h, y, q, s = R.rms_norm(x, w1, 1e-6, res)
    assert torch.equal(c(h1), h) and torch.equal(c(xq).double(), q)
    ref, size, low, tb = R.linear(c(xq), c(xs), c(wo8), c(wos), c(y1), a, b, gate, 2.0)
    assert ((c(o).double() - ref).abs() <= R.linear_bound(size, low, tb, ref, d, r, True)).all()
    h, y, q, s = R.rms_norm(c(o), w2, 1e-6, c(h1))
    assert torch.equal(c(h2), h) and torch.equal(c(oq).double(), q)
    ref, size, low, tb = R.linear(c(oq), c(os), c(h8), c(hs))
    assert ((c(logits).double() - ref).abs() <= R.linear_bound(size, low, tb, ref, d, 0, True)).all()

    # verify, report, gradient
    P = logits.view(B, K, V)
    Q = (P.float() + 0.5 * torch.randn((B, K, V), device="cuda")).to(BF)
    u = torch.rand((B, K, 3), device="cuda")
    tok = torch.empty((B, K), dtype=torch.int32, device="cuda")
    cnt = torch.empty((B,), dtype=torch.int32, device="cuda")
    _lib.uno_block_verify(P, Q, 1.0, 50, 0.95, u, tok, cnt)
    lp, ent, st = torch.empty(M, device="cuda"), torch.empty(M, device="cuda"), torch.empty((M, 2), device="cuda")
    ids, tlp = torch.empty((M, 5), dtype=torch.int32, device="cuda"), torch.empty((M, 5), device="cuda")
    _lib.uno_token_logprobs(logits, tok.view(-1), lp, 1.0, ent, st, ids, tlp)
    tokens = c(tok).view(-1)
    assert ((tokens >= 0).view(B, K).sum(1) == c(cnt)).all()
    _check_logprobs(c(logits), tokens, 1.0, c(lp), c(ent), c(ids), c(tlp))
    grad = torch.empty_like(logits)
    _lib.uno_token_logprobs_grad(logits, tok.view(-1), st, grad, grad_logprob=torch.ones(M, device="cuda"))
    ref, _ = R.logprobs_grad(c(logits), tokens, 1.0, torch.ones(M))
    assert (c(grad)[tokens < 0] == 0).all()
    # (the rounding to bf16 of the value; of the token's own, 1 - p, the float32 p's error of a few
    # 2^-24 is absolute: below 1e-6)
    assert ((c(grad).double() - ref).abs() <= 1.02 * R.HALF_BF16 * ref.abs() + 1e-6).all()
    assert _lib.uno_read_device_status() == _lib.UNO_OK


V_ = W.VerifyWorkload("drv", 4242, B=4, K=16, V=32000, sigma=3.0, rho=0.8, temperature=1.0, top_k=50, top_p=0.95)
L_ = W.GatedLoraWorkload("drv", 4243, M=4 * 16, block=16, rank=16, scale=2.0,
                         shapes=(W.LinearShape("q", 512, 512), W.LinearShape("k", 512, 128), W.LinearShape("o", 512, 512),
                                 W.LinearShape("gate", 512, 1024), W.LinearShape("down", 1024, 512)))


def test_two_host_threads_at_once():
    """Two threads call the same entry points, each on a stream of its own, with other sizes: each
    gets what it gets alone, and a refusal in one does not show in the other."""
    def operands(M, d, V, seed):
        g = torch.Generator().manual_seed(seed)
        o = {"x": torch.randn((M, d), generator=g).to(BF).cuda(), "w": torch.ones(d, dtype=BF, device="cuda")}
        w = (0.1 * torch.randn((V, d), generator=g)).to(BF).cuda()
        o["w8"], o["ws"] = torch.empty((V, d), dtype=R.F8, device="cuda"), \
            torch.empty((-(-V // 128), -(-d // 128)), device="cuda")
        _lib.uno_fp8_quantize(w, o["w8"], o["ws"], 128)
        o["a"], o["b"] = (0.1 * torch.randn((16, d), generator=g)).to(BF).cuda(), \
            torch.randn((V, 16), generator=g).to(BF).cuda()
        o["gate"], o["tok"] = torch.ones(M, device="cuda"), torch.arange(M, dtype=torch.int32, device="cuda")
        return o

    def run(o):
        M, d = o["x"].shape
        q, s = torch.empty((M, d), dtype=R.F8, device="cuda"), torch.empty((M, -(-d // 128)), device="cuda")
        _lib.uno_rms_norm_fp8(o["x"], o["w"], 1e-6, q, s)
        logits = torch.empty((M, o["w8"].shape[0]), dtype=BF, device="cuda")
        _lib.uno_fp8_gated_lora_linear(q, s, o["w8"], o["ws"], logits, x=o["x"], lora_a=o["a"], lora_b=o["b"],
                                       row_gate=o["gate"], scale=0.5)
        lp, ent = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        _lib.uno_token_logprobs(logits, o["tok"], lp, 0.7, ent)
        return logits, lp, ent

    sets = [operands(40, 512, 3001, 1), operands(300, 1040, 1504, 2)]
    alone = [run(o) for o in sets]
    torch.cuda.synchronize()
    bad = []

    def thread(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for n in range(60):
                    got = run(sets[i])
                    if i and n % 5 == 0:
                        with pytest.raises(_lib.UnoError, match="temperature"):
                            _lib.uno_token_logprobs(got[0], sets[i]["tok"], got[1], 0.0, got[2])
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, alone[i])):
                        bad.append((i, n))
                stream.synchronize()
        except BaseException as e:  # noqa: BLE001 (reported below, by the test's own thread)
            bad.append((i, repr(e)))

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:4]
    assert _lib.uno_read_device_status() == _lib.UNO_OK


def _steps(graph, base="fp8", report=5):
    d = DraftVerifyDriver(L_, V_, base=base, report=report)
    out = []
    for s in range(4):
        if graph and s == 1:
            d.capture()
        tok, cnt, nxt = d.step()
        torch.cuda.synchronize()
        o = dict(tok=tok, cnt=cnt, nxt=nxt, gate=d.gate)
        for i, L in enumerate(d.lin):
            o[f"y{i}"] = L["y"]
        if report is not None:
            o |= dict(lp=d.logprob, ent=d.entropy)
        if report:
            o |= dict(ids=d.top_ids, tlp=d.top_logprobs)
        if base == "fp8":
            for i, a in enumerate(d.act8.values()):
                o |= {f"q{i}": a["q"], f"s{i}": a["s"], f"a{i}": a["y"], f"x{i}": a["x"]}
        out.append({k: v.cpu().clone() for k, v in o.items()})
    return d, out


def test_driver_on_an_8bit_base():
    d, out = _steps(graph=False)
    for o in out:
        for i, a in enumerate(d.act8.items()):
            (normed, width), _ = a
            x = o[f"x{i}"]
            if normed:
                _, y, q, s = R.rms_norm(x, torch.ones(width, dtype=BF), d.NORM_EPS)
                assert ((o[f"a{i}"].double() - y).abs() <= 1.01 * R.HALF_BF16 * y.abs()).all()
            else:
                q, s = R.quantize(x.double(), 1)
            assert torch.equal(o[f"q{i}"].double(), q)
            # (roundings of 2^-24 in a scale: half of those in the sum of squares, at most d / 512 + 18
            # on the way of one square, and six more; 16 of them at these widths)
            assert ((o[f"s{i}"].double() - s).abs() <= 2.0 ** -20 * s).all()
        for i, L in enumerate(d.lin):
            k = list(d.act8).index(L["act"])
            ref, size, low, tb = R.linear(o[f"q{k}"], o[f"s{k}"], L["w8"].cpu(), L["w8s"].cpu(), o[f"a{k}"], L["a"].cpu(),
                                          L["b"].cpu(), o["gate"], L_.scale)
            bound = R.linear_bound(size, low, tb, ref, L["shape"].d_in, L_.rank, True)
            assert ((o[f"y{i}"].double() - ref).abs() <= bound).all()
        _check_logprobs(d.P.cpu().view(V_.B * V_.K, V_.V), o["tok"].view(-1), V_.temperature, o["lp"], o["ent"], o["ids"],
                        o["tlp"])
    assert any((out[0]["y0"] != o["y0"]).any() for o in out[1:])  # the steps' activations differ


def test_driver_graph_equals_eager_and_options_leave_the_rest():
    _, eager = _steps(graph=False)
    _, graph = _steps(graph=True)
    for a, b in zip(eager, graph):
        for k in a:
            assert torch.equal(a[k].view(torch.uint8) if a[k].dtype == R.F8 else a[k],
                               b[k].view(torch.uint8) if b[k].dtype == R.F8 else b[k]), k
    _, plain = _steps(graph=False, base="bf16", report=None)
    _, only = _steps(graph=False, base="bf16", report=0)
    for a, b, c in zip(eager, plain, only):
        for k in ("tok", "cnt", "nxt", "gate"):
            assert torch.equal(a[k], b[k]) and torch.equal(b[k], c[k])
        assert torch.equal(b["y0"], c["y0"]) and torch.equal(a["lp"], c["lp"])
