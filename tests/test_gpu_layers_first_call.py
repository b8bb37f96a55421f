"""The first calls of a process, made inside a graph capture: nothing that the library looks up
or sets on its first use may break the capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
from diffusion_drafted_lossless_b200 import _lib
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
M, d, V, r = 24, 512, 5000, 16
g = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn((M, d), generator=g, device="cuda").to(BF)
w = torch.randn((V, d), generator=g, device="cuda").to(BF)
a = torch.randn((r, d), generator=g, device="cuda").to(BF)
b = torch.randn((V, r), generator=g, device="cuda").to(BF)
nw, gate = torch.ones(d, dtype=BF, device="cuda"), torch.ones(M, device="cuda")
tok = torch.arange(M, dtype=torch.int32, device="cuda")

def outputs():
    e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")
    return dict(wq=e(V, d, t=F8), ws=e(-(-V // 128), 4), xq=e(M, d, t=F8), xs=e(M, 4), y=e(M, d, t=BF),
                lg=e(M, V, t=BF), lp=e(M), ent=e(M), st=e(M, 2), ids=e(M, 3, t=torch.int32), tl=e(M, 3), gr=e(M, V, t=BF),
                work=torch.empty(_lib.uno_fp8_gated_lora_linear_workspace_size(M, d, V, r), dtype=torch.uint8, device="cuda"))

def calls(o):
    _lib.uno_fp8_quantize(w, o["wq"], o["ws"], 128)
    _lib.uno_rms_norm_fp8(x, nw, 1e-6, o["xq"], o["xs"], out_y=o["y"])
    _lib.uno_fp8_gated_lora_linear(o["xq"], o["xs"], o["wq"], o["ws"], o["lg"], x=o["y"], lora_a=a, lora_b=b, row_gate=gate,
                                   scale=0.5, workspace=o["work"])
    _lib.uno_token_logprobs(o["lg"], tok, o["lp"], 1.0, o["ent"], o["st"], o["ids"], o["tl"])
    _lib.uno_token_logprobs_grad(o["lg"], tok, o["st"], o["gr"], grad_logprob=gate, entropy=o["ent"], grad_entropy=gate)

one, two = outputs(), outputs()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls(one)
graph.replay()
calls(two)
torch.cuda.synchronize()
for k in one:
    if k != "work":
        p, q = one[k], two[k]
        assert torch.equal(p.view(torch.uint8) if p.dtype == F8 else p, q.view(torch.uint8) if q.dtype == F8 else q), k
assert _lib.uno_read_device_status() == _lib.UNO_OK
print("captured")
"""


def test_first_calls_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
