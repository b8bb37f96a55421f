"""uno_rms_norm_fp8's launch forms: rows whose shared memory lies at the border of what a launch
has without asking, each as the first call of a process; and many rows, which run with CTAs of
four warps."""
import os
import subprocess
import sys

import pytest
import torch

from diffusion_drafted_lossless_b200 import _lib
from tests import layers_ref as R
from tests.test_gpu_norm_fp8 import EPS, _norm, _same, _stat_bound, _x

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import sys, torch
from diffusion_drafted_lossless_b200 import _lib
dtype, d = getattr(torch, sys.argv[1]), int(sys.argv[2])
x, w = torch.ones((3, d), dtype=dtype, device="cuda"), torch.ones(d, dtype=dtype, device="cuda")
y = torch.zeros_like(x)
_lib.uno_rms_norm_fp8(x, w, 1e-6, out_y=y)
assert ((y - 1).abs() <= 1e-6).all()  # (1 / sqrt(1 + eps), half of eps below 1)
"""


@pytest.mark.parametrize("dtype,d", [("float32", 12272), ("float32", 12288), ("bfloat16", 24544), ("bfloat16", 24560),
                                     ("bfloat16", 24576)])
def test_first_call_of_a_process(dtype, d):
    r = subprocess.run([sys.executable, "-c", FIRST, dtype, str(d)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def _check(x, w, r, inplace):
    h, y, q, s = R.rms_norm(x, w, EPS, r)
    gq, gs, gres, gy = _norm(x, w, r, inplace=inplace)
    if r is not None:
        assert torch.equal(gres, h)
    _same(gq, q)
    tol = _stat_bound(x.shape[1], x.dtype) + x.shape[1] / 128 * R.F32 / 2  # (128 threads: four times as many adds)
    assert ((gs.double() - s).abs() <= tol * s).all()
    half = R.HALF_BF16 if x.dtype == BF else R.F32
    assert ((gy.double() - y).abs() <= (half + tol) * y.abs() * 1.01).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,d,res,inplace", [(592, 128, True, False), (600, 2576, True, True),
                                             (593, 4112, False, False), (700, 4112, True, False),
                                             (640, 1040, True, True), (600, 16, False, False)])
def test_many_rows(M, d, res, inplace, dtype):
    """From four rows an SM on: several turns of a CTA's 128 threads, the last of them partial."""
    assert M >= 4 * torch.cuda.get_device_properties(0).multi_processor_count
    x, w = _x(M, d, dtype, d), (1 + 0.2 * _x(1, d, F32, 1, False)[0]).to(dtype)
    _check(x, w, _x(M, d, dtype, 2) if res else None, inplace)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_rows_one_output_each(dtype):
    M, d = 600, 2576
    x, r, w = _x(M, d, dtype, 1), _x(M, d, dtype, 2), _x(1, d, dtype, 3)[0]
    full = _norm(x, w, r)
    for q, y in ((True, False), (False, True)):
        for a, b in zip(full, _norm(x, w, r, q=q, y=y)):
            assert b is None or torch.equal(a.float(), b.float())
    assert _lib.uno_read_device_status() == _lib.UNO_OK
