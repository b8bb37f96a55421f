"""Plain 64-bit forms of the operators of include/uno_layers.h, on the CPU: what the tests
hold the kernels to. Elementary torch operations on float64 tensors."""
import math

import torch

F8 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126

# the 127 finite non-negative e4m3 values in ascending order (code 126 is 448)
CODES = torch.arange(127, dtype=torch.uint8).view(F8).double()
HALF_BF16 = 2.0 ** -8   # half a step of bf16, relative
F32 = 2.0 ** -24        # and of float32


def nearest_e4m3(t):
    """t (float64) to the nearest e4m3 value, ties to the even code, as float64; NaN stays."""
    a = t.abs().clamp(max=E4M3_MAX)
    up = torch.searchsorted(CODES, a.nan_to_num(0.0).contiguous()).clamp(1, 126)
    lo, hi = CODES[up - 1], CODES[up]
    mid = (lo + hi) / 2
    v = torch.where((a > mid) | ((a == mid) & (up % 2 == 0)), hi, lo)
    return torch.where(torch.isnan(t), t, torch.copysign(v, t))


def pad_blocks(x, rows):
    M, d = x.shape
    p = torch.nn.functional.pad(x, (0, -d % 128, 0, -M % rows))
    return p.view(p.shape[0] // rows, rows, p.shape[1] // 128, 128)


def quantize(x, rows, factor=None):
    """(values as float64 [M, d], scales float64) of a float64 matrix; factor [M] per row
    (rows = 1) goes to the scales."""
    M, d = x.shape
    b = pad_blocks(x, rows)
    a = b.abs().nan_to_num(nan=0.0, posinf=math.inf).amax(dim=(1, 3))
    f = torch.ones_like(a) if factor is None else factor[:, None].expand_as(a)
    top = torch.maximum(a, E4M3_MAX * MIN_SCALE / f)
    q = nearest_e4m3(b * E4M3_MAX / top[:, None, :, None])
    return q.view(b.shape[0] * rows, -1)[:M, :d], top * f / E4M3_MAX


def rms_norm(x, weight, eps, residual=None):
    """x, residual, weight in their storage dtype -> (h stored, y, values, scales) in float64."""
    h = x if residual is None else (x.double() + residual.double()).to(x.dtype)
    hd = h.double()
    u = hd * weight.double()
    rstd = 1.0 / torch.sqrt((hd * hd).mean(1) + eps)
    q, s = quantize(u, 1, rstd)
    return h, u * rstd[:, None], q, s


def expand_scales(s, rows, M, d):
    return s.double().repeat_interleave(128, 1)[:, :d].repeat_interleave(rows, 0)[:M]


def linear(xq, xs, wq, ws, x=None, a=None, b=None, gate=None, scale=1.0):
    """(y, sum of the sizes of base products, sum of the sizes of adapter products, |T| |B|)
    in float64."""
    X = xq.double() * expand_scales(xs, 1, *xq.shape)
    W = wq.double() * expand_scales(ws, 128, *wq.shape)
    y, size = X @ W.T, X.abs() @ W.abs().T
    low = torch.zeros_like(y)
    tb = torch.zeros_like(y)
    if a is not None and gate is not None:
        sg = (scale * gate.double())[:, None]
        on = sg != 0
        t = x.double() @ a.double().T
        ta = x.double().abs() @ a.double().abs().T
        term = torch.where(on, sg * (t @ b.double().T), torch.zeros_like(y))
        y = y + term
        low = torch.where(on, sg.abs() * (ta @ b.double().abs().T), torch.zeros_like(y))
        tb = torch.where(on, sg.abs() * (t.abs() @ b.double().abs().T), torch.zeros_like(y))
    return y, size, low, tb


def linear_bound(size, low, tb, y, d_in, rank, bf16):
    """How far a kernel's y may be from the exact one. A K block is four tensor-core steps of
    32 products added to a float32 sum; a step's terms are aligned to its largest and kept to
    at least 23 bits, so each of its 33 terms is off by at most 2^-23 of the largest, and the
    largest is at most the sum of sizes: 4 x 33 x 2^-23. Then one float32 multiply-add for
    each block and two roundings of its factor. The adapter: the same over X A^T (64 columns
    a block) and T B^T, and T's rounding to bf16. Then y's own rounding."""
    nk = -(-d_in // 128)
    base = (132 * 2.0 ** -23 + (nk + 3) * F32) * size
    low_blocks = -(-d_in // 64) + -(-max(rank, 1) // 64)
    adapter = (264 * 2.0 ** -23 + (low_blocks + nk + 4) * F32) * low + HALF_BF16 * 1.01 * tb
    out = (HALF_BF16 if bf16 else F32) * y.abs()
    return (base + adapter) * 1.01 + out + 1e-37


def logprobs(logits, tokens, T):
    """Rows' float64 log softmax, and (logprob, entropy, kept) by the entry point's rules."""
    N, V = logits.shape
    keep = torch.ones(N, dtype=torch.bool) if tokens is None else (tokens >= 0) & (tokens < V)
    x = logits.double()
    mx = x.amax(1)
    empty = mx == -math.inf
    z = (x - torch.where(empty, torch.zeros_like(mx), mx)[:, None]) / T
    logs = torch.where(empty, torch.zeros_like(mx), torch.exp(z).sum(1).log())
    lp = z - logs[:, None]
    p = torch.exp(lp)
    ent = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    at = None
    if tokens is not None:
        at = lp.gather(1, tokens.clamp(0, V - 1).long()[:, None])[:, 0]
        at = torch.where(keep, at, torch.zeros_like(at))
    return {"lp": lp, "p": p, "keep": keep, "empty": empty, "max": mx, "logs": logs, "logprob": at,
            "entropy": torch.where(keep & ~empty, ent, torch.zeros_like(ent)), "h": ent}


def top(logits, r, k):
    """(ids, log probabilities) by value descending, id ascending; (-1, -inf) beyond."""
    N, V = logits.shape
    v, i = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    kk = min(k, V)
    ids = torch.full((N, k), -1, dtype=torch.int64)
    lps = torch.full((N, k), -math.inf, dtype=torch.float64)
    fine = (v[:, :kk] > -math.inf) & r["keep"][:, None]
    ids[:, :kk] = torch.where(fine, i[:, :kk], torch.full_like(i[:, :kk], -1))
    lps[:, :kk] = torch.where(fine, r["lp"].gather(1, i[:, :kk]), torch.full((N, kk), -math.inf, dtype=torch.float64))
    return ids, lps


def logprobs_grad(logits, tokens, T, g_lp=None, g_ent=None):
    r = logprobs(logits, tokens, T)
    lp, p = r["lp"], r["p"]
    g = torch.zeros_like(p)
    if g_lp is not None:
        one = torch.zeros_like(p).scatter_(1, tokens.clamp(0, p.shape[1] - 1).long()[:, None], 1.0)
        g += g_lp.double()[:, None] * (one - p)
    if g_ent is not None:
        g -= g_ent.double()[:, None] * torch.where(p > 0, p * (lp + r["h"][:, None]), torch.zeros_like(p))
    return torch.where((r["keep"] & ~r["empty"])[:, None], g / T, torch.zeros_like(g)), r


def adds(V):
    """Most additions one after another in a thread's share of a row, and across the block."""
    return V / 512 + 8 + 20


def logs_bound(V):
    """Error of log s: the exponentials' own (2^-22, and 2^-23 for each octave below the
    maximum where the weight lies, at most about 24) and one rounding for each addition."""
    return (4 + 2 * 24 + adds(V)) * F32
