"""The operators of a model with an 8-bit frozen base around draft and verify, as perf cases.

Three operators, each with its plain form (elementary torch operations) and the calls of
this package that a user makes instead:
  norm       h = x + residual, RMS norm of h, e4m3 values with one scale per 128 columns
  quantize   e4m3 values of a matrix, one scale per 1 x 128 or per 128 x 128 block
  linear     y = (x_q x_s) (w_q w_s)^T, with the row-gated bf16 adapter where a rank is given
  logprobs   log probabilities of given tokens, entropy, the most probable alternatives
  train      the same rows with the gradient of both outputs
(quantize is how weights and un-normed activations reach the product; train is the
backward direction of logprobs.)

Where the module's `own` is false, `run` computes the plain form; where it is true, it
calls diffusion_drafted_lossless_b200.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128


def listed():
    return [
        # one sequence's block of 16 positions between two projections (hidden 4096): latency
        {"name": "norm_block16_4096", "op": "norm", "M": 16, "d": 4096, "dtype": "bf16", "residual": True, "y": True},
        # 8 sequences x 2048 tokens of a looped-3B prompt or training batch (hidden 2560)
        {"name": "norm_prompt_16384x2560", "op": "norm", "M": 16384, "d": 2560, "dtype": "bf16", "residual": True,
         "y": False},
        # the MLP's inner activations before the down projection, 64 sequences x block 16
        {"name": "quantize_mlp_1024x12288", "op": "quantize", "M": 1024, "d": 12288, "dtype": "f32", "block_rows": 1},
        # a base weight made 8-bit, as done at load time and after an adapter is merged
        {"name": "quantize_weight_9728x2560", "op": "quantize", "M": 9728, "d": 2560, "dtype": "bf16",
         "block_rows": 128},
        # one drafting sequence: a block of 16 rows through the q projection with its adapter
        {"name": "linear_q_m16", "op": "linear", "M": 16, "d_in": 4096, "d_out": 4096, "rank": 128, "block": 16,
         "y": "bf16"},
        # the flagship draft step: 64 sequences x block 16 through the gate projection
        {"name": "linear_gate_m1024", "op": "linear", "M": 1024, "d_in": 4096, "d_out": 12288, "rank": 128,
         "block": 16, "y": "bf16"},
        # a long prompt through the looped-3B up projection (no adapter on prompt rows)
        {"name": "linear_up_m8192", "op": "linear", "M": 8192, "d_in": 2560, "d_out": 9728, "rank": 0, "block": 8,
         "y": "bf16"},
        # the vocabulary head over 4 sequences x block 16: the weight is what has to be read
        {"name": "linear_head_m64", "op": "linear", "M": 64, "d_in": 4096, "d_out": 151936, "rank": 0, "block": 16,
         "y": "bf16"},
        # a ragged batch through an odd head in float32: no size is a multiple of a tile
        {"name": "linear_ragged_f32", "op": "linear", "M": 777, "d_in": 2576, "d_out": 1001, "rank": 0, "block": 8,
         "y": "f32"},
        # what a served step reports for one verified block: 20 alternatives for each position
        {"name": "logprobs_block16_top20", "op": "logprobs", "M": 16, "V": 151936, "dtype": "bf16", "top": 20,
         "temperature": 1.0, "skip": 0.0},
        # the whole looped-3B verify batch; positions behind the accepted prefix are left out
        {"name": "logprobs_looped_2048", "op": "logprobs", "M": 2048, "V": 166144, "dtype": "bf16", "top": 5,
         "temperature": 0.8, "skip": 0.4},
        # training on log probabilities with an entropy term, padding rows among the responses
        {"name": "train_1024", "op": "train", "M": 1024, "V": 151936, "dtype": "bf16", "temperature": 1.0,
         "skip": 0.1},
    ]


def _size(rng, lo, hi, multiple=1):
    """A size between lo and hi, spread over its logarithm, a multiple of `multiple`."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v) // multiple * multiple))


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear", "linear", "logprobs", "train"])
    if op == "norm":
        d = _size(rng, 256, 12288, 16)
        return {"op": op, "M": _size(rng, 1, min(16384, 40_000_000 // d)), "d": d,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "residual": rng.random() < 0.7,
                "y": rng.random() < 0.5}
    if op == "quantize":
        d = _size(rng, 256, 12288, 16)
        return {"op": op, "M": _size(rng, 1, min(16384, 24_000_000 // d)), "d": d,
                "dtype": rng.choice(["bf16", "f32"]), "block_rows": rng.choice([1, 128])}
    if op == "linear":
        d_in = _size(rng, 512, 12288, 16)
        d_out = _size(rng, 256, 16384)
        most = min(8192, int(2.0e11 / (d_in * d_out)))
        rank = rng.choice([0, 0, 8, 64, 128, 200])
        if rank:
            d_out = max(256, d_out // 8 * 8)
        return {"op": op, "M": _size(rng, 1, most), "d_in": d_in, "d_out": d_out, "rank": rank,
                "block": rng.choice([1, 8, 16]), "y": "bf16" if rank or rng.random() < 0.7 else "f32"}
    V = _size(rng, 2000, 166144)
    case = {"op": op, "M": _size(rng, 1, min(4096, 150_000_000 // V)), "V": V,
            "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "logprobs":
        case["top"] = rng.choice([0, 1, 5, 20, 32])
    case["temperature"] = rng.choice([1.0, 0.7, 1.3])
    case["skip"] = rng.choice([0.0, 0.3])
    return case


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _activations(M, d, g):
    """Normal draws with a few wide columns, as a residual stream has them."""
    x = torch.randn((M, d), generator=g, device="cuda")
    wide = torch.randint(0, d, (max(1, d // 256),), generator=g, device="cuda")
    x[:, wide] *= 12.0
    return x


def _blocks(x, rows):
    """x zero-padded to whole rows x 128 blocks: [row blocks, rows, column blocks, 128]."""
    M, d = x.shape
    pad = torch.nn.functional.pad(x, (0, -d % BLOCK, 0, -M % rows))
    return pad.view(pad.shape[0] // rows, rows, pad.shape[1] // BLOCK, BLOCK)


def _round_e4m3(t):
    """t (float64, at most 448 in size) rounded to e4m3, ties to even: 3 mantissa bits down to
    2^-6, steps of 2^-9 below."""
    _, e = torch.frexp(t)
    step = torch.ldexp(torch.ones_like(t), (e - 4).clamp_min(-9))
    return (torch.round(t / step) * step).to(torch.float32).to(torch.float8_e4m3fn)


def _quantize(x, rows, factor=None):
    """e4m3 values and float32 scales of x by rows x 128 blocks. A scale is the block's
    largest size / 448, at least 2^-126; a value is 448 x / that size, rounded once. In 64
    bits, since a value next to a border goes to the wrong side in 32. With `factor` [M, 1]
    the matrix is x * factor; the factor leaves the values as they are (rows = 1)."""
    M, d = x.shape
    b = _blocks(x.double(), rows)
    amax = b.abs().amax(dim=(1, 3), keepdim=True)
    f = torch.ones_like(amax) if factor is None else factor[:, :, None, None]
    amax = torch.maximum(amax, E4M3_MAX * 2.0 ** -126 / f)
    q = _round_e4m3(b * E4M3_MAX / amax)
    q = q.view(b.shape[0] * rows, -1)[:M, :d].contiguous()
    return q, (amax * f / E4M3_MAX).float().view(b.shape[0], b.shape[2])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    dev = torch.device("cuda")
    s = dict(case)
    op = case["op"]
    if op == "norm":
        M, d, t = case["M"], case["d"], _dtype(case["dtype"])
        s["x"] = _activations(M, d, g).mul_(0.5).to(t)
        s["res"] = _activations(M, d, g).to(t) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn((d,), generator=g, device=dev)).to(t)
        s["out_q"] = torch.empty((M, d), dtype=torch.float8_e4m3fn, device=dev)
        s["out_s"] = torch.empty((M, -(-d // BLOCK)), device=dev)
        s["out_res"] = torch.empty((M, d), dtype=t, device=dev) if case["residual"] else None
        s["out_y"] = torch.empty((M, d), dtype=t, device=dev) if case["y"] else None
    elif op == "quantize":
        M, d, t, r = case["M"], case["d"], _dtype(case["dtype"]), case["block_rows"]
        s["x"] = (_activations(M, d, g) if r == 1 else 0.02 * torch.randn((M, d), generator=g, device=dev)).to(t)
        s["out_q"] = torch.empty((M, d), dtype=torch.float8_e4m3fn, device=dev)
        s["out_s"] = torch.empty((-(-M // r), -(-d // BLOCK)), device=dev)
    elif op == "linear":
        M, d_in, d_out, r = case["M"], case["d_in"], case["d_out"], case["rank"]
        x = _activations(M, d_in, g).to(torch.bfloat16)
        s["xq"], s["xs"] = _quantize(x, 1)
        # (the weight in slabs of whole blocks: its 64-bit form would take gigabytes)
        parts = [_quantize((0.02 * torch.randn((min(16384, d_out - at), d_in), generator=g, device=dev))
                           .to(torch.bfloat16), BLOCK) for at in range(0, d_out, 16384)]
        s["wq"], s["ws"] = torch.cat([p[0].view(torch.uint8) for p in parts]).view(torch.float8_e4m3fn), \
            torch.cat([p[1] for p in parts])
        s["y_out"] = torch.empty((M, d_out), dtype=_dtype(case["y"]), device=dev)
        s["x"] = s["a"] = s["b"] = s["gate"] = None
        s["scale"] = 2.0
        if r:
            s["x"] = x
            s["a"] = (0.02 * torch.randn((r, d_in), generator=g, device=dev)).to(torch.bfloat16)
            s["b"] = (0.02 * torch.randn((d_out, r), generator=g, device=dev)).to(torch.bfloat16)
            # position 0 of each block is an exact row: no adapter there
            s["gate"] = (torch.arange(M, device=dev) % case["block"] != 0).float() if case["block"] > 1 \
                else torch.ones((M,), device=dev)
    else:
        M, V = case["M"], case["V"]
        s["logits"] = (3.0 * torch.randn((M, V), generator=g, device=dev)).to(_dtype(case["dtype"]))
        # ids behind the tokenizer's own are never produced: the model's head masks them
        s["logits"][:, V - V // 500:] = -math.inf
        tok = torch.randint(0, V - V // 500, (M,), generator=g, device=dev, dtype=torch.int32)
        # most given tokens are probable ones
        some = torch.randint(0, V - V // 500, (M, 64), generator=g, device=dev)
        best = some.gather(1, s["logits"].gather(1, some).float().argmax(1, keepdim=True))[:, 0].int()
        tok = torch.where(torch.rand((M,), generator=g, device=dev) < 0.7, best, tok)
        s["tokens"] = torch.where(torch.rand((M,), generator=g, device=dev) < case["skip"],
                                  torch.full_like(tok, -1), tok)
        s["logprob"] = torch.empty((M,), device=dev)
        s["entropy"] = torch.empty((M,), device=dev)
        if op == "logprobs":
            k = case["top"]
            s["ids"] = torch.empty((M, k), dtype=torch.int32, device=dev) if k else None
            s["top_lp"] = torch.empty((M, k), device=dev) if k else None
        else:
            s["stats"] = torch.empty((M, 2), device=dev)
            s["grad"] = torch.empty_like(s["logits"])
            s["g_lp"] = torch.randn((M,), generator=g, device=dev) / M
            s["g_ent"] = 0.01 * torch.rand((M,), generator=g, device=dev) / M
    return s


# ---------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------
EPS = 1e-6


def _plain_norm(s):
    x = s["x"]
    h = x if s["res"] is None else (x.float() + s["res"].float()).to(x.dtype)
    # 64 bits: the values next to a border of e4m3 have to go to the right side
    hd = h.double()
    u = hd * s["weight"].double()
    rstd = 1.0 / torch.sqrt((hd * hd).mean(1, keepdim=True) + EPS)
    q, sc = _quantize(u, 1, rstd)
    return {"q": q, "scale": sc, "residual": None if s["res"] is None else h,
            "y": (u * rstd).to(x.dtype) if s["out_y"] is not None else None}


def _dequantize(q, sc, rows):
    M, d = q.shape
    full = sc.repeat_interleave(BLOCK, 1)[:, :d]
    return q.float() * (full if rows == 1 else full.repeat_interleave(rows, 0)[:M])


def _plain_linear(s):
    y = _dequantize(s["xq"], s["xs"], 1) @ _dequantize(s["wq"], s["ws"], BLOCK).T
    if s["rank"]:
        t = s["x"].float() @ s["a"].float().T
        y = y + (s["scale"] * s["gate"])[:, None] * (t @ s["b"].float().T)
    return {"y": y.to(s["y_out"].dtype)}


def _plain_rows(s):
    """Per row: kept or not, log softmax, probabilities."""
    keep = (s["tokens"] >= 0) & (s["tokens"] < s["V"])
    z = s["logits"].float() / s["temperature"]
    z = z - z.amax(1, keepdim=True)
    lp = z - torch.exp(z).sum(1, keepdim=True).log()
    p = torch.exp(lp)
    ent = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    at = lp.gather(1, s["tokens"].clamp(0, s["V"] - 1).long()[:, None])[:, 0]
    zero = torch.zeros_like(at)
    return keep, lp, p, torch.where(keep, at, zero), torch.where(keep, ent, zero), ent


def _plain_logprobs(s):
    keep, lp, _, at, ent, _ = _plain_rows(s)
    out = {"logprob": at, "entropy": ent}
    if s["top"]:
        # values in an order of whole numbers, the lower id first among equal ones
        bits = (s["logits"].float() + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -(bits + 2 ** 31) - 1, bits)
        ids = torch.arange(s["V"], device=bits.device)
        best = torch.topk(order * 2 ** 31 + (s["V"] - 1 - ids), s["top"], dim=1).values
        ids = s["V"] - 1 - best % 2 ** 31
        top = lp.gather(1, ids)
        shown = keep[:, None] & (top > -math.inf)
        out["top_ids"] = torch.where(shown, ids, torch.full_like(ids, -1)).int()
        out["top_logprobs"] = torch.where(shown, top, torch.full_like(top, -math.inf))
    return out


def _plain_train(s):
    keep, lp, p, at, ent, h = _plain_rows(s)
    gl, ge = s["g_lp"][:, None], s["g_ent"][:, None]
    g = -gl * p - ge * torch.where(p > 0, p * (lp + h[:, None]), torch.zeros_like(p))
    g.scatter_add_(1, s["tokens"].clamp(0, s["V"] - 1).long()[:, None], gl)
    g = torch.where(keep[:, None], g / s["temperature"], torch.zeros_like(g))
    return {"logprob": at, "entropy": ent, "grad": g.to(s["logits"].dtype)}


def run(state):
    s, op = state, state["op"]
    if own:
        import diffusion_drafted_lossless_b200 as uno
        if op == "norm":
            uno.uno_rms_norm_fp8(s["x"], s["weight"], EPS, s["out_q"], s["out_s"], residual=s["res"],
                                 out_residual=s["out_res"], out_y=s["out_y"])
            return {"q": s["out_q"], "scale": s["out_s"], "residual": s["out_res"], "y": s["out_y"]}
        if op == "quantize":
            uno.uno_fp8_quantize(s["x"], s["out_q"], s["out_s"], block_rows=s["block_rows"])
            return {"q": s["out_q"], "scale": s["out_s"]}
        if op == "linear":
            uno.uno_fp8_gated_lora_linear(s["xq"], s["xs"], s["wq"], s["ws"], s["y_out"], x=s["x"], lora_a=s["a"],
                                          lora_b=s["b"], row_gate=s["gate"], scale=s["scale"])
            return {"y": s["y_out"]}
        if op == "logprobs":
            uno.uno_token_logprobs(s["logits"], s["tokens"], s["logprob"], temperature=s["temperature"],
                                   out_entropy=s["entropy"], out_top_ids=s["ids"], out_top_logprobs=s["top_lp"])
            out = {"logprob": s["logprob"], "entropy": s["entropy"]}
            return out if s["ids"] is None else {**out, "top_ids": s["ids"], "top_logprobs": s["top_lp"]}
        uno.uno_token_logprobs(s["logits"], s["tokens"], s["logprob"], temperature=s["temperature"],
                               out_entropy=s["entropy"], out_stats=s["stats"])
        uno.uno_token_logprobs_grad(s["logits"], s["tokens"], s["stats"], s["grad"], grad_logprob=s["g_lp"],
                                    entropy=s["entropy"], grad_entropy=s["g_ent"], temperature=s["temperature"])
        return {"logprob": s["logprob"], "entropy": s["entropy"], "grad": s["grad"]}
    if op == "norm":
        return _plain_norm(s)
    if op == "quantize":
        q, sc = _quantize(s["x"], s["block_rows"])
        return {"q": q, "scale": sc}
    if op == "linear":
        return _plain_linear(s)
    return _plain_logprobs(s) if op == "logprobs" else _plain_train(s)


# ---------------------------------------------------------------------------------------
# what a pass cannot do without, and the exact values
# ---------------------------------------------------------------------------------------
def work(case):
    op, M = case["op"], case["M"]
    if op in ("norm", "quantize"):
        d, e = case["d"], 4 if case["dtype"] == "f32" else 2
        if op == "quantize":
            return {"bytes": M * d * (e + 1) + 4 * -(-M // case["block_rows"]) * -(-d // BLOCK), "flops": 3 * M * d}
        return {"bytes": M * d * (e * (1 + 2 * case["residual"] + case["y"]) + 1) + 4 * M * -(-d // BLOCK) + e * d,
                "flops": 6 * M * d}
    if op == "linear":
        i, o, r = case["d_in"], case["d_out"], case["rank"]
        kb = -(-i // BLOCK)
        nbytes = M * i + o * i + 4 * M * kb + 4 * -(-o // BLOCK) * kb + M * o * (4 if case["y"] == "f32" else 2)
        flops = 2 * M * i * o
        if r:
            gated = M - -(-M // case["block"]) if case["block"] > 1 else M
            nbytes += 2 * (M * i + r * i + o * r) + 4 * M
            flops += 2 * gated * r * (i + o)
        return {"bytes": nbytes, "flops": flops}
    V, e = case["V"], 4 if case["dtype"] == "f32" else 2
    rows = M * (1 - case["skip"])  # rows left out need not be read
    if op == "logprobs":
        return {"bytes": int(rows * V * e + M * (12 + 8 * case["top"])), "flops": int(rows * V * 5)}
    return {"bytes": int((rows + M) * V * e + M * 20), "flops": int(rows * V * 12)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x, w = s["x"].double(), s["weight"].double()
        # (a sum of two stored values is exact in 64 bits or rounds the same way)
        h = x if s["res"] is None else (x + s["res"].double()).to(s["x"].dtype).double()
        rstd = (h.square().sum(1, keepdim=True) / case["d"] + EPS).rsqrt()
        # a row's rstd is in its scales and cancels in its values
        q, sc = _exact_blocks(h * w, 1)
        return {"q": q, "scale": sc * rstd, "residual": None if s["res"] is None else h,
                "y": h * w * rstd if s["out_y"] is not None else None}
    if op == "quantize":
        q, sc = _exact_blocks(s["x"].double(), case["block_rows"])
        return {"q": q, "scale": sc}
    if op == "linear":
        d_in, d_out, M = case["d_in"], case["d_out"], case["M"]
        col = torch.arange(d_in, device="cuda") // BLOCK
        x = s["xq"].double() * s["xs"].double()[:, col]
        y = torch.empty((M, d_out), dtype=torch.float64, device="cuda")
        for at in range(0, d_out, 8192):
            row = torch.arange(at, min(at + 8192, d_out), device="cuda")
            w = s["wq"].view(torch.uint8)[row].view(torch.float8_e4m3fn).double()
            w *= s["ws"].double()[row // BLOCK][:, col]
            y[:, at:at + 8192] = x @ w.T
        if case["rank"]:
            low = (s["x"].double() @ s["a"].double().T) * s["gate"].double()[:, None]
            y += s["scale"] * (low @ s["b"].double().T)
        return {"y": y}
    return _exact_rows(case, s)


def _exact_blocks(y, rows):
    """e4m3 values (from the 256 codes' own values, by nearest neighbour, ties to the even
    code) and scales of a float64 matrix."""
    M, d = y.shape
    amax = torch.zeros((-(-M // rows), -(-d // BLOCK)), dtype=torch.float64, device=y.device)
    for c in range(amax.shape[1]):
        m = y[:, c * BLOCK:(c + 1) * BLOCK].abs().amax(1)
        m = torch.nn.functional.pad(m, (0, -M % rows))
        amax[:, c] = m.view(-1, rows).amax(1)
    amax.clamp_min_(E4M3_MAX * 2.0 ** -126)
    codes = torch.arange(127, dtype=torch.uint8, device=y.device).view(torch.float8_e4m3fn).double()
    r = torch.arange(M, device=y.device) // rows
    c = torch.arange(d, device=y.device) // BLOCK
    q = torch.empty((M, d), dtype=torch.float8_e4m3fn, device=y.device)
    for at in range(0, M, 2048):
        part = y[at:at + 2048]
        t = part * E4M3_MAX / amax[r[at:at + 2048]][:, c]
        up = torch.searchsorted(codes, t.abs().contiguous()).clamp(1, 126)
        below, above = codes[up - 1], codes[up]
        mid = (below + above) / 2
        take_up = (t.abs() > mid) | ((t.abs() == mid) & (up % 2 == 0))
        v = torch.where(take_up, above, below) * torch.sign(t)
        q.view(torch.uint8)[at:at + 2048] = v.float().to(torch.float8_e4m3fn).view(torch.uint8)
    return q, amax / E4M3_MAX


def _exact_rows(case, s):
    M, V, T = case["M"], case["V"], case["temperature"]
    out = {"logprob": torch.zeros((M,), dtype=torch.float64, device="cuda"),
           "entropy": torch.zeros((M,), dtype=torch.float64, device="cuda")}
    train = case["op"] == "train"
    k = 0 if train else case["top"]
    if train:
        out["grad"] = torch.zeros((M, V), dtype=torch.float64, device="cuda")
    if k:
        out["top_ids"] = torch.full((M, k), -1, dtype=torch.int32, device="cuda")
        out["top_logprobs"] = torch.full((M, k), -math.inf, dtype=torch.float64, device="cuda")
    rows = torch.nonzero((s["tokens"] >= 0) & (s["tokens"] < V))[:, 0]
    for part in rows.split(128):
        lp = torch.log_softmax(s["logits"][part].double() / T, dim=1)
        p = lp.exp()
        ent = torch.special.entr(p).sum(1)
        tok = s["tokens"][part].long()[:, None]
        out["logprob"][part] = lp.gather(1, tok)[:, 0]
        out["entropy"][part] = ent
        if train:
            onehot = torch.zeros_like(p).scatter_(1, tok, 1.0)
            d_ent = torch.special.entr(p) - p * ent[:, None]
            out["grad"][part] = (s["g_lp"][part].double()[:, None] * (onehot - p) +
                                 s["g_ent"][part].double()[:, None] * d_ent) / T
        if k:
            v, i = torch.sort(s["logits"][part].float(), dim=1, descending=True, stable=True)
            fine = v[:, :k] > -math.inf
            i = i[:, :k]
            out["top_ids"][part] = torch.where(fine, i, -torch.ones_like(i)).int()
            out["top_logprobs"][part] = lp.gather(1, i).masked_fill(~fine, -math.inf)
    return out
