"""Linear draft/verify step driver: the decode step's operations chained on one stream.

Per step (LoopUno project page, "How it works": a block is drafted in one forward with the
LoRA on the noise positions only, the unmodified model verifies it, the longest correct
prefix is kept and the first position is the exact AR token):
  1. uno_block_noise: the block's input tokens — position 0 is the token carried from the
     previous step (its correction token; -1 when every draft was accepted, or at the
     first step), positions 1..K-1 random_uniform noise — and the row gate (0 at
     position 0, 1 on the noise rows);
  2. uno_gated_lora_linear over the seven projections of one decoder layer on the block's
     B x K rows, gated by that row gate;
  3. uno_block_verify with pos0_tokens = the carried tokens (an entry < 0 draws x_0 from
     p_0), drafts sampled in the kernel;
  4. the correction token becomes the next step's carried token.
There is no model: the projections' activations and the verifier / drafter logits are
seeded synthetic inputs of the right shapes (a model's forward would compute them from the
noised tokens). Each step's activations and uniforms come from a small pool and are copied
into the step's input buffers before its launches, so consecutive steps compute on
different data. Every step is the same sequence of launches, so it can be captured once in
a CUDA graph and replayed.
tokens_per_forward() is the mean accepted count per sequence and step.

With base="fp8" step 2 runs on an e4m3 copy of the base weights (made once, 128 x 128 blocks):
the step's hidden activations go through uno_rms_norm_fp8 (unit weight), which the q, k, v,
gate and up projections read; o and down read their inputs through uno_fp8_quantize; and the
projections are uno_fp8_gated_lora_linear, their adapters on the bf16 activations.
With report=n (0 to 32) a step ends with uno_token_logprobs over the verifier's rows: the log
probability of each emitted token, the entropy of its position and the n most probable
alternatives; positions behind the accepted prefix are left out.
"""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

from . import _lib
from . import workloads as W


class DraftVerifyDriver:
    NORMED = ("q", "k", "v", "gate", "up")  # projections that read the normed hidden activations
    NORM_EPS = 1e-6

    def __init__(self, linears: W.GatedLoraWorkload, verify: W.VerifyWorkload, pool: int = 3, device: str = "cuda",
                 base: str = "bf16", report: int | None = None):
        v = verify
        assert linears.M == v.B * v.K, "the projections run on the block's B x K rows"
        assert base in ("bf16", "fp8"), "the base weights are bf16 or e4m3"
        self.base, self.report = base, report
        self.lw, self.v, self.dev = linears, v, torch.device(device)
        bf = torch.bfloat16

        def t(a):
            return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(bf).to(self.dev)

        self.lin = []
        self.x = {}  # the step's activations, one buffer per input width (read by the captured launches)
        for sh in linears.shapes:
            inp = W.linear_inputs(linears, sh)
            ws = torch.empty(_lib.uno_gated_lora_linear_workspace_size(linears.M, sh.d_in, sh.d_out, linears.rank),
                             dtype=torch.uint8, device=self.dev)
            if sh.d_in not in self.x:
                self.x[sh.d_in] = torch.empty((linears.M, sh.d_in), dtype=bf, device=self.dev)
            self.lin.append(dict(shape=sh, x=self.x[sh.d_in], w0=t(inp["w0"]), a=t(inp["a"]), b=t(inp["b"]), ws=ws,
                                 y=torch.empty((linears.M, sh.d_out), dtype=bf, device=self.dev)))
        if base == "fp8":
            self._make_fp8()
        # pool entry s draws its activations from the workload's seed + s (entry 0 is the
        # workload's own X); they stay on the device and are copied in per step
        self.pool_x = []
        for s in range(pool):
            lw = dataclasses.replace(linears, seed=linears.seed + s)
            self.pool_x.append({d: t(W.linear_inputs(lw, next(sh for sh in linears.shapes if sh.d_in == d))["x"])
                                for d in self.x})
        P, Q = W.verify_logits(v)
        self.P_host, self.Q_host = P, Q
        self.P = t(P).view(v.B, v.K, v.V)
        self.Q = t(Q).view(v.B, v.K, v.V)
        self.pool_u = [W.uniforms(v.seed + 2000 + s, (v.B, v.K, 3)) for s in range(pool)]
        self.pool_noise = [W.uniforms(v.seed + 3000 + s, (v.B, v.K)) for s in range(pool)]
        self.u = torch.empty((v.B, v.K, 3), device=self.dev)
        self.u_noise = torch.empty((v.B, v.K), device=self.dev)
        self.carry = torch.full((v.B, v.K), -1, dtype=torch.int32, device=self.dev)  # column 0 is read
        self.noised = torch.empty((v.B, v.K), dtype=torch.int32, device=self.dev)
        self.gate = torch.empty((v.B * v.K,), device=self.dev)
        self.pos0 = torch.empty((v.B,), dtype=torch.int32, device=self.dev)
        self.tokens = torch.empty((v.B, v.K), dtype=torch.int32, device=self.dev)
        self.count = torch.empty((v.B,), dtype=torch.int32, device=self.dev)
        self.next = torch.empty((v.B,), dtype=torch.int32, device=self.dev)
        self.vws = torch.empty(_lib.uno_block_verify_workspace_size(v.B, v.K, v.V, v.top_k, v.top_p),
                               dtype=torch.uint8, device=self.dev)
        if report is not None:
            n = v.B * v.K
            self.logprob = torch.empty((n,), device=self.dev)
            self.entropy = torch.empty((n,), device=self.dev)
            self.top_ids = torch.empty((n, report), dtype=torch.int32, device=self.dev) if report else None
            self.top_logprobs = torch.empty((n, report), device=self.dev) if report else None
        self.steps = 0
        self.graph = None

    def _make_fp8(self):
        """e4m3 base weights, and the step's e4m3 activations: one pair for the normed hidden
        activations, one for each width that is read as it is."""
        M, f8 = self.lw.M, torch.float8_e4m3fn

        def pair(rows, cols, block_rows):
            return (torch.empty((rows, cols), dtype=f8, device=self.dev),
                    torch.empty((rows if block_rows == 1 else _lib._blocks(rows), _lib._blocks(cols)), device=self.dev))

        self.act8 = {}  # (normed, width) -> dict of what the projections read
        for L in self.lin:
            sh = L["shape"]
            L["w8"], L["w8s"] = pair(sh.d_out, sh.d_in, 128)
            _lib.uno_fp8_quantize(L["w0"], L["w8"], L["w8s"], block_rows=128)
            L["w0"] = None
            key = L["act"] = (sh.name in self.NORMED, sh.d_in)
            if key not in self.act8:
                q, s = pair(M, sh.d_in, 1)
                bf = torch.bfloat16
                self.act8[key] = dict(x=L["x"], q=q, s=s, y=torch.empty_like(L["x"]) if key[0] else L["x"],
                                      weight=torch.ones((sh.d_in,), dtype=bf, device=self.dev))
            L["ws"] = torch.empty(_lib.uno_fp8_gated_lora_linear_workspace_size(M, sh.d_in, sh.d_out, self.lw.rank),
                                  dtype=torch.uint8, device=self.dev)

    def pool_inputs(self, s: int):
        """The uniforms of step s (verify [B, K, 3], noise [B, K])."""
        return self.pool_u[s % len(self.pool_u)], self.pool_noise[s % len(self.pool_noise)]

    def pool_linear_workload(self, s: int) -> W.GatedLoraWorkload:
        """The workload whose X (W.linear_inputs) step s's projections read."""
        return dataclasses.replace(self.lw, seed=self.lw.seed + s % len(self.pool_x))

    def _ops(self):
        v, lw = self.v, self.lw
        _lib.uno_block_noise(self.carry, self.u_noise, v.V, self.noised, self.gate)
        if self.base == "fp8":
            for (normed, _), a in self.act8.items():
                if normed:
                    _lib.uno_rms_norm_fp8(a["x"], a["weight"], self.NORM_EPS, a["q"], a["s"], out_y=a["y"])
                else:
                    _lib.uno_fp8_quantize(a["x"], a["q"], a["s"])
            for L in self.lin:
                a = self.act8[L["act"]]
                _lib.uno_fp8_gated_lora_linear(a["q"], a["s"], L["w8"], L["w8s"], L["y"], x=a["y"], lora_a=L["a"],
                                               lora_b=L["b"], row_gate=self.gate, scale=lw.scale, workspace=L["ws"])
        else:
            for L in self.lin:
                _lib.uno_gated_lora_linear(L["x"], L["w0"], L["a"], L["b"], self.gate, lw.scale, L["y"],
                                           workspace=L["ws"])
        self.pos0.copy_(self.noised[:, 0])
        _lib.uno_block_verify(self.P, self.Q, v.temperature, v.top_k, v.top_p, self.u, self.tokens, self.count,
                              self.next, pos0_tokens=self.pos0, workspace=self.vws)
        self.carry[:, 0].copy_(self.next)
        if self.report is not None:
            _lib.uno_token_logprobs(self.P.view(v.B * v.K, v.V), self.tokens.view(-1), self.logprob, v.temperature,
                                    self.entropy, None, self.top_ids, self.top_logprobs)

    def capture(self):
        """Capture one step in a CUDA graph; later steps replay it."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self._ops()
        self.graph = g

    def step(self):
        """One decode step; returns (tokens [B, K], count [B], next [B]) on the device."""
        u, un = self.pool_inputs(self.steps)
        self.u.copy_(torch.from_numpy(u))
        self.u_noise.copy_(torch.from_numpy(un))
        for d, x in self.pool_x[self.steps % len(self.pool_x)].items():
            self.x[d].copy_(x)
        if self.graph is not None:
            self.graph.replay()
        else:
            self._ops()
        self.steps += 1
        return self.tokens, self.count, self.next

    @staticmethod
    def tokens_per_forward(counts) -> float:
        return float(np.mean([np.asarray(c).mean() for c in counts]))
