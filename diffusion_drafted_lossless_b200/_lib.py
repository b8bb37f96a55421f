"""ctypes binding of libuno.so (include/uno.h, include/uno_layers.h). Argument marshalling only.

Each function has the C entry point's name and takes torch tensors (device memory) where
the C ABI takes device pointers; it checks shapes/dtypes enough to build the call, passes
`torch.cuda.current_stream()` unless a stream is given, and raises UnoError on any status
other than UNO_OK. All computation happens in the library's CUDA kernels: there is no
fallback path, and a missing or unloadable libuno.so is an error.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from pathlib import Path

import torch

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libuno.so"

UNO_OK, UNO_ERR_INVALID_ARG, UNO_ERR_UNSUPPORTED, UNO_ERR_CUDA, UNO_ERR_TIMEOUT, UNO_ERR_WORKSPACE = range(6)
UNO_BF16, UNO_F32 = 0, 1

EXPORTED = (
    "uno_status_string", "uno_last_error_string", "uno_version", "uno_read_device_status",
    "uno_gated_lora_linear_workspace_size", "uno_gated_lora_linear",
    "uno_block_verify_workspace_size", "uno_block_verify_min_workspace_size", "uno_block_verify",
    "uno_block_verify_noalloc",
    "uno_tv_loss_workspace_size", "uno_tv_loss", "uno_block_noise",
)
# include/uno_layers.h
EXPORTED_LAYERS = (
    "uno_rms_norm_fp8", "uno_fp8_quantize", "uno_fp8_gated_lora_linear_workspace_size", "uno_fp8_gated_lora_linear",
    "uno_token_logprobs", "uno_token_logprobs_grad",
)


class UnoError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{_status_name(status)}: {detail}")


_lib = None
_vp, _sz, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


def load(path: str | os.PathLike | None = None) -> ctypes.CDLL:
    """Load libuno.so (build it first with `python -m diffusion_drafted_lossless_b200.build`)."""
    global _lib
    if _lib is not None:
        return _lib
    p = Path(path) if path else LIB_PATH
    if not p.exists():
        raise RuntimeError(f"{p} is missing: build it with `python -m diffusion_drafted_lossless_b200.build` "
                           "(the CUDA library is required; there is no fallback)")
    lib = ctypes.CDLL(str(p))
    lib.uno_status_string.restype = ctypes.c_char_p
    lib.uno_status_string.argtypes = [ctypes.c_int]
    lib.uno_last_error_string.restype = ctypes.c_char_p
    lib.uno_version.restype = ctypes.c_int
    lib.uno_read_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    lib.uno_gated_lora_linear_workspace_size.restype = _sz
    lib.uno_gated_lora_linear_workspace_size.argtypes = [_i64, _i64, _i64, _i64, ctypes.c_int]
    lib.uno_gated_lora_linear.argtypes = [_vp, _vp, _vp, _vp, _vp, _f32, _i64, _i64, _i64, _i64, ctypes.c_int,
                                          _vp, _vp, _sz, _vp]
    lib.uno_block_verify_workspace_size.restype = _sz
    lib.uno_block_verify_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _f32, ctypes.c_int]
    lib.uno_block_verify_min_workspace_size.restype = _sz
    lib.uno_block_verify_min_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _f32, ctypes.c_int]
    lib.uno_block_verify.argtypes = [_vp, _vp, ctypes.c_int, _i32, _i32, _i32, _f32, _i32, _f32,
                                     _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.uno_block_verify_noalloc.argtypes = [_vp, _vp, ctypes.c_int, _i32, _i32, _i32, _f32, _i32, _f32,
                                             _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.uno_block_verify_noalloc.restype = ctypes.c_int
    lib.uno_tv_loss_workspace_size.restype = _sz
    lib.uno_tv_loss_workspace_size.argtypes = [_i64, _i64, ctypes.c_int]
    lib.uno_tv_loss.argtypes = [_vp, _vp, ctypes.c_int, _i64, _i64, _vp, _f32, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.uno_block_noise.argtypes = [_vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp]
    lib.uno_block_noise.restype = ctypes.c_int
    for fn in ("uno_gated_lora_linear", "uno_block_verify", "uno_tv_loss"):
        getattr(lib, fn).restype = ctypes.c_int
    lib.uno_read_device_status.restype = ctypes.c_int
    lib.uno_rms_norm_fp8.argtypes = [_vp, _vp, _vp, ctypes.c_int, _i64, _i64, _f32, _vp, _vp, _vp, _vp, _vp]
    lib.uno_fp8_quantize.argtypes = [_vp, ctypes.c_int, _i64, _i64, _i32, _vp, _vp, _vp]
    lib.uno_fp8_gated_lora_linear_workspace_size.restype = _sz
    lib.uno_fp8_gated_lora_linear_workspace_size.argtypes = [_i64, _i64, _i64, _i64]
    lib.uno_fp8_gated_lora_linear.argtypes = [_vp] * 8 + [_f32, _i64, _i64, _i64, _i64, _vp, ctypes.c_int, _vp, _sz, _vp]
    lib.uno_token_logprobs.argtypes = [_vp, ctypes.c_int, _i64, _i64, _f32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.uno_token_logprobs_grad.argtypes = [_vp, ctypes.c_int, _i64, _i64, _f32] + [_vp] * 7
    for fn in ("uno_rms_norm_fp8", "uno_fp8_quantize", "uno_fp8_gated_lora_linear", "uno_token_logprobs",
               "uno_token_logprobs_grad"):
        getattr(lib, fn).restype = ctypes.c_int
    _lib = lib
    return lib


def _status_name(s: int) -> str:
    return load().uno_status_string(int(s)).decode()


def _check(status: int) -> None:
    if status != UNO_OK:
        raise UnoError(status, load().uno_last_error_string().decode())


def _ptr(t):
    """Device address of a tensor argument (None passes NULL). The C ABI takes row-major
    contiguous device memory, so anything else is refused here rather than misread there."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous CUDA tensors "
                         f"(got {type(t).__name__}{'' if not isinstance(t, torch.Tensor) else f' on {t.device}, contiguous={t.is_contiguous()}'})")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return UNO_BF16
    if t.dtype == torch.float32:
        return UNO_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


_NO_STREAM = contextlib.nullcontext()


def _allocating_on(stream):
    """Allocations inside come from `stream`'s pool (None: the current stream's, as they do anyway)."""
    return _NO_STREAM if stream is None else torch.cuda.stream(stream)


def _workspace(nbytes: int, device, workspace, stream):
    if nbytes == 0:
        return None, 0
    if workspace is None:
        with _allocating_on(stream):
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size()


def uno_version() -> int:
    return int(load().uno_version())


def uno_read_device_status() -> int:
    code = ctypes.c_uint32(0)
    _check(load().uno_read_device_status(ctypes.byref(code)))
    return int(code.value)


# ---------------------------------------------------------------------------------------
def uno_gated_lora_linear_workspace_size(M, d_in, d_out, rank, dtype=UNO_BF16) -> int:
    return int(load().uno_gated_lora_linear_workspace_size(M, d_in, d_out, rank, dtype))


def uno_gated_lora_linear(x, w0, lora_a, lora_b, row_gate, scale, y, workspace=None, stream=None):
    """y = x w0^T + scale * diag(row_gate) (x lora_a^T) lora_b^T  (see include/uno.h)."""
    M, d_in = x.shape
    d_out, rank = w0.shape[0], lora_a.shape[0]
    code = _dtype_code(x)
    ws, nb = _workspace(uno_gated_lora_linear_workspace_size(M, d_in, d_out, rank, code), x.device, workspace, stream)
    _check(load().uno_gated_lora_linear(_ptr(x), _ptr(w0), _ptr(lora_a), _ptr(lora_b), _ptr(row_gate),
                                        float(scale), M, d_in, d_out, rank, code, _ptr(y), _ptr(ws), nb,
                                        _stream(stream)))
    return y


# ---------------------------------------------------------------------------------------
def uno_block_verify_workspace_size(B, K, V, top_k, top_p, dtype=UNO_BF16) -> int:
    return int(load().uno_block_verify_workspace_size(B, K, V, top_k, top_p, dtype))


def uno_block_verify_min_workspace_size(B, K, V, top_k, top_p, dtype=UNO_BF16) -> int:
    return int(load().uno_block_verify_min_workspace_size(B, K, V, top_k, top_p, dtype))


def uno_block_verify(verifier_logits, drafter_logits, temperature, top_k, top_p, uniforms,
                     out_tokens, out_count, out_next_token=None, out_p_tok=None, out_q_tok=None, out_tv=None,
                     draft_tokens=None, pos0_tokens=None, workspace=None, stream=None):
    """Lossless block verify over [B, K, V] logits (see include/uno.h)."""
    B, K, V = verifier_logits.shape
    code = _dtype_code(verifier_logits)
    ws, nb = _workspace(uno_block_verify_workspace_size(B, K, V, top_k, top_p, code),
                        verifier_logits.device, workspace, stream)
    _check(load().uno_block_verify(
        _ptr(verifier_logits), _ptr(drafter_logits), code, B, K, V, float(temperature), int(top_k), float(top_p),
        _ptr(draft_tokens), _ptr(pos0_tokens), _ptr(uniforms), _ptr(out_tokens), _ptr(out_count),
        _ptr(out_next_token), _ptr(out_p_tok), _ptr(out_q_tok), _ptr(out_tv), _ptr(ws), nb, _stream(stream)))


def uno_block_verify_noalloc(verifier_logits, drafter_logits, temperature, top_k, top_p, uniforms,
                             out_tokens, out_count, out_next_token=None, out_p_tok=None, out_q_tok=None,
                             out_tv=None, draft_tokens=None, pos0_tokens=None, stream=None):
    """uno_block_verify with the library's fixed scratch array instead of a workspace, for
    callers that cannot allocate device memory (see include/uno.h)."""
    B, K, V = verifier_logits.shape
    code = _dtype_code(verifier_logits)
    _check(load().uno_block_verify_noalloc(
        _ptr(verifier_logits), _ptr(drafter_logits), code, B, K, V, float(temperature), int(top_k), float(top_p),
        _ptr(draft_tokens), _ptr(pos0_tokens), _ptr(uniforms), _ptr(out_tokens), _ptr(out_count),
        _ptr(out_next_token), _ptr(out_p_tok), _ptr(out_q_tok), _ptr(out_tv), _stream(stream)))


# ---------------------------------------------------------------------------------------
def uno_tv_loss_workspace_size(N, V, dtype=UNO_BF16) -> int:
    return int(load().uno_tv_loss_workspace_size(N, V, dtype))


def uno_tv_loss(teacher_logits, student_logits, out_tv, out_mean, grad_student=None, response_mask=None,
                grad_scale=1.0, workspace=None, stream=None):
    """TV self-distillation loss and gradient over [N, V] logits (see include/uno.h)."""
    N, V = teacher_logits.shape
    code = _dtype_code(teacher_logits)
    ws, nb = _workspace(uno_tv_loss_workspace_size(N, V, code), teacher_logits.device, workspace, stream)
    _check(load().uno_tv_loss(_ptr(teacher_logits), _ptr(student_logits), code, N, V, _ptr(response_mask),
                              float(grad_scale), _ptr(out_tv), _ptr(out_mean), _ptr(grad_student), _ptr(ws), nb,
                              _stream(stream)))


# ---------------------------------------------------------------------------------------
def uno_block_noise(clean_tokens, uniforms, V, noised_tokens, row_gate=None, stream=None):
    """Block-noised copy, noise mode random_uniform: position 0 kept, draft positions
    min(V - 1, floor(u V)); optional row gate (see include/uno.h)."""
    B, K = clean_tokens.shape
    _check(load().uno_block_noise(_ptr(clean_tokens), _ptr(uniforms), B, K, int(V), _ptr(noised_tokens),
                                  _ptr(row_gate), _stream(stream)))
    return noised_tokens


# ---------------------------------------------------------------------------------------
# include/uno_layers.h: every tensor's shape, dtype and device is checked here, and the call
# runs on the tensors' device whichever one is current. The checks stand on the path of every
# small call: they compare first and look for what to say only where a comparison fails.
_F8, _BF16, _F32, _I32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32
_CODES = {torch.bfloat16: UNO_BF16, torch.float32: UNO_F32}


def _arg(name, t, shape, dtype, index):
    """Device address of tensor `t` (None passes NULL) after checking what it has to be:
    contiguous, of this shape and dtype, on CUDA device `index`."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index \
            and t.is_contiguous():
        return t.data_ptr()
    _ptr(t)
    raise ValueError(f"{name}: expected {tuple(shape)} {dtype} on cuda:{index}, "
                     f"got {tuple(t.shape)} {t.dtype} on {t.device}")


def _lead(name, t, dtypes):
    """(shape, device address) of a contiguous CUDA matrix of one of the dtypes: an argument
    whose shape the others are checked against."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.dim() == 2 and t.is_contiguous():
        return t.shape, t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _ptr(t)
        raise ValueError(f"{name}: a contiguous CUDA tensor is required")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    _ptr(t)
    raise ValueError(f"{name}: expected a matrix, got {tuple(t.shape)}")


def _current_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# (torch's own accessor of the handle, without the Stream object, where this torch has it: a
# microsecond of a small call)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(fn, index, stream, *args):
    """One library call on CUDA device `index`, enqueued on `stream` (default: that device's
    current one)."""
    if stream is None:
        handle = _current_stream(index)
    elif stream.device_index != index:
        raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors are on cuda:{index}")
    else:
        handle = stream.cuda_stream
    if index == _current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            status = fn(*args, handle)
    if status != UNO_OK:
        _check(status)


def _blocks(n: int) -> int:
    return (n + 127) // 128


def uno_rms_norm_fp8(x, weight, eps, out_q=None, out_scale=None, residual=None, out_residual=None, out_y=None,
                     stream=None):
    """RMS norm of x (+ residual) with e4m3 values and a scale per 128 columns, and / or the
    norm in x's dtype (see include/uno_layers.h)."""
    shape, px = _lead("x", x, _CODES)
    M, d = shape
    i, t = x.get_device(), x.dtype
    _call(load().uno_rms_norm_fp8, i, stream, px, _arg("residual", residual, shape, t, i),
          _arg("weight", weight, (d,), t, i), _CODES[t], M, d, eps,
          _arg("out_residual", out_residual, shape, t, i), _arg("out_q", out_q, shape, _F8, i),
          _arg("out_scale", out_scale, (M, _blocks(d)), _F32, i), _arg("out_y", out_y, shape, t, i))


def uno_fp8_quantize(x, out_q, out_scale, block_rows=1, stream=None):
    """e4m3 values and scales of x by block_rows x 128 blocks, block_rows 1 (activations) or
    128 (weights) (see include/uno_layers.h)."""
    shape, px = _lead("x", x, _CODES)
    M, d = shape
    i, t = x.get_device(), x.dtype
    _call(load().uno_fp8_quantize, i, stream, px, _CODES[t], M, d, block_rows, _arg("out_q", out_q, shape, _F8, i),
          _arg("out_scale", out_scale, (M if block_rows == 1 else _blocks(M), _blocks(d)), _F32, i))


@functools.lru_cache(maxsize=1024)
def uno_fp8_gated_lora_linear_workspace_size(M, d_in, d_out, rank) -> int:
    return int(load().uno_fp8_gated_lora_linear_workspace_size(M, d_in, d_out, rank))


def uno_fp8_gated_lora_linear(x_q, x_scale, w_q, w_scale, y, x=None, lora_a=None, lora_b=None, row_gate=None,
                              scale=1.0, workspace=None, stream=None):
    """y = (x_q x_scale)(w_q w_scale)^T + scale * diag(row_gate) (x lora_a^T) lora_b^T, the
    adapter only where lora_a is given (see include/uno_layers.h)."""
    x_shape, px_q = _lead("x_q", x_q, (_F8,))
    (d_out, w_in), pw_q = _lead("w_q", w_q, (_F8,))
    y_shape, py = _lead("y", y, _CODES)
    M, d_in = x_shape
    i = x_q.get_device()
    if w_in != d_in or y_shape != (M, d_out) or w_q.get_device() != i or y.get_device() != i:
        raise ValueError(f"x_q {tuple(x_shape)}, w_q {(d_out, w_in)} and y {tuple(y_shape)} do not belong together "
                         "or are on different devices")
    rank, pa, pb, px, pg, ws, nb = 0, None, None, None, None, None, 0
    if lora_a is not None:
        (rank, _), _ = _lead("lora_a", lora_a, (_BF16,))
        pa, pb = _arg("lora_a", lora_a, (rank, d_in), _BF16, i), _arg("lora_b", lora_b, (d_out, rank), _BF16, i)
        px, pg = _arg("x", x, x_shape, _BF16, i), _arg("row_gate", row_gate, (M,), _F32, i)
    if rank:
        nb = uno_fp8_gated_lora_linear_workspace_size(M, d_in, d_out, rank)
        if workspace is None:
            # from the pool of the stream that the call runs on: a block of another stream's may still be
            # in use by what that one has queued (bf16; nb is a multiple of 256 bytes)
            with _allocating_on(stream):
                workspace = lora_a.new_empty(nb >> 1)
        elif workspace.get_device() != i:
            raise ValueError(f"workspace is on {workspace.device}, the tensors are on cuda:{i}")
        else:
            nb = workspace.numel() * workspace.element_size()
        ws = _ptr(workspace)
    _call(load().uno_fp8_gated_lora_linear, i, stream, px_q, _arg("x_scale", x_scale, (M, _blocks(d_in)), _F32, i),
          pw_q, _arg("w_scale", w_scale, (_blocks(d_out), _blocks(d_in)), _F32, i), px, pa, pb, pg, scale, M, d_in,
          d_out, rank, py, _CODES[y.dtype], ws, nb)
    return y


def uno_token_logprobs(logits, tokens, out_logprob=None, temperature=1.0, out_entropy=None, out_stats=None,
                       out_top_ids=None, out_top_logprobs=None, stream=None):
    """Log probability of each row's token, entropy, the most probable tokens (as many as
    out_top_ids has columns), and the statistics the gradient needs; rows whose token is not
    in [0, V) are left out (see include/uno_layers.h)."""
    (N, V), p = _lead("logits", logits, _CODES)
    i, t = logits.get_device(), logits.dtype
    k, ids, lps = 0, None, None
    if out_top_ids is not None or out_top_logprobs is not None:
        (_, k), _ = _lead("out_top_ids", out_top_ids, (_I32,))
        if k:
            ids = _arg("out_top_ids", out_top_ids, (N, k), _I32, i)
            lps = _arg("out_top_logprobs", out_top_logprobs, (N, k), _F32, i)
    _call(load().uno_token_logprobs, i, stream, p, _CODES[t], N, V, temperature, _arg("tokens", tokens, (N,), _I32, i),
          k, _arg("out_logprob", out_logprob, (N,), _F32, i), _arg("out_entropy", out_entropy, (N,), _F32, i),
          _arg("out_stats", out_stats, (N, 2), _F32, i), ids, lps)


def uno_token_logprobs_grad(logits, tokens, stats, grad_logits, grad_logprob=None, entropy=None, grad_entropy=None,
                            temperature=1.0, stream=None):
    """Gradient of uno_token_logprobs' log probabilities and entropies with respect to the
    logits; grad_logits may be logits itself (see include/uno_layers.h)."""
    shape, p = _lead("logits", logits, _CODES)
    N, V = shape
    i, t = logits.get_device(), logits.dtype
    _call(load().uno_token_logprobs_grad, i, stream, p, _CODES[t], N, V, temperature,
          _arg("tokens", tokens, (N,), _I32, i), _arg("stats", stats, (N, 2), _F32, i),
          _arg("entropy", entropy, (N,), _F32, i), _arg("grad_logprob", grad_logprob, (N,), _F32, i),
          _arg("grad_entropy", grad_entropy, (N,), _F32, i), _arg("grad_logits", grad_logits, shape, t, i))
