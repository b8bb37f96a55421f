"""Uno draft-and-verify hot path on NVIDIA B200 (sm_100a).

The computation lives in libuno.so (CUDA kernels behind the C ABI of include/uno.h and
include/uno_layers.h): the row-gated LoRA linear, the lossless block verify and the TV
self-distillation loss; an 8-bit base under the projections (RMS norm and quantiser to e4m3
with block scales, the gated LoRA linear on an e4m3 weight), and token log probabilities with
entropy, alternatives and their gradient.
This package is its thin Python binding (plus `driver`, the decode step chained on one
stream); `workloads` holds the seeded synthetic inputs.
"""
from ._lib import (  # noqa: F401
    UNO_BF16, UNO_F32, UNO_OK, UnoError, load, uno_block_noise, uno_block_verify, uno_block_verify_workspace_size,
    uno_block_verify_min_workspace_size,
    uno_fp8_gated_lora_linear, uno_fp8_gated_lora_linear_workspace_size, uno_fp8_quantize,
    uno_gated_lora_linear, uno_gated_lora_linear_workspace_size, uno_read_device_status, uno_rms_norm_fp8,
    uno_token_logprobs, uno_token_logprobs_grad, uno_tv_loss, uno_tv_loss_workspace_size, uno_version,
)
