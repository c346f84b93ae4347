"""GB300-native fused image normalisation (FusedNormalization on sm_103a).

One memory pass over a uint8 NHWC batch: ToTensor, per-channel Normalize,
optional horizontal flip and optional erase rectangle per image, binary32 or
binary16 output in NHWC, NCHW or 4-channel NHWC.  The work runs in the CUDA
kernels of libtrfn.so (C ABI in include/tr_fused_norm.h); this package is
its thin binding plus the seeded synthetic-input generators (synth).

Token-row operators for what follows the batch (C ABI in
include/tr_token_ops.h): RMS norm with the residual's addition, output in the
input's type or in 8 bits, and its gradients; 8-bit quantisation of rows; the
8-bit integer matrix product with a scale for each token and channel.
"""
from .api import (LAUNCH_OVERLAP_PREVIOUS, LAYOUT_NCHW, LAYOUT_NHWC, LAYOUT_NHWC4, OUT_F16, OUT_F32, PRESETS, STAGE_FAST,
                  STAGE_REPRODUCIBLE, VARIANT_AUTO, Staging, tr_stage_zone_bytes,
                  VARIANT_GENERIC, VARIANT_TILED, TransferStation, out_shape, tr_device_status,
                  tr_fused_norm, tr_fused_norm_batches, tr_fused_norm_crop, tr_fused_norm_geometry, tr_fused_norm_plan, tr_fused_norm_sampled, tr_launch_count, tr_norm_preset, tr_sample_aug_params,
                  tr_sample_aug_params_device,
                  tr_ts_slot_bytes, tr_tune_tiled, tr_validate_aug_params, tr_workspace_bytes)
from .tokens import (ELEM_BF16, ELEM_F16, ELEM_F32, ELEM_I8, tr_dequantize_rows, tr_int8_matmul,
                     tr_int8_matmul_workspace_bytes, tr_quantize_rows, tr_rms_norm, tr_rms_norm_backward,
                     tr_rms_norm_backward_workspace_bytes)
from ._native import LIB_PATH, TrError

__all__ = [
    "LAUNCH_OVERLAP_PREVIOUS", "LAYOUT_NCHW", "LAYOUT_NHWC", "LAYOUT_NHWC4", "OUT_F16", "OUT_F32", "PRESETS", "VARIANT_AUTO",
    "VARIANT_GENERIC", "VARIANT_TILED", "TransferStation", "out_shape", "tr_device_status", "tr_fused_norm",
    "tr_fused_norm_batches",
    "tr_fused_norm_crop", "tr_fused_norm_geometry", "tr_sample_aug_params_device", "tr_fused_norm_sampled",
    "tr_fused_norm_plan", "tr_launch_count", "tr_norm_preset", "tr_sample_aug_params", "tr_ts_slot_bytes",
    "tr_tune_tiled", "tr_workspace_bytes",
    "tr_validate_aug_params", "LIB_PATH", "TrError", "STAGE_FAST", "STAGE_REPRODUCIBLE", "Staging",
    "tr_stage_zone_bytes",
    "ELEM_BF16", "ELEM_F16", "ELEM_F32", "ELEM_I8", "tr_dequantize_rows", "tr_int8_matmul",
    "tr_int8_matmul_workspace_bytes", "tr_quantize_rows", "tr_rms_norm", "tr_rms_norm_backward",
    "tr_rms_norm_backward_workspace_bytes",
]
