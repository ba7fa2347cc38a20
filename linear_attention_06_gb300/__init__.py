"""GB300-native Kimi Delta Attention (KDA): prefill and decode behind the C ABI
of libkda (include/kda.h).  This package is the thin Python side of it."""
from ._lib import (KdaError, KdaLatentShape, KdaShape, kda_check_cu_seqlens, kda_decode_step,  # noqa: F401
                   kda_decode_step_gated, kda_device_status, kda_frontend, kda_latent_append,
                   kda_latent_append_q8, kda_latent_decode, kda_latent_decode_q8, kda_latent_decode_q8_workspace_size,
                   kda_latent_decode_workspace_size, kda_latent_gather, kda_latent_gather_q8, kda_latent_prefill, kda_prefill, kda_prefill_checkpointed,
                   kda_prefill_frontend, kda_prefill_gated, kda_prefill_split, kda_prefill_split_workspace_size, kda_selftest_timeout, lib,
                   status_string, version)
from . import workloads  # noqa: F401

__all__ = ["kda_prefill", "kda_prefill_checkpointed", "kda_prefill_frontend", "kda_prefill_gated",
           "kda_prefill_split",
           "kda_prefill_split_workspace_size", "kda_decode_step",
           "kda_decode_step_gated", "kda_frontend", "kda_check_cu_seqlens",
           "kda_latent_append", "kda_latent_gather", "kda_latent_decode", "kda_latent_decode_workspace_size",
           "kda_latent_append_q8", "kda_latent_gather_q8", "kda_latent_decode_q8", "kda_latent_decode_q8_workspace_size",
           "kda_latent_prefill",
           "kda_device_status", "kda_selftest_timeout",
           "status_string", "version", "lib", "KdaError", "KdaShape", "KdaLatentShape", "workloads"]
