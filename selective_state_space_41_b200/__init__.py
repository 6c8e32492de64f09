"""libselscan: the Mamba selective scan, and the operators around it in a
layer (normalisation, causal convolution, gated recurrence), as hand-written
sm_100a CUDA kernels behind a C ABI (``include/selscan.h``), with a thin
Python binding.

    from selective_state_space_41_b200 import selective_scan_fwd
    y, last = selective_scan_fwd(u, delta, A, B, C, D, z, delta_bias,
                                 delta_softplus=True, return_last_state=True)

``workloads`` and ``gen`` hold the synthetic workloads and their seeded input
generator.
"""
from .selscan import (SS_BF16, SS_F32, SelscanError, lib, selective_scan_bwd, selective_scan_fwd,  # noqa: F401
                      ss_bwd, ss_bwd_workspace_bytes, ss_fwd, ss_step,
                      ss_fwd_heuristic, ss_fwd_hostio, ss_fwd_noalloc, ss_fwd_workspace_bytes,
                      ss_status_string, ss_fwd_dtproj, ss_fwd_xdbl, ss_bwd_heuristic, ss_device_status,
                      ss_fwd_ckpt, ss_bwd_ckpt, ss_bwd_ckpt_workspace_bytes, ckpt_shape,
                      SelectiveScanFn, selective_scan_fn,
                      ss_version, workspace_for)
from .layer_ops import (CausalConvFn, GatedRecurrenceFn, LayerNormFn, causal_conv_bwd, causal_conv_fn,  # noqa: F401
                        causal_conv_fwd, causal_conv_step, gated_recurrence_bwd, gated_recurrence_fn,
                        gated_recurrence_fwd, gated_recurrence_step, layer_norm_bwd, layer_norm_fn, layer_norm_fwd,
                        ss_conv_bwd, ss_conv_fwd, ss_conv_step, ss_glr_bwd, ss_glr_ckpt_elems, ss_glr_fwd,
                        ss_glr_step, ss_norm_bwd, ss_norm_bwd_workspace_bytes, ss_norm_fwd)

__all__ = ["selective_scan_fwd", "selective_scan_bwd", "ss_bwd", "ss_bwd_workspace_bytes", "ss_fwd", "ss_step", "ss_fwd_heuristic", "ss_fwd_hostio", "ss_fwd_noalloc",
           "ss_fwd_workspace_bytes", "workspace_for", "ss_status_string", "ss_version",
           "ss_fwd_dtproj", "ss_fwd_xdbl", "ss_bwd_heuristic", "ss_device_status",
           "ss_fwd_ckpt", "ss_bwd_ckpt", "ss_bwd_ckpt_workspace_bytes", "ckpt_shape",
           "SelectiveScanFn", "selective_scan_fn",
           "ss_norm_fwd", "ss_norm_bwd", "ss_norm_bwd_workspace_bytes",
           "layer_norm_fwd", "layer_norm_bwd", "layer_norm_fn", "LayerNormFn",
           "ss_conv_fwd", "ss_conv_bwd", "ss_conv_step",
           "causal_conv_fwd", "causal_conv_bwd", "causal_conv_step", "causal_conv_fn", "CausalConvFn",
           "ss_glr_fwd", "ss_glr_bwd", "ss_glr_step", "ss_glr_ckpt_elems",
           "gated_recurrence_fwd", "gated_recurrence_bwd", "gated_recurrence_step", "gated_recurrence_fn",
           "GatedRecurrenceFn", "SelscanError", "SS_F32", "SS_BF16", "lib"]
