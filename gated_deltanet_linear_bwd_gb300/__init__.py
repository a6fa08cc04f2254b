"""Gated DeltaNet chunked prefill (forward + backward) for one GB300 (sm_103a).

The computation runs in libgdn.so (C ABI in include/gdn.h); this package is
its thin Python binding.  Importing it loads the library and fails loudly if
it has not been built.
"""
from . import _abi, _abi_layer
from ._abi import (GDN_BF16, GDN_CP_AUTO, GDN_CP_FORCE, GDN_CP_OFF, GDN_FP32, GdnError,
                   gdn_abi_version, gdn_bwd_workspace_size, gdn_chunk_bwd, gdn_chunk_fwd,
                   gdn_fwd_ctx_size, gdn_fwd_workspace_size, gdn_last_error, gdn_profile_begin, gdn_profile_end,
                   gdn_recurrent_step, gdn_set_spin_limit, gdn_sync_status)
from .api import (chunk_gated_delta_rule, chunk_gated_delta_rule_bwd,
                  chunk_gated_delta_rule_fwd, recurrent_step)
from .feed_forward import gated_feed_forward, gated_feed_forward_bwd, gated_feed_forward_fwd
from .layer import (MxTensor, add_rms_norm, add_rms_norm_bwd, add_rms_norm_fwd,
                    gated_linear_recurrence, gated_linear_recurrence_bwd,
                    gated_linear_recurrence_fwd, gated_linear_recurrence_step, mx_dequantize,
                    mx_from_parts, mx_linear, mx_matmul, mx_quantize)
from .state_space import (causal_convolution, causal_convolution_bwd, causal_convolution_fwd,
                          causal_convolution_step, state_space_scan, state_space_scan_bwd,
                          state_space_scan_fwd, state_space_step)

_abi.load()
_abi_layer.load()

__all__ = ["chunk_gated_delta_rule", "chunk_gated_delta_rule_fwd", "chunk_gated_delta_rule_bwd",
           "recurrent_step", "gdn_recurrent_step",
           "gdn_abi_version", "gdn_fwd_workspace_size", "gdn_fwd_ctx_size", "gdn_chunk_fwd",
           "gdn_bwd_workspace_size", "gdn_chunk_bwd", "gdn_sync_status", "gdn_last_error",
           "gdn_set_spin_limit", "gdn_profile_begin", "gdn_profile_end", "GdnError", "GDN_FP32", "GDN_BF16", "GDN_CP_AUTO",
           "GDN_CP_OFF", "GDN_CP_FORCE",
           "gated_linear_recurrence", "gated_linear_recurrence_fwd",
           "gated_linear_recurrence_bwd", "gated_linear_recurrence_step",
           "add_rms_norm", "add_rms_norm_fwd", "add_rms_norm_bwd",
           "MxTensor", "mx_quantize", "mx_dequantize", "mx_from_parts", "mx_matmul", "mx_linear",
           "causal_convolution", "causal_convolution_fwd", "causal_convolution_bwd", "causal_convolution_step",
           "state_space_scan", "state_space_scan_fwd", "state_space_scan_bwd", "state_space_step",
           "gated_feed_forward", "gated_feed_forward_fwd", "gated_feed_forward_bwd"]
