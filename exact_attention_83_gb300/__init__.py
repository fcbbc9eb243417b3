"""Exact scaled-dot-product attention (FlashAttention-2 form) for GB300.

The compute path is libfa (hand-written CUDA for sm_103a behind the C ABI in
include/fa.h); `fa` is its thin Python binding.
"""

from .fa import (FAError, Rotary, attention, attention_bwd, attention_decode, attention_fwd,
                 attention_varlen_prefix, bwd, bwd_preprocess, device_status, fwd, load_library,
                 qk_norm_rotary, rotary, set_path, set_wait_timeout_ns)

__all__ = ["FAError", "Rotary", "attention", "attention_bwd", "attention_decode", "attention_fwd",
           "attention_varlen_prefix", "bwd", "bwd_preprocess", "device_status", "fwd",
           "load_library", "qk_norm_rotary", "rotary", "set_path", "set_wait_timeout_ns"]
