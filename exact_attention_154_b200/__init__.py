"""B200 (sm_100a) exact attention: the forward and its gradient.

``fwd`` / ``fwd_qkvpacked`` / ``fwd_varlen`` / ``fwd_fp8`` and ``bwd`` / ``bwd_noalloc``, and
``fwd_sinks`` / ``bwd_sinks`` / ``decode_sinks`` and ``qk_norm_rope`` / ``qk_norm_rope_bwd`` /
``rope_table`` call the C ABI of
``libfa_sm100.so`` (declared in ``include/fa.h``); ``synth`` draws the seeded
synthetic inputs.
"""
from .fa import (FaError, bwd, bwd_noalloc, bwd_sinks, decode_sinks, device_status, fwd, fwd_fp8,
                 fwd_qkvpacked, fwd_sinks, fwd_varlen, launch_ctas, load, qk_norm_rope,
                 qk_norm_rope_bwd, rope_table, strerror, version, watchdog_selftest)

__all__ = ["FaError", "bwd", "bwd_noalloc", "bwd_sinks", "decode_sinks", "device_status", "fwd",
           "fwd_fp8", "fwd_qkvpacked", "fwd_sinks", "fwd_varlen", "launch_ctas", "load",
           "qk_norm_rope", "qk_norm_rope_bwd", "rope_table", "strerror", "version",
           "watchdog_selftest"]
