"""Row-wise RMSNorm and fused residual-add RMSNorm for NVIDIA GB300 (sm_103a).

The compute runs in hand-written CUDA kernels behind the C ABI of ``libks`` (include/ks.h).
This package is the thin Python binding over it: it marshals torch tensors into pointers and
sizes and never computes anything itself. There is no CPU fallback: without the built library
every op raises ``KsLibraryMissing``.
"""
from ._abi import KsError, KsLibraryMissing  # noqa: F401
from .decode import (paged_attention, paged_attention_workspace, rotary,  # noqa: F401
                     rotary_steps, rotary_to_pages)
from .cache4 import (empty_pages_4bit, paged_attention_4bit, paged_attention_4bit_workspace,  # noqa: F401
                     pages_4bit_to_rows, rotary_to_pages_4bit)
from .ops import (fused_add_rms_norm, fused_add_rms_norm_host, gated_add_rms_norm,  # noqa: F401
                  layer_norm, rms_norm, rms_norm_host, silu_and_mul, softmax)

__all__ = ["rms_norm", "fused_add_rms_norm", "rms_norm_host", "fused_add_rms_norm_host",
           "silu_and_mul", "softmax", "layer_norm", "rotary_steps", "rotary", "rotary_to_pages",
           "paged_attention", "paged_attention_workspace", "gated_add_rms_norm", "empty_pages_4bit",
           "rotary_to_pages_4bit", "pages_4bit_to_rows", "paged_attention_4bit",
           "paged_attention_4bit_workspace", "KsError", "KsLibraryMissing"]
