"""GB300-native INT4 per-token-head KV cache with a randomized Hadamard
rotation, and paged attention over it; also an FP8 cache with block scales and
the query/key norm and rotary step before a write.

The compute lives in libkvint4.so (hand-written CUDA for sm_103a behind the C
ABI in include/kvint4.h); this package only marshals torch tensors to it.
"""

from ._lib import (DEV_BAD_BLOCK, DEV_BAD_POS, DEV_BAD_SEQ, DEV_BAD_SIGNS, DEV_BAD_SLOT, DEV_NONFINITE, KvInt4Error,
                   attention, attention_fp8, attention_fp8_shared, attention_mass_fp8, attention_shared_workspace_size,
                   attention_workspace_size, evict_fp8, library_path, load, qk_norm_rope, qk_norm_rope_axes, read_fp8, rope_axes, status_string, write, write_fp8)

__all__ = ["write", "attention", "write_fp8", "read_fp8", "attention_fp8", "attention_fp8_shared", "attention_mass_fp8",
           "evict_fp8", "qk_norm_rope", "qk_norm_rope_axes", "rope_axes",
           "attention_workspace_size", "attention_shared_workspace_size", "load", "library_path",
           "status_string", "KvInt4Error", "DEV_BAD_SLOT", "DEV_BAD_BLOCK", "DEV_BAD_SEQ", "DEV_BAD_SIGNS",
           "DEV_NONFINITE", "DEV_BAD_POS"]
