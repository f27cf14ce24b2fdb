"""GB300-native (sm_103a) KDA gated delta-rule serving step.

The product is the C-ABI library libkda_gb300.so (include/kda.h): kda_decode,
kda_verify, kda_verify_ring and, for the attention layers of a hybrid decoder
(include/kda_paged.h), kda_paged_plan, kda_rope_append and kda_paged_attention,
with kda_rope_append_fp8, kda_paged_attention_fp8 and kda_paged_read_fp8 for a
cache in 8 bits (include/kda_paged_fp8.h). This package holds its CUDA sources (csrc/), its in-tree build (_build.py), a ctypes binding with the same names (kda.py)
and seeded synthetic workloads (workloads.py).
"""

from . import kda, workloads  # noqa: F401
from .kda import (  # noqa: F401
    KdaError,
    kda_decode,
    kda_verify,
    kda_verify_ring,
    kda_paged_plan,
    kda_rope_append,
    kda_paged_attention,
    kda_rope_append_fp8,
    kda_paged_attention_fp8,
    kda_paged_read_fp8,
    kda_select_config,
    kda_num_configs,
    kda_config_tile_v,
    kda_last_error,
    load_library,
)
