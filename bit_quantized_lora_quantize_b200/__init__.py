"""Frozen-NF4 linear layer with a LoRA adapter (QLoRA's data-parallel hot
path) for NVIDIA B200 (sm_100a).

The product is the C-ABI library ``libqlora.so`` (include/qlora.h) built from
``csrc/`` by ``build.py``; ``qlora`` is its thin Python binding and
``synthetic`` the seeded input generator used by tests and the benchmark;
``rows`` the binding of the row-wise operators around the linears (dropout,
layer norm, the linear with adapter dropout), ``int8`` that of the linear on
8-bit integer weights, ``dp`` the data-parallel gradient bucket and ``paged``
the paged AdamW of the adapters.
"""

from .qlora import (  # noqa: F401
    CODES,
    LIB_PATH,
    PackedNF4,
    QloraError,
    lib,
    new_workspace,
    qlora_check_status,
    qlora_codebook,
    qlora_get_wait_timeout,
    qlora_set_wait_timeout,
    qlora_silu_gate_bwd,
    qlora_silu_gate_fwd,
    qlora_dequantize_nf4,
    qlora_linear_bwd,
    qlora_linear_fwd,
    qlora_nf4_codebook,
    qlora_profile_start,
    qlora_profile_stop,
    qlora_quantize_nf4,
    qlora_workspace_bytes,
)
from .rows import (  # noqa: F401
    new_dropout_workspace,
    new_layernorm_workspace,
    qlora_dropout_add_layernorm_bwd,
    qlora_dropout_add_layernorm_fwd,
    qlora_dropout_bwd,
    qlora_dropout_fwd,
    qlora_dropout_workspace_bytes,
    qlora_layernorm_bwd,
    qlora_layernorm_fwd,
    qlora_layernorm_workspace_bytes,
    qlora_linear_bwd_dropout,
    qlora_linear_fwd_dropout,
)
from .int8 import (  # noqa: F401
    PackedInt8,
    new_int8_workspace,
    qlora_int8_workspace_bytes,
    qlora_linear_int8_fwd,
    qlora_matmul_int8,
    qlora_quantize_int8,
)
