"""Differential attention (V1 and V2) for NVIDIA GB300, sm_103a.

The operator lives in the C-ABI library ``libdiffattn.so`` (``include/diffattn.h``);
``binding`` is its thin Python binding.  Build with
``python -m differential_attention_diff_gb300.build``.
"""

from .binding import (  # noqa: F401
    DiffAttnError,
    diffattn_get_device_status,
    diffattn_kv4_append,
    diffattn_kv4_read,
    diffattn_kv4_record_bytes,
    diffattn_kv_evict,
    diffattn_kv_evict_workspace_size,
    diffattn_lambda_init,
    diffattn_paged_append,
    diffattn_qk_rope_bwd,
    diffattn_qk_rope_bwd_workspace_size,
    diffattn_qk_rope_fwd,
    diffattn_rope_inv_freq,
    diffattn_v1_bwd,
    diffattn_v1_fwd,
    diffattn_v2_decode,
    diffattn_v2_decode_kv4,
    diffattn_v2_decode_kv4_workspace_size,
    diffattn_v2_decode_num_splits,
    diffattn_v2_decode_weighted,
    diffattn_v2_decode_weighted_workspace_size,
    diffattn_v2_decode_workspace_size,
    diffattn_v2_fwd,
    diffattn_v2_gate,
    diffattn_v2_paged_fwd,
    diffattn_v2_paged_fwd_workspace_size,
    load,
)
