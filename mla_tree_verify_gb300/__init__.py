"""MLA tree-verify attention for GB300 (sm_103a).

The computation runs in ``libmla_tree_verify.so`` (CUDA kernels behind the C ABIs of
``include/mla_tree_verify.h``, ``include/mla_kv_q8.h`` and ``include/causal_conv1d_dedup.h``);
``binding`` marshals torch tensors to it.  Build the library with ``mla_tree_verify_gb300.build.build()``.
"""
from .binding import (APPEND_BAD_POS, APPEND_BAD_SCALE, APPEND_BAD_SLOT,  # noqa: F401
                      APPEND_BAD_VALUE, APPEND_PAD_SLOT, DEV_BAD_SCALE, KV_TYPE_BF16,
                      KV_TYPE_E4M3, kv_append, kv_gather_q8, mla_tree_verify_q8,
                      mla_tree_verify_q8_debug_ex, mla_tree_verify_q8_debug_merge,
                      Q8_MERGE_ALONE, Q8_MERGE_AUTO, Q8_MERGE_NO_TMEM, workspace_bytes_q8)
from .binding import (CONV1D_BAD_ACCEPT, CONV1D_BAD_SLOT, CONV1D_DTYPE_BF16,  # noqa: F401
                      CONV1D_DTYPE_F32, CONV1D_PAD_SLOT,
                      DEV_BAD_INDPTR, DEV_BAD_MASK, DEV_BAD_SLOT, DEV_TIMEOUT,
                      GATHER_BAD_ARGS, GATHER_BAD_SLOT, MERGE_AUTO, MERGE_NO_TMEM,
                      MERGE_PREFER_TMEM, MlaTreeVerifyError, conv1d_update, kv_gather,
                      mla_tree_verify, mla_tree_verify_debug, mla_tree_verify_debug_ex,
                      plan_header, prepare, read_device_status, split_grid, workspace_bytes)
