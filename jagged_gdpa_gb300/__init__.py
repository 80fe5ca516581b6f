"""jagged_gdpa_gb300: jagged Generalized Dot-Product Attention on GB300 (sm_103a).

The computation lives in libjgdpa.so (C ABI in include/jgdpa.h, CUDA kernels
under csrc/).  This package only builds and binds it.
"""

from ._lib import (  # noqa: F401
    ACT,
    ALU_LIB_PATH,
    LIB_PATH,
    EXPORTS,
    JgdpaError,
    jgdpa_bwd,
    jgdpa_bwd_shared_q,
    jgdpa_cache4_append,
    jgdpa_cache4_fwd,
    jgdpa_cache4_fwd_workspace_bytes,
    jgdpa_cache4_read,
    jgdpa_cache_append,
    jgdpa_cache_append_rotated,
    jgdpa_cache_fwd,
    jgdpa_cache_fwd_workspace_bytes,
    jgdpa_cache_plan,
    jgdpa_cache_plan_workspace_bytes,
    jgdpa_fwd_shared_q,
    jgdpa_shared_q_workspace_bytes,
    jgdpa_ds_scratch_bytes,
    jgdpa_eval_activation,
    jgdpa_fwd,
    jgdpa_fwd_noalloc,
    jgdpa_norm_rotate,
    jgdpa_norm_rotate_bwd,
    jgdpa_norm_rotate_workspace_bytes,
    jgdpa_read_device_status,
    jgdpa_set_wait_limit_ns,
    jgdpa_status_string,
    jgdpa_verify,
    jgdpa_verify_workspace_bytes,
    jgdpa_workspace_bytes,
    load,
)
