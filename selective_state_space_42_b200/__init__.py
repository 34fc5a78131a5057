"""libselscan: the Mamba-1 selective scan, its gradient, its single-token
state update and the scalar-A-per-head (Mamba-2) scan in chunked form, as
hand-written CUDA for B200 (sm_100a) behind a C ABI (include/selscan.h);
next to them linear attention with a decay for each head (forward, gradient,
single token) and the norm/gate/residual junction between blocks.

The Python functions below are a thin ctypes binding with the same names as
the C entry points; see ``selscan.py``, ``linattn.py`` and ``block_norm.py``.
"""
from .block_norm import selscan_block_norm_bwd, selscan_block_norm_fwd
from .linattn import selscan_linattn_bwd, selscan_linattn_fwd, selscan_linattn_step
from .selscan import (LIB_PATH, SELSCAN_BF16, SELSCAN_F32, SELSCAN_MAX_DSTATE,
                      SELSCAN_MAX_DSTATE_BWD,
                      SELSCAN_NOALLOC_WORKSPACE_BYTES,
                      SelscanError, SelscanUnavailable, load_library,
                      selscan_bwd, selscan_bwd_workspace_bytes,
                      selscan_device_status, selscan_fwd, selscan_fwd_noalloc,
                      selscan_fwd_plan,
                      selscan_last_cuda_error,
                      selscan_ssd_fwd, selscan_state_update, selscan_status_string)

__all__ = ["selscan_linattn_fwd", "selscan_linattn_bwd", "selscan_linattn_step",
           "selscan_block_norm_fwd", "selscan_block_norm_bwd", "selscan_bwd", "selscan_bwd_workspace_bytes", "selscan_device_status", "selscan_fwd", "selscan_fwd_noalloc", "selscan_fwd_plan", "selscan_state_update", "selscan_ssd_fwd", "selscan_status_string",
           "selscan_last_cuda_error", "load_library", "SelscanError",
           "SelscanUnavailable", "LIB_PATH", "SELSCAN_F32", "SELSCAN_BF16",
           "SELSCAN_MAX_DSTATE", "SELSCAN_MAX_DSTATE_BWD", "SELSCAN_NOALLOC_WORKSPACE_BYTES"]
