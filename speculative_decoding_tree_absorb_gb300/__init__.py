"""GB300-native (sm_103a) DDTree tree-verify MLA-absorb attention.

The compute path is libkdt.so (C ABI in include/kdt.h, CUDA kernels in csrc/);
this package holds the build script and a thin ctypes binding with the same names.
"""
from .kdt import (  # noqa: F401
    DEFAULT_SCALE, EXPORTS, IMPLS, KdtError, LatentWriteArgs, RopeArgs, VerifyArgs, VerifyQ8Args,
    build_visibility, host_buffer_size, kv_compact, kv_compact_q8, latent_read_q8, latent_write_q8, lib, make_args,
    merge_attn_states, plan, rope_neox, status_str, tree_accept, tree_build,
    tree_sample, verify_attn,
    vc_up_proj, verify_attn_host, verify_attn_noalloc, verify_attn_q8, verify_attn_q8_plan,
    verify_attn_q8_workspace_size, workspace_size,
)

__version__ = "0.1.0"
