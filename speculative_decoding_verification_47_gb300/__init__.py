"""GB300-native batched lossless speculative-decoding verification.

The product is the C-ABI library ``libspecverify.so`` (CUDA kernels for
sm_103a; header ``include/specverify.h``).  ``binding`` exposes its calls to
Python under the same names; ``build`` compiles it in-tree; ``workloads``
draws seeded synthetic inputs.
"""

from .binding import (  # noqa: F401
    SVError,
    sv_kv4_append,
    sv_kv4_attention,
    sv_kv4_read,
    sv_kv_commit,
    sv_kv_compact,
    sv_kv_copy_pages,
    sv_kv_fork,
    sv_kv_free,
    sv_last_error,
    sv_linear,
    sv_linear_w4,
    sv_lmhead_rmsnorm,
    sv_lmhead_workspace_size,
    sv_prefix_attention,
    sv_read_device_flags,
    sv_rmsnorm_residual,
    sv_spec_verify,
    sv_version,
    sv_workspace_size,
)
