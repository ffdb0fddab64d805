"""GB300-native FP8 linear layer: quantize-cast kernels (delayed, tensorwise, MXFP8,
blockwise) and scaled FP8 GEMMs on the sm_103a tensor core, behind a C ABI
(include/fp8lin.h). This package is the build step plus a thin Python binding."""
from . import _lib  # noqa: F401
from .binding import (  # noqa: F401
    BranchGrads, Checkpoint, DelayedState, GradList, QTensor, Recipe, amax_update,
    branch_rmsnorm_bwd, branch_rmsnorm_bwd_workspace_bytes, branch_rmsnorm_quantize, checkpoint,
    checkpoint_quantize, checkpoint_read, dgelu_quantize, empty_checkpoint, empty_qtensor,
    gelu_quantize, grad_clip, grad_norm, grad_workspace_bytes, linear_bwd, linear_dgrad_dgelu,
    linear_fwd, linear_fwd_gelu, quantize, quantize_group, quantize_master,
    quantize_static_scratch, rmsnorm, rmsnorm_bwd, rmsnorm_bwd_workspace_bytes, rmsnorm_quantize,
    rmsnorm_workspace_bytes, workspace_bytes,
)
