"""GB300-native decode-time MoE layer with FloE-style contextually sparse SwiGLU experts.

The compute runs in a CUDA library built for sm_103a (``build.py``) behind a C ABI
(``include/sparse_expert_swiglu.h``); this package is its thin Python binding plus
the seeded synthetic-input generator.
"""

from ._lib import (  # noqa: F401
    DenseExperts,
    DenseLayer,
    EAMC,
    EXPORTED,
    ExpertCache,
    Experts,
    Int8Experts,
    Layer,
    MoeError,
    Workspace,
    eam_add_counts,
    expert_dense_swiglu,
    expert_dense_workspace_bytes,
    expert_int8_swiglu,
    expert_int8_workspace_bytes,
    expert_sparse_swiglu,
    expert_workspace_bytes,
    layer_decode,
    layer_decode_host_rows,
    layer_dense_decode,
    layer_dense_workspace_bytes,
    layer_host_rows_workspace_bytes,
    layer_path,
    layer_workspace_bytes,
    lib,
    lib_path,
    linear,
    linear_int8,
    linear_int8_workspace_bytes,
    linear_workspace_bytes,
    pack_int2_up,
    packed_bytes,
    prefetch_experts,
    quantize_int8,
    residual_norm,
    route_topk,
    route_topk_noalloc,
    route_workspace_bytes,
    unpack_int2_up,
)
from . import build as _build_module  # noqa: E402

build_library = _build_module.build
