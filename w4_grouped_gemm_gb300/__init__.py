"""GB300 (sm_103a) W4 MoE expert layer: GPU-resident routing, fused-dequant
tcgen05 grouped GEMMs and a W4 GEMV decode path behind a C ABI
(include/lily_moe.h), and the attention side of a decoder block
(include/lily_attn.h).  This package is the thin Python binding; the compute
runs in liblily_moe.so, built by ``build.build()``."""
from ._lib import *  # noqa: F401,F403
from ._attn import (ATTN_EXPORTS, AttnDims, NormDims, PagedCache, RopeDims, LILY_DTYPE_E4M3,  # noqa: F401
                    LILY_DTYPE_F16, LILY_PREFIX_NONE, LILY_PREFIX_TENSOR, LILY_PREFIX_WARP,
                    LILY_STATUS_BAD_LEN, LILY_STATUS_BAD_PAGE,
                    LILY_STATUS_BAD_SLOT, lily_attn_add_rmsnorm, lily_attn_prefix_kernel,
                    lily_attn_rope_append, lily_attn_set_wait_ns, lily_attn_shared_prefix,
                    lily_attn_workspace_bytes, make_attn_dims, make_norm_dims, make_rope_dims)
from ._lib import (Dims, LayerWeights, RoutingBuffers, LilyError, alloc_workspace, make_dims,
                   lib, EXPORTS, LIB_PATH)  # noqa: F401
