"""MI355X (gfx950) MoE route-count / dispatch / combine.

The compute path lives in libmoe_route.so (hand-written HIP kernels behind a
C ABI, declared in include/moe_route.h); this package is its thin Python
binding (_lib: moe_route.h; _train: moe_train.h; _experts: moe_experts.h).  Import is
cheap: the library is loaded on first use and its absence raises instead of falling back
to anything else.
"""
from ._experts import (expert_product_mxfp4, experts_decode, experts_decode_workspace,
                       experts_decode_workspace_size, mxfp4_dequantize, mxfp4_quantize, swiglu,
                       swiglu_backward)
from ._lib import (DedupOut, DedupPlan, DispatchOut, MoeError, combine, combine_fp4, combine_fp8,
                   copy16,
                   dedup_dispatch, dispatch, dispatch_noalloc, dispatch_prequant, dispatch_replay, fp8_dequant,
                   geometry, load, route_count, version, workspace, workspace_size)
from ._train import (combine_backward, dispatch_backward, embedding, embedding_backward,
                     embedding_workspace, embedding_workspace_size, gate, gate_backward)

__all__ = ["DedupOut", "DedupPlan", "DispatchOut", "MoeError", "combine", "combine_backward", "combine_fp4",
           "combine_fp8", "copy16", "dedup_dispatch", "dispatch", "dispatch_backward",
           "dispatch_noalloc", "dispatch_prequant", "dispatch_replay", "embedding",
           "embedding_backward", "embedding_workspace", "embedding_workspace_size",
           "expert_product_mxfp4", "experts_decode", "experts_decode_workspace",
           "experts_decode_workspace_size", "fp8_dequant", "gate", "gate_backward", "geometry",
           "load", "mxfp4_dequantize", "mxfp4_quantize", "route_count", "swiglu",
           "swiglu_backward", "version", "workspace", "workspace_size"]
