"""GB300 (sm_103a) local MoE forward: route -> dispatch -> SwiGLU experts -> combine.

The compute lives in ``libmoe.so`` (hand-written CUDA kernels behind the C ABI declared in
``include/moe.h``); ``binding`` marshals torch tensors into that ABI and nothing else, as do ``front``
(``include/moe_front.h``: the norm and the grouped softmax router) and ``mx8`` (``include/moe_mx8.h``).
"""
from .binding import (MoeError, moe_combine_backward, moe_dispatch_backward,  # noqa: F401
                      moe_experts_backward, dispatch_workspace_bytes, experts_workspace_bytes,  # noqa: F401
                      forward_workspace_bytes, moe_combine, moe_device_status, moe_dispatch,
                      moe_experts_forward_dispatched, moe_forward, moe_forward_fused,
                      moe_forward_sigmoid_grouped,
                      moe_forward_with_events, moe_mx4_dequantize,
                      moe_mx4_experts_forward_dispatched, moe_mx4_forward_tokens,
                      moe_mx4_product, moe_mx4_quantize, mx4_experts_workspace_bytes,
                      mx4_tokens_workspace_bytes, moe_route, moe_route_sigmoid_grouped,
                      moe_selected_router_backward, moe_selected_router_weights,
                      moe_wait_selftest)
from .front import (moe_forward_softmax_grouped, moe_rms_norm, moe_rms_norm_backward,  # noqa: F401
                    moe_route_softmax_grouped, rms_norm_backward_workspace_bytes)
from .mx8 import (moe_mx8_dequantize, moe_mx8_dispatch,  # noqa: F401
                  moe_mx8_experts_forward_dispatched, moe_mx8_forward, moe_mx8_product,
                  moe_mx8_quantize, mx8_experts_workspace_bytes, mx8_forward_workspace_bytes)
