"""GB300-native routed mixture-of-experts FFN over a prompt chunk.

The compute runs in the CUDA library ``libmoe_gb300.so`` (see
``routed_expert_prefill_gb300.moe`` for the Python binding of the routed block
and ``routed_expert_prefill_gb300.layer`` for that of the layer operators
around it).  Importing this package does not load the library; ``import
routed_expert_prefill_gb300.moe`` (or touching one of the names below) does.
"""

_MOE = ["moe_route_topk", "moe_build_csr", "moe_experts_fwd"]
_LAYER = ["moe_add_rms_norm", "moe_qmv", "KvCache", "moe_kv_append", "moe_kv_attention"]
__all__ = _MOE + _LAYER


def __getattr__(name):
    if name in _MOE:
        from . import moe

        return getattr(moe, name)
    if name in _LAYER:
        from . import layer

        return getattr(layer, name)
    raise AttributeError(name)
