"""B200-native BitStack residual-block linear.

The C ABI (include/bitstack.h) is implemented by libbitstack_b200.so, built from
csrc/ for sm_100a by ``residual_block_decomp_b200.build``; ``binding`` exposes it
under the same names and ``layer`` wraps a stack in torch-allocated device memory.
Attributes are resolved on first use, so the builder can run before the library
exists; using any binding name without the library fails loudly.
"""
import importlib

_BINDING_NAMES = (
    "BS_BF16", "BS_ERR_ALIGNMENT", "BS_ERR_CAPACITY", "BS_ERR_CUDA", "BS_ERR_INVALID_ARG", "BS_ERR_NO_DEVICE",
    "BS_ERR_RANGE", "BS_ERR_TIMEOUT", "BS_ERR_UNSUPPORTED_SHAPE", "BS_F16", "BS_F32", "BS_OK", "BS_ORDER_AVERAGE",
    "BS_ORDER_GREEDY", "BS_ORDER_RANDOM", "EXPORTS",
    "LIB_PATH", "BsError", "bs_append_block", "bs_block_bytes", "bs_decompose", "bs_decompose_workspace_bytes", "bs_debug_set_wait", "bs_drop_block",
    "bs_get_device_error", "bs_group_workspace_bytes", "bs_linear", "bs_linear_group", "bs_linear_no_alloc", "bs_pack_record", "bs_plain_block_bytes",
    "bs_plain_rank", "bs_plain_stack_create", "bs_plain_stack_device_bytes", "bs_plain_workspace_bytes",
    "bs_plan_budget", "bs_plan_order", "bs_reconstruct",
    "bs_stack_create", "bs_stack_destroy", "bs_stack_device_bytes", "bs_stack_num_blocks", "bs_status_string",
    "bs_unpack_signs", "bs_workspace_bytes", "lib",
    "CacheStep", "bs_cache_append", "bs_cache_attention", "bs_cache_attention_workspace_bytes", "bs_cache_create",
    "bs_cache_debug_set_wait", "bs_cache_destroy", "bs_cache_device_bytes", "bs_cache_get_device_error", "bs_cache_page_bytes", "bs_cache_read",
)
_LAYER_NAMES = ("BitStackAttention", "BitStackCache", "BitStackLinear", "PageTable")
__all__ = list(_BINDING_NAMES) + list(_LAYER_NAMES)


def __getattr__(name):
    if name in _BINDING_NAMES:
        value = getattr(importlib.import_module(".binding", __name__), name)
    elif name in _LAYER_NAMES:
        value = getattr(importlib.import_module(".layer", __name__), name)
    else:
        raise AttributeError(name)
    globals()[name] = value   # found directly from now on
    return value
