"""ctypes view of libmea.so (the C ABI in include/mea.h). Marshalling only."""
from __future__ import annotations

import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmea.so")

# mea_status values (include/mea.h)
MEA_OK = 0
MEA_ERR_NULL = -1
MEA_ERR_SHAPE = -2
MEA_ERR_HEADS = -3
MEA_ERR_HEAD_DIM = -4
MEA_ERR_DTYPE = -5
MEA_ERR_ALIGN = -6
MEA_ERR_MASK = -7
MEA_ERR_WORKSPACE = -8
MEA_ERR_CUDA = -9
MEA_ERR_DEVICE_TIMEOUT = -10
MEA_ERR_DEVICE = -11
MEA_ERR_SCALE = -12
MEA_ERR_SCRATCH_LIMIT = -13

MEA_F16 = 0
MEA_BF16 = 1
MEA_MASK_NONE = 0
MEA_MASK_CAUSAL = 1
MEA_SELFTEST_WAIT_CODE = 0x7F01

EXPORTS = ("mea_forward", "mea_forward_fp8", "mea_backward_workspace_size", "mea_backward",
           "mea_decode_workspace_size", "mea_decode_splitkv", "mea_decode_paged",
           "mea_decode_splitkv_noalloc", "mea_block_key_bounds", "mea_select_blocks",
           "mea_decode_selected_workspace_size", "mea_decode_selected",
           "mea_decode_weights_workspace_size", "mea_decode_weights",
           "mea_attention_weights_workspace_size", "mea_attention_weights",
           "mea_evict_paged", "mea_decode_tree_workspace_size", "mea_decode_tree", "mea_call",
           "mea_status_string", "mea_device_error",
           "mea_set_wait_timeout_ns", "mea_wait_selftest", "mea_version")

# mea_call: entry number and the words of each call (include/mea.h), the scale as a double.
CALLS = {
    "mea_block_key_bounds": (1, struct.Struct("qqqqqqqqqqqqqq")),
    "mea_select_blocks": (2, struct.Struct("qqqqqqqqqqqqqqqqqq")),
    "mea_decode_selected": (3, struct.Struct("qqqqqqqqqqqqqqqqdqqqqq")),
    "mea_decode_weights": (4, struct.Struct("qqqqqqqqqqqqqqqqqqqdqqqqqq")),
    "mea_attention_weights": (5, struct.Struct("qqqqqqqqqqqqqqqdqqqqqqq")),
    "mea_evict_paged": (6, struct.Struct("qqqqqqqqqqqqqqqqqqqqqqqqq")),
    "mea_decode_tree": (7, struct.Struct("qqqqqqqqqqqqqqqqqqqqdqqqqq")),
}

_lib = None


def load() -> ctypes.CDLL:
    """Loads libmea.so (raises if it has not been built: there is no fallback path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmea.so not built at {LIB_PATH}; run "
                          "`python -m memory_efficient_attention_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, ci, cf, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.mea_forward.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, cf, ci,
                                vp, ci, vp]
    lib.mea_forward.restype = ci
    lib.mea_forward_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, cf,
                                    ci, vp, cf, cf, cf, ci, vp]
    lib.mea_forward_fp8.restype = ci
    lib.mea_backward_workspace_size.argtypes = [ci, ci]
    lib.mea_backward_workspace_size.restype = sz
    lib.mea_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci,
                                 ci, ci, ci, cf, ci, vp, ci, vp, sz, vp]
    lib.mea_backward.restype = ci
    lib.mea_decode_workspace_size.argtypes = [ci, ci, ci, ci, ci, ci]
    lib.mea_decode_workspace_size.restype = sz
    lib.mea_decode_splitkv.argtypes = [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, ci, vp,
                                       ci, vp, sz, ci, vp]
    lib.mea_decode_splitkv.restype = ci
    lib.mea_decode_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, ci,
                                     ci, cf, ci, vp, ci, vp, sz, ci, vp]
    lib.mea_decode_paged.restype = ci
    lib.mea_decode_splitkv_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf,
                                               ci, vp, ci, ci, vp]
    lib.mea_decode_splitkv_noalloc.restype = ci
    ll = ctypes.c_longlong
    lib.mea_block_key_bounds.argtypes = [vp] * 5 + [ci] * 8 + [vp]
    lib.mea_block_key_bounds.restype = ci
    lib.mea_select_blocks.argtypes = [vp] * 5 + [ci] * 12 + [vp]
    lib.mea_select_blocks.restype = ci
    lib.mea_decode_selected_workspace_size.argtypes = [ci] * 6
    lib.mea_decode_selected_workspace_size.restype = sz
    lib.mea_decode_selected.argtypes = [vp] * 8 + [ci] * 8 + [cf, vp, ci, vp, sz, vp]
    lib.mea_decode_selected.restype = ci
    lib.mea_decode_weights_workspace_size.argtypes = [ci] * 6
    lib.mea_decode_weights_workspace_size.restype = sz
    lib.mea_decode_weights.argtypes = [vp] * 9 + [ll] + [ci] * 9 + [cf, vp, ci, vp, sz, ci, vp]
    lib.mea_decode_weights.restype = ci
    lib.mea_attention_weights_workspace_size.argtypes = [ci]
    lib.mea_attention_weights_workspace_size.restype = sz
    lib.mea_attention_weights.argtypes = [vp] * 6 + [ll] + [ci] * 8 + [cf, ci, vp, ci, ci, vp, sz,
                                                                       vp]
    lib.mea_attention_weights.restype = ci
    lib.mea_evict_paged.argtypes = [vp] * 5 + [ll] + [vp] * 6 + [ci] * 12 + [vp]
    lib.mea_evict_paged.restype = ci
    lib.mea_decode_tree_workspace_size.argtypes = [ci] * 3
    lib.mea_decode_tree_workspace_size.restype = sz
    lib.mea_decode_tree.argtypes = [vp] * 9 + [ci] * 11 + [cf, vp, ci, vp, sz, vp]
    lib.mea_decode_tree.restype = ci
    lib.mea_call.argtypes = [ci, ctypes.c_char_p]
    lib.mea_call.restype = ci
    lib.mea_status_string.argtypes = [ci]
    lib.mea_status_string.restype = ctypes.c_char_p
    lib.mea_device_error.argtypes = [ctypes.POINTER(ci), ci]
    lib.mea_device_error.restype = ci
    lib.mea_set_wait_timeout_ns.argtypes = [ctypes.c_ulonglong]
    lib.mea_set_wait_timeout_ns.restype = None
    lib.mea_wait_selftest.argtypes = [ctypes.c_ulonglong, ci, vp]
    lib.mea_wait_selftest.restype = ci
    lib.mea_version.argtypes = []
    lib.mea_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(rc: int) -> str:
    return load().mea_status_string(int(rc)).decode()


class MeaError(RuntimeError):
    def __init__(self, rc: int, where: str = ""):
        self.rc = rc
        super().__init__(f"{where}: {status_string(rc)} ({rc})" if where else status_string(rc))


def check(rc: int, where: str) -> None:
    if rc != MEA_OK:
        raise MeaError(rc, where)
