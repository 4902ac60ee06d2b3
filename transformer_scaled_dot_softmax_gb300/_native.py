"""ctypes view of libmha.so (the C ABI in include/mha.h).

Loading never touches the GPU.  If the library has not been built the import
fails loudly: there is no fallback implementation."""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
# MHA_LIBRARY may name another build of this same library (the tests load the
# build with device-side bounds checks that way); by default the in-tree build.
LIB_PATH = os.environ.get("MHA_LIBRARY") or os.path.join(_HERE, "_build", "libmha.so")

MHA_OK, MHA_ERR_INVALID_ARG, MHA_ERR_UNSUPPORTED, MHA_ERR_WORKSPACE = 0, 1, 2, 3
MHA_ERR_MISALIGNED, MHA_ERR_CUDA, MHA_ERR_TIMEOUT, MHA_ERR_BOUNDS = 4, 5, 6, 7
MHA_F32, MHA_BF16, MHA_INT8 = 0, 1, 2
MHA_STATIC_WORKSPACE_BYTES = 32 << 20
MHA_MASK_NONE, MHA_MASK_CAUSAL, MHA_MASK_KEY_PADDING, MHA_MASK_CAUSAL_KEY_PADDING = 0, 1, 2, 3



class ScoreForm(ctypes.Structure):
    """mha_score_form of include/mha.h."""
    _fields_ = [("cap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("bucket_starts", ctypes.c_void_p), ("num_buckets", ctypes.c_int),
                ("bidirectional", ctypes.c_int), ("prefix_lens", ctypes.c_void_p),
                ("doc_ids", ctypes.c_void_p)]


class PagedCache(ctypes.Structure):
    """mha_paged_cache of include/mha.h."""
    _fields_ = [("dtype", ctypes.c_int), ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("page_stride", ctypes.c_longlong), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("row_starts", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("B", ctypes.c_int),
                ("h_kv", ctypes.c_int), ("page_rows", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("max_pages", ctypes.c_int)]


# The same as bytes, a call's fields in one packing (attribute by attribute they
# take longer than the launch); bytes pass as the pointer they are.
pack_paged_cache = struct.Struct("@iPPqPPPPPiiiii").pack

# Every symbol include/mha.h declares, with its ctypes signature.
_vp, _ci, _cf, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ll = ctypes.c_longlong
SIGNATURES = {
    "sdpa_forward": (_ci, [_ci, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _ci, _ci, _cf, _ci, _vp,
                           _vp, _vp]),
    "sdpa_forward_lse": (_ci, [_ci, _vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _ci, _ci, _cf,
                               _ci, _vp, _vp, _vp]),
    "sdpa_bf16_key_split": (_ci, [_ci, _ci, _ci]),
    "sdpa_forward_timeout_drill": (_ci, [_vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _cf, _ci, _vp,
                                         ctypes.c_ulonglong, _ci, _vp, _vp]),
    "sdpa_forward_host_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _ci, _ci, _ci]),
    "sdpa_forward_host": (_ci, [_ci, _vp, _vp, _vp, _vp, _vp, _sz, _ci, _ci, _ci, _ci, _ci, _ci,
                                _cf, _ci, _vp, _vp, _vp]),
    "sdpa_backward_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _ci, _ci]),
    "sdpa_backward": (_ci, [_ci, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _ci, _ci,
                            _ci, _ci, _ci, _ci, _cf, _ci, _vp, _vp, _vp]),
    "positional_encoding_add": (_ci, [_vp, _vp, _ci, _ci, _ci, _ci, _vp]),
    "encoder_layer_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _ci]),
    "encoder_layer_forward": (_ci, [_vp] * 13 + [_cf, _vp, _vp, _sz, _ci, _ci, _ci, _ci, _ci, _cf,
                                                _ci, _vp, _vp, _vp]),
    "sdpa_decode_forward": (_ci, [_vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _ci, _ci, _cf, _vp,
                                  _vp]),
    "sdpa_scored_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _vp]),
    "sdpa_scored_forward": (_ci, [_ci] + [_vp] * 7 + [_sz] + [_ci] * 7 +
                            [_cf, _ci, _vp, _vp, _vp, _vp]),
    "sdpa_scored_backward_workspace_bytes": (_sz, [_ci] * 5 + [_vp]),
    "sdpa_scored_backward": (_ci, [_ci] + [_vp] * 12 + [_sz] + [_ci] * 7 +
                             [_cf, _ci, _vp, _vp, _vp, _vp]),
    "sdpa_decode_shared_workspace_bytes": (_sz, [_ci] * 6 + [_vp]),
    "sdpa_decode_shared_forward": (_ci, [_vp] * 7 + [_sz] + [_ci] * 8 +
                                   [_cf, _ci, _vp, _vp, _vp, _vp]),
    "paged_cache_append": (_ci, [_vp, _vp, _ll, _ll, _vp, _ll, _ll, _ci, _ci, _vp]),
    "paged_cache_read": (_ci, [_vp, _vp, _vp, _ci, _ci, _vp]),
    "sdpa_paged_workspace_bytes": (_sz, [_vp, _ci, _ci, _ci]),
    "sdpa_paged_forward": (_ci, [_vp, _vp, _ll, _ll, _vp, _ll, _ll, _vp, _sz, _ci, _ci, _ci, _ci,
                                 _cf, _ci, _vp, _vp]),
    "mha_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _ci, _ci]),
    "mha_forward": (_ci, [_ci, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _ci, _ci, _ci, _ci,
                          _ci, _ci, _ci, _cf, _ci, _vp, _vp, _vp]),
    "mha_forward_add_layernorm": (_ci, [_ci, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _cf, _vp, _vp,
                                        _sz, _ci, _ci, _ci, _ci, _ci, _ci, _ci, _cf, _ci, _vp, _vp,
                                        _vp]),
    "mha_forward_static_workspace": (_ci, [_ci, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci,
                                           _ci, _ci, _ci, _ci, _cf, _ci, _vp, _vp, _vp]),
    "mha_status_string": (ctypes.c_char_p, [_ci]),
    "mha_last_error": (ctypes.c_char_p, []),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            "libmha.so is not built (%s); run transformer_scaled_dot_softmax_gb300.build.build() "
            "or __graft_entry__.build() -- there is no CPU fallback" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()
