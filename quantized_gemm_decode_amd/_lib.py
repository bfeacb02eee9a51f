"""ctypes declarations of the C ABI in include/qlinear.h (argument marshalling only)."""

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libqlinear.so")

c_i32, c_i64, c_vp, c_cp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_char_p


class QLConfig(ctypes.Structure):
    _fields_ = [(n, c_i32) for n in ("algo", "swap_ab", "split_k", "waves_n", "waves_k", "rows_per_wave",
                                     "prefetch", "a_mode", "w_lds", "w_layout", "tile_m", "tile_n")]


class QLPlanFacts(ctypes.Structure):
    _fields_ = [("source", c_i32), ("chunks", c_i32), ("chunk_k", c_i32), ("workgroups", c_i32),
                ("threads", c_i32), ("lds_bytes", c_i32), ("workspace_bytes", c_i64), ("epilogue", c_i32)]


class QLRows(ctypes.Structure):
    _fields_ = [("data", c_vp), ("token_stride", c_i64), ("head_stride", c_i64)]


class QLKvCache(ctypes.Structure):
    _fields_ = ([(n, c_vp) for n in ("k", "v", "k_scale", "v_scale")]
                + [(n, c_i64) for n in ("k_page_stride", "k_token_stride", "k_head_stride", "v_page_stride",
                                        "v_token_stride", "v_head_stride", "num_pages")]
                + [(n, c_i32) for n in ("type", "page_size", "kv_heads", "head_dim")])


class QLNormRope(ctypes.Structure):
    _fields_ = [("q_weight", c_vp), ("k_weight", c_vp), ("cos_sin", c_vp), ("max_pos", c_i64), ("rot_dim", c_i32),
                ("interleaved", c_i32), ("eps", ctypes.c_float)]


class QLAttentionShape(ctypes.Structure):
    _fields_ = ([(n, c_i64) for n in ("batch", "tokens", "max_q", "max_kv")]
                + [(n, c_i32) for n in ("q_heads", "kv_heads", "head_dim", "page_size", "kv_type", "causal", "window")]
                + [("scale", ctypes.c_float)])


class QLAttentionFacts(ctypes.Structure):
    _fields_ = [(n, c_i32) for n in ("stream_rows", "slots", "tile_rows", "row_blocks", "splits", "chunk")] + [("workspace_bytes", c_i64)]


c_rows, c_cache = ctypes.POINTER(QLRows), ctypes.POINTER(QLKvCache)

# name -> (restype, argtypes); exactly the functions declared in include/qlinear.h
SIGNATURES = {
    "qlinear_version": (c_i32, []),
    "qlinear_status_string": (c_cp, [c_i32]),
    "qlinear_last_error": (c_cp, []),
    "qlinear_quantize_act": (c_i32, [c_i32, c_vp, c_i64, c_i64, c_vp, c_vp, c_vp]),
    "qlinear_quantize_weight": (c_i32, [c_i32, c_vp, c_i64, c_i64, c_vp, c_vp, c_vp]),
    "qlinear_packed_act_bytes": (c_i64, [c_i64, c_i64]),
    "qlinear_quantize_act_packed": (c_i32, [c_i32, c_vp, c_i64, c_i64, c_vp, c_vp, c_vp]),
    "qlinear_packed_weight_bytes": (c_i64, [c_i64, c_i64]),
    "qlinear_encode_e4m3": (c_i32, [c_vp, c_i64, c_vp, c_vp]),
    "qlinear_stream_read": (c_i32, [c_vp, c_i64, c_i32, c_i32, c_i32, c_vp, c_vp]),
    "qlinear_stream_read_bcast": (c_i32, [c_vp, c_i64, c_vp, c_i64, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp]),
    "qlinear_pack_weight": (c_i32, [c_vp, c_i64, c_i64, c_vp, c_vp]),
    "qlinear_packed_mx_scale_bytes": (c_i64, [c_i64, c_i64]),
    "qlinear_packed_weight_bytes_fp4": (c_i64, [c_i64, c_i64]),
    "qlinear_pack_weight_fp4": (c_i32, [c_vp, c_i64, c_i64, c_vp, c_vp]),
    "qlinear_pack_mx_scales": (c_i32, [c_vp, c_i64, c_i64, c_vp, c_vp]),
    "qlinear_table_load": (c_i32, [c_cp, ctypes.POINTER(c_i64)]),
    "qlinear_table_clear": (None, []),
    "qlinear_plan": (c_i32, [c_i32, c_i64, c_i64, c_i64, ctypes.POINTER(c_vp)]),
    "qlinear_plan_packed": (c_i32, [c_i32, c_i64, c_i64, c_i64, ctypes.POINTER(c_vp)]),
    "qlinear_plan_layouts": (c_i32, [c_i32, c_i64, c_i64, c_i64, c_i32, c_i32, ctypes.POINTER(c_vp)]),
    "qlinear_plan_from_table": (c_i32, [c_i32, c_i64, c_i64, c_i64, ctypes.POINTER(c_vp)]),
    "qlinear_plan_with_config": (c_i32, [c_i32, c_i64, c_i64, c_i64, ctypes.POINTER(QLConfig),
                                         ctypes.POINTER(c_vp)]),
    "qlinear_plan_info": (c_i32, [c_vp, ctypes.POINTER(QLConfig), ctypes.POINTER(QLPlanFacts)]),
    "qlinear_plan_glu": (c_i32, [c_i32, c_i64, c_i64, c_i64, c_i32, ctypes.POINTER(c_vp)]),
    "qlinear_plan_glu_with_config": (c_i32, [c_i32, c_i64, c_i64, c_i64, ctypes.POINTER(QLConfig),
                                             ctypes.POINTER(c_vp)]),
    "qlinear_workspace_bytes": (c_i64, [c_vp]),
    "qlinear_plan_destroy": (None, [c_vp]),
    "qlinear_run": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "qlinear_run_debug_acc": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "qlinear_forward": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "qlinear_forward_noalloc": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "qlinear_forward_glu_amax": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "qlinear_forward_amax": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "qlinear_qk_norm_rope": (c_i32, [ctypes.POINTER(QLNormRope), c_i64, c_i32, c_i32, c_i32, c_rows, c_rows, c_vp, c_rows,
                                     c_rows, c_vp]),
    "qlinear_qkv_append": (c_i32, [ctypes.POINTER(QLNormRope), c_i64, c_i32, c_rows, c_rows, c_rows, c_vp, c_vp, c_rows,
                                   c_cache, c_vp]),
    "qlinear_attention_plan": (c_i32, [ctypes.POINTER(QLAttentionShape), ctypes.POINTER(c_vp)]),
    "qlinear_attention_plan_info": (c_i32, [c_vp, ctypes.POINTER(QLAttentionFacts)]),
    "qlinear_attention_workspace_bytes": (c_i64, [c_vp]),
    "qlinear_attention_plan_destroy": (None, [c_vp]),
    "qlinear_attention": (c_i32, [c_vp, c_rows, c_cache, c_vp, c_i64, c_vp, c_vp, c_rows, c_vp, c_vp, c_vp]),
    "qlinear_verify_workspace_bytes": (c_i64, [c_i64, c_i64]),
    "qlinear_verify_draft": (c_i32, [c_i64] * 4 + [c_vp] * 10),
    "qlinear_graph_begin": (c_i32, [c_vp]),
    "qlinear_graph_end": (c_i32, [c_vp, ctypes.POINTER(c_vp)]),
    "qlinear_graph_launch": (c_i32, [c_vp, c_vp]),
    "qlinear_graph_destroy": (None, [c_vp]),
}

_lib = None


def load(path=LIB_PATH):
    """Load libqlinear.so (built in-tree) and declare every exported function.

    Raises OSError when the library is missing: there is no fallback path.
    """
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError("libqlinear.so is not built (%s); run python -m quantized_gemm_decode_amd.build" % path)
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib
