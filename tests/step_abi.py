"""The C ABI of include/qlora_step.h through ctypes, for the tests."""
import ctypes

import decoder_abi as dec

_vp, _i64, _i32, _sz, _f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float


class Rows(ctypes.Structure):
    _fields_ = [("data", _vp), ("stride", _i64)]


class Norm(ctypes.Structure):
    _fields_ = [("pre", _vp), ("post", _vp), ("gate", _vp), ("gate_rows", _i64), ("norm_pre", _i32), ("norm_post", _i32),
                ("dtype", ctypes.c_int), ("scale", _f), ("eps", _f)]


class Tensor(ctypes.Structure):
    _fields_ = [("data", _vp), ("n", _i64), ("dtype", ctypes.c_int)]


class Rules(ctypes.Structure):
    _fields_ = [("history", _vp), ("history_stride", _i64), ("history_width", _i64), ("lengths", _vp), ("prompts", _vp),
                ("repetition", _f), ("presence", _f), ("frequency", _f), ("repetitions", _vp), ("presences", _vp),
                ("frequencies", _vp), ("bias_ids", _vp), ("bias_ids_stride", _i64), ("bias", _vp), ("bias_stride", _i64),
                ("biases", _i64), ("allowed", _vp), ("allowed_stride", _i64)]


def library():
    L = dec._library()
    p = ctypes.POINTER
    L.qlora_block_norm_fwd.restype = ctypes.c_int
    L.qlora_block_norm_fwd.argtypes = [p(Norm), _i64, _i64, ctypes.c_int] + [p(Rows)] * 4 + [_vp]
    L.qlora_block_norm_bwd.restype = ctypes.c_int
    L.qlora_block_norm_bwd.argtypes = [p(Norm), _i64, _i64, ctypes.c_int] + [p(Rows)] * 6 + [_vp, _vp, _vp, _vp, _sz, _vp]
    L.qlora_block_norm_bwd_workspace_bytes.restype = _sz
    L.qlora_block_norm_bwd_workspace_bytes.argtypes = [_i64, _i64, _i64, _i32, _i32, _i32]
    L.qlora_grad_norm_workspace_bytes.restype = _sz
    L.qlora_grad_norm_workspace_bytes.argtypes = [p(Tensor), _i64]
    L.qlora_grad_norm.restype = ctypes.c_int
    L.qlora_grad_norm.argtypes = [p(Tensor), _i64, ctypes.c_double, _vp, _vp, _vp, _sz, _vp]
    L.qlora_grad_clip_workspace_bytes.restype = _sz
    L.qlora_grad_clip_workspace_bytes.argtypes = [p(Tensor), _i64]
    L.qlora_grad_clip.restype = ctypes.c_int
    L.qlora_grad_clip.argtypes = [p(Tensor), p(Tensor), _i64, ctypes.c_double, _vp, _vp, _sz, _vp]
    L.qlora_kv_attention_window_workspace_bytes.restype = _sz
    L.qlora_kv_attention_window_workspace_bytes.argtypes = [p(dec._Cache), p(dec._Batch), _i32, _i64, _i64, _i64, _i64]
    L.qlora_kv_attention_window.restype = ctypes.c_int
    L.qlora_kv_attention_window.argtypes = [p(dec._Cache), p(dec._Batch), p(dec._Heads), p(dec._Heads), _f, _i64, _i64, _i64, _i64,
                                            _vp, _sz, _vp]
    L.qlora_logits_shape.restype = ctypes.c_int
    L.qlora_logits_shape.argtypes = [p(Rules), _i64, _i64, ctypes.c_int, p(Rows), p(Rows), _vp]
    return L
