"""ctypes binding of ``libqlin.so`` (the C ABI declared in ``include/qlin.h``).

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the CUDA stream, statuses become exceptions.  Every step of
the computation runs in the library's CUDA kernels (or, for t158_pack /
t158_unpack, its host C code).  If the library is not built this module
raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

from .build import LIB

T158_NMAT = 7
ERR_TIMEOUT = 5  # QLIN_ERR_TIMEOUT
_lock = threading.Lock()
_lib = None
_raw_stream = None  # torch's functions behind _stream, once CUDA is in use


class QlinError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        self.status = status
        super().__init__(f"{fn} -> {status_name(status)}: {detail}")


class T158ModelC(ctypes.Structure):
    """Mirror of ``t158_model``."""

    _fields_ = [
        ("n_layers", ctypes.c_int32), ("dim", ctypes.c_int32), ("n_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("ffn", ctypes.c_int32),
        ("vocab", ctypes.c_int32), ("max_pos", ctypes.c_int32),
        ("eps", ctypes.c_float), ("reserved0", ctypes.c_float),
        ("w", ctypes.c_void_p * T158_NMAT), ("pitch", ctypes.c_int64 * T158_NMAT),
        ("scales", ctypes.c_void_p), ("g_attn", ctypes.c_void_p), ("g_ffn", ctypes.c_void_p),
        ("g_final", ctypes.c_void_p), ("emb", ctypes.c_void_p), ("rope_cos", ctypes.c_void_p),
        ("rope_sin", ctypes.c_void_p),
    ]


class T158SketchC(ctypes.Structure):
    """Mirror of ``t158_sketch``."""

    _fields_ = [
        ("emb_t", ctypes.c_void_p), ("signs", ctypes.c_void_p), ("perm", ctypes.c_void_p), ("c_e", ctypes.c_void_p),
        ("k", ctypes.c_int32), ("n_cand", ctypes.c_int32),
    ]


class QlinKvC(ctypes.Structure):
    """Mirror of ``qlin_kv``."""

    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("seq_stride", ctypes.c_int64),
        ("row_stride", ctypes.c_int64), ("n_seqs", ctypes.c_int32), ("rows", ctypes.c_int32),
        ("type", ctypes.c_int32), ("reserved0", ctypes.c_int32),
    ]


KV_F32, KV_BF16 = 0, 1


class QlinKv4C(ctypes.Structure):
    """Mirror of ``qlin_kv4``."""

    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
        ("n_pages", ctypes.c_int32), ("page_rows", ctypes.c_int32), ("n_seqs", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
    ]


class T158PromptsC(ctypes.Structure):
    """Mirror of ``t158_prompts``."""

    _fields_ = [("kv", ctypes.c_void_p), ("len", ctypes.c_void_p), ("n_prompts", ctypes.c_int32),
                ("rows", ctypes.c_int32)]


class T158Kv4C(ctypes.Structure):
    """Mirror of ``t158_kv4``."""

    _fields_ = [("kv", QlinKv4C), ("code_bytes", ctypes.c_int64), ("scale_bytes", ctypes.c_int64)]


_P, _I, _I64, _F, _D, _SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                             ctypes.c_size_t)
_ST = ctypes.c_int
# name -> (argtypes, restype), in the order of include/qlin.h
SIGNATURES = {
    "qlin_status_str": ([_I], ctypes.c_char_p),
    "qlin_last_error": ([], ctypes.c_char_p),
    "qlin_version": ([], _I),
    "t158_pitch": ([_I64], _I64),
    "t158_pack": ([_P, _I64, _I64, _P, _I64], _ST),
    "t158_unpack": ([_P, _I64, _I64, _I64, _P], _ST),
    "qlin_w8_quantize": ([_P, _I64, _I64, _P, _I64, _P, _P], _ST),
    "qlin_quant_i8": ([_P, _P, _P, _I, _I, _P], _ST),
    "qlin_t158_i8": ([_P, _P, _P, _I64, _F, _P, _P, _I, _I, _I, _P], _ST),
    "qlin_t158_i8_workspace_size": ([_I, _I], _SZ),
    "qlin_t158_i8_ws": ([_P, _P, _P, _I64, _F, _P, _P, _I, _I, _I, _P, _SZ, _P], _ST),
    "qlin_w8_f32": ([_P, _P, _I64, _F, _P, _I, _I, _I, _P], _ST),
    "qlin_w8_f32_workspace_size": ([_I, _I], _SZ),
    "qlin_w8_f32_ws": ([_P, _P, _I64, _F, _P, _I, _I, _I, _P, _SZ, _P], _ST),
    "qlin_w8g_quantize": ([_P, _I64, _I64, _I, _P, _I64, _P, _I64, _P], _ST),
    "qlin_w8g_f32": ([_P, _P, _I64, _P, _I64, _I, _P, _I, _I, _I, _P], _ST),
    "qlin_embed_bf16": ([_P, _I, _I, _P, _P, _P, _P], _ST),
    "qlin_rmsnorm": ([_P, _P, _P, _I, _I, _F, _P], _ST),
    "t158_rope_table": ([_P, _P, _I, _I, _D, _P], _ST),
    "qlin_rope_kv_append": ([_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P], _ST),
    "qlin_attention_workspace_size": ([_I, _I, _I], _SZ),
    "qlin_attention_decode": ([_P, _P, _P, _I, _I, _I, _I, _P, _P, _SZ, _P], _ST),
    "qlin_attention_decode_noalloc": ([_P, _P, _P, _I, _I, _I, _I, _P, _P], _ST),
    "qlin_geglu": ([_P, _P, _P, _I, _P], _ST),
    "qlin_lm_head_workspace_size": ([_I], _SZ),
    "qlin_lm_head_argmax": ([_P, _P, _I, _I, _P, _P, _P, _SZ, _P], _ST),
    "qlin_sketch_emb_t_pitch": ([_I], ctypes.c_int64),
    "qlin_sketch_signs_bytes": ([_I, _I], _SZ),
    "qlin_sketch_prepare": ([_P, _I, _I, _P, _P, _P, _P, _P, _P], _ST),
    "qlin_sketch_workspace_size": ([_I], _SZ),
    "qlin_sketch_head": ([_P, _P, _P, _P, _P, _I, _I, _P, _I, _I, _P, _P, _P, _P, _P, _SZ, _P], _ST),
    "qlin_sketch_head_status": ([_P, _P], _ST),
    "decode_step_t158_workspace_size": ([ctypes.POINTER(T158ModelC), ctypes.POINTER(_SZ)], _ST),
    "decode_step_t158": ([ctypes.POINTER(T158ModelC), _P, _P, _SZ, _P, ctypes.c_int32, _P, _P, _P], _ST),
    "decode_step_t158_launches": ([ctypes.POINTER(T158ModelC)], _I),
    "decode_step_t158_status": ([_P, _P], _ST),
    "decode_step_t158_set_wait_limit": ([ctypes.c_uint64], None),
    "decode_step_t158_test_withhold": ([ctypes.c_int], None),
    "decode_step_t158_sketch_workspace_size": ([ctypes.POINTER(T158ModelC), ctypes.POINTER(T158SketchC),
                                                ctypes.POINTER(_SZ)], _ST),
    "decode_step_t158_sketch": ([ctypes.POINTER(T158ModelC), ctypes.POINTER(T158SketchC), _P, _P, _SZ, _P,
                                 ctypes.c_int32, _P, _P], _ST),
    "t158_group_pitch": ([_I64], _I64),
    "t158_pack_groups": ([_P, _I64, _I64, _P, _I64], _ST),
    "qlin_t158_skip_workspace_size": ([_I], _SZ),
    "qlin_t158_i8_skip": ([_P, _P, _P, _I64, _F, _P, _P, _I, _I, _P, _SZ, _P], _ST),
    "qlin_lm_head_lanes_workspace_size": ([_I, _I], _SZ),
    "qlin_lm_head_lanes": ([_P, _P, _I, _I, _I, _P, _P, _P, _SZ, _P], _ST),
    "qlin_lm_head_lanes_status": ([_P, _P], _ST),
    "decode_lanes_t158_workspace_size": ([ctypes.POINTER(T158ModelC), _I, ctypes.POINTER(_SZ)], _ST),
    "decode_lanes_t158": ([ctypes.POINTER(T158ModelC), _P, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _I, _P], _ST),
    "decode_lanes_t158_launches": ([ctypes.POINTER(T158ModelC), _I], _I),
    "decode_lanes_t158_status": ([_P, _P], _ST),
    "decode_step_t158_sketch_status": ([ctypes.POINTER(T158ModelC), ctypes.POINTER(T158SketchC), _P, _P], _ST),
    "qlin_attention_lanes_workspace_size": ([_I, _I, _I, _I], _SZ),
    "qlin_attention_on_tensor_cores": ([ctypes.POINTER(QlinKvC), ctypes.POINTER(QlinKvC), _I, _I, _I, _I, _I, _I], _I),
    "qlin_attention_lanes": ([_P, ctypes.POINTER(QlinKvC), _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P], _ST),
    "qlin_attention_prefix": ([_P, ctypes.POINTER(QlinKvC), _P, _P, ctypes.POINTER(QlinKvC), _P, _P, _I, _I, _I, _I,
                               _I, _I, _P, _P, _P, _SZ, _P], _ST),
    "decode_lanes_t158_prefix_workspace_size": ([ctypes.POINTER(T158ModelC), _I, ctypes.POINTER(_SZ)], _ST),
    "decode_lanes_t158_prefix": ([ctypes.POINTER(T158ModelC), ctypes.POINTER(T158PromptsC), _P, _P, _I, _I, _I, _P, _P,
                                  _P, _P, _P, _P, _SZ, _I, _P], _ST),
    "qlin_beam_select_workspace_size": ([_I, _I, _I, _I], _SZ),
    "qlin_beam_select": ([_P, _I64, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _SZ, _P], _ST),
    "qlin_beam_reorder": ([_P, _I64, _I64, _I, _I64, _I, _P, _P, _I, _I, _P, _P], _ST),
    "qlin_kv4_append": ([ctypes.POINTER(QlinKv4C), _P, _P, _I64, _P, _I64, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P,
                         _P], _ST),
    "qlin_kv4_read": ([ctypes.POINTER(QlinKv4C), _P, _P, _I, _I, _I, _P, _P, _P, _P], _ST),
    "qlin_sample": ([_P, _I64, _P, _P, _P, _P, _P, _I, _I, _P, _P, _P, _P], _ST),
    "qlin_attention_kv4_workspace_size": ([_I, _I, _I, _I], _SZ),
    "decode_lanes_t158_kv4_workspace_size": ([ctypes.POINTER(T158ModelC), _I, ctypes.POINTER(_SZ)], _ST),
    "decode_lanes_t158_kv4": ([ctypes.POINTER(T158ModelC), ctypes.POINTER(T158Kv4C), _I, _P, _P, _P, _P, _P, _P, _SZ, _I,
                               _P], _ST),
    "qlin_attention_kv4_on_tensor_cores": ([ctypes.POINTER(QlinKv4C), _I, _I, _I, _I, _I, _I], _I),
    "qlin_attention_kv4": ([_P, ctypes.POINTER(QlinKv4C), _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P], _ST),
}


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB):
                raise RuntimeError(f"{LIB} is missing: build it with `python -m weight_streaming_gemv_gb300.build` "
                                   "(there is no fallback implementation)")
            L = ctypes.CDLL(LIB)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = res
            _lib = L
    return _lib


def status_name(s: int) -> str:
    return lib().qlin_status_str(int(s)).decode()


def _check(fn: str, s: int):
    if s != 0:
        raise QlinError(fn, s, lib().qlin_last_error().decode())


def _ptr(t):
    """Device/host address of a torch tensor or numpy array; ints pass through; None is NULL."""
    if t is None:
        return None
    if type(t) is not int:
        try:  # (looking data_ptr up first: 0.16 us a tensor against 0.11, of nine in a call of 5)
            return t.data_ptr()
        except AttributeError:
            pass
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    if isinstance(t, int):
        return t
    raise TypeError(f"not a tensor, an array or an address: {type(t).__name__}")


def _stream(stream):
    if stream is None:
        global _raw_stream
        if _raw_stream is None:
            import torch
            current = torch.cuda.current_stream().cuda_stream  # (and CUDA is initialised from here on)
            c = torch._C
            # (current_stream() makes an object: 3 us of a 13 us call on a Grace core, this 0.2)
            if not (hasattr(c, "_cuda_getCurrentRawStream") and hasattr(c, "_cuda_getDevice")):
                return current
            _raw_stream = c._cuda_getCurrentRawStream, c._cuda_getDevice
        handle, device = _raw_stream
        return handle(device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------------ host packing
def t158_pitch(K: int) -> int:
    return int(lib().t158_pitch(K))


def t158_pack(trits: np.ndarray, pitch: int | None = None) -> np.ndarray:
    t = np.ascontiguousarray(trits, np.int8)
    N, K = t.shape
    pitch = t158_pitch(K) if pitch is None else pitch
    out = np.empty((N, pitch), np.uint8)
    _check("t158_pack", lib().t158_pack(_ptr(t), N, K, _ptr(out), pitch))
    return out


def t158_unpack(packed: np.ndarray, K: int) -> np.ndarray:
    pk = np.ascontiguousarray(packed, np.uint8)
    N, pitch = pk.shape
    out = np.empty((N, K), np.int8)
    _check("t158_unpack", lib().t158_unpack(_ptr(pk), N, K, pitch, _ptr(out)))
    return out


# ------------------------------------------------------------------ device calls
def qlin_w8_quantize(w, N, K, w8, w_pitch, scale, stream=None):
    _check("qlin_w8_quantize", lib().qlin_w8_quantize(_ptr(w), N, K, _ptr(w8), w_pitch, _ptr(scale), _stream(stream)))


def qlin_quant_i8(x, xq, x_scale, M, K, stream=None):
    _check("qlin_quant_i8", lib().qlin_quant_i8(_ptr(x), _ptr(xq), _ptr(x_scale), M, K, _stream(stream)))


def qlin_t158_i8(xq, x_scale, w_packed, w_pitch, w_scale, y, acc, M, N, K, stream=None):
    _check("qlin_t158_i8", lib().qlin_t158_i8(_ptr(xq), _ptr(x_scale), _ptr(w_packed), w_pitch, float(w_scale),
                                              _ptr(y), _ptr(acc), M, N, K, _stream(stream)))


def qlin_t158_i8_workspace_size(M, K):
    return int(lib().qlin_t158_i8_workspace_size(M, K))


def qlin_t158_i8_ws(xq, x_scale, w_packed, w_pitch, w_scale, y, acc, M, N, K, workspace, workspace_bytes,
                    stream=None):
    _check("qlin_t158_i8_ws", lib().qlin_t158_i8_ws(_ptr(xq), _ptr(x_scale), _ptr(w_packed), w_pitch,
                                                    float(w_scale), _ptr(y), _ptr(acc), M, N, K, _ptr(workspace),
                                                    workspace_bytes, _stream(stream)))


def qlin_w8_f32(x, w8, w_pitch, w_scale, y, M, N, K, stream=None):
    _check("qlin_w8_f32", lib().qlin_w8_f32(_ptr(x), _ptr(w8), w_pitch, float(w_scale), _ptr(y), M, N, K,
                                            _stream(stream)))


def qlin_w8_f32_workspace_size(M, K):
    return int(lib().qlin_w8_f32_workspace_size(M, K))


def qlin_w8_f32_ws(x, w8, w_pitch, w_scale, y, M, N, K, workspace, workspace_bytes, stream=None):
    _check("qlin_w8_f32_ws", lib().qlin_w8_f32_ws(_ptr(x), _ptr(w8), w_pitch, float(w_scale), _ptr(y), M, N, K,
                                                  _ptr(workspace), workspace_bytes, _stream(stream)))


def qlin_w8g_quantize(w, N, K, G, w8, w_pitch, scales, s_pitch, stream=None):
    _check("qlin_w8g_quantize", lib().qlin_w8g_quantize(_ptr(w), N, K, G, _ptr(w8), w_pitch, _ptr(scales), s_pitch,
                                                        _stream(stream)))


def qlin_w8g_f32(x, w8, w_pitch, scales, s_pitch, G, y, M, N, K, stream=None):
    _check("qlin_w8g_f32", lib().qlin_w8g_f32(_ptr(x), _ptr(w8), w_pitch, _ptr(scales), s_pitch, G, _ptr(y), M, N, K,
                                              _stream(stream)))


def qlin_embed_bf16(emb, vocab, dim, token, h, status_word=None, stream=None):
    _check("qlin_embed_bf16", lib().qlin_embed_bf16(_ptr(emb), vocab, dim, _ptr(token), _ptr(h), _ptr(status_word),
                                                    _stream(stream)))


def qlin_rmsnorm(x, gamma, out, M, n, eps, stream=None):
    _check("qlin_rmsnorm", lib().qlin_rmsnorm(_ptr(x), _ptr(gamma), _ptr(out), M, n, float(eps), _stream(stream)))


def t158_rope_table(cos_t, sin_t, max_pos, head_dim, base, stream=None):
    _check("t158_rope_table", lib().t158_rope_table(_ptr(cos_t), _ptr(sin_t), max_pos, head_dim, float(base),
                                                    _stream(stream)))


def qlin_rope_kv_append(q, k, v, k_cache, v_cache, cos_t, sin_t, pos, n_heads, n_kv, head_dim, stream=None):
    _check("qlin_rope_kv_append", lib().qlin_rope_kv_append(_ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache),
                                                            _ptr(cos_t), _ptr(sin_t), pos, n_heads, n_kv, head_dim,
                                                            _stream(stream)))


def qlin_attention_workspace_size(max_pos, n_heads, head_dim) -> int:
    return int(lib().qlin_attention_workspace_size(max_pos, n_heads, head_dim))


def qlin_attention_decode(q, k_cache, v_cache, pos, n_heads, n_kv, head_dim, out, workspace, workspace_bytes,
                          stream=None):
    _check("qlin_attention_decode", lib().qlin_attention_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), pos, n_heads,
                                                                n_kv, head_dim, _ptr(out), _ptr(workspace),
                                                                workspace_bytes, _stream(stream)))


ATTENTION_NOALLOC_SCRATCH_BYTES = 262144


def qlin_attention_decode_noalloc(q, k_cache, v_cache, pos, n_heads, n_kv, head_dim, out, stream=None):
    """Decode attention without a workspace argument, for callers that cannot allocate
    device memory: the partials go to a fixed 256 KiB array inside the library.  Calls
    that overlap on the GPU share that array and race."""
    _check("qlin_attention_decode_noalloc",
           lib().qlin_attention_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), pos, n_heads, n_kv, head_dim,
                                               _ptr(out), _stream(stream)))


def qlin_geglu(g, u, a, n, stream=None):
    _check("qlin_geglu", lib().qlin_geglu(_ptr(g), _ptr(u), _ptr(a), n, _stream(stream)))


def qlin_lm_head_workspace_size(vocab) -> int:
    return int(lib().qlin_lm_head_workspace_size(vocab))


def qlin_lm_head_argmax(emb, x, vocab, dim, logits, next_token, workspace, workspace_bytes, stream=None):
    _check("qlin_lm_head_argmax", lib().qlin_lm_head_argmax(_ptr(emb), _ptr(x), vocab, dim, _ptr(logits),
                                                            _ptr(next_token), _ptr(workspace), workspace_bytes,
                                                            _stream(stream)))


def qlin_sketch_emb_t_pitch(vocab) -> int:
    return int(lib().qlin_sketch_emb_t_pitch(vocab))


def qlin_sketch_signs_bytes(vocab, dim) -> int:
    return int(lib().qlin_sketch_signs_bytes(vocab, dim))


def qlin_sketch_prepare(emb, vocab, dim, dim_scale, emb_t, signs, perm, c_e, stream=None):
    _check("qlin_sketch_prepare", lib().qlin_sketch_prepare(_ptr(emb), vocab, dim, _ptr(dim_scale), _ptr(emb_t),
                                                            _ptr(signs), _ptr(perm), _ptr(c_e), _stream(stream)))


def qlin_sketch_workspace_size(vocab) -> int:
    return int(lib().qlin_sketch_workspace_size(vocab))


def qlin_sketch_head(emb, emb_t, signs, perm, c_e, vocab, dim, x, k, n_cand, approx, cand, cand_logits,
                     next_token, workspace, workspace_bytes, stream=None):
    _check("qlin_sketch_head", lib().qlin_sketch_head(
        _ptr(emb), _ptr(emb_t), _ptr(signs), _ptr(perm), _ptr(c_e), vocab, dim, _ptr(x), k, n_cand, _ptr(approx),
        _ptr(cand), _ptr(cand_logits), _ptr(next_token), _ptr(workspace), workspace_bytes, _stream(stream)))


def qlin_sketch_head_status(workspace, stream=None):
    _check("qlin_sketch_head_status", lib().qlin_sketch_head_status(_ptr(workspace), _stream(stream)))


def decode_step_t158_workspace_size(model: T158ModelC) -> int:
    n = ctypes.c_size_t()
    _check("decode_step_t158_workspace_size", lib().decode_step_t158_workspace_size(ctypes.byref(model), ctypes.byref(n)))
    return n.value


def decode_step_t158(model: T158ModelC, kv_cache, workspace, workspace_bytes, token, pos, logits, next_token,
                     stream=None):
    _check("decode_step_t158", lib().decode_step_t158(ctypes.byref(model), _ptr(kv_cache), _ptr(workspace),
                                                      workspace_bytes, _ptr(token), int(pos), _ptr(logits),
                                                      _ptr(next_token), _stream(stream)))


def decode_step_t158_launches(model: T158ModelC) -> int:
    return int(lib().decode_step_t158_launches(ctypes.byref(model)))


def decode_step_t158_status(workspace, stream=None):
    _check("decode_step_t158_status", lib().decode_step_t158_status(_ptr(workspace), _stream(stream)))


def decode_step_t158_set_wait_limit(ns: int):
    lib().decode_step_t158_set_wait_limit(int(ns))


def decode_step_t158_test_withhold(layer: int):
    lib().decode_step_t158_test_withhold(int(layer))


def decode_step_t158_sketch_workspace_size(model: T158ModelC, sk: T158SketchC) -> int:
    n = ctypes.c_size_t()
    _check("decode_step_t158_sketch_workspace_size",
           lib().decode_step_t158_sketch_workspace_size(ctypes.byref(model), ctypes.byref(sk), ctypes.byref(n)))
    return n.value


def decode_step_t158_sketch(model: T158ModelC, sk: T158SketchC, kv_cache, workspace, workspace_bytes, token, pos,
                            next_token, stream=None):
    _check("decode_step_t158_sketch", lib().decode_step_t158_sketch(
        ctypes.byref(model), ctypes.byref(sk), _ptr(kv_cache), _ptr(workspace), workspace_bytes, _ptr(token), pos,
        _ptr(next_token), _stream(stream)))


def decode_step_t158_sketch_status(model: T158ModelC, sk: T158SketchC, workspace, stream=None):
    _check("decode_step_t158_sketch_status", lib().decode_step_t158_sketch_status(
        ctypes.byref(model), ctypes.byref(sk), _ptr(workspace), _stream(stream)))


def decode_lanes_t158_workspace_size(model: T158ModelC, max_lanes: int) -> int:
    n = ctypes.c_size_t()
    _check("decode_lanes_t158_workspace_size",
           lib().decode_lanes_t158_workspace_size(ctypes.byref(model), max_lanes, ctypes.byref(n)))
    return n.value


def decode_lanes_t158(model: T158ModelC, kv_caches, n_seqs, n_lanes, tokens, positions, seqs, logits, next_tokens,
                      workspace, workspace_bytes, max_lanes, stream=None):
    _check("decode_lanes_t158", lib().decode_lanes_t158(
        ctypes.byref(model), _ptr(kv_caches), n_seqs, n_lanes, _ptr(tokens), _ptr(positions), _ptr(seqs),
        _ptr(logits), _ptr(next_tokens), _ptr(workspace), workspace_bytes, max_lanes, _stream(stream)))


def decode_lanes_t158_launches(model: T158ModelC, n_lanes: int) -> int:
    return int(lib().decode_lanes_t158_launches(ctypes.byref(model), n_lanes))


def decode_lanes_t158_status(workspace, stream=None):
    _check("decode_lanes_t158_status", lib().decode_lanes_t158_status(_ptr(workspace), _stream(stream)))


def qlin_lm_head_lanes_workspace_size(vocab, dim) -> int:
    return int(lib().qlin_lm_head_lanes_workspace_size(vocab, dim))


def qlin_lm_head_lanes(emb, x, vocab, dim, n_lanes, logits, next_tokens, workspace, workspace_bytes, stream=None):
    _check("qlin_lm_head_lanes", lib().qlin_lm_head_lanes(_ptr(emb), _ptr(x), vocab, dim, n_lanes, _ptr(logits),
                                                          _ptr(next_tokens), _ptr(workspace), workspace_bytes,
                                                          _stream(stream)))


def qlin_lm_head_lanes_status(workspace, stream=None):
    _check("qlin_lm_head_lanes_status", lib().qlin_lm_head_lanes_status(_ptr(workspace), _stream(stream)))


def t158_group_pitch(N: int) -> int:
    return int(lib().t158_group_pitch(N))


def t158_pack_groups(trits, gpitch=None):
    """Host packing by input group (for qlin_t158_i8_skip): [ceil(K/4)][gpitch] uint8."""
    t = np.ascontiguousarray(trits, np.int8)
    N, K = t.shape
    gpitch = t158_group_pitch(N) if gpitch is None else gpitch
    out = np.empty(((K + 3) // 4, gpitch), np.uint8)
    _check("t158_pack_groups", lib().t158_pack_groups(t.ctypes.data, N, K, out.ctypes.data, gpitch))
    return out


def qlin_t158_skip_workspace_size(N) -> int:
    return int(lib().qlin_t158_skip_workspace_size(N))


def qlin_t158_i8_skip(xq, x_scale, w_groups, gpitch, w_scale, y, acc, N, K, workspace, workspace_bytes, stream=None):
    _check("qlin_t158_i8_skip", lib().qlin_t158_i8_skip(_ptr(xq), _ptr(x_scale), _ptr(w_groups), gpitch, w_scale,
                                                        _ptr(y), _ptr(acc), N, K, _ptr(workspace), workspace_bytes,
                                                        _stream(stream)))


def kv_cache(k, v) -> QlinKvC:
    """The ``qlin_kv`` of two tensors [n_seqs][rows][n_kv * head_dim] (float32, bfloat16, or int16 holding bf16
    bits; any strides but the last's), which the caller keeps."""
    if k.dim() != 3 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.stride(2) != 1:
        raise ValueError("kv_cache: k and v are [n_seqs][rows][n_kv * head_dim] tensors of one shape, type and "
                         "strides, the last axis contiguous")
    kinds = {"torch.float32": KV_F32, "torch.bfloat16": KV_BF16, "torch.int16": KV_BF16}
    if str(k.dtype) not in kinds:
        raise ValueError(f"kv_cache: type {k.dtype}")
    c = QlinKvC()
    c.k, c.v, c.type = k.data_ptr(), v.data_ptr(), kinds[str(k.dtype)]
    c.seq_stride, c.row_stride = k.stride(0), k.stride(1)
    c.n_seqs, c.rows = k.shape[0], k.shape[1]
    return c


def qlin_attention_lanes_workspace_size(n_lanes, n_heads, n_kv, head_dim) -> int:
    return int(lib().qlin_attention_lanes_workspace_size(n_lanes, n_heads, n_kv, head_dim))


def qlin_attention_on_tensor_cores(prefix, kv: QlinKvC, n_lanes, n_heads, n_kv, head_dim, window, sinks) -> bool:
    r = lib().qlin_attention_on_tensor_cores(None if prefix is None else ctypes.byref(prefix), ctypes.byref(kv), n_lanes,
                                             n_heads, n_kv, head_dim, window, sinks)
    if r < 0:
        _check("qlin_attention_on_tensor_cores", -r)
    return bool(r)


def qlin_attention_lanes(q, kv: QlinKvC, positions, seqs, n_lanes, n_heads, n_kv, head_dim, window, sinks, out,
                         status_word, workspace, workspace_bytes, stream=None):
    _check("qlin_attention_lanes", lib().qlin_attention_lanes(
        _ptr(q), ctypes.byref(kv), _ptr(positions), _ptr(seqs), n_lanes, n_heads, n_kv, head_dim, window, sinks,
        _ptr(out), _ptr(status_word), _ptr(workspace), workspace_bytes, _stream(stream)))


def qlin_attention_prefix(q, prefix: QlinKvC, prefix_len, prefix_of, kv: QlinKvC, positions, seqs, n_lanes, n_heads,
                          n_kv, head_dim, window, sinks, out, status_word, workspace, workspace_bytes, stream=None):
    _check("qlin_attention_prefix", lib().qlin_attention_prefix(
        _ptr(q), ctypes.byref(prefix), _ptr(prefix_len), _ptr(prefix_of), ctypes.byref(kv), _ptr(positions),
        _ptr(seqs), n_lanes, n_heads, n_kv, head_dim, window, sinks, _ptr(out), _ptr(status_word), _ptr(workspace),
        workspace_bytes, _stream(stream)))


def decode_lanes_t158_prefix_workspace_size(model: T158ModelC, max_lanes: int) -> int:
    n = ctypes.c_size_t()
    _check("decode_lanes_t158_prefix_workspace_size",
           lib().decode_lanes_t158_prefix_workspace_size(ctypes.byref(model), max_lanes, ctypes.byref(n)))
    return n.value


def decode_lanes_t158_prefix(model: T158ModelC, prompts: T158PromptsC, prefix_of, kv_caches, own_rows, n_seqs, n_lanes,
                             tokens, positions, seqs, logits, next_tokens, workspace, workspace_bytes, max_lanes,
                             stream=None):
    _check("decode_lanes_t158_prefix", lib().decode_lanes_t158_prefix(
        ctypes.byref(model), ctypes.byref(prompts), _ptr(prefix_of), _ptr(kv_caches), own_rows, n_seqs, n_lanes,
        _ptr(tokens), _ptr(positions), _ptr(seqs), _ptr(logits), _ptr(next_tokens), _ptr(workspace), workspace_bytes,
        max_lanes, _stream(stream)))


def qlin_beam_select_workspace_size(n_groups, beams, vocab, n_out) -> int:
    return int(lib().qlin_beam_select_workspace_size(n_groups, beams, vocab, n_out))


def qlin_beam_select(logits, row_stride, scores, finished, eos, n_groups, beams, vocab, n_out, out_scores, parents,
                     tokens, workspace, workspace_bytes, stream=None):
    _check("qlin_beam_select", lib().qlin_beam_select(
        _ptr(logits), row_stride, _ptr(scores), _ptr(finished), eos, n_groups, beams, vocab, n_out, _ptr(out_scores),
        _ptr(parents), _ptr(tokens), _ptr(workspace), workspace_bytes, _stream(stream)))


def qlin_beam_reorder(cache, seq_stride, plane_stride, n_planes, row_bytes, max_rows, parents, n_rows, n_groups,
                      beams, status_word=None, stream=None):
    _check("qlin_beam_reorder", lib().qlin_beam_reorder(
        _ptr(cache), seq_stride, plane_stride, n_planes, row_bytes, max_rows, _ptr(parents), _ptr(n_rows), n_groups,
        beams, _ptr(status_word), _stream(stream)))


def kv4_cache(k, v, k_scale, v_scale, table) -> QlinKv4C:
    """The ``qlin_kv4`` of four contiguous uint8 tensors, codes [n_pages][n_kv][page_rows][head_dim / 2] and scales
    [n_pages][n_kv][page_rows][head_dim / 32], and an int32 table [n_seqs][pages of a sequence] (any stride between
    its rows from a row on), all on one device, which the caller keeps."""
    for t in (k, v, k_scale, v_scale):
        if t.dim() != 4 or str(t.dtype) != "torch.uint8" or not t.is_contiguous() or t.shape[:3] != k.shape[:3]:
            raise ValueError("kv4_cache: codes and scales are contiguous uint8 tensors [n_pages][n_kv][page_rows][...]")
    if v.shape != k.shape or k.shape[3] != 16 * k_scale.shape[3] or v_scale.shape != k_scale.shape:
        raise ValueError(f"kv4_cache: codes {tuple(k.shape)}, {tuple(v.shape)} and scales {tuple(k_scale.shape)}, "
                         f"{tuple(v_scale.shape)}")
    if table.dim() != 2 or str(table.dtype) != "torch.int32" or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("kv4_cache: the table is int32 [n_seqs][pages], its rows contiguous")
    if any(t.device != k.device for t in (v, k_scale, v_scale, table)):
        raise ValueError("kv4_cache: codes, scales and the table are on one device")
    if table.shape[0] > 1 and table.stride(0) < table.shape[1]:
        raise ValueError(f"kv4_cache: the table's rows of {table.shape[1]} pages lie in one another (stride {table.stride(0)})")
    c = QlinKv4C()
    c.k, c.v, c.k_scale, c.v_scale = k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr()
    c.table, c.table_stride = table.data_ptr(), max(table.stride(0), table.shape[1])
    c.n_pages, c.page_rows = k.shape[0], k.shape[2]
    c.n_seqs, c.max_pages = table.shape
    return c


def qlin_kv4_append(kv: QlinKv4C, k, v, kv_stride, q, q_stride, q_out, cos_t, sin_t, rope_rows, positions, seqs,
                    n_lanes, n_heads, n_kv, head_dim, status_word=None, stream=None):
    _check("qlin_kv4_append", lib().qlin_kv4_append(
        ctypes.byref(kv), _ptr(k), _ptr(v), kv_stride, _ptr(q), q_stride, _ptr(q_out), _ptr(cos_t), _ptr(sin_t),
        rope_rows, _ptr(positions), _ptr(seqs), n_lanes, n_heads, n_kv, head_dim, _ptr(status_word), _stream(stream)))


def qlin_kv4_read(kv: QlinKv4C, positions, seqs, n_lanes, n_kv, head_dim, k_out, v_out, status_word=None, stream=None):
    _check("qlin_kv4_read", lib().qlin_kv4_read(
        ctypes.byref(kv), _ptr(positions), _ptr(seqs), n_lanes, n_kv, head_dim, _ptr(k_out), _ptr(v_out),
        _ptr(status_word), _stream(stream)))


def qlin_attention_kv4_workspace_size(n_lanes, n_heads, n_kv, head_dim) -> int:
    return int(lib().qlin_attention_kv4_workspace_size(n_lanes, n_heads, n_kv, head_dim))


def qlin_attention_kv4_on_tensor_cores(kv: QlinKv4C, n_lanes, n_heads, n_kv, head_dim, window, sinks) -> bool:
    r = lib().qlin_attention_kv4_on_tensor_cores(ctypes.byref(kv), n_lanes, n_heads, n_kv, head_dim, window, sinks)
    if r < 0:
        _check("qlin_attention_kv4_on_tensor_cores", -r)
    return bool(r)


def qlin_attention_kv4(q, kv: QlinKv4C, positions, seqs, n_lanes, n_heads, n_kv, head_dim, window, sinks, out,
                       status_word, workspace, workspace_bytes, stream=None):
    _check("qlin_attention_kv4", lib().qlin_attention_kv4(
        _ptr(q), ctypes.byref(kv), _ptr(positions), _ptr(seqs), n_lanes, n_heads, n_kv, head_dim, window, sinks,
        _ptr(out), _ptr(status_word), _ptr(workspace), workspace_bytes, _stream(stream)))


def qlin_sample(logits, row_stride, u, temperature, top_k, top_p, min_p, n_rows, vocab, tokens, probs=None, kept=None,
                stream=None):
    _check("qlin_sample", lib().qlin_sample(
        _ptr(logits), row_stride, _ptr(u), _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p), n_rows, vocab,
        _ptr(tokens), _ptr(probs), _ptr(kept), _stream(stream)))


def decode_lanes_t158_kv4_workspace_size(model: T158ModelC, max_lanes: int) -> int:
    n = ctypes.c_size_t()
    _check("decode_lanes_t158_kv4_workspace_size",
           lib().decode_lanes_t158_kv4_workspace_size(ctypes.byref(model), max_lanes, ctypes.byref(n)))
    return n.value


def decode_lanes_t158_kv4(model: T158ModelC, cache: T158Kv4C, n_lanes, tokens, positions, seqs, logits, next_tokens,
                          workspace, workspace_bytes, max_lanes, stream=None):
    _check("decode_lanes_t158_kv4", lib().decode_lanes_t158_kv4(
        ctypes.byref(model), ctypes.byref(cache), n_lanes, _ptr(tokens), _ptr(positions), _ptr(seqs), _ptr(logits),
        _ptr(next_tokens), _ptr(workspace), workspace_bytes, max_lanes, _stream(stream)))
