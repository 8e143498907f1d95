"""ctypes binding of ``libmclayer.so`` (the C ABI in ``include/mc_layer.h``).

Argument marshalling only: every function here has the name of the C entry
point it calls and forwards plain integers (device pointers, sizes, a
cudaStream_t handle).  Anything with a ``data_ptr()`` method (a torch tensor)
is accepted where a pointer is expected.  No computation happens in Python.

The index and constant arrays of positions and masks (offsets, prefixes, key
bounds, tables, positions, inverse frequencies, slopes) come as int64 or as
expanded views easily, which a pointer does not show: given as tensors, their
type, layout and length are checked here (TypeError, ValueError).  Without a
`stream` those calls go to torch's current one; the other stage calls to the
legacy default stream, which side streams are not ordered with.
"""
from __future__ import annotations

import ctypes
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
# MC_LAYER_DEBUG=1 selects the debug build (-DMC_DEBUG: every global store's
# indices are checked on the device; see build.py).
LIB_PATH = os.path.join(PKG_DIR, "libmclayer_debug.so" if os.environ.get("MC_LAYER_DEBUG") == "1"
                        else "libmclayer.so")

MC_OK = 0
MC_ERR_SHAPE = -1
MC_ERR_UNSUPPORTED = -2
MC_ERR_NULLPTR = -3
MC_ERR_ALIGN = -4
MC_ERR_WORKSPACE = -5
MC_ERR_CUDA = -6
MC_ERR_DEVICE_TIMEOUT = -7
MC_ERR_DEVICE_BOUNDS = -8
MC_ERR_ARGUMENT = -9
MC_ERR_SCRATCH_LIMIT = -10

MC_ACCUMULATE_GRADS = 1
MC_RECOMPUTE_ACTIVATIONS = 2
MC_SEQUENCE_PARALLEL = 4
MC_FP8_HYBRID = 8
MC_ATTN_DQ_RECOMPUTE = 16
MC_BUILD_DEBUG = 1
MC_BUILD_NVTX = 2

MC_EPI_STORE_F32 = 0
MC_EPI_STORE_BF16 = 1
MC_EPI_BIAS_BF16 = 2
MC_EPI_BIAS_GELU = 3
MC_EPI_BIAS_RESID_F32 = 4
MC_EPI_GELU_BWD = 5

PARAM_ORDER = ("ln1_g", "ln1_b", "w_qkv", "b_qkv", "w_o", "b_o",
               "ln2_g", "ln2_b", "w_fc1", "b_fc1", "w_fc2", "b_fc2")


class McError(RuntimeError):
    def __init__(self, code: int, where: str = ""):
        self.code = code
        super().__init__(f"{where}: {code} ({mc_strerror(code)})" if where else
                         f"{code} ({mc_strerror(code)})")


class mc_layer_shape(ctypes.Structure):  # noqa: N801 (C name)
    _fields_ = [("micro_batch", ctypes.c_int32), ("seq_len", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("ffn_hidden", ctypes.c_int32), ("tp_parts", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class mc_layer_weights(ctypes.Structure):  # noqa: N801
    _fields_ = [(n, ctypes.c_void_p) for n in PARAM_ORDER]


class mc_layer_grads(ctypes.Structure):  # noqa: N801
    _fields_ = [(n, ctypes.c_void_p) for n in PARAM_ORDER]


MC_ROTARY_MAX_AXES = 4
MC_ROTARY_ADJACENT_PAIRS = 1
MC_ROTARY_DEAL_AXES = 2
_RotarySections = ctypes.c_int32 * MC_ROTARY_MAX_AXES


class mc_rotary_spec(ctypes.Structure):  # noqa: N801
    _fields_ = [("rot_dim", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("sections", _RotarySections), ("flags", ctypes.c_uint32)]


class mc_attention_options(ctypes.Structure):  # noqa: N801
    lengths = (1 << 62,) * 3  # rows, table integers, slopes (make_attention_options)
    _fields_ = [("key_lo", ctypes.c_void_p), ("key_hi", ctypes.c_void_p),
                ("tables", ctypes.c_void_p), ("slopes", ctypes.c_void_p),
                ("softcap", ctypes.c_float), ("causal", ctypes.c_int32)]


class mc_layer_rotary(ctypes.Structure):  # noqa: N801
    length = 1 << 62  # of positions (make_layer_rotary)
    _fields_ = [("spec", mc_rotary_spec), ("positions", ctypes.c_void_p),
                ("inv_freq", ctypes.c_void_p)]


MC_QK_NORM_CENTRED = 1


class mc_qk_norm(ctypes.Structure):  # noqa: N801
    lengths = (1 << 62,) * 2  # shortest of the queries' and of the keys' arrays (make_qk_norm)
    _fields_ = [("q_gain", ctypes.c_void_p), ("q_shift", ctypes.c_void_p),
                ("k_gain", ctypes.c_void_p), ("k_shift", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("flags", ctypes.c_uint32)]


class mc_qk_norm_grads(ctypes.Structure):  # noqa: N801
    lengths = (1 << 62,) * 2
    _fields_ = [("q_gain", ctypes.c_void_p), ("q_shift", ctypes.c_void_p),
                ("k_gain", ctypes.c_void_p), ("k_shift", ctypes.c_void_p)]


class mc_layer_qk_norm(ctypes.Structure):  # noqa: N801
    parts = (None, None)  # norm and gradients with their lengths (make_layer_qk_norm)
    _fields_ = [("norm", mc_qk_norm), ("grads", mc_qk_norm_grads)]


class mc_cross_attention(ctypes.Structure):  # noqa: N801
    _fields_ = [("sequences", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("q_rows", ctypes.c_int32), ("kv_rows", ctypes.c_int32),
                ("max_q", ctypes.c_int32), ("max_kv", ctypes.c_int32),
                ("ld_q", ctypes.c_int64), ("ld_kv", ctypes.c_int64), ("ld_o", ctypes.c_int64),
                ("q_offsets", ctypes.c_void_p), ("q_lens", ctypes.c_void_p),
                ("kv_offsets", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
                ("scale", ctypes.c_float)]


_lib = None

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_SZ = ctypes.c_size_t

_OPT = ctypes.POINTER(mc_attention_options)
_ROT = ctypes.POINTER(mc_layer_rotary)
_NORM = ctypes.POINTER(mc_qk_norm)
_LNORM = ctypes.POINTER(mc_layer_qk_norm)
_CROSS = ctypes.POINTER(mc_cross_attention)

_SIGNATURES = {
    "mc_layer_check_shape": (_INT, [ctypes.POINTER(mc_layer_shape)]),
    "mc_layer_saved_bytes": (_SZ, [ctypes.POINTER(mc_layer_shape)]),
    "mc_layer_workspace_bytes": (_SZ, [ctypes.POINTER(mc_layer_shape)]),
    "mc_layer_forward": (_INT, [ctypes.POINTER(mc_layer_shape), ctypes.POINTER(mc_layer_weights),
                                _P, _P, _P, _P, _SZ, _P]),
    "mc_layer_backward": (_INT, [ctypes.POINTER(mc_layer_shape), ctypes.POINTER(mc_layer_weights),
                                 _P, _P, _P, _P, ctypes.POINTER(mc_layer_grads), _P, _SZ, _P]),
    "mc_layer_device_status": (_INT, [_P, _P]),
    "mc_strerror": (ctypes.c_char_p, [_INT]),
    "mc_layernorm_forward": (_INT, [_P, _P, _P, _P, _P, _P, _I64, _I32, _P, _P]),
    "mc_layernorm_backward": (_INT, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _INT, _P,
                                     _I64, _I32, _P, _P]),
    "mc_layernorm_backward_scratch_floats": (_SZ, [_I64, _I32]),
    "mc_gemm": (_INT, [_I64, _I64, _I64, _P, _I64, _INT, _P, _I64, _INT, _P, _I64, _INT, _P, _P,
                       _I64, _INT, _INT, _P, _P]),
    "mc_attention_forward": (_INT, [_P, _P, _P, _I32, _I32, _I32, _I32, _P, _P]),
    "mc_attention_backward": (_INT, [_P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _P]),
    "mc_attention_backward_noalloc": (_INT, [_P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _P]),
    "mc_attention_backward_ws_bytes": (_SZ, [_I32, _I32, _I32, _I32]),
    "mc_build_features": (_INT, []),
    "mc_attention_backward_ws": (_INT, [_P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _SZ,
                                        _P, _P]),
    "mc_selftest_wait_timeout": (_INT, [_I64, _P, _P]),
    "mc_selftest_bounds_check": (_INT, [_I64, _I64, _P, _P, _P]),
    "mc_fp8_scratch_floats": (_SZ, []),
    "mc_fp8_quantize": (_INT, [_P, _I32, _I64, _I32, _P, _P, _P, _P, _P]),
    "mc_fp8_quantize_2d": (_INT, [_P, _I32, _I64, _I64, _I32, _P, _P, _P, _P, _P]),
    "mc_gemm_fp8": (_INT, [_I64, _I64, _I64, _P, _I64, _I32, _P, _I64, _I32, _P, _P, _P, _I64,
                           _I32, _P, _P, _I64, _I32, _I32, _P, _P]),
    "mc_cp_schedule": (_INT, [_I32, _I32, _I32, ctypes.POINTER(_I32)]),
    "mc_cp_launch_plan": (_INT, [_I32, ctypes.POINTER(_I32), _I32]),
    "mc_attention_cp_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "mc_attention_forward_cp": (_INT, [_P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _SZ, _P, _P]),
    "mc_attention_backward_cp": (_INT, [_P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P,
                                        _SZ, _P, _P]),
    "mc_rotary_forward": (_INT, [_P, _P, _I32, _I64, _I32, _I32, _I64, _I64, _P, _P,
                                 ctypes.POINTER(mc_rotary_spec), _P, _P]),
    "mc_rotary_backward": (_INT, [_P, _P, _I32, _I64, _I32, _I32, _I64, _I64, _P, _P,
                                  ctypes.POINTER(mc_rotary_spec), _P, _P]),
    "mc_attention_mask_table_ints": (_SZ, [_I32, _I32]),
    "mc_attention_mask_documents": (_INT, [_P, _I32, _P, _I32, _I32, _I32, _I32, _P, _P, _P, _P,
                                           _P]),
    "mc_attention_mask_intervals": (_INT, [_I32, _I32, _P, _P, _P, _P, _P]),
    "mc_attention_forward_opt": (_INT, [_P, _P, _P, _I32, _I32, _I32, _I32, _OPT, _P, _P]),
    "mc_attention_backward_opt_ws_bytes": (_SZ, [_I32, _I32, _I32, _I32, _OPT]),
    "mc_attention_backward_opt": (_INT, [_P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _OPT, _P,
                                         _SZ, _P, _P]),
    "mc_qk_norm_forward": (_INT, [_P, _P, _I32, _I64, _I32, _I32, _I32, _I64, _I64, _NORM, _P, _P,
                                  ctypes.POINTER(mc_rotary_spec), _P, _P]),
    "mc_qk_norm_scratch_floats": (_SZ, [_I64, _I32, _I32, _I32]),
    "mc_qk_norm_backward": (_INT, [_P, _P, _P, _I32, _I64, _I32, _I32, _I32, _I64, _I64, _I64,
                                   _NORM, _P, _P, ctypes.POINTER(mc_rotary_spec),
                                   ctypes.POINTER(mc_qk_norm_grads), _I32, _P, _P, _P]),
    "mc_layer_saved_bytes_norm": (_SZ, [ctypes.POINTER(mc_layer_shape), _LNORM]),
    "mc_layer_workspace_bytes_norm": (_SZ, [ctypes.POINTER(mc_layer_shape), _LNORM, _OPT]),
    "mc_layer_forward_norm": (_INT, [ctypes.POINTER(mc_layer_shape),
                                     ctypes.POINTER(mc_layer_weights), _LNORM, _ROT, _OPT, _P, _P,
                                     _P, _P, _SZ, _P]),
    "mc_layer_backward_norm": (_INT, [ctypes.POINTER(mc_layer_shape),
                                      ctypes.POINTER(mc_layer_weights), _LNORM, _ROT, _OPT, _P, _P,
                                      _P, _P, ctypes.POINTER(mc_layer_grads), _P, _SZ, _P]),
    "mc_attention_forward_cross": (_INT, [_P, _P, _P, _P, _P, _CROSS, _P, _P]),
    "mc_attention_backward_cross_ws_bytes": (_SZ, [_CROSS]),
    "mc_attention_backward_cross": (_INT, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _CROSS, _P, _SZ,
                                           _P, _P]),
    "mc_layer_workspace_bytes_opt": (_SZ, [ctypes.POINTER(mc_layer_shape), _OPT]),
    "mc_layer_forward_opt": (_INT, [ctypes.POINTER(mc_layer_shape),
                                    ctypes.POINTER(mc_layer_weights), _ROT, _OPT, _P, _P, _P, _P,
                                    _SZ, _P]),
    "mc_layer_backward_opt": (_INT, [ctypes.POINTER(mc_layer_shape),
                                     ctypes.POINTER(mc_layer_weights), _ROT, _OPT, _P, _P, _P, _P,
                                     ctypes.POINTER(mc_layer_grads), _P, _SZ, _P]),
}


def lib() -> ctypes.CDLL:
    """Loads libmclayer.so (or the debug build, see LIB_PATH), built in-tree;
    raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} not found: build it with "
                               "`python -m megatron_transformer_layer_gb300.build` "
                               "(`--debug` for the debug build)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s) -> int | None:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream  # torch.cuda.Stream


def make_shape(micro_batch, seq_len, hidden, heads, ffn_hidden, tp_parts=1, head_dim=0, flags=0):
    return mc_layer_shape(micro_batch, seq_len, hidden, heads, ffn_hidden, tp_parts, head_dim, flags)


def make_weights(tensors: dict) -> mc_layer_weights:
    return mc_layer_weights(*[_ptr(tensors[n]) for n in PARAM_ORDER])


def make_grads(tensors: dict) -> mc_layer_grads:
    return mc_layer_grads(*[_ptr(tensors[n]) for n in PARAM_ORDER])


# ---- the C entry points, same names ----------------------------------------

def mc_layer_check_shape(shape: mc_layer_shape) -> int:
    return lib().mc_layer_check_shape(ctypes.byref(shape))


def mc_layer_saved_bytes(shape: mc_layer_shape) -> int:
    return lib().mc_layer_saved_bytes(ctypes.byref(shape))


def mc_layer_workspace_bytes(shape: mc_layer_shape) -> int:
    return lib().mc_layer_workspace_bytes(ctypes.byref(shape))


def mc_layer_forward(shape, weights, x, y, saved, ws, ws_bytes, stream=None) -> int:
    return lib().mc_layer_forward(ctypes.byref(shape), ctypes.byref(weights), _ptr(x), _ptr(y),
                                  _ptr(saved), _ptr(ws), ws_bytes, _stream(stream))


def mc_layer_backward(shape, weights, x, dy, saved, dx, grads, ws, ws_bytes, stream=None) -> int:
    return lib().mc_layer_backward(ctypes.byref(shape), ctypes.byref(weights), _ptr(x), _ptr(dy),
                                   _ptr(saved), _ptr(dx), ctypes.byref(grads), _ptr(ws), ws_bytes,
                                   _stream(stream))


def mc_layer_device_status(ws, stream=None) -> int:
    return lib().mc_layer_device_status(_ptr(ws), _stream(stream))


def mc_strerror(code: int) -> str:
    try:
        return lib().mc_strerror(code).decode()
    except RuntimeError:
        return "libmclayer.so not loaded"


def mc_layernorm_forward(x, gamma, beta, out, mean, rstd, rows, h, status=None, stream=None) -> int:
    return lib().mc_layernorm_forward(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(out), _ptr(mean),
                                      _ptr(rstd), rows, h, _ptr(status), _stream(stream))


def mc_layernorm_backward(dout, x, mean, rstd, gamma, resid, dx, dx_bf16, dgamma, dbeta, colsum_dx,
                          accumulate, partials, rows, h, status=None, stream=None) -> int:
    return lib().mc_layernorm_backward(_ptr(dout), _ptr(x), _ptr(mean), _ptr(rstd), _ptr(gamma),
                                       _ptr(resid), _ptr(dx), _ptr(dx_bf16), _ptr(dgamma),
                                       _ptr(dbeta), _ptr(colsum_dx), accumulate, _ptr(partials),
                                       rows, h, _ptr(status), _stream(stream))


def mc_layernorm_backward_scratch_floats(rows: int, h: int) -> int:
    return lib().mc_layernorm_backward_scratch_floats(rows, h)


def mc_gemm(M, N, K, A, lda, a_layout, B, ldb, b_layout, out, ldc, epilogue, bias=None, aux=None,
            ldaux=0, accumulate=0, k_parts=1, status=None, stream=None) -> int:
    return lib().mc_gemm(M, N, K, _ptr(A), lda, a_layout, _ptr(B), ldb, b_layout, _ptr(out), ldc,
                         epilogue, _ptr(bias), _ptr(aux), ldaux, accumulate, k_parts, _ptr(status),
                         _stream(stream))


def mc_attention_forward(qkv, o, lse, micro_batch, seq_len, heads, head_dim, status=None,
                         stream=None) -> int:
    return lib().mc_attention_forward(_ptr(qkv), _ptr(o), _ptr(lse), micro_batch, seq_len, heads,
                                      head_dim, _ptr(status), _stream(stream))


def mc_attention_backward(qkv, o, lse, dout, dqkv, delta, micro_batch, seq_len, heads, head_dim,
                          status=None, stream=None) -> int:
    return lib().mc_attention_backward(_ptr(qkv), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dqkv),
                                       _ptr(delta), micro_batch, seq_len, heads, head_dim,
                                       _ptr(status), _stream(stream))


def mc_attention_backward_ws_bytes(micro_batch, seq_len, heads, head_dim) -> int:
    return lib().mc_attention_backward_ws_bytes(micro_batch, seq_len, heads, head_dim)


def mc_attention_backward_ws(qkv, o, lse, dout, dqkv, delta, micro_batch, seq_len, heads,
                             head_dim, ds_workspace, ds_workspace_bytes, status=None,
                             stream=None) -> int:
    """mc_attention_backward whose dQ is formed from dS^T tiles written by the
    dK/dV kernel into `ds_workspace` (uint8 device tensor)."""
    return lib().mc_attention_backward_ws(_ptr(qkv), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dqkv),
                                          _ptr(delta), micro_batch, seq_len, heads, head_dim,
                                          _ptr(ds_workspace), ds_workspace_bytes, _ptr(status),
                                          _stream(stream))


def mc_attention_backward_noalloc(qkv, o, lse, dout, dqkv, micro_batch, seq_len, heads, head_dim,
                                  status=None, stream=None) -> int:
    """Allocation-free attention backward (fixed in-library scratch)."""
    return lib().mc_attention_backward_noalloc(_ptr(qkv), _ptr(o), _ptr(lse), _ptr(dout),
                                               _ptr(dqkv), micro_batch, seq_len, heads, head_dim,
                                               _ptr(status), _stream(stream))


def mc_cp_schedule(cp_parts, rank, step):
    """(query chunk, key chunk) pairs of a virtual CP rank in a ring step
    (host only); raises on an invalid argument."""
    buf = (_I32 * 8)()
    n = lib().mc_cp_schedule(cp_parts, rank, step, buf)
    if n < 0:
        raise ValueError(mc_strerror(n))
    return [(buf[2 * k], buf[2 * k + 1]) for k in range(n)]


def mc_cp_launch_plan(cp_parts):
    """The context-parallel launch plan (host only): one tuple (launch,
    query chunk, key chunk, mode of the query chunk, mode of the key chunk)
    per chunk pair, in launch order; raises on an invalid argument."""
    n_pairs = cp_parts * (2 * cp_parts + 1) if cp_parts > 0 else 1
    buf = (_I32 * (5 * n_pairs))()
    n = lib().mc_cp_launch_plan(cp_parts, buf, n_pairs)
    if n < 0:
        raise ValueError(mc_strerror(n))
    return [tuple(buf[5 * k + e] for e in range(5)) for k in range(n)]


def mc_attention_cp_workspace_bytes(micro_batch, seq_len, heads, head_dim, cp_parts) -> int:
    return lib().mc_attention_cp_workspace_bytes(micro_batch, seq_len, heads, head_dim, cp_parts)


def mc_attention_forward_cp(qkv, o, lse, micro_batch, seq_len, heads, head_dim, cp_parts,
                            workspace, workspace_bytes, status=None, stream=None) -> int:
    return lib().mc_attention_forward_cp(_ptr(qkv), _ptr(o), _ptr(lse), micro_batch, seq_len,
                                         heads, head_dim, cp_parts, _ptr(workspace),
                                         workspace_bytes, _ptr(status), _stream(stream))


def mc_attention_backward_cp(qkv, o, lse, dout, dqkv, delta, micro_batch, seq_len, heads,
                             head_dim, cp_parts, workspace, workspace_bytes, status=None,
                             stream=None) -> int:
    return lib().mc_attention_backward_cp(_ptr(qkv), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dqkv),
                                          _ptr(delta), micro_batch, seq_len, heads, head_dim,
                                          cp_parts, _ptr(workspace), workspace_bytes,
                                          _ptr(status), _stream(stream))


FP8_E4M3 = 0
FP8_E5M2 = 1


def mc_fp8_scratch_floats() -> int:
    return lib().mc_fp8_scratch_floats()


def mc_fp8_quantize(x, out, scale_inv, scratch, fmt, status=None, stream=None) -> int:
    """Per-tensor current scaling of x (fp32 or bf16 tensor) to 8-bit bytes."""
    import torch
    in_bf16 = 1 if x.dtype == torch.bfloat16 else 0
    return lib().mc_fp8_quantize(_ptr(x), in_bf16, x.numel(), fmt, _ptr(out), _ptr(scale_inv),
                                 _ptr(scratch), _ptr(status), _stream(stream))


def mc_fp8_quantize_2d(x, out, out_t, scale_inv, scratch, fmt, stream=None) -> int:
    """Per-tensor current scaling of a 2-D x (fp32 or bf16) to 8-bit bytes,
    written as is (out) and/or transposed (out_t); either may be None."""
    import torch
    in_bf16 = 1 if x.dtype == torch.bfloat16 else 0
    rows, cols = x.shape
    return lib().mc_fp8_quantize_2d(_ptr(x), in_bf16, rows, cols, fmt, _ptr(out), _ptr(out_t),
                                    _ptr(scale_inv), _ptr(scratch), _stream(stream))


def mc_gemm_fp8(M, N, K, A, lda, a_format, B, ldb, b_format, a_scale_inv, b_scale_inv, out, ldc,
                epilogue, bias=None, aux=None, ldaux=0, accumulate=0, k_parts=1, status=None,
                stream=None) -> int:
    return lib().mc_gemm_fp8(M, N, K, _ptr(A), lda, a_format, _ptr(B), ldb, b_format,
                             _ptr(a_scale_inv), _ptr(b_scale_inv), _ptr(out), ldc, epilogue,
                             _ptr(bias), _ptr(aux), ldaux, accumulate, k_parts, _ptr(status),
                             _stream(stream))


# ---- rotary positions, interval masks and attention over them

def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


_TYPES = {}  # torch's types by name, filled when a tensor first comes


def _array(x, what, dtype, n):
    """Pointer of an array of at least n elements: a contiguous tensor on the GPU
    of the torch type named `dtype`, or a bare pointer, which is not checked."""
    if x is None:
        return None
    try:
        if x.dtype is _TYPES[dtype] and x.is_contiguous() and x.numel() >= n and x.is_cuda:
            return x.data_ptr()
    except (AttributeError, KeyError):  # no tensor, or the first one
        pass
    return _other_array(x, what, dtype, n)


def _other_array(x, what, dtype, n):
    if isinstance(x, int):
        return x
    import torch
    _TYPES[dtype] = getattr(torch, dtype)
    if isinstance(x, torch.Tensor):
        if x.dtype is not _TYPES[dtype]:
            raise TypeError(f"{what}: {dtype} expected, got {x.dtype}")
        if not x.is_contiguous():
            raise ValueError(f"{what}: a contiguous tensor expected, got strides {x.stride()}")
        if x.numel() < n:
            raise ValueError(f"{what}: {n} elements expected, got {x.numel()}")
        if not x.is_cuda:
            raise ValueError(f"{what}: a tensor on the GPU expected, got one on {x.device}")
    return x.data_ptr()


def _on(stream, x):
    """A call's stream: without one, torch's current stream of x's device, as the
    layer's calls (for a bare pointer the legacy default stream)."""
    if stream is None and getattr(x, "is_cuda", False):
        import torch
        return torch.cuda.current_stream(x.device).cuda_stream
    return _stream(stream)


def _length(x):
    """Elements of a tensor; of what is not one, as many as it takes."""
    return x.numel() if hasattr(x, "numel") else 1 << 62


def make_rotary_spec(rot_dim, sections=None, interleaved_pairs=False, interleaved_axes=False):
    """`sections`: pairs of each axis (default: one axis).  `interleaved_pairs`:
    pairs are neighbours (2p, 2p + 1); `interleaved_axes`: axes dealt in turn."""
    if sections is None:
        sections = (rot_dim // 2,)
    if not 1 <= len(sections) <= MC_ROTARY_MAX_AXES:
        raise ValueError(f"1 to {MC_ROTARY_MAX_AXES} axes, got {len(sections)}")
    flags = (MC_ROTARY_ADJACENT_PAIRS if interleaved_pairs else 0) | \
        (MC_ROTARY_DEAL_AXES if interleaved_axes else 0)
    return mc_rotary_spec(rot_dim, len(sections), _RotarySections(*sections), flags)


def make_layer_rotary(spec, positions, inv_freq):
    """positions: int32 [axes, tokens], inv_freq: float32 [rot_dim / 2].  Keeps a
    reference to the tensors it points to."""
    out = mc_layer_rotary(spec, _array(positions, "positions", "int32", 0),
                          _array(inv_freq, "inv_freq", "float32", spec.rot_dim // 2))
    out.tensors = (positions, inv_freq)
    out.length = _length(positions)
    return out


def make_attention_options(key_lo, key_hi, tables, slopes=None, softcap=0.0, causal=True):
    """key_lo, key_hi, tables: int32, slopes: float32 [heads].  Keeps a reference
    to the tensors it points to."""
    out = mc_attention_options(_array(key_lo, "key_lo", "int32", 0),
                               _array(key_hi, "key_hi", "int32", 0),
                               _array(tables, "tables", "int32", 0),
                               _array(slopes, "slopes", "float32", 0),
                               float(softcap), 1 if causal else 0)
    out.tensors = (key_lo, key_hi, tables, slopes)
    out.lengths = (min(_length(key_lo), _length(key_hi)), _length(tables), _length(slopes))
    return out


def _options(options, micro_batch, seq_len, heads):
    """options for a call of this shape, which its arrays must cover."""
    if options is None:
        return None
    rows, tables, slopes = options.lengths
    if rows < micro_batch * seq_len:
        raise ValueError(f"key_lo, key_hi: {micro_batch * seq_len} elements expected, got {rows}")
    if tables < 8 * micro_batch * ((seq_len + 127) // 128):
        raise ValueError(f"tables: {8 * micro_batch * ((seq_len + 127) // 128)} elements expected, "
                         f"got {tables}")
    if slopes < heads:
        raise ValueError(f"slopes: {heads} elements expected, got {slopes}")
    return ctypes.byref(options)


def _rotary(rotary, shape):
    """rotary for a layer of this shape, which its positions must cover."""
    if rotary is None:
        return None
    n = rotary.spec.axes * shape.micro_batch * shape.seq_len
    if rotary.length < n:
        raise ValueError(f"positions: {n} elements expected, got {rotary.length}")
    return ctypes.byref(rotary)


def _is_bf16(x, what="rotary positions"):
    import torch
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"{what} take bf16 or fp32, got {x.dtype}")
    return 1 if x.dtype == torch.bfloat16 else 0


def mc_rotary_forward(x, out, tokens, heads, head_dim, ld_in, ld_out, positions, inv_freq, spec,
                      status=None, stream=None) -> int:
    """Rotary positions over `heads` heads at the start of each row of x (a
    bf16 or fp32 tensor; `out` of the same type, or x itself)."""
    if out.dtype != x.dtype:
        raise TypeError(f"rotary positions: {x.dtype} in, {out.dtype} out")
    return lib().mc_rotary_forward(_ptr(x), _ptr(out), _is_bf16(x), tokens, heads, head_dim, ld_in,
                                   ld_out, _array(positions, "positions", "int32",
                                                  spec.axes * tokens),
                                   _array(inv_freq, "inv_freq", "float32", spec.rot_dim // 2),
                                   ctypes.byref(spec), _ptr(status), _on(stream, x))


def mc_rotary_backward(dout, din, tokens, heads, head_dim, ld_dout, ld_din, positions, inv_freq,
                       spec, status=None, stream=None) -> int:
    if din.dtype != dout.dtype:
        raise TypeError(f"rotary positions: {dout.dtype} in, {din.dtype} out")
    return lib().mc_rotary_backward(_ptr(dout), _ptr(din), _is_bf16(dout), tokens, heads, head_dim,
                                    ld_dout, ld_din, _array(positions, "positions", "int32",
                                                            spec.axes * tokens),
                                    _array(inv_freq, "inv_freq", "float32", spec.rot_dim // 2),
                                    ctypes.byref(spec), _ptr(status), _on(stream, dout))


# ---- norms of queries and keys with their rotation

def _norm_struct(cls, dtype, n, q_gain, q_shift, k_gain, k_shift, *rest):
    arrays = (q_gain, q_shift, k_gain, k_shift)
    names = ("q_gain", "q_shift", "k_gain", "k_shift")
    out = cls(*[_array(x, w, dtype, n) for x, w in zip(arrays, names)], *rest)
    out.tensors = arrays
    out.lengths = tuple(min(_length(x) for x in arrays[2 * i: 2 * i + 2]) for i in range(2))
    return out


def make_qk_norm(q_gain=None, k_gain=None, q_shift=None, k_shift=None, eps=1e-5, centred=False):
    """Gains and shifts: bfloat16 [head_dim], None for ones and zeros; `centred`
    takes the mean off (LayerNorm).  Keeps a reference to the tensors."""
    return _norm_struct(mc_qk_norm, "bfloat16", 0, q_gain, q_shift, k_gain, k_shift, float(eps),
                        MC_QK_NORM_CENTRED if centred else 0)


def make_qk_norm_grads(q_gain=None, k_gain=None, q_shift=None, k_shift=None):
    """Where the gradients of the gains and shifts go: float32 [head_dim], None
    for those that are not wanted.  Keeps a reference to the tensors."""
    return _norm_struct(mc_qk_norm_grads, "float32", 0, q_gain, q_shift, k_gain, k_shift)


def _norm_ref(struct, what, q_heads, k_heads, head_dim):
    """struct for a call of these heads, which its arrays must cover."""
    if struct is None:
        return None
    for n, used, of in zip(struct.lengths, (q_heads, k_heads), "qk"):
        if used and n < head_dim:
            raise ValueError(f"{what} of {of}: {head_dim} elements expected, got {n}")
    return ctypes.byref(struct)


def _turning(positions, inv_freq, spec, tokens):
    if spec is None:
        return None, None, None
    return (_array(positions, "positions", "int32", spec.axes * tokens),
            _array(inv_freq, "inv_freq", "float32", spec.rot_dim // 2), ctypes.byref(spec))


def _token_rows(x, what, tokens, ld, width):
    """Pointer of a tensor whose `tokens` rows of `width` elements lie ld apart: of
    rows, of heads [tokens, heads, head_dim], or of any contiguous shape whose last
    dimension rows are whole numbers of."""
    try:
        (n, w), (s0, s1) = x.shape, x.stride()
        if n >= tokens and w >= width and s1 == 1 and (s0 == ld or tokens == 1) and x.is_cuda:
            return x.data_ptr()
    except ValueError:  # not two dimensions
        pass
    if not x.is_cuda:
        raise ValueError(f"{what}: a tensor on the GPU expected, got one on {x.device}")
    if x.dim() > 1 and x.stride(0) == ld and x.shape[0] >= max(tokens, 1):
        covers = x[0].is_contiguous() and x[0].numel() >= width
    else:
        covers = x.dim() > 0 and x.is_contiguous() and x.numel() >= (tokens - 1) * ld + width and \
            (x.dim() == 1 or tokens == 1 or (x.shape[-1] > 0 and ld % x.shape[-1] == 0))
    if not covers:
        raise ValueError(f"{what}: {tokens} rows of {width} elements, {ld} apart, expected, got shape "
                         f"{tuple(x.shape)}, strides {x.stride()}")
    return x.data_ptr()


def mc_qk_norm_forward(x, out, tokens, q_heads, k_heads, head_dim, ld_in, ld_out, norm,
                       positions=None, inv_freq=None, spec=None, status=None, stream=None) -> int:
    """Norms (and, with a spec, rotary positions) over q_heads + k_heads heads at
    the start of each row of x (a bf16 or fp32 tensor; `out` of the same type, or
    x itself)."""
    if out.dtype != x.dtype:
        raise TypeError(f"norms of queries and keys: {x.dtype} in, {out.dtype} out")
    width = (q_heads + k_heads) * head_dim
    return lib().mc_qk_norm_forward(_token_rows(x, "x", tokens, ld_in, width),
                                    _token_rows(out, "out", tokens, ld_out, width),
                                    _is_bf16(x, "norms of queries and keys"), tokens, q_heads, k_heads,
                                    head_dim, ld_in, ld_out,
                                    _norm_ref(norm, "norm", q_heads, k_heads, head_dim),
                                    *_turning(positions, inv_freq, spec, tokens), _ptr(status),
                                    _on(stream, x))


def mc_qk_norm_scratch_floats(tokens, q_heads, k_heads, head_dim) -> int:
    return lib().mc_qk_norm_scratch_floats(tokens, q_heads, k_heads, head_dim)


def mc_qk_norm_backward(x, dout, din, tokens, q_heads, k_heads, head_dim, ld_in, ld_dout, ld_din,
                        norm, positions=None, inv_freq=None, spec=None, grads=None, accumulate=0,
                        scratch=None, status=None, stream=None) -> int:
    """The gradients of mc_qk_norm_forward: din from x and dout (all of one
    type), and those of the gains and shifts that `grads` asks for (scratch:
    mc_qk_norm_scratch_floats float32)."""
    if dout.dtype != x.dtype or din.dtype != x.dtype:
        raise TypeError(f"norms of queries and keys: {x.dtype} in, {dout.dtype} and {din.dtype} "
                        "for its gradients")
    need = 0 if grads is None else mc_qk_norm_scratch_floats(tokens, q_heads, k_heads, head_dim)
    width = (q_heads + k_heads) * head_dim
    return lib().mc_qk_norm_backward(_token_rows(x, "x", tokens, ld_in, width),
                                     _token_rows(dout, "dout", tokens, ld_dout, width),
                                     _token_rows(din, "din", tokens, ld_din, width),
                                     _is_bf16(x, "norms of queries and keys"), tokens, q_heads,
                                     k_heads, head_dim, ld_in, ld_dout, ld_din,
                                     _norm_ref(norm, "norm", q_heads, k_heads, head_dim),
                                     *_turning(positions, inv_freq, spec, tokens),
                                     _norm_ref(grads, "gradient", q_heads, k_heads, head_dim),
                                     accumulate, _array(scratch, "scratch", "float32", need),
                                     _ptr(status), _on(stream, x))


def make_layer_qk_norm(norm, grads=None):
    """norm: make_qk_norm, grads: make_qk_norm_grads or None.  Keeps a reference to
    their tensors."""
    out = mc_layer_qk_norm(norm, mc_qk_norm_grads() if grads is None else grads)
    out.parts = (norm, grads)
    return out


def _layer_norm(qk_norm, shape):
    """qk_norm for a layer of this shape, whose heads its arrays must cover."""
    if qk_norm is None:
        return None
    d = shape.head_dim or shape.hidden // max(shape.heads, 1)
    for part, what in zip(qk_norm.parts, ("norm", "gradient")):
        _norm_ref(part, what, 1, 1, d)
    return ctypes.byref(qk_norm)


def mc_layer_saved_bytes_norm(shape, qk_norm) -> int:
    return lib().mc_layer_saved_bytes_norm(ctypes.byref(shape), _ref(qk_norm))


def mc_layer_workspace_bytes_norm(shape, qk_norm, attention) -> int:
    return lib().mc_layer_workspace_bytes_norm(ctypes.byref(shape), _ref(qk_norm), _ref(attention))


def mc_layer_forward_norm(shape, weights, qk_norm, rotary, attention, x, y, saved, ws, ws_bytes,
                          stream=None) -> int:
    return lib().mc_layer_forward_norm(ctypes.byref(shape), ctypes.byref(weights),
                                       _layer_norm(qk_norm, shape), _rotary(rotary, shape),
                                       _options(attention, shape.micro_batch, shape.seq_len,
                                                shape.heads),
                                       _ptr(x), _ptr(y), _ptr(saved), _ptr(ws), ws_bytes,
                                       _on(stream, x))


def mc_layer_backward_norm(shape, weights, qk_norm, rotary, attention, x, dy, saved, dx, grads, ws,
                           ws_bytes, stream=None) -> int:
    return lib().mc_layer_backward_norm(ctypes.byref(shape), ctypes.byref(weights),
                                        _layer_norm(qk_norm, shape), _rotary(rotary, shape),
                                        _options(attention, shape.micro_batch, shape.seq_len,
                                                 shape.heads),
                                        _ptr(x), _ptr(dy), _ptr(saved), _ptr(dx),
                                        ctypes.byref(grads), _ptr(ws), ws_bytes, _on(stream, x))


# ---- attention to keys and values of another length

def make_cross_attention(sequences, q_rows, kv_rows, heads, kv_heads, head_dim, ld_q=None,
                         ld_kv=None, ld_o=None, q_offsets=None, q_lens=None, kv_offsets=None,
                         kv_lens=None, max_q=0, max_kv=0, scale=0.0):
    """Row strides default to the heads' own width.  Offsets int32 [sequences +
    1], lengths int32 [sequences].  With offsets state max_q and max_kv, the most
    rows of a sequence: without them each counts as long as all rows together, in
    the backward pass's workspace too.  Keeps a reference to the tensors."""
    arrays = (q_offsets, q_lens, kv_offsets, kv_lens)
    names = ("q_offsets", "q_lens", "kv_offsets", "kv_lens")
    out = mc_cross_attention(
        sequences, heads, kv_heads, head_dim, q_rows, kv_rows, max_q, max_kv,
        heads * head_dim if ld_q is None else ld_q, kv_heads * head_dim if ld_kv is None else ld_kv,
        heads * head_dim if ld_o is None else ld_o,
        *[_array(x, w, "int32", sequences + 1 - (i & 1)) for i, (x, w) in enumerate(zip(arrays, names))],
        float(scale))
    out.tensors = arrays
    return out


def _rows(x, what, rows, ld, width):
    """Pointer of a bf16 tensor of rows that are ld elements apart, which it must
    cover (a bare pointer is not checked)."""
    try:
        if x.dtype is _TYPES["bfloat16"] and x.is_cuda:
            (n, w), (s0, s1) = x.shape, x.stride()
            if n >= rows and w >= width and s1 == 1 and (s0 == ld or rows == 1):
                return x.data_ptr()
    except (AttributeError, KeyError, ValueError):  # no tensor, the first one, or not of rows
        pass
    return _other_rows(x, what, rows, ld, width)


def _other_rows(x, what, rows, ld, width):
    if x is None or isinstance(x, int):
        return x
    import torch
    _TYPES["bfloat16"] = torch.bfloat16
    if x.dtype is not torch.bfloat16:
        raise TypeError(f"{what}: bfloat16 expected, got {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"{what}: a tensor on the GPU expected, got one on {x.device}")
    if x.dim() != 2 or x.shape[0] < rows or x.shape[1] < width or x.stride(1) != 1 \
            or (rows > 1 and x.stride(0) != ld):
        raise ValueError(f"{what}: {rows} rows of {width} elements, {ld} apart, expected, got shape "
                         f"{tuple(x.shape)}, strides {x.stride()}")
    return x.data_ptr()


def mc_attention_forward_cross(q, k, v, o, lse, cross, status=None, stream=None) -> int:
    """Attention of the rows of q to those of k and v, see make_cross_attention
    (bf16 tensors [rows, heads * head_dim] or views of wider rows; lse float32
    [heads, q_rows])."""
    c = cross
    a, akv = c.heads * c.head_dim, c.kv_heads * c.head_dim
    n, nkv, ld_kv = c.q_rows, c.kv_rows, c.ld_kv
    return lib().mc_attention_forward_cross(
        _rows(q, "q", n, c.ld_q, a), _rows(k, "k", nkv, ld_kv, akv), _rows(v, "v", nkv, ld_kv, akv),
        _rows(o, "o", n, c.ld_o, a), _array(lse, "lse", "float32", c.heads * n), ctypes.byref(c),
        _ptr(status), _on(stream, q))


def mc_attention_backward_cross_ws_bytes(cross) -> int:
    return lib().mc_attention_backward_cross_ws_bytes(ctypes.byref(cross))


def mc_attention_backward_cross(q, k, v, o, lse, dout, dq, dk, dv, delta, cross, ws, ws_bytes,
                                status=None, stream=None) -> int:
    c = cross
    a, akv = c.heads * c.head_dim, c.kv_heads * c.head_dim
    n, nkv, ld_q, ld_kv, ld_o = c.q_rows, c.kv_rows, c.ld_q, c.ld_kv, c.ld_o
    return lib().mc_attention_backward_cross(
        _rows(q, "q", n, ld_q, a), _rows(k, "k", nkv, ld_kv, akv), _rows(v, "v", nkv, ld_kv, akv),
        _rows(o, "o", n, ld_o, a), _array(lse, "lse", "float32", c.heads * n),
        _rows(dout, "dout", n, ld_o, a), _rows(dq, "dq", n, ld_q, a),
        _rows(dk, "dk", nkv, ld_kv, akv), _rows(dv, "dv", nkv, ld_kv, akv),
        _array(delta, "delta", "float32", c.heads * n), ctypes.byref(c), _ptr(ws), ws_bytes,
        _ptr(status), _on(stream, q))


def mc_attention_mask_table_ints(micro_batch, seq_len) -> int:
    return lib().mc_attention_mask_table_ints(micro_batch, seq_len)


def mc_attention_mask_documents(offsets, n_docs, prefix, causal, window, micro_batch, seq_len,
                                key_lo, key_hi, tables, status=None, stream=None) -> int:
    rows, ints = micro_batch * seq_len, 8 * micro_batch * ((seq_len + 127) // 128)
    return lib().mc_attention_mask_documents(_array(offsets, "offsets", "int32", n_docs + 1), n_docs,
                                             _array(prefix, "prefix", "int32", n_docs), causal,
                                             window, micro_batch, seq_len,
                                             _array(key_lo, "key_lo", "int32", rows),
                                             _array(key_hi, "key_hi", "int32", rows),
                                             _array(tables, "tables", "int32", ints),
                                             _ptr(status), _on(stream, key_lo))


def mc_attention_mask_intervals(micro_batch, seq_len, key_lo, key_hi, tables, status=None,
                                stream=None) -> int:
    rows, ints = micro_batch * seq_len, 8 * micro_batch * ((seq_len + 127) // 128)
    return lib().mc_attention_mask_intervals(micro_batch, seq_len,
                                             _array(key_lo, "key_lo", "int32", rows),
                                             _array(key_hi, "key_hi", "int32", rows),
                                             _array(tables, "tables", "int32", ints),
                                             _ptr(status), _on(stream, key_lo))


def mc_attention_forward_opt(qkv, o, lse, micro_batch, seq_len, heads, head_dim, options,
                             status=None, stream=None) -> int:
    return lib().mc_attention_forward_opt(_ptr(qkv), _ptr(o), _ptr(lse), micro_batch, seq_len,
                                          heads, head_dim,
                                          _options(options, micro_batch, seq_len, heads),
                                          _ptr(status), _on(stream, qkv))


def mc_attention_backward_opt_ws_bytes(micro_batch, seq_len, heads, head_dim, options) -> int:
    return lib().mc_attention_backward_opt_ws_bytes(micro_batch, seq_len, heads, head_dim,
                                                    _ref(options))


def mc_attention_backward_opt(qkv, o, lse, dout, dqkv, delta, micro_batch, seq_len, heads,
                              head_dim, options, ds_workspace=None, ds_workspace_bytes=0,
                              status=None, stream=None) -> int:
    return lib().mc_attention_backward_opt(_ptr(qkv), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dqkv),
                                           _ptr(delta), micro_batch, seq_len, heads, head_dim,
                                           _options(options, micro_batch, seq_len, heads),
                                           _ptr(ds_workspace), ds_workspace_bytes, _ptr(status),
                                           _on(stream, qkv))


def mc_layer_workspace_bytes_opt(shape, attention) -> int:
    return lib().mc_layer_workspace_bytes_opt(ctypes.byref(shape), _ref(attention))


def mc_layer_forward_opt(shape, weights, rotary, attention, x, y, saved, ws, ws_bytes,
                         stream=None) -> int:
    return lib().mc_layer_forward_opt(ctypes.byref(shape), ctypes.byref(weights),
                                      _rotary(rotary, shape),
                                      _options(attention, shape.micro_batch, shape.seq_len,
                                               shape.heads),
                                      _ptr(x), _ptr(y), _ptr(saved), _ptr(ws), ws_bytes,
                                      _on(stream, x))


def mc_layer_backward_opt(shape, weights, rotary, attention, x, dy, saved, dx, grads, ws, ws_bytes,
                          stream=None) -> int:
    return lib().mc_layer_backward_opt(ctypes.byref(shape), ctypes.byref(weights),
                                       _rotary(rotary, shape),
                                       _options(attention, shape.micro_batch, shape.seq_len,
                                                shape.heads),
                                       _ptr(x), _ptr(dy), _ptr(saved), _ptr(dx),
                                       ctypes.byref(grads), _ptr(ws), ws_bytes, _on(stream, x))


def mc_selftest_bounds_check(index, extent, buf, status, stream=None) -> int:
    """Runs the index check of a debug build on one index (failure-path test)."""
    return lib().mc_selftest_bounds_check(index, extent, _ptr(buf), _ptr(status), _stream(stream))


def mc_selftest_wait_timeout(timeout_ns, status, stream=None) -> int:
    """Runs a kernel whose bounded wait is made to run out (failure-path test)."""
    return lib().mc_selftest_wait_timeout(timeout_ns, _ptr(status), _stream(stream))
