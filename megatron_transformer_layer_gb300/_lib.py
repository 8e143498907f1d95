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


_lib = None

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_SZ = ctypes.c_size_t

_OPT = ctypes.POINTER(mc_attention_options)
_ROT = ctypes.POINTER(mc_layer_rotary)

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


def _is_bf16(x):
    import torch
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"rotary positions take bf16 or fp32, got {x.dtype}")
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
