"""Thin Python binding of libgemm_decode.so (ctypes).

Argument marshalling only: each function checks that tensors live on a HIP
device with the expected dtype, size and contiguity, passes their
``data_ptr()`` and torch's current stream to the C entry point of the same
name (declared in include/gemm_decode.h), and raises on a non-zero status.
Every step of the computation runs in the library's HIP kernels; there is no
fallback. Importing this package fails loudly if the library is not built.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgemm_decode.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
        "(or python gemm_decode_amd/build.py) first")

_lib = ctypes.CDLL(LIB_PATH)

GD_OK, GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_EHIP, GD_ERANGE = 0, -1, -2, -3, -4, -5

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_F32 = ctypes.c_float
_F64 = ctypes.c_double
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t


class GemmDecodeError(RuntimeError):
    def __init__(self, status: int, text: str):
        self.status = status
        name = _lib.gemm_decode_status_string(status).decode()
        super().__init__(f"{name}: {text}")


class Q1Problem(ctypes.Structure):
    """gd_q1_problem: one batch-1 problem of q1_q8_gemv_grouped."""
    _fields_ = [("bits_plane", _P), ("scale_plane", _P), ("a_q8", _P), ("y", _P), ("rows", _I64)]


class TernaryProblem(ctypes.Structure):
    """gd_ternary_problem: one problem of ternary_gemv_grouped."""
    _fields_ = [("w_pos", _P), ("w_neg", _P), ("x_planes", _P), ("y", _P),
                ("dot_out", _P), ("w_scale", _F32), ("x_scale", _F32), ("x_scale_dev", _P)]


class _KVQ8(ctypes.Structure):
    """gd_kv_q8."""
    _fields_ = [("k_codes", _P), ("k_scales", _P), ("v_codes", _P), ("v_scales", _P), ("n_pages", _I64),
                ("page_size", _I64), ("n_kv_heads", _I64), ("head_dim", _I64)]


ROPE_NONE, ROPE_LINEAR, ROPE_NTK, ROPE_YARN, ROPE_LLAMA3 = range(5)


class RopeScaling(ctypes.Structure):
    """gd_rope_scaling: how rope_table scales the rotary frequencies for long contexts."""
    _fields_ = [("kind", _I32), ("reserved", _I32), ("factor", _F64), ("original_len", _F64), ("low", _F64),
                ("high", _F64), ("attention", _F64)]

    def __init__(self, kind, factor=1.0, original_len=0.0, low=0.0, high=0.0, attention=0.0):
        super().__init__(kind, 0, factor, original_len, low, high, attention)


def _declare():
    L = _lib
    L.gemm_decode_status_string.argtypes = [ctypes.c_int]
    L.gemm_decode_status_string.restype = ctypes.c_char_p
    L.gemm_decode_last_error.argtypes = []
    L.gemm_decode_last_error.restype = ctypes.c_char_p
    L.gemm_decode_abi_version.restype = ctypes.c_int
    sig = {
        "q1_planes_bytes": [_I64, _I64, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)],
        "q1_repack": [_P, _I64, _I64, _P, _P, _P],
        "q1_q8_gemv": [_P, _P, _P, _P, _I64, _I64, _I64, _P],
        "q1_q8_gemv_grouped": [_P, _I64, _I64, _I64, _P],
        "q1_sign_gemm": [_P, _P, _P, _P, _I64, _I64, _I64, _P, ctypes.c_size_t, _P],
        "q1_sign_gemm_workspace_bytes": [_I64, _I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
        "q1_sign_packed_bytes": [_I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
        "q1_sign_pack": [_P, _P, _I64, _I64, _P, _P],
        "q1_sign_gemm_packed": [_P, _P, _P, _I64, _I64, _I64, _P, ctypes.c_size_t, _P],
        "q1_sign_gemv": [_P, _P, _P, _I64, _I64, _I64, _P],
        "q1_sign_gemm_lut4": [_P, _P, _P, _I64, _I64, _I64, _P],
        "blockq8_matmul_nt": [_P, _P, _P, _P, _I64, _I64, _I64, _P],
        "ternary_act_bitplanes": [_P, _I64, _I64, _P, _P],
        "ternary_gemv": [_P, _P, _F32, _P, _F32, _P, _P, _I64, _I64, _P],
        "ternary_gemv_grouped": [_P, _I64, _I64, _I64, _P],
        "q8_0_quantize": [_P, _P, _I64, _I64, _P],
        "attn_decode_workspace_bytes": [_I64, _I64, _I64, _I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
        "attn_decode_splitk": [_P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _F32, _I64, _P, ctypes.c_size_t, _P],
        "attn_decode_splitk_noalloc": [_P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _F32, _I64, _P],
        "ternary_quantize_act": [_P, _I64, _I64, _P, _P, _P],
        "rmsnorm_q8_0": [_P, _P, _P, _P, _P, _I64, _I64, _F32, _I32, _P],
        "rmsnorm_ternary_act": [_P, _P, _P, _P, _P, _P, _I64, _I64, _F32, _I32, _P],
        "q8_0_dequantize": [_P, _P, _I64, _I64, _I32, _P],
        "ternary_dequantize_act": [_P, _P, _P, _I64, _I64, _I32, _P],
        "rope_table": [_P, _I64, _I64, _F64, _P, _P],
        "kv_q8_store": [_P, _P, _I64, _P, _I64, _P, _I64, _P, _P, _I64, _I64, _I32, _P, _P, _I64, _I64, _I32, _P],
        "kv_q8_load": [_P, _P, _P, _P, _I64, _I32, _P],
        "attn_decode_q8": [_P, _P, _P, _P, _I64, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _F32, _F32, _I32, _P, _SZ,
                           _P],
        "attn_decode_q8_workspace_bytes": [_I64, _I64, _I64, _I64, _I64, _I64, _I64, ctypes.POINTER(_SZ)],
        "rmsnorm_sandwich_q8_0": [_P, _P, _P, _I64, _P, _P, _F32, _F32, _P, _P, _P, _I64, _I64, _F32, _I32, _P],
        "rmsnorm_sandwich_ternary_act": [_P, _P, _P, _I64, _P, _P, _F32, _F32, _P, _P, _P, _P, _I64, _I64, _F32, _I32,
                                         _P],
        "q1_q8_linear": [_P, _P, _P, _P, _I32, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _SZ, _P],
        "q1_q8_gated": [_P, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _I64, _I64, _I64, _I32, _P, _SZ, _P],
        "q1_q8_linear_workspace_bytes": [_I64, _I64, ctypes.POINTER(_SZ)],
        "token_logprobs": [_P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _F32, _F32, _I32, _P, _SZ, _P],
        "token_logprobs_workspace_bytes": [_I64, _I64, _I64, ctypes.POINTER(_SZ)],
        "gemm_decode_fill": [_P, ctypes.c_size_t, ctypes.c_uint32, _P],
        "gemm_decode_stream_read": [_P, ctypes.c_size_t, ctypes.c_int32, _P, _I64, _P],
    }
    for name, args in sig.items():
        fn = getattr(L, name, None)
        if fn is None:
            continue
        fn.argtypes = args
        fn.restype = ctypes.c_int


_declare()

# The problem structs below mirror the header of this ABI version; a library
# built from other sources would read them with another layout.
ABI_VERSION = 4
if _lib.gemm_decode_abi_version() != ABI_VERSION:
    raise ImportError(f"{LIB_PATH} has ABI version {_lib.gemm_decode_abi_version()}, this binding needs "
                      f"{ABI_VERSION}: rebuild it")


def lib():
    return _lib


def _check(status: int):
    if status != GD_OK:
        raise GemmDecodeError(status, _lib.gemm_decode_last_error().decode())


def _stream():
    import torch
    return torch.cuda.current_stream().cuda_stream


def _dev(t, dtype, numel=None, name="tensor"):
    """data_ptr of a contiguous device tensor of the given dtype (and size)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a HIP device, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")
    return t.data_ptr()


# --------------------------------------------------------------- Q1_0.q8_0

def q1_planes_bytes(rows: int, K: int):
    b, s = ctypes.c_size_t(), ctypes.c_size_t()
    _check(_lib.q1_planes_bytes(rows, K, ctypes.byref(b), ctypes.byref(s)))
    return b.value, s.value


def q1_repack(w_aos, rows: int, K: int, bits_plane, scale_plane):
    import torch
    bb, sb = q1_planes_bytes(rows, K)
    _check(_lib.q1_repack(_dev(w_aos, torch.uint8, rows * (K // 128) * 18, "w_aos"), rows, K,
                          _dev(bits_plane, torch.uint8, bb, "bits_plane"),
                          _dev(scale_plane, torch.uint8, sb, "scale_plane"), _stream()))


def q1_alloc_planes(rows: int, K: int, device="cuda"):
    """Allocates (bits_plane, scale_plane) uint8 device tensors of the right size."""
    import torch
    bb, sb = q1_planes_bytes(rows, K)
    return (torch.empty(bb, dtype=torch.uint8, device=device),
            torch.empty(sb, dtype=torch.uint8, device=device))


def q1_q8_gemv(bits_plane, scale_plane, a_q8, y, rows: int, K: int, n_act: int = 1):
    import torch
    bb, sb = q1_planes_bytes(rows, K)
    _check(_lib.q1_q8_gemv(_dev(bits_plane, torch.uint8, bb, "bits_plane"),
                           _dev(scale_plane, torch.uint8, sb, "scale_plane"),
                           _dev(a_q8, torch.uint8, n_act * (K // 32) * 34, "a_q8"),
                           _dev(y, torch.float32, n_act * rows, "y"), rows, K, n_act, _stream()))


def q1_q8_gemv_grouped(problems, count: int, rows: int, K: int):
    """problems: device uint8 tensor holding `count` gd_q1_problem structs
    (see make_q1_problems)."""
    import torch
    _check(_lib.q1_q8_gemv_grouped(_dev(problems, torch.uint8, count * ctypes.sizeof(Q1Problem), "problems"),
                                   count, rows, K, _stream()))


def make_q1_problems(entries, device="cuda"):
    """Device array of gd_q1_problem from [(bits_plane, scale_plane, a_q8, y[, rows]), ...]
    (rows 0 or absent: the launch's rows)."""
    import torch
    arr = (Q1Problem * len(entries))()
    for i, e in enumerate(entries):
        b, s, a, y = e[:4]
        arr[i] = Q1Problem(b.data_ptr(), s.data_ptr(), a.data_ptr(), y.data_ptr(), e[4] if len(e) > 4 else 0)
    host = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8)
    return host.to(device)


# --------------------------------------------------------- sign-bit GEMM

def q1_sign_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    out = ctypes.c_size_t()
    _check(_lib.q1_sign_gemm_workspace_bytes(M, N, K, ctypes.byref(out)))
    return out.value


_sign_ws = {}


def _sign_workspace(M: int, N: int, K: int, device=None):
    """The per-device cached sign-GEMM workspace, grown to the call's need."""
    import torch
    need = q1_sign_gemm_workspace_bytes(M, N, K) if K >= 32 and K % 32 == 0 else 16
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    ws = _sign_ws.get(dev)
    if ws is None or ws.numel() < need:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        _sign_ws[dev] = ws
    return ws


def q1_sign_gemm(x, w_bits, w_scales, y, M: int, N: int, K: int, workspace=None):
    """y = x @ w^T for sign-bit weights. `workspace` (a uint8 CUDA tensor of
    at least q1_sign_gemm_workspace_bytes(M, N, K)) defaults to one cached per
    device, grown as needed and shared by every call on that device that
    passes none: pass your own to run calls on several streams at once."""
    import torch
    G = K // 32 if K % 32 == 0 else -1
    if workspace is None:
        workspace = _sign_workspace(M, N, K, x.device)
    _check(_lib.q1_sign_gemm(_dev(x, torch.float32, M * K, "x"),
                             _dev(w_bits, torch.int32, N * G if G > 0 else None, "w_bits"),
                             _dev(w_scales, torch.float32, N * G if G > 0 else None, "w_scales"),
                             _dev(y, torch.float32, M * N, "y"), M, N, K,
                             _dev(workspace, torch.uint8, None, "workspace"), workspace.numel(), _stream()))


def q1_sign_packed_bytes(N: int, K: int) -> int:
    b = ctypes.c_size_t()
    _check(_lib.q1_sign_packed_bytes(N, K, ctypes.byref(b)))
    return b.value


def q1_sign_pack(w_bits, w_scales, N: int, K: int, w_packed):
    """One-time repack of sign words + scales (uint8 [q1_sign_packed_bytes])."""
    import torch
    G = K // 32 if K % 32 == 0 else None
    _check(_lib.q1_sign_pack(_dev(w_bits, torch.int32, N * G if G else None, "w_bits"),
                             _dev(w_scales, torch.float32, N * G if G else None, "w_scales"), N, K,
                             _dev(w_packed, torch.uint8, q1_sign_packed_bytes(N, K) if G else None, "w_packed"),
                             _stream()))


def q1_sign_gemm_packed(x, w_packed, y, M: int, N: int, K: int, workspace=None):
    import torch
    if workspace is None:
        workspace = _sign_workspace(M, N, K, x.device)
    _check(_lib.q1_sign_gemm_packed(_dev(x, torch.float32, M * K, "x"),
                                    _dev(w_packed, torch.uint8, None, "w_packed"),
                                    _dev(y, torch.float32, M * N, "y"), M, N, K,
                                    _dev(workspace, torch.uint8, None, "workspace"), workspace.numel(), _stream()))


def q1_sign_gemv(x, w_packed, y, M: int, N: int, K: int):
    import torch
    _check(_lib.q1_sign_gemv(_dev(x, torch.float32, M * K, "x"), _dev(w_packed, torch.uint8, None, "w_packed"),
                             _dev(y, torch.float32, M * N, "y"), M, N, K, _stream()))


def q1_sign_gemm_lut4(x, w_packed, y, M: int, N: int, K: int):
    import torch
    _check(_lib.q1_sign_gemm_lut4(_dev(x, torch.float32, M * K, "x"), _dev(w_packed, torch.uint8, None, "w_packed"),
                                  _dev(y, torch.float32, M * N, "y"), M, N, K, _stream()))


# ------------------------------------------------------ block-Q8 matmul_nt

def blockq8_matmul_nt(x, quants, scales, y, m: int, k: int, n: int):
    import torch
    _check(_lib.blockq8_matmul_nt(_dev(x, torch.float32, m * k, "x"),
                                  _dev(quants, torch.int32, n * k // 4 if k % 4 == 0 else None, "quants"),
                                  _dev(scales, torch.float32, n * (k // 32) if k % 32 == 0 else None, "scales"),
                                  _dev(y, torch.float32, m * n, "y"), m, k, n, _stream()))


# ----------------------------------------------------------------- ternary

def ternary_act_bitplanes(x_q, count: int, K: int, planes):
    import torch
    _check(_lib.ternary_act_bitplanes(_dev(x_q, torch.int8, count * K, "x_q"), count, K,
                                      _dev(planes, torch.int32, count * 8 * (K // 32) if K % 32 == 0 else None,
                                           "planes"), _stream()))


def ternary_gemv(w_pos, w_neg, w_scale: float, x_planes, x_scale: float, y, dot_out, rows: int, K: int):
    import torch
    W = K // 32 if K % 32 == 0 else None
    dp = None if dot_out is None else _dev(dot_out, torch.int32, rows, "dot_out")
    _check(_lib.ternary_gemv(_dev(w_pos, torch.int32, rows * W if W else None, "w_pos"),
                             _dev(w_neg, torch.int32, rows * W if W else None, "w_neg"), float(w_scale),
                             _dev(x_planes, torch.int32, 8 * W if W else None, "x_planes"), float(x_scale),
                             _dev(y, torch.float32, rows, "y"), dp, rows, K, _stream()))


def make_ternary_problems(entries, device="cuda"):
    """Device array of gd_ternary_problem from
    [(w_pos, w_neg, x_planes, y, dot_out_or_None, w_scale, x_scale), ...];
    x_scale is a float, or a one-element device f32 tensor (x_scale_dev)."""
    import torch
    arr = (TernaryProblem * len(entries))()
    for i, (p, n, xp, y, d, ws, xs) in enumerate(entries):
        if isinstance(xs, torch.Tensor):
            xs_val, xs_dev = 0.0, _dev(xs, torch.float32, None, "x_scale")
        else:
            xs_val, xs_dev = float(xs), None
        arr[i] = TernaryProblem(p.data_ptr(), n.data_ptr(), xp.data_ptr(), y.data_ptr(),
                                None if d is None else d.data_ptr(), float(ws), xs_val, xs_dev)
    host = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8)
    return host.to(device)


def ternary_gemv_grouped(problems, count: int, rows: int, K: int):
    import torch
    _check(_lib.ternary_gemv_grouped(
        _dev(problems, torch.uint8, count * ctypes.sizeof(TernaryProblem), "problems"), count, rows, K, _stream()))


# ------------------------------------------------- activation quantization

def q8_0_quantize(x, a_q8, n: int, K: int):
    """f32 x [n, K] -> q8_0 blocks (uint8 [n * K/32 * 34]), on the device."""
    import torch
    _check(_lib.q8_0_quantize(_dev(x, torch.float32, n * K, "x"),
                              _dev(a_q8, torch.uint8, n * (K // 32) * 34 if K % 32 == 0 else None, "a_q8"),
                              n, K, _stream()))


def ternary_quantize_act(x, count: int, K: int, planes, x_scale):
    """f32 x [count, K] -> int8 bit planes (int32 [count * 8 * K/32]) and
    scales (f32 [count]), on the device."""
    import torch
    _check(_lib.ternary_quantize_act(_dev(x, torch.float32, count * K, "x"), count, K,
                                     _dev(planes, torch.int32, count * 8 * (K // 32) if K % 32 == 0 else None,
                                          "planes"),
                                     _dev(x_scale, torch.float32, count, "x_scale"), _stream()))


# ------------------------------------------------------ decode attention

def attn_decode_workspace_bytes(n_heads: int, n_kv_heads: int, head_dim: int, kv_len: int,
                                num_splits: int = 0) -> int:
    b = ctypes.c_size_t()
    _check(_lib.attn_decode_workspace_bytes(n_heads, n_kv_heads, head_dim, kv_len, num_splits, ctypes.byref(b)))
    return b.value


def attn_decode_splitk(q, k_cache, v_cache, out, n_heads: int, n_kv_heads: int, head_dim: int, kv_len: int,
                       kv_stride: int, scale: float, num_splits: int = 0, workspace=None):
    """Split-K decode attention for one token; the workspace (uint8) is
    allocated here when not given."""
    import torch
    need = attn_decode_workspace_bytes(n_heads, n_kv_heads, head_dim, kv_len, num_splits)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    cache_n = n_kv_heads * kv_stride * head_dim
    _check(_lib.attn_decode_splitk(_dev(q, torch.float32, n_heads * head_dim, "q"),
                                   _dev(k_cache, torch.float32, cache_n, "k_cache"),
                                   _dev(v_cache, torch.float32, cache_n, "v_cache"),
                                   _dev(out, torch.float32, n_heads * head_dim, "out"),
                                   n_heads, n_kv_heads, head_dim, kv_len, kv_stride, float(scale), num_splits,
                                   _dev(workspace, torch.uint8, None, "workspace"), workspace.numel(), _stream()))


def attn_decode_splitk_noalloc(q, k_cache, v_cache, out, n_heads: int, n_kv_heads: int, head_dim: int,
                               kv_len: int, kv_stride: int, scale: float, num_splits: int = 0):
    """attn_decode_splitk with the split partials in the library's own
    scratch (no workspace, nothing allocated; calls that overlap on one
    device race)."""
    import torch
    cache_n = n_kv_heads * kv_stride * head_dim
    _check(_lib.attn_decode_splitk_noalloc(_dev(q, torch.float32, n_heads * head_dim, "q"),
                                           _dev(k_cache, torch.float32, cache_n, "k_cache"),
                                           _dev(v_cache, torch.float32, cache_n, "v_cache"),
                                           _dev(out, torch.float32, n_heads * head_dim, "out"),
                                           n_heads, n_kv_heads, head_dim, kv_len, kv_stride, float(scale),
                                           num_splits, _stream()))


# -------------------------------------------- norm with an 8-bit output

_dtype_code = {}
_attn_bytes = {}   # workspace bytes by sizes: a pure function of them, called for each launch


def _dtype(t, name):
    """The GD_F32 / GD_F16 / GD_BF16 code of a tensor's type."""
    if not _dtype_code:
        import torch
        _dtype_code.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
    try:
        return _dtype_code[t.dtype]
    except (KeyError, AttributeError):
        raise TypeError(f"{name} must be a float32, float16 or bfloat16 tensor") from None


_device_and_stream = []   # how torch is asked for the current device and its stream


def _current():
    """(index of the current device, torch's current stream on it)."""
    if not _device_and_stream:
        import torch
        if not torch.cuda.is_initialized():
            torch.cuda.init()
        # The calls below torch.cuda's: 0.1 us, where a torch.cuda.Stream object takes 1.1. They are not public: a torch
        # without them is asked the public way.
        device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
        _device_and_stream[:] = device, stream
    device, stream = _device_and_stream
    i = device()
    return i, stream(i)


def _on(index, t, dtype, numel, name):
    """data_ptr of a contiguous tensor of this type and size on device `index`, the one the call launches on."""
    try:
        if t.dtype == dtype and t.get_device() == index and t.is_contiguous() and (numel is None or t.numel() == numel):
            return t.data_ptr()
    except AttributeError:
        pass
    p = _dev(t, dtype, numel, name)   # says what is wrong
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{index}")
    return p


def _rows_on(index, t, dtype, n, heads, head_dim, name):
    """_on of n rows of `heads` head rows: [n, heads, head_dim], or those with the leading or the last axes joined or split
    up. Rows in another order of the axes, the heads first for instance, are refused (where their sizes tell)."""
    try:
        if (t.dtype == dtype and t.get_device() == index and t.is_contiguous()
                and t.shape == (n, heads, head_dim)):
            return t.data_ptr()
    except AttributeError:
        pass
    p, s = _on(index, t, dtype, None, name), t.shape
    if t.numel() != n * heads * head_dim or len(s) > 1 and s[-1] != heads * head_dim and (
            s[-1] != head_dim or len(s) > 2 and s[-2] != heads):
        raise ValueError(f"{name} must be [{n}, {heads}, {head_dim}], got {list(s)}")
    return p


def rmsnorm_q8_0(x, residual, weight, h_out, a_q8, n: int, K: int, eps: float):
    """h = x + residual, and the RMS norm of h times `weight` as q8_0 blocks
    (uint8 [n * K/32 * 34], what q1_q8_gemv reads). x, residual (or None) and
    h_out (or None; may be x or residual) are [n, K] of one type (float32,
    float16, bfloat16); weight float32 [K]."""
    import torch
    dt, (i, stream) = _dtype(x, "x"), _current()
    _check(_lib.rmsnorm_q8_0(_on(i, x, x.dtype, n * K, "x"),
                             None if residual is None else _on(i, residual, x.dtype, n * K, "residual"),
                             _on(i, weight, torch.float32, K, "weight"),
                             None if h_out is None else _on(i, h_out, x.dtype, n * K, "h_out"),
                             _on(i, a_q8, torch.uint8, n * (K // 32) * 34 if K % 32 == 0 else None, "a_q8"),
                             n, K, eps, dt, stream))


def rmsnorm_ternary_act(x, residual, weight, h_out, planes, x_scale, n: int, K: int, eps: float):
    """rmsnorm_q8_0 with one scale per row: int8 bit planes (int32
    [n * 8 * K/32]) and scales (float32 [n]), what ternary_gemv reads."""
    import torch
    dt, (i, stream) = _dtype(x, "x"), _current()
    _check(_lib.rmsnorm_ternary_act(_on(i, x, x.dtype, n * K, "x"),
                                    None if residual is None else _on(i, residual, x.dtype, n * K, "residual"),
                                    _on(i, weight, torch.float32, K, "weight"),
                                    None if h_out is None else _on(i, h_out, x.dtype, n * K, "h_out"),
                                    _on(i, planes, torch.int32, n * 8 * (K // 32) if K % 32 == 0 else None, "planes"),
                                    _on(i, x_scale, torch.float32, n, "x_scale"), n, K, eps, dt, stream))


def _sandwich(i, x, post_weight, residual, weight, h_out, gate, gate_index, n, K):
    """The arguments that the sandwich norms share, checked."""
    import torch
    rows, n_gates = n * K, 0
    if gate is not None:
        n_gates, rest = divmod(gate.numel(), K) if K > 0 else (0, 1)
        if rest or n_gates == 0 or gate.shape[-1] != K:
            raise ValueError(f"gate must be [n_gates, {K}], got {list(gate.shape)}")
    return (_on(i, x, x.dtype, rows, "x"),
            None if post_weight is None else _on(i, post_weight, torch.float32, K, "post_weight"),
            None if gate is None else _on(i, gate, x.dtype, None, "gate"), n_gates,
            None if gate_index is None else _on(i, gate_index, torch.int32, n, "gate_index"),
            _on(i, residual, x.dtype, rows, "residual"), _on(i, weight, torch.float32, K, "weight"),
            None if h_out is None else _on(i, h_out, x.dtype, rows, "h_out"))


def rmsnorm_sandwich_q8_0(x, post_weight, residual, weight, h_out, a_q8, n: int, K: int, eps: float, gate=None,
                          gate_index=None, residual_scale: float = 1.0, block_scale: float = 1.0):
    """The norms behind and before a block: h = residual_scale * residual +
    block_scale * gate * u, u the RMS norm of the block's output x times
    post_weight (None: x itself), and the RMS norm of h times `weight` as q8_0
    blocks. x, residual, h_out (or None; may be x or residual) are [n, K] of one
    type, gate (or None) [n_gates, K] of the same; gate_index int32 [n] names each
    row's gate (None: one gate for all rows, or one per row); weights float32 [K]."""
    import torch
    dt, (i, stream) = _dtype(x, "x"), _current()
    xp, pp, gp, ng, ip, rp, wp, hp = _sandwich(i, x, post_weight, residual, weight, h_out, gate, gate_index, n, K)
    _check(_lib.rmsnorm_sandwich_q8_0(xp, pp, gp, ng, ip, rp, residual_scale, block_scale, wp, hp,
                                      _on(i, a_q8, torch.uint8, n * (K // 32) * 34 if K % 32 == 0 else None, "a_q8"),
                                      n, K, eps, dt, stream))


def rmsnorm_sandwich_ternary_act(x, post_weight, residual, weight, h_out, planes, x_scale, n: int, K: int, eps: float,
                                 gate=None, gate_index=None, residual_scale: float = 1.0, block_scale: float = 1.0):
    """rmsnorm_sandwich_q8_0 with one scale per row: int8 bit planes (int32
    [n * 8 * K/32]) and scales (float32 [n])."""
    import torch
    dt, (i, stream) = _dtype(x, "x"), _current()
    xp, pp, gp, ng, ip, rp, wp, hp = _sandwich(i, x, post_weight, residual, weight, h_out, gate, gate_index, n, K)
    _check(_lib.rmsnorm_sandwich_ternary_act(
        xp, pp, gp, ng, ip, rp, residual_scale, block_scale, wp, hp,
        _on(i, planes, torch.int32, n * 8 * (K // 32) if K % 32 == 0 else None, "planes"),
        _on(i, x_scale, torch.float32, n, "x_scale"), n, K, eps, dt, stream))


def q8_0_dequantize(a_q8, y, n: int, K: int):
    """The values of q8_0 blocks: y [n, K] (float32, float16 or bfloat16)."""
    import torch
    dt, (i, stream) = _dtype(y, "y"), _current()
    _check(_lib.q8_0_dequantize(_on(i, a_q8, torch.uint8, n * (K // 32) * 34 if K % 32 == 0 else None, "a_q8"),
                                _on(i, y, y.dtype, n * K, "y"), n, K, dt, stream))


def ternary_dequantize_act(planes, x_scale, y, n: int, K: int):
    """The values of int8 bit planes and scales: y [n, K]."""
    import torch
    dt, (i, stream) = _dtype(y, "y"), _current()
    _check(_lib.ternary_dequantize_act(_on(i, planes, torch.int32, n * 8 * (K // 32) if K % 32 == 0 else None, "planes"),
                                       _on(i, x_scale, torch.float32, n, "x_scale"), _on(i, y, y.dtype, n * K, "y"),
                                       n, K, dt, stream))


# ---------------------------------------------- products with an epilogue

ACT_NONE, ACT_RELU, ACT_RELU2, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(6)

_plane_bytes = {}    # of a weight by its sizes, and
_linear_bytes = {}   # workspace bytes: pure functions, asked for at each launch


def _kept(table, sizes, of):
    """of(*sizes), kept in `table`."""
    got = table.get(sizes)
    if got is None:
        got = of(*sizes)
        if len(table) >= 4096:
            table.clear()
        table[sizes] = got
    return got


def q1_q8_linear_workspace_bytes(K: int, n_act: int) -> int:
    """Workspace bytes of q1_q8_linear and q1_q8_gated (0 up to four columns)."""
    b = ctypes.c_size_t()
    _check(_lib.q1_q8_linear_workspace_bytes(K, n_act, ctypes.byref(b)))
    return b.value


def _linear(i, a_q8, y, y_q8, rows, K, n_act, residual, workspace):
    """What q1_q8_linear and q1_q8_gated check alike: (a_q8, residual, y, y_q8, dtype, workspace tensor, its address and
    bytes)."""
    import torch
    if y is None:
        dtype, code = (torch.float32, 0) if residual is None else (residual.dtype, _dtype(residual, "residual"))
    else:
        dtype, code = y.dtype, _dtype(y, "y")
    need = _kept(_linear_bytes, (K, n_act), q1_q8_linear_workspace_bytes)
    space = None
    if workspace is not None:
        need, space = workspace.numel(), _on(i, workspace, torch.uint8, None, "workspace")
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=a_q8.device)
        space = workspace.data_ptr()
    return (_on(i, a_q8, torch.uint8, n_act * (K // 32) * 34, "a_q8"),
            None if residual is None else _on(i, residual, dtype, n_act * rows, "residual"),
            None if y is None else _on(i, y, dtype, n_act * rows, "y"),
            None if y_q8 is None else _on(i, y_q8, torch.uint8, n_act * (rows // 32) * 34 if rows % 32 == 0 else None, "y_q8"),
            code, workspace, space, need)


def q1_q8_linear(bits_plane, scale_plane, a_q8, y, rows: int, K: int, n_act: int = 1, bias=None, act: int = ACT_NONE,
                 residual=None, y_q8=None, workspace=None):
    """y = act(W a + bias) + residual for Q1 planes of a [rows, K] weight and
    n_act q8_0 columns: y and residual [n_act, rows] (float32, float16 or
    bfloat16; y may be residual), bias float32 [rows], and the same values as
    q8_0 blocks in y_q8 (uint8 [n_act * rows/32 * 34]) where that is given; y may
    then be None. The workspace (uint8) is allocated here when one is needed and
    not given."""
    import torch
    i, stream = _current()
    bb, sb = _kept(_plane_bytes, (rows, K), q1_planes_bytes)
    ap, rp, yp, qp, dt, workspace, space, need = _linear(i, a_q8, y, y_q8, rows, K, n_act, residual, workspace)
    _check(_lib.q1_q8_linear(_on(i, bits_plane, torch.uint8, bb, "bits_plane"),
                             _on(i, scale_plane, torch.uint8, sb, "scale_plane"), ap,
                             None if bias is None else _on(i, bias, torch.float32, rows, "bias"), act, rp, yp, qp, rows, K,
                             n_act, dt, space, need, stream))


def q1_q8_gated(gate_bits, gate_scales, up_bits, up_scales, a_q8, y, rows: int, K: int, n_act: int = 1,
                act: int = ACT_SILU, gate_bias=None, up_bias=None, y_q8=None, workspace=None):
    """y = act(G a + gate_bias) * (U a + up_bias) for the Q1 planes of a gated
    feed-forward block's two [rows, K] weights; y, y_q8 and the workspace as
    q1_q8_linear's."""
    import torch
    i, stream = _current()
    bb, sb = _kept(_plane_bytes, (rows, K), q1_planes_bytes)
    ap, _, yp, qp, dt, workspace, space, need = _linear(i, a_q8, y, y_q8, rows, K, n_act, None, workspace)
    _check(_lib.q1_q8_gated(_on(i, gate_bits, torch.uint8, bb, "gate_bits"),
                            _on(i, gate_scales, torch.uint8, sb, "gate_scales"),
                            _on(i, up_bits, torch.uint8, bb, "up_bits"), _on(i, up_scales, torch.uint8, sb, "up_scales"), ap,
                            None if gate_bias is None else _on(i, gate_bias, torch.float32, rows, "gate_bias"),
                            None if up_bias is None else _on(i, up_bias, torch.float32, rows, "up_bias"), act, yp, qp, rows,
                            K, n_act, dt, space, need, stream))


# ------------------------------------------------------------ 8-bit cache

class KVCacheQ8:
    """A pool of pages of 8-bit keys and values (gd_kv_q8): codes int8
    [n_pages, n_kv_heads, page_size, head_dim] and scales float16
    [n_pages, n_kv_heads, page_size, head_dim/32] for keys and for values. The
    handle checks the four tensors' shapes and types once and keeps them alive."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        import torch
        if not isinstance(k_codes, torch.Tensor) or k_codes.dim() != 4:
            raise ValueError("k_codes must be [n_pages, n_kv_heads, page_size, head_dim]")
        shape = k_codes.shape
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = shape
        scales = shape[:3] + (self.head_dim // 32,)
        given = ((k_codes, "k_codes", torch.int8, shape), (k_scales, "k_scales", torch.float16, scales),
                 (v_codes, "v_codes", torch.int8, shape), (v_scales, "v_scales", torch.float16, scales))
        for t, name, _, want in given:   # a plane of another order would be misread
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if t.shape != want:
                raise ValueError(f"{name} must be {list(want)}, got {list(t.shape)}")
        planes = [_dev(t, dtype, None, name) for t, name, dtype, _ in given]
        self.device = k_codes.device
        if any(t.device != self.device for t in (k_scales, v_codes, v_scales)):
            raise ValueError("the cache's planes must be on one device")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self._c = _KVQ8(*planes, self.n_pages, self.page_size, self.n_kv_heads, self.head_dim)
        self._ref = ctypes.addressof(self._c)

    def _on(self, index):
        if self.device.index != index:
            raise ValueError(f"the cache is on {self.device}, the current device is cuda:{index}")
        return self._ref


def kv_q8_alloc(n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, device="cuda") -> KVCacheQ8:
    """Allocates a cache pool (contents undefined until stored)."""
    import torch
    shape = (n_pages, n_kv_heads, page_size)
    codes = [torch.empty(shape + (head_dim,), dtype=torch.int8, device=device) for _ in range(2)]
    scales = [torch.empty(shape + (head_dim // 32,), dtype=torch.float16, device=device) for _ in range(2)]
    return KVCacheQ8(codes[0], scales[0], codes[1], scales[1])


def rope_table(table, n_pos: int, rot_dim: int, base: float = 10000.0, scaling: RopeScaling = None):
    """Fills table (float32 [n_pos, rot_dim/2, 2]) with the (cos, sin) of every
    position's rotary angles, frequencies scaled by `scaling` if given."""
    import torch
    i, stream = _current()
    if scaling is not None and not isinstance(scaling, RopeScaling):
        raise TypeError("scaling must be a RopeScaling")
    _check(_lib.rope_table(_on(i, table, torch.float32, n_pos * (rot_dim // 2) * 2, "table"), n_pos, rot_dim, base,
                           None if scaling is None else ctypes.addressof(scaling), stream))


def _token_rows(i, t, dtype, n_tok, width, name, head_dim=None):
    """(data_ptr, stride between tokens) of a tensor of n_tok rows of `width`
    elements: [n_tok, width] or [n_tok, heads, head_dim] (or the heads joined,
    [n_tok, 1, width]), each row contiguous."""
    try:
        good = t.dtype == dtype and t.get_device() == i
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if not good:
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{i}")
    shape, strides = t.shape, t.stride()
    if len(shape) == 3:
        rows, inner = shape[1] * shape[2], strides[2] == 1 and (strides[1] == shape[2] or shape[1] == 1)
        if head_dim is not None and shape[2] != head_dim and shape[1] != 1:
            raise ValueError(f"{name} must be [{n_tok}, {width // head_dim}, {head_dim}], got {list(shape)}")
    elif len(shape) == 2:
        rows, inner = shape[1], strides[1] == 1
    else:
        raise ValueError(f"{name} must be [n_tok, heads, head_dim] or [n_tok, heads * head_dim]")
    if shape[0] != n_tok or rows != width:
        raise ValueError(f"{name} must hold {n_tok} rows of {width} elements, got {tuple(shape)}")
    if not inner:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.data_ptr(), strides[0] if n_tok > 1 else width


def kv_q8_store(cache: KVCacheQ8, k, v, slots, n_tok: int, q=None, q_out=None, n_heads: int = 0, rope=None,
                positions=None, interleaved: bool = False):
    """Rotates q and k (rope from rope_table, positions int32 [n_tok]; both or
    neither), writes q_out, and stores k and v in the cache at `slots` (int64
    [n_tok]; -1: not stored). q, k and v may be parts of one projection's rows
    (token strides are free); q_out [n_tok, n_heads, head_dim] may be q."""
    import torch
    dt, (i, stream) = _dtype(k, "k"), _current()
    ref, D = cache._on(i), cache.head_dim
    kp, ks = _token_rows(i, k, k.dtype, n_tok, cache.n_kv_heads * D, "k", D)
    vp, vs = _token_rows(i, v, k.dtype, n_tok, cache.n_kv_heads * D, "v", D)
    qp = qo = None
    qs = 0
    if n_heads:
        qp, qs = _token_rows(i, q, k.dtype, n_tok, n_heads * D, "q", D)
        qo = _rows_on(i, q_out, k.dtype, n_tok, n_heads, D, "q_out")
    elif q is not None or q_out is not None:
        raise ValueError("q and q_out need n_heads")
    rp = pp = None
    n_pos = rot = 0
    if rope is not None:
        rp = _on(i, rope, torch.float32, None, "rope")
        if rope.dim() != 3 or rope.shape[2] != 2:
            raise ValueError("rope must be [n_pos, rot_dim/2, 2]")
        if rope.numel() == 0:   # its address would be NULL, which asks for no rotation
            raise ValueError("rope is empty")
        n_pos, rot = rope.shape[0], 2 * rope.shape[1]
    if positions is not None:
        pp = _on(i, positions, torch.int32, n_tok, "positions")
    _check(_lib.kv_q8_store(ref, qp, qs, kp, ks, vp, vs, qo, rp, n_pos, rot, bool(interleaved), pp,
                            _on(i, slots, torch.int64, n_tok, "slots"), n_tok, n_heads, dt, stream))


def kv_q8_load(cache: KVCacheQ8, slots, k_out, v_out, n_tok: int):
    """The cached rows at `slots` (int64 [n_tok]; outside the pool: zeros) as
    k_out and v_out [n_tok, n_kv_heads, head_dim]; either may be None."""
    import torch
    one = v_out if k_out is None else k_out
    dt, (i, stream) = _dtype(one, "k_out" if k_out is not None else "v_out"), _current()
    H, D = cache.n_kv_heads, cache.head_dim
    _check(_lib.kv_q8_load(cache._on(i), _on(i, slots, torch.int64, n_tok, "slots"),
                           None if k_out is None else _rows_on(i, k_out, one.dtype, n_tok, H, D, "k_out"),
                           None if v_out is None else _rows_on(i, v_out, one.dtype, n_tok, H, D, "v_out"), n_tok, dt,
                           stream))


def attn_decode_q8_workspace_bytes(n_seqs: int, n_q: int, n_heads: int, n_kv_heads: int, head_dim: int, max_q: int,
                                   max_kv_len: int) -> int:
    """Workspace bytes that serve this call and every one no larger in n_seqs, n_q, max_q and max_kv_len."""
    b = ctypes.c_size_t()
    _check(_lib.attn_decode_q8_workspace_bytes(n_seqs, n_q, n_heads, n_kv_heads, head_dim, max_q, max_kv_len,
                                               ctypes.byref(b)))
    return b.value


def attn_decode_q8(q, cache: KVCacheQ8, page_table, kv_lens, q_start, tree_mask, out, n_heads: int, max_q: int,
                   max_kv_len: int, scale: float, softcap: float = 0.0, workspace=None):
    """Attention of each sequence's last tokens over the 8-bit cache. q and out
    are [n_q, n_heads, head_dim]; page_table int32 [n_seqs, max_pages] or None
    (sequence b is page b); kv_lens int32 [n_seqs]; q_start int32 [n_seqs + 1]
    or None (max_q rows per sequence); tree_mask int64 [n_q] (the bits of each
    word: the drafted tokens of its sequence that the row sees) or None (a
    chain). The workspace (uint8) is allocated here when not given."""
    import torch
    dt, (i, stream) = _dtype(q, "q"), _current()
    ref, D = cache._on(i), cache.head_dim
    lens = _on(i, kv_lens, torch.int32, None, "kv_lens")
    n_seqs = kv_lens.numel()
    n_q, rest = divmod(q.numel(), n_heads * D) if n_heads > 0 else (0, 1)
    if rest or n_q == 0:
        raise ValueError(f"q must be [n_q, {n_heads}, {D}], got {tuple(q.shape)}")
    qp, op = _rows_on(i, q, q.dtype, n_q, n_heads, D, "q"), _rows_on(i, out, q.dtype, n_q, n_heads, D, "out")
    table, max_pages = None, 1
    if page_table is not None:
        table = _on(i, page_table, torch.int32, None, "page_table")
        if page_table.dim() != 2 or page_table.shape[0] != n_seqs:
            raise ValueError(f"page_table must be [{n_seqs}, max_pages], got {tuple(page_table.shape)}")
        if page_table.numel() == 0:   # its address would be NULL, which stands for no table
            raise ValueError("page_table is empty")
        max_pages = page_table.shape[1]
    if workspace is None:
        sizes = (n_seqs, n_q, n_heads, cache.n_kv_heads, D, max_q, max_kv_len)
        need = _attn_bytes.get(sizes)
        if need is None:
            need = attn_decode_q8_workspace_bytes(*sizes)
            if len(_attn_bytes) >= 4096:
                _attn_bytes.clear()
            _attn_bytes[sizes] = need
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        space = workspace.data_ptr()
    else:
        need, space = workspace.numel(), _on(i, workspace, torch.uint8, None, "workspace")
    _check(_lib.attn_decode_q8(ref, qp, op, table, max_pages, lens,
                               None if q_start is None else _on(i, q_start, torch.int32, n_seqs + 1, "q_start"),
                               None if tree_mask is None else _on(i, tree_mask, torch.int64, n_q, "tree_mask"),
                               n_seqs, n_q, n_heads, max_q, max_kv_len, scale, softcap, dt,
                               space, need, stream))


# -------------------------------------------------------- log probabilities

_logprobs_bytes = {}   # workspace bytes by sizes


def token_logprobs_workspace_bytes(n: int, V: int, k: int) -> int:
    """Workspace bytes that serve this call and every one no larger in n, V and k."""
    b = ctypes.c_size_t()
    _check(_lib.token_logprobs_workspace_bytes(n, V, k, ctypes.byref(b)))
    return b.value


def token_logprobs(logits, tokens, logprobs, entropy, top_ids, top_logprobs, n: int, V: int, scale: float = 1.0,
                   softcap: float = 0.0, workspace=None):
    """Natural log probabilities of logits [n, V] (float32, float16 or bfloat16;
    rows may be apart, as logits[:, :V] of a padded vocabulary), scaled (1 /
    temperature) and capped: of tokens (int64 [n, n_given], -1: padding) into
    logprobs (float32, the same shape), of each row's entropy (float32 [n]), and of the
    k <= 64 largest logits (top_ids int64 [n, k], top_logprobs float32 [n, k]).
    Pairs that are not asked for are None. The workspace (uint8) is allocated
    here when one is needed and not given."""
    import torch
    dt, (i, stream) = _dtype(logits, "logits"), _current()
    if logits.get_device() != i:
        raise ValueError(f"logits is on {logits.device}, the current device is cuda:{i}")
    shape = logits.shape
    if len(shape) == 1 and n == 1 and shape[0] == V and logits.stride(0) == 1:
        stride = V
    elif len(shape) == 2 and shape[0] == n and shape[1] == V and (logits.stride(1) == 1 or V == 1):
        stride = logits.stride(0) if n > 1 else V
    else:
        raise ValueError(f"logits must be [{n}, {V}] with contiguous rows, got {list(shape)}")

    def of(a, b, first, second, names):
        if (a is None) != (b is None):
            raise ValueError(f"{names[0]} and {names[1]} come together")
        if a is None:
            return None, None, 0
        if len(a.shape) not in (1, 2) or a.shape[0] != n or a.shape != b.shape:
            raise ValueError(f"{names[0]} and {names[1]} must be [{n}, number each], got {list(a.shape)} and {list(b.shape)}")
        if a.numel() == 0:
            raise ValueError(f"{names[0]} is empty")
        return _on(i, a, first, None, names[0]), _on(i, b, second, None, names[1]), a.numel() // n
    tp, lp, n_given = of(tokens, logprobs, torch.int64, torch.float32, ("tokens", "logprobs"))
    kp, kl, k = of(top_ids, top_logprobs, torch.int64, torch.float32, ("top_ids", "top_logprobs"))
    space, need = None, 0
    if workspace is not None:
        need, space = workspace.numel(), _on(i, workspace, torch.uint8, None, "workspace")
    else:
        need = _kept(_logprobs_bytes, (n, V, k), token_logprobs_workspace_bytes)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=logits.device)
            space = workspace.data_ptr()
    _check(_lib.token_logprobs(logits.data_ptr(), stride, tp, n_given, lp,
                               None if entropy is None else _on(i, entropy, torch.float32, n, "entropy"), kp, kl, k, n, V,
                               scale, softcap, dt, space, need, stream))


# ------------------------------------------------------------ measurement

def gemm_decode_fill(buf, seed: int = 1):
    import torch
    _check(_lib.gemm_decode_fill(_dev(buf, torch.uint8, None, "buf"), buf.numel(), seed, _stream()))


def gemm_decode_stream_read(buf, passes: int, sink):
    import torch
    _check(_lib.gemm_decode_stream_read(_dev(buf, torch.uint8, None, "buf"), buf.numel(), passes,
                                        _dev(sink, torch.int32, None, "sink"), sink.numel(), _stream()))
