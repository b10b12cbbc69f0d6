"""ctypes binding of libbitlinear (include/bitlinear.h).

Argument marshalling only: each function checks that its torch tensors are on
the GPU, contiguous and of the right dtype, allocates outputs (and the
workspace) with torch when the caller gives none, and passes raw device
pointers and the current HIP stream to the C entry point of the same name.
Every step of the computation runs in libbitlinear's kernels.  There is no
fallback: if the library is missing, ``load()`` raises.

The calls on the paged caches are made by ``_calls`` (csrc/torch_calls.cpp) where
nothing about their arguments is out of the ordinary, as a decode step waits for
the host otherwise; what that leaves is made, or refused, here, and so are all
calls where ``_calls`` has not been built.
"""
import collections
import ctypes
import importlib
import os
import sys
import warnings

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libbitlinear.so")

BL_F32 = 0
BL_BF16 = 1
BL_OP_QUANT_WEIGHT = 0
BL_OP_FFN_RELU2 = 1
BL_MAX_K = 131072

STATUS = {0: "BL_OK", 1: "BL_ERR_NULL", 2: "BL_ERR_SHAPE", 3: "BL_ERR_DTYPE",
          4: "BL_ERR_ALIGN", 5: "BL_ERR_WORKSPACE", 6: "BL_ERR_ARCH", 7: "BL_ERR_HIP"}

EXPORTS = ["quant_weight_absmean_pack", "quant_weight_absmean_pack_noalloc", "quant_act_absmax_i8",
           "quant_act_absmax_i4", "bitlinear_a4", "bitlinear_gemv",
           "bitlinear_gemm", "bitlinear_gemv_fused", "bitlinear_ffn_relu2",
           "bitlinear_decode_stack", "bitlinear_decode_stack_status",
           "bitlinear_backward_input", "bitlinear_backward_weight",
           "bitlinear_t5_row_bytes", "bitlinear_repack_t5", "bitlinear_gemv_t5",
           "bitlinear_kv8_append", "bitlinear_kv8_attention", "bitlinear_kv8_attention_ws_bytes",
           "bitlinear_kv8_append_rope", "bitlinear_kv8_read", "bitlinear_kv4_append", "bitlinear_kv4_read",
           "bitlinear_kv4_attention", "bitlinear_kv4_attention_ws_bytes",
           "bitlinear_decode_stack_kv", "bitlinear_decode_stack_kv_ws_bytes",
           "bitlinear_decode_stack_kv_rope", "bitlinear_decode_stack_kv4", "bitlinear_decode_stack_kv4_ws_bytes",
           "quant_weight_absmax_i4", "dequant_weight_i4", "bitlinear_gemv_w4",
           "bl_workspace_bytes", "bl_status_string", "bl_last_error", "bl_abi_version"]
BL_OP_DECODE_STACK = 2
BL_OP_BACKWARD_INPUT = 3
BL_OP_BACKWARD_WEIGHT = 4
LAYER_WEIGHTS = ("Wq", "Wk", "Wv", "Wo", "Wg", "Wu", "Wd")
LAYER_GAMMAS = ("gq", "gk", "gv", "go", "gg", "gu", "gd")


class Layer(ctypes.Structure):
    """bl_layer (include/bitlinear.h)."""
    _fields_ = [(n, ctypes.c_void_p) for n in LAYER_WEIGHTS + LAYER_GAMMAS + ("ffn_norm",)]


class StackDims(ctypes.Structure):
    """bl_stack_dims (include/bitlinear.h)."""
    _fields_ = [("H", ctypes.c_int64), ("KV", ctypes.c_int64), ("F", ctypes.c_int64),
                ("D", ctypes.c_int64), ("eps", ctypes.c_float), ("path", ctypes.c_int32),
                ("wait_us", ctypes.c_int32), ("reserved", ctypes.c_int32)]


BL_STACK_AUTO = 0
BL_STACK_LAUNCHES = 1
BL_STACK_PERSISTENT = 2
BL_MAX_JOBS = 8


class GemvJob(ctypes.Structure):
    """bl_gemv_job (include/bitlinear.h)."""
    _fields_ = [("X", ctypes.c_void_p), ("Wp", ctypes.c_void_p), ("gamma", ctypes.c_void_p),
                ("Y", ctypes.c_void_p), ("Xq", ctypes.c_void_p), ("d", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Kv8(ctypes.Structure):
    """bl_kv8 (include/bitlinear.h)."""
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("sk", ctypes.c_void_p),
                ("sv", ctypes.c_void_p), ("n_blocks", ctypes.c_int64), ("KVH", ctypes.c_int64),
                ("T", ctypes.c_int64), ("D", ctypes.c_int64)]


class Kv4(ctypes.Structure):
    """bl_kv4 (include/bitlinear.h)."""
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("zk", ctypes.c_void_p),
                ("zv", ctypes.c_void_p), ("n_blocks", ctypes.c_int64), ("KVH", ctypes.c_int64),
                ("T", ctypes.c_int64), ("D", ctypes.c_int64)]


class BlRope(ctypes.Structure):
    """bl_rope (include/bitlinear.h)."""
    _fields_ = [("cos_sin", ctypes.c_void_p), ("rows", ctypes.c_int64), ("rot", ctypes.c_int64),
                ("interleaved", ctypes.c_int32), ("reserved", ctypes.c_int32)]


# An 8-bit key/value cache: K int8 [n_blocks, KVH, T, D], V int8 [n_blocks,
# KVH, D, T], sk and sv fp32 [n_blocks, KVH].  Calls take any such 4-tuple.
Kv8Cache = collections.namedtuple("Kv8Cache", ("K", "V", "sk", "sv"))
# A 4-bit one: K uint8 [n_blocks, KVH, T, D/2], V uint8 [n_blocks, KVH, T/16, D,
# 8], zk and zv fp16 [n_blocks, KVH, T, 2] (least value and step).
Kv4Cache = collections.namedtuple("Kv4Cache", ("K", "V", "zk", "zv"))
# A rotation: cos_sin fp32 [positions, rot], rot / 2 cosines and then rot / 2
# sines a row; pairs (2i, 2i + 1) where interleaved, else (i, i + rot / 2).
Rope = collections.namedtuple("Rope", ("cos_sin", "interleaved"), defaults=(False,))

_lib = None
_calls = None
_ENTRIES = ("bitlinear_kv8_append", "bitlinear_kv8_append_rope", "bitlinear_kv4_append", "bitlinear_kv8_read",
            "bitlinear_kv4_read", "bitlinear_kv8_attention", "bitlinear_kv4_attention",
            "bitlinear_kv8_attention_ws_bytes", "bitlinear_kv4_attention_ws_bytes")
_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t


class BitLinearError(RuntimeError):
    def __init__(self, call, status, detail):
        self.call, self.status, self.detail = call, status, detail
        super().__init__(f"{call}: {STATUS.get(status, status)}: {detail}")


def _bind(lib, calls):
    calls.bind(_check, *(ctypes.cast(getattr(lib, name), _p).value for name in _ENTRIES))


def _short_way(lib):
    """_calls on the library's entry points, or None: it saves 5 us of host time a call
    and nothing else, so where it was not built, or for another torch or Python, the calls are
    made through ctypes."""
    try:
        calls = importlib.import_module("._calls", __package__)
    except ImportError as e:
        why = str(e)
    else:
        here = f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"
        built_for = getattr(calls, "built_for", "another torch")
        if built_for == here:
            _bind(lib, calls)
            return calls
        why = f"it was built for {built_for}, this is {here}"
    warnings.warn(f"_calls.so is not used, calls on the paged caches take 5 us more of host time ({why}); run "
                  "`python -m ternary_weight_linear_absmean_amd.build`", RuntimeWarning, stacklevel=3)
    return None


def load():
    """Load libbitlinear.so (built in-tree by build.py), and _calls.so if it is there;
    raise if the library is missing."""
    global _lib, _calls
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run "
                          "`python -m ternary_weight_linear_absmean_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    st = ctypes.c_int
    lib.quant_weight_absmean_pack.restype = st
    lib.quant_weight_absmean_pack.argtypes = [_p, _i64, _i64, _p, _p, _p, _sz, _p]
    lib.quant_weight_absmean_pack_noalloc.restype = st
    lib.quant_weight_absmean_pack_noalloc.argtypes = [_p, _i64, _i64, _p, _p, _p]
    lib.quant_act_absmax_i8.restype = st
    lib.quant_act_absmax_i8.argtypes = [_p, ctypes.c_int, _i64, _i64, _p, _p, _p]
    lib.quant_act_absmax_i4.restype = st
    lib.quant_act_absmax_i4.argtypes = [_p, ctypes.c_int, _i64, _i64, _p, _p, _p]
    for name in ("bitlinear_gemv", "bitlinear_gemm", "bitlinear_a4"):
        f = getattr(lib, name)
        f.restype = st
        f.argtypes = [_p, _p, _i64, _p, _p, _i64, _i64, _p, _p, _p]
    lib.bitlinear_gemv_fused.restype = st
    lib.bitlinear_gemv_fused.argtypes = [ctypes.POINTER(GemvJob), ctypes.c_int, _i64, _p]
    lib.bitlinear_decode_stack.restype = st
    lib.bitlinear_decode_stack.argtypes = [ctypes.POINTER(Layer), ctypes.c_int,
                                           ctypes.POINTER(StackDims), _p, _p, _p, _sz, _p]
    lib.bitlinear_decode_stack_status.restype = st
    lib.bitlinear_decode_stack_status.argtypes = [_p, _sz, ctypes.POINTER(StackDims),
                                                  ctypes.POINTER(ctypes.c_int32)]
    lib.bitlinear_ffn_relu2.restype = st
    lib.bitlinear_ffn_relu2.argtypes = [_p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _p,
                                        ctypes.c_float, _p, _p, _i64, _p, _p, _p, _p, _sz, _p]
    lib.bl_workspace_bytes.restype = _sz
    for name in ("bitlinear_backward_input", "bitlinear_backward_weight"):
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = [_p, _i64, _i64, _p, _p, _i64, _p, _p, _sz, _p]
    lib.bl_workspace_bytes.argtypes = [ctypes.c_int, _i64, _i64, _i64, _i64]
    lib.bitlinear_t5_row_bytes.restype = _sz
    lib.bitlinear_t5_row_bytes.argtypes = [_i64]
    lib.bitlinear_repack_t5.restype = st
    lib.bitlinear_repack_t5.argtypes = [_p, _i64, _i64, _p, _p]
    lib.bitlinear_gemv_t5.restype = st
    lib.bitlinear_gemv_t5.argtypes = [_p, _p, _i64, _p, _p, _i64, _i64, _p, _p, _p]
    i32 = ctypes.c_int
    lib.bitlinear_kv8_append.restype = st
    lib.bitlinear_kv8_append.argtypes = [_p, _p, i32, _i64, _p, _p, _p, _i64, _i64,
                                         ctypes.POINTER(Kv8), _p]
    lib.bitlinear_kv8_attention.restype = st
    lib.bitlinear_kv8_attention.argtypes = [_p, i32, _i64, _i64, _p, _p, _p, _i64, _i64,
                                            ctypes.POINTER(Kv8), ctypes.c_float, _p, _p, _sz, _p]
    lib.bitlinear_kv8_attention_ws_bytes.restype = _sz
    lib.bitlinear_kv8_attention_ws_bytes.argtypes = [_i64] * 7
    lib.bitlinear_kv8_append_rope.restype = st
    lib.bitlinear_kv8_append_rope.argtypes = [_p, _p, _p, _p, i32, _i64, _i64, _p, _p, _p, _i64, _i64,
                                              ctypes.POINTER(Kv8), ctypes.POINTER(BlRope), _p]
    lib.bitlinear_kv4_append.restype = st
    lib.bitlinear_kv4_append.argtypes = [_p, _p, _p, _p, i32, _i64, _i64, _p, _p, _p, _i64, _i64,
                                         ctypes.POINTER(Kv4), ctypes.POINTER(BlRope), _p]
    lib.bitlinear_kv4_attention.restype = st
    lib.bitlinear_kv4_attention.argtypes = [_p, i32, _i64, _i64, _p, _p, _p, _i64, _i64,
                                            ctypes.POINTER(Kv4), ctypes.c_float, _p, _p, _sz, _p]
    lib.bitlinear_kv4_attention_ws_bytes.restype = _sz
    lib.bitlinear_kv4_attention_ws_bytes.argtypes = [_i64] * 7
    for name, kind in (("bitlinear_kv8_read", Kv8), ("bitlinear_kv4_read", Kv4)):
        f = getattr(lib, name)
        f.restype = st
        f.argtypes = [ctypes.POINTER(kind), _p, _p, _p, _i64, _i64, _i64, _p, _p, i32, _p]
    lib.bitlinear_decode_stack_kv.restype = st
    lib.bitlinear_decode_stack_kv.argtypes = [
        ctypes.POINTER(Layer), ctypes.POINTER(Kv8), i32, ctypes.POINTER(StackDims), _p, _p, _p, _i64,
        ctypes.c_float, _p, _p, _p, _sz, _p]
    lib.bitlinear_decode_stack_kv_ws_bytes.restype = _sz
    lib.bitlinear_decode_stack_kv_ws_bytes.argtypes = [ctypes.POINTER(StackDims), _i64, _i64]
    for name, kind in (("bitlinear_decode_stack_kv_rope", Kv8), ("bitlinear_decode_stack_kv4", Kv4)):
        f = getattr(lib, name)
        f.restype = st
        f.argtypes = [ctypes.POINTER(Layer), ctypes.POINTER(kind), i32, ctypes.POINTER(StackDims), _p, _p, _p, _i64,
                      ctypes.POINTER(BlRope), ctypes.c_float, _p, _p, _p, _sz, _p]
    lib.bitlinear_decode_stack_kv4_ws_bytes.restype = _sz
    lib.bitlinear_decode_stack_kv4_ws_bytes.argtypes = [ctypes.POINTER(StackDims), _i64, _i64]
    lib.quant_weight_absmax_i4.restype = st
    lib.quant_weight_absmax_i4.argtypes = [_p, i32, _i64, _i64, _i64, _p, _p, _p]
    lib.dequant_weight_i4.restype = st
    lib.dequant_weight_i4.argtypes = [_p, _p, _i64, _i64, _i64, _p, i32, _p]
    lib.bitlinear_gemv_w4.restype = st
    lib.bitlinear_gemv_w4.argtypes = [_p, i32, _i64, _p, _p, _i64, _i64, _i64, _p, _p]
    lib.bl_status_string.restype = ctypes.c_char_p
    lib.bl_status_string.argtypes = [ctypes.c_int]
    lib.bl_last_error.restype = ctypes.c_char_p
    lib.bl_last_error.argtypes = []
    lib.bl_abi_version.restype = ctypes.c_int
    lib.bl_abi_version.argtypes = []
    _lib, _calls = lib, _short_way(lib)
    return lib


def _check(call, status):
    if status != 0:
        raise BitLinearError(call, status, load().bl_last_error().decode())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t, dtype, name):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def workspace_bytes(op, M=0, N=0, K=0, F=0):
    return int(load().bl_workspace_bytes(op, M, N, K, F))


def quant_weight_absmean_pack(W, Wp=None, gamma=None, ws=None, stream=None):
    """fp32 W [N, K] -> (packed uint8 [N, K/4], gamma fp32 [1]) on the GPU."""
    _dev(W, torch.float32, "W")
    N, K = W.shape
    dev = W.device
    Wp = _dev(Wp, torch.uint8, "Wp") if Wp is not None else torch.empty(
        (N, K // 4), dtype=torch.uint8, device=dev)
    gamma = _dev(gamma, torch.float32, "gamma") if gamma is not None else torch.empty(
        (1,), dtype=torch.float32, device=dev)
    need = workspace_bytes(BL_OP_QUANT_WEIGHT, 0, N, K, 0)
    if ws is None:
        ws = torch.empty((max(need, 16),), dtype=torch.uint8, device=dev)
    _check("quant_weight_absmean_pack", load().quant_weight_absmean_pack(
        _ptr(W), N, K, _ptr(Wp), _ptr(gamma), _ptr(ws), ws.numel(), _stream(stream)))
    return Wp, gamma


def quant_weight_absmean_pack_noalloc(W, Wp=None, gamma=None, stream=None):
    """quant_weight_absmean_pack with the library's own scratch (no workspace);
    N * K <= 2^27.  Pass Wp and gamma to keep the call itself free of
    allocation (torch allocates them here when they are absent)."""
    _dev(W, torch.float32, "W")
    N, K = W.shape
    dev = W.device
    Wp = _dev(Wp, torch.uint8, "Wp") if Wp is not None else torch.empty(
        (N, K // 4), dtype=torch.uint8, device=dev)
    gamma = _dev(gamma, torch.float32, "gamma") if gamma is not None else torch.empty(
        (1,), dtype=torch.float32, device=dev)
    _check("quant_weight_absmean_pack_noalloc", load().quant_weight_absmean_pack_noalloc(
        _ptr(W), N, K, _ptr(Wp), _ptr(gamma), _stream(stream)))
    return Wp, gamma


def quant_act_absmax_i8(X, Xq=None, d=None, stream=None):
    """X [M, K] (fp32 or bf16) -> (Xq int8 [M, K], d fp32 [M])."""
    if X.dtype == torch.float32:
        dt = BL_F32
    elif X.dtype == torch.bfloat16:
        dt = BL_BF16
    else:
        raise TypeError("X must be float32 or bfloat16")
    _dev(X, X.dtype, "X")
    M, K = X.shape
    Xq = _dev(Xq, torch.int8, "Xq") if Xq is not None else torch.empty(
        (M, K), dtype=torch.int8, device=X.device)
    d = _dev(d, torch.float32, "d") if d is not None else torch.empty(
        (M,), dtype=torch.float32, device=X.device)
    _check("quant_act_absmax_i8", load().quant_act_absmax_i8(
        _ptr(X), dt, M, K, _ptr(Xq), _ptr(d), _stream(stream)))
    return Xq, d


def _product(call, Xq, d, Wp, gamma, Y, acc, want_acc, stream, a4=False):
    _dev(Xq, torch.uint8 if a4 else torch.int8, "Xq4" if a4 else "Xq")
    _dev(d, torch.float32, "d")
    _dev(Wp, torch.uint8, "Wp")
    _dev(gamma, torch.float32, "gamma")
    M, K = Xq.shape
    if a4:
        K *= 2
    N = Wp.shape[0]
    if Wp.dim() != 2 or Wp.shape[1] * 4 != K:
        raise ValueError(f"Wp must be [N, K/4] = [*, {K // 4}], got {tuple(Wp.shape)}")
    if d.shape != (M,):
        raise ValueError("d must be [M]")
    Y = _dev(Y, torch.float32, "Y") if Y is not None else torch.empty(
        (M, N), dtype=torch.float32, device=Xq.device)
    if acc is None and want_acc:
        acc = torch.empty((M, N), dtype=torch.int32, device=Xq.device)
    _dev(acc, torch.int32, "acc")
    _check(call, getattr(load(), call)(_ptr(Xq), _ptr(d), M, _ptr(Wp), _ptr(gamma), N, K,
                                       _ptr(Y), _ptr(acc), _stream(stream)))
    return (Y, acc) if want_acc or acc is not None else Y


def bitlinear_gemv(Xq, d, Wp, gamma, Y=None, acc=None, want_acc=False, stream=None):
    """Y [M, N] fp32 for 1 <= M <= 64 tokens; with want_acc also int32 acc."""
    return _product("bitlinear_gemv", Xq, d, Wp, gamma, Y, acc, want_acc, stream)


def bitlinear_gemm(Xq, d, Wp, gamma, Y=None, acc=None, want_acc=False, stream=None):
    """Y [M, N] fp32 for any M on int8 MFMA; with want_acc also int32 acc."""
    return _product("bitlinear_gemm", Xq, d, Wp, gamma, Y, acc, want_acc, stream)


def quant_act_absmax_i4(X, Xq4=None, d=None, stream=None):
    """X [M, K] (fp32 or bf16, K even) -> (Xq4 uint8 [M, K/2] 4-bit codes, d fp32 [M])."""
    if X.dtype == torch.float32:
        dt = BL_F32
    elif X.dtype == torch.bfloat16:
        dt = BL_BF16
    else:
        raise TypeError("X must be float32 or bfloat16")
    _dev(X, X.dtype, "X")
    M, K = X.shape
    Xq4 = _dev(Xq4, torch.uint8, "Xq4") if Xq4 is not None else torch.empty(
        (M, K // 2), dtype=torch.uint8, device=X.device)
    d = _dev(d, torch.float32, "d") if d is not None else torch.empty(
        (M,), dtype=torch.float32, device=X.device)
    _check("quant_act_absmax_i4", load().quant_act_absmax_i4(
        _ptr(X), dt, M, K, _ptr(Xq4), _ptr(d), _stream(stream)))
    return Xq4, d


def bitlinear_a4(Xq4, d, Wp, gamma, Y=None, acc=None, want_acc=False, stream=None):
    """Y [M, N] fp32 from 4-bit activation codes Xq4 uint8 [M, K/2]; with
    want_acc also the int32 accumulator."""
    return _product("bitlinear_a4", Xq4, d, Wp, gamma, Y, acc, want_acc, stream, a4=True)


def t5_row_bytes(K):
    """Bytes per row of the five-weights-per-byte format (0 if K is out of range)."""
    return int(load().bitlinear_t5_row_bytes(K))


def bitlinear_repack_t5(Wp, K=None, Wt5=None, stream=None):
    """2-bit packed Wp [N, K/4] -> Wt5 uint8 [N, t5_row_bytes(K)] (same weights)."""
    _dev(Wp, torch.uint8, "Wp")
    N = Wp.shape[0]
    K = Wp.shape[1] * 4 if K is None else K
    if Wp.dim() != 2 or Wp.shape[1] * 4 != K:
        raise ValueError(f"Wp must be [N, K/4], got {tuple(Wp.shape)} for K={K}")
    rb = t5_row_bytes(K)
    Wt5 = _dev(Wt5, torch.uint8, "Wt5") if Wt5 is not None else torch.empty(
        (N, rb), dtype=torch.uint8, device=Wp.device)
    if tuple(Wt5.shape) != (N, rb):
        raise ValueError(f"Wt5 must be [{N}, {rb}]")
    _check("bitlinear_repack_t5", load().bitlinear_repack_t5(_ptr(Wp), N, K, _ptr(Wt5),
                                                             _stream(stream)))
    return Wt5


def bitlinear_gemv_t5(Xq, d, Wt5, gamma, Y=None, acc=None, want_acc=False, stream=None):
    """Y [M, N] fp32 from five-per-byte weights, 1 <= M <= 8; with want_acc
    also the int32 accumulator."""
    _dev(Xq, torch.int8, "Xq")
    _dev(d, torch.float32, "d")
    _dev(Wt5, torch.uint8, "Wt5")
    _dev(gamma, torch.float32, "gamma")
    M, K = Xq.shape
    N = Wt5.shape[0]
    if Wt5.dim() != 2 or Wt5.shape[1] != t5_row_bytes(K):
        raise ValueError(f"Wt5 must be [N, {t5_row_bytes(K)}], got {tuple(Wt5.shape)}")
    if d.shape != (M,):
        raise ValueError("d must be [M]")
    Y = _dev(Y, torch.float32, "Y") if Y is not None else torch.empty(
        (M, N), dtype=torch.float32, device=Xq.device)
    if acc is None and want_acc:
        acc = torch.empty((M, N), dtype=torch.int32, device=Xq.device)
    _dev(acc, torch.int32, "acc")
    _check("bitlinear_gemv_t5", load().bitlinear_gemv_t5(
        _ptr(Xq), _ptr(d), M, _ptr(Wt5), _ptr(gamma), N, K, _ptr(Y), _ptr(acc),
        _stream(stream)))
    return (Y, acc) if want_acc or acc is not None else Y


def bitlinear_gemv_fused(jobs, stream=None):
    """Fused decode step: each job is a dict with X ([M, K] fp32 / bf16), Wp,
    gamma and optional Y, Xq, d (allocated when absent; Xq / d only when the
    key is present with None meaning "allocate").  Returns the list of jobs
    with their output tensors filled in."""
    if not 1 <= len(jobs) <= BL_MAX_JOBS:
        raise ValueError(f"1..{BL_MAX_JOBS} jobs")
    arr = (GemvJob * len(jobs))()
    M = None
    out = []
    for i, j in enumerate(jobs):
        X = j["X"]
        if X.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("X must be float32 or bfloat16")
        _dev(X, X.dtype, "X")
        _dev(j["Wp"], torch.uint8, "Wp")
        _dev(j["gamma"], torch.float32, "gamma")
        m, K = X.shape
        if M is None:
            M = m
        elif m != M:
            raise ValueError("all jobs must have the same number of tokens")
        N = j["Wp"].shape[0]
        if j["Wp"].shape[1] * 4 != K:
            raise ValueError("Wp must be [N, K/4]")
        dev = X.device
        r = dict(j)
        r["Y"] = _dev(j.get("Y"), torch.float32, "Y") if j.get("Y") is not None else \
            torch.empty((M, N), dtype=torch.float32, device=dev)
        if "Xq" in j:
            r["Xq"] = j["Xq"] if j["Xq"] is not None else torch.empty((M, K), dtype=torch.int8,
                                                                        device=dev)
            _dev(r["Xq"], torch.int8, "Xq")
        if "d" in j:
            r["d"] = j["d"] if j["d"] is not None else torch.empty((M,), dtype=torch.float32,
                                                                     device=dev)
            _dev(r["d"], torch.float32, "d")
        arr[i] = GemvJob(X.data_ptr(), j["Wp"].data_ptr(), j["gamma"].data_ptr(),
                         r["Y"].data_ptr(), r["Xq"].data_ptr() if r.get("Xq") is not None else None,
                         r["d"].data_ptr() if r.get("d") is not None else None, N, K,
                         BL_BF16 if X.dtype == torch.bfloat16 else BL_F32, 0)
        out.append(r)
    _check("bitlinear_gemv_fused", load().bitlinear_gemv_fused(arr, len(jobs), M, _stream(stream)))
    return out


def bitlinear_ffn_relu2(Xq, d, Wg, gamma_g, Wu, gamma_u, Wd, gamma_d, norm_w=None, eps=1e-5,
                        Y=None, Hq=None, dh=None, want_debug=False, ws=None, stream=None):
    """ReLU^2 FFN tail; returns Y [M, N] (and Hq int8 [M, F], dh fp32 [M] with
    want_debug)."""
    _dev(Xq, torch.int8, "Xq")
    _dev(d, torch.float32, "d")
    for t, n in ((Wg, "Wg"), (Wd, "Wd")):
        _dev(t, torch.uint8, n)
    _dev(Wu, torch.uint8, "Wu")
    _dev(gamma_g, torch.float32, "gamma_g")
    _dev(gamma_d, torch.float32, "gamma_d")
    _dev(gamma_u, torch.float32, "gamma_u")
    _dev(norm_w, torch.float32, "norm_w")
    M, K = Xq.shape
    F = Wg.shape[0]
    N = Wd.shape[0]
    if Wg.shape[1] * 4 != K or (Wu is not None and tuple(Wu.shape) != tuple(Wg.shape)) \
            or Wd.shape[1] * 4 != F:
        raise ValueError("weight shapes do not chain: Wg/Wu [F, K/4], Wd [N, F/4]")
    dev = Xq.device
    Y = _dev(Y, torch.float32, "Y") if Y is not None else torch.empty(
        (M, N), dtype=torch.float32, device=dev)
    if want_debug:
        Hq = Hq if Hq is not None else torch.empty((M, F), dtype=torch.int8, device=dev)
        dh = dh if dh is not None else torch.empty((M,), dtype=torch.float32, device=dev)
    _dev(Hq, torch.int8, "Hq")
    _dev(dh, torch.float32, "dh")
    need = workspace_bytes(BL_OP_FFN_RELU2, M, N, K, F)
    if ws is None:
        ws = torch.empty((max(need, 16),), dtype=torch.uint8, device=dev)
    _check("bitlinear_ffn_relu2", load().bitlinear_ffn_relu2(
        _ptr(Xq), _ptr(d), M, K, F, _ptr(Wg), _ptr(gamma_g), _ptr(Wu), _ptr(gamma_u),
        _ptr(norm_w), float(eps), _ptr(Wd), _ptr(gamma_d), N, _ptr(Y), _ptr(Hq), _ptr(dh),
        _ptr(ws), ws.numel(), _stream(stream)))
    return (Y, Hq, dh) if want_debug else Y


def bitlinear_decode_stack(layers, x, H, KV, F, D, eps=1e-5, trace=False, ws=None, stream=None,
                           path=BL_STACK_AUTO, wait_us=0):
    """One decode token through len(layers) layers; x fp32 [H] is updated in
    place.  Each layer is a dict with packed weights Wq..Wd (uint8), gammas
    gq..gd (fp32 [1]) and optional ffn_norm (fp32 [F]).  With trace=True
    returns the per-layer trace [n_layers, 5 H + 2 KV] (x_in, q, k, v, o,
    x_mid, y).  path: BL_STACK_AUTO, BL_STACK_LAUNCHES or BL_STACK_PERSISTENT;
    wait_us: limit of each wait of the persistent path (0 = 1 s)."""
    _dev(x, torch.float32, "x")
    n = len(layers)
    arr = (Layer * max(1, n))()
    for i, L in enumerate(layers):
        vals = []
        for k in LAYER_WEIGHTS:
            vals.append(_dev(L[k], torch.uint8, k).data_ptr())
        for k in LAYER_GAMMAS:
            vals.append(_dev(L[k], torch.float32, k).data_ptr())
        nw = L.get("ffn_norm")
        vals.append(_dev(nw, torch.float32, "ffn_norm").data_ptr() if nw is not None else None)
        arr[i] = Layer(*vals)
    dims = StackDims(H, KV, F, D, float(eps), int(path), int(wait_us), 0)
    tr = None
    if trace:
        tr = torch.empty((n, 5 * H + 2 * KV), dtype=torch.float32, device=x.device)
    need = workspace_bytes(BL_OP_DECODE_STACK, 1, H, KV, F)
    if ws is None:
        ws = torch.empty((max(need, 16),), dtype=torch.uint8, device=x.device)
    _check("bitlinear_decode_stack", load().bitlinear_decode_stack(
        arr, n, ctypes.byref(dims), _ptr(x), _ptr(tr), _ptr(ws), ws.numel(), _stream(stream)))
    return tr


def bitlinear_decode_stack_status(ws, H, KV, F, D, path=BL_STACK_AUTO):
    """Status of the last bitlinear_decode_stack call on workspace ws (uint8
    device tensor): 0 = it ran to the end, 1 = a wait gave up (x holds NaN).
    Blocking read; call it once that call's work has finished."""
    _dev(ws, torch.uint8, "ws")
    dims = StackDims(H, KV, F, D, 0.0, int(path), 0, 0)
    out = ctypes.c_int32(-1)
    _check("bitlinear_decode_stack_status", load().bitlinear_decode_stack_status(
        _ptr(ws), ws.numel(), ctypes.byref(dims), ctypes.byref(out)))
    return int(out.value)


def bitlinear_backward_input(dY, Wp, gamma, dX=None, ws=None, stream=None):
    """Straight-through gradient of the layer input: dX [M, K] = gamma (dY . Wq)
    for dY fp32 [M, N] and the forward's packed Wp [N, K/4], gamma [1]."""
    _dev(dY, torch.float32, "dY")
    _dev(Wp, torch.uint8, "Wp")
    _dev(gamma, torch.float32, "gamma")
    M, N = dY.shape
    if Wp.dim() != 2 or Wp.shape[0] != N:
        raise ValueError(f"Wp must be [N, K/4] with N = {N}, got {tuple(Wp.shape)}")
    K = Wp.shape[1] * 4
    dX = _dev(dX, torch.float32, "dX") if dX is not None else torch.empty(
        (M, K), dtype=torch.float32, device=dY.device)
    if tuple(dX.shape) != (M, K):
        raise ValueError(f"dX must be [{M}, {K}]")
    need = workspace_bytes(BL_OP_BACKWARD_INPUT, M, N, K, 0)
    if ws is None:
        ws = torch.empty((max(need, 16),), dtype=torch.uint8, device=dY.device)
    _check("bitlinear_backward_input", load().bitlinear_backward_input(
        _ptr(dY), M, N, _ptr(Wp), _ptr(gamma), K, _ptr(dX), _ptr(ws), ws.numel(), _stream(stream)))
    return dX


def bitlinear_backward_weight(dY, Xq, d, dW=None, ws=None, stream=None):
    """Straight-through gradient of the latent weights: dW [N, K] =
    (dY o d)^T . Xq for dY fp32 [M, N] and the forward's Xq int8 [M, K], d [M]."""
    _dev(dY, torch.float32, "dY")
    _dev(Xq, torch.int8, "Xq")
    _dev(d, torch.float32, "d")
    M, N = dY.shape
    if Xq.dim() != 2 or Xq.shape[0] != M or tuple(d.shape) != (M,):
        raise ValueError(f"Xq must be [{M}, K] and d [{M}]")
    K = Xq.shape[1]
    dW = _dev(dW, torch.float32, "dW") if dW is not None else torch.empty(
        (N, K), dtype=torch.float32, device=dY.device)
    if tuple(dW.shape) != (N, K):
        raise ValueError(f"dW must be [{N}, {K}]")
    need = workspace_bytes(BL_OP_BACKWARD_WEIGHT, M, N, K, 0)
    if ws is None:
        ws = torch.empty((max(need, 16),), dtype=torch.uint8, device=dY.device)
    _check("bitlinear_backward_weight", load().bitlinear_backward_weight(
        _ptr(dY), M, N, _ptr(Xq), _ptr(d), K, _ptr(dW), _ptr(ws), ws.numel(), _stream(stream)))
    return dW


# The calls below run on their tensors' device whichever is current, and their
# outputs and workspaces are allocated on the stream that the kernels run on.

_DTYPES = {torch.float32: BL_F32, torch.bfloat16: BL_BF16}


def _at(t, dtype, dev, shape, name):
    """Address of tensor t, which must be contiguous, of dtype, on GPU dev (its
    number: comparing devices takes twice the time), of shape."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == shape \
            and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _rows(t, dim, name):
    """GPU, bl_dtype, address and shape of a contiguous fp32 / bf16 tensor
    with dim dimensions on the GPU."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    shape = t.shape
    if len(shape) != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {list(shape)}")
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be float32 or bfloat16")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.get_device(), dt, t.data_ptr(), shape


class _Nowhere:
    """A context that changes nothing (contextlib's costs 0.2 us a call)."""
    __slots__ = ()

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_HERE = _Nowhere()


def _where(dev, stream):
    """The HIP stream to run on, and the context to allocate and launch in."""
    if stream is None:
        # the handle alone: a Stream object costs 1.8 us, as much as a small launch
        return (torch._C._cuda_getCurrentRawStream(dev),
                _HERE if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev))
    if stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{dev}")
    return stream.cuda_stream, torch.cuda.stream(stream)


def kv8_cache(n_blocks, KVH, T=64, D=128, device="cuda"):
    """A zeroed Kv8Cache."""
    def z(*shape, dtype):
        return torch.zeros(shape, dtype=dtype, device=device)
    return Kv8Cache(z(n_blocks, KVH, T, D, dtype=torch.int8), z(n_blocks, KVH, D, T, dtype=torch.int8),
                    z(n_blocks, KVH, dtype=torch.float32), z(n_blocks, KVH, dtype=torch.float32))


def _kv8(cache, dev):
    K, V, sk, sv = cache
    if not isinstance(K, torch.Tensor) or K.dim() != 4:
        raise ValueError("the cache's K must be a tensor [n_blocks, KVH, T, D]")
    nb, KVH, T, D = K.shape
    return Kv8(_at(K, torch.int8, dev, (nb, KVH, T, D), "cache K"),
               _at(V, torch.int8, dev, (nb, KVH, D, T), "cache V"),
               _at(sk, torch.float32, dev, (nb, KVH), "cache sk"),
               _at(sv, torch.float32, dev, (nb, KVH), "cache sv"), nb, KVH, T, D)


def kv4_cache(n_blocks, KVH, T=64, D=128, device="cuda"):
    """A zeroed Kv4Cache."""
    def z(*shape, dtype=torch.uint8):
        return torch.zeros(shape, dtype=dtype, device=device)
    return Kv4Cache(z(n_blocks, KVH, T, D // 2), z(n_blocks, KVH, T // 16, D, 8),
                    z(n_blocks, KVH, T, 2, dtype=torch.float16), z(n_blocks, KVH, T, 2, dtype=torch.float16))


def _kv4(cache, dev):
    K, V, zk, zv = cache
    if not isinstance(K, torch.Tensor) or K.dim() != 4:
        raise ValueError("the cache's K must be a tensor [n_blocks, KVH, T, D/2]")
    nb, KVH, T, half = K.shape
    return Kv4(_at(K, torch.uint8, dev, (nb, KVH, T, half), "cache K"),
               _at(V, torch.uint8, dev, (nb, KVH, T // 16, 2 * half, 8), "cache V"),
               _at(zk, torch.float16, dev, (nb, KVH, T, 2), "cache zk"),
               _at(zv, torch.float16, dev, (nb, KVH, T, 2), "cache zv"), nb, KVH, T, 2 * half)


def _rope(rope, dev):
    cos_sin, interleaved = rope
    if not isinstance(cos_sin, torch.Tensor) or cos_sin.dim() != 2:
        raise ValueError("the rotation's cos_sin must be a tensor [positions, rot]")
    rows, rot = cos_sin.shape
    return BlRope(_at(cos_sin, torch.float32, dev, (rows, rot), "cos_sin"), rows, rot, bool(interleaved), 0)


def _seqs(q_start, lengths, table, dev):
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a tensor [B, max_blocks]")
    B, nb = table.shape
    return (_at(q_start, torch.int32, dev, (B + 1,), "q_start"),
            _at(lengths, torch.int32, dev, (B,), "lengths"),
            _at(table, torch.int32, dev, (B, nb), "table"), B, nb)


def bitlinear_kv8_append(k, v, q_start, lengths, table, cache, stream=None):
    """The new tokens' rows k, v [n_tok, KVH, D] (fp32 or bf16) into the cache
    (Kv8Cache, updated in place).  int32 on the GPU: q_start [B + 1], lengths
    [B] (with the new tokens), table [B, max_blocks]."""
    if stream is None and _calls is not None:
        if _calls.append(8, k, v, q_start, lengths, table, cache, None, None, None) is not NotImplemented:
            return
    dev, dt, kp, shape = _rows(k, 3, "k")
    c = _kv8(cache, dev)
    n = shape[0]
    if shape[1] != c.KVH or shape[2] != c.D:
        raise ValueError(f"k must be [n_tok, {c.KVH}, {c.D}], got {list(shape)}")
    vp = _at(v, k.dtype, dev, shape, "v")
    meta = _seqs(q_start, lengths, table, dev)
    handle, context = _where(dev, stream)
    with context:
        st = load().bitlinear_kv8_append(kp, vp, dt, n, *meta, c, handle)
    if st:
        _check("bitlinear_kv8_append", st)


def _append_turned(call, device_cache, k, v, q_start, lengths, table, cache, rope, q, q_out, stream):
    dev, dt, kp, shape = _rows(k, 3, "k")
    c = device_cache(cache, dev)
    n = shape[0]
    if shape[1] != c.KVH or shape[2] != c.D:
        raise ValueError(f"k must be [n_tok, {c.KVH}, {c.D}], got {list(shape)}")
    vp = _at(v, k.dtype, dev, shape, "v")
    meta = _seqs(q_start, lengths, table, dev)
    r = None if rope is None else _rope(rope, dev)
    qp, op, QH = None, None, 0
    if q is not None:
        if r is None:
            raise ValueError("q is rotated with the keys: without rope there is nothing to do with it")
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError(f"q must be a tensor [{n}, QH, {c.D}]")
        QH = q.shape[1]
        qp = _at(q, k.dtype, dev, (n, QH, c.D), "q")
    if q_out is not None:
        if q is None:
            raise ValueError("q_out without q")
        op = _at(q_out, k.dtype, dev, (n, QH, c.D), "q_out")
    handle, context = _where(dev, stream)
    with context:
        if q is not None and q_out is None:
            q_out = torch.empty_like(q)
            op = q_out.data_ptr()
        st = getattr(load(), call)(kp, vp, qp, op, dt, n, QH, *meta, c, r, handle)
    if st:
        _check(call, st)
    return q_out


def bitlinear_kv8_append_rope(k, v, q_start, lengths, table, cache, rope, q=None, q_out=None, stream=None):
    """bitlinear_kv8_append of the keys rotated by their tokens' positions (rope:
    Rope, a row of cos_sin for each of the table's positions at least).  Returns q
    [n_tok, QH, D] rotated the same way, in q_out if given (which may be q), None
    without q; its rows of no sequence are left as they are."""
    if rope is None:
        raise ValueError("bitlinear_kv8_append_rope without rope")
    if stream is None and _calls is not None:
        r = _calls.append(8, k, v, q_start, lengths, table, cache, rope, q, q_out)
        if r is not NotImplemented:
            return r
    return _append_turned("bitlinear_kv8_append_rope", _kv8, k, v, q_start, lengths, table, cache, rope, q,
                          q_out, stream)


def bitlinear_kv4_append(k, v, q_start, lengths, table, cache, rope=None, q=None, q_out=None, stream=None):
    """The new tokens' rows k, v [n_tok, KVH, D] (fp32 or bf16) into the 4-bit cache
    (Kv4Cache, updated in place), as they are or, with rope, keys and q rotated as
    by bitlinear_kv8_append_rope (which see for q and what is returned)."""
    if stream is None and _calls is not None:
        r = _calls.append(4, k, v, q_start, lengths, table, cache, rope, q, q_out)
        if r is not NotImplemented:
            return r
    return _append_turned("bitlinear_kv4_append", _kv4, k, v, q_start, lengths, table, cache, rope, q, q_out,
                          stream)


def _read(call, device_cache, q_start, lengths, table, cache, n_tok, dtype, k, v, stream):
    K = cache[0]
    if not isinstance(K, torch.Tensor) or not K.is_cuda:
        raise TypeError("the cache's K must be a CUDA (HIP) tensor")
    dev = K.get_device()
    c = device_cache(cache, dev)
    meta = _seqs(q_start, lengths, table, dev)
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float32 or bfloat16")
    if n_tok < 0:
        raise ValueError(f"n_tok must not be negative, got {n_tok}")
    shape = (n_tok, c.KVH, c.D)
    for t, name in ((k, "k"), (v, "v")):
        if t is not None:
            _at(t, dtype, dev, shape, name)
    handle, context = _where(dev, stream)
    with context:
        if k is None:
            k = torch.empty(shape, dtype=dtype, device=K.device)
        if v is None:
            v = torch.empty(shape, dtype=dtype, device=K.device)
        st = getattr(load(), call)(c, *meta, n_tok, k.data_ptr(), v.data_ptr(), _DTYPES[dtype], handle)
    if st:
        _check(call, st)
    return k, v


def bitlinear_kv8_read(q_start, lengths, table, cache, n_tok, dtype=torch.float32, k=None, v=None, stream=None):
    """The cached tokens of rows 0 .. n_tok - 1 of a call as values, k and v
    [n_tok, KVH, D] of dtype (fp32 or bf16): the n_b rows of sequence b are its
    last n_b tokens.  q_start, lengths, table as for bitlinear_kv8_append."""
    if stream is None and _calls is not None:
        r = _calls.read(8, q_start, lengths, table, cache, n_tok, dtype, k, v)
        if r is not NotImplemented:
            return r
    return _read("bitlinear_kv8_read", _kv8, q_start, lengths, table, cache, n_tok, dtype, k, v, stream)


def bitlinear_kv4_read(q_start, lengths, table, cache, n_tok, dtype=torch.float32, k=None, v=None, stream=None):
    """bitlinear_kv8_read of a 4-bit cache."""
    if stream is None and _calls is not None:
        r = _calls.read(4, q_start, lengths, table, cache, n_tok, dtype, k, v)
        if r is not NotImplemented:
            return r
    return _read("bitlinear_kv4_read", _kv4, q_start, lengths, table, cache, n_tok, dtype, k, v, stream)


def bitlinear_kv8_attention(q, q_start, lengths, table, cache, scale=None, out=None, ws=None,
                            stream=None):
    """Causal attention of q [n_tok, QH, D] (fp32 or bf16) over the cache:
    out [n_tok, QH, D].  scale defaults to D ** -0.5; q_start, lengths, table
    as for bitlinear_kv8_append.  Rows of no sequence are left as they are.
    out may not overlap q."""
    if stream is None and _calls is not None:
        r = _calls.attention(8, q, q_start, lengths, table, cache, scale, out, ws)
        if r is not NotImplemented:
            return r
    dev, dt, qp, (n, QH, D) = _rows(q, 3, "q")
    c = _kv8(cache, dev)
    if D != c.D:
        raise ValueError(f"q must be [n_tok, QH, {c.D}], got {list(q.shape)}")
    meta = _seqs(q_start, lengths, table, dev)
    if out is not None:
        _at(out, q.dtype, dev, (n, QH, D), "out")
    wp = size = 0
    if ws is not None:
        size = ws.numel()
        wp = _at(ws, torch.uint8, dev, (size,), "ws")
    lib = load()
    handle, context = _where(dev, stream)
    with context:
        if ws is None:
            size = lib.bitlinear_kv8_attention_ws_bytes(n, QH, meta[3], meta[4], c.KVH, c.T, D)
            if size:
                ws = torch.empty((size,), dtype=torch.uint8, device=dev)
                wp = ws.data_ptr()
        if out is None:
            out = torch.empty_like(q)
        st = lib.bitlinear_kv8_attention(
            qp, dt, n, QH, *meta, c, D ** -0.5 if scale is None else scale, out.data_ptr(), wp, size,
            handle)
    if st:
        _check("bitlinear_kv8_attention", st)
    return out


def bitlinear_kv4_attention(q, q_start, lengths, table, cache, scale=None, out=None, ws=None,
                            stream=None):
    """bitlinear_kv8_attention over a 4-bit cache (Kv4Cache)."""
    if stream is None and _calls is not None:
        r = _calls.attention(4, q, q_start, lengths, table, cache, scale, out, ws)
        if r is not NotImplemented:
            return r
    dev, dt, qp, (n, QH, D) = _rows(q, 3, "q")
    c = _kv4(cache, dev)
    if D != c.D:
        raise ValueError(f"q must be [n_tok, QH, {c.D}], got {list(q.shape)}")
    meta = _seqs(q_start, lengths, table, dev)
    if out is not None:
        _at(out, q.dtype, dev, (n, QH, D), "out")
    wp = size = 0
    if ws is not None:
        size = ws.numel()
        wp = _at(ws, torch.uint8, dev, (size,), "ws")
    lib = load()
    handle, context = _where(dev, stream)
    with context:
        if ws is None:
            size = lib.bitlinear_kv4_attention_ws_bytes(n, QH, meta[3], meta[4], c.KVH, c.T, D)
            if size:
                ws = torch.empty((size,), dtype=torch.uint8, device=dev)
                wp = ws.data_ptr()
        if out is None:
            out = torch.empty_like(q)
        st = lib.bitlinear_kv4_attention(
            qp, dt, n, QH, *meta, c, D ** -0.5 if scale is None else scale, out.data_ptr(), wp, size,
            handle)
    if st:
        _check("bitlinear_kv4_attention", st)
    return out


def _stack_cached(call, ws_call, kind, device_cache, layers, caches, x, q_start, lengths, table, H, KV, F, D, rope,
                  eps, scale, trace, ws, stream):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA (HIP) tensor")
    dev, n = x.get_device(), len(layers)
    if len(caches) != n:
        raise ValueError(f"{n} layers and {len(caches)} caches")
    xp = _at(x, torch.float32, dev, (H,), "x")
    arr, kvs = (Layer * max(1, n))(), (kind * max(1, n))()
    wide = {"Wd": F}
    rows = {"Wq": H, "Wk": KV, "Wv": KV, "Wo": H, "Wg": F, "Wu": F, "Wd": H}
    for i, L in enumerate(layers):
        vals = [_at(L[k], torch.uint8, dev, (rows[k], wide.get(k, H) // 4), k) for k in LAYER_WEIGHTS]
        vals += [_at(L[k], torch.float32, dev, (1,), k) for k in LAYER_GAMMAS]
        nw = L.get("ffn_norm")
        arr[i] = Layer(*vals, None if nw is None else _at(nw, torch.float32, dev, (F,), "ffn_norm"))
        kvs[i] = device_cache(caches[i], dev)
    qp, lp, tp, B, nb = _seqs(q_start, lengths, table, dev)
    if B != 1:
        raise ValueError(f"one sequence, got {B}")
    turn = () if call == "bitlinear_decode_stack_kv" else (None if rope is None else _rope(rope, dev),)
    dims = StackDims(H, KV, F, D, float(eps), BL_STACK_AUTO, 0, 0)
    lib = load()
    handle, context = _where(dev, stream)
    with context:
        tr = torch.empty((n, 5 * H + 2 * KV), dtype=torch.float32, device=dev) if trace else None
        if ws is None:
            need = getattr(lib, ws_call)(ctypes.byref(dims), kvs[0].T if n else 64, nb)
            ws = torch.empty((max(need, 16),), dtype=torch.uint8, device=dev)
        st = getattr(lib, call)(
            arr, kvs, n, ctypes.byref(dims), qp, lp, tp, nb, *turn, D ** -0.5 if scale is None else scale, xp,
            None if tr is None else tr.data_ptr(), _at(ws, torch.uint8, dev, (ws.numel(),), "ws"),
            ws.numel(), handle)
    if st:
        _check(call, st)
    return tr


def bitlinear_decode_stack_kv(layers, caches, x, q_start, lengths, table, H, KV, F, D, eps=1e-5,
                              scale=None, trace=False, ws=None, stream=None):
    """bitlinear_decode_stack with the attention over 8-bit caches: one token of
    one sequence through len(layers) layers, each appending to its Kv8Cache and
    attending over it, q and k as their BitLinears give them (not rotated).
    q_start int32 [2] = [0, 1], lengths int32 [1] (with the
    new token) and table int32 [1, max_blocks] on the GPU.  x fp32 [H] is
    updated in place; scale defaults to D ** -0.5."""
    return _stack_cached("bitlinear_decode_stack_kv", "bitlinear_decode_stack_kv_ws_bytes", Kv8, _kv8, layers,
                         caches, x, q_start, lengths, table, H, KV, F, D, None, eps, scale, trace, ws, stream)


def bitlinear_decode_stack_kv_rope(layers, caches, x, q_start, lengths, table, H, KV, F, D, rope, eps=1e-5,
                                   scale=None, trace=False, ws=None, stream=None):
    """bitlinear_decode_stack_kv with q and k rotated by the token's position (rope:
    Rope, the same in all layers); the trace holds them as their BitLinears do."""
    if rope is None:
        raise ValueError("bitlinear_decode_stack_kv_rope without rope")
    return _stack_cached("bitlinear_decode_stack_kv_rope", "bitlinear_decode_stack_kv_ws_bytes", Kv8, _kv8, layers,
                         caches, x, q_start, lengths, table, H, KV, F, D, rope, eps, scale, trace, ws, stream)


def bitlinear_decode_stack_kv4(layers, caches, x, q_start, lengths, table, H, KV, F, D, rope=None, eps=1e-5,
                               scale=None, trace=False, ws=None, stream=None):
    """bitlinear_decode_stack_kv over 4-bit caches (Kv4Cache), q and k rotated by the
    token's position where rope (Rope) is given."""
    return _stack_cached("bitlinear_decode_stack_kv4", "bitlinear_decode_stack_kv4_ws_bytes", Kv4, _kv4, layers,
                         caches, x, q_start, lengths, table, H, KV, F, D, rope, eps, scale, trace, ws, stream)


def quant_weight_absmax_i4(W, group=128, Wq4=None, s=None, stream=None):
    """W [N, K] (fp32 or bf16) -> (Wq4 uint8 [N, K/2] 4-bit codes, s bf16
    [N, K/group]); group 32, 64 or 128."""
    dev, dt, wp, (N, K) = _rows(W, 2, "W")
    if group not in (32, 64, 128) or K % group:
        raise ValueError(f"group must be 32, 64 or 128 and divide K = {K}, got {group}")
    if Wq4 is not None:
        _at(Wq4, torch.uint8, dev, (N, K // 2), "Wq4")
    if s is not None:
        _at(s, torch.bfloat16, dev, (N, K // group), "s")
    handle, context = _where(dev, stream)
    with context:
        if Wq4 is None:
            Wq4 = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
        if s is None:
            s = torch.empty((N, K // group), dtype=torch.bfloat16, device=dev)
        st = load().quant_weight_absmax_i4(wp, dt, N, K, group, Wq4.data_ptr(), s.data_ptr(), handle)
    if st:
        _check("quant_weight_absmax_i4", st)
    return Wq4, s


def _w4(Wq4, s):
    """(GPU, N, K, group, addresses) of 4-bit weights."""
    if not isinstance(Wq4, torch.Tensor) or not Wq4.is_cuda:
        raise TypeError("Wq4 must be a CUDA (HIP) tensor")
    packed = Wq4.shape
    if len(packed) != 2 or not isinstance(s, torch.Tensor) or s.dim() != 2:
        raise ValueError("Wq4 must be [N, K/2] and s [N, K/group]")
    N, K2 = packed
    groups, dev = s.shape[1], Wq4.get_device()
    group = 2 * K2 // groups if groups else 128
    if 2 * K2 != group * groups or group not in (32, 64, 128):
        raise ValueError(f"Wq4 {list(packed)} and s {list(s.shape)} do not make groups of 32, 64 or "
                         "128")
    return (dev, N, 2 * K2, group, _at(Wq4, torch.uint8, dev, packed, "Wq4"),
            _at(s, torch.bfloat16, dev, (N, groups), "s"))


def dequant_weight_i4(Wq4, s, dtype=torch.float32, W=None, stream=None):
    """The weights [N, K] of dtype (fp32 or bf16) that 4-bit codes stand for."""
    dev, N, K, group, wp, sp = _w4(Wq4, s)
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float32 or bfloat16")
    if W is not None:
        _at(W, dtype, dev, (N, K), "W")
    handle, context = _where(dev, stream)
    with context:
        if W is None:
            W = torch.empty((N, K), dtype=dtype, device=dev)
        st = load().dequant_weight_i4(wp, sp, N, K, group, W.data_ptr(), _DTYPES[dtype], handle)
    if st:
        _check("dequant_weight_i4", st)
    return W


def bitlinear_gemv_w4(X, Wq4, s, Y=None, stream=None):
    """Y [M, N] fp32 = X W^T for X [M, K] (fp32 or bf16), 1 <= M <= 16, and
    4-bit weights (Wq4 [N, K/2], s [N, K/group])."""
    dev, dt, xp, (M, cols) = _rows(X, 2, "X")
    wdev, N, K, group, wp, sp = _w4(Wq4, s)
    if wdev != dev:
        raise ValueError(f"Wq4 is on cuda:{wdev}, not on cuda:{dev}")
    if cols != K:
        raise ValueError(f"X must be [M, {K}], got {[M, cols]}")
    if Y is not None:
        _at(Y, torch.float32, dev, (M, N), "Y")
    handle, context = _where(dev, stream)
    with context:
        if Y is None:
            Y = torch.empty((M, N), dtype=torch.float32, device=dev)
        st = load().bitlinear_gemv_w4(xp, dt, M, wp, sp, N, K, group, Y.data_ptr(), handle)
    if st:
        _check("bitlinear_gemv_w4", st)
    return Y
