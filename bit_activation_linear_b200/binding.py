"""Python binding of libbitnet_b200.so: argument marshalling only.

Every function here has the name of the C entry point it calls (include/bitnet.h), takes torch
CUDA tensors, checks dtype / device / contiguity, allocates outputs and workspace with torch
(the library itself never allocates) and passes raw pointers plus the current torch stream.  All
arithmetic runs in the library's kernels; there is no fallback of any kind: if the shared
library is missing or cannot load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbitnet_b200.so")
_lock = threading.Lock()
_lib = None

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE = 0, -1, -2, -3, -4, -5
ACT_RELU2, ACT_SWIGLU = 1, 2  # bitnet_activation
PATH_DECODE, PATH_TC, PATH_TC_SKINNY, PATH_TC_TMEM = 1, 2, 3, 4  # bitnet_product_path
QUANT_PLAIN, QUANT_FWHT, QUANT_HADAMARD_TC = 1, 2, 3  # bitnet_quant_path


class BitnetError(RuntimeError):
    """A non-zero status from the library, with its text and the library's detail message."""

    def __init__(self, status: int, where: str):
        lib = load_library()
        self.status = status
        text = lib.bitnet_status_string(status).decode()
        detail = lib.bitnet_last_error().decode()
        super().__init__(f"{where}: {text} ({status}): {detail}")


class _CKvCache(ctypes.Structure):  # bitnet_kv_cache
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("scale_tokens", ctypes.c_int32)]


class _CKvBatch(ctypes.Structure):  # bitnet_kv_batch
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("batch", ctypes.c_int64),
                ("max_pages", ctypes.c_int64), ("tokens", ctypes.c_int64)]


_SIGS = {
    "bitnet_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "bitnet_last_error": (ctypes.c_char_p, []),
    "bitnet_launch_count": (ctypes.c_uint64, []),
    "bitnet_packed_weight_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "bitnet_weight_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "bitnet_quantize_pack_weights": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                                    ctypes.c_int64, ctypes.c_void_p,
                                                    ctypes.c_void_p, ctypes.c_void_p,
                                                    ctypes.c_size_t, ctypes.c_void_p]),
    "bitnet_quantize_pack_weights_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                                            ctypes.c_int64, ctypes.c_void_p,
                                                            ctypes.c_void_p, ctypes.c_void_p]),
    "bitnet_act_codes_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "bitnet_act_quant": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "bitnet_fwht_f32": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                       ctypes.c_void_p, ctypes.c_void_p]),
    "bitnet_ternary_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "bitnet_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                 ctypes.c_int]),
    "bitnet_product_plan": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                           ctypes.POINTER(ctypes.c_int)]),
    "bitnet_act_quant_plan": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                             ctypes.POINTER(ctypes.c_int)]),
    "bitnet_bitlinear_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                                ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                                ctypes.c_size_t, ctypes.c_void_p]),
    "bitnet_hbitlinear_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                                 ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                                 ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.c_size_t, ctypes.c_void_p]),
    "bitnet_act_quant_norm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                             ctypes.c_void_p, ctypes.c_float, ctypes.c_int,
                                             ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_void_p]),
    "bitnet_norm_transform_f32": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                                 ctypes.c_void_p, ctypes.c_float, ctypes.c_int,
                                                 ctypes.c_void_p, ctypes.c_void_p]),
    "bitnet_norm_bitlinear_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                                     ctypes.c_int64, ctypes.c_void_p,
                                                     ctypes.c_float, ctypes.c_int, ctypes.c_void_p,
                                                     ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                                     ctypes.c_void_p, ctypes.c_void_p,
                                                     ctypes.c_size_t, ctypes.c_void_p]),
    "bitnet_ternary_gemm_act": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                               ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                               ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "bitnet_bitlinear_forward_act": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                                    ctypes.c_int64, ctypes.c_void_p,
                                                    ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                                    ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                                    ctypes.c_void_p, ctypes.c_size_t,
                                                    ctypes.c_void_p]),
    "bitnet_weight_workspace_bytes_rotated": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "bitnet_quantize_pack_weights_rotated": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                                            ctypes.c_int64, ctypes.c_void_p,
                                                            ctypes.c_void_p, ctypes.c_void_p,
                                                            ctypes.c_size_t, ctypes.c_void_p]),
    "bitnet_act_quant_absmax4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                                 ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.c_void_p, ctypes.c_void_p]),
    "bitnet_bitlinear_forward_absmax4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                                         ctypes.c_int64, ctypes.c_void_p,
                                                         ctypes.c_void_p, ctypes.c_int64,
                                                         ctypes.c_int, ctypes.c_void_p,
                                                         ctypes.c_void_p, ctypes.c_size_t,
                                                         ctypes.c_void_p]),
    "bitnet_base3_weight_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "bitnet_quantize_pack_weights_base3": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                                          ctypes.c_int64, ctypes.c_void_p,
                                                          ctypes.c_void_p, ctypes.c_void_p,
                                                          ctypes.c_size_t, ctypes.c_void_p]),
    "bitnet_ternary_gemv_base3": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                                 ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                                 ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.c_void_p]),
    "bitnet_bitlinear_forward_base3": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64,
                                                      ctypes.c_int64, ctypes.c_void_p,
                                                      ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                                      ctypes.c_int, ctypes.c_void_p,
                                                      ctypes.c_void_p, ctypes.c_size_t,
                                                      ctypes.c_void_p]),
    "bitnet_state_codes_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "bitnet_quant_states": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p]),
    "bitnet_act_quant_residual_norm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p,
                                                      ctypes.c_int64, ctypes.c_int64,
                                                      ctypes.c_void_p, ctypes.c_float,
                                                      ctypes.c_int, ctypes.c_void_p,
                                                      ctypes.c_void_p, ctypes.c_void_p,
                                                      ctypes.c_void_p, ctypes.c_void_p]),
    "bitnet_residual_norm_bitlinear_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p,
                                                              ctypes.c_int64, ctypes.c_int64,
                                                              ctypes.c_void_p, ctypes.c_float,
                                                              ctypes.c_void_p, ctypes.c_void_p,
                                                              ctypes.c_int64, ctypes.c_int,
                                                              ctypes.c_void_p, ctypes.c_void_p,
                                                              ctypes.c_void_p, ctypes.c_size_t,
                                                              ctypes.c_void_p]),
    "bitnet_kv_cache_append": (ctypes.c_int, [ctypes.POINTER(_CKvCache),
                                              ctypes.POINTER(_CKvBatch), ctypes.c_void_p,
                                              ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                              ctypes.c_void_p]),
    "bitnet_kv_cache_read": (ctypes.c_int, [ctypes.POINTER(_CKvCache), ctypes.POINTER(_CKvBatch),
                                            ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                            ctypes.c_int64, ctypes.c_void_p]),
    "bitnet_kv_attention_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(_CKvCache),
                                                              ctypes.POINTER(_CKvBatch),
                                                              ctypes.c_int64, ctypes.c_int64]),
    "bitnet_kv_attention": (ctypes.c_int, [ctypes.POINTER(_CKvCache), ctypes.POINTER(_CKvBatch),
                                           ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_int64, ctypes.c_float, ctypes.c_int,
                                           ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "bitnet_sync_status": (ctypes.c_int, [ctypes.c_void_p]),
    "bitnet_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_int64, ctypes.c_void_p]),
}

EXPORTED = tuple(_SIGS)


def load_library(path: str | None = None):
    """Load (once) and return the ctypes handle of libbitnet_b200.so.  Raises if it is absent."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(
                    f"{p} is missing: build it with `python -m bit_activation_linear_b200.build`"
                    " (nvcc, sm_100a). There is no fallback implementation.")
            lib = ctypes.CDLL(p)
            for name, (res, args) in _SIGS.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(t: torch.Tensor, name: str, dtype=None, dim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions")


def _nbytes_at_least(t: torch.Tensor, need: int, name: str):
    have = t.numel() * t.element_size()
    if have < need:
        raise ValueError(f"{name} holds {have} bytes, {need} needed")


def _rc(status: int, where: str):
    if status != OK:
        raise BitnetError(status, where)


def bitnet_launch_count() -> int:
    return int(load_library().bitnet_launch_count())


def bitnet_packed_weight_bytes(N: int, K: int) -> int:
    return int(load_library().bitnet_packed_weight_bytes(N, K))


def bitnet_weight_workspace_bytes(N: int, K: int) -> int:
    return int(load_library().bitnet_weight_workspace_bytes(N, K))


def bitnet_act_codes_bytes(M: int, K: int, act_bits: int) -> int:
    return int(load_library().bitnet_act_codes_bytes(M, K, act_bits))


def bitnet_workspace_bytes(M: int, K: int, N: int, act_bits: int) -> int:
    return int(load_library().bitnet_workspace_bytes(M, K, N, act_bits))


def bitnet_product_plan(M: int, K: int, N: int, act_bits: int):
    """(path, k_split) of the product of this shape on the current device (PATH_* values)."""
    path, split = ctypes.c_int(0), ctypes.c_int(0)
    _rc(load_library().bitnet_product_plan(M, K, N, int(act_bits), ctypes.byref(path),
                                           ctypes.byref(split)), "bitnet_product_plan")
    return path.value, split.value


def bitnet_act_quant_plan(K: int, hadamard: bool, norm: bool = False) -> int:
    """Which kernel quantises a K-wide row (QUANT_* values); host only, no device needed."""
    path = ctypes.c_int(0)
    _rc(load_library().bitnet_act_quant_plan(K, int(bool(hadamard)), int(bool(norm)),
                                             ctypes.byref(path)), "bitnet_act_quant_plan")
    return path.value


def bitnet_quantize_pack_weights(W: torch.Tensor, Wp: torch.Tensor | None = None,
                                 gamma: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                                 stream=None):
    """absmean-ternarise and pack bf16 W [N, K].  Returns (Wp uint8 [N, K/4], gamma float [1])."""
    L = load_library()
    _check(W, "W", torch.bfloat16, 2)
    N, K = W.shape
    if Wp is None:
        Wp = torch.empty((N, K // 4), dtype=torch.uint8, device=W.device)
    _nbytes_at_least(Wp, int(L.bitnet_packed_weight_bytes(N, K)), "Wp")
    if gamma is None:
        gamma = torch.empty(1, dtype=torch.float32, device=W.device)
    need = int(L.bitnet_weight_workspace_bytes(N, K))
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=W.device)
    _rc(L.bitnet_quantize_pack_weights(W.data_ptr(), N, K, Wp.data_ptr(), gamma.data_ptr(),
                                       ws.data_ptr(), ws.numel() * ws.element_size(),
                                       _stream(stream)), "bitnet_quantize_pack_weights")
    return Wp, gamma


def bitnet_quantize_pack_weights_noalloc(W: torch.Tensor, Wp: torch.Tensor | None = None,
                                         gamma: torch.Tensor | None = None, stream=None):
    """As bitnet_quantize_pack_weights, with the library's fixed device scratch instead of a
    workspace (for callers that cannot allocate device memory).  Returns (Wp, gamma)."""
    L = load_library()
    _check(W, "W", torch.bfloat16, 2)
    N, K = W.shape
    if Wp is None:
        Wp = torch.empty((N, K // 4), dtype=torch.uint8, device=W.device)
    _nbytes_at_least(Wp, int(L.bitnet_packed_weight_bytes(N, K)), "Wp")
    if gamma is None:
        gamma = torch.empty(1, dtype=torch.float32, device=W.device)
    _rc(L.bitnet_quantize_pack_weights_noalloc(W.data_ptr(), N, K, Wp.data_ptr(),
                                               gamma.data_ptr(), _stream(stream)),
        "bitnet_quantize_pack_weights_noalloc")
    return Wp, gamma


def bitnet_act_quant(X: torch.Tensor, hadamard: bool, act_bits: int, codes=None, scales=None,
                     rowsum=None, stream=None):
    """Per-token (Hadamard +) quantisation: absmax INT8 or absmean INT4.  Returns (codes,
    scales, rowsum)."""
    L = load_library()
    _check(X, "X", torch.bfloat16, 2)
    M, K = X.shape
    if codes is None:
        codes = torch.empty((M, K if act_bits == 8 else K // 2),
                            dtype=torch.int8 if act_bits == 8 else torch.uint8, device=X.device)
    if scales is None:
        scales = torch.empty(M, dtype=torch.float32, device=X.device)
    if rowsum is None:
        rowsum = torch.empty(M, dtype=torch.int32, device=X.device)
    _nbytes_at_least(codes, int(L.bitnet_act_codes_bytes(M, K, act_bits)), "codes")
    _nbytes_at_least(scales, 4 * M, "scales")
    _nbytes_at_least(rowsum, 4 * M, "rowsum")
    _rc(L.bitnet_act_quant(X.data_ptr(), M, K, int(bool(hadamard)), int(act_bits),
                           codes.data_ptr(), scales.data_ptr(), rowsum.data_ptr(),
                           _stream(stream)), "bitnet_act_quant")
    return codes, scales, rowsum


def bitnet_fwht_f32(X: torch.Tensor, Z: torch.Tensor | None = None, stream=None):
    """Z = H_K X / sqrt(K) per row in fp32 (debug / parity entry)."""
    L = load_library()
    _check(X, "X", torch.bfloat16, 2)
    M, K = X.shape
    if Z is None:
        Z = torch.empty((M, K), dtype=torch.float32, device=X.device)
    _rc(L.bitnet_fwht_f32(X.data_ptr(), M, K, Z.data_ptr(), _stream(stream)), "bitnet_fwht_f32")
    return Z


def bitnet_ternary_gemm(codes: torch.Tensor, scales: torch.Tensor, rowsum: torch.Tensor, K: int,
                        Wp: torch.Tensor, gamma: torch.Tensor, act_bits: int, want_acc=False,
                        want_y=True, acc=None, Y=None, stream=None):
    """Ternary x integer product (+ rescale).  Returns (acc int32 [M, N] or None, Y bf16 or None)."""
    L = load_library()
    for t, n in ((codes, "codes"), (scales, "scales"), (rowsum, "rowsum"), (Wp, "Wp"),
                 (gamma, "gamma")):
        _check(t, n)
    M = scales.numel()
    N = Wp.shape[0]
    _nbytes_at_least(codes, int(L.bitnet_act_codes_bytes(M, K, act_bits)), "codes")
    _nbytes_at_least(rowsum, 4 * M, "rowsum")
    _nbytes_at_least(Wp, int(L.bitnet_packed_weight_bytes(N, K)), "Wp")
    if want_acc and acc is None:
        acc = torch.empty((M, N), dtype=torch.int32, device=codes.device)
    if want_y and Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=codes.device)
    _rc(L.bitnet_ternary_gemm(codes.data_ptr(), scales.data_ptr(), rowsum.data_ptr(), M, K,
                              Wp.data_ptr(), gamma.data_ptr(), N, int(act_bits),
                              acc.data_ptr() if acc is not None else None,
                              Y.data_ptr() if Y is not None else None, _stream(stream)),
        "bitnet_ternary_gemm")
    return acc, Y


def _forward(fn_name: str, X, Wp, gamma, act_bits, Y, ws, stream):
    L = load_library()
    _check(X, "X", torch.bfloat16, 2)
    _check(Wp, "Wp")
    _check(gamma, "gamma", torch.float32)
    M, K = X.shape
    N = Wp.shape[0]
    _nbytes_at_least(Wp, int(L.bitnet_packed_weight_bytes(N, K)), "Wp")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _nbytes_at_least(Y, 2 * M * N, "Y")
    need = int(L.bitnet_workspace_bytes(M, K, N, act_bits))
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=X.device)
    _rc(getattr(L, fn_name)(X.data_ptr(), M, K, Wp.data_ptr(), gamma.data_ptr(), N,
                            int(act_bits), Y.data_ptr(), ws.data_ptr(),
                            ws.numel() * ws.element_size(), _stream(stream)), fn_name)
    return Y


def bitnet_bitlinear_forward(X, Wp, gamma, act_bits=8, Y=None, ws=None, stream=None):
    """Y = BitLinear(X) for bf16 X [M, K] and packed ternary Wp [N, K/4]."""
    return _forward("bitnet_bitlinear_forward", X, Wp, gamma, act_bits, Y, ws, stream)


def bitnet_hbitlinear_forward(X, Wp, gamma, act_bits=8, Y=None, ws=None, stream=None):
    """Y = H-BitLinear(X): online Hadamard transform, then BitLinear."""
    return _forward("bitnet_hbitlinear_forward", X, Wp, gamma, act_bits, Y, ws, stream)


def _act_cols(N: int, activation: int) -> int:
    return N // 2 if activation == ACT_SWIGLU else N


def bitnet_ternary_gemm_act(codes, scales, rowsum, K: int, Wp, gamma, act_bits: int,
                            activation: int, Y=None, stream=None):
    """Y = activation(rescaled product): squared ReLU [M, N] or SwiGLU over interleaved gate/up
    features [M, N/2] (bf16)."""
    L = load_library()
    for t, n in ((codes, "codes"), (scales, "scales"), (rowsum, "rowsum"), (Wp, "Wp"),
                 (gamma, "gamma")):
        _check(t, n)
    M = scales.numel()
    N = Wp.shape[0]
    _nbytes_at_least(codes, int(L.bitnet_act_codes_bytes(M, K, act_bits)), "codes")
    _nbytes_at_least(Wp, int(L.bitnet_packed_weight_bytes(N, K)), "Wp")
    if Y is None:
        Y = torch.empty((M, _act_cols(N, activation)), dtype=torch.bfloat16, device=Wp.device)
    _nbytes_at_least(Y, 2 * M * _act_cols(N, activation), "Y")
    _rc(L.bitnet_ternary_gemm_act(codes.data_ptr(), scales.data_ptr(), rowsum.data_ptr(), M, K,
                                  Wp.data_ptr(), gamma.data_ptr(), N, int(act_bits),
                                  int(activation), Y.data_ptr(), _stream(stream)),
        "bitnet_ternary_gemm_act")
    return Y


def bitnet_bitlinear_forward_act(X, Wp, gamma, act_bits, hadamard, activation, Y=None, ws=None,
                                 stream=None):
    """Y = activation((H-)BitLinear(X)) with the activation in the product's epilogue."""
    L = load_library()
    _check(X, "X", torch.bfloat16, 2)
    _check(Wp, "Wp")
    _check(gamma, "gamma", torch.float32)
    M, K = X.shape
    N = Wp.shape[0]
    _nbytes_at_least(Wp, int(L.bitnet_packed_weight_bytes(N, K)), "Wp")
    if Y is None:
        Y = torch.empty((M, _act_cols(N, activation)), dtype=torch.bfloat16, device=X.device)
    _nbytes_at_least(Y, 2 * M * _act_cols(N, activation), "Y")
    need = int(L.bitnet_workspace_bytes(M, K, N, act_bits))
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=X.device)
    _rc(L.bitnet_bitlinear_forward_act(X.data_ptr(), M, K, Wp.data_ptr(), gamma.data_ptr(), N,
                                       int(act_bits), int(bool(hadamard)), int(activation),
                                       Y.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
                                       _stream(stream)),
        "bitnet_bitlinear_forward_act")
    return Y


def _gain_ptr(gain, K):
    if gain is None:
        return None
    _check(gain, "norm_gain", torch.bfloat16, 1)
    if gain.numel() != K:
        raise ValueError(f"norm_gain has {gain.numel()} entries, K = {K}")
    return gain.data_ptr()


def bitnet_act_quant_norm(X: torch.Tensor, norm_gain, eps: float, hadamard: bool, act_bits: int,
                          codes=None, scales=None, rowsum=None, stream=None):
    """RMS normalisation (gain norm_gain bf16 [K] or None, eps) fused with per-token
    (Hadamard +) absmax quantisation.  Returns (codes, scales, rowsum)."""
    L = load_library()
    _check(X, "X", torch.bfloat16, 2)
    M, K = X.shape
    if codes is None:
        codes = torch.empty((M, K if act_bits == 8 else K // 2),
                            dtype=torch.int8 if act_bits == 8 else torch.uint8, device=X.device)
    if scales is None:
        scales = torch.empty(M, dtype=torch.float32, device=X.device)
    if rowsum is None:
        rowsum = torch.empty(M, dtype=torch.int32, device=X.device)
    _nbytes_at_least(codes, int(L.bitnet_act_codes_bytes(M, K, act_bits)), "codes")
    _nbytes_at_least(scales, 4 * M, "scales")
    _nbytes_at_least(rowsum, 4 * M, "rowsum")
    _rc(L.bitnet_act_quant_norm(X.data_ptr(), M, K, _gain_ptr(norm_gain, K), float(eps),
                                int(bool(hadamard)), int(act_bits), codes.data_ptr(),
                                scales.data_ptr(), rowsum.data_ptr(), _stream(stream)),
        "bitnet_act_quant_norm")
    return codes, scales, rowsum


def bitnet_norm_transform_f32(X: torch.Tensor, norm_gain, eps: float, hadamard: bool,
                              Z: torch.Tensor | None = None, stream=None):
    """The normalised rows (and their Hadamard transform) in fp32 (debug / parity entry)."""
    L = load_library()
    _check(X, "X", torch.bfloat16, 2)
    M, K = X.shape
    if Z is None:
        Z = torch.empty((M, K), dtype=torch.float32, device=X.device)
    _rc(L.bitnet_norm_transform_f32(X.data_ptr(), M, K, _gain_ptr(norm_gain, K), float(eps),
                                    int(bool(hadamard)), Z.data_ptr(), _stream(stream)),
        "bitnet_norm_transform_f32")
    return Z


def bitnet_norm_bitlinear_forward(X, norm_gain, eps, hadamard, Wp, gamma, act_bits=8, Y=None,
                                  ws=None, stream=None):
    """Y = (H-)BitLinear(RMSNorm(X)) with the normalisation fused into the quantiser."""
    L = load_library()
    _check(X, "X", torch.bfloat16, 2)
    _check(Wp, "Wp")
    _check(gamma, "gamma", torch.float32)
    M, K = X.shape
    N = Wp.shape[0]
    _nbytes_at_least(Wp, int(L.bitnet_packed_weight_bytes(N, K)), "Wp")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _nbytes_at_least(Y, 2 * M * N, "Y")
    need = int(L.bitnet_workspace_bytes(M, K, N, act_bits))
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=X.device)
    _rc(L.bitnet_norm_bitlinear_forward(X.data_ptr(), M, K, _gain_ptr(norm_gain, K), float(eps),
                                        int(bool(hadamard)), Wp.data_ptr(), gamma.data_ptr(), N,
                                        int(act_bits), Y.data_ptr(), ws.data_ptr(),
                                        ws.numel() * ws.element_size(), _stream(stream)),
        "bitnet_norm_bitlinear_forward")
    return Y


def bitnet_weight_workspace_bytes_rotated(N: int, K: int) -> int:
    return int(load_library().bitnet_weight_workspace_bytes_rotated(N, K))


def bitnet_quantize_pack_weights_rotated(W: torch.Tensor, Wp: torch.Tensor | None = None,
                                         gamma: torch.Tensor | None = None,
                                         ws: torch.Tensor | None = None, stream=None):
    """Weight half of the weight + activation Hadamard rotation: ternarise and pack the rows of
    W H / sqrt(K).  Returns (Wp uint8 [N, K/4], gamma float [1]) for bitnet_hbitlinear_forward."""
    L = load_library()
    _check(W, "W", torch.bfloat16, 2)
    N, K = W.shape
    if Wp is None:
        Wp = torch.empty((N, K // 4), dtype=torch.uint8, device=W.device)
    _nbytes_at_least(Wp, int(L.bitnet_packed_weight_bytes(N, K)), "Wp")
    if gamma is None:
        gamma = torch.empty(1, dtype=torch.float32, device=W.device)
    need = int(L.bitnet_weight_workspace_bytes_rotated(N, K))
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=W.device)
    _rc(L.bitnet_quantize_pack_weights_rotated(W.data_ptr(), N, K, Wp.data_ptr(),
                                               gamma.data_ptr(), ws.data_ptr(),
                                               ws.numel() * ws.element_size(), _stream(stream)),
        "bitnet_quantize_pack_weights_rotated")
    return Wp, gamma


def bitnet_act_quant_absmax4(X: torch.Tensor, hadamard: bool, codes=None, scales=None,
                             rowsum=None, stream=None):
    """Variant INT4 quantiser with a per-token absmax scale (Q = 7).  Returns (codes uint8
    [M, K/2] nibbles, scales, rowsum), consumed by the product with act_bits 4."""
    L = load_library()
    _check(X, "X", torch.bfloat16, 2)
    M, K = X.shape
    if codes is None:
        codes = torch.empty((M, K // 2), dtype=torch.uint8, device=X.device)
    if scales is None:
        scales = torch.empty(M, dtype=torch.float32, device=X.device)
    if rowsum is None:
        rowsum = torch.empty(M, dtype=torch.int32, device=X.device)
    _nbytes_at_least(codes, int(L.bitnet_act_codes_bytes(M, K, 4)), "codes")
    _nbytes_at_least(scales, 4 * M, "scales")
    _nbytes_at_least(rowsum, 4 * M, "rowsum")
    _rc(L.bitnet_act_quant_absmax4(X.data_ptr(), M, K, int(bool(hadamard)), codes.data_ptr(),
                                   scales.data_ptr(), rowsum.data_ptr(), _stream(stream)),
        "bitnet_act_quant_absmax4")
    return codes, scales, rowsum


def bitnet_bitlinear_forward_absmax4(X, Wp, gamma, hadamard: bool, Y=None, ws=None, stream=None):
    """Y = (H-)BitLinear(X) with the variant absmax INT4 activation quantiser."""
    L = load_library()
    _check(X, "X", torch.bfloat16, 2)
    _check(Wp, "Wp")
    _check(gamma, "gamma", torch.float32)
    M, K = X.shape
    N = Wp.shape[0]
    _nbytes_at_least(Wp, int(L.bitnet_packed_weight_bytes(N, K)), "Wp")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _nbytes_at_least(Y, 2 * M * N, "Y")
    need = int(L.bitnet_workspace_bytes(M, K, N, 4))
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=X.device)
    _rc(L.bitnet_bitlinear_forward_absmax4(X.data_ptr(), M, K, Wp.data_ptr(), gamma.data_ptr(),
                                           N, int(bool(hadamard)), Y.data_ptr(), ws.data_ptr(),
                                           ws.numel() * ws.element_size(), _stream(stream)),
        "bitnet_bitlinear_forward_absmax4")
    return Y


def bitnet_base3_weight_bytes(N: int, K: int) -> int:
    return int(load_library().bitnet_base3_weight_bytes(N, K))


def bitnet_quantize_pack_weights_base3(W: torch.Tensor, Wp3: torch.Tensor | None = None,
                                       gamma: torch.Tensor | None = None,
                                       ws: torch.Tensor | None = None, stream=None):
    """absmean-ternarise bf16 W [N, K] into base-3 rows (five weights a byte).
    Returns (Wp3 uint8 [N, 4 * ceil(K/20)], gamma float [1])."""
    L = load_library()
    _check(W, "W", torch.bfloat16, 2)
    N, K = W.shape
    if Wp3 is None:
        Wp3 = torch.empty((N, 4 * ((K + 19) // 20)), dtype=torch.uint8, device=W.device)
    _nbytes_at_least(Wp3, int(L.bitnet_base3_weight_bytes(N, K)), "Wp3")
    if gamma is None:
        gamma = torch.empty(1, dtype=torch.float32, device=W.device)
    need = int(L.bitnet_weight_workspace_bytes(N, K))
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=W.device)
    _rc(L.bitnet_quantize_pack_weights_base3(W.data_ptr(), N, K, Wp3.data_ptr(),
                                             gamma.data_ptr(), ws.data_ptr(),
                                             ws.numel() * ws.element_size(), _stream(stream)),
        "bitnet_quantize_pack_weights_base3")
    return Wp3, gamma


def bitnet_ternary_gemv_base3(codes, scales, rowsum, K: int, Wp3, gamma, activation: int = 0,
                              want_acc=False, want_y=True, acc=None, Y=None, stream=None):
    """Product of INT8 codes (M <= 8 tokens) with base-3 weights Wp3 [N, 4 * ceil(K/20)].
    Returns (acc int32 [M, N] or None, Y bf16 [M, N] ([M, N/2] for SwiGLU) or None)."""
    L = load_library()
    for t, n in ((codes, "codes"), (scales, "scales"), (rowsum, "rowsum"), (Wp3, "Wp3"),
                 (gamma, "gamma")):
        _check(t, n)
    M = scales.numel()
    N = Wp3.shape[0]
    _nbytes_at_least(codes, int(L.bitnet_act_codes_bytes(M, K, 8)), "codes")
    _nbytes_at_least(rowsum, 4 * M, "rowsum")
    _nbytes_at_least(Wp3, int(L.bitnet_base3_weight_bytes(N, K)), "Wp3")
    if want_acc and acc is None:
        acc = torch.empty((M, N), dtype=torch.int32, device=codes.device)
    if want_y and Y is None:
        Y = torch.empty((M, _act_cols(N, activation)), dtype=torch.bfloat16, device=codes.device)
    if Y is not None:
        _nbytes_at_least(Y, 2 * M * _act_cols(N, activation), "Y")
    _rc(L.bitnet_ternary_gemv_base3(codes.data_ptr(), scales.data_ptr(), rowsum.data_ptr(), M, K,
                                    Wp3.data_ptr(), gamma.data_ptr(), N, int(activation),
                                    acc.data_ptr() if acc is not None else None,
                                    Y.data_ptr() if Y is not None else None, _stream(stream)),
        "bitnet_ternary_gemv_base3")
    return acc, Y


def bitnet_bitlinear_forward_base3(X, Wp3, gamma, hadamard: bool, activation: int = 0, Y=None,
                                   ws=None, stream=None):
    """Y = activation((H-)BitLinear(X)) for M <= 8 tokens on base-3 weights, INT8 activations."""
    L = load_library()
    _check(X, "X", torch.bfloat16, 2)
    _check(Wp3, "Wp3")
    _check(gamma, "gamma", torch.float32)
    M, K = X.shape
    N = Wp3.shape[0]
    _nbytes_at_least(Wp3, int(L.bitnet_base3_weight_bytes(N, K)), "Wp3")
    if Y is None:
        Y = torch.empty((M, _act_cols(N, activation)), dtype=torch.bfloat16, device=X.device)
    _nbytes_at_least(Y, 2 * M * _act_cols(N, activation), "Y")
    need = int(L.bitnet_workspace_bytes(M, K, N, 8))
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=X.device)
    _rc(L.bitnet_bitlinear_forward_base3(X.data_ptr(), M, K, Wp3.data_ptr(), gamma.data_ptr(), N,
                                         int(bool(hadamard)), int(activation), Y.data_ptr(),
                                         ws.data_ptr(), ws.numel() * ws.element_size(),
                                         _stream(stream)),
        "bitnet_bitlinear_forward_base3")
    return Y


def bitnet_state_codes_bytes(M: int, C: int, bits: int) -> int:
    return int(load_library().bitnet_state_codes_bytes(M, C, bits))


def bitnet_quant_states(X: torch.Tensor, group: int, bits: int = 3, codes=None, scales=None,
                        stream=None):
    """Low-bit absmax codes of bf16 Q/K/V states [M, C], per group of `group` features.
    Returns (codes uint8 [M, C * bits / 8] bit streams, scales float [M, C / group])."""
    L = load_library()
    _check(X, "X", torch.bfloat16, 2)
    M, C = X.shape
    if codes is None:
        codes = torch.empty((M, C * bits // 8), dtype=torch.uint8, device=X.device)
    if scales is None:
        scales = torch.empty((M, max(C // group, 1)), dtype=torch.float32, device=X.device)
    _nbytes_at_least(codes, int(L.bitnet_state_codes_bytes(M, C, bits)), "codes")
    _nbytes_at_least(scales, 4 * M * (C // group), "scales")
    _rc(L.bitnet_quant_states(X.data_ptr(), M, C, int(group), int(bits), codes.data_ptr(),
                              scales.data_ptr(), _stream(stream)), "bitnet_quant_states")
    return codes, scales


def _device_of(t, name: str) -> int:
    """The CUDA device of a tensor, which has to be the current one: the library launches there."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return dev


def _plain(t, name: str, dtype, dim, dev: int) -> int:
    """The address of a contiguous tensor of this type on device `dev`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and (dim is None or t.dim() == dim)
            and t.get_device() == dev and t.is_contiguous()):
        _check(t, name, dtype, dim)  # says what is wrong
        raise ValueError("all tensors must be on one device")
    return t.data_ptr()


# the current stream's handle without a Stream object around it (a microsecond and a half)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(stream, dev: int) -> int:
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream)


_empty_strided = torch.empty_strided


def _empty(rows: int, cols: int, dtype, device, stream):
    """A new [rows, cols] tensor ([rows] where cols is 0), in the pool of the stream that the call
    launches on, so that memory which is freed right after the call is not handed to another
    stream while the kernels still use it.  (empty_strided costs a microsecond less than empty.)"""
    size, stride = ((rows, cols), (cols, 1)) if cols else ((rows,), (1,))
    if stream is None:
        return _empty_strided(size, stride, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(raw, device=device)
    with torch.cuda.stream(stream):
        return _empty_strided(size, stride, dtype=dtype, device=device)


def _residual_args(X, R, norm_gain, H, stream):
    """Checked (device, M, K, pointers of X, R and the gain, H)."""
    dev = _device_of(X, "X")
    x = _plain(X, "X", torch.bfloat16, 2, dev)
    r = _plain(R, "R", torch.bfloat16, 2, dev)
    if R.shape != X.shape:
        raise ValueError(f"R is {tuple(R.shape)}, X is {tuple(X.shape)}")
    M, K = X.shape
    gain = None
    if norm_gain is not None:
        gain = _plain(norm_gain, "norm_gain", torch.bfloat16, 1, dev)
        if norm_gain.shape[0] != K:
            raise ValueError(f"norm_gain has {norm_gain.numel()} entries, K = {K}")
    if H is None:
        H = _empty(M, K, torch.bfloat16, X.device, stream)
    else:
        _plain(H, "H", torch.bfloat16, None, dev)
        _nbytes_at_least(H, 2 * M * K, "H")
    return dev, M, K, x, r, gain, H


def bitnet_act_quant_residual_norm(X: torch.Tensor, R: torch.Tensor, norm_gain, eps: float,
                                   act_bits: int, H=None, codes=None, scales=None, rowsum=None,
                                   stream=None):
    """Residual addition, RMS normalisation and per-token quantisation in one pass: H = X + R
    (bf16; may be X or R), codes of the normalised H.  Returns (H, codes, scales, rowsum)."""
    L = _lib or load_library()
    dev, M, K, x, r, gain, H = _residual_args(X, R, norm_gain, H, stream)
    if codes is None:
        codes = _empty(M, K if act_bits == 8 else K // 2,
                       torch.int8 if act_bits == 8 else torch.uint8, X.device, stream)
    else:
        _plain(codes, "codes", codes.dtype, None, dev)
        _nbytes_at_least(codes, int(L.bitnet_act_codes_bytes(M, K, act_bits)), "codes")
    if scales is None:
        scales = _empty(M, 0, torch.float32, X.device, stream)
    else:
        _plain(scales, "scales", torch.float32, None, dev)
        _nbytes_at_least(scales, 4 * M, "scales")
    if rowsum is None:
        rowsum = _empty(M, 0, torch.int32, X.device, stream)
    else:
        _plain(rowsum, "rowsum", torch.int32, None, dev)
        _nbytes_at_least(rowsum, 4 * M, "rowsum")
    _rc(L.bitnet_act_quant_residual_norm(x, r, M, K, gain, eps, act_bits, H.data_ptr(),
                                         codes.data_ptr(), scales.data_ptr(), rowsum.data_ptr(),
                                         _stream_on(stream, dev)),
        "bitnet_act_quant_residual_norm")
    return H, codes, scales, rowsum


def bitnet_residual_norm_bitlinear_forward(X, R, norm_gain, eps, Wp, gamma, act_bits=8, H=None,
                                           Y=None, ws=None, stream=None):
    """H = X + R (bf16; may be X or R), Y = BitLinear(RMSNorm(H)).  Returns (H, Y)."""
    L = _lib or load_library()
    dev, M, K, x, r, gain, H = _residual_args(X, R, norm_gain, H, stream)
    wp = _plain(Wp, "Wp", Wp.dtype, None, dev)
    g = _plain(gamma, "gamma", torch.float32, None, dev)
    N = Wp.shape[0]
    _nbytes_at_least(Wp, N * K // 4, "Wp")
    if Y is None:
        Y = _empty(M, N, torch.bfloat16, X.device, stream)
    else:
        _plain(Y, "Y", torch.bfloat16, None, dev)
        _nbytes_at_least(Y, 2 * M * N, "Y")
    if ws is None:
        ws = _empty(max(int(L.bitnet_workspace_bytes(M, K, N, act_bits)), 256), 0, torch.uint8,
                    X.device, stream)
    else:
        _plain(ws, "ws", ws.dtype, None, dev)
    _rc(L.bitnet_residual_norm_bitlinear_forward(
        x, r, M, K, gain, eps, wp, g, N, act_bits, H.data_ptr(), Y.data_ptr(), ws.data_ptr(),
        ws.numel() * ws.element_size(), _stream_on(stream, dev)),
        "bitnet_residual_norm_bitlinear_forward")
    return H, Y


class KvCache:
    """A paged 8-bit K/V cache (bitnet_kv_cache) over the caller's tensors: k_codes, v_codes int8
    [num_pages, kv_heads, page_tokens, head_dim]; k_scales, v_scales float
    [num_pages, kv_heads, page_tokens / scale_tokens].  It only holds and describes them."""

    __slots__ = ("k_codes", "v_codes", "k_scales", "v_scales", "num_pages", "kv_heads",
                 "page_tokens", "head_dim", "scale_tokens", "device", "_c", "_ref", "_sizes")

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        for t, n in ((k_codes, "k_codes"), (v_codes, "v_codes")):
            _check(t, n, torch.int8, 4)
        for t, n in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            _check(t, n, torch.float32, 3)
        pages, heads, page, dim = k_codes.shape
        blocks = k_scales.shape[2]
        if v_codes.shape != k_codes.shape or v_scales.shape != k_scales.shape:
            raise ValueError("K and V differ in shape")
        if k_scales.shape[:2] != (pages, heads) or blocks < 1 or page % blocks:
            raise ValueError(f"scales {tuple(k_scales.shape)} do not fit codes "
                             f"{tuple(k_codes.shape)}")
        if len({t.get_device() for t in (k_codes, v_codes, k_scales, v_scales)}) != 1:
            raise ValueError("all tensors must be on one device")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = (k_codes, v_codes, k_scales,
                                                                    v_scales)
        self.num_pages, self.kv_heads, self.page_tokens, self.head_dim = pages, heads, page, dim
        self.scale_tokens = page // blocks
        self._c = _CKvCache(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(),
                            v_scales.data_ptr(), pages, heads, dim, page, self.scale_tokens)
        self._ref = ctypes.byref(self._c)
        self.device = k_codes.get_device()
        self._sizes = {}  # workspace bytes by the sizes of a batch

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, head_dim: int, page_tokens: int = 64,
              scale_tokens: int = 16, device="cuda") -> "KvCache":
        """A cache of its own tensors, not cleared (new pages need no clearing)."""
        if scale_tokens < 1 or page_tokens % scale_tokens:
            raise ValueError(f"page_tokens {page_tokens} is no multiple of scale_tokens "
                             f"{scale_tokens}")
        codes = [torch.empty((num_pages, kv_heads, page_tokens, head_dim), dtype=torch.int8,
                             device=device) for _ in range(2)]
        scales = [torch.empty((num_pages, kv_heads, page_tokens // scale_tokens),
                              dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*codes, *scales)


def _kv_batch(cache: KvCache, q_start, kv_len, page_table, tokens: int) -> _CKvBatch:
    dev, i32 = cache.device, torch.int32
    if dev != torch.cuda.current_device():
        raise ValueError(f"the cache is on cuda:{dev}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    starts = _plain(q_start, "q_start", i32, 1, dev)
    lengths = _plain(kv_len, "kv_len", i32, 1, dev)
    table = _plain(page_table, "page_table", i32, 2, dev)
    batch = kv_len.shape[0]
    rows, max_pages = page_table.shape
    if q_start.shape[0] != batch + 1 or rows != batch:
        raise ValueError(f"kv_len has {batch} sequences, q_start {q_start.shape[0]} entries, "
                         f"page_table {rows} rows")
    return _CKvBatch(starts, lengths, table, batch, max_pages, tokens)


def _rows(t, name: str, width: int, tokens, dev: int):
    """(pointer, row distance in elements) of a bf16 matrix of `width` columns on device `dev` whose
    rows may lie apart; [tokens, heads, head_dim] counts as [tokens, heads * head_dim]."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        raise ValueError("all tensors must be on one device" if t.is_cuda
                         else f"{name} must be a CUDA tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        cols = shape[1]
        if cols > 1 and stride[1] != 1 and shape[0]:
            raise ValueError(f"the columns of {name} must be contiguous")
    elif len(shape) == 3:
        cols = shape[1] * shape[2]
        if not t.is_contiguous() and shape[0] and (
                stride[2] != 1 or shape[1] > 1 and stride[1] != shape[2]):
            raise ValueError(f"the heads of a row of {name} must lie one after the other")
    else:
        raise ValueError(f"{name} must have 2 or 3 dimensions")
    if cols != width:
        raise ValueError(f"{name} has rows of {cols}, {width} wanted")
    if tokens is not None and shape[0] != tokens:
        raise ValueError(f"{name} has {shape[0]} rows, {tokens} wanted")
    # a single row has no distance to the next one, and no rows have no strides at all
    return t.data_ptr(), stride[0] if shape[0] > 1 else width


def bitnet_kv_cache_append(cache: KvCache, K: torch.Tensor, V: torch.Tensor, q_start, kv_len,
                           page_table, stream=None) -> None:
    """Quantise the new tokens' K and V (bf16 [tokens, kv_heads * head_dim], rows may lie apart)
    into the cache.  q_start int32 [batch + 1], kv_len int32 [batch] (with the new tokens),
    page_table int32 [batch, max_pages]."""
    L = _lib or load_library()
    width, dev = cache.kv_heads * cache.head_dim, cache.device
    k, ldk = _rows(K, "K", width, None, dev)
    tokens = K.shape[0]
    v, ldv = _rows(V, "V", width, tokens, dev)
    batch = _kv_batch(cache, q_start, kv_len, page_table, tokens)
    _rc(L.bitnet_kv_cache_append(cache._ref, batch, k, ldk, v, ldv, _stream_on(stream, dev)),
        "bitnet_kv_cache_append")


def bitnet_kv_cache_read(cache: KvCache, tokens: int, q_start, kv_len, page_table, K=None, V=None,
                         stream=None):
    """The last q_start[s + 1] - q_start[s] tokens of each sequence as bf16, packed: returns
    (K, V), each [tokens, kv_heads * head_dim]."""
    L = _lib or load_library()
    width, dev = cache.kv_heads * cache.head_dim, cache.device
    if K is None:
        K = _empty(tokens, width, torch.bfloat16, cache.k_codes.device, stream)
    if V is None:
        V = _empty(tokens, width, torch.bfloat16, cache.k_codes.device, stream)
    k, ldk = _rows(K, "K", width, tokens, dev)
    v, ldv = _rows(V, "V", width, tokens, dev)
    batch = _kv_batch(cache, q_start, kv_len, page_table, tokens)
    _rc(L.bitnet_kv_cache_read(cache._ref, batch, k, ldk, v, ldv, _stream_on(stream, dev)),
        "bitnet_kv_cache_read")
    return K, V


def bitnet_kv_attention_workspace_bytes(cache: KvCache, tokens: int, batch: int, max_pages: int,
                                        q_heads: int, max_new: int) -> int:
    """Bytes of workspace bitnet_kv_attention needs for such a batch (host only)."""
    key = (tokens, batch, max_pages, q_heads, max_new)
    need = cache._sizes.get(key)
    if need is None:
        one = 16  # the query looks at sizes, not at the arrays
        b = _CKvBatch(one, one, one, batch, max_pages, tokens)
        need = int(load_library().bitnet_kv_attention_workspace_bytes(
            cache._ref, ctypes.byref(b), q_heads, max_new))
        if len(cache._sizes) < 4096:
            cache._sizes[key] = need
    return need


def bitnet_kv_attention(cache: KvCache, Q: torch.Tensor, q_heads: int, q_start, kv_len,
                        page_table, max_new: int, scale: float | None = None,
                        causal: bool = True, Y=None, lse=None, want_lse: bool = False, ws=None,
                        stream=None):
    """Attention of new tokens Q (bf16 [tokens, q_heads * head_dim], rows may lie apart) over the
    cached states of their sequences.  max_new: the most new tokens of any sequence; it chooses the
    kernel for the whole batch, so prompts and single tokens belong in calls of their own.  scale
    defaults to 1 / sqrt(head_dim).  Returns (Y bf16 [tokens, q_heads * head_dim], lse float
    [tokens, q_heads] or None)."""
    L = _lib or load_library()
    width, dev = q_heads * cache.head_dim, cache.device
    q, ldq = _rows(Q, "Q", width, None, dev)
    tokens = Q.shape[0]
    batch = _kv_batch(cache, q_start, kv_len, page_table, tokens)
    if Y is None:
        Y = _empty(tokens, width, torch.bfloat16, Q.device, stream)
        y, ldy = Y.data_ptr(), width
    else:
        y, ldy = _rows(Y, "Y", width, tokens, dev)
    lse_ptr = None
    if lse is not None:
        lse_ptr = _plain(lse, "lse", torch.float32, None, dev)
        _nbytes_at_least(lse, 4 * tokens * q_heads, "lse")
    elif want_lse:
        lse = _empty(tokens, q_heads, torch.float32, Q.device, stream)
        lse_ptr = lse.data_ptr()
    ws_ptr, ws_bytes = None, 0
    if ws is not None:
        ws_ptr, ws_bytes = _plain(ws, "ws", ws.dtype, None, dev), ws.numel() * ws.element_size()
    else:
        ws_bytes = bitnet_kv_attention_workspace_bytes(cache, tokens, batch.batch,
                                                       batch.max_pages, q_heads, max_new)
        if ws_bytes:
            ws = _empty(ws_bytes, 0, torch.uint8, Q.device, stream)
            ws_ptr = ws.data_ptr()
    _rc(L.bitnet_kv_attention(cache._ref, batch, q, ldq, q_heads, max_new,
                              cache.head_dim ** -0.5 if scale is None else scale,
                              1 if causal else 0, y, ldy, lse_ptr, ws_ptr, ws_bytes,
                              _stream_on(stream, dev)), "bitnet_kv_attention")
    return Y, lse


def bitnet_selftest_wait_timeout(limit_cycles: int, stream=None) -> None:
    """Enqueue the failure-detection self-test: one bounded wait that runs out after
    limit_cycles SM cycles and records a time-out for the next bitnet_sync_status()."""
    st = load_library().bitnet_selftest_wait_timeout(int(limit_cycles), _stream(stream))
    _rc(st, "bitnet_selftest_wait_timeout")


def bitnet_sync_status(stream=None) -> int:
    """Synchronise the stream and raise BitnetError if a kernel reported a fault or time-out."""
    st = load_library().bitnet_sync_status(_stream(stream))
    _rc(st, "bitnet_sync_status")
    return st
