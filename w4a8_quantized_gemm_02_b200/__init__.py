"""Python binding of ``libqoq.so``: the B200 (sm_100a) W4A8 GEMM with
progressive group quantization (QoQ, "QServe: W4A8KV4 Quantization and System
Co-design for Efficient LLM Serving", Methods 1) Algorithm: QoQ and
2) System: QServe).

This module only marshals arguments (torch tensors -> device pointers, the
current CUDA stream) into the C ABI declared in ``include/qoq.h``; every step
of the computation runs in the library's CUDA kernels.  There is no CPU
fallback: if the library is not built, or a call fails, an exception is
raised.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqoq.so")

QOQ_OK = 0
QOQ_ERR_INVALID_ARG = 1
QOQ_ERR_UNSUPPORTED = 2
QOQ_ERR_CUDA = 3
QOQ_ERR_WORKSPACE = 4

# Every symbol the public header declares.
EXPORTS = (
    "qoq_status_str", "qoq_version", "qoq_protective_range",
    "qoq_packed_block_bytes", "qoq_packed_weight_bytes",
    "qoq_quantize_weights", "qoq_pack_codes", "qoq_unpack_weights",
    "qoq_quantize_act_per_token", "qoq_w4a8_gemm", "qoq_w4a8_gemm_i32",
    "qoq_w4a8_gemm_config", "qoq_w4a8_linear", "qoq_gemm_plan", "qoq_device_error",
    "qoq_gemm_workspace_bytes", "qoq_gemm_workspace_bytes_config",
    "qoq_w4a8_gemm_static_ws", "qoq_selftest_wait_timeout", "qoq_w4a8_linear_fused",
    "qoq_smooth_factors", "qoq_quantize_weights_smoothed", "qoq_quantize_act_per_token_smoothed",
    "qoq_quantize_weights_gate_up", "qoq_w4a8_gate_up_silu",
    "qoq_kv4_cache_bytes", "qoq_kv4_quantize", "qoq_kv4_attention_workspace_bytes",
    "qoq_kv4_decode_attention",
    "qoq_kv4_paged_bytes", "qoq_kv4_paged_append", "qoq_kv4_paged_attention_workspace_bytes",
    "qoq_kv4_paged_attention", "qoq_lora_workspace_bytes", "qoq_lora_add",
)

_lock = threading.Lock()
_lib = None


class QoQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """Load ``libqoq.so`` (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m w4a8_quantized_gemm_02_b200.build`")
            L = ctypes.CDLL(LIB_PATH)
            P, I = ctypes.c_void_p, ctypes.c_int
            sz = ctypes.c_size_t
            L.qoq_status_str.restype = ctypes.c_char_p
            L.qoq_status_str.argtypes = [I]
            L.qoq_version.restype = I
            L.qoq_version.argtypes = []
            L.qoq_protective_range.restype = I
            L.qoq_protective_range.argtypes = []
            L.qoq_packed_block_bytes.restype = sz
            L.qoq_packed_block_bytes.argtypes = [I]
            L.qoq_packed_weight_bytes.restype = sz
            L.qoq_packed_weight_bytes.argtypes = [I, I, I]
            L.qoq_quantize_weights.restype = I
            L.qoq_quantize_weights.argtypes = [P, I, I, I, P, P, P]
            L.qoq_pack_codes.restype = I
            L.qoq_pack_codes.argtypes = [P, P, P, I, I, I, P, P]
            L.qoq_unpack_weights.restype = I
            L.qoq_unpack_weights.argtypes = [P, I, I, I, P, P, P, P, P]
            L.qoq_quantize_act_per_token.restype = I
            L.qoq_quantize_act_per_token.argtypes = [P, I, I, P, P, P]
            L.qoq_quantize_weights_gate_up.restype = I
            L.qoq_quantize_weights_gate_up.argtypes = [P, I, I, I, P, P, P]
            L.qoq_w4a8_gate_up_silu.restype = I
            L.qoq_w4a8_gate_up_silu.argtypes = [P, P, P, P, I, I, I, I, P, P, P, P]
            L.qoq_smooth_factors.restype = I
            L.qoq_smooth_factors.argtypes = [P, I, P, I, I, P, P]
            L.qoq_quantize_weights_smoothed.restype = I
            L.qoq_quantize_weights_smoothed.argtypes = [P, P, I, I, I, P, P, P]
            L.qoq_quantize_act_per_token_smoothed.restype = I
            L.qoq_quantize_act_per_token_smoothed.argtypes = [P, P, I, I, P, P, P]
            L.qoq_w4a8_gemm.restype = I
            L.qoq_w4a8_gemm.argtypes = [P, P, P, P, I, I, I, I, P, P, sz, P]
            L.qoq_selftest_wait_timeout.restype = I
            L.qoq_selftest_wait_timeout.argtypes = [P]
            L.qoq_w4a8_gemm_static_ws.restype = I
            L.qoq_w4a8_gemm_static_ws.argtypes = [P, P, P, P, I, I, I, I, P, P]
            L.qoq_w4a8_gemm_i32.restype = I
            L.qoq_w4a8_gemm_i32.argtypes = [P, P, I, I, I, I, P, P, sz, P]
            L.qoq_w4a8_gemm_config.restype = I
            L.qoq_w4a8_gemm_config.argtypes = [P, P, P, P, I, I, I, I, P, P, I, I, P, sz, P]
            L.qoq_w4a8_linear.restype = I
            L.qoq_w4a8_linear.argtypes = [P, I, I, P, P, I, I, P, P, P, P, sz, P]
            L.qoq_w4a8_linear_fused.restype = I
            L.qoq_w4a8_linear_fused.argtypes = [P, I, I, P, P, I, I, P, P, P, P, sz, P]
            L.qoq_gemm_workspace_bytes.restype = sz
            L.qoq_gemm_workspace_bytes.argtypes = [I, I, I, I]
            L.qoq_gemm_workspace_bytes_config.restype = sz
            L.qoq_gemm_workspace_bytes_config.argtypes = [I, I, I, I, I, I]
            L.qoq_gemm_plan.restype = I
            L.qoq_gemm_plan.argtypes = [I, I, I, I] + [ctypes.POINTER(I)] * 4
            L.qoq_kv4_cache_bytes.restype = I
            L.qoq_kv4_cache_bytes.argtypes = [I, I, I, I] + [ctypes.POINTER(sz)] * 3
            L.qoq_kv4_quantize.restype = I
            L.qoq_kv4_quantize.argtypes = [P, P, I, I, I, I, I, I, P, P, P, P]
            L.qoq_kv4_attention_workspace_bytes.restype = sz
            L.qoq_kv4_attention_workspace_bytes.argtypes = [I, I, I, I, I]
            L.qoq_kv4_decode_attention.restype = I
            L.qoq_kv4_decode_attention.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P, sz, P]
            L.qoq_kv4_paged_bytes.restype = I
            L.qoq_kv4_paged_bytes.argtypes = [I, I, I, I] + [ctypes.POINTER(sz)] * 3
            L.qoq_kv4_paged_append.restype = I
            L.qoq_kv4_paged_append.argtypes = ([P, sz, I, I, I, I, P, P, I, P, I, I, I, P, I, I,
                                                ctypes.c_double] + [P] * 7)
            L.qoq_kv4_paged_attention_workspace_bytes.restype = sz
            L.qoq_kv4_paged_attention_workspace_bytes.argtypes = [I] * 8
            L.qoq_kv4_paged_attention.restype = I
            L.qoq_kv4_paged_attention.argtypes = [P, sz, I, I, I, I, P, P, P, P, P, I, P, I, I, I,
                                                  I, ctypes.c_float, P, P, sz, P]
            L.qoq_lora_workspace_bytes.restype = sz
            L.qoq_lora_workspace_bytes.argtypes = [I] * 5
            L.qoq_lora_add.restype = I
            L.qoq_lora_add.argtypes = [P, P, I, I, I, P, P, I, I, P, P, P, P, sz, P]
            L.qoq_device_error.restype = I
            L.qoq_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint), I]
            _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().qoq_status_str(int(status)).decode()


def _check(status: int, where: str):
    if status != QOQ_OK:
        raise QoQError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need_cuda(t, name, dtype=None, ndim=None, shape=None, device=None, min_bytes=None):
    """Reject anything the library would read or write through a bad pointer:
    a host tensor, another device's tensor, a strided view, the wrong dtype,
    shape or size."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if min_bytes is not None and t.numel() * t.element_size() < min_bytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, "
                         f"needs {min_bytes}")


def _need_packed(packed, N, K, group, device):
    import torch
    nbytes = packed_weight_bytes(N, K, group)
    if nbytes == 0:
        raise QoQError(QOQ_ERR_INVALID_ARG, "qoq_packed_weight_bytes")
    _need_cuda(packed, "packed", torch.uint8, device=device, min_bytes=nbytes)


def _need_gemm_operands(X8, sx, packed, s1, N, group):
    """X8 (M, K) int8 and, where given, sx (M,) fp16, s1 (N,) fp16 and the
    packed weights of an N x K layer, all on X8's device.  Returns M, K."""
    import torch
    _need_cuda(X8, "X8", torch.int8, 2)
    M, K = X8.shape
    dev = X8.device
    if sx is not None:
        _need_cuda(sx, "sx", torch.float16, shape=(M,), device=dev)
    if s1 is not None:
        _need_cuda(s1, "s1", torch.float16, shape=(N,), device=dev)
    _need_packed(packed, N, K, group, dev)
    return M, K


def _out(out, shape, dtype, device):
    """The caller's output tensor after checking it, or a new one."""
    import torch
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need_cuda(out, "out", dtype, shape=shape, device=device)
    return out


def _need_ws(ws, device):
    import torch
    if ws is not None:
        _need_cuda(ws, "ws", torch.uint8, device=device)


# ---------------------------------------------------------------------------
# sizes / plan
# ---------------------------------------------------------------------------

def packed_block_bytes(group: int = 128) -> int:
    return int(lib().qoq_packed_block_bytes(group))


def packed_weight_bytes(N: int, K: int, group: int = 128) -> int:
    return int(lib().qoq_packed_weight_bytes(N, K, group))


def gemm_plan(M: int, N: int, K: int, group: int = 128) -> dict:
    vals = [ctypes.c_int() for _ in range(4)]
    _check(lib().qoq_gemm_plan(M, N, K, group, *[ctypes.byref(v) for v in vals]),
           "qoq_gemm_plan")
    return dict(zip(("tok_tile", "splits", "ctas", "stages"), (v.value for v in vals)))


def gemm_workspace_bytes(M: int, N: int, K: int, group: int = 128, tok_tile: int = 0,
                         splits: int = 0) -> int:
    if tok_tile or splits:
        return int(lib().qoq_gemm_workspace_bytes_config(M, N, K, group, tok_tile, splits))
    return int(lib().qoq_gemm_workspace_bytes(M, N, K, group))


_ws_cache = {}


def workspace(nbytes: int, device, stream=None, kind: str = "gemm"):
    """A reusable, zero-initialized device workspace of at least `nbytes`
    bytes.  There is one buffer per (device, stream, kind), grown on demand
    and allocated and zeroed on that stream: the split-K counters in the
    GEMM's assume that the calls sharing it run one after another, which
    calls on one stream do.  The attention's partial results go to a buffer
    of their own (kind "kv4"), which leaves the GEMM's counters at zero."""
    import torch
    if nbytes <= 0:
        return None
    device = torch.device(device)
    if stream is None:
        stream = torch.cuda.current_stream(device)
    key = (device.index, stream.cuda_stream, kind)
    with _lock:
        buf = _ws_cache.get(key)
        if buf is None or buf.numel() < nbytes:
            with torch.cuda.stream(stream):
                buf = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
            _ws_cache[key] = buf
    return buf


def _ws_args(ws):
    if ws is None:
        return None, 0
    return ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size()


def selftest_wait_timeout(stream=None):
    """Launch the bounded-wait self-test kernel (about 2 s on the device);
    afterwards device_error() has bit 64 set."""
    _check(lib().qoq_selftest_wait_timeout(_stream(stream)), "qoq_selftest_wait_timeout")


def device_error(clear: bool = True) -> int:
    v = ctypes.c_uint()
    _check(lib().qoq_device_error(ctypes.byref(v), int(clear)), "qoq_device_error")
    return int(v.value)


# ---------------------------------------------------------------------------
# offline weight quantization
# ---------------------------------------------------------------------------

def quantize_weights(W, group: int = 128, stream=None):
    """W: (N, K) float16 CUDA tensor -> (packed uint8 tensor, s1 float16[N])."""
    import torch
    _need_cuda(W, "W", torch.float16, 2)
    N, K = W.shape
    nbytes = packed_weight_bytes(N, K, group)
    if nbytes == 0:
        raise QoQError(QOQ_ERR_INVALID_ARG, "qoq_packed_weight_bytes")
    packed = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    s1 = torch.empty(N, dtype=torch.float16, device=W.device)
    _check(lib().qoq_quantize_weights(_ptr(W), N, K, group, _ptr(packed), _ptr(s1),
                                      _stream(stream)), "qoq_quantize_weights")
    return packed, s1


def pack_codes(q, s2, z, group: int = 128, stream=None):
    """Canonical codes (uint8 N x K, int8 N x K/G, uint8 N x K/G) -> packed."""
    import torch
    _need_cuda(q, "q", torch.uint8, 2)
    N, K = q.shape
    if group <= 0 or K % group:
        raise QoQError(QOQ_ERR_INVALID_ARG, "qoq_pack_codes")
    _need_cuda(s2, "s2", torch.int8, shape=(N, K // group), device=q.device)
    _need_cuda(z, "z", torch.uint8, shape=(N, K // group), device=q.device)
    nbytes = packed_weight_bytes(N, K, group)
    if nbytes == 0:
        raise QoQError(QOQ_ERR_INVALID_ARG, "qoq_packed_weight_bytes")
    packed = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _check(lib().qoq_pack_codes(_ptr(q), _ptr(s2), _ptr(z), N, K, group, _ptr(packed),
                                _stream(stream)), "qoq_pack_codes")
    return packed


def unpack_weights(packed, N: int, K: int, group: int = 128, stream=None):
    """packed -> (q uint8 N x K, s2 int8, z uint8, dq int8 N x K)."""
    import torch
    _need_cuda(packed, "packed", torch.uint8)
    dev = packed.device
    _need_packed(packed, N, K, group, dev)
    q = torch.empty((N, K), dtype=torch.uint8, device=dev)
    s2 = torch.empty((N, K // group), dtype=torch.int8, device=dev)
    z = torch.empty((N, K // group), dtype=torch.uint8, device=dev)
    dq = torch.empty((N, K), dtype=torch.int8, device=dev)
    _check(lib().qoq_unpack_weights(_ptr(packed), N, K, group, _ptr(q), _ptr(s2), _ptr(z),
                                    _ptr(dq), _stream(stream)), "qoq_unpack_weights")
    return q, s2, z, dq


# ---------------------------------------------------------------------------
# online path
# ---------------------------------------------------------------------------

def quantize_act_per_token(X, out=None, stream=None):
    """X: (M, K) float16 -> (X8 int8 (M, K), sx float16 (M,))."""
    import torch
    _need_cuda(X, "X", torch.float16, 2)
    M, K = X.shape
    if out is None:
        X8 = torch.empty((M, K), dtype=torch.int8, device=X.device)
        sx = torch.empty(M, dtype=torch.float16, device=X.device)
    else:
        X8, sx = out
        _need_cuda(X8, "X8", torch.int8, shape=(M, K), device=X.device)
        _need_cuda(sx, "sx", torch.float16, shape=(M,), device=X.device)
    _check(lib().qoq_quantize_act_per_token(_ptr(X), M, K, _ptr(X8), _ptr(sx),
                                            _stream(stream)), "qoq_quantize_act_per_token")
    return X8, sx


def quantize_weights_gate_up(W, group: int = 128, stream=None):
    """A fused gate_up weight W (2I, K) float16 (gate rows first) ->
    (packed, s1 float16[2I]) in the interleaved tile order."""
    import torch
    _need_cuda(W, "W", torch.float16, 2)
    N2, K = W.shape
    if N2 % 128:
        raise ValueError("W must have 2I rows with I % 64 == 0")
    nbytes = packed_weight_bytes(N2, K, group)
    if nbytes == 0:
        raise QoQError(QOQ_ERR_INVALID_ARG, "qoq_packed_weight_bytes")
    packed = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    s1 = torch.empty(N2, dtype=torch.float16, device=W.device)
    _check(lib().qoq_quantize_weights_gate_up(_ptr(W), N2 // 2, K, group, _ptr(packed), _ptr(s1),
                                              _stream(stream)), "qoq_quantize_weights_gate_up")
    return packed, s1


def w4a8_gate_up_silu(X8, sx, packed, s1, I: int, group: int = 128, out=None, stream=None):
    """H = silu(gate) * up (M, I) float16 from the gate_up weight, and its
    per-token INT8 quantization (H8, sh) for the down projection."""
    import torch
    M, K = _need_gemm_operands(X8, sx, packed, s1, 2 * I, group)
    dev = X8.device
    if out is None:
        H = torch.empty((M, I), dtype=torch.float16, device=dev)
        H8 = torch.empty((M, I), dtype=torch.int8, device=dev)
        sh = torch.empty(M, dtype=torch.float16, device=dev)
    else:
        H, H8, sh = out
        _need_cuda(H, "H", torch.float16, shape=(M, I), device=dev)
        _need_cuda(H8, "H8", torch.int8, shape=(M, I), device=dev)
        _need_cuda(sh, "sh", torch.float16, shape=(M,), device=dev)
    _check(lib().qoq_w4a8_gate_up_silu(_ptr(X8), _ptr(sx), _ptr(packed), _ptr(s1), M, I, K, group,
                                       _ptr(H), _ptr(H8), _ptr(sh), _stream(stream)),
           "qoq_w4a8_gate_up_silu")
    return H, H8, sh


def kv4_cache_bytes(B: int, Hkv: int, L: int, d: int = 128):
    """(k_bytes, v_bytes, scale_bytes) of a 4-bit KV cache."""
    k, v, sc = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().qoq_kv4_cache_bytes(B, Hkv, L, d, ctypes.byref(k), ctypes.byref(v),
                                     ctypes.byref(sc)), "qoq_kv4_cache_bytes")
    return k.value, v.value, sc.value


def kv4_cache(B: int, Hkv: int, L: int, device, d: int = 128):
    """An empty cache: (k_codes uint8, v_codes uint8, scales float16) device
    tensors, (B, Hkv, L // 16, 1024), (B, Hkv, L // 16, 1024) and
    (B, Hkv, L, 4)."""
    import torch
    kv4_cache_bytes(B, Hkv, L, d)
    kc = torch.zeros((B, Hkv, L // 16, 1024), dtype=torch.uint8, device=device)
    vc = torch.zeros((B, Hkv, L // 16, 1024), dtype=torch.uint8, device=device)
    sc = torch.zeros((B, Hkv, L, 4), dtype=torch.float16, device=device)
    return kc, vc, sc


def kv4_quantize(K, V, cache, t0: int = 0, stream=None):
    """Write K, V ((B, Hkv, T, 128) float16) into cache slots t0 .. t0+T-1."""
    import torch
    kc, vc, sc = cache
    _need_cuda(K, "K", torch.float16, 4)
    B, Hkv, T, d = K.shape
    _need_cuda(V, "V", torch.float16, shape=tuple(K.shape), device=K.device)
    L = sc.shape[2]
    _need_cuda(kc, "k_codes", torch.uint8, shape=(B, Hkv, L // 16, 1024), device=K.device)
    _need_cuda(vc, "v_codes", torch.uint8, shape=(B, Hkv, L // 16, 1024), device=K.device)
    _need_cuda(sc, "scales", torch.float16, shape=(B, Hkv, L, 4), device=K.device)
    _check(lib().qoq_kv4_quantize(_ptr(K), _ptr(V), B, Hkv, T, d, L, t0, _ptr(kc), _ptr(vc),
                                  _ptr(sc), _stream(stream)), "qoq_kv4_quantize")


def kv4_decode_attention(Q, cache, seqlen, out=None, ws=None, stream=None):
    """Decode attention of Q ((B, Hq, 128) float16) over the 4-bit cache for
    the first seqlen[b] tokens (int32 CUDA tensor (B,)); returns (B, Hq, 128)
    float16."""
    import torch
    kc, vc, sc = cache
    _need_cuda(Q, "Q", torch.float16, 3)
    B, Hq, d = Q.shape
    Hkv, L = sc.shape[1], sc.shape[2]
    _need_cuda(kc, "k_codes", torch.uint8, shape=(B, Hkv, L // 16, 1024), device=Q.device)
    _need_cuda(vc, "v_codes", torch.uint8, shape=(B, Hkv, L // 16, 1024), device=Q.device)
    _need_cuda(sc, "scales", torch.float16, shape=(B, Hkv, L, 4), device=Q.device)
    _need_cuda(seqlen, "seqlen", torch.int32, shape=(B,), device=Q.device)
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float16, device=Q.device)
    else:
        _need_cuda(out, "out", torch.float16, shape=(B, Hq, d), device=Q.device)
    need = int(lib().qoq_kv4_attention_workspace_bytes(B, Hq, Hkv, L, d))
    if ws is None:
        ws = workspace(need, Q.device, stream, kind="kv4")
    _check(lib().qoq_kv4_decode_attention(_ptr(Q), _ptr(kc), _ptr(vc), _ptr(sc), _ptr(seqlen), B,
                                          Hq, Hkv, L, d, _ptr(out), _ptr(ws),
                                          ws.numel() * ws.element_size(), _stream(stream)),
           "qoq_kv4_decode_attention")
    return out


# ---------------------------------------------------------------------------
# paged 4-bit KV cache
# ---------------------------------------------------------------------------

def _on(t, stream):
    """A context with the device of `t` as the current one and `stream` (if one
    is given) as its current stream."""
    import contextlib

    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("the inputs must be CUDA tensors")
    if stream is not None and stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(t.device))
    stack.enter_context(torch.cuda.stream(stream))
    return stack


_calls = None


def _load_calls():
    """The extension that makes calls whose arguments are all as the kernels take
    them, on the current device and stream, in a tenth of the time; it returns
    None for any other."""
    global _calls
    import torch  # noqa: F401  (its libraries come first)
    try:
        from . import _torch_calls
    except ImportError as e:
        raise RuntimeError(f"the extension _torch_calls has not been built: {e}") from e
    _calls = _torch_calls
    return _calls


def _elsewhere(t, stream):
    """Whether a call on `t` is not simply one on the current device's current
    stream.  Such a call is made again inside _on, so that its outputs and
    workspace belong to the stream it runs on."""
    import torch
    return stream is not None or t.get_device() != torch.cuda.current_device()


def _need_rows(t, name, dtype, width, device=None):
    """A CUDA tensor of rows of `width` contiguous elements, the rows any
    multiple of 16 bytes apart; returns (rows, elements between rows)."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() == 0:
        raise ValueError(f"{name} must be a CUDA tensor of rows")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    rows, at = t.shape[0], 1
    if t.is_contiguous() and rows * width == t.numel() and rows:
        return rows, width
    for size, step in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and step != at:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        at *= size
    if at != width:
        raise ValueError(f"{name} must have rows of {width} elements, got {at}")
    ld = t.stride(0) if rows > 1 else width
    if ld < width or ld * t.element_size() % 16:
        raise ValueError(f"{name}: rows must be {width} or more elements and a multiple of 16 "
                         f"bytes apart, got {ld}")
    return rows, ld


def _need_batch(cache, q_start, seqlen, block_table, dev):
    """Checks a paged cache and a ragged batch; returns (pages, Hkv, page, B, width)."""
    import torch
    kc, vc, sc = cache
    shape = getattr(sc, "shape", ())
    if len(shape) != 4 or shape[3] != 4 or shape[2] % 16:
        raise ValueError("scales must have shape (pages, Hkv, page, 4), page a multiple of 16")
    pages, Hkv, page, _ = shape
    _need_cuda(sc, "scales", torch.float16, shape=shape, device=dev)
    shape = (pages, Hkv, page // 16, 1024)
    _need_cuda(kc, "k_codes", torch.uint8, shape=shape, device=dev)
    _need_cuda(vc, "v_codes", torch.uint8, shape=shape, device=dev)
    shape = getattr(block_table, "shape", ())
    if len(shape) != 2:
        raise ValueError("block_table must have 2 dims")
    B, width = shape
    _need_cuda(block_table, "block_table", torch.int32, shape=shape, device=dev)
    _need_cuda(seqlen, "seqlen", torch.int32, shape=(B,), device=dev)
    _need_cuda(q_start, "q_start", torch.int32, shape=(B + 1,), device=dev)
    return pages, Hkv, page, B, width


def kv4_paged_bytes(pages: int, Hkv: int, page: int, d: int = 128):
    """(k_bytes, v_bytes, scale_bytes) of a paged 4-bit KV cache."""
    k, v, sc = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().qoq_kv4_paged_bytes(pages, Hkv, page, d, ctypes.byref(k), ctypes.byref(v),
                                     ctypes.byref(sc)), "qoq_kv4_paged_bytes")
    return k.value, v.value, sc.value


def kv4_paged_cache(pages: int, Hkv: int, page: int, device, d: int = 128):
    """An empty pool of `pages` pages of `page` tokens: (k_codes uint8, v_codes
    uint8, scales float16), (pages, Hkv, page // 16, 1024) twice and
    (pages, Hkv, page, 4)."""
    import torch
    kv4_paged_bytes(pages, Hkv, page, d)
    kc = torch.zeros((pages, Hkv, page // 16, 1024), dtype=torch.uint8, device=device)
    vc = torch.zeros((pages, Hkv, page // 16, 1024), dtype=torch.uint8, device=device)
    sc = torch.zeros((pages, Hkv, page, 4), dtype=torch.float16, device=device)
    return kc, vc, sc


def rope_frequencies(rot: int = 128, base: float = 10000.0, scaling=None, device="cuda"):
    """(inv_freq, factor) of a rotary embedding over `rot` dimensions: the
    radians per position of its rot / 2 pairs as a float64 tensor, and the
    factor on rotated values, for kv4_paged_append.

    scaling: None, or a dict with "type" and the type's numbers, for contexts
    longer than the trained one:
      "linear"  factor: positions divided by it
      "ntk"     factor: base * factor ** (rot / (rot - 2))
      "llama3"  factor, low_freq_factor, high_freq_factor, original_length:
                wavelengths over original_length / low_freq_factor are divided,
                those under original_length / high_freq_factor kept, those
                between interpolated
      "yarn"    factor, original_length, beta_fast (32), beta_slow (1),
                attention_factor (0.1 ln factor + 1): pairs that turn less than
                beta_slow times over the trained length divided, more than
                beta_fast times kept, a ramp between."""
    import torch
    if rot <= 0 or rot > 128 or rot % 16:
        raise ValueError("rot must be a multiple of 16 in 16 .. 128")
    if not base > 1.0:
        raise ValueError("base must be over 1")
    scaling = dict(scaling or {"type": "none"})
    kind = scaling.pop("type", None)
    allowed = {"none": (), "linear": ("factor",), "ntk": ("factor",),
               "llama3": ("factor", "low_freq_factor", "high_freq_factor", "original_length"),
               "yarn": ("factor", "original_length", "beta_fast", "beta_slow",
                        "attention_factor")}
    if kind not in allowed:
        raise ValueError(f"unknown scaling type {kind!r}")
    if set(scaling) - set(allowed[kind]):
        raise ValueError(f"{kind} scaling takes {allowed[kind]}, got {sorted(scaling)}")
    missing = set(allowed[kind]) - set(scaling) - {"beta_fast", "beta_slow", "attention_factor"}
    if missing:
        raise ValueError(f"{kind} scaling needs {sorted(missing)}")
    factor = float(scaling.get("factor", 1.0))
    if not factor > 0.0:
        raise ValueError("factor must be positive")
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2))
    freq = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
    attention = 1.0
    if kind == "linear":
        freq = [f / factor for f in freq]
    elif kind == "llama3":
        length = float(scaling["original_length"])
        low, high = float(scaling["low_freq_factor"]), float(scaling["high_freq_factor"])
        if not high > low:
            raise ValueError("high_freq_factor must be over low_freq_factor")
        turns = [length * f / (2.0 * math.pi) for f in freq]
        keep = [min(1.0, max(0.0, (t - low) / (high - low))) for t in turns]
        freq = [(1.0 - k) * f / factor + k * f for f, k in zip(freq, keep)]
    elif kind == "yarn":
        length = float(scaling["original_length"])
        fast, slow = float(scaling.get("beta_fast", 32.0)), float(scaling.get("beta_slow", 1.0))

        def pair_of(turns):   # the pair that turns so often over the trained length
            return rot * math.log(length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        lo, hi = max(0, math.floor(pair_of(fast))), min(rot - 1, math.ceil(pair_of(slow)))
        ramp = [min(1.0, max(0.0, (j - lo) / max(hi - lo, 1e-3))) for j in range(rot // 2)]
        freq = [f / factor * r + f * (1.0 - r) for f, r in zip(freq, ramp)]
        attention = float(scaling.get("attention_factor", 0.1 * math.log(factor) + 1.0
                                      if factor > 1.0 else 1.0))
    return torch.tensor(freq, dtype=torch.float64, device=device), attention


_DEFAULT_SCALE = 1.0 / math.sqrt(128.0)
_ROPE_LAYOUTS = {"half": 0, "interleaved": 1}


def kv4_paged_append(qkv, cache, q_start, seqlen, block_table, Hq: int, inv_freq=None,
                     rope_layout: str = "half", rope_factor: float = 1.0, q_out=None, values=None,
                     stream=None):
    """Rotate the queries and keys of qkv ((T, (Hq + 2 Hkv) * 128) float16, rows
    may be strided) to their positions, quantize keys and values into their
    pages, and return the queries, (T, Hq, 128) float16.

    q_start (B + 1) and seqlen (B), int32: sequence b has the rows q_start[b] ..
    q_start[b + 1] - 1, its last tokens of seqlen[b]; block_table (B, width)
    int32.  inv_freq: float64 (rot / 2) from rope_frequencies (None: no
    rotation), rope_layout "half" or "interleaved".  values: (K, V), each
    (T, Hkv, 128) float16, written with the values that the cache then holds.
    Rows of no sequence are not written (in a new tensor: they hold anything)."""
    if rope_layout not in _ROPE_LAYOUTS:
        raise ValueError(f"rope_layout must be one of {sorted(_ROPE_LAYOUTS)}")
    if stream is None:
        q = (_calls or _load_calls()).paged_append(
            qkv, cache, q_start, seqlen, block_table, Hq, inv_freq, _ROPE_LAYOUTS[rope_layout],
            rope_factor, q_out, values)
        if q is not None:
            return q
    import torch
    if not isinstance(qkv, torch.Tensor) or not qkv.is_cuda:
        raise ValueError("qkv must be a CUDA tensor")
    if _elsewhere(qkv, stream):
        with _on(qkv, stream):
            return kv4_paged_append(qkv, cache, q_start, seqlen, block_table, Hq, inv_freq,
                                    rope_layout, rope_factor, q_out, values)
    dev = qkv.device
    pages, Hkv, page, B, width = _need_batch(cache, q_start, seqlen, block_table, dev)
    T, ld = _need_rows(qkv, "qkv", torch.float16, (Hq + 2 * Hkv) * 128)
    rot = freq = k_at = v_at = 0
    if inv_freq is not None:
        _need_cuda(inv_freq, "inv_freq", torch.float64, 1, device=dev)
        rot, freq = 2 * inv_freq.shape[0], inv_freq.data_ptr()
    if values is not None:
        kh, vh = values
        _need_cuda(kh, "values[0]", torch.float16, shape=(T, Hkv, 128), device=dev)
        _need_cuda(vh, "values[1]", torch.float16, shape=(T, Hkv, 128), device=dev)
        k_at, v_at = kh.data_ptr(), vh.data_ptr()
    if q_out is None:
        q_out = qkv.new_empty((T, Hq, 128))
    else:
        _need_cuda(q_out, "q_out", torch.float16, shape=(T, Hq, 128), device=dev)
    st = lib().qoq_kv4_paged_append(
        qkv.data_ptr(), ld, T, Hq, Hkv, 128, q_start.data_ptr(), seqlen.data_ptr(), B,
        block_table.data_ptr(), width, pages, page, freq, rot, _ROPE_LAYOUTS[rope_layout],
        rope_factor, q_out.data_ptr(), cache[0].data_ptr(), cache[1].data_ptr(),
        cache[2].data_ptr(), k_at, v_at, torch.cuda.current_stream(dev).cuda_stream)
    if st:
        _check(st, "qoq_kv4_paged_append")
    return q_out


def kv4_paged_attention(Q, cache, q_start, seqlen, block_table, max_q=None, scale=None, out=None,
                        ws=None, stream=None):
    """Causal attention of the rows of Q ((T, Hq, 128) float16, rows may be
    strided) over the paged cache; returns (T, Hq, 128) float16.

    The batch as for kv4_paged_append, after the append.  max_q: the largest
    number of rows of a sequence (1 for a decode step; default: T).  scale:
    default 1 / sqrt(128).  ws: a uint8 workspace of
    kv4_paged_attention_workspace_bytes (default: allocated for the call).  Rows
    of no sequence, and of one with more than max_q, are not written (in a new
    tensor: they hold anything)."""
    scale = _DEFAULT_SCALE if scale is None else scale
    if stream is None:
        o = (_calls or _load_calls()).paged_attention(Q, cache, q_start, seqlen, block_table,
                                                      max_q, scale, out, ws)
        if o is not None:
            return o
    import torch
    if not isinstance(Q, torch.Tensor) or Q.dim() != 3 or Q.shape[2] != 128:
        raise ValueError("Q must have shape (T, Hq, 128)")
    if not Q.is_cuda:
        raise ValueError("Q must be a CUDA tensor")
    if _elsewhere(Q, stream):
        with _on(Q, stream):
            return kv4_paged_attention(Q, cache, q_start, seqlen, block_table, max_q, scale, out,
                                       ws)
    Hq, dev = Q.shape[1], Q.device
    T, ldq = _need_rows(Q, "Q", torch.float16, Hq * 128)
    pages, Hkv, page, B, width = _need_batch(cache, q_start, seqlen, block_table, dev)
    max_q = max(T, 1) if max_q is None else max_q
    if out is None:
        out = Q.new_empty((T, Hq, 128))
    else:
        _need_cuda(out, "out", torch.float16, shape=(T, Hq, 128), device=dev)
    if ws is None:
        ws = cache[0].new_empty(kv4_paged_attention_workspace_bytes(T, Hq, Hkv, B, width, page,
                                                                    max_q))
    else:
        _need_ws(ws, dev)
    st = lib().qoq_kv4_paged_attention(
        Q.data_ptr(), ldq, T, Hq, Hkv, 128, cache[0].data_ptr(), cache[1].data_ptr(),
        cache[2].data_ptr(), q_start.data_ptr(), seqlen.data_ptr(), B, block_table.data_ptr(),
        width, pages, page, max_q, scale, out.data_ptr(), ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream(dev).cuda_stream)
    if st:
        _check(st, "qoq_kv4_paged_attention")
    return out


def kv4_paged_attention_workspace_bytes(T: int, Hq: int, Hkv: int, B: int, width: int, page: int,
                                        max_q: int) -> int:
    return int(lib().qoq_kv4_paged_attention_workspace_bytes(T, Hq, Hkv, 128, B, width, page,
                                                             max_q))


def smooth_factors(Xcal, W, stream=None):
    """Per-input-channel smoothing factors (float16[K]) from a calibration
    batch Xcal (Mc, K) and the weight W (N, K), both float16 CUDA tensors."""
    import torch
    _need_cuda(Xcal, "Xcal", torch.float16, 2)
    Mc, K = Xcal.shape
    _need_cuda(W, "W", torch.float16, 2, device=Xcal.device)
    N, K2 = W.shape
    if K2 != K:
        raise ValueError("Xcal and W must have the same number of input channels")
    s = torch.empty(K, dtype=torch.float16, device=W.device)
    _check(lib().qoq_smooth_factors(_ptr(Xcal), Mc, _ptr(W), N, K, _ptr(s), _stream(stream)),
           "qoq_smooth_factors")
    return s


def quantize_weights_smoothed(W, smooth, group: int = 128, stream=None):
    """quantize_weights of W * smooth[k] (the factors folded into s1)."""
    import torch
    _need_cuda(W, "W", torch.float16, 2)
    N, K = W.shape
    _need_cuda(smooth, "smooth", torch.float16, shape=(K,), device=W.device)
    nbytes = packed_weight_bytes(N, K, group)
    if nbytes == 0:
        raise QoQError(QOQ_ERR_INVALID_ARG, "qoq_packed_weight_bytes")
    packed = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    s1 = torch.empty(N, dtype=torch.float16, device=W.device)
    _check(lib().qoq_quantize_weights_smoothed(_ptr(W), _ptr(smooth), N, K, group, _ptr(packed),
                                               _ptr(s1), _stream(stream)),
           "qoq_quantize_weights_smoothed")
    return packed, s1


def quantize_act_per_token_smoothed(X, smooth, out=None, stream=None):
    """quantize_act_per_token of X / smooth[k]."""
    import torch
    _need_cuda(X, "X", torch.float16, 2)
    M, K = X.shape
    _need_cuda(smooth, "smooth", torch.float16, shape=(K,), device=X.device)
    if out is None:
        X8 = torch.empty((M, K), dtype=torch.int8, device=X.device)
        sx = torch.empty(M, dtype=torch.float16, device=X.device)
    else:
        X8, sx = out
        _need_cuda(X8, "X8", torch.int8, shape=(M, K), device=X.device)
        _need_cuda(sx, "sx", torch.float16, shape=(M,), device=X.device)
    _check(lib().qoq_quantize_act_per_token_smoothed(_ptr(X), _ptr(smooth), M, K, _ptr(X8),
                                                     _ptr(sx), _stream(stream)),
           "qoq_quantize_act_per_token_smoothed")
    return X8, sx


_AUTO = object()


def _auto_ws(ws, M, N, K, group, device, tok_tile=0, splits=0, stream=None):
    if ws is _AUTO:
        return workspace(gemm_workspace_bytes(M, N, K, group, tok_tile, splits), device,
                         stream)
    _need_ws(ws, device)
    return ws


def w4a8_gemm(X8, sx, packed, s1, N: int, group: int = 128, out=None, ws=_AUTO, stream=None):
    """Y = (X8 . dq^T) * sx[m] * s1[n] as float16 (M, N).  `ws`: a uint8
    device tensor for the split-K workspace (default: a cached one; None:
    do not split K)."""
    import torch
    M, K = _need_gemm_operands(X8, sx, packed, s1, N, group)
    Y = _out(out, (M, N), torch.float16, X8.device)
    w, wb = _ws_args(_auto_ws(ws, M, N, K, group, X8.device, stream=stream))
    _check(lib().qoq_w4a8_gemm(_ptr(X8), _ptr(sx), _ptr(packed), _ptr(s1), M, N, K, group,
                               _ptr(Y), w, wb, _stream(stream)), "qoq_w4a8_gemm")
    return Y


def w4a8_gemm_static_ws(X8, sx, packed, s1, N: int, group: int = 128, out=None, stream=None):
    """The same GEMM without a workspace argument: the library uses its own
    fixed device array (shared by every call on the device, so calls must not
    overlap in time).  Raises QoQError (unsupported) for shapes needing more
    split-K scratch than that array holds."""
    import torch
    M, K = _need_gemm_operands(X8, sx, packed, s1, N, group)
    Y = _out(out, (M, N), torch.float16, X8.device)
    _check(lib().qoq_w4a8_gemm_static_ws(_ptr(X8), _ptr(sx), _ptr(packed), _ptr(s1), M, N, K,
                                         group, _ptr(Y), _stream(stream)),
           "qoq_w4a8_gemm_static_ws")
    return Y


def w4a8_gemm_i32(X8, packed, N: int, group: int = 128, out=None, ws=_AUTO, stream=None):
    """Raw INT32 accumulator acc = X8 . dq^T (M, N)."""
    import torch
    M, K = _need_gemm_operands(X8, None, packed, None, N, group)
    acc = _out(out, (M, N), torch.int32, X8.device)
    w, wb = _ws_args(_auto_ws(ws, M, N, K, group, X8.device, stream=stream))
    _check(lib().qoq_w4a8_gemm_i32(_ptr(X8), _ptr(packed), M, N, K, group, _ptr(acc), w, wb,
                                   _stream(stream)), "qoq_w4a8_gemm_i32")
    return acc


def w4a8_gemm_config(X8, sx, packed, s1, N: int, group: int = 128, *, tok_tile=0, splits=0,
                     int32_out=False, out=None, ws=_AUTO, stream=None):
    """The GEMM with an explicit token tile / split count (0 = auto)."""
    import torch
    if int32_out:
        M, K = _need_gemm_operands(X8, None, packed, None, N, group)
        acc = _out(out, (M, N), torch.int32, X8.device)
        Y = None
    else:
        M, K = _need_gemm_operands(X8, sx, packed, s1, N, group)
        Y = _out(out, (M, N), torch.float16, X8.device)
        acc = None
    w, wb = _ws_args(_auto_ws(ws, M, N, K, group, X8.device, tok_tile, splits, stream))
    _check(lib().qoq_w4a8_gemm_config(_ptr(X8), _ptr(sx), _ptr(packed), _ptr(s1), M, N, K, group,
                                      _ptr(Y), _ptr(acc), tok_tile, splits, w, wb,
                                      _stream(stream)), "qoq_w4a8_gemm_config")
    return acc if int32_out else Y


def w4a8_linear(X, packed, s1, N: int, group: int = 128, out=None, scratch=None, ws=_AUTO,
                stream=None):
    """Y = X . W^T: per-token activation quantization + W4A8 GEMM in one call
    (the GEMM overlaps the quantizer's tail).  ``scratch`` = (X8, sx),
    written."""
    import torch
    _need_cuda(X, "X", torch.float16, 2)
    M, K = X.shape
    dev = X.device
    _need_cuda(s1, "s1", torch.float16, shape=(N,), device=dev)
    _need_packed(packed, N, K, group, dev)
    if scratch is None:
        X8 = torch.empty((M, K), dtype=torch.int8, device=dev)
        sx = torch.empty(M, dtype=torch.float16, device=dev)
    else:
        X8, sx = scratch
        _need_cuda(X8, "X8", torch.int8, shape=(M, K), device=dev)
        _need_cuda(sx, "sx", torch.float16, shape=(M,), device=dev)
    Y = _out(out, (M, N), torch.float16, dev)
    w, wb = _ws_args(_auto_ws(ws, M, N, K, group, dev, stream=stream))
    _check(lib().qoq_w4a8_linear(_ptr(X), M, K, _ptr(packed), _ptr(s1), N, group, _ptr(X8),
                                 _ptr(sx), _ptr(Y), w, wb, _stream(stream)), "qoq_w4a8_linear")
    return Y


def w4a8_linear_fused(X, packed, s1, N: int, group: int = 128, out=None, scratch=None,
                      ws=_AUTO, stream=None):
    """w4a8_linear as one kernel that quantizes its own activations (a few
    decode rows: M * K * 2 <= 49152 and a 16-token plan without a cluster
    split; else QoQError, unsupported)."""
    import torch
    _need_cuda(X, "X", torch.float16, 2)
    M, K = X.shape
    dev = X.device
    _need_cuda(s1, "s1", torch.float16, shape=(N,), device=dev)
    _need_packed(packed, N, K, group, dev)
    if scratch is None:
        X8 = torch.empty((M, K), dtype=torch.int8, device=dev)
        sx = torch.empty(M, dtype=torch.float16, device=dev)
    else:
        X8, sx = scratch
        _need_cuda(X8, "X8", torch.int8, shape=(M, K), device=dev)
        _need_cuda(sx, "sx", torch.float16, shape=(M,), device=dev)
    Y = _out(out, (M, N), torch.float16, dev)
    # up to four rows the kernel runs its own 16-token plan (the automatic
    # plan would be the GEMV): the workspace is that plan's
    tok = 16 if M <= 4 else 0
    w, wb = _ws_args(_auto_ws(ws, M, N, K, group, dev, tok_tile=tok, stream=stream))
    _check(lib().qoq_w4a8_linear_fused(_ptr(X), M, K, _ptr(packed), _ptr(s1), N, group,
                                       _ptr(X8), _ptr(sx), _ptr(Y), w, wb, _stream(stream)),
           "qoq_w4a8_linear_fused")
    return Y


def lora_workspace_bytes(T: int, K: int, N: int, R: int, n: int) -> int:
    return int(lib().qoq_lora_workspace_bytes(T, K, N, R, n))


def lora_add(Y, X, A, B, ids, scaling, out=None, ws=None, stream=None):
    """Y[t] + scaling[a] * B[a] @ (A[a] @ X[t]) with a = ids[t] (Y[t] where
    ids[t] is outside [0, n)): the adapters of every row's request beside a
    shared projection.

    Y (T, N), X (T, K), A (n, R, K), B (n, N, R) float16, ids (T,) int32,
    scaling (n,) float32.  out: a (T, N) float16 tensor, which may be Y
    (default: a new one)."""
    if stream is None:
        o = (_calls or _load_calls()).lora_add(Y, X, A, B, ids, scaling, out, ws)
        if o is not None:
            return o
    import torch
    if not isinstance(X, torch.Tensor) or not X.is_cuda or X.dim() != 2:
        raise ValueError("X must be a CUDA tensor with 2 dims")
    if _elsewhere(X, stream):
        with _on(X, stream):
            return lora_add(Y, X, A, B, ids, scaling, out, ws)
    (T, K), dev = X.shape, X.device
    shape = getattr(B, "shape", ())
    if len(shape) != 3:
        raise ValueError("B must have 3 dims")
    n, N, R = shape
    _need_cuda(X, "X", torch.float16, shape=(T, K), device=dev)
    _need_cuda(Y, "Y", torch.float16, shape=(T, N), device=dev)
    _need_cuda(A, "A", torch.float16, shape=(n, R, K), device=dev)
    _need_cuda(B, "B", torch.float16, shape=shape, device=dev)
    _need_cuda(ids, "ids", torch.int32, shape=(T,), device=dev)
    _need_cuda(scaling, "scaling", torch.float32, shape=(n,), device=dev)
    if out is None:
        out = torch.empty_like(Y)
    elif out is not Y:
        _need_cuda(out, "out", torch.float16, shape=(T, N), device=dev)
    if ws is None:
        ws = torch.empty(lora_workspace_bytes(T, K, N, R, n), dtype=torch.uint8, device=dev)
    else:
        _need_ws(ws, dev)
    st = lib().qoq_lora_add(Y.data_ptr(), X.data_ptr(), T, K, N, A.data_ptr(), B.data_ptr(), R, n,
                            ids.data_ptr(), scaling.data_ptr(), out.data_ptr(), ws.data_ptr(),
                            ws.numel(), torch.cuda.current_stream(dev).cuda_stream)
    if st:
        _check(st, "qoq_lora_add")
    return out


class QoQLinear:
    """A linear layer y = x W^T with W stored in the packed W4 format.

    Calling it quantizes the activations per token and runs the W4A8 GEMM;
    both steps are CUDA kernels of ``libqoq.so``.  With ``adapters`` = (A, B,
    scaling) and ``ids``, every row's low-rank adapter is added (lora_add)."""

    def __init__(self, W, group: int = 128):
        self.N, self.K = W.shape
        self.group = group
        self.packed, self.s1 = quantize_weights(W, group)

    def __call__(self, X, out=None, scratch=None, stream=None, adapters=None, ids=None):
        if (adapters is None) != (ids is None):
            raise ValueError("adapters and ids go together")
        Y = w4a8_linear(X, self.packed, self.s1, self.N, self.group, out=out,
                        scratch=scratch, stream=stream)
        if adapters is not None:
            A, B, scaling = adapters
            lora_add(Y, X, A, B, ids, scaling, out=Y, stream=stream)
        return Y
