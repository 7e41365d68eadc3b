"""Refusals of qoq_lora_add and its workspace sizes, on the host."""
import ctypes

import pytest

import w4a8_quantized_gemm_02_b200 as qoq

FAKE = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def L():
    return qoq.lib()


def _add(L, Y=FAKE, X=FAKE, T=3, K=256, N=128, A=FAKE, B=FAKE, R=16, n=2, ids=FAKE, s=FAKE,
         out=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return L.qoq_lora_add(Y, X, T, K, N, A, B, R, n, ids, s, out, ws, ws_bytes, None)


def test_refusals(L):
    for name in ("Y", "X", "A", "B", "ids", "s", "out"):
        assert _add(L, **{name: None}) == qoq.QOQ_ERR_INVALID_ARG, name
        odd = ctypes.c_void_p(0x10002)
        assert _add(L, **{name: odd}) == qoq.QOQ_ERR_INVALID_ARG, name
    for bad in (dict(T=-1), dict(K=0), dict(K=200), dict(N=0), dict(N=100), dict(R=0), dict(n=0)):
        assert _add(L, **bad) == qoq.QOQ_ERR_INVALID_ARG, bad
    for bad in (dict(R=12), dict(R=136), dict(K=133248), dict(T=(1 << 20) + 1),
                dict(n=4097)):
        assert _add(L, **bad) == qoq.QOQ_ERR_UNSUPPORTED, bad
    need = L.qoq_lora_workspace_bytes(3, 256, 128, 16, 2)
    for bad in (dict(ws=None), dict(ws=ctypes.c_void_p(0x10008)), dict(ws_bytes=need - 1)):
        assert _add(L, **bad) == qoq.QOQ_ERR_WORKSPACE, bad
    assert _add(L, T=0, ws=None, ws_bytes=0) == qoq.QOQ_OK


def test_workspace(L):
    f = L.qoq_lora_workspace_bytes
    assert f(0, 256, 128, 16, 2) == 0 and f(4, 200, 128, 16, 2) == 0
    for T, K, R, n in ((1, 128, 8, 1), (48, 8192, 32, 64), (2500, 14336, 64, 6),
                       (1 << 20, 256, 128, 3), (4096, 256, 128, 4096)):
        need = f(T, K, 128, R, n)
        # h in two FP16 parts and a factor a row, a row list a unit
        assert T * (4 * R + 4) <= need <= T * (4 * (R + 31) + 4) + (T + 256) * 264 + 1024
