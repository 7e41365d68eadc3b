"""Prompt chunks with rows that see no token, whole slots of 256 rows among them: zeros, and
what lies beside them as ever.  (A slot without tokens has no products to wait for: its rows
must not be staged where other warps still put their queries.)"""
import numpy as np
import pytest


pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU container
    pytest.skip("no CUDA device", allow_module_level=True)

import paged_exact as exact  # noqa: E402
import w4a8_quantized_gemm_02_b200 as qoq  # noqa: E402

D = 128


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 1), (8, 2)])
@pytest.mark.parametrize("q,seqlen", [
    ([40], [0]), ([300], [-5]), ([300], [7]), ([600], [200]), ([257], [1]),
    ([40, 300, 300], [0, -5, 7]), ([129, 1, 64], [0, 0, 64]), ([50, 50], [3000, 0])])
def test_rows_that_see_nothing_are_zero(q, seqlen, Hq, Hkv):
    rng = np.random.default_rng(sum(q) + Hq)
    total = np.maximum(seqlen, 1)
    every = lambda v: lambda b, t: np.full(t, v)  # noqa: E731
    kc, vc, sc, table = exact.pool_of(rng, total, 16, Hkv, every(0.3), every(-2.2), every(0.25),
                                      every(-1.9))
    q_start = (1 + np.concatenate([[0], np.cumsum(q)])).astype(np.int32)
    T, lens = int(q_start[-1]) + 2, np.array(seqlen, np.int32)
    Q = rng.choice([96.0, -96.0], (T, Hq, D)).astype(np.float16)     # (not to be taken for a zero)
    scale = 0.001
    want, tol = exact.attention(Q, kc, vc, sc, q_start, lens, table, scale)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    args = (dev(Q), (dev(kc), dev(vc), dev(sc)), dev(q_start), dev(lens), dev(table))
    pos = np.concatenate([np.arange(s - n, s) for n, s in zip(q, seqlen)])
    blind = torch.from_numpy(1 + np.nonzero(pos < 0)[0]).cuda()
    for _ in range(5):
        out = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
        qoq.kv4_paged_attention(*args, scale=scale, out=out)
        assert bool((out[blind] == 0.0).all())
        assert bool((out[[0, T - 2, T - 1]] == 7.0).all())
        rows = slice(1, T - 2)
        assert bool(((out[rows].double() - want[rows]).abs() <= tol[rows]).all())
    assert qoq.device_error() == 0
