"""Prompt attention over more slots than are put in order (128) or than the threads that list
them take in one turn, and over more sequences than are held in shared memory (1024)."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU container
    pytest.skip("no CUDA device", allow_module_level=True)

import paged_exact as exact  # noqa: E402
import w4a8_quantized_gemm_02_b200 as qoq  # noqa: E402

D = 128


def _batch(kind):
    rng = np.random.default_rng(len(kind))
    if kind == "one long prompt":                 # 131 slots, the longer ones split
        return [8300], [0], 4, 1
    if kind == "many short chunks":               # 130 sequences of 24 rows
        return [3] * 130, rng.integers(0, 400, 130).tolist(), 8, 1
    if kind == "many and one long":               # past 128 slots, few of them split
        return [5] * 150 + [20], rng.integers(0, 40, 150).tolist() + [9000], 8, 2
    # more than 1024 sequences: single tokens, chunks, ones without rows
    q = [(1, 3, 0, 1, 40)[b % 5] if b % 50 < 5 else 1 for b in range(1100)]
    return q, rng.integers(0, 60, 1100).tolist(), 8, 1


@pytest.mark.parametrize("kind", ["one long prompt", "many short chunks", "many and one long",
                                  "over 1024 sequences"])
def test_matches_reference(kind):
    q, past, Hq, Hkv = _batch(kind)
    rng = np.random.default_rng(7)
    total = np.maximum(np.add(q, past), 1)
    kc, vc, sc, table = exact.pool_of(
        rng, total, 64, Hkv, lambda b, t: rng.uniform(0.1, 0.5, t),
        lambda b, t: -rng.uniform(1.0, 4.0, t), lambda b, t: rng.uniform(0.1, 0.4, t),
        lambda b, t: -rng.uniform(1.0, 3.0, t))
    q_start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    seqlen = np.add(q, past).astype(np.int32)
    Q = rng.choice([0.5, 0.0, -0.5], (int(q_start[-1]), Hq, D)).astype(np.float16)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    got = qoq.kv4_paged_attention(dev(Q), (dev(kc), dev(vc), dev(sc)), dev(q_start), dev(seqlen),
                                  dev(table), max_q=max(q)).double()
    want, tol = exact.attention(Q, kc, vc, sc, q_start, seqlen, table, 1.0 / math.sqrt(D))
    worst = float(((got - want).abs() / tol).max())
    assert worst <= 1.0, f"{worst:.3g} of the allowance"
    assert qoq.device_error() == 0
