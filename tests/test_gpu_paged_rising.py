"""Paged attention where the running maximum rises at every half step of 64 tokens,
or never again after the first: every raise waits for the products issued before it
and rescales them."""
import math

import numpy as np
import pytest

import paged_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a8_quantized_gemm_02_b200 as qoq  # noqa: E402

D = 128


@pytest.mark.parametrize("rise", [0.44, 0.05, -0.44])
@pytest.mark.parametrize("q,past,Hq,Hkv", [
    ([1], [1500], 4, 1), ([1], [1500], 16, 1), ([128], [0], 1, 1), ([70], [1500], 4, 1),
    ([40], [3500], 4, 2), ([300], [45], 8, 1), ([64, 1, 9], [700, 2000, 333], 4, 1)])
def test_maximum_that_moves(q, past, Hq, Hkv, rise):
    """`rise`: of the keys' offset over 64 tokens, 5 in the score for 0.44."""
    page = 32
    rng = np.random.default_rng(sum(past) + Hq)
    total = np.add(q, past)
    need = -(-total // page)
    width, pages = int(need.max()), int(need.sum())
    table = np.full((len(q), width), -1, np.int32)
    order = rng.permutation(pages)
    shape = (pages, Hkv, page // 16, 16, D)
    kc = ref.pack(rng.integers(0, 16, shape).astype(np.uint8), ref.K_AT)
    vc = ref.pack(rng.integers(0, 16, shape).astype(np.uint8), ref.V_AT)
    sc = np.empty((pages, Hkv, page, 4), np.float16)
    sc[..., 0] = 0.02
    sc[..., 2] = rng.uniform(0.1, 0.4, sc.shape[:3])
    sc[..., 3] = -rng.uniform(1.0, 3.0, sc.shape[:3])
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        t = np.arange(n * page).reshape(n, 1, page)
        sc[table[b, :n], :, :, 1] = np.broadcast_to(rise * t / 64.0, (n, Hkv, page))
    q_start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    Q = (1.0 + 0.1 * rng.standard_normal((int(q_start[-1]), Hq, D))).astype(np.float16)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    seqlen = total.astype(np.int32)
    got = qoq.kv4_paged_attention(dev(Q), (dev(kc), dev(vc), dev(sc)), dev(q_start), dev(seqlen),
                                  dev(table), max_q=max(q)).cpu().numpy().astype(np.float64)
    want, tol = ref.attention(Q, kc, vc, sc, q_start, seqlen, table, 1.0 / math.sqrt(D))
    # scores reach 2^9 in log2 units, where FP32 rounds by 2^-16: three roundings, 2^-14.4 or
    # 3.2e-5 of a weight; the single-token kernel's queries are fixed point, half a unit of
    # 1.6 / 32512, by codes of up to 15 * 0.02 in 128 dimensions and the scale: at most
    # 8.4e-5; twice their sum (numerator and denominator) is under 2^-12 of the values
    vmax = float((15 * sc[..., 2].astype(np.float64)).max() + 3.0)
    off = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (off <= tol + 2.0 ** -12 * vmax).all(), float((off - tol).max() / vmax)
    assert qoq.device_error() == 0
