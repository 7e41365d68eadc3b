"""Paged attention over values of any size: the cache's scales reach from FP16's smallest
numbers to its largest, and a row's weight may lie on one token or be spread over many that
are thousands of times lighter.  Neither may cost the weights their digits."""
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
SCALE = 1.0 / math.sqrt(D)


def _queries(rng, T, Hq, a=0.5):
    """0 and +-a, more of them positive: exact in every format of the kernels."""
    return (rng.choice([a, a, a, 0.0, -a], (T, Hq, D))).astype(np.float16)


def _run(rng, q, past, Hq, Hkv, page, v_scale, v_offset, rise, codes=(0, 16)):
    """rise(sequence, tokens): the score of every token in log2 units, about (by the keys'
    offset: the mean query sums to 128 * 0.2)."""
    total = np.add(q, past)
    per = SCALE * math.log2(math.e) * 128 * 0.2
    kc, vc, sc, table = exact.pool_of(
        rng, total, page, Hkv, lambda b, t: np.full(t, 0.02), lambda b, t: rise(b, t) / per - 0.15,
        v_scale, v_offset, codes)
    q_start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    seqlen = total.astype(np.int32)
    Q = _queries(rng, int(q_start[-1]), Hq)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    got = qoq.kv4_paged_attention(dev(Q), (dev(kc), dev(vc), dev(sc)), dev(q_start), dev(seqlen),
                                  dev(table), max_q=max(q)).double()
    want, tol = exact.attention(Q, kc, vc, sc, q_start, seqlen, table, SCALE)
    # (FP16 ends at 65504 and rounds to infinity from 65520 on: with scales of 8736, the FP16
    # number next to 8732, and offsets of -65504 a code of 15 stands for 65536)
    over = want.abs() - tol >= 65520.0
    assert bool((got[over] == want[over].sign() * math.inf).all())
    near = ~over & (want.abs() + tol >= 65520.0)
    got = torch.where(over | near & got.isinf(), want, got)
    assert bool(torch.isfinite(got).all())
    worst = float(((got - want).abs() / tol).max())
    assert worst <= 1.0, f"{worst:.3g} of the allowance"
    assert qoq.device_error() == 0


# q, past, Hq, Hkv: the single-token kernel with 4, 8 and 16 rows, whole and split over many
# CTAs; the prompt kernel, whole and split
SHAPES = [
    ([1], [0], 4, 1), ([1, 1], [700, 4095], 4, 1), ([1], [32767], 8, 2), ([1], [9000], 8, 1),
    ([1], [5000], 16, 1), ([3], [600], 4, 1),
    ([128], [0], 1, 1), ([65, 300], [64, 4000], 4, 1), ([40], [32000], 4, 1), ([20], [700], 16, 2),
]
SPREAD = {
    "flat": lambda b, t: np.zeros(t),
    "sink 12": lambda b, t: 12.0 * (np.arange(t) == 0),
    "sink 20": lambda b, t: 20.0 * (np.arange(t) == 0),
    "late sink": lambda b, t: 16.0 * (np.arange(t) == min(t - 1, 417)),
}


@pytest.mark.parametrize("spread", SPREAD)
@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 1e-4, 1e4])
@pytest.mark.parametrize("q,past,Hq,Hkv", SHAPES)
def test_values_of_every_size(q, past, Hq, Hkv, size, spread):
    rng = np.random.default_rng(sum(past) + Hq + int(size * 1e4))
    s = size * 0.3
    _run(rng, q, past, Hq, Hkv, 64, lambda b, t: s * rng.uniform(0.7, 1.3, t),
         lambda b, t: -7.0 * s * rng.uniform(0.8, 1.2, t), SPREAD[spread])


@pytest.mark.parametrize("kind", ["spread", "light sink", "heavy but far", "heavy later", "constant",
                                  "largest"])
@pytest.mark.parametrize("q,past,Hq,Hkv", SHAPES)
def test_values_of_different_sizes_in_a_row(q, past, Hq, Hkv, kind):
    rng = np.random.default_rng(sum(past) + Hq)
    every = lambda t, v: np.full(t, v)  # noqa: E731
    flat = SPREAD["flat"]
    if kind == "spread":                 # scales over 20 powers of two
        scale, rise = (lambda b, t: 2.0 ** rng.uniform(-18, 2, t)), flat
    elif kind == "light sink":           # the token that has the weight has hardly a value
        scale = lambda b, t: np.where(np.arange(t) == 0, 2.0 ** -18, 0.3)  # noqa: E731
        rise = SPREAD["sink 12"]
    elif kind == "heavy but far":        # large values that no row attends to
        scale = lambda b, t: np.where(np.arange(t) % 97 == 5, 8000.0, 1e-3)  # noqa: E731
        rise = lambda b, t: -60.0 * (np.arange(t) % 97 == 5)  # noqa: E731
    elif kind == "heavy later":          # ... growing over the sequence
        scale, rise = (lambda b, t: 2.0 ** np.linspace(-20, 8, t)), flat
    elif kind == "constant":             # vectors of one value: their scale is 0
        scale, rise = (lambda b, t: np.where(np.arange(t) % 3 == 0, 0.0, 1e-3)), flat
    else:                                # the largest scale of a finite vector
        scale, rise = (lambda b, t: every(t, 8732.0)), flat
    offset = {"constant": lambda b, t: rng.uniform(-2.0, 2.0, t),
              "largest": lambda b, t: every(t, -65504.0)}.get(kind, lambda b, t: every(t, 0.0))
    _run(rng, q, past, Hq, Hkv, 32, scale, offset, rise)


def test_constant_values_only():
    """Every scale 0: the outputs are averages of the offsets."""
    rng = np.random.default_rng(5)
    for q, past in (([1], [900]), ([70], [900])):
        _run(rng, q, past, 4, 1, 16, lambda b, t: np.zeros(t), lambda b, t: rng.uniform(-2.0, 2.0, t),
             SPREAD["sink 12"])


@pytest.mark.parametrize("q,past,Hq,Hkv", SHAPES)
def test_negative_scales(q, past, Hq, Hkv):
    """Scales that no append writes, but a caller's own cache may hold."""
    rng = np.random.default_rng(sum(past))
    _run(rng, q, past, Hq, Hkv, 32, lambda b, t: rng.choice([-0.4, -0.3, 0.2], t),
         lambda b, t: rng.uniform(-1.0, 1.0, t), SPREAD["sink 12"])
