"""Infinities and NaN in the paged cache and in queries stay with the rows that see them."""
import math

import numpy as np
import pytest

import paged_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU container
    pytest.skip("no CUDA device", allow_module_level=True)

import w4a8_quantized_gemm_02_b200 as qoq  # noqa: E402

D = 128


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _case(rng, q, past, page, Hq, Hkv):
    total = np.add(q, past)
    need = -(-total // page)
    pages = int(need.sum()) + 1
    table = np.full((len(q), int(need.max())), -1, np.int32)
    order, at = rng.permutation(pages), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (pages, Hkv, page // 16, 16, D)
    kc = ref.pack(rng.integers(0, 16, shape).astype(np.uint8), ref.K_AT)
    vc = ref.pack(rng.integers(0, 16, shape).astype(np.uint8), ref.V_AT)
    sc = np.empty((pages, Hkv, page, 4), np.float16)
    sc[..., 0] = rng.uniform(0.1, 0.5, sc.shape[:3])
    sc[..., 1] = -rng.uniform(1.0, 4.0, sc.shape[:3])
    sc[..., 2] = rng.uniform(0.1, 0.4, sc.shape[:3])
    sc[..., 3] = -rng.uniform(1.0, 3.0, sc.shape[:3])
    q_start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    Q = rng.standard_normal((int(q_start[-1]), Hq, D)).astype(np.float16)
    return Q, kc, vc, sc, q_start, total.astype(np.int32), table


def _attend(c, max_q):
    Q, kc, vc, sc, q_start, seqlen, table = (_dev(a) for a in c)
    out = qoq.kv4_paged_attention(Q, (kc, vc, sc), q_start, seqlen, table, max_q=max_q)
    return out.cpu().numpy().astype(np.float64)


# (up to 16 rows: the single-token kernel; more: the prompt kernel, whole and split)
SHAPES = [([5], [90], 2, 1), ([4], [2000], 4, 2), ([70], [0], 4, 1), ([70, 130], [333, 1], 4, 2),
          ([60], [3000], 4, 1)]


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("q,past,Hq,Hkv", SHAPES)
def test_a_token_is_not_seen_by_earlier_rows(q, past, Hq, Hkv, which, bad):
    """A scale or offset of one query token is no number (its codes are then 0, as the quantizer
    leaves them): the rows before it are what they are without it, the rows from it on are no
    numbers either."""
    rng = np.random.default_rng(sum(q) + which)
    page = 32
    case = _case(rng, q, past, page, Hq, Hkv)
    Q, kc, vc, sc, q_start, seqlen, table = case
    want, tol = ref.attention(Q, kc, vc, sc, q_start, seqlen, table, 1 / math.sqrt(D))
    dirty, first = sc.copy(), []
    ck, cv = ref.unpack(kc, ref.K_AT), ref.unpack(vc, ref.V_AT)
    for b in range(len(q)):
        i = q[b] // 2 + 1
        first.append(i)
        t = past[b] + i
        dirty[table[b, t // page], :, t % page, which] = bad
        for c in (ck, cv):
            c[table[b, t // page], :, t % page // 16, t % 16] = 0
    got = _attend((Q, ref.pack(ck, ref.K_AT), ref.pack(cv, ref.V_AT), dirty, q_start, seqlen, table),
                  max(q))
    for b in range(len(q)):
        lo, mid, hi = q_start[b], q_start[b] + first[b], q_start[b + 1]
        assert np.isfinite(got[lo:mid]).all()
        assert (np.abs(got[lo:mid] - want[lo:mid]) <= tol[lo:mid]).all()
        if which in (0, 2) or which == 1 and bad != bad:
            assert np.isnan(got[mid:hi]).all()            # 0 * inf, or a NaN
        elif which == 3:
            assert (~np.isfinite(got[mid:hi])).all()
        # (an infinite offset of a key makes its score infinite: with a negative one the token
        # has no weight)
    assert qoq.device_error() == 0


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("q,past,Hq,Hkv", [([1], [3], 4, 1), ([1, 1, 1], [900, 40, 5000], 4, 2),
                                           ([3], [4000], 4, 1)] + SHAPES)
def test_queries_that_are_no_numbers(q, past, Hq, Hkv, bad):
    """The row is NaN (scores inf - inf), the others are what they were."""
    rng = np.random.default_rng(sum(past) + 1)
    case = _case(rng, q, past, 16, Hq, Hkv)
    want, tol = ref.attention(*case, 1 / math.sqrt(D))
    Q, hit = case[0].copy(), np.zeros(case[0].shape[:2], bool)
    for r in range(0, Q.shape[0], 3):
        h = int(rng.integers(0, Hq))
        Q[r, h, int(rng.integers(0, D))] = bad
        hit[r, h] = True
    got = _attend((Q, *case[1:]), max(q))
    assert np.isnan(got[hit]).all()
    assert (np.abs(got - want)[~hit] <= np.broadcast_to(tol, want.shape)[~hit]).all()


def test_keys_that_are_no_numbers_at_all():
    """Every key of a sequence is NaN, and of another none."""
    rng = np.random.default_rng(3)
    for q in ([1, 1], [40, 50]):
        case = _case(rng, q, [700, 700], 16, 4, 1)
        want, tol = ref.attention(*case, 1 / math.sqrt(D))
        sc = case[3].copy()
        sc[case[6][0]] = np.nan
        got = _attend((*case[:3], sc, *case[4:]), max(q))
        n = q[0]
        assert np.isnan(got[:n]).all()
        assert (np.abs(got[n:] - want[n:]) <= tol[n:]).all()


@pytest.mark.parametrize("which", [2, 3])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("q,past,Hq,Hkv", [([1], [127], 4, 1), ([1], [5000], 8, 2), ([3], [700], 4, 1),
                                           ([40], [300], 4, 1), ([40], [6000], 4, 1)])
def test_a_value_with_hardly_any_weight_counts(q, past, Hq, Hkv, bad, which):
    """The value that is no number stands among tokens 2^-200 below the others, alone in their
    part of the sums: any weight of it is too much."""
    rng = np.random.default_rng(9)
    page = 16
    Q, kc, vc, sc, q_start, seqlen, table = _case(rng, q, past, page, Hq, Hkv)
    Q[:] = rng.choice([0.5, 0.25], Q.shape)
    sc[..., 0], sc[..., 1] = 0.01, 0.0
    for t in range(32):
        sc[table[0, t // page], :, t % page, 1] = -200 / (math.log2(math.e) / math.sqrt(D) * 48)
    sc[table[0, 0], :, 5, which] = bad
    assert np.isnan(_attend((Q, kc, vc, sc, q_start, seqlen, table), max(q))).all()
