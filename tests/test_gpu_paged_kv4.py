"""The paged 4-bit KV cache ("QServe: Cuantificación W4A8KV4 ...", abstract: the
KV cache in 4 bits) against plain references in binary64.

* qoq_kv4_paged_append: the whole pool, codes and scales, must equal the pool
  before with the rows' slots replaced by the oracle's quantization of the
  binary64 rotation, bit for bit; the queries lie within half an FP16 step and
  one binary32 step of the rotated values' size.
* qoq_kv4_paged_attention: within the allowance derived in
  paged_reference.attention.
"""
import math

import numpy as np
import pytest

import paged_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU container
    pytest.skip("no CUDA device", allow_module_level=True)

import w4a8_quantized_gemm_02_b200 as qoq  # noqa: E402

DEV = torch.device("cuda:0")
D = 128


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _batch(rng, q, past, page, spare=2, pages=None):
    """(q_start, seqlen, table, pages): q[b] rows on top of past[b] tokens, every
    sequence's pages scattered over the pool."""
    q, past = np.asarray(q), np.asarray(past)
    total = q + past
    need = -(-total // page)
    pages = pages or int(need.sum()) + spare
    table = np.full((len(q), max(1, int(need.max()))), -1, np.int32)
    order = rng.permutation(pages)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return (np.concatenate([[0], np.cumsum(q)]).astype(np.int32), total.astype(np.int32), table,
            pages)


def _pool(rng, pages, Hkv, page):
    """A pool holding the quantization of random vectors."""
    kc = ref.pack(rng.integers(0, 16, (pages, Hkv, page // 16, 16, D)).astype(np.uint8), ref.K_AT)
    vc = ref.pack(rng.integers(0, 16, (pages, Hkv, page // 16, 16, D)).astype(np.uint8), ref.V_AT)
    sc = np.empty((pages, Hkv, page, 4), np.float16)
    sc[..., 0] = rng.uniform(0.1, 0.5, sc.shape[:3])
    sc[..., 1] = -rng.uniform(1.0, 4.0, sc.shape[:3])
    sc[..., 2] = rng.uniform(0.1, 0.4, sc.shape[:3])
    sc[..., 3] = -rng.uniform(1.0, 3.0, sc.shape[:3])
    return kc, vc, sc


def _append_reference(oracle, pool, qkv, q_start, seqlen, table, Hq, Hkv, freq, layout, factor):
    kc, vc, sc = (a.copy() for a in pool)
    pages, _, page = sc.shape[:3]
    k_codes, v_codes = ref.unpack(kc, ref.K_AT), ref.unpack(vc, ref.V_AT)
    T = qkv.shape[0]
    x = qkv.reshape(T, Hq + 2 * Hkv, D)
    rows = ref.rows(q_start, seqlen)
    q_out = np.full((T, Hq, D), np.nan)
    kv = {}
    for b, r, p in rows:
        y = ref.rotate(x[r:r + 1, :Hq + Hkv], [p], freq, layout, factor)[0]
        q_out[r] = y[:Hq]
        kv[r] = (y[Hq:].astype(np.float32).astype(np.float16), x[r, Hq + Hkv:])
    hat = np.full((2, T, Hkv, D), np.nan)
    for b, r, p in rows:
        both = [oracle.kv4_quant(np.ascontiguousarray(a)[None, :, None, :]) for a in kv[r]]
        for i, (q, s, m) in enumerate(both):
            hat[i, r] = q[0, :, 0] * s[0].astype(np.float64) + m[0].astype(np.float64)
        if not (0 <= p < table.shape[1] * page):
            continue
        pid = int(table[b, p // page])
        if not 0 <= pid < pages:
            continue
        slot = p % page
        k_codes[pid, :, slot // 16, slot % 16] = both[0][0][0, :, 0]
        v_codes[pid, :, slot // 16, slot % 16] = both[1][0][0, :, 0]
        for i in range(2):
            sc[pid, :, slot, 2 * i] = both[i][1][0, :, 0]
            sc[pid, :, slot, 2 * i + 1] = both[i][2][0, :, 0]
    return (ref.pack(k_codes, ref.K_AT), ref.pack(v_codes, ref.V_AT), sc), q_out, hat


def _check_pool(cache, want):
    for got, exp, name in zip(cache, want, ("k_codes", "v_codes", "scales")):
        g = got.cpu().numpy()
        if name == "scales":
            g, exp = g.view(np.uint16), exp.view(np.uint16)
        bad = np.argwhere(g != exp)
        assert bad.size == 0, f"{name}: {len(bad)} differ, first at {bad[0]}"


def _check_queries(got, want, qkv, Hq, factor):
    """Half an FP16 step, and a binary32 rounding of the two products: of the
    pair's size at most."""
    got = got.astype(np.float64)
    known = ~np.isnan(want)
    size = factor * 2.0 * np.abs(qkv.astype(np.float64)).max()
    tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2.0 ** -22 * size
    assert (np.abs(got - want)[known] <= tol[known]).all()


FREQ = {rot: 500000.0 ** (-np.arange(0, rot, 2) / rot) for rot in (16, 48, 64, 128)}

APPEND = [
    # q, past, page, Hq, Hkv, rot, layout
    ([1], [0], 16, 4, 1, 128, "half"),
    ([1, 1, 1], [0, 15, 16], 16, 4, 2, 128, "interleaved"),
    ([1] * 9, [0, 1, 7, 8, 9, 31, 32, 47, 100], 48, 5, 1, 64, "half"),
    ([17, 0, 1, 33], [0, 5, 30, 15], 32, 3, 3, 64, "interleaved"),
    ([40, 3, 130], [3, 0, 61], 64, 8, 2, 48, "half"),
    ([16, 32], [16, 0], 16, 2, 2, 0, "half"),
    ([5, 64, 64], [11, 0, 64], 128, 6, 2, 16, "interleaved"),
]


@pytest.mark.parametrize("q,past,page,Hq,Hkv,rot,layout", APPEND)
def test_append_matches_reference(oracle, q, past, page, Hq, Hkv, rot, layout):
    rng = np.random.default_rng(sum(q) + page)
    q_start, seqlen, table, pages = _batch(rng, q, past, page)
    T = int(q_start[-1])
    qkv = (rng.standard_normal((T, (Hq + 2 * Hkv) * D)) * 1.5).astype(np.float16)
    qkv.reshape(T, -1, D)[0, Hq] = 2.5          # a constant key ...
    qkv.reshape(T, -1, D)[0, Hq + Hkv] = -0.75  # ... and value
    pool = _pool(rng, pages, Hkv, page)
    cache = tuple(_dev(a) for a in pool)
    freq, factor = (FREQ[rot], 1.25) if rot else (None, 1.0)
    values = tuple(torch.empty(T, Hkv, D, dtype=torch.float16, device=DEV) for _ in range(2))
    got = qoq.kv4_paged_append(_dev(qkv), cache, _dev(q_start), _dev(seqlen), _dev(table), Hq,
                               inv_freq=None if freq is None else _dev(freq), rope_layout=layout,
                               rope_factor=factor, values=values)
    want, q_out, hat = _append_reference(oracle, pool, qkv, q_start, seqlen, table, Hq, Hkv, freq,
                                         layout, factor)
    _check_pool(cache, want)
    _check_queries(got.cpu().numpy(), q_out, qkv, Hq, factor)
    for v, h in zip(values, hat):
        # one FP32 multiply-add and the FP16 rounding
        assert (np.abs(v.cpu().numpy() - h) <= 2.0 ** -11 * np.abs(h) + 2.0 ** -20).all()


def test_append_without_rotation_is_kv4_quantize():
    """The pages of one sequence, in order, hold what kv4_quantize writes."""
    rng = np.random.default_rng(5)
    Hkv, T = 2, 64
    x = _dev(rng.standard_normal((T, (2 + 2 * Hkv) * D)).astype(np.float16))
    flat = qoq.kv4_cache(1, Hkv, T, DEV)
    k, v = (x.view(T, -1, D)[:, a:a + Hkv].permute(1, 0, 2)[None].contiguous() for a in (2, 4))
    qoq.kv4_quantize(k, v, flat)
    cache = qoq.kv4_paged_cache(4, Hkv, 16, DEV)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    qoq.kv4_paged_append(x, cache, i32([0, T]), i32([T]), i32([[0, 1, 2, 3]]), 2)
    for got, exp, per in zip(cache, flat, (1, 1, 16)):
        got = got.permute(1, 0, *range(2, got.dim())).reshape(exp.shape[1:])
        assert torch.equal(got.view(torch.uint8), exp[0].view(torch.uint8))


@pytest.mark.parametrize("pos", [(1 << 20) - 3, 131071, 12345678])
def test_append_far_positions(oracle, pos):
    rng = np.random.default_rng(pos)
    page, Hq, Hkv = 128, 2, 1
    width = pos // page + 2
    table = np.full((1, width), -1, np.int32)
    for t in range(pos, pos + 5):
        table[0, t // page] = t // page - pos // page
    qkv = rng.standard_normal((5, 4 * D)).astype(np.float16)
    pool = _pool(rng, 2, Hkv, page)
    cache = tuple(_dev(a) for a in pool)
    q_start, seqlen = np.array([0, 5], np.int32), np.array([pos + 5], np.int32)
    got = qoq.kv4_paged_append(_dev(qkv), cache, _dev(q_start), _dev(seqlen), _dev(table), Hq,
                               inv_freq=_dev(FREQ[128]))
    want, q_out, _ = _append_reference(oracle, pool, qkv, q_start, seqlen, table, Hq, Hkv,
                                       FREQ[128], "half", 1.0)
    _check_pool(cache, want)
    _check_queries(got.cpu().numpy(), q_out, qkv, Hq, 1.0)


def test_append_rows_without_a_slot(oracle):
    """Page numbers outside the pool, positions past the table and before 0, and
    rows outside every sequence: nothing else changes."""
    rng = np.random.default_rng(8)
    page, Hq, Hkv, pages = 16, 2, 1, 4
    q_start = np.array([2, 20, 24, 30, 33], np.int32)
    seqlen = np.array([18, 40, 3, 3], np.int32)     # past the table; n > seqlen
    table = np.array([[0, pages], [1, -1], [2, 2], [3, 0x7fffffff]], np.int32)
    T = 36
    qkv = rng.standard_normal((T, 4 * D)).astype(np.float16)
    pool = _pool(rng, pages, Hkv, page)
    cache = tuple(_dev(a) for a in pool)
    q_out = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device=DEV)
    qoq.kv4_paged_append(_dev(qkv), cache, _dev(q_start), _dev(seqlen), _dev(table), Hq,
                         inv_freq=_dev(FREQ[128]), q_out=q_out)
    want, q_ref, _ = _append_reference(oracle, pool, qkv, q_start, seqlen, table, Hq, Hkv,
                                       FREQ[128], "half", 1.0)
    _check_pool(cache, want)
    got = q_out.cpu().numpy()
    outside = [0, 1, 33, 34, 35]
    assert (got[outside] == 7.0).all()
    _check_queries(got, q_ref, qkv, Hq, 1.0)


def test_append_sequences_sharing_a_page(oracle):
    """Two sequences that append to different slots of one block, also of one
    word, in one call; the page is in both tables."""
    rng = np.random.default_rng(9)
    page, Hq, Hkv = 16, 2, 2
    q_start = np.arange(9, dtype=np.int32)
    seqlen = np.array([1, 9, 2, 10, 3, 11, 16, 8], np.int32)
    table = np.zeros((8, 1), np.int32)
    qkv = rng.standard_normal((8, 6 * D)).astype(np.float16)
    pool = _pool(rng, 1, Hkv, page)
    for _ in range(10):
        cache = tuple(_dev(a) for a in pool)
        qoq.kv4_paged_append(_dev(qkv), cache, _dev(q_start), _dev(seqlen), _dev(table), Hq)
        want, _, _ = _append_reference(oracle, pool, qkv, q_start, seqlen, table, Hq, Hkv, None,
                                       "half", 1.0)
        _check_pool(cache, want)


def test_append_strided_rows_and_wild_row_ranges(oracle):
    rng = np.random.default_rng(10)
    page, Hq, Hkv, T = 32, 4, 1, 50
    wide = rng.standard_normal((T, 7 * D)).astype(np.float16)
    q_start, seqlen, table, pages = _batch(rng, [20, 30], [5, 40], page)
    pool = _pool(rng, pages, Hkv, page)
    cache = tuple(_dev(a) for a in pool)
    view = _dev(wide)[:, D // 2:D // 2 + 6 * D]
    qoq.kv4_paged_append(view, cache, _dev(q_start), _dev(seqlen), _dev(table), Hq)
    want, _, _ = _append_reference(oracle, pool, wide[:, D // 2:D // 2 + 6 * D], q_start, seqlen,
                                   table, Hq, Hkv, None, "half", 1.0)
    _check_pool(cache, want)
    # ranges that are none: past the rows, negative, running backwards
    for bad in ([0, T + 1, T], [-3, 5, 2], [40, 10, 5], [T, T, T]):
        cache = tuple(_dev(a) for a in pool)
        q_out = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device=DEV)
        qoq.kv4_paged_append(view, cache, _dev(np.array(bad, np.int32)), _dev(seqlen),
                             _dev(table), Hq, q_out=q_out)
        _check_pool(cache, pool)
        assert bool((q_out == 7.0).all())


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _run_attention(rng, q, past, page, Hq, Hkv, scale=None, q_scale=1.0, max_q=None, pages=None):
    q_start, seqlen, table, pages = _batch(rng, q, past, page, pages=pages)
    T = int(q_start[-1])
    Q = (rng.standard_normal((T, Hq, D)) * q_scale).astype(np.float16)
    pool = _pool(rng, pages, Hkv, page)
    out = qoq.kv4_paged_attention(_dev(Q), tuple(_dev(a) for a in pool), _dev(q_start),
                                  _dev(seqlen), _dev(table),
                                  max_q=max(q) if max_q is None else max_q, scale=scale)
    want, tol = ref.attention(Q, *pool, q_start, seqlen, table,
                              scale if scale is not None else 1.0 / math.sqrt(D))
    return out.cpu().numpy().astype(np.float64), want, tol


def _check(got, want, tol):
    known = ~np.isnan(want)       # rows of a sequence
    tol = np.broadcast_to(tol, want.shape)[known]
    off = np.abs(got[known] - want[known])
    assert np.isfinite(got[known]).all()
    assert (off <= tol).all(), f"worst {np.max(off / np.maximum(tol, 1e-30), initial=0):.3g} of the allowance"


DECODE = [
    # past, page, Hq, Hkv
    ([0], 16, 1, 1),
    ([0, 1, 14, 15, 16, 17, 31, 32, 33], 16, 4, 1),
    ([100, 7, 64], 48, 8, 1),
    ([511, 512, 513, 30], 32, 5, 5),
    ([700, 1, 1500], 64, 6, 2),
    ([300, 40], 16, 14, 1),          # more than 8 heads a KV head
    ([90, 200], 32, 40, 2),          # more than 16
    ([5000], 128, 8, 2),
]


@pytest.mark.parametrize("past,page,Hq,Hkv", DECODE)
def test_decode_matches_reference(past, page, Hq, Hkv):
    rng = np.random.default_rng(sum(past) + Hq)
    _check(*_run_attention(rng, [1] * len(past), past, page, Hq, Hkv))


def test_decode_many_sequences():
    """More sequences than the threads that look lengths up, mixed with ones
    without rows."""
    rng = np.random.default_rng(3)
    past = rng.integers(0, 90, 300)
    past[7] = 3000
    q = [0 if b % 11 == 5 else 1 for b in range(300)]
    _check(*_run_attention(rng, q, past, 16, 2, 1))


PROMPT = [
    # q, past, page, Hq, Hkv
    ([2], [0], 16, 4, 1),
    ([3, 2], [70, 15], 16, 4, 2),            # 8 or fewer rows, masked borders
    ([4, 1, 0, 3], [40, 600, 9, 0], 32, 4, 1),   # up to 16 rows
    ([17], [0], 16, 1, 1),
    ([64], [0], 64, 4, 1),
    ([65, 1, 20], [0, 333, 100], 48, 4, 2),
    ([130, 7], [129, 1000], 128, 2, 2),
    ([33, 100], [500, 28], 16, 7, 1),
    ([300], [45], 64, 8, 1),
    ([40, 2], [3, 900], 32, 20, 1),
    ([128, 256], [0, 0], 64, 1, 1),
    ([40, 5], [3500, 2100], 64, 4, 1),       # split over the tokens
    ([9], [1500], 16, 17, 1),
    ([70, 3, 20], [1100, 0, 5000], 32, 4, 1),
]


@pytest.mark.parametrize("q,past,page,Hq,Hkv", PROMPT)
def test_prompt_matches_reference(q, past, page, Hq, Hkv):
    rng = np.random.default_rng(sum(q) + sum(past))
    _check(*_run_attention(rng, q, past, page, Hq, Hkv))
    assert qoq.device_error() == 0


@pytest.mark.parametrize("q,past", [([1, 1], [800, 33]), ([90], [200]), ([50], [2500])])
def test_attention_saturated_scores(q, past):
    """Scores of hundreds: the softmax picks few tokens and its maximum keeps
    rising."""
    rng = np.random.default_rng(12)
    got, want, tol = _run_attention(rng, q, past, 32, 4, 1, q_scale=60.0)
    # the FP32 score error grows with the scores: 60 times the allowance
    _check(got, want, tol + 59 * 5e-5 * np.abs(np.nan_to_num(want)).max() + 59 * 5e-5 * 3.0)


@pytest.mark.parametrize("scale", [0.0, -0.07, 0.5])
def test_attention_scale(scale):
    rng = np.random.default_rng(13)
    got, want, tol = _run_attention(rng, [1, 40], [300, 50], 16, 4, 1, scale=scale)
    # scores are |scale| sqrt(128) times the default's
    _check(got, want, tol * max(1.0, abs(scale) * math.sqrt(D)))


def test_attention_rows_that_see_nothing_and_absent_pages():
    """Rows before position 0, sequences of length 0 or less, pages outside the
    pool, a table shorter than the length: zeros where nothing is seen; rows of
    no sequence stay as they were."""
    rng = np.random.default_rng(14)
    page, Hq, Hkv, pages = 16, 4, 2, 6
    pool = _pool(rng, pages, Hkv, page)
    cache = tuple(_dev(a) for a in pool)
    cases = [
        # q, seqlen
        ([1, 1, 1, 1], [0, -5, 20, 64]),
        ([6, 2, 40, 3], [4, 0, 38, 50]),
        ([30, 30, 1, 1], [20, 70, 33, 1]),
    ]
    table = np.array([[-1, -1, -1], [pages, 0, 1], [2, -1, 3], [4, 5, 1 << 30]], np.int32)
    for q, seqlen in cases:
        q_start = (2 + np.concatenate([[0], np.cumsum(q)])).astype(np.int32)
        T = int(q_start[-1]) + 3
        Q = rng.standard_normal((T, Hq, D)).astype(np.float16)
        seqlen = np.array(seqlen, np.int32)
        out = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device=DEV)
        qoq.kv4_paged_attention(_dev(Q), cache, _dev(q_start), _dev(seqlen), _dev(table), out=out)
        want, tol = ref.attention(Q, *pool, q_start, seqlen, table, 1.0 / math.sqrt(D))
        got = out.cpu().numpy().astype(np.float64)
        _check(got, want, tol)
        assert (got[np.isnan(want)] == 7.0).all()


def test_attention_ignores_what_lies_past_the_length():
    """Slots behind the last token hold NaN and infinite scales; entries of the
    table behind the last page are absurd."""
    rng = np.random.default_rng(15)
    page, Hq, Hkv = 32, 4, 1
    for q in ([1, 1], [50, 21]):
        q_start, seqlen, table, pages = _batch(rng, q, [70, 3], page)
        pool = _pool(rng, pages, Hkv, page)
        T = int(q_start[-1])
        Q = rng.standard_normal((T, Hq, D)).astype(np.float16)
        wide = np.full((2, table.shape[1] + 4), 1 << 29, np.int32)
        wide[:, :table.shape[1]] = table
        dirty = pool[2].copy()
        for b in range(2):
            used = int(seqlen[b])
            for p in range(-(-used // page)):
                dirty[table[b, p], :, max(0, used - p * page):] = \
                    rng.choice([np.nan, np.inf, -np.inf], (Hkv, page - min(page, used - p * page), 4))
        clean, tol = ref.attention(Q, *pool, q_start, seqlen, table, 1.0 / math.sqrt(D))
        out = qoq.kv4_paged_attention(_dev(Q), (_dev(pool[0]), _dev(pool[1]), _dev(dirty)),
                                      _dev(q_start), _dev(seqlen), _dev(wide), max_q=max(q))
        _check(out.cpu().numpy().astype(np.float64), clean, tol)


def test_attention_leaves_sequences_over_max_q():
    rng = np.random.default_rng(16)
    q_start, seqlen, table, pages = _batch(rng, [1, 5, 1], [50, 60, 70], 16)
    pool = _pool(rng, pages, 1, 16)
    Q = rng.standard_normal((7, 4, D)).astype(np.float16)
    out = torch.full((7, 4, D), 7.0, dtype=torch.float16, device=DEV)
    qoq.kv4_paged_attention(_dev(Q), tuple(_dev(a) for a in pool), _dev(q_start), _dev(seqlen),
                            _dev(table), max_q=1, out=out)
    want, tol = ref.attention(Q, *pool, q_start, seqlen, table, 1.0 / math.sqrt(D))
    got = out.cpu().numpy().astype(np.float64)
    assert (got[1:6] == 7.0).all()
    _check(got[[0, 6]], want[[0, 6]], tol[[0, 6]])


def test_append_then_attention_in_a_captured_graph(oracle):
    """A decode step, rotation and append and then attention over what was
    appended, captured once and replayed as the sequences grow; two graphs with
    their own workspaces replayed at once on two streams give what they give one
    after the other."""
    rng = np.random.default_rng(17)
    page, Hq, Hkv, B = 16, 8, 2, 5
    past = np.array([0, 15, 700, 31, 1200])
    q_start, seqlen, table, pages = _batch(rng, [8] * B, past, page)
    q_start = np.arange(B + 1, dtype=np.int32)
    pool = _pool(rng, pages, Hkv, page)
    freq = _dev(FREQ[128])

    class Step:
        def __init__(self):
            self.cache = tuple(_dev(a) for a in pool)
            self.qkv = torch.empty(B, (Hq + 2 * Hkv) * D, dtype=torch.float16, device=DEV)
            self.len = _dev((past + 1).astype(np.int32))
            self.start, self.table = _dev(q_start), _dev(table)
            self.stream = torch.cuda.Stream()
            self.graph = torch.cuda.CUDAGraph()
            self.qkv.zero_()
            torch.cuda.synchronize()
            with torch.cuda.graph(self.graph, stream=self.stream):
                q = qoq.kv4_paged_append(self.qkv, self.cache, self.start, self.len, self.table,
                                         Hq, inv_freq=freq)
                self.out = qoq.kv4_paged_attention(q, self.cache, self.start, self.len,
                                                   self.table, max_q=1)

    steps = [Step(), Step()]
    x = [rng.standard_normal((4, B, (Hq + 2 * Hkv) * D)).astype(np.float16) for _ in steps]
    want_pools = [pool, pool]
    for t in range(4):
        for s, data in zip(steps, x):
            s.qkv.copy_(_dev(data[t]))
            s.len.copy_(_dev((past + 1 + t).astype(np.int32)))
        torch.cuda.synchronize()
        for s in steps:
            with torch.cuda.stream(s.stream):
                s.graph.replay()
        torch.cuda.synchronize()
        for i, s in enumerate(steps):
            now = (past + 1 + t).astype(np.int32)
            want_pools[i], q_ref, _ = _append_reference(oracle, want_pools[i], x[i][t], q_start,
                                                        now, table, Hq, Hkv, FREQ[128], "half", 1.0)
            _check_pool(s.cache, want_pools[i])
            # the attention's own query: rotated and rounded to FP16
            q16 = q_ref.astype(np.float32).astype(np.float16)
            want, tol = ref.attention(q16, *want_pools[i], q_start, now, table, 1 / math.sqrt(D))
            # a query half an FP16 step off (2^-11 relative) moves a score by at most
            # 2^-11 sum |q k^| scale, and an output by twice that times max |v^|; a
            # binary32 rotation rounds to another FP16 value once in thousands
            slack = 2.0 * 2.0 ** -11 * 3.0
            _check(s.out.cpu().numpy().astype(np.float64), want, tol + slack)


def test_calls_on_another_stream():
    """Inputs of one stream used on another that waits for it, outputs read back
    after the reverse wait; the default workspace belongs to the call's stream."""
    rng = np.random.default_rng(18)
    q_start, seqlen, table, pages = _batch(rng, [1] * 4, [900, 20, 3, 2000], 32)
    pool = _pool(rng, pages, 2, 32)
    Q = rng.standard_normal((4, 8, D)).astype(np.float16)
    args = (_dev(Q), tuple(_dev(a) for a in pool), _dev(q_start), _dev(seqlen), _dev(table))
    base = qoq.kv4_paged_attention(*args, max_q=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [qoq.kv4_paged_attention(*args, max_q=1, stream=side) for _ in range(5)]
    torch.cuda.current_stream().wait_stream(side)
    for o in outs:
        assert torch.equal(o, base)


def test_attention_is_deterministic_and_takes_strided_queries():
    rng = np.random.default_rng(19)
    q_start, seqlen, table, pages = _batch(rng, [1, 70, 1], [900, 20, 3], 32)
    pool = tuple(_dev(a) for a in _pool(rng, pages, 2, 32))
    T = int(q_start[-1])
    qkv = _dev(rng.standard_normal((T, 12 * D)).astype(np.float16))
    view = qkv.view(T, 12, D)[:, :8]
    args = (pool, _dev(q_start), _dev(seqlen), _dev(table))
    a = qoq.kv4_paged_attention(view, *args)
    b = qoq.kv4_paged_attention(view.contiguous(), *args)
    assert torch.equal(a, b)
    for _ in range(3):
        assert torch.equal(a, qoq.kv4_paged_attention(view, *args))


def test_empty_calls():
    cache = qoq.kv4_paged_cache(2, 1, 16, DEV)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    none = torch.empty(0, 4 * D, dtype=torch.float16, device=DEV)
    q = qoq.kv4_paged_append(none, cache, i32([0, 0]), i32([3]), i32([[0]]), 2)
    assert q.shape == (0, 2, D)
    assert qoq.kv4_paged_attention(q, cache, i32([0, 0]), i32([3]), i32([[0]])).shape == (0, 2, D)
    x = torch.zeros(3, 4 * D, dtype=torch.float16, device=DEV)
    table = torch.empty(0, 1, dtype=torch.int32, device=DEV)
    seqlen = torch.empty(0, dtype=torch.int32, device=DEV)
    q = qoq.kv4_paged_append(x, cache, i32([0]), seqlen, table, 2)
    qoq.kv4_paged_attention(q, cache, i32([0]), seqlen, table)
    torch.cuda.synchronize()
    assert int(cache[0].sum()) == 0
