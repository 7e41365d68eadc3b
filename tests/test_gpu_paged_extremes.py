"""Calls of the paged cache that its documentation allows and that are far from an ordinary
step: a captured mixed batch whose lengths change from replay to replay, a pool past 2^32
bytes, row ranges that are none, lengths at the ends of int32."""
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


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _pool(rng, total, page, Hkv):
    return exact.pool_of(rng, total, page, Hkv, lambda b, t: rng.uniform(0.1, 0.5, t),
                         lambda b, t: -rng.uniform(1.0, 4.0, t),
                         lambda b, t: rng.uniform(0.1, 0.4, t),
                         lambda b, t: -rng.uniform(1.0, 3.0, t))


def test_mixed_batches_in_captured_graphs():
    """One graph for every batch of up to 4 sequences and 430 rows: prompts, chunks, single
    tokens, padded sequences, in changing places; two graphs at once on two streams."""
    rng = np.random.default_rng(1)
    T, B, Hq, Hkv, page, most = 430, 4, 8, 2, 32, 2200
    kc, vc, sc, table = _pool(rng, [most] * B, page, Hkv)

    class Step:
        def __init__(self):
            self.cache = (_dev(kc), _dev(vc), _dev(sc))
            self.Q = torch.zeros(T, Hq, D, dtype=torch.float16, device="cuda")
            self.start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
            self.len = torch.zeros(B, dtype=torch.int32, device="cuda")
            self.table = _dev(table)
            self.out = torch.zeros(T, Hq, D, dtype=torch.float16, device="cuda")
            self.stream, self.graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(self.graph, stream=self.stream):
                qoq.kv4_paged_attention(self.Q, self.cache, self.start, self.len, self.table,
                                        max_q=300, out=self.out)

    steps = [Step(), Step()]
    batches = [
        ([300, 1, 100, 3], [300, 2200, 1500, 900]), ([1, 1, 1, 1], [5, 2000, 1, 700]),
        ([0, 0, 0, 0], [0, 9, 0, 3]), ([100, 300, 0, 20], [0, 40, 77, 2000]),
        ([1, 2, 300, 100], [2000, 2, 2200, -7]), ([50, 50, 50, 50], [50, 1000, 60, 50])]
    for i in range(0, len(batches), 2):
        for s, (q, lens) in zip(steps, batches[i:i + 2]):
            s.q = (2 + np.concatenate([[0], np.cumsum(q)])).astype(np.int32)
            s.lens = np.array(lens, np.int32)
            s.host = rng.choice([0.5, 0.0, -0.5], (T, Hq, D)).astype(np.float16)
            s.Q.copy_(_dev(s.host))
            s.start.copy_(_dev(s.q))
            s.len.copy_(_dev(s.lens))
            s.out.fill_(7.0)
        torch.cuda.synchronize()
        for s in steps:
            with torch.cuda.stream(s.stream):
                s.graph.replay()
        torch.cuda.synchronize()
        for s in steps:
            want, tol = exact.attention(s.host, kc, vc, sc, s.q, s.lens, table, SCALE)
            mine = ~torch.isnan(want)
            got = s.out.double()
            assert bool((got[~mine] == 7.0).all())
            assert bool(((got - want).abs()[mine] <= tol[mine]).all())
    assert qoq.device_error() == 0


def test_a_pool_past_32_bits():
    """Codes at offsets over 2^32 bytes, block numbers over 2^22: appended and read as in a
    small pool."""
    Hq, Hkv, page, pages = 8, 8, 512, 16500
    assert pages * Hkv * page // 16 * 1024 > 1 << 32
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator("cuda").manual_seed(2)
    results = []
    for n, at in ((pages, [pages - 1, 3, pages - 2]), (3, [2, 0, 1])):
        cache = (torch.empty(n, Hkv, page // 16, 1024, dtype=torch.uint8, device="cuda"),
                 torch.empty(n, Hkv, page // 16, 1024, dtype=torch.uint8, device="cuda"),
                 torch.empty(n, Hkv, page, 4, dtype=torch.float16, device="cuda"))
        for c in cache:
            for p in at:
                c[p].zero_()
        table = i32([[at[0], at[1]], [at[2], -1]])
        outs = []
        for q, lens in (([600, 40], [600, 40]), ([1, 1], [601, 41]), ([100, 3], [701, 44])):
            T = sum(q)
            g.manual_seed(T)
            x = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda").half()
            start = i32([0, q[0], T])
            Q = qoq.kv4_paged_append(x, cache, start, i32(lens), table, Hq)
            outs += [Q, qoq.kv4_paged_attention(Q, cache, start, i32(lens), table, max_q=max(q))]
        results.append(outs + [c[p] for c in cache for p in at])
        del cache
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert qoq.device_error() == 0


@pytest.mark.parametrize("bad", [[0, 51, 50], [-3, 5, 2], [40, 10, 5], [50, 50, 50], [0, 0, 0],
                                 [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1]])
@pytest.mark.parametrize("max_q", [1, 4, 50])
def test_row_ranges_that_are_none(bad, max_q):
    rng = np.random.default_rng(3)
    T, Hq, Hkv = 50, 4, 1
    kc, vc, sc, table = _pool(rng, [700, 90], 16, Hkv)
    Q = rng.standard_normal((T, Hq, D)).astype(np.float16)
    out = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
    qoq.kv4_paged_attention(_dev(Q), (_dev(kc), _dev(vc), _dev(sc)), _dev(np.array(bad, np.int32)),
                            _dev(np.array([700, 90], np.int32)), _dev(table), max_q=max_q, out=out)
    assert bool((out == 7.0).all()) and qoq.device_error() == 0


@pytest.mark.parametrize("q", [[1, 1, 1], [4, 1, 3], [60, 300, 20]])
def test_lengths_at_the_ends_of_int32(q):
    """The smallest int32 and 0 see nothing; the largest sees what the table holds."""
    rng = np.random.default_rng(4)
    Hq, Hkv, page = 4, 1, 16
    kc, vc, sc, table = _pool(rng, [330] * 3, page, Hkv)
    q_start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    lens = np.array([-2 ** 31, 2 ** 31 - 1, 0], np.int32)
    Q = rng.choice([0.5, 0.0, -0.5], (int(q_start[-1]), Hq, D)).astype(np.float16)
    cache = (_dev(kc), _dev(vc), _dev(sc))
    got = qoq.kv4_paged_attention(_dev(Q), cache, _dev(q_start), _dev(lens), _dev(table),
                                  max_q=max(q)).double()
    want, tol = exact.attention(Q, kc, vc, sc, q_start, lens, table, SCALE)
    assert bool(((got - want).abs() <= tol).all())
    assert bool((got[:q[0]] == 0).all()) and bool((got[-q[2]:] == 0).all())
    # appending there writes queries only
    before = [c.clone() for c in cache]
    x = _dev(rng.standard_normal((int(q_start[-1]), (Hq + 2 * Hkv) * D)).astype(np.float16))
    r = qoq.kv4_paged_append(x, cache, _dev(q_start), _dev(lens), _dev(table), Hq)
    assert torch.equal(r.view(-1, Hq * D), x[:, :Hq * D])
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
    assert qoq.device_error() == 0


@pytest.mark.parametrize("by_rows", [False, True])
def test_appending_values_that_are_no_numbers(by_rows):
    """Infinities, NaN, the largest and the smallest numbers in keys and values: codes, scales
    and offsets are those of kv4_quantize, as one prompt (whole words) and as single tokens."""
    rng = np.random.default_rng(6)
    Hkv, T = 2, 64
    x = rng.standard_normal((T, 2 + 2 * Hkv, D)).astype(np.float16)
    odd = [np.inf, -np.inf, np.nan, 65504.0, -65504.0, 2.0 ** -24, 0.0, -0.0]
    for t in range(T):
        if t % 4 == 3:
            continue
        x[t, 2:, rng.integers(0, D, 1 + t % 3)] = odd[t % 8]
        if t % 5 == 0:
            x[t, 2:, rng.integers(0, D)] = odd[(t + 3) % 8]
        if t % 16 == 1:
            x[t, 2:] = odd[t // 16 * 2]                       # the whole vector
    x = _dev(x.reshape(T, -1))
    flat = qoq.kv4_cache(1, Hkv, T, "cuda")
    k, v = (x.view(T, -1, D)[:, a:a + Hkv].permute(1, 0, 2)[None].contiguous() for a in (2, 4))
    qoq.kv4_quantize(k, v, flat)
    cache = qoq.kv4_paged_cache(4, Hkv, 16, "cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    if by_rows:
        qoq.kv4_paged_append(x, cache, i32(list(range(T + 1))), i32(list(range(1, T + 1))),
                             i32([[0, 1, 2, 3]] * T), 2)
    else:
        qoq.kv4_paged_append(x, cache, i32([0, T]), i32([T]), i32([[0, 1, 2, 3]]), 2)
    for got, exp in zip(cache, flat):
        got = got.permute(1, 0, *range(2, got.dim())).reshape(exp.shape[1:])
        if got.dtype == torch.float16:          # (a NaN is a NaN, whatever its bits)
            same = (got == exp[0]) & (got.signbit() == exp[0].signbit()) | got.isnan() & exp[0].isnan()
            assert bool(same.all())
        else:
            assert torch.equal(got, exp[0])
