"""qoq_lora_add against binary64, and the operators of a decode step in a row.

Allowance of an output: half an FP16 step of it (2^-11 relative, 2^-25 below the
normal range), plus, of the sum of the products' sizes |x| |A| |B|: one FP32 rounding
(2^-24) for each of the K / 16 + R / 16 steps of the sums and a few more at their
ends, and 2^-21 for the 22 bits of the middle values.  For K <= 4096 that is under
2^-24 * (256 + 8 + 16) + 2^-21 < 2^-15."""
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


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _case(rng, T, K, N, R, n, ids):
    X = rng.standard_normal((T, K)).astype(np.float16)
    X[:, rng.integers(0, K, 3)] *= 20
    A = (rng.standard_normal((n, R, K)) / math.sqrt(K)).astype(np.float16)
    B = (rng.standard_normal((n, N, R)) * 0.1).astype(np.float16)
    Y = rng.standard_normal((T, N)).astype(np.float16)
    scaling = rng.uniform(0.25, 2.0, n).astype(np.float32)
    return Y, X, A, B, np.asarray(ids, np.int32), scaling


def _reference(Y, X, A, B, ids, scaling):
    out, size = Y.astype(np.float64), np.zeros(Y.shape)
    for a in range(len(scaling)):
        r = np.nonzero(ids == a)[0]
        if r.size:
            x, wa, wb = X[r].astype(np.float64), A[a].astype(np.float64), B[a].astype(np.float64)
            out[r] += float(scaling[a]) * ((x @ wa.T) @ wb.T)
            size[r] += float(scaling[a]) * ((np.abs(x) @ np.abs(wa).T) @ np.abs(wb).T)
    return out, 2.0 ** -11 * np.abs(out) + 2.0 ** -25 + 2.0 ** -15 * size


def _check(got, args):
    want, tol = _reference(*args)
    off = np.abs(got.cpu().numpy().astype(np.float64) - want)
    assert (off <= tol).all(), f"worst {np.max(off / tol):.3g} of the allowance"


def _ids(rng, T, n, kind):
    if kind == "distinct":
        return rng.permutation(max(T, n))[:T] % n
    if kind == "random":
        return rng.integers(-1, n, T)
    if kind == "one":
        return np.full(T, n - 1)
    if kind == "none":
        return np.full(T, -1)
    if kind == "wild":
        return rng.choice([-2 ** 31, -1, 0, n - 1, n, 2 ** 31 - 1], T)
    at, ids = 0, np.empty(T, np.int64)          # runs
    while at < T:
        step = int(rng.integers(1, 60))
        ids[at:at + step] = rng.integers(-1, n)
        at += step
    return ids


CASES = [
    # T, K, N, R, n, kind
    (1, 128, 128, 8, 1, "one"),
    (1, 4096, 6144, 16, 4, "random"),
    (2, 256, 384, 24, 3, "distinct"),
    (9, 1024, 128, 40, 20, "distinct"),
    (16, 512, 256, 128, 5, "random"),
    (33, 640, 512, 64, 33, "distinct"),
    (48, 2048, 1280, 32, 64, "random"),
    (70, 384, 256, 72, 3, "wild"),
    (100, 256, 128, 16, 7, "none"),
    (130, 1152, 640, 56, 6, "runs"),
    (513, 512, 256, 64, 6, "runs"),
    (700, 256, 384, 128, 40, "random"),
    (1000, 384, 128, 8, 1, "one"),
    (4200, 128, 128, 16, 300, "random"),       # rows are taken by adapter within 4096
    (9000, 128, 128, 8, 5, "runs"),
    (65, 256, 128, 112, 4096, "distinct"),
]


@pytest.mark.parametrize("T,K,N,R,n,kind", CASES)
def test_matches_reference(T, K, N, R, n, kind):
    rng = np.random.default_rng(T + R)
    args = _case(rng, T, K, N, R, n, _ids(rng, T, n, kind))
    Y, X, A, B, ids, scaling = (_dev(a) for a in args)
    got = qoq.lora_add(Y, X, A, B, ids, scaling)
    _check(got, args)
    # again, and in place: the same bits
    assert torch.equal(qoq.lora_add(Y, X, A, B, ids, scaling), got)
    qoq.lora_add(Y, X, A, B, ids, scaling, out=Y)
    assert torch.equal(Y, got)


def test_large_and_small_values():
    """Middle values past FP16's range (scaled back by small B), and subnormal
    ones."""
    rng = np.random.default_rng(4)
    for up, down in ((3000.0, 1e-6), (1e-4, 300.0)):
        Y, X, A, B, ids, scaling = _case(rng, 20, 512, 256, 32, 3, _ids(rng, 20, 3, "random"))
        X = (X * 0.02).astype(np.float16)
        A, B = (A * up).astype(np.float16), (B * down).astype(np.float16)
        args = (Y, (X * 50).astype(np.float16), A, B, ids, scaling)
        _check(qoq.lora_add(*(_dev(a) for a in args)), args)


def test_rows_of_no_adapter_keep_their_bits():
    rng = np.random.default_rng(6)
    args = _case(rng, 40, 256, 256, 16, 2, _ids(rng, 40, 2, "random"))
    Y = args[0].copy()
    Y[0, :4] = [np.inf, -np.inf, -0.0, 65504]
    args[4][0] = -1
    out = qoq.lora_add(_dev(Y), *(_dev(a) for a in args[1:])).cpu().numpy()
    rows = args[4] < 0
    assert np.array_equal(out[rows].view(np.uint16), Y[rows].view(np.uint16))


def test_empty_call_and_other_stream():
    rng = np.random.default_rng(7)
    args = tuple(_dev(a) for a in _case(rng, 50, 512, 256, 32, 4, _ids(rng, 50, 4, "random")))
    none = (args[0][:0], args[1][:0], *args[2:4], args[4][:0], args[5])
    assert qoq.lora_add(*none).shape == (0, 256)
    base = qoq.lora_add(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [qoq.lora_add(*args, stream=side) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(o, base) for o in outs)


def test_two_graphs_do_not_share_a_workspace():
    rng = np.random.default_rng(8)
    steps = []
    for k in range(2):
        host = _case(rng, 64, 1024, 512, 32, 9, _ids(rng, 64, 9, "random"))
        args = tuple(_dev(a) for a in host)
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            out = qoq.lora_add(*args)
        steps.append((host, args, s, g, out))
    for _ in range(5):
        for _, _, s, g, _ in steps:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for host, _, _, _, out in steps:
        _check(out, host)


def test_layer_step_in_a_row(oracle):
    """QKV projection with adapters, rotation and append, attention, output
    projection: a prompt step and then decode steps, every part against its
    reference on the values that it was given."""
    rng = np.random.default_rng(9)
    Hq, Hkv, D, hidden, page, n, R = 4, 2, 128, 512, 16, 3, 16
    wq = _dev((rng.standard_normal(((Hq + 2 * Hkv) * D, hidden)) * 0.05).astype(np.float16))
    wo = _dev((rng.standard_normal((hidden, Hq * D)) * 0.05).astype(np.float16))
    qkv_proj, o_proj = qoq.QoQLinear(wq), qoq.QoQLinear(wo)
    A = (rng.standard_normal((n, R, hidden)) / 23).astype(np.float16)
    B = (rng.standard_normal((n, (Hq + 2 * Hkv) * D, R)) * 0.1).astype(np.float16)
    scaling = np.array([0.5, 1.0, 2.0], np.float32)
    adapters = (_dev(A), _dev(B), _dev(scaling))
    freq, factor = qoq.rope_frequencies(128, 500000.0, device=DEV)
    cache = qoq.kv4_paged_cache(12, Hkv, page, DEV)
    table = _dev(rng.permutation(12).reshape(3, 4).astype(np.int32))
    lens = np.zeros(3, np.int32)
    for q in ([20, 33, 1], [1, 1, 1], [1, 0, 1], [2, 3, 1]):
        start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        lens = (lens + q).astype(np.int32)
        T = int(start[-1])
        ids = np.repeat([2, -1, 0], q).astype(np.int32)
        x = rng.standard_normal((T, hidden)).astype(np.float16)
        plain = qkv_proj(_dev(x))
        qkv = qkv_proj(_dev(x), adapters=adapters, ids=_dev(ids))
        _check(qkv, (plain.cpu().numpy(), x, A, B, ids, scaling))
        qr = qoq.kv4_paged_append(qkv, cache, _dev(start), _dev(lens), table, Hq, inv_freq=freq,
                                  rope_factor=factor)
        out = qoq.kv4_paged_attention(qr, cache, _dev(start), _dev(lens), table, max_q=max(q))
        y = o_proj(out.view(T, Hq * D))
        assert y.shape == (T, hidden) and bool(torch.isfinite(y).all())
        host = qkv.cpu().numpy().reshape(T, -1, D)
        pos = [p for _, _, p in ref.rows(start, lens)]
        want_q = ref.rotate(host[:, :Hq], pos, freq.cpu().numpy(), "half", factor)
        assert np.abs(qr.cpu().numpy() - want_q).max() <= 2.0 ** -10 * np.abs(want_q).max()
        want, tol = ref.attention(qr.cpu().numpy(), *(c.cpu().numpy() for c in cache), start, lens,
                                  table.cpu().numpy(), 1 / math.sqrt(D))
        assert (np.abs(out.cpu().numpy() - want) <= tol).all()
    assert qoq.device_error() == 0


def test_refusals():
    rng = np.random.default_rng(10)
    Y, X, A, B, ids, s = (_dev(a) for a in _case(rng, 4, 256, 256, 16, 2, [0, 1, 0, -1]))
    bad = [
        (Y, X, A[:, :12].contiguous(), B[:, :, :12].contiguous(), ids, s),        # rank
        (Y, X[:, :200].contiguous(), A[:, :, :200].contiguous(), B, ids, s),      # K
    ]
    for args in bad:
        with pytest.raises(qoq.QoQError):
            qoq.lora_add(*args)
    wrong = [
        (Y, X, A, B, ids[:3], s), (Y, X, A, B, ids.long(), s), (Y, X, A, B[:, :128], ids, s),
        (Y, X, A.float(), B, ids, s), (Y[:2], X, A, B, ids, s), (Y, X, A, B, ids, s[:1]),
        (Y, X.t(), A, B, ids, s), (Y.cpu(), X, A, B, ids, s),
    ]
    for args in wrong:
        with pytest.raises(ValueError):
            qoq.lora_add(*args)
    with pytest.raises(qoq.QoQError) as e:
        qoq.lora_add(Y, X, A, B, ids, s, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == qoq.QOQ_ERR_WORKSPACE
    layer = qoq.QoQLinear(_dev(rng.standard_normal((256, 256)).astype(np.float16)))
    with pytest.raises(ValueError):
        layer(X, adapters=(A, B, s))
