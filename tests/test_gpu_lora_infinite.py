"""Adapters whose middle values are infinite: the sums decide, as in the formula."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU container
    pytest.skip("no CUDA device", allow_module_level=True)

import w4a8_quantized_gemm_02_b200 as qoq  # noqa: E402


@pytest.mark.parametrize("T", [1, 5, 70])
@pytest.mark.parametrize("R", [8, 40])
def test_infinite_inputs(T, R):
    """Row 0 has one infinite input; A and B keep its sign in every rank, or mix signs."""
    rng = np.random.default_rng(T + R)
    K, N = 256, 256
    A = rng.uniform(0.01, 0.1, (2, R, K)).astype(np.float16)
    B = rng.uniform(0.01, 0.1, (2, N, R)).astype(np.float16)
    B[:, ::2] *= -1                               # columns of either sign
    B[1, 1::4, 0] *= -1                           # ... and, of adapter 1, of both: inf - inf
    X = rng.standard_normal((T, K)).astype(np.float16)
    X[0, 3] = np.inf
    Y = rng.standard_normal((T, N)).astype(np.float16)
    scaling = np.array([0.5, 2.0], np.float32)
    for a in range(2):
        ids = np.full(T, a, np.int32)
        dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
        got = qoq.lora_add(dev(Y), dev(X), dev(A), dev(B), dev(ids), dev(scaling)).cpu().numpy()
        with np.errstate(invalid="ignore"):
            want = Y.astype(np.float64) + scaling[a] * (
                (X.astype(np.float64) @ A[a].astype(np.float64).T) @ B[a].astype(np.float64).T)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        inf = np.isinf(want)
        assert inf.any() and np.array_equal(got[inf], want[inf].astype(np.float16))
        ok = np.isfinite(want)
        assert np.isfinite(got[ok]).all()
        # half an FP16 step; of the products' sizes, 2^-24 for each of K / 16 + R / 16 + 8
        # additions (27 at most) and 2^-21 for the 22 bits of the middle values: under 2^-18
        size = scaling[a] * ((np.abs(np.where(np.isinf(X), 0, X).astype(np.float64)) @
                              A[a].astype(np.float64).T) @ np.abs(B[a].astype(np.float64)).T)
        tol = 2.0 ** -11 * np.abs(want[ok]) + 2.0 ** -25 + 2.0 ** -18 * size[ok]
        assert (np.abs(got[ok] - want[ok]) <= tol).all()
