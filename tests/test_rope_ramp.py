"""Values in the middle of the ramps that rope_frequencies lays between kept and divided
frequencies, against the published formulas written out for one pair."""
import math

import pytest

import w4a8_quantized_gemm_02_b200 as qoq

pytest.importorskip("torch")


def test_llama3_between_the_wavelengths():
    rot, base, factor, low, high, length = 128, 500000.0, 8.0, 1.0, 4.0, 8192
    got, _ = qoq.rope_frequencies(rot, base, {
        "type": "llama3", "factor": factor, "low_freq_factor": low, "high_freq_factor": high,
        "original_length": length}, device="cpu")
    between = 0
    for j in range(rot // 2):
        f = math.exp(-2 * j / rot * math.log(base))
        wavelength = 2 * math.pi / f
        if wavelength > length / low:
            want = f / factor
        elif wavelength < length / high:
            want = f
        else:
            smooth = (length / wavelength - low) / (high - low)
            want = (1 - smooth) * (f / factor) + smooth * f
            between += 1
        assert math.isclose(float(got[j]), want, rel_tol=1e-12), j
    assert between > 3


@pytest.mark.parametrize("rot,base,factor,length,fast,slow", [
    (128, 10000.0, 4.0, 4096, 32.0, 1.0), (64, 1000000.0, 16.0, 32768, 32.0, 1.0),
    (128, 500000.0, 8.0, 8192, 48.0, 2.0)])
def test_yarn_on_the_ramp(rot, base, factor, length, fast, slow):
    got, attention = qoq.rope_frequencies(rot, base, {
        "type": "yarn", "factor": factor, "original_length": length, "beta_fast": fast,
        "beta_slow": slow}, device="cpu")
    assert math.isclose(attention, 0.1 * math.log(factor) + 1.0)

    # pair j turns length * base^(-2 j / rot) / (2 pi) times over the trained length
    def pair(turns):
        return rot / 2 * math.log(length / (2 * math.pi * turns)) / math.log(base)
    first, last = math.floor(pair(fast)), math.ceil(pair(slow))
    first, last = max(first, 0), min(last, rot - 1)
    between = 0
    for j in range(rot // 2):
        f = math.exp(-2 * j / rot * math.log(base))
        divided = min(max((j - first) / (last - first), 0.0), 1.0)
        between += 0.0 < divided < 1.0
        want = (f / factor) * divided + f * (1.0 - divided)
        assert math.isclose(float(got[j]), want, rel_tol=1e-12), j
    assert between > 3
