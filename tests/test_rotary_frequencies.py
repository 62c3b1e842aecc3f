"""Frequencies for long contexts, value by value (no GPU)."""
import math

import pytest

from exact_io_aware_64_b200 import binding


def close(f, want):
    # float32 of a float64 value: half a step, 2^-24 of it
    assert len(f) == len(want)
    for a, b in zip(f.tolist(), want):
        assert abs(a - b) <= 2.0 ** -24 * 1.01 * b


@pytest.mark.parametrize("rot,base,factor,length", [(64, 10000.0, 4.0, 2048), (128, 500000.0, 8.0, 8192),
                                                    (32, 10000.0, 1.0, 4096), (2, 10000.0, 16.0, 100),
                                                    (128, 10000.0, 0.5, 4096), (96, 10000.0, 40.0, 10)])
def test_values(rot, base, factor, length):
    plain = [base ** (-2.0 * k / rot) for k in range(rot // 2)]
    kw = {"base": base, "factor": factor, "original_len": length, "device": "cpu"}
    f, m = binding.rotary_frequencies(rot, scaling="linear", **kw)
    close(f, [x / factor for x in plain])
    assert m == 1.0
    f, m = binding.rotary_frequencies(rot, scaling="base", **kw)
    # raised so that the slowest frequency is divided by factor, the fastest stays
    far = [x * factor ** (-2.0 * k / (rot - 2)) for k, x in enumerate(plain)] if rot > 2 else plain
    close(f, far)
    assert m == 1.0
    f, m = binding.rotary_frequencies(rot, scaling="parts", **kw)
    want = []
    for x in plain:
        turns = length * x / (2 * math.pi)
        if turns >= 32:
            want.append(x)
        elif turns <= 1:
            want.append(x / factor)
        else:
            place = math.log(turns, 32)
            want.append(place * x + (1 - place) * x / factor)
    close(f, want)
    assert m == pytest.approx(0.1 * math.log(factor) + 1 if factor > 1 else 1.0, abs=1e-15)


def test_the_parts_meet_all_three_kinds():
    f, _ = binding.rotary_frequencies(128, factor=8.0, scaling="parts", original_len=4096, device="cpu")
    p, _ = binding.rotary_frequencies(128, device="cpu")
    r = (p / f).tolist()
    assert r[0] == 1.0 and r[-1] == pytest.approx(8.0) and any(1.01 < x < 7.99 for x in r)


@pytest.mark.parametrize("kw", [{"original_len": 0}, {"original_len": -4096}, {"factor": math.inf},
                                {"factor": math.nan}, {"base": math.inf}, {"base": -1.0}])
def test_refusals(kw):
    with pytest.raises(ValueError):
        binding.rotary_frequencies(64, scaling="parts", device="cpu", **kw)
