"""Rotary frequencies for longer contexts, every pair against its rule, written
here in plain Python one pair at a time."""
import math

import pytest

import precision_quantized_gemm_b200 as qg


def _turns(frequency, original):
    return original * frequency / (2 * math.pi)


def _rule(scaling, dim, base, j, factor, original, low=1.0, high=4.0, fast=32.0, slow=1.0):
    f = base ** (-2.0 * j / dim)
    if scaling is None:
        return f
    if scaling == "linear":
        return f / factor
    if scaling == "base":
        return (base * factor ** (dim / (dim - 2))) ** (-2.0 * j / dim)
    if scaling == "bands":
        turns = _turns(f, original)
        if turns >= high:
            return f
        if turns <= low:
            return f / factor
        kept = (turns - low) / (high - low)
        return kept * f + (1 - kept) * f / factor

    # "ramp": from the pair that turns `fast` times to the one that turns `slow` times, a real number of pairs
    # each, rounded outwards, within the head's channels
    def pair(turns):
        return dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

    begin, end = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), dim - 1)
    divided = min(max((j - begin) / (end - begin), 0.0), 1.0)
    return divided * f / factor + (1 - divided) * f


@pytest.mark.parametrize("scaling", [None, "linear", "base", "bands", "ramp"])
@pytest.mark.parametrize("dim,base,original", [(64, 10000.0, 4096), (128, 10000.0, 8192), (128, 10000.0, 65536),
                                               (128, 10000.0, 131072), (96, 10000.0, 262144), (128, 500000.0, 131072),
                                               (32, 1000.0, 32768)])
@pytest.mark.parametrize("factor", [1.0, 4.0, 32.0])
def test_every_pair(scaling, dim, base, original, factor):
    """Also where the slowest pair still turns in the original context.  64 bits and a few operations: 2^-40."""
    got, _ = qg.rope_frequencies(dim, base, scaling=scaling, factor=factor, original=original, device="cpu")
    for j, f in enumerate(got.tolist()):
        assert f == pytest.approx(_rule(scaling, dim, base, j, factor, original), rel=2.0 ** -40, abs=0.0)


def test_ramp_keeps_what_turns():
    """A pair that turns more than `slow` times in the original context is not divided in full."""
    plain, _ = qg.rope_frequencies(128, 10000.0, device="cpu")
    f, _ = qg.rope_frequencies(128, 10000.0, scaling="ramp", factor=4.0, original=131072, device="cpu")
    assert _turns(plain[-1].item(), 131072) > 2 and f[-1] > 1.2 * plain[-1] / 4
