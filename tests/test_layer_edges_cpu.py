"""Why the attention subtracts its reference before it scales: the arithmetic of a score's power of
two in fp32, pinned on the CPU."""
import numpy as np
import pytest


def _largest_exponents(size, seed=0, n=20000):
    """log2 p of a row's own maximum s, reference m = s: by fma(s, c, -round(m c)), and by (s - m) c."""
    rng = np.random.default_rng(seed)
    s = (rng.uniform(1, 2, n) * size).astype(np.float32)
    c = rng.uniform(1, 2, n).astype(np.float32)
    m = s * c  # rounded once to fp32
    fused = (s.astype(np.longdouble) * c - m).astype(np.float32)  # exact product (48 bits), rounded once
    return fused, (s - s) * c


@pytest.mark.parametrize("bits", [10, 22, 28, 32, 60])
def test_the_power_of_a_rows_own_maximum(bits):
    fused, first = _largest_exponents(2.0 ** bits)
    assert (first == 0).all()
    # the fused form is off by up to half a unit of s c (below 2^(bits + 2)): harmless for
    # scores of some millions, past fp16's range from 2^28 on
    half = 2.0 ** (bits + 1 - 24)
    assert np.abs(fused).max() <= half
    assert (fused.max() > 15) == (bits >= 28) and (fused.max() < 1) == (bits <= 22)
