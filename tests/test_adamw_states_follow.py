"""How 8-bit states follow gradients whose size changes, by the header's definition of the codes (CPU)."""
import numpy as np
import pytest

from training_ref import F, decode, encode


def root_after(beta2, before, after, n=1024):
    """The median of the held root over the exact one, of the half of a block's values whose gradients fell to a tenth."""
    r = np.random.default_rng(0)
    codes = encode(np.zeros(n, F), np.zeros(n, F))
    exact, low = np.zeros(n), np.arange(n) % 2 == 0
    for t in range(before + after):
        g = r.standard_normal(n).astype(F) * F(1e-3)
        if t >= before:
            g[low] *= F(0.1)
        m, v = decode(*codes)
        codes = encode(m * F(0.9) + g * F(0.1), v * F(beta2) + (g * g) * F(1 - beta2))
        exact = exact * beta2 + g.astype(np.float64) ** 2 * (1 - beta2)
    return float(np.median((np.sqrt(decode(*codes)[1]) / np.sqrt(exact))[low]))


@pytest.mark.parametrize("beta2", [0.9, 0.95, 0.97])
def test_followed(beta2):
    assert abs(root_after(beta2, 500, 1000) - 1) < 0.06


def test_not_followed():
    """What the header warns of: a thousandth of v a step is less than half a step of any code."""
    assert root_after(0.999, 1500, 5000) > 4
