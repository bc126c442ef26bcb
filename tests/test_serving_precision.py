"""The tests' tolerances tell what they are meant to tell: planted in the
definition, without a GPU."""
import numpy as np
import pytest

from tests.block_util import to_bf16


def fine_tolerance(out, mass, size, d, tokens, softcap=0.0):
    """Of weights that enter as two bf16, their rounding and what it left, each to nearest: 2^-17 of a weight. Sums of
    `tokens` products in 32 bits, at most a rounding of 2^-24 each; 2^-20 of exp2; tanh within 2^-21 of the cap. A score's
    error changes weights and their sum."""
    score = size * ((d + 10) * 2.0 ** -24 + 2.0 ** -20) + softcap * 2.0 ** -21
    weight = 2.0 ** -17 + 2.0 ** -20 + (tokens + 10) * 2.0 ** -24 + 2 * score
    return 2.0 ** -8 * np.abs(out) + weight[..., None] * mass * 1.01 + 2.0 ** -133


@pytest.mark.parametrize("n,d", [(77, 64), (300, 128), (200, 256)])
def test_weights_in_one_part_are_told(n, d):
    """Softmax weights rounded to one bf16 leave the tolerance of two in some of a few rows' outputs; in two they do not, nor
    where the second part is scaled wrongly."""
    g = np.random.Generator(np.random.PCG64(n))
    bad = {"one": 0, "two": 0, "half of the second": 0}
    for _ in range(8):
        q, k, v = 0.1 * g.standard_normal(d), g.standard_normal((n, d)), g.standard_normal((n, d))
        s = k @ q * d ** -0.5
        e = np.exp2((s - s.max()) * np.log2(np.e))
        want, mass, size = e @ v / e.sum(), e @ np.abs(v) / e.sum(), np.max(np.abs(k) @ np.abs(q)) * d ** -0.5
        hi = to_bf16(e)
        lo = to_bf16(e - hi)
        tol = fine_tolerance(want[None], mass[None], np.array([size]), d, n)[0]
        for name, w in (("one", hi), ("two", hi + lo), ("half of the second", hi + 0.5 * lo)):
            bad[name] += int((np.abs(to_bf16(w @ v / e.sum()) - want) > tol).sum())
    assert bad["two"] == 0 and bad["one"] > 20 and bad["half of the second"] > 20, bad
