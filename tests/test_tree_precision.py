"""The rounding that nq_tree_attend states for its rotated keys, on the CPU: the
kernel's f16 arithmetic step by step in numpy, against fp64."""
import numpy as np
import pytest

EPS = 2.0 ** -11  # half a step of f16, relative


def rotated(x, y, pos, w):
    """(o, o') of the pairs (x, y) = (k_i, k_i') before their scale, as the kernel
    rounds them: u = (x + y) / 2 and v = (x - y) / 2 are integers, the angles'
    combinations f16, one product and one fma in f16 per coordinate (their exact
    values fit fp64, so that each rounding is one)."""
    u, v = (x + y) / 2, (x - y) / 2
    c, s = np.cos(pos * w).astype(np.float32), np.sin(pos * w).astype(np.float32)
    cp, sp = (c - s).astype(np.float16).astype(float), (c + s).astype(np.float16).astype(float)
    r16 = lambda z: z.astype(np.float16).astype(float)  # noqa: E731
    return r16(u * cp + r16(v * sp)), r16(-v * cp + r16(u * sp))


@pytest.mark.parametrize("theta", [1e4, 5e5, 1e6])
@pytest.mark.parametrize("bits", [2, 3])
def test_rotated_keys_keep_the_stated_bound(theta, bits):
    """|o - k| <= 2^-11 (2 r + |k|), r the pair's length: the combinations
    c' = cos - sin and s' = cos + sin are below sqrt 2, so rounded by 2^-11 at
    most, against |u| + |v| <= r; the product v s' is at most r; the sum is |k|.
    (The products of two roundings are below 2^-9 of that, and the fp32 angles
    take 2^-22 r.)"""
    rng = np.random.default_rng(bits)
    n = 400_000
    # the two products with H64 of a lattice point's halves: integers up to 64 (2^b - 1)
    u, v = rng.integers(-64 * (2 ** bits - 1), 64 * (2 ** bits - 1) + 1, (2, n)).astype(float)
    pos, w = rng.integers(0, 131072, n), theta ** (-rng.integers(0, 64, n) / 64.0)
    x, y = u + v, u - v
    o, p = rotated(x, y, pos, w)
    c, s = np.cos(pos * w), np.sin(pos * w)
    k, l, r = x * c - y * s, y * c + x * s, np.hypot(x, y)
    for got, want in ((o, k), (p, l)):
        assert (np.abs(got - want) <= EPS * (2 * r + np.abs(want)) * (1 + 2.0 ** -9) + 2.0 ** -22 * r).all()
        # and no bound relative to the coordinate alone holds: pairs cancel
        assert (np.abs(got - want) > EPS * np.abs(want)).mean() > 0.05
