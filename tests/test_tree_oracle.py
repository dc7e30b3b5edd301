"""The accuracy checks of tree attention against mistakes planted in the oracle
(CPU): the kernel's own roundings pass, and what a broken pipeline would give does
not - values of a neighbouring tile, a tile lost or counted twice, stale scales,
sums rescaled by a wrong factor."""
import numpy as np
import pytest

from tests.tree_oracle import D, Expected, angles, check_all, dequant, hadamard, lattice

THETA = 5e5


def store(n, bits, seed):
    """Random lattice points (codes 0 .. 2^b - 2, with the coset bit one more, so
    that their mean is 0) and scales about one."""
    rng = np.random.default_rng(seed)
    half = rng.integers(0, 2, (n, 16))
    j = rng.integers(0, 2 ** bits - 1 + half.repeat(8, -1))
    b = ((j[..., None] >> np.arange(bits)) & 1).reshape(n, -1).astype(np.uint8)
    codes = np.packbits(b, axis=-1, bitorder="little").view(np.uint32)
    sig = np.exp(0.2 * rng.standard_normal(n)).astype(np.float16).view(np.uint16).astype(np.uint32)
    return codes, (half << np.arange(16)).sum(-1).astype(np.uint32) | (sig << 16)


def bf16(x):
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


def f16(x):
    return x.astype(np.float16).astype(np.float64)


def as_kernel(q, ks, vs, kn, vn, see, scale, order=None, raised=0.0):
    """The kernel's roundings in one pass: (out, lse).  order: the token whose
    values meet token t's weight (-1: its weight is lost); raised: log2 of the
    largest weight."""
    n = len(ks[0])
    t, kap = lattice(*ks)
    h64 = hadamard()[:64, :64]
    u, v = t[:, :64] @ h64, t[:, 64:] @ h64
    c, s = (x.astype(np.float32) for x in angles(np.arange(n), THETA))
    cp, sp = f16(c - s), f16(c + s)
    o = np.concatenate([f16(u * cp + f16(v * sp)), f16(-v * cp + f16(u * sp))], -1)
    sc = scale * (q @ o.T) * kap
    sn = np.where(see, scale * (q @ kn.T), -np.inf)
    top = np.maximum(sc.max(-1), sn.max(-1))[:, None]
    w, wn = np.exp(sc - top) * 2.0 ** (4 + raised), np.exp(sn - top) * 2.0 ** (4 + raised)
    l = w.sum(-1) + wn.sum(-1)
    val, sig = dequant(*vs), (vs[1] >> 16).astype(np.uint16).view(np.float16).astype(np.float64)
    m = sig / 2.0 ** np.floor(np.log2(sig))
    wr = f16(w * m) / m
    if order is not None:
        wr, val = np.where(order >= 0, wr, 0), val[np.maximum(order, 0)]
    return bf16((wr @ val + wn @ vn) / l[:, None]), top[:, 0] + np.log(l) - (4 + raised) * np.log(2)


def case(n, rows, bk=3, bv=2, seed=0, nodes=4):
    rng = np.random.default_rng(seed)
    q, kn, vn = (bf16(rng.standard_normal((r, D))) for r in (rows, nodes, nodes))
    see = rng.random((rows, nodes)) < 0.5
    return q, (*store(n, bk, seed + 1), bk), (*store(n, bv, seed + 2), bv), kn, vn, see


def expected(q, ks, vs, kn, vn, see, scale):
    return Expected(q, dequant(*ks, np.arange(len(ks[0])), THETA), dequant(*vs), kn, vn, see, scale)


@pytest.mark.parametrize("n,rows,scale", [(300, 4, D ** -0.5), (2000, 16, D ** -0.5), (12345, 8, 0.03),
                                          (20000, 4, D ** -0.5), (2000, 8, 0.5), (900, 8, -0.3)])
@pytest.mark.parametrize("bk,bv", [(3, 2), (2, 3)])
def test_the_kernels_roundings_pass(n, rows, scale, bk, bv):
    a = case(n, rows, bk, bv, seed=n)
    for raised in (0.0, 9.0):
        e, (o, l) = expected(*a, scale), as_kernel(*a, scale, raised=raised)
        e.check(o, l)
        assert check_all([(e, o)]) < 2.0 ** -8


def planted(n):
    t = np.arange(n)
    tiles = -(-n // 128)
    lost = t.copy()
    lost[t // 128 == tiles // 2] = -1
    stale = t.copy()
    one = t // 128 == tiles // 3
    stale[one] = t[one] - 128
    return {"zeros": None, "the next tile's values": np.minimum(t + 128, n - 1), "a tile's values lost": lost,
            "a tile's values stale": stale, "one token off": np.minimum(t + 1, n - 1)}


FLAT = 0.02  # random codes are wider than encoded rows: scores of half a nat


@pytest.mark.parametrize("n", [12345, 16300, 40000])
@pytest.mark.parametrize("what", list(planted(1000)))
def test_planted_mistakes_fail(n, what):
    """One tile among 97 to 313 is enough, with scores that leave no token most of
    the weight."""
    a = case(n, 4, seed=3)
    e = expected(*a, FLAT)
    good, lse = as_kernel(*a, FLAT)
    e.check(good, lse)
    order = planted(n)[what]
    o = np.zeros_like(good) if order is None else as_kernel(*a, FLAT, order=order)[0]
    for check in (lambda: e.check(o, lse), lambda: check_all([(e, o)])):
        with pytest.raises(AssertionError):
            check()


@pytest.mark.parametrize("n", [12345, 40000])
def test_a_lost_tile_shows_in_the_sum(n):
    a = case(n, 4, seed=5)
    e = expected(*a, FLAT)
    o, lse = as_kernel(*a, FLAT)
    mid = slice(128 * (n // 256), 128 * (n // 256) + 128)
    with pytest.raises(AssertionError, match="lse"):
        e.check(o, lse + np.log1p(-e.p[:, mid].sum(-1)))


@pytest.mark.parametrize("scale", [0.1, 0.4, -0.4])
def test_growing_scores_leave_the_check_meaningful(scale):
    """Keys along the query at a growing strength, where errors are counted as if
    they were alike: the tolerance stays below a tenth of what the output could
    be, and a rescaling by another power of two fails."""
    rng = np.random.default_rng(7)
    n = 2000
    q, ks, vs, kn, vn, see = case(n, 6, seed=7)
    k = dequant(*ks, np.arange(n), THETA)
    k = k * 0.2 + q[:1] / np.linalg.norm(q[0]) * np.linspace(-30, 30, n)[:, None]
    v = dequant(*vs)
    e = Expected(q, k, v, kn, vn, see, scale)
    to, _ = e.tolerance(alike=True)
    assert (to <= 0.1 * (e.p @ np.sqrt((np.concatenate([v, vn]) ** 2).sum(-1)))).all()
    e.check(bf16(e.out), e.lse, alike=True)
    p = e.p.copy()
    p[:, :n // 2] *= 2.0 ** 10  # the first half's sums not rescaled
    p[:, n - 128:n] *= 0.5 + 0.1 * rng.random()
    p /= p.sum(-1, keepdims=True)
    with pytest.raises(AssertionError):
        e.check(bf16(p @ np.concatenate([v, vn])), e.lse, alike=True)
