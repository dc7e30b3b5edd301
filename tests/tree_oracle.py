"""fp64 evaluation of tree attention for one KV head, in numpy, with what the
kernel's roundings can move: the GPU tests compare with it, and the CPU tests
plant mistakes in it.

Errors, per query row with exact weights p_t (all norms over the 128 coordinates):
- a rotated key is formed from f16 angle combinations c', s' by a rounded f16
  product and an f16 fma, u c' + v s' with u^2 + v^2 = r^2 / 2 over the pair's
  length r.  Each of the four roundings is uniform within half a step (2^-11
  relative: variance 2^-22 / 3).  The combinations give (q^2 + q'^2)(u^2 + v^2)
  (c'^2 + s'^2) = |q pair|^2 r^2 of it, the product q^2 (v s')^2 + q'^2 (u s')^2
  <= |q pair|^2 r^2, the sum <= |q pair|^2 r^2.  Together, for the score,
    sigma_t^2 <= scale^2 2^-22 sum over pairs (q_i^2 + q_i'^2)(k_ti^2 + k_ti'^2);
- a weight is rounded to f16, 2^-11 of itself or 2^-29 of the largest (f16 has
  no smaller step below 2^-14, and the largest weight is 2^4 at least);
- a score error moves the output by p_t ds (v_t - out), a weight error by p_t e
  v_t.  Errors of different tokens are independent (they act on coordinates that
  are), so they add as variances:
    V = sum_t p_t^2 sigma_t^2 |v_t - out|^2 + max(2^-11 p_t, 2^-29 p_max)^2 / 3 |v_t|^2;
  where keys are made alike on purpose they may add as they are:
    C = sum_t p_t sigma_t |v_t - out|;
- the output's rounding to bf16 is uniform within 2^-8 of each coordinate: 2^-8
  |out| surely, 2^-8 / sqrt 3 |out| as a root mean square at most;
- fp32 sums: 2^-18 of sum p |v|, of sum |q k| in the scores 2^-19.
"""
import math

import numpy as np

D = 128


def hadamard():
    h = np.ones((1, 1))
    for _ in range(7):
        h = np.kron(np.array([[1.0, 1.0], [1.0, -1.0]]), h)
    return h


def lattice(codes, meta, bits):
    """t = 2q [n][128] (integers) and kappa [n] of packed vectors: codes uint32
    [n][4 bits], meta uint32 [n]."""
    c = np.concatenate([codes.astype(np.uint64), np.zeros((len(codes), 1), np.uint64)], -1)
    i = np.arange(D)
    w, off = bits * i // 32, (bits * i % 32).astype(np.uint64)
    j = ((c[:, w] | (c[:, w + 1] << np.uint64(32))) >> off) & np.uint64(2 ** bits - 1)
    half = (meta[:, None] >> (i // 8).astype(np.uint32)) & 1
    sig = (meta >> 16).astype(np.uint16).view(np.float16).astype(np.float64)
    return 2.0 * j.astype(np.float64) - 2 ** bits + 2 - half, sig / (2 * math.sqrt(D))


def rotate(x, c, s):
    a, b = x[..., :64], x[..., 64:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def angles(pos, theta):
    a = np.asarray(pos, np.float64)[:, None] * theta ** (-np.arange(64) / 64.0)
    return np.cos(a), np.sin(a)


def dequant(codes, meta, bits, pos=None, theta=None):
    """fp64 vectors, rotated to their positions where given."""
    t, kap = lattice(codes, meta, bits)
    x = (t @ hadamard()) * kap[:, None]
    return x if pos is None else rotate(x, *angles(pos, theta))


class Expected:
    """Rows q [R][128] over keys k and values v [n][128] (held: which tokens
    count) and over draft keys and values kn, vn [m][128] where see [R][m]."""

    def __init__(self, q, k, v, kn, vn, see, scale, held=None):
        n = len(k)
        ka, va = np.concatenate([k, kn]), np.concatenate([v, vn])
        sc = scale * (q @ ka.T)
        if held is not None:
            sc[:, :n] = np.where(held, sc[:, :n], -np.inf)
        sc[:, n:] = np.where(see, sc[:, n:], -np.inf)
        top = sc.max(-1, keepdims=True, initial=-np.inf)
        top = np.where(np.isinf(top), 0, top)
        e = np.exp(sc - top)
        l = e.sum(-1, keepdims=True)
        p = np.divide(e, l, out=np.zeros_like(e), where=l > 0)
        self.out, self.p = p @ va, p
        with np.errstate(divide="ignore"):
            self.lse = top[:, 0] + np.log(l[:, 0])
        pair = lambda x: x[:, :64] ** 2 + x[:, 64:] ** 2  # noqa: E731
        sig = abs(scale) * 2.0 ** -11 * np.sqrt(pair(q) @ pair(k).T)
        v2 = (va ** 2).sum(-1)
        away = v2[None, :n] - 2 * self.out @ v.T + (self.out ** 2).sum(-1, keepdims=True)
        away = np.maximum(away, 0)
        pk, most = p[:, :n], p.max(-1, keepdims=True, initial=0)
        w2 = np.maximum(2.0 ** -11 * pk, np.where(pk > 0, 2.0 ** -29 * most, 0)) ** 2 / 3
        self.V = (pk ** 2 * sig ** 2 * away + w2 * v2[None, :n]).sum(-1)
        self.C = (pk * sig * np.sqrt(away)).sum(-1)
        self.sums = 2.0 ** -18 * (p @ np.sqrt(v2))
        self.size = np.linalg.norm(self.out, axis=-1)
        self.lse_v, self.lse_c = (pk ** 2 * sig ** 2).sum(-1), (pk * sig).sum(-1)
        qk = abs(scale) * (np.abs(q) @ np.abs(ka).T).max(-1, initial=0)
        finite = np.where(np.isinf(self.lse), 0, self.lse)
        self.lse_sums = 2.0 ** -16 + 2.0 ** -18 * np.abs(finite) + 2.0 ** -19 * qk

    def tolerance(self, alike=False):
        """Per row, on the error's norm and on lse: four standard deviations
        (alike: four times the plain sum) beside what rounds surely."""
        four = self.C if alike else np.sqrt(self.V)
        out = 2.0 ** -8 * self.size + 4 * four + 4 * np.sqrt(self.V) * alike + self.sums
        return out, 4 * (self.lse_c if alike else np.sqrt(self.lse_v)) + self.lse_sums

    def check(self, out, lse, alike=False):
        """Asserts a kernel's rows (fp64 [R][128], [R])."""
        to, tl = self.tolerance(alike)
        empty = np.isinf(self.lse)
        assert np.isfinite(out).all() and (out[empty] == 0).all()
        assert (np.isneginf(lse) == empty).all()
        err = np.linalg.norm(out - self.out, axis=-1)
        assert (err <= to).all(), ("row", int((err - to).argmax()), err.max(), to.min())
        gap = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, self.lse))
        assert (gap <= tl).all(), ("lse", int((gap - tl).argmax()), gap.max(), tl.min())


def check_all(rows):
    """Asserts the norm of many rows' errors together, [(Expected, out)]: root mean
    squares add, and a quarter covers what the sum of some hundred squares of
    uniform errors strays from its mean.  Returns the relative error."""
    err = sum(((o - e.out) ** 2).sum() for e, o in rows)
    want = sum((2.0 ** -16 / 3 * e.size ** 2 + e.V).sum() for e, _ in rows)
    sums = math.sqrt(sum((e.sums ** 2).sum() for e, _ in rows))
    assert math.sqrt(err) <= 1.25 * math.sqrt(want) + sums, (math.sqrt(err), math.sqrt(want), sums)
    return math.sqrt(err / max(sum((e.size ** 2).sum() for e, _ in rows), 1e-300))
