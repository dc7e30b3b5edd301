"""Accuracy of tree attention where the worst-case bounds say little: long caches,
many tiles per CTA, references that move.  Against fp64 with the statistical
tolerances of tests/tree_oracle.py (derived there; tests/test_tree_oracle.py plants
the mistakes that they have to find)."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_serve import check_tree, gen, i32, nq, tree_mask, see_of, u32  # noqa: F401
from tests.tree_oracle import D, Expected, check_all, dequant, hadamard

pytestmark = pytest.mark.gpu
UNITS, HEADS = 18, 8  # 144 pairs: a wave of CTAs, each with all tiles of its pair


def splits(nq, G, nodes, n, shared, ragged, units=UNITS, heads=HEADS):
    """Splits of the cache, from the workspace: partial sums of 130 floats per row
    and split (rounded up to 256 bytes), 32 KB of angles per tile."""
    tiles = -(-n // 128)
    b = nq.lib().nq_tree_attend_workspace_bytes(units, heads, G, nodes, n, int(shared), int(ragged))
    b -= (1 if shared else units) * tiles * 16 * 128 * 16
    return b // (units * heads * G * nodes * 130 * 4)


def encode(nq, x, bits, key_pos=None, tab=None, max_pos=0):
    """Rows x [units][heads][n][128] (fp32) packed, unit by unit; key_pos: rotated
    keys at these positions."""
    U, H, n, _ = x.shape
    st = nq.PackedStore.empty(U, H, n, bits)
    for u in range(U):
        row = x[u:u + 1].to(torch.bfloat16)
        one = st.select_units(slice(u, u + 1))
        if key_pos is None:
            nq.nq_encode(None, row, None, one, n)
        else:
            # the listed positions' rows of a cache that holds them there
            full = torch.zeros(1, H, max_pos, D, dtype=torch.bfloat16, device="cuda")
            full[:, :, key_pos[u].long()] = row
            nq.nq_encode(full, None, one, None, n, tab, max_pos, kept=key_pos[u:u + 1])
    return st


def to_pages(nq, ks, vs, P, seed):
    """The same caches in shuffled pages of P: (stores, table)."""
    U, H, n = ks.meta.shape
    width = -(-n // P)
    ids = torch.from_numpy(np.random.default_rng(seed).permutation(U * width + 3)).cuda()
    table = ids[:U * width].view(U, width)
    out = []
    for s in (ks, vs):
        p = nq.PackedStore.empty(U * width + 3, H, P, s.bits)
        for a, b in ((s.codes, p.codes), (s.meta, p.meta)):
            pad = torch.zeros(U, H, width * P, *a.shape[3:], dtype=a.dtype, device="cuda")
            pad[:, :, :n] = a
            b[table.flatten()] = pad.unflatten(2, (width, P)).transpose(1, 2).flatten(0, 1)
        out.append(p)
    return *out, table.to(torch.int32).contiguous()


class Call:
    """One call over stores of UNITS x HEADS caches, and its oracle for some pairs."""

    def __init__(self, nq, q, Kn, Vn, ks, vs, theta, tab, max_pos, lens=None, pos=None, mask=None,
                 scale=D ** -0.5, page=0):
        self.q, self.Kn, self.Vn, self.ks, self.vs, self.theta = q, Kn, Vn, ks, vs, theta
        self.lens, self.pos, self.mask, self.scale, self.n = lens, pos, mask, scale, ks.meta.shape[2]
        a, b, table = (ks, vs, None) if not page else to_pages(nq, ks, vs, page, 5)
        lt = None if lens is None else i32(lens)
        self.out, self.lse = nq.nq_tree_attend(q, Kn, Vn, a, b, self.n, tab, max_pos, mask=mask, lens=lt,
                                               table=table, positions=pos, scale=scale, lse=True)
        torch.cuda.synchronize()
        assert nq.device_error() == 0

    def pair(self, u, h):
        """(Expected, out, lse) of the rows of KV head h of unit u, [G * nodes]."""
        U, Hq, M, _ = self.q.shape
        G = Hq // self.Kn.shape[1]
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        m = self.n if self.lens is None else self.lens[u]
        at = np.arange(m) if self.pos is None else self.pos[u, :m].cpu().numpy()
        k = dequant(u32(self.ks.codes[u, h, :m]), u32(self.ks.meta[u, h, :m]), self.ks.bits, at, self.theta)
        v = dequant(u32(self.vs.codes[u, h, :m]), u32(self.vs.meta[u, h, :m]), self.vs.bits)
        see = np.tile(see_of(self.mask, U, M)[u], (G, 1))
        e = Expected(f(self.q[u, h * G:(h + 1) * G]).reshape(G * M, D), k, v, f(self.Kn[u, h]),
                     f(self.Vn[u, h]), see, self.scale)
        return e, f(self.out[u, h * G:(h + 1) * G]).reshape(G * M, D), \
            f(self.lse[u, h * G:(h + 1) * G]).reshape(G * M)


def drafts(seed, G, nodes, q_scale=1.0):
    g = gen(seed)
    mk = lambda h: torch.randn(UNITS, h, nodes, D, generator=g, device="cuda")  # noqa: E731
    return (mk(HEADS * G) * q_scale).to(torch.bfloat16), mk(HEADS).to(torch.bfloat16), mk(HEADS).to(torch.bfloat16)


PAIRS = ((0, 0), (UNITS // 2, 3), (UNITS - 1, HEADS - 1))


@pytest.mark.parametrize("nodes,G,n,page,ragged,kept,bk,bv", [
    (1, 4, 16300, 0, False, False, 3, 2), (4, 8, 9000, 64, True, False, 2, 2),
    (16, 4, 16384, 64, False, False, 2, 3), (32, 4, 12345, 0, True, False, 3, 3),
    (32, 8, 8000, 48, False, False, 3, 2), (19, 7, 9001, 0, False, True, 3, 2)])
def test_long_pipelines_against_the_oracle(nq, nodes, G, n, page, ragged, kept, bk, bv):  # noqa: F811
    """Twelve tiles at least pass through a CTA (every buffer and barrier phase is
    used again), scores flat enough that each tile counts."""
    theta, max_pos = 5e5, n + n // 2 if kept else n
    g = gen(n)
    tab = nq.rope_tables(theta, max_pos)
    pos = torch.stack([torch.randperm(max_pos, generator=g, device="cuda")[:n].sort()[0]
                       for _ in range(UNITS)]).to(torch.int32) if kept else None
    at = pos if kept else torch.arange(n, dtype=torch.int32, device="cuda").expand(UNITS, n).contiguous()
    x = lambda: torch.randn(UNITS, HEADS, n, D, generator=g, device="cuda")  # noqa: E731
    ks, vs = encode(nq, x(), bk, at, tab, max_pos), encode(nq, x(), bv)
    lens = None
    if ragged:
        lens = [int(z) for z in torch.randint(n // 2, n + 1, (UNITS,), generator=g, device="cuda")]
        lens[0], lens[1], lens[UNITS - 1] = n, 0, n - 129
    assert splits(nq, G, nodes, n, not kept, ragged) * 12 <= -(-n // 128)
    call = Call(nq, *drafts(n, G, nodes, 0.5), ks, vs, theta, tab, max_pos, lens, pos,
                tree_mask(UNITS, nodes, "tree", n), page=page)
    rows = []
    for u, h in PAIRS + (((1, 2),) if ragged else ()):
        e, o, l = call.pair(u, h)
        e.check(o, l)
        rows.append((e, o))
    assert check_all(rows) < 0.003


@pytest.mark.parametrize("nodes,G", [(1, 4), (4, 8), (16, 4), (32, 4)])
@pytest.mark.parametrize("page", [0, 64])
def test_every_tile_counts_once(nq, nodes, G, page):  # noqa: F811
    """The values of tile j are along row j of H, so coefficient j of an output in
    that basis is tile j's weight: lost, repeated and stale tiles show one by one.
    A coefficient's error: bf16 roundings, independent and within 2^-8 |o_i|, six
    standard deviations 2^-8 |o| / (128 sqrt 3); the tokens' errors by 4 sqrt V
    and the fp32 sums along a unit vector, over sqrt 128."""
    n, theta = 16300, 1e6  # 128 tiles
    g = gen(nodes)
    tab = nq.rope_tables(theta, n)
    at = torch.arange(n, dtype=torch.int32, device="cuda").expand(UNITS, n).contiguous()
    H = torch.from_numpy(hadamard()).float().cuda()
    v = H[torch.arange(n, device="cuda") // 128].expand(UNITS, HEADS, n, D) + \
        0.1 * torch.randn(UNITS, HEADS, n, D, generator=g, device="cuda")
    ks = encode(nq, torch.randn(UNITS, HEADS, n, D, generator=g, device="cuda"), 3, at, tab, n)
    vs = encode(nq, v, 2)
    del v
    assert splits(nq, G, nodes, n, True, False) == 1
    call = Call(nq, *drafts(3, G, nodes, 0.25), ks, vs, theta, tab, n,
                mask=torch.zeros(UNITS, nodes, 1, dtype=torch.int64, device="cuda"), page=page)
    h = hadamard() / D
    for u, kv in PAIRS:
        e, o, l = call.pair(u, kv)
        e.check(o, l)
        got, want = o @ h, e.out @ h
        tol = 6 * 2.0 ** -8 * e.size / (D * math.sqrt(3)) + (4 * np.sqrt(e.V) + e.sums) / math.sqrt(D)
        assert (tol < 0.25 * np.abs(want).min(-1)).all()
        assert (np.abs(got - want) <= tol[:, None]).all(), np.argwhere(np.abs(got - want) > tol[:, None])[:4]


def along(d, amp, noise, g):
    """Keys along unit rows d [units][heads][128] at strengths amp [n]."""
    x = torch.randn(*d.shape[:2], len(amp), D, generator=g, device="cuda") * noise
    return x + d[:, :, None] * torch.as_tensor(amp, dtype=torch.float32, device="cuda")[:, None]


@pytest.mark.parametrize("nodes,G", [(3, 2), (16, 2), (16, 4), (32, 4)])
@pytest.mark.parametrize("shape", ["rising", "saw"])
def test_moving_references(nq, nodes, G, shape):  # noqa: F811
    """Scores that rise along the cache, in one sweep or in rising teeth, by up to
    hundreds of powers of two with all tiles in one CTA: references move at many
    tiles, at different ones for different rows, and the sums in tensor memory are
    rescaled.  Errors are counted as alike (the keys are), and the tolerance stays
    below a tenth of sum p |v|."""
    n, theta = 2100, 1e4
    g = gen(nodes)
    t = np.arange(n)
    amp = 60 * t / n - 30 if shape == "rising" else 20 * (t % 700) / 700 + 20 * (t // 700) - 30
    q, Kn, Vn = drafts(nodes, G, nodes)
    d = torch.randn(UNITS, HEADS, D, generator=g, device="cuda")
    d = d / d.norm(dim=-1, keepdim=True)
    # row i of a head's queries: along +-d by strengths that differ, and its own part
    lead = (11.0 - 0.3 * torch.arange(nodes, device="cuda")) * (1 - 2 * (torch.arange(nodes, device="cuda") % 3 == 1).float())
    q = (q.float() * 0.3 + d.repeat_interleave(G, 1)[:, :, None] * lead[:, None]).to(torch.bfloat16)
    tab = nq.rope_tables(theta, n)
    at = torch.arange(n, dtype=torch.int32, device="cuda").expand(UNITS, n).contiguous()
    ks = encode(nq, along(d, amp, 0.5, g), 3, at, tab, n)
    vs = encode(nq, torch.randn(UNITS, HEADS, n, D, generator=g, device="cuda"), 2)
    assert splits(nq, G, nodes, n, True, False) == 1
    for scale in (0.1, 0.4, -0.4):
        call = Call(nq, q, Kn, Vn, ks, vs, theta, tab, n, mask=tree_mask(UNITS, nodes, "tree", 1), scale=scale)
        for u, h in PAIRS:
            e, o, l = call.pair(u, h)
            spread = e.sums * 2.0 ** 18  # sum p |v|
            assert (e.tolerance(alike=True)[0] <= 0.1 * spread).all()
            e.check(o, l, alike=True)


@pytest.mark.parametrize("nodes,G", [(1, 4), (16, 4), (32, 4)])
@pytest.mark.parametrize("where", [0, 7000, 16299])
def test_a_sink_token_of_no_value(nq, nodes, G, where):  # noqa: F811
    """One token takes most of the weight (its score is 15 nats, 22 powers of two,
    above the others before its key is coded, which may take a tenth off) and its
    value is 0, as at the start of many caches: what is left is the sum of the small
    weights, rounded by 2^-29 of the largest.  (For most rows the tolerance has to
    stay below a tenth of the output: sums not rescaled, or flushed, are off by more.)"""
    n, theta = 16300, 5e5
    g = gen(where + nodes)
    d = torch.ones(UNITS, HEADS, D, device="cuda") / math.sqrt(D)
    q, Kn, Vn = drafts(where, G, nodes, 0.5)
    q = (q.float() + 6 * d[0, 0]).to(torch.bfloat16)
    amp = np.zeros(n)
    amp[where] = 15 / (6 * D ** -0.5)
    tab = nq.rope_tables(theta, n)
    at = torch.arange(n, dtype=torch.int32, device="cuda").expand(UNITS, n).contiguous()
    k = along(d, amp, 1.0, g)
    k[:, :, where] = d * amp[where]
    v = torch.randn(UNITS, HEADS, n, D, generator=g, device="cuda")
    v[:, :, where] = 0
    ks, vs = encode(nq, k, 3, at, tab, n), encode(nq, v, 2)
    del k, v
    call = Call(nq, q, Kn, Vn, ks, vs, theta, tab, n,
                mask=torch.zeros(UNITS, nodes, 1, dtype=torch.int64, device="cuda"))
    for u, h in PAIRS:
        e, o, l = call.pair(u, h)
        assert (e.p[:, where] > 0.5).all() and np.median(e.tolerance()[0] / e.size) < 0.1
        e.check(o, l)


SMALL = [dict(units=2, heads=4, G=4, nodes=5, n=n) for n in (0, 1, 2, 127, 128, 129, 257, 1000)] + \
    [dict(units=1, heads=2, G=G, nodes=7, n=300, bk=bk, bv=bv) for G in (1, 3, 8) for bk in (2, 3) for bv in (2, 3)] + \
    [dict(units=1, heads=1, G=G, nodes=m, n=260, kind=k) for m, G in ((1, 1), (17, 4), (64, 4), (130, 8), (1024, 1))
     for k in ("chain", "tree")] + \
    [dict(units=5, heads=3, G=2, nodes=6, n=290, P=P, lens=[290, 0, 1, 128, 131], kind="sparse") for P in (1, 16, 100)] + \
    [dict(units=2, heads=8, G=4, nodes=9, n=700, kept=True, theta=1e6),
     dict(units=2, heads=4, G=7, nodes=9, n=700, kept=True, pos_base=60000, theta=1e6, layout="head"),
     dict(units=1, heads=2, G=4, nodes=8, n=400, sigma_v=1000.0),
     dict(units=1, heads=2, G=4, nodes=8, n=400, sigma_v=2.0 ** -9),
     dict(units=2, heads=1, G=3, nodes=5, n=12345), dict(units=3, heads=1, G=4, nodes=7, n=21001, P=64,
                                                        lens=[21001, 7000, 20872])]


@pytest.mark.parametrize("case", range(len(SMALL)))
def test_relative_error(nq, case):  # noqa: F811
    """The error's norm over the output's, beside the bounds per element: unit-normal
    queries and keys give sigma_t^2 <= 2^-21 (two coordinates' squares per pair and
    side, 64 pairs, over 128), the weights 2^-22 / 3, the output 2^-16 / 3: 1.25
    times their root is 0.003."""
    assert check_tree(nq, seed=100 + case, **SMALL[case]) < 0.003
