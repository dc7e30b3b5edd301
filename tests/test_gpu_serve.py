"""GPU tests of the serving calls around the packed cache: page tables, norms
with RoPE, encode into slots, tree attention, and a run of them together.

Integers (page tables, slots, codes) must be equal.  Norms: see norm_bound.
Tree attention, per output element with the exact softmax weights p_t and
scores s_t of the row (fp64):
  |out - ref| <= 2^-8 |ref| + B sum_t p_t |v_t|,   B = 2 ds + 2^-10 + 2^-16,
  |lse - ref| <= ds + 2^-18 (1 + |lse|),
with ds the largest score error.  A rotated key pair of length r (r <= |k_i| +
|k_i'| over RoPE partners i, i') is formed in f16 as u c' + v s', u = (x_i +
x_i')/2 and v = (x_i - x_i')/2 exact, c' = cos - sin, s' = cos + sin: |u| + |v| =
max(|x_i|, |x_i'|) <= r, |v| <= r / sqrt 2 and |u| likewise.  c' and s' are below
sqrt 2, rounded by at most 2^-11 (together 2^-11 r), the product v s' by 2^-11
of at most r, the sum by 2^-11 |k_i|: at most 2^-11 (2 r + |k_i|), so
  ds = scale max_t sum_i (|q_i| + |q_i'|) |k_ti| 2^-11 * 3
(sum_i |q_i| r <= sum_i (|q_i| + |q_i'|) |k_ti| pair by pair, and |q_i| |k_ti|
is part of it; the fp32 sums add below 2^-20 of the same sum: 2^-18); the
weights are rounded to f16 (2^-11; the scaled codes are exact), a weight error
e^ds acts on numerator and sum (2 ds), fp32 sums add below 2^-16, and the
output is rounded to bf16 (half a step: 2^-8 relative).
"""
import ctypes
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def nq():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from e8_lattice_vector_nq_b200 import build, nq as nqmod

    build.build()
    return nqmod


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def u32(t):
    return t.detach().cpu().contiguous().numpy().view(np.uint32)


# ------------------------------------------------------------- page tables
def ref_pages(lens, counts, P, free, taken, table, rows):
    """The definition, one token at a time."""
    S, W = table.shape
    table = table.copy()
    slots, pos = np.full(rows, -1, np.int64), np.zeros(rows, np.int64)
    at, row, flags = max(taken, 0), 0, 0
    starts, out = [], []
    for s in range(S):
        l, c = max(int(lens[s]), 0), max(int(counts[s]), 0)
        have, need = -(-l // P), min(-(-(l + c) // P), W)
        if c and l % P and l // P < W and table[s, l // P] < 0:
            flags |= 2
        if c and -(-(l + c) // P) > W:
            flags |= 2
        for j in range(have, need):
            table[s, j] = free[at] if at < len(free) else -1
            at += 1
        starts.append(row)
        out.append(l + c)
        for t in range(l, l + c):
            if row < rows:
                page = int(table[s, t // P]) if t // P < W else -1
                slots[row] = page * P + t % P if page >= 0 and page * P + t % P < 2 ** 31 else -1
                pos[row] = t
            row += 1
    flags |= (1 if at > len(free) else 0) | (4 if row > rows else 0)
    return table, out, starts + [row], slots, pos, [at, flags]


def run_pages(nq, lens, counts, P, free, table, rows, taken=None, **kw):
    tt = i32(table)
    r = nq.nq_page_tables(i32(lens), i32(counts), P, i32(free), tt, rows,
                          taken=None if taken is None else i32([taken]), **kw)
    want = ref_pages(lens, counts, P, free, taken or 0, np.asarray(table), rows)
    for name, g, w in zip(("table", "lens", "starts", "slots", "positions", "used"),
                          (tt, r.lens, r.starts, r.slots, r.positions, r.used), want):
        np.testing.assert_array_equal(g.cpu().numpy(), np.asarray(w), err_msg=name)
    return tt, r


def page_case(seed, S, P, max_len, max_new, W=None):
    rng = np.random.default_rng(seed)
    lens, counts = rng.integers(0, max_len + 1, S), rng.integers(0, max_new + 1, S)
    have, need = -(-lens // P), -(-(lens + counts) // P)
    pages = rng.permutation(int(need.sum()) + 3)
    W = int(need.max()) + 1 if W is None else W
    table = np.full((S, W), -1, np.int32)
    at = 0
    for s in range(S):
        k = min(have[s], W)
        table[s, :k] = pages[at:at + k]
        at += have[s]
    return lens, counts, pages[at:], table


@pytest.mark.parametrize("S,P,max_len,max_new", [(1, 1, 0, 1), (1, 16, 100, 0), (3, 7, 50, 20),
                                                 (64, 64, 4000, 1), (513, 16, 300, 40),
                                                 (1021, 256, 9, 700), (8192, 100, 300, 3)])
@pytest.mark.parametrize("pad", [0, 5])
def test_page_tables(nq, S, P, max_len, max_new, pad):
    lens, counts, free, table = page_case(S, S, P, max_len, max_new)
    run_pages(nq, lens, counts, P, free, table, int(counts.sum()) + pad)


def test_page_tables_edges(nq):
    lens, counts, free, table = page_case(5, 40, 16, 200, 60)
    rows = int(counts.sum())
    run_pages(nq, lens, counts, 16, free[:3], table, rows)            # list too short
    run_pages(nq, lens, counts, 16, [], table, rows)                  # none left
    run_pages(nq, lens, counts, 16, free, table, rows - 7)            # too few rows
    run_pages(nq, lens, counts, 16, free, table, 0)                   # no rows
    run_pages(nq, lens, counts, 16, free, table[:, :4].copy(), rows)  # table rows too short
    run_pages(nq, lens, counts, 16, np.concatenate([[9] * 11, free]), table, rows, taken=11)
    run_pages(nq, lens, counts, 16, free, table, rows, taken=-4)
    bad = table.copy()
    bad[:, :] = -1                                                    # started pages lost
    run_pages(nq, lens, counts, 16, free, bad, rows)
    neg = lens.copy()
    neg[::3] = -5
    nc = counts.copy()
    nc[1::4] = -9
    run_pages(nq, neg, nc, 16, np.arange(300), table, rows)
    run_pages(nq, lens, counts, 16, free + 2 ** 27, table, rows)      # slots past 31 bits
    run_pages(nq, [7], [3], 65536, [5, 6], [[2]], 4)


def test_page_tables_repeat_offset_outputs_and_no_requests(nq):
    lens, counts, free, table = page_case(9, 33, 8, 100, 30)
    rows = int(counts.sum()) + 9
    tt, r = run_pages(nq, lens, counts, 8, free, table, rows)
    again = nq.nq_page_tables(i32(lens), i32(counts), 8, i32(free), tt, rows)
    for x in ("lens", "starts", "slots", "positions", "used"):
        assert torch.equal(getattr(r, x), getattr(again, x))
    buf = torch.full((2 * rows + 8,), 77, dtype=torch.int32, device="cuda")
    out = nq.PageTables(torch.empty_like(r.lens), torch.empty_like(r.starts), buf[1:1 + rows],
                        buf[rows + 3:2 * rows + 3], torch.empty_like(r.used))
    nq.nq_page_tables(i32(lens), i32(counts), 8, i32(free), tt, rows, out=out)
    assert torch.equal(out.slots, r.slots) and torch.equal(out.positions, r.positions)
    assert buf[0] == 77 and (buf[rows + 1:rows + 3] == 77).all() and (buf[2 * rows + 3:] == 77).all()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    e = nq.nq_page_tables(none, none, 8, none, none.view(0, 4), 6)
    assert e.slots.tolist() == [-1] * 6 and e.positions.tolist() == [0] * 6
    assert e.starts.tolist() == [0] and e.used.tolist() == [0, 0]


# ------------------------------------------------------------- norm + RoPE
def ref_norm(x, w, eps, pos, theta):
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double()
    ang = pos.double()[:, None, :, None] * theta ** (-torch.arange(64, device=x.device).double() / 64)
    c, s = torch.cos(ang), torch.sin(ang)
    a, b = y[..., :64], y[..., 64:]
    return torch.cat([a * c - b * s, b * c + a * s], -1), y


def norm_bound(ref, y, dtype):
    """y: 19 additions and 16 squares in the sum (halved by the square root),
    the mean's scaling, eps, the root and two products: 13 roundings of 2^-24;
    cos and sin: two table values and two roundings each, under 3 * 2^-24
    absolute; the rotation: two roundings.  Together below 20 * 2^-24 of
    |y_i| + |y_i'|; then the output's rounding, half a bf16 step."""
    pair = y.abs() + torch.cat([y[..., 64:], y[..., :64]], -1).abs()
    b = 20 * 2.0 ** -24 * pair
    return b + (2.0 ** -8 * (ref.abs() + b) if dtype == torch.bfloat16 else 0)


@pytest.mark.parametrize("units,rows,hq,hk,din,dq,dk,layout", [
    (1, 1, 1, 1, "b", "b", "b", "token"), (2, 3, 8, 2, "b", "f", "b", "token"),
    (1, 77, 28, 4, "b", "f", "b", "fused"), (3, 130, 5, 1, "f", "f", "b", "head"),
    (1, 2048, 32, 8, "b", "b", "b", "fused"), (64, 1, 32, 8, "b", "b", "b", "fused"),
    (2, 9, 12, 0, "f", "b", "b", "token"), (2, 301, 0, 7, "b", "b", "f", "head"),
])
def test_norm_rope(nq, units, rows, hq, hk, din, dq, dk, layout):
    T = {"b": torch.bfloat16, "f": torch.float32}
    g = gen(rows)
    theta, max_pos = 5e5, 100000
    if layout == "head":
        mk = lambda h: torch.randn(units, h, rows, D, generator=g, device="cuda").to(T[din])  # noqa: E731
        q, k = mk(hq) if hq else None, mk(hk) if hk else None
    else:
        extra = 3 if layout == "fused" else 0
        f = torch.randn(units, rows, hq + hk + extra, D, generator=g, device="cuda") * 3
        f = f.to(T[din]).permute(0, 2, 1, 3)
        q, k = f[:, :hq] if hq else None, f[:, hq:hq + hk] if hk else None
    for t in (q, k):
        if t is not None:
            t[:, :, -1] = 0  # a zero row
            t[0, 0, 0] *= 1e4
    wq = torch.randn(D, generator=g, device="cuda") if rows != 77 else None
    wk = torch.rand(D, generator=g, device="cuda") if hk != 7 else None
    pos = torch.randint(0, max_pos, (units, rows), generator=g, device="cuda", dtype=torch.int32)
    pos[0, 0] = max_pos - 1
    tab = nq.rope_tables(theta, max_pos)
    keep = [t.clone() if t is not None else None for t in (q, k)]
    for p, base in ((pos, 0), (None, max_pos - rows), (pos // 2, 33)):
        qo, ko = nq.nq_qk_norm_rope(q, k, tab, max_pos, positions=p, pos_base=base, q_weight=wq,
                                    k_weight=wk, eps=1e-5, q_dtype=T[dq] if hq else None,
                                    k_dtype=T[dk] if hk else None)
        at = base + (p if p is not None else torch.arange(rows, device="cuda")[None].expand(units, rows))
        for x, w, o, kept in ((q, wq, qo, keep[0]), (k, wk, ko, keep[1])):
            if x is None:
                assert o is None
                continue
            ref, y = ref_norm(x, w, 1e-5, at, theta)
            assert (o.double() - ref).abs().le(norm_bound(ref, y, o.dtype)).all()
            assert torch.equal(x, kept)


def test_norm_rope_in_place_views_and_shared_positions(nq):
    g = gen(4)
    f = torch.randn(2, 11, 10, 160, generator=g, device="cuda").to(torch.bfloat16)
    base = f.clone()
    q, k = f[:, :, :7, :D].permute(0, 2, 1, 3), f[:, :, 7:9, 32:].permute(0, 2, 1, 3)
    tab = nq.rope_tables(1e4, 512)
    pos = torch.randint(0, 512, (1, 11), generator=g, device="cuda", dtype=torch.int32).expand(2, 11)
    want = nq.nq_qk_norm_rope(q, k, tab, 512, positions=pos)
    got = nq.nq_qk_norm_rope(q, k, tab, 512, positions=pos, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    # nothing beside the views moved
    assert torch.equal(f[:, :, 9], base[:, :, 9])
    assert torch.equal(f[:, :, :7, D:], base[:, :, :7, D:])
    assert torch.equal(f[:, :, 7:9, :32], base[:, :, 7:9, :32])


def test_norm_rope_gives_what_the_codec_undoes(nq):
    """Keys rotated here and encoded come back as they were normalised: the
    encode's RoPE removal is this rotation's inverse (3-bit error scale)."""
    g = gen(8)
    k = torch.randn(1, 2, 300, D, generator=g, device="cuda").to(torch.bfloat16)
    tab = nq.rope_tables(1e4, 300)
    _, kr = nq.nq_qk_norm_rope(None, k, tab, 300, k_dtype=torch.bfloat16)
    st = nq.PackedStore.empty(1, 2, 300, 3)
    nq.nq_encode(kr, None, st, None, 300, tab, 300)
    back = torch.empty_like(kr)
    nq.nq_decode(st, None, 300, back, None, tab, 300)
    err = (back.float() - kr.float()).norm(dim=-1) / kr.float().norm(dim=-1)
    assert err.max() < 0.35


# ------------------------------------------------------- encode into slots
@pytest.mark.parametrize("rows,heads,P,bk,bv", [(1, 1, 1, 3, 2), (17, 8, 16, 2, 2), (300, 3, 7, 3, 3),
                                                (64, 12, 64, 2, 3), (1100, 8, 100, 3, 2)])
def test_encode_slots_matches_the_oracle(nq, oq, rows, heads, P, bk, bv):
    g, rng = gen(rows), np.random.default_rng(rows)
    max_pos, theta = 4 * rows + 300, 1e6
    # token-major rows, as a model leaves them
    kv = torch.randn(rows, 2 * heads, D, generator=g, device="cuda").to(torch.bfloat16)
    K, V = kv[:, :heads].permute(1, 0, 2), kv[:, heads:].permute(1, 0, 2)
    pages = -(-rows // P) + 2
    slot = rng.permutation(pages * P)[:rows].astype(np.int32)
    drop = rng.random(rows) < 0.2
    slot[drop] = np.where(np.arange(drop.sum()) % 2 == 0, -1, pages * P + 5)
    pos = rng.permutation(max_pos)[:rows].astype(np.int32)
    ks, vs = nq.PackedStore.empty(pages, heads, P, bk), nq.PackedStore.empty(pages, heads, P, bv)
    for t in (ks.codes, ks.meta, vs.codes, vs.meta):
        t.fill_(0x5A5A5A5A)
    tab = nq.rope_tables(theta, max_pos)
    nq.nq_encode_slots(K, V, ks, vs, i32(slot), i32(pos), tab, max_pos)
    torch.cuda.synchronize()
    # the oracle encodes a cache that holds the rows at their positions
    full = torch.zeros(2, heads, max_pos, D, dtype=torch.bfloat16)
    full[0][:, pos], full[1][:, pos] = K.cpu(), V.cpu()
    u16 = lambda t: t.contiguous().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    r = oq.encode_unit(u16(full[0]), u16(full[1]), rows, kept=pos, theta=theta, bits_k=bk, bits_v=bv)
    used = np.flatnonzero((slot >= 0) & (slot < pages * P))
    pg, off = slot[used] // P, slot[used] % P
    for st, c, m in ((ks, "k_codes", "k_meta"), (vs, "v_codes", "v_meta")):
        want_c = np.full(st.codes.shape, 0x5A5A5A5A, np.uint32)
        want_m = np.full(st.meta.shape, 0x5A5A5A5A, np.uint32)
        want_c[pg, :, off] = np.asarray(r[c]).reshape(heads, rows, -1)[:, used].transpose(1, 0, 2)
        want_m[pg, :, off] = np.asarray(r[m]).reshape(heads, rows)[:, used].T
        np.testing.assert_array_equal(u32(st.codes), want_c)
        np.testing.assert_array_equal(u32(st.meta), want_m)


def test_encode_slots_one_side_contiguous_cache_and_repeated_positions(nq):
    """Pages as whole sequences (page_size = cap), keys alone and values alone,
    several rows at one position: the same bits as nq_encode row by row."""
    g = gen(2)
    K = torch.randn(4, 6, D, generator=g, device="cuda").to(torch.bfloat16)
    V = torch.randn(4, 6, D, generator=g, device="cuda").to(torch.bfloat16)
    tab = nq.rope_tables(1e4, 64)
    ks, vs = nq.PackedStore.empty(3, 4, 50, 3), nq.PackedStore.empty(3, 4, 50, 2)
    for t in (ks.codes, ks.meta, vs.codes, vs.meta):
        t.zero_()
    slot, pos = [0, 50, 100, 49, 99, 149], [13, 13, 13, 0, 63, 63]
    nq.nq_encode_slots(K, None, ks, None, i32(slot), i32(pos), tab, 64)
    nq.nq_encode_slots(None, V, None, vs, i32(slot))
    k1, v1 = nq.PackedStore.empty(1, 4, 1, 3), nq.PackedStore.empty(1, 4, 1, 2)
    for r, (s, p) in enumerate(zip(slot, pos)):
        nq.nq_encode(K[None, :, r:r + 1].contiguous(), V[None, :, r:r + 1].contiguous(), k1, v1, 1,
                     tab, 64, pos_base=p)
        for a, b in ((ks, k1), (vs, v1)):
            assert torch.equal(a.codes[s // 50, :, s % 50], b.codes[0, :, 0])
            assert torch.equal(a.meta[s // 50, :, s % 50], b.meta[0, :, 0])
    assert torch.count_nonzero(ks.meta) == 24 and torch.count_nonzero(vs.meta) == 24
    none = torch.empty(4, 0, D, dtype=torch.bfloat16, device="cuda")
    nq.nq_encode_slots(none, none, ks, vs, i32([]), i32([]), tab, 64)


# ---------------------------------------------------------- tree attention
def unpack(codes, meta, bits):
    """fp64 values before RoPE: kappa * H t, [..., 128]."""
    c, m = u32(codes).astype(np.uint64), u32(meta)
    i = np.arange(D)
    w, off = bits * i // 32, bits * i % 32
    c = np.concatenate([c, np.zeros(c.shape[:-1] + (1,), np.uint64)], -1)
    j = ((c[..., w] | (c[..., w + 1] << np.uint64(32))) >> off.astype(np.uint64)) & np.uint64(2 ** bits - 1)
    half = (m[..., None] >> (i // 8).astype(np.uint32)) & 1
    t = 2.0 * j.astype(np.float64) - 2 ** bits + 2 - half
    h = np.ones((1, 1))
    for _ in range(7):
        h = np.kron(np.array([[1, 1], [1, -1]]), h)
    sig = (m >> 16).astype(np.uint16).view(np.float16).astype(np.float64)
    return (t @ h) * (sig / (2 * math.sqrt(D)))[..., None]


def see_of(mask, units, nodes):
    if mask is None:
        return np.broadcast_to(np.tril(np.ones((nodes, nodes), bool)), (units, nodes, nodes))
    b = np.unpackbits(mask.cpu().numpy().view(np.uint8), axis=-1, bitorder="little")[..., :nodes]
    return np.broadcast_to(b.astype(bool), (units, nodes, nodes))


def ref_tree(q, Kn, Vn, ks, vs, lens, table, P, positions, pos_base, theta, mask, scale):
    """(out, lse, bound on out, bound on lse), fp64 numpy."""
    U, Hq, M, _ = q.shape
    H = Kn.shape[1]
    G = Hq // H
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    q, Kn, Vn = f(q), f(Kn), f(Vn)
    out, ob = np.zeros(q.shape), np.zeros(q.shape)
    lse, lb = np.zeros((U, Hq, M)), np.zeros((U, Hq, M))
    see = see_of(mask, U, M)
    w = theta ** (-np.arange(64) / 64.0)
    for u in range(U):
        n = lens[u]
        t = np.arange(n)
        ok = np.ones(n, bool)
        if n:
            if table is None:
                kc, km, vc, vm = (x[u, :, :n] for x in (ks.codes, ks.meta, vs.codes, vs.meta))
            else:
                pg = table[u].cpu().numpy()[t // P].astype(np.int64)
                ok = (pg >= 0) & (pg < ks.meta.shape[0])
                pg = torch.tensor(np.where(ok, pg, 0), device="cuda")
                off = torch.tensor(t % P, device="cuda")
                kc, km, vc, vm = (x[pg, :, off].transpose(0, 1) for x in (ks.codes, ks.meta, vs.codes, vs.meta))
            k, v = unpack(kc, km, ks.bits), unpack(vc, vm, vs.bits)
            p = pos_base + (t if positions is None else positions[u, :n].cpu().numpy())
            c, s = np.cos(p[:, None] * w), np.sin(p[:, None] * w)
            k = np.concatenate([k[..., :64] * c - k[..., 64:] * s, k[..., 64:] * c + k[..., :64] * s], -1)
        else:
            k = v = np.zeros((H, 0, D))
        for j in range(Hq):
            h = j // G
            ka, va = np.concatenate([k[h], Kn[u, h]]), np.concatenate([v[h], Vn[u, h]])
            sc = scale * q[u, j] @ ka.T
            sc[:, :n] = np.where(ok, sc[:, :n], -np.inf)
            sc[:, n:] = np.where(see[u], sc[:, n:], -np.inf)
            m = sc.max(-1, keepdims=True)
            e = np.exp(sc - np.where(np.isinf(m), 0, m))
            l = e.sum(-1, keepdims=True)
            pr = np.divide(e, l, out=np.zeros_like(e), where=l > 0)
            out[u, j] = pr @ va
            with np.errstate(divide="ignore"):
                lse[u, j] = (np.where(np.isinf(m), 0, m) + np.log(l))[:, 0]
            qq = np.abs(q[u, j]) + np.abs(np.roll(q[u, j], 64, -1))
            ds = abs(scale) * (qq @ np.abs(k[h]).T).max(-1) * 3 * 2.0 ** -11 if n else np.zeros(M)
            ds = ds + 2.0 ** -18
            ob[u, j] = 2.0 ** -8 * np.abs(out[u, j]) + \
                (2 * ds + (2.0 ** -10 if n else 0) + 2.0 ** -16)[:, None] * (pr @ np.abs(va))
            lb[u, j] = ds + 2.0 ** -18 * (1 + np.abs(np.where(np.isinf(lse[u, j]), 0, lse[u, j])))
    return out, lse, ob, lb


def fill_store(nq, lead, heads, cap, bits, seed, sigma=1.0):
    """A store as the codec leaves it: normal rows encoded (no RoPE needed)."""
    g = gen(seed)
    x = torch.randn(lead, heads, max(cap, 1), D, generator=g, device="cuda") * sigma
    st = nq.PackedStore.empty(lead, heads, max(cap, 1), bits)
    nq.nq_encode(None, x.to(torch.bfloat16), None, st, max(cap, 1))
    return st


def tree_mask(units, nodes, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "chain":
        return None
    see = np.zeros((units, nodes, nodes), bool)
    for u in range(units):
        for i in range(nodes):
            if kind == "tree":
                p = int(rng.integers(-1, i)) if i else -1
                if p >= 0:
                    see[u, i] = see[u, p]
                see[u, i, i] = True
            elif kind == "sparse":
                see[u, i] = rng.random(nodes) < 0.3
            elif kind == "full":
                see[u, i] = True
    W = (nodes + 63) // 64
    b = np.zeros((units, nodes, 64 * W), np.uint8)
    b[..., :nodes] = see
    if kind == "full":
        b[:] = 1  # bits past the last node are not read as nodes
    m = np.packbits(b, axis=-1, bitorder="little").view(np.int64)
    return torch.from_numpy(m.reshape(units, nodes, W).copy()).cuda()


def check_tree(nq, units, heads, G, nodes, n, bk=3, bv=2, P=0, lens=None, kept=False, kind="tree",
               theta=1e4, pos_base=0, scale=None, seed=0, q_scale=1.0, hole=None, layout="token",
               sigma_k=1.0, sigma_v=1.0, shared_mask=False):
    g, rng = gen(seed), np.random.default_rng(seed)
    hl = [n] * units if lens is None else list(lens)
    if P:
        need = [-(-x // P) for x in hl]
        W = -(-n // P) + 1 if n else 1
        pool = rng.permutation(sum(need) + 2).astype(np.int32)
        tb = np.full((units, W), -7, np.int32)
        at = 0
        for u in range(units):
            tb[u, :need[u]] = pool[at:at + need[u]]
            at += need[u]
        if hole is not None:
            tb[hole] = len(pool) + 3
        table, lead, cap = torch.from_numpy(tb).cuda(), len(pool), P
    else:
        table, lead, cap = None, units, n
    ks = fill_store(nq, lead, heads, cap, bk, seed + 1, sigma_k)
    vs = fill_store(nq, lead, heads, cap, bv, seed + 2, sigma_v)
    max_pos = 2 * n + pos_base + 1
    tab = nq.rope_tables(theta, max_pos)
    positions = None
    if kept:
        positions = torch.from_numpy(np.stack([np.sort(rng.permutation(max_pos - pos_base)[:n])
                                               for _ in range(units)]).astype(np.int32)).cuda()
    mk = lambda h: torch.randn(units, nodes, h, D, generator=g, device="cuda")  # noqa: E731
    q = (mk(heads * G) * q_scale).to(torch.bfloat16).permute(0, 2, 1, 3)
    Kn, Vn = (mk(heads).to(torch.bfloat16).permute(0, 2, 1, 3) for _ in range(2))
    if layout == "head":
        q, Kn, Vn = (t.contiguous() for t in (q, Kn, Vn))
    mask = tree_mask(1 if shared_mask else units, nodes, kind, seed)
    if shared_mask and mask is not None:
        mask = mask[0]
    sc = D ** -0.5 if scale is None else scale
    lt = None if lens is None else i32([x if u % 2 else x for u, x in enumerate(lens)])
    ws = nq.tree_attend_workspace(units, heads, G, nodes, n, positions is None, lens is not None)
    ws.fill_(float("nan"))  # nothing of the workspace is read before it is written
    guard = torch.full((units, nodes + 1, heads * G, D), 3.25, dtype=torch.bfloat16, device="cuda")
    buf = guard[:, :nodes].permute(0, 2, 1, 3)
    out, lse = nq.nq_tree_attend(q, Kn, Vn, ks, vs, n, tab, max_pos, mask=mask, lens=lt, table=table,
                                 positions=positions, pos_base=pos_base, scale=sc, out=buf, lse=True,
                                 ws=ws)
    torch.cuda.synchronize()
    assert nq.device_error() == 0
    assert out is buf and (guard[:, nodes] == 3.25).all()
    ref, rl, ob, lb = ref_tree(q, Kn, Vn, ks, vs, hl, table, P, positions, pos_base, theta, mask, sc)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o).all()
    empty = np.isinf(rl)
    assert (np.isneginf(l) == empty).all() and (o[empty] == 0).all()
    bad = np.abs(o - ref) > ob
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:3], np.abs(o - ref).max())
    ld = np.abs(np.where(empty, 0, l) - np.where(empty, 0, rl))
    assert (ld <= lb).all(), ld.max()
    return np.linalg.norm(o - ref) / max(np.linalg.norm(ref), 1e-30)


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 127, 128, 129, 255, 257, 1000])
def test_tree_lengths(nq, n):
    check_tree(nq, 2, 4, 4, 5, n, seed=n)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("bk,bv", [(3, 2), (2, 3), (2, 2), (3, 3)])
def test_tree_groups_and_formats(nq, G, bk, bv):
    check_tree(nq, 1, 2, G, 7, 300, bk, bv, seed=10 * G + bk)


@pytest.mark.parametrize("nodes,G", [(1, 1), (1, 4), (3, 8), (16, 4), (17, 4), (31, 1), (33, 2), (64, 2),
                                     (64, 4), (65, 4), (127, 1), (130, 8), (256, 1), (1024, 1)])
@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_tree_nodes(nq, nodes, G, kind):
    check_tree(nq, 1, 1, G, nodes, 260, kind=kind, seed=nodes + G)


@pytest.mark.parametrize("P", [1, 5, 16, 64, 100, 128, 300])
def test_tree_pages_and_ragged_lengths(nq, P):
    check_tree(nq, 5, 3, 2, 6, 290, P=P, lens=[290, 0, 1, 128, 131], kind="sparse", seed=P)


def test_tree_ragged_contiguous_all_empty(nq):
    check_tree(nq, 3, 2, 4, 4, 200, lens=[0, 0, 0], kind="sparse", seed=3)
    check_tree(nq, 3, 2, 4, 4, 200, lens=[0, 200, 3], kind="full", seed=4)


def test_tree_missing_pages_are_left_out(nq):
    check_tree(nq, 2, 2, 4, 3, 200, P=16, hole=(1, 3), seed=5)
    check_tree(nq, 2, 2, 4, 3, 200, P=16, hole=(1, slice(None)), kind="sparse", seed=6)


def test_tree_bad_positions_and_empty_batches(nq):
    """Positions past the table (out of contract) read some row of it and fault
    nothing; a batch of no units and a pool of no pages are accepted."""
    ks, vs = fill_store(nq, 1, 2, 200, 3, 1), fill_store(nq, 1, 2, 200, 2, 2)
    tab = nq.rope_tables(1e4, 300)
    z = lambda u: torch.randn(u, 2, 3, D, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, K = z(1), z(1)
    bad = torch.full((1, 200), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    bad[0, ::2] = -(2 ** 31)
    for base in (0, 250):
        out = nq.nq_tree_attend(q, K, K, ks, vs, 200, tab, 300, positions=bad, pos_base=base)
        assert torch.isfinite(out).all()
    qk = nq.nq_qk_norm_rope(q, K, tab, 300, positions=bad[:, :3], pos_base=7)
    assert torch.isfinite(qk[0]).all()
    nq.nq_encode_slots(K[0], K[0], ks, vs, i32([1, 2, 3]), bad[0, :3], tab, 300)
    none = nq.nq_tree_attend(z(0), z(0), z(0), ks, vs, 200, tab, 300)
    assert none.shape == (0, 2, 3, D)
    torch.cuda.synchronize()
    # through the C interface: a pool of no pages leaves the draft alone
    L, p = nq.lib(), lambda t: ctypes.c_void_p(t.data_ptr())
    out, want = torch.empty_like(q), nq.nq_tree_attend(q, K, K, None, None, 0)
    ws = nq.tree_attend_workspace(1, 2, 1, 3, 200)
    st = lambda t: nq.KVStrides(*t.stride()[:3])  # noqa: E731
    kd, vd, tb = ks.desc(), vs.desc(), i32([[0, 0]])
    status = L.nq_tree_attend(p(q), st(q), p(K), st(K), p(K), st(K), 1, 2, 1, 3, ctypes.byref(kd),
                              ctypes.byref(vd), 200, None, p(tb), 2, 100, 0, None, 0, 0, p(tab), 300,
                              None, 0, D ** -0.5, p(out), st(out), None, p(ws),
                              ws.numel() * 4, None)
    torch.cuda.synchronize()
    assert status == 0 and torch.equal(out, want)


def test_tree_kept_positions_base_and_layout(nq):
    check_tree(nq, 2, 8, 4, 9, 700, kept=True, theta=1e6, seed=7)
    check_tree(nq, 2, 4, 7, 9, 700, kept=True, pos_base=60000, theta=1e6, layout="head", seed=8)
    check_tree(nq, 2, 2, 2, 70, 150, pos_base=131072, theta=5e5, kind="tree", shared_mask=True, seed=9)


def test_tree_sharp_flat_and_negative_scores(nq):
    check_tree(nq, 1, 2, 4, 8, 2000, q_scale=8.0, seed=11)
    check_tree(nq, 1, 2, 4, 8, 2000, scale=0.0, seed=12)
    check_tree(nq, 1, 2, 4, 8, 2000, scale=-0.2, q_scale=4.0, seed=13)
    check_tree(nq, 1, 2, 4, 8, 500, q_scale=2.0 ** -60, scale=2.0 ** 57, seed=14)
    check_tree(nq, 1, 2, 4, 8, 500, q_scale=2.0 ** 60, scale=2.0 ** -63, seed=15)


@pytest.mark.parametrize("nodes,G,n,page,ragged", [
    (1, 4, 40000, 0, False), (7, 4, 21001, 64, True), (16, 4, 30000, 0, True), (5, 3, 12345, 0, False),
    (32, 4, 17000, 48, False), (24, 8, 26000, 0, True)])
def test_tree_many_tiles_per_cta(nq, nodes, G, n, page, ragged):
    """Long caches: many tiles pass through each CTA's pipeline (the barriers'
    phases wrap many times).  Against the simple arithmetic in fp64 for one
    head, repeated calls equal bit for bit, no wait run out."""
    units = 3 if ragged else 2
    lens = [n, n // 3, n - 129] if ragged else None
    check_tree(nq, units, 1, G, nodes, n, P=page, lens=lens, seed=n)
    ks, vs = fill_store(nq, 40, 8, 1500, 3, 1), fill_store(nq, 40, 8, 1500, 2, 2)
    tab = nq.rope_tables(1e4, 1500)
    g = gen(n)
    q = torch.randn(40, 8 * G, nodes, D, generator=g, device="cuda").to(torch.bfloat16)
    Kn = torch.randn(40, 8, nodes, D, generator=g, device="cuda").to(torch.bfloat16)
    first = nq.nq_tree_attend(q, Kn, Kn, ks, vs, 1500, tab, 1500)
    for _ in range(20):
        assert torch.equal(nq.nq_tree_attend(q, Kn, Kn, ks, vs, 1500, tab, 1500), first)
    assert nq.device_error() == 0


def test_tree_value_and_key_scales(nq):
    """fp16 scales far from one (values are averaged in scaled codes)."""
    check_tree(nq, 1, 2, 4, 8, 400, sigma_v=1000.0, seed=16)
    check_tree(nq, 1, 2, 4, 8, 400, sigma_v=2.0 ** -9, seed=17)
    check_tree(nq, 1, 2, 4, 8, 400, sigma_k=100.0, scale=1e-3, seed=18)
    check_tree(nq, 1, 2, 4, 8, 400, sigma_k=1e-3, scale=50.0, seed=19)


def test_tree_growing_maximum(nq):
    """Scores that grow along the cache: the running maximum moves at every tile."""
    units, heads, n = 1, 2, 1500
    g = gen(1)
    q = torch.randn(units, heads, 3, D, generator=g, device="cuda")
    tab = nq.rope_tables(1e4, n)
    # keys along the query at position-dependent strength (rotated to their positions)
    amp = torch.linspace(-30, 30, n, device="cuda")[None, None, :, None]
    x = q[:, :, :1] / q[:, :, :1].norm(dim=-1, keepdim=True) * amp + \
        0.5 * torch.randn(units, heads, n, D, generator=g, device="cuda")
    ks, vs = nq.PackedStore.empty(units, heads, n, 3), fill_store(nq, units, heads, n, 2, 2)
    nq.nq_encode(x.to(torch.bfloat16), None, ks, None, n, tab, n)
    q = q.to(torch.bfloat16)
    Kn, Vn = (torch.randn(units, heads, 3, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    for scale in (0.1, 1.0, -1.0):
        out, lse = nq.nq_tree_attend(q, Kn, Vn, ks, vs, n, tab, n, scale=scale, lse=True)
        ref, rl, ob, lb = ref_tree(q, Kn, Vn, ks, vs, [n], None, 0, None, 0, 1e4, None, scale)
        assert (np.abs(out.double().cpu().numpy() - ref) <= ob).all()
        assert (np.abs(lse.double().cpu().numpy() - rl) <= lb).all()


def test_tree_rows_are_independent(nq):
    """A row of huge queries changes nothing in its neighbours, and the draft
    nodes that a row does not see may hold anything, NaN included."""
    g = gen(21)
    ks, vs = fill_store(nq, 1, 1, 333, 3, 1), fill_store(nq, 1, 1, 333, 2, 2)
    tab = nq.rope_tables(1e4, 333)
    q, Kn, Vn = (torch.randn(1, 1, 6, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    base = nq.nq_tree_attend(q, Kn, Vn, ks, vs, 333, tab, 333)
    big = q.clone()
    big[:, :, 5] *= 2.0 ** 40
    got = nq.nq_tree_attend(big, Kn, Vn, ks, vs, 333, tab, 333)
    assert torch.equal(got[:, :, :5], base[:, :, :5]) and torch.isfinite(got).all()
    Kn[:, :, 5], Vn[:, :, 5] = float("nan"), float("inf")
    got = nq.nq_tree_attend(q, Kn, Vn, ks, vs, 333, tab, 333)
    assert torch.equal(got[:, :, :5], base[:, :, :5])


def test_tree_agrees_with_single_token_attention(nq):
    """One node that sees nothing of the draft: nq_attend's own answer."""
    n, H, G = 900, 4, 4
    ks, vs = fill_store(nq, 2, H, n, 3, 1), fill_store(nq, 2, H, n, 2, 2)
    tab = nq.rope_tables(1e6, n)
    q = torch.randn(2, H * G, 1, D, generator=gen(3), device="cuda").to(torch.bfloat16)
    Kn = torch.zeros(2, H, 1, D, dtype=torch.bfloat16, device="cuda")
    blind = torch.zeros(2, 1, 1, dtype=torch.int64, device="cuda")
    out, lse = nq.nq_tree_attend(q, Kn, Kn, ks, vs, n, tab, n, mask=blind, lse=True)
    o1, l1 = nq.nq_attend(q[:, :, 0].float().contiguous(), ks, vs, n, G, tab, n)
    assert (out[:, :, 0].float() - o1).norm() <= 4e-3 * o1.norm()
    assert (lse[:, :, 0] - l1).abs().max() < 5e-3


def test_tree_strided_stores_and_long_offsets(nq):
    """Units of a larger store (gaps between them), and a store whose last unit
    lies past 2^31 code words."""
    g = gen(31)
    big_k, big_v = fill_store(nq, 6, 2, 300, 3, 1), fill_store(nq, 6, 2, 300, 2, 2)
    tab = nq.rope_tables(1e4, 300)
    q, Kn, Vn = (torch.randn(3, 2, 4, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    part = nq.nq_tree_attend(q, Kn, Vn, big_k.select_units(slice(0, 6, 2)),
                             big_v.select_units(slice(0, 6, 2)), 190, tab, 300)
    for i in range(3):
        one = nq.nq_tree_attend(q[i:i + 1], Kn[i:i + 1], Vn[i:i + 1],
                                big_k.select_units(slice(2 * i, 2 * i + 1)),
                                big_v.select_units(slice(2 * i, 2 * i + 1)), 190, tab, 300)
        assert (one.float() - part[i:i + 1].float()).norm() <= 4e-3 * one.float().norm()
    far = (2 ** 31 + 2 ** 22) // 12
    kc = torch.zeros(far * 12, dtype=torch.int32, device="cuda")
    km = torch.zeros(far, dtype=torch.int32, device="cuda")
    vc, vm = kc.view(-1)[:far * 8], torch.zeros(far, dtype=torch.int32, device="cuda")
    P = 64
    pages = far // P
    ks = nq.PackedStore(kc[:pages * P * 12].view(pages, 1, P, 12), km[:pages * P].view(pages, 1, P), 3)
    vcod = torch.zeros(pages, 1, P, 8, dtype=torch.int32, device="cuda")
    vs = nq.PackedStore(vcod, vm[:pages * P].view(pages, 1, P), 2)
    src_k, src_v = fill_store(nq, 1, 1, 2 * P, 3, 5), fill_store(nq, 1, 1, 2 * P, 2, 6)
    ids = [pages - 1, 7]
    for a, b in ((ks.codes, src_k.codes), (ks.meta, src_k.meta), (vs.codes, src_v.codes), (vs.meta, src_v.meta)):
        for x, p in enumerate(ids):
            a[p, 0] = b[0, 0, x * P:(x + 1) * P]
    got = nq.nq_tree_attend(q[:1, :1], Kn[:1, :1], Vn[:1, :1], ks, vs, 2 * P, tab, 300, table=i32([ids]))
    want = nq.nq_tree_attend(q[:1, :1], Kn[:1, :1], Vn[:1, :1], src_k, src_v, 2 * P, tab, 300)
    assert torch.equal(got, want)


def test_tree_other_stream_graph_and_repeat(nq):
    """The same bits from a side stream, from two graphs replayed in turn on one
    workspace, and again: no atomics, no state between calls."""
    g = gen(41)
    U, H, G, M, n = 2, 4, 4, 12, 1700
    ks, vs = fill_store(nq, U, H, n, 3, 1), fill_store(nq, U, H, n, 2, 2)
    tab = nq.rope_tables(1e4, n)
    q = torch.randn(U, H * G, M, D, generator=g, device="cuda").to(torch.bfloat16)
    Kn, Vn = (torch.randn(U, H, M, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    lens = i32([n, 900])
    call = lambda x, **kw: nq.nq_tree_attend(x, Kn, Vn, ks, vs, n, tab, n, lens=lens, **kw)  # noqa: E731
    q2 = q.flip(2).contiguous()
    a, b = call(q), call(q2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    side = call(q, stream=s)
    s.synchronize()
    assert torch.equal(side, a)
    ws = nq.tree_attend_workspace(U, H, G, M, n, ragged=True)
    outs, graphs = [torch.empty_like(q), torch.empty_like(q)], []
    for x, o in ((q, outs[0]), (q2, outs[1])):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call(x, out=o, ws=ws)
        graphs.append(gr)
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], a) and torch.equal(outs[1], b)
    lens.copy_(i32([5, n]))  # a captured call reads the lengths of its replay
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], call(q))


def test_binding_refuses_wrong_shapes(nq):
    ks, vs = nq.PackedStore.empty(2, 4, 64, 3), nq.PackedStore.empty(2, 4, 64, 2)
    tab = nq.rope_tables(1e4, 64)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, K = z(2, 8, 5, D), z(2, 4, 5, D)
    bad = [dict(q=z(2, 9, 5, D)), dict(K=z(2, 4, 6, D)), dict(q=q.float()), dict(n=65),
           dict(mask=torch.zeros(2, 5, 2, dtype=torch.int64, device="cuda")),
           dict(mask=torch.zeros(2, 5, 1, dtype=torch.int32, device="cuda")),
           dict(lens=i32([1, 2, 3])), dict(table=i32([[0, 1]])), dict(table=i32([[0], [1]]), n=65),
           dict(positions=torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
           dict(out=z(2, 8, 4, D)), dict(v=nq.PackedStore.empty(2, 4, 32, 2))]
    for kw in bad:
        a = dict(q=q, K=K, v=vs, n=60)
        a.update(kw)
        with pytest.raises(ValueError):
            nq.nq_tree_attend(a["q"], a["K"], a["K"], ks, a["v"], a["n"], tab, 64,
                              mask=a.get("mask"), lens=a.get("lens"), table=a.get("table"),
                              positions=a.get("positions"), out=a.get("out"))
    with pytest.raises(ValueError):
        nq.nq_encode_slots(z(4, 3, D), z(4, 3, D), ks, vs, i32([1, 2]), i32([1, 2, 3]), tab, 64)
    with pytest.raises(ValueError):
        nq.nq_qk_norm_rope(q, K.float(), tab, 64)
    with pytest.raises(ValueError):
        nq.nq_qk_norm_rope(q, K, tab, 64, q_weight=torch.ones(64, device="cuda"))
    with pytest.raises(ValueError):
        nq.nq_page_tables(i32([1]), i32([1, 2]), 16, i32([0]), i32([[0]]), 4)


def test_binding_refuses_short_tables_and_other_types(nq):
    """A table of angles for fewer positions than the call names would be read
    past its end; an output type that the library does not write."""
    ks, vs = nq.PackedStore.empty(2, 4, 512, 3), nq.PackedStore.empty(2, 4, 512, 2)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, K = z(2, 8, 5, D), z(2, 4, 5, D)
    good = nq.rope_tables(1e4, 512)
    for tab, most in ((good[:-1], 512), (good, 513), (good.double(), 512), (good.half(), 512)):
        with pytest.raises(ValueError):
            nq.nq_qk_norm_rope(q, K, tab, most)
        with pytest.raises(ValueError):
            nq.nq_encode_slots(K[0], K[0], ks, vs, i32([0] * 5), i32([1] * 5), tab, most)
        with pytest.raises(ValueError):
            nq.nq_tree_attend(q, K, K, ks, vs, 500, tab, most)
    for kw in (dict(q_dtype=torch.float16), dict(k_dtype=torch.float64)):
        with pytest.raises(ValueError):
            nq.nq_qk_norm_rope(q, K, good, 512, **kw)


def test_paged_store_rounds_up_to_whole_pages(nq):
    """Every token that gets a slot is attended: a request of 23 tokens in pages
    of 16, asked for with max_tokens = 20, has room for 32."""
    store = nq.PagedStore(2, 1, 1, 5, 16, 20, 1e4)
    assert store.n == 32
    plan = store.plan(i32([23, 33]), 60)
    assert plan.used.tolist() == [4, 2]  # the second request's 33rd token has no page
    g = gen(77)
    x = torch.randn(2, 1, 60, D, generator=g, device="cuda").to(torch.bfloat16)
    store.write(0, x[0], x[1], plan.slots, plan.positions)
    store.commit(plan)
    q = torch.randn(2, 1, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    mask = torch.zeros(1, 1, dtype=torch.int64, device="cuda")  # the draft is not seen
    _, lse = store.attend(0, torch.zeros_like(q), q, q, mask, lse=True)
    # a query of zeros: log(tokens), computed as (log2(2^4 tokens) - 4) ln 2.  The
    # logarithm (8.5 and 9, 1 ulp = 2^-20), the difference and the product (half
    # an ulp, 2^-23 each) and ln 2 (2^-25 relative): below 2^-20, and as much
    # again for the expected value's own rounding
    want = torch.tensor([23.0, 32.0], dtype=torch.float64).log()
    assert torch.allclose(lse.flatten().cpu().double(), want, rtol=0, atol=2.0 ** -19)


# ----------------------------------------------------------- the run of them
@pytest.mark.parametrize("captured", [False, True])
def test_speculative_steps_over_a_paged_store(nq, captured):
    """Prompts, then three draft-and-verify steps of a batch: norm + RoPE, tree
    attention, page plan, write of the accepted nodes, new lengths, with the
    batch's lengths on the device only.  After each step the store holds, at
    every token, the bits that nq_encode gives for that token, and the tree's
    attention matches fp64 over them."""
    S, layers, H, G, M, P, cap = 5, 2, 4, 2, 7, 16, 160
    g, rng = gen(51), np.random.default_rng(51)
    store = nq.PagedStore(S, layers, H, 70, P, cap, 1e4)
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    history = [[] for _ in range(S)]  # accepted (rotated K, V) rows per request and layer
    prompt = [37, 0, 16, 64, 5]
    total = sum(prompt)
    plan = store.plan(i32(prompt), total + 3)
    for layer in range(layers):
        x = torch.randn(1, total + 3, 2 * H, D, generator=g, device="cuda").to(torch.bfloat16).permute(0, 2, 1, 3)
        _, K = nq.nq_qk_norm_rope(None, x[:, :H], store.rope, cap, positions=plan.positions[None], k_weight=w)
        store.write(layer, K[0], x[0, H:], plan.slots, plan.positions)
        at = 0
        for s in range(S):
            history[s].append([K[0, :, at:at + prompt[s]].clone(), x[0, H:, at:at + prompt[s]].clone()])
            at += prompt[s]
    store.commit(plan)
    lens = list(prompt)
    # static buffers of the step, as a captured server keeps them
    x = torch.zeros(layers, S, M, (G + 2) * H, D, dtype=torch.bfloat16, device="cuda")
    mask = torch.zeros(S, M, 1, dtype=torch.int64, device="cuda")
    depth = torch.zeros(S, M, dtype=torch.int32, device="cuda")
    outs = torch.empty(layers, S, M, G * H, D, dtype=torch.bfloat16, device="cuda")
    rot = torch.empty(layers, 2, S, M, H, D, dtype=torch.bfloat16, device="cuda")

    def forward():
        pos = (store.lens[:, None] + depth).to(torch.int32)
        for layer in range(layers):
            row = x[layer].permute(0, 2, 1, 3)
            q, K = nq.nq_qk_norm_rope(row[:, :G * H], row[:, G * H:(G + 1) * H], store.rope, cap,
                                      positions=pos, q_weight=w, k_weight=w)
            V = row[:, (G + 1) * H:]
            rot[layer, 0].copy_(K.permute(0, 2, 1, 3))
            rot[layer, 1].copy_(V.permute(0, 2, 1, 3))
            store.attend(layer, q, K, V, mask, out=outs[layer].permute(0, 2, 1, 3))
            qs[layer].copy_(q)

    qs = torch.empty(layers, S, G * H, M, D, dtype=torch.bfloat16, device="cuda")
    graph = None
    for step in range(3):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        mask.copy_(tree_mask(S, M, "tree", step))
        see = see_of(mask, S, M)
        depth.copy_(torch.from_numpy(see.sum(-1).astype(np.int32) - 1))
        if captured and graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                forward()
        if captured:
            graph.replay()
        else:
            forward()
        torch.cuda.synchronize()
        for layer in range(layers):
            ks, vs = store.layer(layer)
            K, V = (rot[layer, i].permute(0, 2, 1, 3) for i in range(2))
            ref, _, ob, _ = ref_tree(qs[layer], K, V, ks, vs, lens, store.table, P, None, 0, 1e4,
                                     mask, D ** -0.5)
            got = outs[layer].permute(0, 2, 1, 3).double().cpu().numpy()
            assert (np.abs(got - ref) <= ob).all()
        # accept a path of each tree: the ancestors of a random node (request 2: nothing)
        paths = [np.flatnonzero(see[s, rng.integers(M)]) if s != 2 else [] for s in range(S)]
        counts = [len(p) for p in paths]
        plan = store.plan(i32(counts), S * M)
        node_slot = np.full((S, M), -1)
        got_slots, starts = plan.slots.cpu().numpy(), plan.starts.cpu().numpy()
        for s in range(S):
            node_slot[s, paths[s]] = got_slots[starts[s]:starts[s] + counts[s]]
        assert plan.used.tolist()[1] == 0
        positions = (store.lens[:, None] + depth).to(torch.int32).reshape(-1)
        for layer in range(layers):
            rows = rot[layer].reshape(2, S * M, H, D).permute(0, 2, 1, 3)
            store.write(layer, rows[0], rows[1], i32(node_slot.reshape(-1)), positions)
            for s in range(S):
                for i in range(2):
                    keep = rot[layer, i, s, torch.as_tensor(np.asarray(paths[s], np.int64), device="cuda")]
                    history[s][layer][i] = torch.cat([history[s][layer][i], keep.permute(1, 0, 2)], 1)
        store.commit(plan)
        lens = [a + b for a, b in zip(lens, counts)]
        assert store.lens.tolist() == lens
        used = store.table[store.table >= 0].tolist()
        assert len(set(used)) == len(used) == int(store.taken)
        # the pages hold what nq_encode gives for each request's own rows
        for s in range(S):
            n = lens[s]
            if n == 0:
                continue
            pg = store.table[s].long()[torch.arange(n, device="cuda") // P]
            off = torch.arange(n, device="cuda") % P
            for layer in range(layers):
                ks, vs = store.layer(layer)
                k1, v1 = nq.PackedStore.empty(1, H, n, 3), nq.PackedStore.empty(1, H, n, 2)
                K, V = history[s][layer]
                nq.nq_encode(K[None].contiguous(), V[None].contiguous(), k1, v1, n, store.rope, cap)
                for a, b in ((ks, k1), (vs, v1)):
                    assert torch.equal(a.codes[pg, :, off].transpose(0, 1), b.codes[0])
                    assert torch.equal(a.meta[pg, :, off].transpose(0, 1), b.meta[0])
    assert nq.device_error() == 0


def test_calls_refuse_longer_angle_tables(nq):
    """A store's table covers its rounded-up length: named with a smaller one
    it is refused by every call, not read at the wrong rows."""
    store = nq.PagedStore(1, 1, 4, 3, 100, 250, 1e4)
    assert store.n == 300
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, K = z(1, 8, 5, D), z(1, 4, 5, D)
    for most in (250, 256):
        with pytest.raises(ValueError):
            nq.nq_qk_norm_rope(q, K, store.rope, most)
        with pytest.raises(ValueError):
            nq.nq_encode_slots(K[0], K[0], *store.layer(0), i32([0] * 5), i32([1] * 5), store.rope, most)
        with pytest.raises(ValueError):
            nq.nq_tree_attend(q, K, K, *store.layer(0), 250, store.rope, most, table=store.table)
    nq.nq_qk_norm_rope(q, K, store.rope, 300)


def test_calls_refuse_strided_slots(nq):
    """Every other slot of a store, which the kernels would read (and write) as
    neighbours."""
    ks, vs = nq.PackedStore.empty(2, 4, 64, 3), nq.PackedStore.empty(2, 4, 64, 2)
    thin = lambda s: nq.PackedStore(s.codes[:, :, ::2], s.meta[:, :, ::2], s.bits)  # noqa: E731
    tab = nq.rope_tables(1e4, 64)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, K = z(2, 8, 5, D), z(2, 4, 5, D)
    for k, v in ((thin(ks), thin(vs)), (thin(ks), nq.PackedStore.empty(2, 4, 32, 2))):
        with pytest.raises(ValueError):
            nq.nq_tree_attend(q, K, K, k, v, 20, tab, 64)
        with pytest.raises(ValueError):
            nq.nq_encode_slots(K[0], K[0], k, v, i32([0] * 5), i32([1] * 5), tab, 64)


def test_paged_store_on_a_side_stream(nq):
    """A whole step on a stream that is never made current and that is busy with
    other work at its start: each call waits for the one before it."""
    S, H, G, P = 4, 2, 2, 16
    counts = ([20, 0, 33, 5], [3, 7, 0, 12])

    def steps(stream):
        g = gen(91)
        store = nq.PagedStore(S, 1, H, 12, P, 64, 1e4)
        outs = []
        for c in counts:
            x = torch.randn(2, H, sum(c) + 2, D, generator=g, device="cuda").to(torch.bfloat16)
            q = torch.randn(S, H * G, 3, D, generator=g, device="cuda").to(torch.bfloat16)
            K, V = (torch.randn(S, H, 3, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
            n = i32(c)
            a = torch.ones(4096, 4096, dtype=torch.bfloat16, device="cuda")
            torch.cuda.synchronize()
            if stream is not None:
                with torch.cuda.stream(stream):
                    for _ in range(40):
                        torch.mm(a, a)
            plan = store.plan(n, sum(c) + 2, stream=stream)
            store.write(0, x[0], x[1], plan.slots, plan.positions, stream=stream)
            store.commit(plan, stream=stream)
            outs.append(store.attend(0, q, K, V, stream=stream))
            (torch.cuda.current_stream() if stream is None else stream).synchronize()
            assert store.lens.tolist() == [sum(z) for z in zip(*counts[:len(outs)])]
        return outs + [store.table, store.lens, store.taken]

    want = steps(None)
    got = steps(torch.cuda.Stream())
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert nq.device_error() == 0


@pytest.mark.parametrize("captured", [False, True])
def test_paged_store_serves_on_as_requests_end(nq, captured):
    """Requests come and go for many steps over a pool that holds a few of them:
    with their pages released nothing runs out, no page is in two rows, and each
    request's attention is that over its own tokens alone (a store of its own, the
    same kernel: two outputs rounded to bf16 differ by a step at most, 2^-7
    relative; two sets of weights rounded to f16 by 2^-10 of sum p |v|, which is
    below 8 norms of sum p v for 66 keys of independent values, 2^-7 again; a
    wrong page is off by about the norm itself).  Captured: plan, write, commit, attention and release of a
    step are one graph, replayed with other counts and endings."""
    S, H, G, P, pages, rows, T = 3, 2, 2, 16, 14, 96, 64
    g, rng = gen(93), np.random.default_rng(93)
    store = nq.PagedStore(S, 1, H, pages, P, T, 1e4)
    counts, done = i32([0] * S), torch.zeros(S, dtype=torch.bool, device="cuda")
    x = torch.zeros(2, H, rows, D, dtype=torch.bfloat16, device="cuda")
    q = torch.randn(S, H * G, 2, D, generator=g, device="cuda").to(torch.bfloat16)
    K, V = (torch.randn(S, H, 2, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    out, used = torch.zeros_like(q), i32([0, 0])

    def step():
        plan = store.plan(counts, rows)
        store.write(0, x[0], x[1], plan.slots, plan.positions)
        store.commit(plan)
        used.copy_(plan.used)
        store.attend(0, q, K, V, out=out)
        store.release(done)

    graph = None
    if captured:
        step()  # (nothing to do: counts and endings are 0)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    tokens = [[torch.zeros(H, 0, D, dtype=torch.bfloat16, device="cuda")] * 2 for _ in range(S)]
    total = 0
    for it in range(12):
        c = [int(rng.integers(0, min(32, T - t[0].shape[1]) + 1)) for t in tokens]
        end = rng.random(S) < 0.4
        total += sum(-(-n // P) for n in c)
        counts.copy_(i32(c))
        done.copy_(torch.from_numpy(end))
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        if captured:
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert used.tolist()[1] == 0
        at = 0
        for s in range(S):
            for i in range(2):
                tokens[s][i] = torch.cat([tokens[s][i], x[i, :, at:at + c[s]]], 1)
            at += c[s]
            n = tokens[s][0].shape[1]
            ks, vs = nq.PackedStore.empty(1, H, max(n, 1), 3), nq.PackedStore.empty(1, H, max(n, 1), 2)
            if n:
                nq.nq_encode(tokens[s][0][None], tokens[s][1][None], ks, vs, n, store.rope, store.n)
            one = nq.nq_tree_attend(q[s:s + 1], K[s:s + 1], V[s:s + 1], ks, vs, n, store.rope, store.n)
            assert (out[s:s + 1].float() - one.float()).norm() <= 2.0 ** -6 * one.float().norm()
            if end[s]:
                tokens[s] = [t[:, :0] for t in tokens[s]]
        assert store.lens.tolist() == [t[0].shape[1] for t in tokens]
        held = [p for s, row in enumerate(store.table.tolist()) for p in row[:-(-tokens[s][0].shape[1] // P)]]
        rest = store.free[int(store.taken):].tolist()
        assert sorted(held + rest) == list(range(pages))
    assert total > 2 * pages and nq.device_error() == 0
    with pytest.raises(ValueError):
        store.release(done.int())
    with pytest.raises(ValueError):
        store.release(done[:2])
    with pytest.raises(ValueError):
        store.release(done.cpu())


def test_page_tables_lengths_past_31_bits(nq):
    """A request whose new tokens pass 2^31 - 1: lengths and positions saturate,
    slots and pages go on."""
    P, last = 65536, 2 ** 31 - 1
    table = torch.full((1, 32769), 7, dtype=torch.int32, device="cuda")
    table[0, 32768] = -1
    r = nq.nq_page_tables(i32([last - 2]), i32([5]), P, i32([3, 4]), table, 6)
    assert r.lens.tolist() == [last] and r.starts.tolist() == [0, 5] and r.used.tolist() == [1, 0]
    assert r.positions.tolist() == [last - 2, last - 1, last, last, last, 0]
    assert r.slots.tolist() == [8 * P - 3, 8 * P - 2, 8 * P - 1, 3 * P, 3 * P + 1, -1]
    assert table[0, 32767:].tolist() == [7, 3]


@pytest.mark.parametrize("size", [2.0 ** 60, 2.0 ** -60, 1.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_rope_large_and_small_rows(nq, size, dtype):
    """At the ends of the range that the sum of squares has: 128 * 2^120 and
    128 * 2^-120 are still normal in fp32."""
    x = torch.rand(1, 3, 40, D, generator=gen(6), device="cuda") * 2 - 1
    x[..., 5] = 1.0  # (the largest of a row)
    x = (x * size).to(dtype)
    tab, pos = nq.rope_tables(1e4, 40), torch.arange(40, device="cuda")[None]
    q, _ = nq.nq_qk_norm_rope(x, None, tab, 40, eps=0.0)
    ref, y = ref_norm(x, None, 0.0, pos, 1e4)
    assert (q.double() - ref).abs().le(norm_bound(ref, y, dtype)).all()


def test_encode_and_norm_at_offsets_past_32_bits(nq):
    """Rows written to the last pages of a store of more than 2^31 code words, and
    heads normed in place in a buffer of more than 2^31 elements."""
    g = gen(97)
    H, P = 8, 64
    pages = (2 ** 31 + 2 ** 23) // (H * P * 12)
    ks, vs = nq.PackedStore.empty(pages, H, P, 3), nq.PackedStore.empty(pages, H, P, 2)
    K, V = (torch.randn(H, 5, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    tab = nq.rope_tables(1e4, 5)
    slot = [pages * P - 1, pages * P - 64, 0, pages * P - 130, pages * P]
    nq.nq_encode_slots(K, V, ks, vs, i32(slot), i32(range(5)), tab, 5)
    k1, v1 = nq.PackedStore.empty(1, H, 5, 3), nq.PackedStore.empty(1, H, 5, 2)
    nq.nq_encode(K[None], V[None], k1, v1, 5, tab, 5)
    for r in range(4):
        for a, b in ((ks, k1), (vs, v1)):
            assert torch.equal(a.codes[slot[r] // P, :, slot[r] % P], b.codes[0, :, r])
            assert torch.equal(a.meta[slot[r] // P, :, slot[r] % P], b.meta[0, :, r])
    del ks, vs
    far = 2 ** 31 + 2 ** 20
    buf = torch.zeros(far + 4096, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, 3, 5, D), (far, 5 * D, D, 1))
    x.copy_(torch.randn(2, 3, 5, D, generator=g, device="cuda"))
    want, _ = nq.nq_qk_norm_rope(x.contiguous(), None, tab, 5)
    nq.nq_qk_norm_rope(x, None, tab, 5, q_out=x)
    assert torch.equal(x, want)


def test_calls_under_way_on_two_streams(nq):
    """Two steps at once, each on its own stream with its own workspace: neither
    changes the other's bits."""
    g = gen(98)
    U, H, G, M, n = 6, 8, 4, 12, 3000
    ks, vs = fill_store(nq, U, H, n, 3, 1), fill_store(nq, U, H, n, 2, 2)
    tab = nq.rope_tables(1e4, n)
    pos = torch.arange(M, dtype=torch.int32, device="cuda").expand(U, M).contiguous()
    x = [torch.randn(U, M, (G + 2) * H, D, generator=g, device="cuda").to(torch.bfloat16).permute(0, 2, 1, 3)
         for _ in range(2)]
    lens = [i32([n, 5, 1700, 0, 128, 2999]), None]

    def step(i, stream):
        q, k = nq.nq_qk_norm_rope(x[i][:, :G * H], x[i][:, G * H:(G + 1) * H], tab, n, positions=pos, stream=stream)
        return nq.nq_tree_attend(q, k, x[i][:, (G + 1) * H:], ks, vs, n, tab, n, lens=lens[i], stream=stream)

    want = [step(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(15):
        for i in range(2):
            got[i].append(step(i, streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])
    assert nq.device_error() == 0
