"""Argument checks of the serving calls (page tables, norms with RoPE, encode
into slots, tree attention), on the CPU: every refused call returns its status
before anything is launched (the pointers are never dereferenced), empty work
is accepted without a device, and host tensors are refused by the binding."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def nq():
    from e8_lattice_vector_nq_b200 import build, nq as nqmod

    build.build()
    return nqmod


def ptr(x):
    return ctypes.c_void_p(x)


A, B, C, E, F, G, H = (0x10000000 * i for i in range(1, 8))  # far apart, 16-byte aligned


def pages(nq, **kw):
    a = dict(lens=A, counts=B, requests=4, page=16, free=C, n_free=100, taken=None, table=E,
             stride=8, lens_out=F, starts=G, slots=H, positions=H + 0x1000000, rows=64,
             used=H + 0x2000000)
    a.update(kw)
    p = lambda k: None if a[k] is None else ptr(a[k])  # noqa: E731
    return nq.lib().nq_page_tables(p("lens"), p("counts"), a["requests"], a["page"], p("free"),
                                   a["n_free"], p("taken"), p("table"), a["stride"],
                                   p("lens_out"), p("starts"), p("slots"), p("positions"),
                                   a["rows"], p("used"), None)


@pytest.mark.parametrize("kw,status", [
    (dict(requests=-1), 1), (dict(page=0), 1), (dict(stride=0), 1), (dict(n_free=-1), 1),
    (dict(rows=-1), 1), (dict(requests=8193), 4), (dict(page=65537), 4), (dict(rows=1 << 31), 4),
    (dict(stride=(1 << 24) + 1), 4), (dict(lens=None), 1), (dict(table=None), 1),
    (dict(starts=None), 1), (dict(used=None), 1), (dict(free=None), 1), (dict(slots=None), 1),
    (dict(slots=H + 2), 1), (dict(taken=C + 1), 1),
    # in-place lengths, slots over the free list, a cursor inside used, tables over lens
    (dict(lens_out=A), 1), (dict(slots=C + 16), 1), (dict(taken=H + 0x2000000), 1),
    (dict(table=A - 64), 1), (dict(positions=H + 128), 1),
])
def test_page_tables_refusals(nq, kw, status):
    assert pages(nq, **kw) == status, nq.lib().nq_last_error()


def norm(nq, **kw):
    S = nq.KVStrides
    a = dict(q=A, qs=S(0, 128, 4096), qh=32, k=B, ks=S(0, 128, 1024), kh=8, t=0, units=1, rows=4,
             wq=None, wk=None, eps=1e-6, pos=None, pstride=0, base=0, tab=C, maxp=64, qo=E,
             qos=S(0, 128, 4096), qt=0, ko=F, kos=S(0, 128, 1024), kt=0)
    a.update(kw)
    p = lambda k: None if a[k] is None else ptr(a[k])  # noqa: E731
    return nq.lib().nq_qk_norm_rope(p("q"), a["qs"], a["qh"], p("k"), a["ks"], a["kh"], a["t"],
                                    a["units"], a["rows"], p("wq"), p("wk"), a["eps"], p("pos"),
                                    a["pstride"], a["base"], p("tab"), a["maxp"], p("qo"),
                                    a["qos"], a["qt"], p("ko"), a["kos"], a["kt"], None)


def test_norm_rope_refusals(nq):
    S = nq.KVStrides
    inv, uns = nq.NQ_ERR_INVALID, nq.NQ_ERR_UNSUPPORTED
    assert norm(nq, qh=0, kh=0) == inv
    assert norm(nq, qh=1025) == inv and norm(nq, rows=-1) == inv and norm(nq, base=-1) == inv
    assert norm(nq, eps=-1.0) == inv and norm(nq, eps=float("nan")) == inv
    assert norm(nq, eps=float("inf")) == inv
    assert norm(nq, t=2) == inv and norm(nq, qt=-1) == inv and norm(nq, kt=3) == inv
    assert norm(nq, q=None) == inv and norm(nq, ko=None) == inv and norm(nq, q=A + 8) == inv
    assert norm(nq, qs=S(0, 128, 4100)) == inv and norm(nq, qs=S(0, -128, 4096)) == inv
    # outputs that several rows would write
    assert norm(nq, qos=S(0, 0, 4096)) == inv and norm(nq, qos=S(0, 128, 0)) == inv
    assert norm(nq, units=2) == inv
    # in place only as it is
    assert norm(nq, qo=A, qos=S(0, 512, 128)) == inv and norm(nq, qo=A, qt=1) == inv
    assert norm(nq, wq=C + 4) == inv
    assert norm(nq, tab=None) == inv and norm(nq, base=61) == inv and norm(nq, maxp=0) == inv
    assert norm(nq, units=2, pos=F, pstride=3, qos=S(1 << 20, 128, 4096),
                kos=S(1 << 20, 128, 1024)) == inv
    assert norm(nq, rows=1 << 30, maxp=1 << 31) == uns
    assert norm(nq, units=0) == 0 and norm(nq, rows=0) == 0


def slots(nq, **kw):
    S = nq.KVStrides
    pk = nq.Packed(0x20000, 0x30000, 64, 8, 3)
    a = dict(K=A, ks=S(0, 128, 1024), V=B, vs=S(0, 128, 1024), heads=8, rows=4, slots=C,
             positions=E, page=8, pages=4, tab=F, maxp=64, kout=pk, vout=pk)
    a.update(kw)
    p = lambda k: None if a[k] is None else ptr(a[k])  # noqa: E731
    d = lambda k: None if a[k] is None else ctypes.byref(a[k])  # noqa: E731
    return nq.lib().nq_encode_slots(p("K"), a["ks"], p("V"), a["vs"], a["heads"], a["rows"],
                                    p("slots"), p("positions"), a["page"], a["pages"], p("tab"),
                                    a["maxp"], d("kout"), d("vout"), None)


def test_encode_slots_refusals(nq):
    S = nq.KVStrides
    inv, uns = nq.NQ_ERR_INVALID, nq.NQ_ERR_UNSUPPORTED
    assert slots(nq, K=None, V=None) == inv
    for kw in (dict(heads=0), dict(rows=-1), dict(page=0), dict(pages=-1), dict(slots=None),
               dict(slots=C + 2), dict(positions=None), dict(tab=None), dict(maxp=0),
               dict(kout=None), dict(vout=None, K=None),
               dict(kout=nq.Packed(0x20000, 0x30000, 64, 8, 4)), dict(ks=S(0, 128, 1020)),
               dict(K=A + 2)):
        assert slots(nq, **kw) == inv, kw
    assert slots(nq, rows=1 << 29) == uns and slots(nq, pages=1 << 29) == uns
    assert slots(nq, rows=0) == 0


def tree(nq, **kw):
    S = nq.KVStrides
    pk = nq.Packed(0x20000, 0x30000, 4096, 512, 3)
    a = dict(q=A, qs=S(1 << 16, 128, 4096), K=B, ks=S(1 << 14, 128, 1024), V=C,
             vs=S(1 << 14, 128, 1024), units=2, heads=8, G=4, nodes=5, kin=pk, vin=pk, n=100,
             lens=None, table=None, tstride=0, page=1, pages=0, pos=None, pstride=0, base=0,
             tab=E, maxp=100, mask=None, mstride=0, scale=0.1, out=F, os=S(1 << 16, 128, 4096),
             lse=None, ws=G, wsb=1 << 40)
    a.update(kw)
    p = lambda k: None if a[k] is None else ptr(a[k])  # noqa: E731
    d = lambda k: None if a[k] is None else ctypes.byref(a[k])  # noqa: E731
    return nq.lib().nq_tree_attend(
        p("q"), a["qs"], p("K"), a["ks"], p("V"), a["vs"], a["units"], a["heads"], a["G"],
        a["nodes"], d("kin"), d("vin"), a["n"], p("lens"), p("table"), a["tstride"], a["page"],
        a["pages"], p("pos"), a["pstride"], a["base"], p("tab"), a["maxp"], p("mask"),
        a["mstride"], a["scale"], p("out"), a["os"], p("lse"), p("ws"), a["wsb"], None)


def test_tree_attend_refusals(nq):
    S = nq.KVStrides
    inv, uns = nq.NQ_ERR_INVALID, nq.NQ_ERR_UNSUPPORTED
    for kw in (dict(units=-1), dict(heads=0), dict(G=0), dict(G=9), dict(nodes=0),
               dict(nodes=1025), dict(n=-1), dict(base=-1), dict(scale=float("nan")),
               dict(q=None), dict(K=None), dict(V=None), dict(out=None), dict(q=A + 2),
               dict(qs=S(1 << 16, 128, 4097)), dict(os=S(0, 128, 4096)), dict(os=S(1 << 16, 0, 4096)),
               dict(out=A), dict(out=B), dict(lse=F + 2), dict(lens=F + 1), dict(mask=F + 4),
               dict(mask=F, mstride=4), dict(kin=None), dict(vin=None), dict(tab=None),
               dict(kin=nq.Packed(0x20000, 0x30000, 64, 8, 1)), dict(maxp=99), dict(base=1),
               dict(pos=F, pstride=99), dict(table=F, tstride=6, page=16), dict(table=F, page=0),
               dict(table=F, tstride=7, page=16, pages=-1), dict(table=F + 2, tstride=7, page=16),
               dict(ws=None), dict(ws=G + 8)):
        assert tree(nq, **kw) == inv, kw
    assert tree(nq, wsb=16) == nq.NQ_ERR_WORKSPACE
    assert tree(nq, n=1 << 31, maxp=1 << 32) == uns
    assert tree(nq, units=1 << 20, nodes=1024) == uns
    assert tree(nq, units=0) == 0


def test_tree_workspace_sizes(nq):
    L = nq.lib()
    assert L.nq_tree_attend_workspace_bytes(1, 8, 4, 1, 0, 1, 0) == 0
    assert L.nq_tree_attend_workspace_bytes(0, 8, 4, 1, 100, 1, 0) == 0
    small = L.nq_tree_attend_workspace_bytes(1, 8, 4, 1, 100, 1, 0)
    assert 0 < small < L.nq_tree_attend_workspace_bytes(1, 8, 4, 64, 100, 1, 0)
    assert small <= L.nq_tree_attend_workspace_bytes(1, 8, 4, 1, 100000, 1, 0)


def test_binding_refuses_host_tensors(nq):
    bf = torch.zeros(1, 8, 4, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    st = nq.PackedStore.empty(4, 8, 16, 3, "cpu")
    tab = torch.zeros(16)
    calls = {
        "page_tables": lambda: nq.nq_page_tables(i, i, 16, i, i.view(4, 1), 8),
        "norm_rope": lambda: nq.nq_qk_norm_rope(bf, bf, tab, 64),
        "encode_slots": lambda: nq.nq_encode_slots(bf[0], bf[0], st, st, i, i, tab, 64),
        "tree_attend": lambda: nq.nq_tree_attend(bf, bf, bf, st, st, 16, tab, 64),
    }
    for name, call in calls.items():
        with pytest.raises(ValueError, match="no CPU path"):
            call()


@pytest.mark.parametrize("built,named", [(131072, 1000), (300, 250), (257, 256), (512, 1), (256, 257)])
def test_binding_refuses_angle_tables_of_another_length(nq, built, named):
    """The fine rows follow the coarse ones at row ceil(max_pos / 256), so a
    table of more positions than the call names is read at the wrong rows just
    as a shorter one is read past its end."""
    tab = nq.rope_tables(1e4, built, "cpu")
    nq._rope_table(tab, built)
    with pytest.raises(ValueError, match="table"):
        nq._rope_table(tab, named)


def test_binding_takes_tables_of_the_same_rows(nq):
    """Lengths that round up to the same number of coarse rows share a table."""
    tab = nq.rope_tables(1e4, 300, "cpu")
    assert torch.equal(tab, nq.rope_tables(1e4, 512, "cpu"))
    for named in (257, 300, 512):
        nq._rope_table(tab, named)


def test_binding_refuses_stores_laid_out_otherwise(nq):
    """The kernels take two strides per store and find slots side by side:
    strided slots, codes of other slots than meta's, of another type or of
    another width are refused, views that keep the layout are not."""
    ok = nq.PackedStore.empty(4, 8, 16, 3, "cpu")
    c, m = ok.codes, ok.meta
    for st in (ok, ok.select_units(slice(1, 4, 2)), nq.PackedStore(c[:, 2:5], m[:, 2:5], 3),
               nq.PackedStore(c[:, :, 5:9], m[:, :, 5:9], 3), nq.PackedStore.empty(4, 8, 1, 3, "cpu")):
        d = nq._packed(st)
        assert (d.codes, d.meta) == (st.codes.data_ptr(), st.meta.data_ptr())
        assert (d.unit_stride, d.head_stride, d.bits) == (*st.meta.stride()[:2], 3)
    other = torch.empty(4, 8, 16, 24, dtype=torch.int32)[..., ::2]
    for codes, meta, bits in ((c[:, :, ::2], m[:, :, ::2], 3), (c[:, :, :9], m, 3), (c[:3], m, 3),
                              (c[:, :5], m, 3), (c, m, 2), (c[..., :8], m, 2), (c, m, 4),
                              (c.float(), m, 3), (c, m.float(), 3), (other, m, 3),
                              (c, torch.empty(4, 8, 32, dtype=torch.int32)[:, :, ::2], 3)):
        with pytest.raises(ValueError):
            nq._packed(nq.PackedStore(codes, meta, bits))


@pytest.mark.parametrize("S,P,pages,width", [(1, 1, 3, 4), (5, 16, 40, 9), (7, 3, 11, 6), (64, 64, 300, 12),
                                             (3, 8, 0, 2)])
def test_released_pages_return_to_the_list(nq, S, P, pages, width):
    """Random admissions and endings, a free list that runs out among them: after
    every release a page is either in one row or in the list, never both, and the
    rows of the other requests are as they were.  The planning is done here, as
    nq_page_tables defines it."""
    import random

    rng = random.Random(S * 1000 + pages)
    free = torch.arange(pages + 1, dtype=torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32)
    lens, taken = torch.zeros(S, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ran_out = 0
    for _ in range(60):
        new = [rng.randint(0, min(3 * P, width * P - int(x))) if rng.random() < 0.5 else 0 for x in lens]
        at = int(taken)
        for s, c in enumerate(new):
            for j in range(-(-int(lens[s]) // P), -(-(int(lens[s]) + c) // P)):
                table[s, j] = int(free[at]) if at < pages else -1
                at += 1
        if rng.random() < 0.2:  # the plan is dropped: what it wrote stays in the table
            continue
        ran_out += at > pages
        taken.fill_(at)
        lens += torch.tensor(new, dtype=torch.int32)
        done = torch.tensor([rng.random() < 0.3 for _ in range(S)])
        before, held = table.clone(), lens.clone()
        nq._release_pages(done, table, lens, taken, free, P)
        assert torch.equal(table[~done], before[~done]) and (table[done] == -1).all()
        assert torch.equal(lens, torch.where(done, 0, held))
        rows = [int(table[s, j]) for s in range(S) for j in range(-(-int(lens[s]) // P))]
        rows = [x for x in rows if x >= 0]
        assert int(taken) == len(rows)
        assert sorted(rows + free[int(taken):pages].tolist()) == list(range(pages))
    assert pages > 0 or ran_out


def test_binding_takes_a_store_of_one_slot_with_any_slot_stride(nq):
    ok = nq.PackedStore.empty(4, 8, 2, 3, "cpu")
    one = nq.PackedStore(ok.codes[:, :, ::2], ok.meta[:, :, ::2], 3)
    assert nq._packed(one).meta == ok.meta.data_ptr()
    with pytest.raises(ValueError):
        nq._packed(ok, 0)  # a store of the host beside tensors of a device


def test_binding_takes_stores_of_unsigned_words(nq):
    ok = nq.PackedStore.empty(4, 8, 2, 3, "cpu")
    assert nq._packed(nq.PackedStore(ok.codes.view(torch.uint32), ok.meta.view(torch.uint32), 3)).bits == 3
