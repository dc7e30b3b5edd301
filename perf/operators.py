"""The serving operators over the packed KV cache, as workloads to measure.

One verification step of a server that drafts tokens over an E8-packed cache runs
four operators: page tables for the new tokens, per-head norms of queries and keys
with the rotation, attention of the drafted tree over packed cache and draft, and the
write of the accepted rows into their pages.  ``listed()`` names the cases, ``draw``
gives more of the same ranges, ``run`` computes one pass (in plain torch operations, or
with ``own`` through the library) and ``exact`` evaluates the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

D = 128
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # per-head norms + rotation: one decode step of the 64 sequences of the append
        # workload (q and k are views of one fused projection row)
        dict(name="norm_rope_decode_64seq", op="norm_rope", units=64, rows=1, hq=32, hk=8,
             out="bf16", weights=True, positions="list", max_pos=16640, theta=1e4),
        # queries rounded nowhere (fp32, what the single-token attention takes), odd length,
        # Qwen-shaped heads, norms without weights, kept positions
        dict(name="norm_rope_ragged_f32", op="norm_rope", units=3, rows=1237, hq=28, hk=4,
             out="f32", weights=False, positions="list", max_pos=65536, theta=1e6),
        # the prefill of one Mistral-shaped layer
        dict(name="norm_rope_prefill_32k", op="norm_rope", units=1, rows=32768, hq=32, hk=8,
             out="bf16", weights=True, positions="base", max_pos=32768, theta=1e6),
        # page tables: one token for each of 64 running sequences
        dict(name="pages_decode_64seq", op="page_tables", requests=64, page=64, max_len=16384,
             max_new=1, pad=0),
        # admission of a large ragged batch, requests of zero tokens among them, padded rows
        dict(name="pages_prefill_1k", op="page_tables", requests=1021, page=16, max_len=4096,
             max_new=1500, pad=777),
        # accepted rows of 64 sequences into their pages (the append workload's two-bit codes)
        dict(name="encode_slots_decode", op="encode_slots", rows=64, heads=8, bits_k=2, bits_v=2,
             page=64, max_pos=16640, theta=1e4, skip=0.0),
        # a prefill chunk into pages, some rows padded (no slot)
        dict(name="encode_slots_prefill", op="encode_slots", rows=8191, heads=8, bits_k=3,
             bits_v=2, page=64, max_pos=131072, theta=5e5, skip=0.05),
        # tree attention: the smallest call, a chain of 4 drafted tokens over a short cache
        dict(name="tree_chain4_2k", op="tree_attend", units=1, heads=8, G=4, nodes=4, n=2048,
             bits_k=3, bits_v=2, page=0, ragged=False, kept=False, mask="chain", theta=1e4),
        # Qwen-shaped heads (7 query heads a KV head), evicted positions, odd tree and length
        dict(name="tree19_evicted_qwen", op="tree_attend", units=2, heads=4, G=7, nodes=19,
             n=42727, bits_k=3, bits_v=2, page=0, ragged=False, kept=True, mask="tree", theta=1e6),
        # a served batch: paged, ragged lengths (an empty cache among them), two-bit codes
        dict(name="tree16_paged_batch", op="tree_attend", units=32, heads=8, G=4, nodes=16,
             n=16384, bits_k=2, bits_v=2, page=64, ragged=True, kept=False, mask="tree",
             theta=1e4),
        # single new tokens of a served batch over the evicted Mistral-shaped cache length
        dict(name="tree1_batch_13k", op="tree_attend", units=32, heads=8, G=4, nodes=1, n=13147,
             bits_k=3, bits_v=2, page=0, ragged=False, kept=True, mask="chain", theta=1e6),
        # the largest: 64 drafted tokens over one layer of the 128K-token cache
        dict(name="tree64_128k", op="tree_attend", units=1, heads=8, G=4, nodes=64, n=131072,
             bits_k=3, bits_v=2, page=0, ragged=False, kept=False, mask="tree", theta=5e5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "page_tables", "encode_slots", "tree_attend", "tree_attend"])
    if op == "norm_rope":
        units = rng.randint(1, 64)
        hq, hk = rng.choice([(32, 8), (28, 4), (8, 8), (12, 3), (5, 1)])
        rows = _log_int(rng, 1, 32768 // units)
        return dict(op=op, units=units, rows=rows, hq=hq, hk=hk, out=rng.choice(["bf16", "f32"]),
                    weights=rng.random() < 0.7, positions=rng.choice(["base", "list"]),
                    max_pos=max(rows, _log_int(rng, 64, 131072)),
                    theta=rng.choice([1e4, 5e5, 1e6]))
    if op == "page_tables":
        return dict(op=op, requests=_log_int(rng, 1, 4096), page=rng.choice([1, 7, 16, 64, 100, 256]),
                    max_len=_log_int(rng, 1, 16384), max_new=_log_int(rng, 1, 400),
                    pad=rng.choice([0, 1, 513]))
    if op == "encode_slots":
        return dict(op=op, rows=_log_int(rng, 1, 8192), heads=rng.choice([1, 3, 4, 5, 8]),
                    bits_k=rng.choice([2, 3]), bits_v=rng.choice([2, 3]),
                    page=rng.choice([1, 16, 37, 64, 256]), max_pos=_log_int(rng, 300, 131072),
                    theta=rng.choice([1e4, 5e5, 1e6]), skip=rng.choice([0.0, 0.1, 0.5]))
    units = _log_int(rng, 1, 32)
    heads = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 7, 8])
    nodes = _log_int(rng, 1, 128)
    # no more scores than the largest listed case has
    most = min(131072, 64 * 4 * 8 * 131072 // (units * heads * G * nodes), 32 * 8 * 16384 // (units * heads))
    page = rng.choice([0, 0, 16, 48, 64, 100])
    return dict(op=op, units=units, heads=heads, G=G, nodes=nodes, n=_log_int(rng, 1, max(2, most)),
                bits_k=rng.choice([2, 3]), bits_v=rng.choice([2, 3]), page=page,
                ragged=rng.random() < 0.5, kept=page == 0 and rng.random() < 0.4,
                mask=rng.choice(["chain", "tree", "sparse"]), theta=rng.choice([1e4, 5e5, 1e6]))


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _tables(theta, max_pos):
    """The two-level fp32 cos/sin tables: rows of angles 256a*w_i, then of b*w_i (b < 256)."""
    na = (max_pos + 255) // 256
    w = theta ** (-np.arange(64, dtype=np.float64) / 64.0)
    p = np.concatenate([256.0 * np.arange(na), np.arange(256.0)])
    ang = p[:, None] * w[None, :]
    t = np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)
    return torch.from_numpy(t.reshape(-1)).to(DEV)


def _pack(j, bits):
    """Codes [..., 128] (int64) -> uint32 words in int32 [..., 4 * bits], code c at bit bits*c."""
    b = (j[..., None] >> torch.arange(bits, device=j.device)) & 1
    b = b.reshape(j.shape[:-1] + (4 * bits, 32))
    words = (b << torch.arange(32, device=j.device)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _store(g, lead, heads, cap, bits):
    """A filled packed store: codes as the codec leaves them (a normal coordinate whose largest
    of 128 reaches the end of the code range), a coset bit per group, fp16 scales."""
    codes = torch.empty(lead, heads, cap, 4 * bits, dtype=torch.int32, device=DEV)
    meta = torch.empty(lead, heads, cap, dtype=torch.int32, device=DEV)
    amax = (2 ** bits - 1) / 2
    step = max(1, (1 << 18) // max(1, cap))
    flat_c, flat_m = codes.view(lead * heads, cap, -1), meta.view(lead * heads, cap)
    for a in range(0, lead * heads, step):
        b = min(lead * heads, a + step)
        y = torch.randn(b - a, cap, D, generator=g, device=DEV) * (amax / 2.6)
        half = torch.randint(0, 2, (b - a, cap, 16), generator=g, device=DEV)
        hh = half.repeat_interleave(8, -1)
        lim = torch.where(hh > 0, 2 ** bits - 1, 2 ** bits - 2)
        j = torch.where(hh > 0, torch.floor(y) + 2 ** (bits - 1), torch.round(y) + 2 ** (bits - 1) - 1)
        j = torch.minimum(j.long().clamp_(min=0), lim)
        flat_c[a:b] = _pack(j, bits)
        sig = torch.exp(0.25 * torch.randn(b - a, cap, generator=g, device=DEV)) * (2.6 / amax)
        sbits = sig.to(torch.float16).view(torch.int16).long() & 0xFFFF
        mask = (half << torch.arange(16, device=DEV)).sum(-1)
        m = mask | (sbits << 16)
        flat_m[a:b] = torch.where(m >= 1 << 31, m - (1 << 32), m).to(torch.int32)
    return codes, meta


def _tree_mask(case, g, rng):
    """Ancestors and self of each node as 64-bit words [units][nodes][words]; None for a chain.
    "sparse" takes random sets of nodes instead, empty ones among them."""
    if case["mask"] == "chain":
        return None
    U, M = case["units"], case["nodes"]
    see = np.zeros((U, M, M), bool)
    for u in range(U):
        if case["mask"] == "sparse":
            see[u] = rng.random((M, M)) < 0.15
            continue
        for i in range(M):
            p = int(rng.integers(max(-1, i - 9), i)) if i else -1
            if p >= 0:
                see[u, i] = see[u, p]
            see[u, i, i] = True
    words = (M + 63) // 64
    bits = np.zeros((U, M, words * 64), np.uint8)
    bits[:, :, :M] = see
    packed = np.packbits(bits.reshape(U, M, words, 64), axis=-1, bitorder="little")
    return torch.from_numpy(packed.view(np.int64).reshape(U, M, words).copy()).to(DEV)


def _new_tokens(case):
    return case["requests"] * (case["max_new"] + 1) // 2


def prepare(case, seed):
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "norm_rope":
        U, R, hq, hk = case["units"], case["rows"], case["hq"], case["hk"]
        # one projection row holds the queries, keys and values of a token
        qkv = torch.randn(U, R, hq + 2 * hk, D, generator=g, device=DEV)
        qkv *= torch.exp(0.5 * torch.randn(hq + 2 * hk, D, generator=g, device=DEV))
        qkv = qkv.to(torch.bfloat16)
        s["q"] = qkv[:, :, :hq].permute(0, 2, 1, 3)
        s["k"] = qkv[:, :, hq:hq + hk].permute(0, 2, 1, 3)
        s["wq"] = 1 + 0.3 * torch.randn(D, generator=g, device=DEV) if case["weights"] else None
        s["wk"] = 1 + 0.3 * torch.randn(D, generator=g, device=DEV) if case["weights"] else None
        s["eps"] = 1e-6
        s["base"] = 0
        s["pos"] = None
        if case["positions"] == "list":
            s["pos"] = torch.randint(0, case["max_pos"], (U, R), generator=g, device=DEV,
                                     dtype=torch.int32)
        else:
            s["base"] = int(rng.integers(0, case["max_pos"] - R + 1))
        s["tab"] = _tables(case["theta"], case["max_pos"])
    elif op == "page_tables":
        S, P = case["requests"], case["page"]
        lens = rng.integers(0, case["max_len"] + 1, S)
        new = rng.integers(0, case["max_new"] + 1, S)
        total = _new_tokens(case)
        while new.sum() != total:  # a batch of a fixed number of new tokens, spread at random
            off = total - int(new.sum())
            room = np.flatnonzero(new < case["max_new"] if off > 0 else new > 0)
            new[rng.permutation(room)[:abs(off)]] += 1 if off > 0 else -1
        have, need = -(-lens // P), -(-(lens + new) // P)
        pages = rng.permutation(int(need.sum()) + 5)
        width = -(-(case["max_len"] + case["max_new"]) // P)
        table = np.full((S, width), -1, np.int32)
        at = 0
        for i in range(S):
            table[i, :have[i]] = pages[at:at + have[i]]
            at += have[i]
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)  # noqa: E731
        s["lens"], s["new"], s["free"], s["table"] = t(lens), t(new), t(pages[at:]), t(table)
        s["rows"] = total + case["pad"]
    elif op == "encode_slots":
        R, H, P = case["rows"], case["heads"], case["page"]
        for x in ("K", "V"):
            lam = torch.exp((0.5 if x == "K" else 0.3) * torch.randn(H, 1, D, generator=g, device=DEV))
            s[x] = (torch.randn(H, R, D, generator=g, device=DEV) * lam).to(torch.bfloat16)
        pages = (R + P - 1) // P + 3
        slots = rng.permutation(pages * P)[:R].astype(np.int32)
        slots[rng.random(R) < case["skip"]] = -1
        s["slots"] = torch.from_numpy(slots).to(DEV)
        s["pos"] = torch.randint(0, case["max_pos"], (R,), generator=g, device=DEV, dtype=torch.int32)
        s["tab"] = _tables(case["theta"], case["max_pos"])
        for x, b in (("k", case["bits_k"]), ("v", case["bits_v"])):
            s[x + "c"] = torch.zeros(pages, H, P, 4 * b, dtype=torch.int32, device=DEV)
            s[x + "m"] = torch.zeros(pages, H, P, dtype=torch.int32, device=DEV)
    else:
        U, H, G, M, n = (case[x] for x in ("units", "heads", "G", "nodes", "n"))
        lens = rng.integers(0, n + 1, U) if case["ragged"] else np.full(U, n)
        if case["ragged"]:
            lens[int(rng.integers(U))] = n
            if U > 1:
                lens[int(rng.integers(U))] = 0
        s["hlens"] = [int(x) for x in lens]
        s["lens"] = torch.from_numpy(lens.astype(np.int32)).to(DEV) if case["ragged"] else None
        P = case["page"]
        if P:
            width = (n + P - 1) // P
            need = [(x + P - 1) // P for x in s["hlens"]]
            ids = rng.permutation(sum(need) + 3).astype(np.int32)
            table = np.full((U, width), -1, np.int32)
            at = 0
            for u in range(U):
                table[u, :need[u]] = ids[at:at + need[u]]
                at += need[u]
            s["table"] = torch.from_numpy(table).to(DEV)
            lead, cap = len(ids), P
        else:
            s["table"] = None
            lead, cap = U, n
        s["kc"], s["km"] = _store(g, lead, H, cap, case["bits_k"])
        s["vc"], s["vm"] = _store(g, lead, H, cap, case["bits_v"])
        s["pos"] = None
        s["max_pos"] = n
        if case["kept"]:  # ascending positions of the kept tokens of a longer cache
            s["max_pos"] = n + n // 2 + 8
            s["pos"] = torch.stack([torch.randperm(s["max_pos"], generator=g, device=DEV)[:n].sort()[0]
                                    for _ in range(U)]).to(torch.int32)
        s["tab"] = _tables(case["theta"], s["max_pos"])
        s["q"] = (1.5 * torch.randn(U, M, H * G, D, generator=g, device=DEV)).to(torch.bfloat16).permute(0, 2, 1, 3)
        s["K"] = torch.randn(U, M, H, D, generator=g, device=DEV).to(torch.bfloat16).permute(0, 2, 1, 3)
        s["V"] = torch.randn(U, M, H, D, generator=g, device=DEV).to(torch.bfloat16).permute(0, 2, 1, 3)
        s["mask"] = _tree_mask(case, g, rng)
    return s


# ------------------------------------------------------------- plain form
def _cos_sin(pos, theta, dtype=torch.float32):
    w = theta ** (-torch.arange(64, dtype=torch.float64, device=pos.device) / 64.0)
    ang = pos.double()[..., None] * w
    return torch.cos(ang).to(dtype), torch.sin(ang).to(dtype)


def _rotate(x, c, s):
    a, b = x[..., :64], x[..., 64:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _hadamard(dtype):
    h = torch.ones(1, 1, dtype=dtype, device=DEV)
    for _ in range(7):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _norm_rope_plain(s):
    case = s["case"]
    pos = s["pos"] if s["pos"] is not None else s["base"] + torch.arange(case["rows"], device=DEV)[None]
    c, sn = _cos_sin(pos, case["theta"])
    c, sn = c[:, None], sn[:, None]
    out = []
    for x, w, t in ((s["q"], s["wq"], case["out"]), (s["k"], s["wk"], "bf16")):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
        if w is not None:
            y = y * w
        y = _rotate(y, c, sn)
        out.append(y.to(torch.bfloat16) if t == "bf16" else y)
    return tuple(out)


def _page_tables_plain(s):
    P, rows = s["case"]["page"], s["rows"]
    lens, new, free, table = s["lens"].long(), s["new"].long(), s["free"], s["table"].clone()
    S, width = table.shape
    have, need = (lens + P - 1) // P, (lens + new + P - 1) // P
    fresh = need - have
    base = torch.cumsum(fresh, 0) - fresh
    j = torch.arange(width, device=DEV)[None]
    take = (j >= have[:, None]) & (j < need[:, None])
    at = (base[:, None] + j - have[:, None]).clamp(0, free.numel() - 1)
    table = torch.where(take, free[at], table)
    starts = torch.zeros(S + 1, dtype=torch.int64, device=DEV)
    starts[1:] = torch.cumsum(new, 0)
    r = torch.arange(rows, device=DEV)
    req = (torch.searchsorted(starts, r, right=True) - 1).clamp(0, S - 1)
    real = r < starts[-1]
    t = lens[req] + r - starts[req]
    slot = table[req, (t // P).clamp(0, width - 1)].long() * P + t % P
    i32 = torch.int32
    return (table, (lens + new).to(i32), starts.to(i32), torch.where(real, slot, -1).to(i32),
            torch.where(real, t, 0).to(i32))


def _fma(a, b, c):
    return (a.double() * b.double() + c.double()).float()


def _encode_plain(x, bits, cs=None):
    """Codes and meta words of rows x [..., 128] (bf16), the codec's fp32 arithmetic."""
    v = x.float()
    if cs is not None:
        c, s = cs
        a, b = v[..., :64], v[..., 64:]
        v = torch.cat([_fma(a, c, b * s), _fma(b, c, -(a * s))], -1)
    lead = v.shape[:-1]
    h = 1
    while h < D:
        v = v.reshape(lead + (D // (2 * h), 2, h))
        v = torch.stack([v[..., 0, :] + v[..., 1, :], v[..., 0, :] - v[..., 1, :]], -2)
        h *= 2
    v = v.reshape(lead + (D,))
    amax = (2 ** bits - 1) / 2
    G, C = np.float32(1 / (amax * math.sqrt(128))), np.float32(1 / math.sqrt(128))
    sig = (v.abs().amax(-1) * float(G)).clamp(max=65504.0).to(torch.float16)
    sf = sig.float()
    r = torch.where(sf == 0, 0.0, torch.full_like(sf, float(C)) / sf)
    y = (v * r[..., None]).reshape(lead + (16, 8))

    def coset(u):
        f = torch.round(u)
        e = u - f
        d = e[..., 0] * e[..., 0]
        for i in range(1, 8):
            d = _fma(e[..., i], e[..., i], d)
        odd = f.sum(-1).long() % 2 != 0
        m = e.abs().amax(-1)
        d = torch.where(odd, d + _fma(torch.full_like(m, -2.0), m, torch.ones_like(m)), d)
        return f, e, d, odd, m

    A, B = coset(y), coset(y - 0.5)
    half = B[2] < A[2]
    f, e = torch.where(half[..., None], B[0], A[0]), torch.where(half[..., None], B[1], A[1])
    odd, m = torch.where(half, B[3], A[3]), torch.where(half, B[4], A[4])
    first = (e.abs() == m[..., None]).to(torch.int8).argmax(-1, keepdim=True)
    move = torch.where(e >= 0, 1.0, -1.0).gather(-1, first) * odd[..., None]
    f = f.scatter_add(-1, first, move)
    lim = torch.where(half, 2 ** bits - 1, 2 ** bits - 2)[..., None]
    j = f.long() + 2 ** (bits - 1) - 1 + half[..., None]
    j = torch.minimum(j.clamp(min=0), lim).reshape(lead + (D,))
    mask = (half.long() << torch.arange(16, device=x.device)).sum(-1)
    meta = mask | ((sig.view(torch.int16).long() & 0xFFFF) << 16)
    return _pack(j, bits), torch.where(meta >= 1 << 31, meta - (1 << 32), meta).to(torch.int32)


def _encode_slots_plain(s):
    case = s["case"]
    P, bk, bv = case["page"], case["bits_k"], case["bits_v"]
    t = s["tab"].view(-1, 64, 2)
    na = (case["max_pos"] + 255) // 256
    p = s["pos"].long()
    A, B = t[p >> 8], t[na + (p & 255)]
    c = _fma(A[..., 0], B[..., 0], -(A[..., 1] * B[..., 1]))
    sn = _fma(A[..., 1], B[..., 0], A[..., 0] * B[..., 1])
    kc, km = _encode_plain(s["K"], bk, (c, sn))
    vc, vm = _encode_plain(s["V"], bv)
    slot = s["slots"].long()
    row = torch.nonzero(slot >= 0)[:, 0]
    page, off = slot[row] // P, slot[row] % P
    out = []
    for dst, src in ((s["kc"], kc), (s["km"], km), (s["vc"], vc), (s["vm"], vm)):
        dst = dst.clone()
        dst[page, :, off] = src[:, row].transpose(0, 1)
        out.append(dst)
    return tuple(out)


def _unpack(codes, meta, bits):
    """2q of every coordinate (int64 [..., 128]) and the fp16 scale (float32 [...])."""
    w = codes.long() & 0xFFFFFFFF
    w = torch.cat([w, torch.zeros_like(w[..., :1])], -1)
    c = torch.arange(D, device=codes.device)
    wi, off = (bits * c) // 32, (bits * c) % 32
    j = ((w[..., wi] | (w[..., wi + 1] << 32)) >> off) & (2 ** bits - 1)
    m = meta.long() & 0xFFFFFFFF
    half = ((m[..., None] >> (c // 8)) & 1)
    sig = (m >> 16).to(torch.int32).to(torch.int16).view(torch.float16)
    return 2 * j - 2 ** bits + 2 - half, sig.float()


def _unit_rows(s, u, x):
    """Codes and meta of the tokens of unit u, [heads][len][...]."""
    n = s["hlens"][u]
    c, m = s[x + "c"], s[x + "m"]
    if s["table"] is None:
        return c[u, :, :n], m[u, :, :n]
    P = s["case"]["page"]
    t = torch.arange(n, device=DEV)
    page = s["table"][u].long()[t // P]
    return c[page, :, t % P].transpose(0, 1), m[page, :, t % P].transpose(0, 1)


def _see(s):
    """Which draft nodes each node attends: bool [units][nodes][nodes]."""
    U, M = s["case"]["units"], s["case"]["nodes"]
    if s["mask"] is None:
        return torch.ones(M, M, dtype=torch.bool, device=DEV).tril().expand(U, M, M)
    j = torch.arange(M, device=DEV)
    return ((s["mask"][:, :, j // 64] >> (j % 64)) & 1).bool()


def _tree_plain(s):
    case = s["case"]
    U, H, G, M = (case[x] for x in ("units", "heads", "G", "nodes"))
    Hm = _hadamard(torch.float32)
    C = float(np.float32(1 / math.sqrt(128)))
    see = _see(s)
    out = torch.empty(U, H * G, M, D, dtype=torch.bfloat16, device=DEV)
    for u in range(U):
        n = s["hlens"][u]
        c, sn = _cos_sin(s["pos"][u, :n] if s["pos"] is not None else torch.arange(n, device=DEV),
                         case["theta"])
        q = s["q"][u].float().reshape(H, G * M, D)
        Kn, Vn = s["K"][u].float(), s["V"][u].float()
        sd = torch.einsum("hrd,hjd->hrj", q, Kn) * D ** -0.5
        sd = sd.masked_fill(~see[u].repeat(G, 1)[None], -math.inf)
        step = max(1, (1 << 28) // max(1, n * max(G * M, D)))
        kc, km = _unit_rows(s, u, "k")
        vc, vm = _unit_rows(s, u, "v")
        for h in range(0, H, step):
            t, sig = _unpack(kc[h:h + step], km[h:h + step], case["bits_k"])
            k = _rotate((t.float() @ Hm) * (sig * 0.5 * C)[..., None], c, sn)
            t, sig = _unpack(vc[h:h + step], vm[h:h + step], case["bits_v"])
            v = (t.float() @ Hm) * (sig * 0.5 * C)[..., None]
            del t
            sc = torch.cat([q[h:h + step] @ k.transpose(1, 2) * D ** -0.5, sd[h:h + step]], -1)
            m = sc.amax(-1, keepdim=True)
            p = torch.exp(sc - torch.where(m == -math.inf, 0.0, m))
            l = p.sum(-1, keepdim=True)
            o = p[..., :n] @ v + p[..., n:] @ Vn[h:h + step]
            o = torch.where(l > 0, o / l, 0.0)
            out[u, h * G:(h + step) * G] = o.reshape(-1, M, D).to(torch.bfloat16)
    return out


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"norm_rope": _norm_rope_plain, "page_tables": _page_tables_plain,
                "encode_slots": _encode_slots_plain, "tree_attend": _tree_plain}[op](state)
    from e8_lattice_vector_nq_b200 import nq

    s, case = state, state["case"]
    if op == "norm_rope":
        return nq.nq_qk_norm_rope(
            s["q"], s["k"], s["tab"], case["max_pos"], positions=s["pos"], pos_base=s["base"],
            q_weight=s["wq"], k_weight=s["wk"], eps=s["eps"],
            q_dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    if op == "page_tables":
        t = nq.nq_page_tables(s["lens"], s["new"], case["page"], s["free"], s["table"], s["rows"])
        return s["table"], t.lens, t.starts, t.slots, t.positions
    ks = nq.PackedStore(s["kc"], s["km"], case["bits_k"])
    vs = nq.PackedStore(s["vc"], s["vm"], case["bits_v"])
    if op == "encode_slots":
        nq.nq_encode_slots(s["K"], s["V"], ks, vs, s["slots"], s["pos"], s["tab"], case["max_pos"])
        return s["kc"], s["km"], s["vc"], s["vm"]
    return nq.nq_tree_attend(s["q"], s["K"], s["V"], ks, vs, case["n"], s["tab"], s["max_pos"],
                             mask=s["mask"], lens=s["lens"], table=s["table"], positions=s["pos"])


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "norm_rope":
        rows = case["units"] * case["rows"]
        qb = 2 if case["out"] == "bf16" else 4
        elems = rows * D * (case["hq"] + case["hk"])
        return {"bytes": rows * D * (case["hq"] * (2 + qb) + case["hk"] * 4) + 4 * rows, "flops": 8 * elems}
    if op == "page_tables":
        S = case["requests"]
        new = _new_tokens(case)
        return {"bytes": int(8 * S + 8 * S + 8 * (new + case["pad"]) + 8 * new / case["page"]),
                "flops": int(8 * new)}
    if op == "encode_slots":
        vec = case["rows"] * case["heads"] * (1 - case["skip"])
        per = 512 + 16 * (case["bits_k"] + case["bits_v"]) + 8
        return {"bytes": int(vec * per + 8 * case["rows"]), "flops": int(vec * 2 * 128 * 30)}
    U, H, G, M, n = (case[x] for x in ("units", "heads", "G", "nodes", "n"))
    tokens = U * n * (0.5 if case["ragged"] else 1.0)
    vec = tokens * H
    byts = vec * (16 * (case["bits_k"] + case["bits_v"]) + 8) + (4 * tokens if case["kept"] else 0)
    byts += U * M * H * D * 2 * (2 * G + 2)
    return {"bytes": int(byts), "flops": int(4 * D * G * M * vec + 2 * D * G * M * M * U * H)}


# ------------------------------------------------------- 64-bit evaluation
def _exact_norm_rope(s):
    case = s["case"]
    R = case["rows"]
    w = torch.tensor([case["theta"] ** (-i / 64.0) for i in range(64)], dtype=torch.float64, device=DEV)
    if s["pos"] is None:
        pos = torch.arange(s["base"], s["base"] + R, device=DEV).expand(case["units"], R)
    else:
        pos = s["pos"]
    z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                    pos.to(torch.float64)[:, None, :, None] * w)
    out = []
    for x, g in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.to(torch.float64)
        y = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / D + s["eps"])
        y = y if g is None else y * g.to(torch.float64)
        r = torch.complex(y[..., :64].contiguous(), y[..., 64:].contiguous()) * z
        out.append(torch.cat([r.real, r.imag], -1))
    return tuple(out)


def _exact_pages(s):
    P = s["case"]["page"]
    lens, new = s["lens"].tolist(), s["new"].tolist()
    free, table = s["free"].tolist(), s["table"].cpu().numpy().copy()
    slots, pos, starts, used = [], [], [0], 0
    for r, (a, c) in enumerate(zip(lens, new)):
        for t in range(a, a + c):
            if t % P == 0:
                table[r, t // P] = free[used]
                used += 1
            slots.append(int(table[r, t // P]) * P + t % P)
            pos.append(t)
        starts.append(starts[-1] + c)
    pad = s["rows"] - len(slots)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return (torch.from_numpy(table).to(DEV), t([a + c for a, c in zip(lens, new)]), t(starts),
            t(slots + [-1] * pad), t(pos + [0] * pad))


def _fwht64(x):
    for b in range(7):
        y = x.reshape(x.shape[:-1] + (D >> (b + 1), 2, 1 << b))
        lo, hi = y[..., 0, :], y[..., 1, :]
        x = torch.stack((lo + hi, lo - hi), -2).reshape(x.shape)
    return x


def _exact_values(s, u, h, x):
    n, bits = s["hlens"][u], s["case"]["bits_" + x]
    codes, meta = s[x + "c"], s[x + "m"]
    if s["table"] is None:
        codes, meta = codes[u, h, :n], meta[u, h, :n]
    else:
        P = s["case"]["page"]
        pages = s["table"][u, :(n + P - 1) // P].long()
        codes = codes[pages, h].reshape(-1, 4 * bits)[:n]
        meta = meta[pages, h].reshape(-1)[:n]
    by = codes.contiguous().view(torch.uint8).view(n, 16 * bits)
    b = ((by[:, :, None] >> torch.arange(8, dtype=torch.uint8, device=DEV)) & 1).view(n, D, bits)
    j = sum(b[:, :, i].to(torch.float64) * 2 ** i for i in range(bits))
    mb = meta.contiguous().view(torch.uint8).view(n, 4)
    half = ((mb[:, :2, None] >> torch.arange(8, dtype=torch.uint8, device=DEV)) & 1).view(n, 16, 1)
    t = 2 * j.view(n, 16, 8) - (2 ** bits - 2) - half.to(torch.float64)
    sig = meta.contiguous().view(torch.float16).view(n, 2)[:, 1].to(torch.float64)
    return _fwht64(t.reshape(n, D)) * (sig / (2 * math.sqrt(128)))[:, None]


def _exact_tree(s):
    case = s["case"]
    U, H, G, M = (case[x] for x in ("units", "heads", "G", "nodes"))
    w = torch.tensor([case["theta"] ** (-i / 64.0) for i in range(64)], dtype=torch.float64, device=DEV)
    out = torch.zeros(U, H * G, M, D, dtype=torch.float64, device=DEV)
    for u in range(U):
        n = s["hlens"][u]
        pos = torch.arange(n, device=DEV) if s["pos"] is None else s["pos"][u, :n]
        z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                        pos.to(torch.float64)[:, None] * w)
        block = torch.zeros(M, M, dtype=torch.float64, device=DEV)
        if s["mask"] is None:
            block += torch.triu(torch.full((M, M), -math.inf, dtype=torch.float64, device=DEV), 1)
        else:
            words = s["mask"][u].cpu().numpy().view(np.uint8)
            bit = np.unpackbits(words, axis=-1, bitorder="little")[:, :M]
            block[torch.from_numpy(bit == 0).to(DEV)] = -math.inf
        for h in range(H):
            k = _exact_values(s, u, h, "k")
            k = torch.complex(k[:, :64].contiguous(), k[:, 64:].contiguous()) * z
            k = torch.cat([torch.cat([k.real, k.imag], -1), s["K"][u, h].to(torch.float64)])
            v = torch.cat([_exact_values(s, u, h, "v"), s["V"][u, h].to(torch.float64)])
            for g in range(G):
                a = s["q"][u, h * G + g].to(torch.float64) @ k.T / math.sqrt(D)
                a[:, n:] += block
                out[u, h * G + g] = torch.nan_to_num(torch.softmax(a, -1), nan=0.0) @ v
    return out


def exact(case, seed):
    op = case["op"]
    if op == "encode_slots":  # packed codes: no number behind them but the fp32 rule's own
        return None
    if op == "page_tables":
        return _exact_pages(prepare(case, seed))
    if op == "norm_rope":
        return _exact_norm_rope(prepare(case, seed))
    return _exact_tree(prepare(case, seed))
