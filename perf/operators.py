"""Cases of the paged 4-bit KV cache: attention over it, storing and reading tokens, and
copying, forking, compacting and freeing its pages.

A cache is a pool of pages of P tokens of one row (sequence, layer, KV head). A page holds, one after
another, the K codes [P][d/2], the V codes [P][d/2], the K scales [P][G] and the V scales [P][G]
(G = d / quant_group), a scale being two bf16: the step s, then the base m; a value is m + c s.
  K codes of a token: 32-bit words [4][d/32]; word (t, w) holds dims 32 w + 8 t + n in bits 4 n.
  V codes of a token: 16-bit words [8][d/32]; word (p, h) holds dims 32 h + 4 g + n in bits 4 n with
  g = p, or p ^ 4 where bit 1 of the token's place in its page is set.
"""
import math

import torch

own = False
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step, smallest workload: 4 rows of a 1024-token audio at a 40 % budget, fp32
        dict(name="attend_tiny_f32", op="attend", lens="1024", pct=40, layers=1, heads=4, group=1, d=64, dtype="f32",
             qg=32, page=16, nq=1),
        # one layer's call within a decode step of a 3B-class model: latency counts
        dict(name="attend_layer_3b", op="attend", lens="6000", pct=60, layers=1, heads=2, group=8, d=128, dtype="bf16",
             qg=64, page=64, nq=1),
        # every layer of a 30B-class model, 16000 audio tokens at 40 %
        dict(name="attend_30b", op="attend", lens="16000", pct=40, layers=48, heads=4, group=8, d=128, dtype="bf16",
             qg=64, page=64, nq=1),
        # the ragged serving batch, an odd GQA group, one finished (empty) sequence among it
        dict(name="attend_ragged", op="attend", lens="2000,3500,0,5000,7500,9000,12000,14000,16000", pct=25, layers=28,
             heads=4, group=7, d=128, dtype="bf16", qg=32, page=64, nq=1),
        # four tokens verified at once over whole audios (4 bits in place of eviction)
        dict(name="attend_verify_long", op="attend", lens="32768,16000,999", pct=100, layers=4, heads=4, group=8, d=128,
             dtype="bf16", qg=128, page=128, nq=4),
        # a small audio's kept tokens stored and read back, fp32
        dict(name="store_tiny_f32", op="store", lens="1024", pct=40, layers=1, heads=4, group=1, d=64, dtype="f32",
             qg=32, page=16),
        # compression of a 3B-class model's audio: 60 % of 6000 tokens
        dict(name="store_3b", op="store", lens="6000", pct=60, layers=36, heads=2, group=8, d=128, dtype="bf16", qg=64,
             page=64),
        # compression of the ragged batch
        dict(name="store_ragged", op="store", lens="2000,3500,5000,7500,9000,12000,14000,16000", pct=25, layers=28,
             heads=4, group=7, d=128, dtype="bf16", qg=64, page=64),
        # four answers sampled from one audio: fork, one token each, attention, free
        dict(name="branch_3b", op="branch", lens="6000", pct=60, layers=36, heads=2, group=8, d=128, dtype="bf16", qg=64,
             page=64, kids=4),
        # a second question on each audio of a small ragged batch, one layer range's worth of rows
        dict(name="branch_ragged", op="branch", lens="2000,3500,5000,7500", pct=25, layers=4, heads=4, group=7, d=64,
             dtype="bf16", qg=32, page=32, kids=1),
        # a cache re-selected to half its budget
        dict(name="compact_30b", op="compact", lens="16000", pct=40, layers=48, heads=4, group=8, d=128, dtype="bf16",
             qg=64, page=64, keep=50),
        # sequences moved to another pool
        dict(name="copy_ragged", op="copy", lens="2000,3500,5000,7500", pct=25, layers=28, heads=4, group=7, d=128,
             dtype="bf16", qg=128, page=64),
    ]


def draw(rng):
    def logu(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["attend", "attend", "attend", "store", "branch", "compact", "copy"])
    d = rng.choice([64, 128, 128])
    c = dict(op=op, layers=logu(1, 48), heads=rng.choice([1, 2, 4, 5, 8]), group=rng.randint(1, 8), d=d,
             dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), qg=rng.choice([g for g in (32, 64, 128) if g <= d]),
             page=rng.choice([16, 32, 64, 128]), pct=rng.choice([5, 25, 40, 60, 100]))
    # the first sequence holds a token a row at least; the others may be as short as one token, or empty
    first = 1 if c["pct"] == 100 and op != "compact" else 400
    lens = [logu(first, 32768)] + [logu(1, 32768) for _ in range(logu(1, 8) - 1)]
    n = len(lens)
    if n > 2 and rng.random() < 0.5:
        lens[rng.randrange(1, n)] = rng.choice([0, 1])
    kids = rng.randint(1, 4) if op == "branch" else 1
    # no more than the largest listed case; rows are padded to the longest one in the plain form
    while n * kids * c["layers"] * c["heads"] * max(lens) * c["pct"] / 100 * d > 3e8:
        if c["layers"] > 1:
            c["layers"] //= 2
        else:
            lens = [max(1, x // 2) if x else 0 for x in lens]
    c["lens"] = ",".join(map(str, lens))
    if op == "attend":
        c["nq"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
    if op == "branch":
        c["kids"] = kids
    if op == "compact":
        c["keep"] = rng.choice([10, 50, 90, 100])
    return c


def _lens(c):
    return [int(x) for x in c["lens"].split(",")]


def _rows_of(c, L, rs):
    """Tokens held by each of a sequence's rows: a layer's budget split over its heads, half evenly and half by
    relevance; a layer's sum does not depend on the draw."""
    H, nl = c["heads"], c["layers"]
    B = L * H * c["pct"] // 100
    rel = torch.rand(nl, H, generator=rs, dtype=torch.float64) + 0.5
    share = 0.5 / H + 0.5 * rel / rel.sum(1, keepdim=True)
    b = (B * share).floor().to(torch.int64).clamp_(max=L)
    rest = B - b.sum(1)
    for h in range(H):  # what is left goes to the first heads that have room
        give = torch.minimum(rest, L - b[:, h])
        b[:, h] += give
        rest = rest - give
    return b.reshape(-1)


def _longest(c):
    """What no row of _rows_of() is longer than."""
    H, L = c["heads"], max(_lens(c))
    B = L * H * c["pct"] // 100
    return min(L, int(B * (0.5 / H + 0.75 / (1.5 + 0.5 * (H - 1)))) + H)


def _tokens(c):
    return sum(L * c["heads"] * c["pct"] // 100 for L in _lens(c)) * c["layers"]


def work(c):
    d = c["d"]
    eb = 2 if c["dtype"] == "bf16" else 4
    T, per = _tokens(c), c["d"] + 8 * (c["d"] // c["qg"])
    rows = len(_lens(c)) * c["layers"] * c["heads"]
    state = 4 * rows + 4 * T // c["page"]  # the rows' lengths and page lists
    if c["op"] == "attend":
        R = c["nq"] * c["group"]
        return {"bytes": T * per + state + rows * R * (2 * d * eb + 4), "flops": 4.0 * T * R * d}
    if c["op"] == "store":
        return {"bytes": 2 * T * (2 * d * eb + per) + 4 * T + 3 * state, "flops": 0}
    if c["op"] == "branch":
        k, R = c["kids"], c["group"]
        # the children's table entries, their last pages, the parents' pages once, the new tokens
        return {"bytes": T * per + k * rows * (2 * (c["page"] // 2) * per + 2 * d * eb + R * (2 * d * eb + 4))
                + 4 * k * state, "flops": 4.0 * k * T * R * d}
    if c["op"] == "compact":
        T2 = T * c["keep"] // 100
        return {"bytes": T2 * (3 * per + 2 * d * eb + 4) + 4 * state, "flops": 0}
    return {"bytes": T * (3 * per + 2 * d * eb) + 4 * state, "flops": 0}


# ------------------------------------------------- 4-bit rows and their layout
def _quantise(x, qg):
    """Codes [n, d], steps and bases [n, G] (bf16) of rows x."""
    g = x.unflatten(-1, (-1, qg))
    bad = ~torch.isfinite(g).all(-1)
    m = g.amin(-1).to(torch.bfloat16)
    top = g.amax(-1)
    s = ((top.double() - m.double()) / 15).float().clamp(min=0).to(torch.bfloat16)
    t = (g.double() - m.double().unsqueeze(-1)) / s.double().unsqueeze(-1)
    c = torch.where((s == 0).unsqueeze(-1) | bad.unsqueeze(-1), 0.0, t.round().clamp(0, 15)).to(torch.int32)
    nan = torch.full_like(m, math.nan)
    return c.flatten(-2), torch.where(bad, nan, s), torch.where(bad, nan, m)


def _pack_k(c):
    w = c.unflatten(-1, (-1, 4, 8))  # [n, d/32, t, n]
    sh = 4 * torch.arange(8, device=c.device, dtype=torch.int32)
    return (w << sh).sum(-1, dtype=torch.int32).transpose(-1, -2).flatten(-2)


def _pack_v(c, place):
    w = c.unflatten(-1, (-1, 8, 4))  # [n, d/32, g, n]
    sh = 4 * torch.arange(4, device=c.device, dtype=torch.int32)
    w = (w << sh).sum(-1, dtype=torch.int32)
    w = (w - ((w > 32767).to(torch.int32) << 16)).to(torch.int16).transpose(-1, -2)  # [n, g, d/32]
    return torch.where(((place & 2) != 0)[:, None, None], w.roll(4, -2), w).flatten(-2)


def _unpack_k(w, d):
    sh = 4 * torch.arange(8, device=w.device, dtype=torch.int32)
    c = (w.unflatten(-1, (4, d // 32)).unsqueeze(-1) >> sh) & 15  # [.., t, w, n]
    return c.transpose(-3, -2).flatten(-3)


def _unpack_v(w, d, place):
    sh = 4 * torch.arange(4, device=w.device, dtype=torch.int32)
    c = (w.unflatten(-1, (8, d // 32)).to(torch.int32).unsqueeze(-1) >> sh) & 15  # [.., p, h, n]
    c = torch.where(((place & 2) != 0)[..., None, None, None], c.roll(4, -3), c)
    return c.transpose(-3, -2).flatten(-3)


def _views(pages, P, d, G):
    """The four parts of every page: K words, V words, K scales, V scales."""
    a, b = P * d // 2, P * G * 4
    return (pages[:, :a].view(torch.int32).unflatten(1, (P, d // 8)),
            pages[:, a:2 * a].view(torch.int16).unflatten(1, (P, d // 4)),
            pages[:, 2 * a:2 * a + b].view(torch.bfloat16).unflatten(1, (P, G, 2)),
            pages[:, 2 * a + b:2 * a + 2 * b].view(torch.bfloat16).unflatten(1, (P, G, 2)))


def _values(code, scale, qg):
    g = code.unflatten(-1, (-1, qg)).float()
    return (g * scale[..., 0:1].float() + scale[..., 1:2].float()).flatten(-2)


def _store_tokens(pages, P, d, qg, page, place, k, v):
    kw, vw, ks, vs = _views(pages, P, d, d // qg)
    ck, sk, mk = _quantise(k, qg)
    cv, sv, mv = _quantise(v, qg)
    kw[page, place], vw[page, place] = _pack_k(ck), _pack_v(cv, place)
    ks[page, place], vs[page, place] = torch.stack((sk, mk), -1), torch.stack((sv, mv), -1)


def _read_tokens(pages, P, d, qg, page, place):
    kw, vw, ks, vs = _views(pages, P, d, d // qg)
    return (_values(_unpack_k(kw[page, place], d), ks[page, place], qg),
            _values(_unpack_v(vw[page, place], d, place), vs[page, place], qg))


# ------------------------------------------------------------------- inputs
def _keys(n, d, g):
    """Keys with channels of their own offset and size, and values."""
    off = torch.randn(d, generator=g, device=DEV)
    size = 0.3 + torch.rand(d, generator=g, device=DEV)
    k = torch.randn(n, d, generator=g, device=DEV).mul_(size).add_(off)
    return k, torch.randn(n, d, generator=g, device=DEV)


def _flat(b, total):
    """Row and place within its row of each of the rows' tokens."""
    row = torch.repeat_interleave(torch.arange(b.numel(), device=b.device), b, output_size=total)
    start = torch.cumsum(b, 0) - b
    return row, torch.arange(total, device=b.device) - start[row]


def prepare(c, seed):
    g = torch.Generator(DEV).manual_seed(seed * 7919 + 17)
    rs = torch.Generator().manual_seed(seed * 31 + 5)
    lens, d, P, qg = _lens(c), c["d"], c["page"], c["qg"]
    G, dt = d // qg, DT[c["dtype"]]
    nseq, rps = len(lens), c["layers"] * c["heads"]
    b = torch.cat([_rows_of(c, L, rs) for L in lens])
    held = int(b.sum())
    # sequences of the cache: the parents, then room for what forks, copies and compactions make
    kids = c.get("kids", 1) if c["op"] in ("branch", "compact") else 0
    n_seqs = nseq * (1 + kids)
    rows = n_seqs * rps
    max_pages = -(-(_longest(c) + 1) // P)
    used = -(-b // P)
    n_used = int(used.sum())
    spare = {"attend": n_used // 16 + 1, "store": n_used + n_used // 16 + 8, "branch": 2 * kids * nseq * rps + 8,
             "compact": n_used + 8, "copy": 8}[c["op"]]
    n_pages = n_used + spare if c["op"] != "store" else spare
    s = {"case": c, "rps": rps, "nseq": nseq, "n_seqs": n_seqs, "n_pages": n_pages, "max_pages": max_pages,
         "b_host": b.tolist(), "total": held}
    page_bytes = P * (d + 8 * G)
    s["pages"] = torch.zeros(n_pages, page_bytes, dtype=torch.uint8, device=DEV)
    s["table"] = torch.zeros(rows, max_pages, dtype=torch.int32, device=DEV)
    s["len"] = torch.zeros(rows, dtype=torch.int32, device=DEV)
    bd = b.to(DEV)
    s["b"] = bd.to(torch.int32)
    s["seqs"] = list(range(nseq))
    s["off"] = torch.cat((torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(bd + 1, 0)))
    row, t = _flat(bd, held)
    if c["op"] == "store":  # the audio's K and V, and the kept positions of each row
        L_rows = torch.tensor([L for L in lens for _ in range(rps)], device=DEV)
        koff = torch.cumsum(L_rows, 0) - L_rows
        k, v = _keys(int(L_rows.sum()), d, g)
        s["K"], s["V"] = k.to(dt), v.to(dt)
        # ascending positions, spread over the row
        L_t, b_t = L_rows[row], bd[row]
        u = torch.rand(held, generator=g, device=DEV, dtype=torch.float64)
        pos = ((t + u) * L_t / b_t.clamp(min=1)).long()
        pos = torch.minimum(torch.maximum(pos, t), L_t - b_t + t)
        idx = torch.zeros(int(s["off"][-1]), dtype=torch.int32, device=DEV)
        idx[s["off"][row] + t] = pos.to(torch.int32)
        s["idx"], s["koff"] = idx, koff
    else:  # rows already held, their pages scattered over the pool
        perm = torch.randperm(n_pages, generator=g, device=DEV)[:n_used].to(torch.int32)
        ud = used.to(DEV)
        prow, pj = _flat(ud, n_used)
        s["table"][prow, pj] = perm
        s["len"][: nseq * rps] = s["b"]
        page, place = s["table"][row, t // P].long(), t % P
        k, v = _keys(held, d, g)
        k, v = k.to(dt), v.to(dt)
        _store_tokens(s["pages"], P, d, qg, page, place, k, v)
    ref = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    if c["op"] != "store":
        ref[perm.long()] = 1
    s["ref"] = ref
    R = c["group"] * c.get("nq", 1)

    def queries(n):
        """Queries near one of their row's keys."""
        rid = torch.arange(n, device=DEV) % (nseq * rps)
        q = torch.randn(n, R, d, generator=g, device=DEV) * 0.3
        at = torch.rand(n, R, generator=g, device=DEV) * bd[rid][:, None]
        at = torch.minimum(at.long(), bd[rid][:, None] - 1).clamp(min=0) + (torch.cumsum(bd, 0) - bd)[rid][:, None]
        near = k[at.clamp(max=max(held - 1, 0))].float() if held else 0.0
        return (q + 0.5 * near).to(dt)

    if c["op"] == "attend":
        n = nseq * rps
        s["q"] = queries(n)
        s["out"] = torch.zeros(n, R, d, dtype=dt, device=DEV)
        s["lse"] = torch.zeros(n, R, dtype=torch.float32, device=DEV)
    elif c["op"] == "branch":
        n = nseq * kids * rps
        s["src"] = [x for x in range(nseq) for _ in range(kids)]
        s["dst"] = list(range(nseq, nseq + nseq * kids))
        s["src_dev"] = torch.tensor(s["src"], device=DEV)
        parent = (s["src_dev"][:, None] * rps + torch.arange(rps, device=DEV)).flatten()
        q = queries(nseq * rps)[parent]
        s["q"] = (q.float() + 0.1 * torch.randn(q.shape, generator=g, device=DEV)).to(dt)
        kn, vn = _keys(n, d, g)
        s["k_new"], s["v_new"] = kn.to(dt), vn.to(dt)
        s["out"] = torch.zeros(n, R, d, dtype=dt, device=DEV)
        s["lse"] = torch.zeros(n, R, dtype=torch.float32, device=DEV)
    elif c["op"] == "compact":
        s["dst"] = list(range(nseq, 2 * nseq))
        n2 = b * c["keep"] // 100
        s["total2"] = int(n2.sum())
        n2d = n2.to(DEV)
        s["count"] = n2d.to(torch.int32)
        s["off2"] = torch.cat((torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(n2d + 1, 0)))
        row2, t2 = _flat(n2d, s["total2"])
        u = torch.rand(s["total2"], generator=g, device=DEV, dtype=torch.float64)
        pos = ((t2 + u) * bd[row2] / n2d[row2].clamp(min=1)).long()
        pos = torch.minimum(torch.maximum(pos, t2), bd[row2] - n2d[row2] + t2)
        idx = torch.zeros(int(s["off2"][-1]), dtype=torch.int32, device=DEV)
        idx[s["off2"][row2] + t2] = pos.to(torch.int32)
        s["idx"] = idx
    elif c["op"] == "copy":
        # the other pool is a little larger and in part taken by other sequences
        s["pages2"] = torch.zeros(2 * n_pages + 8, page_bytes, dtype=torch.uint8, device=DEV)
        taken = torch.randperm(2 * n_pages + 8, generator=g, device=DEV)[: n_pages // 2]
        s["table2"] = torch.zeros(n_seqs + 1, rps, max_pages, dtype=torch.int32, device=DEV).flatten(0, 1)
        s["len2"] = torch.zeros((n_seqs + 1) * rps, dtype=torch.int32, device=DEV)
        per = min(max_pages, taken.numel() // rps)
        if per:
            taken = taken[: per * rps]
            s["table2"][n_seqs * rps:, :per] = taken.to(torch.int32).view(rps, per)
            s["len2"][n_seqs * rps:] = per * P
        else:
            taken = taken[:0]
        s["ref2"] = torch.zeros(2 * n_pages + 8, dtype=torch.int32, device=DEV)
        s["ref2"][taken] = 1
    if c["op"] in ("store", "copy", "compact"):
        n_out = held + nseq * rps
        s["K_out"] = torch.zeros(n_out, d, dtype=dt, device=DEV)
        s["V_out"] = torch.zeros(n_out, d, dtype=dt, device=DEV)
    s["seq_dev"] = torch.tensor(s["seqs"], device=DEV)
    s["dst_dev"] = torch.tensor(s.get("dst", s["seqs"]), device=DEV)
    if own:  # the handles a program keeps: the same tensors
        import kv_cache_compression_layer_b200 as kv

        def handle(n, pages, table, lens_):
            sh = kv.make_paged_shape(n, c["layers"], c["heads"], c["group"], d,
                                     kv.KV_BF16 if c["dtype"] == "bf16" else kv.KV_F32, pages.shape[0], max_pages,
                                     quant_group=qg, page_tokens=P)
            return kv.PagedCache(sh, pages=pages, table=table, lens=lens_)

        s["cache"] = handle(n_seqs, s["pages"], s["table"], s["len"])
        if c["op"] == "copy":
            s["cache2"] = handle(n_seqs + 1, s["pages2"], s["table2"], s["len2"])
    return s


# ------------------------------------------------------------- the plain forms
def _table_rows(seq_dev, rps):
    return (seq_dev[:, None] * rps + torch.arange(rps, device=DEV)).flatten()


def _claim(table, ref, rows, old, new):
    """Pages old..new of the given rows (counts, int64) from the lowest free ones, in the order of the rows."""
    need = new - old
    base = torch.cumsum(need, 0) - need
    free = ref == 0
    rank = torch.cumsum(free, 0)
    ids = torch.argsort((~free).to(torch.uint8), stable=True)
    j = torch.arange(table.shape[1], device=DEV)
    fresh = (j >= old[:, None]) & (j < new[:, None])
    at = (base[:, None] + j - old[:, None]).clamp(0, ids.numel() - 1)
    table[rows] = torch.where(fresh, ids[at].to(torch.int32), table[rows])
    ref.add_((free & (rank <= need.sum())).to(torch.int32))


def _release(table, ref, lens, rows, P):
    j = torch.arange(table.shape[1], device=DEV)
    held = j < ((lens[rows].long() + P - 1) // P)[:, None]
    ref.index_add_(0, table[rows].flatten().long(), -held.flatten().to(torch.int32))
    lens[rows] = 0


def _plain_attend(s, rows, nq):
    c = s["case"]
    d, P, qg, g = c["d"], c["page"], c["qg"], c["group"]
    kw, vw, ks, vs = _views(s["pages"], P, d, d // qg)
    pg = s["table"][rows].long()
    place = torch.arange(P, device=DEV)
    n = s["len"][rows]
    T = pg.shape[1] * P
    K = _values(_unpack_k(kw[pg], d), ks[pg], qg).flatten(1, 2)  # [rows, T, d]
    S = torch.bmm(s["q"].float(), K.transpose(1, 2)) / math.sqrt(d)
    del K
    lim = (n[:, None] - nq + 1 + torch.arange(nq, device=DEV)).repeat_interleave(g, 1)  # [rows, R]
    seen = torch.arange(T, device=DEV) < lim[:, :, None]
    S = torch.where(seen, S, -math.inf)
    top = S.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(S - top)
    z = p.sum(-1, keepdim=True)
    V = _values(_unpack_v(vw[pg], d, place.expand(pg.shape + (P,))), vs[pg], qg).flatten(1, 2)
    V = torch.where((torch.arange(T, device=DEV) < n[:, None])[:, :, None], V, 0.0)
    o = torch.bmm(p, V) / torch.where(z > 0, z, 1.0)
    return o.to(s["q"].dtype), (top + torch.log(z)).squeeze(-1)


def _plain_load(pages, table, lens, rows, c, b, total, off, K_out, V_out):
    P = c["page"]
    row, t = _flat(b, total)
    page, place = table[rows][row, t // P].long(), t % P
    k, v = _read_tokens(pages, P, c["d"], c["qg"], page, place)
    K_out[off[row] + t], V_out[off[row] + t] = k.to(K_out.dtype), v.to(V_out.dtype)


def _plain(s):
    c = s["case"]
    d, P, qg, rps = c["d"], c["page"], c["qg"], s["rps"]
    table, lens, ref, pages = s["table"], s["len"], s["ref"], s["pages"]
    rows = _table_rows(s["seq_dev"], rps)
    if c["op"] == "attend":
        out, lse = _plain_attend(s, rows, c["nq"])
        return {"out": out, "lse": lse}
    if c["op"] == "store":
        b = s["b"].long()
        _claim(table, ref, rows, torch.zeros_like(b), (b + P - 1) // P)
        row, t = _flat(b, s["total"])
        src = s["koff"][row] + s["idx"][s["off"][row] + t]
        _store_tokens(pages, P, d, qg, table[rows][row, t // P].long(), t % P, s["K"][src], s["V"][src])
        lens[rows] = s["b"]
        _plain_load(pages, table, lens, rows, c, b, s["total"], s["off"], s["K_out"], s["V_out"])
        _release(table, ref, lens, rows, P)
        return {"K": s["K_out"], "V": s["V_out"], "table": table}
    if c["op"] == "branch":
        par, kid = _table_rows(s["src_dev"], rps), _table_rows(s["dst_dev"], rps)
        n = lens[par].long()
        full, all_ = n // P, (n + P - 1) // P
        j = torch.arange(table.shape[1], device=DEV)
        share = j < full[:, None]
        old = table[par]
        table[kid] = torch.where(share, old, table[kid])
        ref.index_add_(0, old.flatten().long(), share.flatten().to(torch.int32))
        _claim(table, ref, kid, full, all_)
        last = (all_ - 1).clamp(min=0)[:, None]
        a, z = old.gather(1, last).flatten().long(), table[kid].gather(1, last).flatten().long()
        z = torch.where(all_ > full, z, a)  # rows without a part-filled page rewrite a page with itself
        pages[z] = pages[a]
        lens[kid] = lens[par]
        _claim(table, ref, kid, all_, (n + P) // P)
        page = table[kid].gather(1, (n // P)[:, None]).flatten().long()
        _store_tokens(pages, P, d, qg, page, n % P, s["k_new"], s["v_new"])
        lens[kid] = lens[kid] + 1
        out, lse = _plain_attend(s, kid, 1)
        _release(table, ref, lens, kid, P)
        return {"out": out, "lse": lse, "table": table}
    if c["op"] == "compact":
        dst = _table_rows(s["dst_dev"], rps)
        n2 = s["count"].long()
        _claim(table, ref, dst, torch.zeros_like(n2), (n2 + P - 1) // P)
        row, t = _flat(n2, s["total2"])
        pos = s["idx"][s["off2"][row] + t].long()
        pa, ia = table[rows][row, pos // P].long(), pos % P
        pb, ib = table[dst][row, t // P].long(), t % P
        kw, vw, ks, vs = _views(pages, P, d, d // qg)
        v = vw[pa, ia].unflatten(-1, (8, d // 32))
        v = torch.where((((ia ^ ib) & 2) != 0)[:, None, None], v.roll(4, -2), v).flatten(-2)
        kw[pb, ib], vw[pb, ib], ks[pb, ib], vs[pb, ib] = kw[pa, ia], v, ks[pa, ia], vs[pa, ia]
        lens[dst] = s["count"]
        _plain_load(pages, table, lens, dst, c, n2, s["total2"], s["off2"], s["K_out"], s["V_out"])
        _release(table, ref, lens, dst, P)
        return {"K": s["K_out"], "V": s["V_out"], "table": table}
    table2, lens2, ref2, pages2 = s["table2"], s["len2"], s["ref2"], s["pages2"]
    n = lens[rows].long()
    np_ = (n + P - 1) // P
    _claim(table2, ref2, rows, torch.zeros_like(n), np_)
    n_used = sum(-(-x // P) for x in s["b_host"])
    prow, pj = _flat(np_, n_used)
    pages2[table2[rows][prow, pj].long()] = pages[table[rows][prow, pj].long()]
    lens2[rows] = lens[rows]
    _plain_load(pages2, table2, lens2, rows, c, n, s["total"], s["off"], s["K_out"], s["V_out"])
    _release(table2, ref2, lens2, rows, P)
    return {"K": s["K_out"], "V": s["V_out"], "table": table2}


# -------------------------------------------------- the framework's own calls
def _own(s):
    c, cache = s["case"], s["cache"]
    if c["op"] == "attend":
        cache.attend(s["seqs"], s["q"], s["out"], lse=s["lse"], n_q=c["nq"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "store":
        cache.append(s["seqs"], s["K"], s["V"], count=s["b"], src_off=s["koff"], idx=s["idx"], idx_off=s["off"])
        cache.load(s["seqs"], s["K_out"], s["V_out"], s["off"])
        cache.free(s["seqs"])
        return {"K": s["K_out"], "V": s["V_out"], "table": s["table"]}
    if c["op"] == "branch":
        cache.fork(s["src"], s["dst"])
        cache.append(s["dst"], s["k_new"], s["v_new"])
        cache.attend(s["dst"], s["q"], s["out"], lse=s["lse"])
        cache.free(s["dst"])
        return {"out": s["out"], "lse": s["lse"], "table": s["table"]}
    if c["op"] == "compact":
        cache.compact(s["seqs"], s["dst"], s["idx"], s["off2"], s["count"])
        cache.load(s["dst"], s["K_out"], s["V_out"], s["off2"])
        cache.free(s["dst"])
        return {"K": s["K_out"], "V": s["V_out"], "table": s["table"]}
    cache.copy_to(s["cache2"], s["seqs"], s["seqs"])
    s["cache2"].load(s["seqs"], s["K_out"], s["V_out"], s["off"])
    s["cache2"].free(s["seqs"])
    return {"K": s["K_out"], "V": s["V_out"], "table": s["table2"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------ 64-bit definition
def _grid(x):
    """x rounded to the nearest bf16, in float64."""
    return x.float().to(torch.bfloat16).double()


def _represented(x, qg):
    """What a group of x stands for once held in 4 bits, in float64, straight from the definition."""
    x = x.double().reshape(x.shape[0], -1, qg)
    lo, hi = x.min(2, keepdim=True).values, x.max(2, keepdim=True).values
    base = _grid(lo)
    step = _grid(torch.relu(hi - base) / 15.0)
    level = torch.zeros_like(x)
    for k in range(1, 16):  # the level is the number of half steps passed; a tie goes to the even level
        edge = (k - 0.5) * step
        up = x - base
        level += ((up >= edge) if k % 2 == 0 else (up > edge)) & (step > 0)
    return (base + level * step).reshape(x.shape[0], -1)


def _exact_token_rows(s, r):
    """K and V in float64 of a row's tokens, nibble by nibble from the page bytes."""
    c = s["case"]
    d, P, qg = c["d"], c["page"], c["qg"]
    n, W, G = s["b_host"][r], d // 32, d // qg
    t = torch.arange(n, device=DEV)
    raw = s["pages"][s["table"][r].long()[t // P]]
    i = torch.arange(d, device=DEV)
    place = (t % P)[:, None]
    kb = place * (d // 2) + ((i % 32 // 8) * W + i // 32) * 4 + i % 8 // 2
    p = (i % 32 // 4) ^ (((place >> 1) & 1) * 4)
    vb = P * d // 2 + place * (d // 2) + (p * W + i // 32) * 2 + i % 4 // 2
    ck = (raw.gather(1, kb).int() >> (4 * (i % 2)).int()) & 15
    cv = (raw.gather(1, vb).int() >> (4 * (i % 2)).int()) & 15
    out = []
    for code, first in ((ck, P * d), (cv, P * d + P * G * 4)):
        at = first + (place * G + (i // qg)) * 4
        half = [raw.gather(1, at + x).long() + 256 * raw.gather(1, at + x + 1).long() for x in (0, 2)]
        step, base = (((h << 16) - ((h >> 15) << 32)).to(torch.int32).view(torch.float32).double() for h in half)
        out.append(base + code.double() * step)
    return out


def _exact_attention(q, K, V, nq, g):
    d = q.shape[-1]
    o = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:1], -math.inf, dtype=torch.float64, device=DEV)
    for t in range(nq):
        m = K.shape[0] - nq + 1 + t
        if m > 0:
            a = q[t * g:(t + 1) * g].double() @ K[:m].T / math.sqrt(d)
            lse[t * g:(t + 1) * g] = torch.logsumexp(a, 1)
            o[t * g:(t + 1) * g] = torch.softmax(a, 1) @ V[:m]
    return o, lse


def exact(c, seed):
    s = prepare(c, seed)
    qg, nr = c["qg"], len(s["b_host"])
    if c["op"] == "attend":
        got = [_exact_attention(s["q"][r], *_exact_token_rows(s, r), c["nq"], c["group"]) for r in range(nr)]
        return {"out": torch.stack([x[0] for x in got]), "lse": torch.stack([x[1] for x in got])}
    if c["op"] == "branch":
        kn, vn = _represented(s["k_new"], qg), _represented(s["v_new"], qg)
        got, i = [], 0
        for x in s["src"]:
            for r in range(x * s["rps"], (x + 1) * s["rps"]):
                K, V = _exact_token_rows(s, r)
                got.append(_exact_attention(s["q"][i], torch.cat((K, kn[i:i + 1])), torch.cat((V, vn[i:i + 1])), 1,
                                            c["group"]))
                i += 1
        return {"out": torch.stack([x[0] for x in got]), "lse": torch.stack([x[1] for x in got]), "table": None}
    K = torch.zeros(s["K_out"].shape, dtype=torch.float64, device=DEV)
    V = torch.zeros_like(K)
    if c["op"] == "store":
        for r in range(nr):
            n, o = s["b_host"][r], int(s["off"][r])
            src = s["koff"][r] + s["idx"][o:o + n]
            if n:
                K[o:o + n], V[o:o + n] = _represented(s["K"][src], qg), _represented(s["V"][src], qg)
        return {"K": K, "V": V, "table": None}
    off = s["off2"] if c["op"] == "compact" else s["off"]
    for r in range(nr):
        k, v = _exact_token_rows(s, r)
        if c["op"] == "compact":
            n = int(s["count"][r])
            at = s["idx"][int(off[r]):int(off[r]) + n].long()
            k, v = k[at], v[at]
        K[int(off[r]):int(off[r]) + len(k)], V[int(off[r]):int(off[r]) + len(v)] = k, v
    return {"K": K, "V": V, "table": None}
