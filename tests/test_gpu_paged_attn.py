"""kv_paged_attn against a softmax in float64 over the values held, within
bounds derived from its arithmetic (tests/_paged.py, Model.attention)."""
import numpy as np
import pytest
import torch

import kv_cache_compression_layer_b200 as kv
from tests import _paged as pg

pytestmark = pytest.mark.gpu


def queries(rng, m, rows, R, dtype, dev):
    """Queries near one of their row's keys."""
    d = m.sh.head_dim
    q = 0.3 * rng.normal(size=(len(rows), R, d))
    for i, r in enumerate(rows):
        if m.len[r]:
            q[i] += 0.5 * m.K[r][rng.integers(0, m.len[r], R), 0]
    return pg.up(np.nan_to_num(q), dtype, dev)


def attend(cache, m, rng, seqs, n_q=1, layers=None, rows_at=None):
    rows = m.call_rows(seqs, layers)
    R = n_q * m.sh.group
    q = queries(rng, m, rows, R, m.sh.dtype, cache.device)
    out, lse = torch.full_like(q, 3.0), torch.full(q.shape[:2], 3.0, device=cache.device)
    cache.attend(seqs, q, out, lse=lse, n_q=n_q, layers=layers)
    assert cache.read_status() == m.status
    m.check_attention(q, out, lse, seqs, n_q, layers, rows_at)
    return q, out, lse


CASES = [  # d, group size, page, type, g, n_q
    (128, 64, 64, kv.KV_BF16, 8, 1), (128, 32, 16, kv.KV_BF16, 7, 1), (128, 128, 128, kv.KV_BF16, 1, 1),
    (64, 64, 32, kv.KV_BF16, 5, 1), (64, 32, 64, kv.KV_BF16, 16, 1), (128, 64, 64, kv.KV_BF16, 8, 4),
    (128, 32, 32, kv.KV_BF16, 3, 5), (128, 128, 16, kv.KV_BF16, 1, 64), (64, 64, 128, kv.KV_BF16, 7, 9),
    (64, 32, 128, kv.KV_BF16, 4, 2), (128, 64, 128, kv.KV_F32, 8, 1), (128, 32, 64, kv.KV_F32, 1, 1),
    (64, 32, 16, kv.KV_F32, 3, 3), (64, 64, 64, kv.KV_F32, 16, 1), (128, 128, 32, kv.KV_F32, 5, 8)]


@pytest.mark.parametrize("d,qg,page,dtype,g,n_q", CASES)
def test_ragged_rows(d, qg, page, dtype, g, n_q):
    """Rows of 0, 1, a few and several hundred tokens, odd ends of pages and tiles."""
    rng = np.random.default_rng(d + qg + page + g + n_q)
    cache, m = pg.make(n_seqs=3, n_layers=2, heads=2, group=g, d=d, qg=qg, page=page, dtype=dtype,
                       max_pages=-(-700 // page))
    pg.fill(cache, m, [0, 1, 2, 15, 16, 17, 63, 64, 65, 129, 333, 700], rng)
    attend(cache, m, rng, [0, 1, 2], n_q)
    attend(cache, m, rng, [2, 0], n_q, layers=(1, 1))


@pytest.mark.parametrize("dtype", [kv.KV_BF16, kv.KV_F32])
@pytest.mark.parametrize("n", [1, 64, 4097, 32768])
def test_one_row(n, dtype):
    """One row over all CTAs: their partials are joined."""
    rng = np.random.default_rng(n)
    cache, m = pg.make(n_seqs=1, n_layers=1, heads=1, group=8, dtype=dtype, max_pages=512)
    pg.fill(cache, m, [n], rng)
    attend(cache, m, rng, [0])
    attend(cache, m, rng, [0], n_q=3)


def test_many_rows():
    """More rows than one launch takes, most of them short, some empty."""
    rng = np.random.default_rng(1)
    cache, m = pg.make(n_seqs=40, n_layers=10, heads=6, group=2, d=64, qg=32, page=16, max_pages=6)
    pg.fill(cache, m, rng.integers(0, 80, m.rows), rng)
    assert m.rows > 2 * 1024
    attend(cache, m, rng, list(range(40)), rows_at=set(range(0, m.rows, 7)))


def test_pages_in_any_place_and_repeatable():
    """The same tokens on other pages give the same bits; so does the same call again."""
    rng = np.random.default_rng(2)
    cache, m = pg.make(n_seqs=2, n_layers=2, heads=2, group=7, page=32, max_pages=24, n_pages=400)
    pg.fill(cache, m, rng.integers(1, 600, m.rows), rng)
    q, out, lse = attend(cache, m, rng, [0, 1])
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    cache.attend([0, 1], q, out2, lse=lse2)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    perm = torch.randperm(400, generator=torch.Generator().manual_seed(0)).to(cache.device)
    table = cache.table.clone()
    moved = torch.zeros_like(cache.pages)
    moved[perm] = cache.pages
    other = kv.PagedCache(cache.shape, pages=moved, table=perm[table.long()].to(torch.int32), lens=cache.lens.clone())
    other.attend([0, 1], q, out2, lse=lse2)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_what_lies_behind_a_row_is_not_read():
    """NaN scales behind the last token, in the part of a page that a row does not fill, reach no output; a NaN token
    does, and only those queries that see it."""
    rng = np.random.default_rng(4)
    for dtype in (kv.KV_BF16, kv.KV_F32):
        cache, m = pg.make(n_seqs=1, n_layers=1, heads=3, group=2, dtype=dtype, max_pages=4)
        cache.pages.fill_(0xff)
        pg.fill(cache, m, [5, 100, 64], rng)
        attend(cache, m, rng, [0])
        attend(cache, m, rng, [0], n_q=4)
        K, V = pg.tokens(rng, 9, 128, dtype)
        V[5, 7] = np.nan  # the second row's last token
        rows = m.call_rows([0])
        Kr, Vr = K.reshape(3, 3, 128), V.reshape(3, 3, 128)
        m.append(rows, Kr, Vr)
        cache.append([0], pg.up(Kr, dtype, cache.device), pg.up(Vr, dtype, cache.device))
        q = queries(rng, m, rows, 4, dtype, cache.device)
        out = torch.empty_like(q)
        cache.attend([0], q, out, n_q=2)
        bad = torch.isnan(out.float()).cpu()
        assert not bad[0].any() and not bad[2].any()
        # the first query does not see it; the second has it in the group of channels that holds the NaN
        assert not bad[1, :2].any() and not bad[1, :, 64:].any() and bad[1, 2:, :64].all()
        out3 = torch.empty(3, 6, 128, dtype=q.dtype, device=cache.device)
        cache.attend([0], queries(rng, m, rows, 6, dtype, cache.device), out3, n_q=3)
        bad = torch.isnan(out3.float()).cpu()
        assert not bad[1, :4].any() and bad[1, 4:, :64].all()


def test_large_logits():
    """Queries that leave all of the weight on one key, and keys in falling and rising order of their logits."""
    rng = np.random.default_rng(9)
    cache, m = pg.make(n_seqs=1, n_layers=1, heads=2, group=4, qg=128, max_pages=8)
    n = 400
    K, V = pg.tokens(rng, 2 * n, 128, 1)
    K = pg.bf16(K * np.concatenate([np.linspace(0.1, 4, n), np.linspace(4, 0.1, n)])[:, None])
    m.append([0, 1], K.reshape(2, n, 128), V.reshape(2, n, 128))
    cache.append([0], pg.up(K, 1, cache.device), pg.up(V, 1, cache.device))
    q = queries(rng, m, [0, 1], 4, 1, cache.device) * 8
    out, lse = torch.empty_like(q), torch.empty(2, 4, device=cache.device)
    cache.attend([0], q, out, lse=lse)
    m.check_attention(q, out, lse, [0], 1)


def test_another_stream_and_graph():
    """A captured step (append, attention) replayed on another stream equals the steps one by one."""
    rng = np.random.default_rng(10)
    cache, m = pg.make(n_seqs=2, n_layers=2, heads=2, group=4, page=16, max_pages=8)
    twin, m2 = pg.make(n_seqs=2, n_layers=2, heads=2, group=4, page=16, max_pages=8)
    counts = rng.integers(0, 40, m.rows)
    pg.fill(cache, m, counts, np.random.default_rng(0))
    pg.fill(twin, m2, counts, np.random.default_rng(0))
    dev = cache.device
    steps = [(pg.tokens(rng, m.rows, 128, 1), 0.5 * rng.normal(size=(m.rows, 4, 128))) for _ in range(6)]
    k, v = (torch.zeros(m.rows, 128, dtype=torch.bfloat16, device=dev) for _ in range(2))
    q = torch.zeros(m.rows, 4, 128, dtype=torch.bfloat16, device=dev)
    out = torch.zeros_like(q)
    st = torch.cuda.Stream(dev)
    st.wait_stream(torch.cuda.current_stream(dev))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        cache.append([0, 1], k, v)
        cache.attend([0, 1], q, out)
    for (K, V), Q in steps:
        with torch.cuda.stream(st):
            k.copy_(pg.up(K, 1, dev)), v.copy_(pg.up(V, 1, dev)), q.copy_(pg.up(Q, 1, dev))
            graph.replay()
        m2.append(m2.call_rows([0, 1]), K[:, None], V[:, None])
        twin.append([0, 1], pg.up(K, 1, dev), pg.up(V, 1, dev))
        want = twin.attend([0, 1], pg.up(Q, 1, dev))
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    m2.check(cache)


def test_a_wait_that_runs_out_is_reported():
    """With no time to wait the call gives up with a status; the next one is sound."""
    rng = np.random.default_rng(12)
    cache, m = pg.make(n_seqs=1, n_layers=2, heads=2, max_pages=32)
    pg.fill(cache, m, rng.integers(200, 2000, m.rows), rng)
    q = queries(rng, m, m.call_rows([0]), 3, 1, cache.device)
    prev = kv.kv_set_wait_limit_ns(0)
    try:
        cache.attend([0], q)
        assert cache.read_status() == kv.KV_DEV_TIMEOUT
    finally:
        kv.kv_set_wait_limit_ns(prev)
    cache.status.zero_()
    attend(cache, m, rng, [0])


def test_bad_page_numbers_are_reported():
    rng = np.random.default_rng(13)
    cache, m = pg.make(n_seqs=2, n_layers=1, heads=1, group=2, max_pages=4)
    pg.fill(cache, m, [200, 200], rng)
    cache.table[0, 1] = -1
    cache.table[0, 2] = cache.shape.n_pages
    q = queries(rng, m, [0, 1], 2, 1, cache.device)
    out = cache.attend([0, 1], q)
    assert cache.read_status() == kv.KV_DEV_BOUNDS
    m.check_attention(q, out, None, [0, 1], 1, rows_at={1})


def test_pages_beyond_four_gigabytes():
    """Pages whose byte offset passes 32 bits are written, read, attended over and copied."""
    rng = np.random.default_rng(14)
    n_pages, low = 480_000, 470_000  # 9216 bytes a page: the free ones start at 4.3e9
    sh = kv.make_paged_shape(3, 1, 1, 4, 128, kv.KV_BF16, n_pages, low, 64, 64)
    table = torch.zeros(3, low, dtype=torch.int32, device="cuda")
    table[0] = torch.arange(low, device="cuda")
    lens = torch.tensor([low * 64, 0, 0], dtype=torch.int32, device="cuda")
    cache = kv.PagedCache(sh, table=table, lens=lens)
    m = pg.Model(sh)
    m.ref[:low] = 1
    m.lists[0], m.len[0] = [-1], low * 64  # held, and not looked at
    K, V = pg.tokens(rng, 300, 128, 1)
    m.append([1], [K], [V])
    assert m.lists[1] == list(range(low, low + 5)) and low * 9216 > 1 << 32
    cache.append([1], pg.up(K, 1, cache.device), pg.up(V, 1, cache.device))
    cache.copy_to(cache, [1], [2])
    m.copy_to(m, [1], [2])
    m.check_values(cache, [1, 2])
    attend(cache, m, rng, [2, 1])
    assert cache.table[1, :5].tolist() == m.lists[1] and cache.table[2, :5].tolist() == m.lists[2]


def test_two_calls_at_once():
    """Two attentions over one pool on two streams, each with a workspace of its own, many times."""
    rng = np.random.default_rng(15)
    cache, m = pg.make(n_seqs=4, n_layers=2, heads=2, group=4, page=16, max_pages=60)
    pg.fill(cache, m, rng.integers(1, 900, m.rows), rng)
    ws = torch.zeros_like(cache.ws)
    second = kv.make_paged_cache(cache.pages, cache.table, cache.lens, cache.ref, cache.free_bits, cache.status, ws)
    q = [queries(rng, m, m.call_rows(s), 4, 1, cache.device) for s in ([0, 1], [1, 2, 3])]
    want = [cache.attend(s, x) for s, x in zip(([0, 1], [1, 2, 3]), q)]
    outs = [[torch.empty_like(x) for _ in range(20)] for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        kv.kv_paged_attn(cache.shape, cache.cache, [0, 1], q[0], outs[0][i], stream=streams[0])
        kv.kv_paged_attn(cache.shape, second, [1, 2, 3], q[1], outs[1][i], stream=streams[1])
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)


def test_a_branch_in_a_graph():
    """Fork, append, attention and free captured once and replayed: every replay gives the same, and leaves the cache
    as it was."""
    rng = np.random.default_rng(16)
    cache, m = pg.make(n_seqs=3, n_layers=2, heads=2, group=2, d=64, qg=32, page=16, max_pages=10)
    counts = np.zeros(m.rows, int)
    counts[: m.rps] = [0, 16, 33, 150]
    pg.fill(cache, m, counts, rng)
    dev = cache.device
    K, V = pg.tokens(rng, 2 * m.rps, 64, 1)
    k, v = pg.up(K, 1, dev), pg.up(V, 1, dev)
    m.fork([0, 0], [1, 2])
    m.append(m.call_rows([1, 2]), K[:, None], V[:, None])
    q = queries(rng, m, m.call_rows([1, 2]), 2, 1, dev)
    out = torch.empty_like(q)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        cache.fork([0, 0], [1, 2])
        cache.append([1, 2], k, v)
        cache.attend([1, 2], q, out)
        cache.free([1, 2])
    lists = [list(x) for x in m.lists]
    for _ in range(3):
        out.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        m.check_attention(q, out, None, [1, 2], 1)
        table = cache.table.cpu().numpy()
        for r in m.call_rows([1, 2]):  # what is behind a row's list stays
            assert table[r, : len(lists[r])].tolist() == lists[r]
    m.free([1, 2])
    m.check(cache)


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e4, 1e30])
def test_values_of_any_size(scale):
    """Steps of V far from 1, and rows in which they grow and shrink by powers of ten."""
    rng = np.random.default_rng(17)
    cache, m = pg.make(n_seqs=1, n_layers=1, heads=2, group=3, qg=32, max_pages=8)
    n = 300
    K, V = pg.tokens(rng, 2 * n, 128, 1)
    V = pg.bf16(V * scale)
    V[n:] = pg.bf16(V[n:] * np.repeat(10.0 ** rng.integers(-3, 4, n // 10), 10)[:, None])
    V[:40] = 0.0  # steps of 0 first
    m.append([0, 1], K.reshape(2, n, 128), V.reshape(2, n, 128))
    cache.append([0], pg.up(K, 1, cache.device), pg.up(V, 1, cache.device))
    q = queries(rng, m, [0, 1], 3, 1, cache.device)
    out = torch.empty_like(q)
    cache.attend([0], q, out)
    m.check_attention(q, out, None, [0], 1)


def test_a_padded_batch():
    """Rows without tokens and queries that are not finite (padding) leave the other queries as they should be."""
    rng = np.random.default_rng(18)
    for dtype, g, n_q in ((kv.KV_BF16, 8, 1), (kv.KV_BF16, 4, 3), (kv.KV_F32, 2, 4)):
        cache, m = pg.make(n_seqs=3, n_layers=1, heads=2, group=g, dtype=dtype, max_pages=8)
        pg.fill(cache, m, [300, 77, 0, 0, 500, 1], rng)
        R = g * n_q
        q = queries(rng, m, list(range(6)), R, dtype, cache.device)
        q[2:4] = float("nan")  # of a sequence without tokens
        spoilt = {(0, 1): float("nan"), (1, R - 1): float("inf"), (4, 0): -float("inf")}
        for at, x in spoilt.items():
            q[at][::3] = x
        out = cache.attend([0, 1, 2], q, n_q=n_q)
        assert cache.read_status() == 0
        Q, O = q.double().cpu().numpy(), out.double().cpu().numpy()
        assert (O[2:4] == 0).all()
        for r in (0, 1, 4, 5):
            good = [i for i in range(R) if (r, i) not in spoilt]
            x = Q[r].copy()
            x[[i for i in range(R) if i not in good]] = 0
            o, _, tol, _ = m.attention(x, r, n_q)
            assert (np.abs(O[r] - o) <= tol)[good].all()


def test_longest_row():
    """2^26 keys (one list that names eight pages over and over): attended over, forked, full, freed."""
    rng = np.random.default_rng(19)
    base, m = pg.make(n_seqs=1, n_layers=1, heads=1, group=2, max_pages=8)
    pg.fill(base, m, [512], rng)
    n, dev = 1 << 26, base.device
    sh = kv.make_paged_shape(2, 1, 1, 2, 128, kv.KV_BF16, 8, n // 64, 64, 64)
    table = torch.zeros(2, n // 64, dtype=torch.int32, device=dev)
    table[0] = torch.arange(n // 64, device=dev) % 8
    cache = kv.PagedCache(sh, pages=base.pages, table=table, lens=torch.tensor([n, 0], dtype=torch.int32, device=dev))
    cache.fork([0], [1])
    q = queries(rng, m, [0], 2, 1, dev)
    lse = torch.empty(2, 1, 2, device=dev)
    o0 = cache.attend([0], q, lse=lse[0])
    o1 = cache.attend([1], q, lse=lse[1])
    assert cache.read_status() == 0 and torch.equal(o0, o1) and torch.equal(lse[0], lse[1])
    o, z, tol, tol_z = m.attention(q[0].double().cpu().numpy(), 0, 1)
    # sums as in Model.attention, over the keys that a block takes (two a multiprocessor at least), a rounding of l and
    # of the base's sum for each key of a lane (32 of its keys are summed in lanes and warps of their own); what is lost
    # of a key's term is lost of its weight too, so those bounds are the 512 keys'
    N = n / (2 * torch.cuda.get_device_properties(dev).multi_processor_count)
    V = m.V[0]
    rel = N / 32 * 2.0 ** -24
    tol = tol + N / 16 * 2.0 ** -23 * (16 * V[:, 1] + np.abs(V[:, 2])).max(0) + 2 * rel * np.abs(V[:, 0]).max(0)
    assert (np.abs(o0[0].double().cpu().numpy() - o) <= tol).all()
    z = z + np.log(n / 512)
    assert (np.abs(lse[0, 0].double().cpu().numpy() - z) <= tol_z + rel + 2.0 ** -22 * np.abs(z)).all()
    one = torch.zeros(1, 128, dtype=torch.bfloat16, device=dev)
    cache.append([1], one, one)  # there is no place behind the last
    assert cache.read_status() == kv.KV_DEV_CAPACITY and cache.lens.tolist() == [n, n]
    cache.free([0])
    assert cache.free_pages() == 0
    cache.free([1])
    assert cache.free_pages() == 8


def test_graphs_that_share_a_workspace():
    """Two captured calls over one workspace, replayed in turn with calls between them, give what they gave."""
    rng = np.random.default_rng(20)
    cache, m = pg.make(n_seqs=4, n_layers=2, heads=2, group=4, page=16, max_pages=60)
    pg.fill(cache, m, rng.integers(1, 900, m.rows), rng)
    sets = [[0, 1], [2], [3, 0, 2]]
    q = [queries(rng, m, m.call_rows(s), 8, 1, cache.device) for s in sets]
    want = [cache.attend(s, x, n_q=2) for s, x in zip(sets, q)]
    outs = [torch.empty_like(x) for x in q]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graphs = []
    for s, x, o in zip(sets[:2], q, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=st):
            cache.attend(s, x, o, n_q=2)
    for i in range(10):
        for o in outs:
            o.fill_(7)
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            graphs[i % 2].replay()
            cache.attend(sets[2], q[2], outs[2], n_q=2)
            graphs[1 - i % 2].replay()
        torch.cuda.current_stream().wait_stream(st)
        assert all(torch.equal(w, o) for w, o in zip(want, outs))


def test_outputs_on_another_stream():
    """An output that the call makes belongs to the stream it was given, so that work still under way on the current
    one does not reach it."""
    rng = np.random.default_rng(21)
    cache, m = pg.make(n_seqs=1, n_layers=2, heads=2, group=8, max_pages=8)
    pg.fill(cache, m, [500] * m.rows, rng)
    q = queries(rng, m, m.call_rows([0]), 8, 1, cache.device)
    want = cache.attend([0], q)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (st, st.cuda_stream):
        held = torch.empty_like(q)
        torch.cuda._sleep(50_000_000)  # some tens of milliseconds, then a write to memory that is free again by then
        held.fill_(9)
        del held
        out = cache.attend([0], q, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert cache._on(0).stream == torch.cuda.default_stream(cache.device)  # 0 names the default stream, not a new one
    with torch.cuda.stream(st):
        st.wait_stream(torch.cuda.default_stream())
        out = cache.attend([0], q, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    with pytest.raises(ValueError):
        cache.attend([0], q, out=q)
    two = torch.empty(2 * q.numel() - 8, dtype=q.dtype, device=q.device)
    with pytest.raises(ValueError):
        cache.attend([0], two[: q.numel()], out=two[q.numel() - 8:])


def test_queries_of_one_large_channel():
    """Channels far below their query's largest, where the matrix unit's alignment cuts products: within the bound,
    and as if they were not there where they are smaller still."""
    rng = np.random.default_rng(22)
    for dtype in (kv.KV_BF16, kv.KV_F32):
        cache, m = pg.make(n_seqs=1, n_layers=1, heads=6, group=2, dtype=dtype, max_pages=8)
        pg.fill(cache, m, [200] * 6, rng)
        q = rng.normal(size=(6, 2, 128))
        for r in range(6):
            q[r] *= 2.0 ** -(4 * r + 4)
            q[r, :, rng.integers(0, 128)] = 3.0
        q = pg.up(q, dtype, cache.device)
        out, lse = torch.empty_like(q), torch.empty(6, 2, device=cache.device)
        cache.attend([0], q, out, lse=lse)
        m.check_attention(q, out, lse, [0], 1)
