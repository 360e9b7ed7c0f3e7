"""kv_paged_append and kv_paged_load against the numpy model: values, codes,
page lists and counts equal bit for bit, over types, group and page sizes."""
import numpy as np
import pytest
import torch

import kv_cache_compression_layer_b200 as kv
from tests import _paged as pg

pytestmark = pytest.mark.gpu

FORMATS = [(128, 32, 64), (128, 64, 64), (128, 128, 128), (64, 32, 16), (64, 64, 32), (128, 64, 16)]


@pytest.mark.parametrize("dtype", [kv.KV_BF16, kv.KV_F32])
@pytest.mark.parametrize("d,qg,page", FORMATS)
def test_ragged_appends(d, qg, page, dtype):
    rng = np.random.default_rng(d + qg + page + dtype)
    cache, m = pg.make(n_seqs=3, n_layers=2, heads=2, d=d, qg=qg, page=page, dtype=dtype, max_pages=20)
    cap = 20 * page
    for top in (5, page + 3, 40):  # rows of 0 .. top tokens, then more behind them
        pg.fill(cache, m, rng.integers(0, top + 1, m.rows), rng)
        m.check(cache)
    assert 0 in m.len or min(m.len) < cap


def test_page_bytes_are_as_documented():
    """The bytes of the pages, read by the header's description alone, give the model's values."""
    rng = np.random.default_rng(0)
    for d, qg, P in FORMATS:
        cache, m = pg.make(n_seqs=1, n_layers=1, heads=2, d=d, qg=qg, page=P)
        pg.fill(cache, m, [2 * P + 5, P - 1], rng)
        raw = cache.pages.cpu().numpy()
        G = d // qg
        for r in range(2):
            for t in range(m.len[r]):
                page, i = raw[m.lists[r][t // P]], t % P
                kc = page[i * d // 2:(i + 1) * d // 2].view(np.uint32).reshape(4, d // 32)
                vc = page[P * d // 2 + i * d // 2:][: d // 2].view(np.uint16).reshape(8, d // 32)
                sc = [page[P * d + x * P * G * 4 + i * G * 4:][: G * 4].view(np.uint32) for x in (0, 1)]
                step = [(s.astype(np.uint32) << 16).view(np.float32).astype(np.float64) for s in sc]
                base = [(s & 0xffff0000).view(np.float32).astype(np.float64) for s in sc]
                for c in range(d):
                    w, x = c // 32, c % 32
                    k = (int(kc[x // 8, w]) >> (4 * (x % 8))) & 15
                    p = (x // 4) ^ (4 if i & 2 else 0)
                    v = (int(vc[p, w]) >> (4 * (x % 4))) & 15
                    assert base[0][c // qg] + k * step[0][c // qg] == m.K[r][t, 0, c]
                    assert base[1][c // qg] + v * step[1][c // qg] == m.V[r][t, 0, c]


@pytest.mark.parametrize("dtype", [kv.KV_BF16, kv.KV_F32])
def test_hard_values(dtype):
    """Ties of the codes and of the steps, equal channels, one outlier, tiny, huge and non-finite values."""
    rng = np.random.default_rng(3)
    d, qg = 128, 64
    rows = [np.zeros(d), np.full(d, -3.5), np.arange(d) % 31 * 0.5, np.arange(d) % 16 * 1.0,
            -(np.arange(d) % 61) / 4.0, 2.0 ** (np.arange(d) % 40 - 20), 1e38 * np.sin(np.arange(d)),
            1e-38 * np.cos(np.arange(d)), 3e-39 * np.cos(np.arange(d)), np.where(np.arange(d) == 77, 1e30, 0.01),
            100 + 0.001 * np.arange(d)]
    for bad in (np.nan, np.inf, -np.inf):
        x = rng.normal(size=d)
        x[3] = bad
        rows.append(x)
    for _ in range(40):  # a coarse grid: many quotients halfway between two codes
        rows.append(rng.integers(-30, 31, d) * 2.0 ** rng.integers(-3, 4))
    x = np.array(rows)
    x = pg.bf16(x) if dtype == kv.KV_BF16 else x.astype(np.float32).astype(np.float64)
    cache, m = pg.make(n_seqs=1, n_layers=1, heads=1, d=d, qg=qg, dtype=dtype)
    m.append([0], [x], [x[::-1]])
    cache.append([0], pg.up(x, dtype, cache.device), pg.up(x[::-1], dtype, cache.device))
    m.check(cache)


@pytest.mark.parametrize("dtype", [kv.KV_BF16, kv.KV_F32])
def test_many_random_groups(dtype):
    """Two million random channels: every code is that of exact arithmetic."""
    rng = np.random.default_rng(11)
    n, d = 8192, 128
    x = rng.normal(size=(2, n, d)) * np.exp(rng.normal(size=(2, n, 1)) * 3) + rng.normal(size=(2, n, 1))
    x = pg.bf16(x) if dtype == kv.KV_BF16 else x.astype(np.float32).astype(np.float64)
    cache, m = pg.make(n_seqs=1, n_layers=1, heads=1, d=d, qg=32, dtype=dtype, page=128, max_pages=64)
    m.append([0], [x[0]], [x[1]])
    cache.append([0], pg.up(x[0], dtype, cache.device), pg.up(x[1], dtype, cache.device))
    m.check(cache)


def test_token_by_token_and_layer_by_layer():
    """One token a row and a layer at a time equals the model's rows; other layers stay as they are."""
    rng = np.random.default_rng(5)
    cache, m = pg.make(n_seqs=4, n_layers=3, heads=2, d=64, qg=32, page=16, max_pages=4)
    for step in range(35):
        seqs = [3, 1] if step % 2 else [0, 1, 2]
        layers = (step % 3, 1) if step % 5 else (0, 3)
        rows = m.call_rows(seqs, layers)
        n = 1 + step % 2
        K, V = pg.tokens(rng, len(rows) * n, 64, kv.KV_BF16)
        m.append(rows, K.reshape(len(rows), n, 64), V.reshape(len(rows), n, 64))
        cache.append(seqs, pg.up(K, 1, cache.device).view(len(rows), n, 64),
                     pg.up(V, 1, cache.device).view(len(rows), n, 64), layers=layers)
        m.check(cache, values=step % 7 == 6)
    m.check_values(cache, [2, 0], layers=(1, 2))


def test_kept_positions_and_bad_sources():
    """idx, idx_off and src_off as selection leaves them; sources that do not exist are stored as zeros."""
    rng = np.random.default_rng(6)
    cache, m = pg.make(n_seqs=2, n_layers=1, heads=2, d=128, qg=64)
    L, dev = [50, 50, 7, 7], cache.device
    K, V = pg.tokens(rng, sum(L), 128, 1)
    koff = np.concatenate([[0], np.cumsum(L)])
    keep = [np.sort(rng.permutation(l)[:k]) for l, k in zip(L, (20, 0, 7, 3))]
    off = np.concatenate([[0], np.cumsum([len(k) + 1 for k in keep])])
    idx = np.full(off[-1], 1 << 30, np.int32)  # spare places are not read
    for k, o in zip(keep, off):
        idx[o:o + len(k)] = k
    m.append(range(4), [K[koff[i] + k] for i, k in enumerate(keep)], [V[koff[i] + k] for i, k in enumerate(keep)])
    args = lambda ix, n: dict(count=torch.tensor(n, dtype=torch.int32, device=dev),  # noqa: E731
                              src_off=torch.from_numpy(koff[:-1].copy()).to(dev),
                              idx=torch.from_numpy(ix).to(dev), idx_off=torch.from_numpy(off).to(dev))
    Kd, Vd = pg.up(K, 1, dev), pg.up(V, 1, dev)
    cache.append([0, 1], Kd, Vd, **args(idx, [len(k) for k in keep]))
    m.check(cache)
    bad = idx.copy()
    bad[off[0] + 1], bad[off[2]], bad[off[3]] = -60, sum(L), 1 << 30
    z = np.zeros((1, 128))
    take = lambda X: [np.concatenate([X[keep[0][:1]], z, X[keep[0][2:3]]]), X[:0],  # noqa: E731
                      np.concatenate([z, X[koff[2] + keep[2][1:3]]]), z]
    m.append(range(4), take(K), take(V))
    m.status |= kv.KV_DEV_RANGE
    cache.append([0, 1], Kd, Vd, **args(bad, [3, -5, 3, 1]))
    m.check(cache)


def test_rows_that_do_not_fit_stay():
    """The pool or a row's list runs out: those rows are untouched, the rest is served."""
    rng = np.random.default_rng(7)
    cache, m = pg.make(n_seqs=4, n_layers=1, heads=1, d=64, qg=64, page=16, n_pages=5, max_pages=4)
    pg.fill(cache, m, [16, 5, 0, 0], rng)
    m.check(cache)
    pg.fill(cache, m, [32, 11, 17, 0], rng)  # 2 pages, none (its page has room), 2 pages of the 1 left
    assert m.status == kv.KV_DEV_PAGES and m.len == [48, 16, 0, 0]
    m.check(cache)
    pg.fill(cache, m, [17, 0, 0, 1], rng)  # row 0 would pass its 4 pages
    assert m.status & kv.KV_DEV_CAPACITY and m.len == [48, 16, 0, 1]
    m.check(cache)


def test_bad_page_numbers_are_reported():
    """A page number outside the pool is neither read nor written."""
    rng = np.random.default_rng(8)
    cache, m = pg.make(n_seqs=2, n_layers=1, heads=1, d=64, qg=64, page=16, max_pages=4)
    pg.fill(cache, m, [20, 20], rng)
    pages = cache.pages.clone()
    cache.table[0, 1] = cache.shape.n_pages
    cache.table[1, 0] = -3
    K = torch.full((40, 64), 5.0, dtype=torch.bfloat16, device=cache.device)
    V = K.clone()
    cache.load([0, 1], K, V, torch.tensor([0, 20, 40], device=cache.device))
    assert cache.read_status() == kv.KV_DEV_BOUNDS
    want = torch.full((40, 64), 5.0)
    want[:16] = torch.from_numpy(m.K[0][:16, 0]).float().bfloat16().float()
    want[36:] = torch.from_numpy(m.K[1][16:, 0]).float().bfloat16().float()
    assert torch.equal(K.float().cpu(), want)
    one = torch.zeros(2, 64, dtype=torch.bfloat16, device=cache.device)
    cache.append([0, 1], one, one)
    torch.cuda.synchronize()
    changed = (cache.pages != pages).any(1).nonzero().flatten().tolist()
    assert changed in ([], [m.lists[1][1]])


def test_a_group_that_rounds_to_infinity():
    """float32 values above the largest bf16: as the smallest of a group they round to an infinity, and the group
    holds NaN; as the largest they only make the step."""
    cache, _ = pg.make(n_seqs=1, n_layers=1, heads=1, d=64, qg=32, dtype=kv.KV_F32)
    top = float(np.finfo(np.float32).max)
    x = torch.full((1, 64), top, device=cache.device)
    x[0, 32:] = torch.arange(32, device=cache.device) / 31 * top
    y = -x
    cache.append([0], x, y)
    K, V = torch.empty_like(x), torch.empty_like(x)
    cache.load([0], K, V, torch.tensor([0, 1], device=cache.device))
    assert cache.read_status() == 0
    assert torch.isnan(K[0, :32]).all() and torch.isnan(V[0]).all()  # -top is the smallest of both groups of V
    want = pg.quantise(x.double().cpu().numpy(), 32)[0][0, 32:]
    assert np.array_equal(K[0, 32:].double().cpu().numpy(), want.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("dtype", [kv.KV_BF16, kv.KV_F32])
def test_channels_far_apart(dtype):
    """Groups that hold zeros and channels 2^-10 to 2^-40 of the rest, next to halves between codes: x - m is
    rounded in float32 there, and the codes are still those of exact arithmetic."""
    rng = np.random.default_rng(12)
    n, d = 512, 128
    x = rng.integers(-30, 31, (n, d)) * 0.5  # steps and halves that are met exactly
    tiny = rng.random((n, d)) < 0.2
    x = np.where(tiny, rng.normal(size=(n, d)) * 2.0 ** rng.integers(-40, -9, (n, 1)), x)
    x[rng.random((n, d)) < 0.1] = 0.0
    x[:, 0], x[:, 1] = 0.0, 15.0  # m = 0 or below, steps of a power of two among them
    x[: n // 2] = np.abs(x[: n // 2])
    x = pg.bf16(x)
    for qg in (32, 128):
        cache, m = pg.make(n_seqs=1, n_layers=1, heads=1, d=d, qg=qg, page=16, max_pages=64, dtype=dtype)
        m.append([0], [x], [-x])
        cache.append([0], pg.up(x, dtype, cache.device), pg.up(-x, dtype, cache.device))
        m.check(cache)
