"""Forking, copying, compacting and freeing pages against the numpy model:
page lists, counts, the free set and every value equal."""
import numpy as np
import pytest
import torch

import kv_cache_compression_layer_b200 as kv
from tests import _paged as pg
from tests.test_gpu_paged_attn import attend

pytestmark = pytest.mark.gpu


def keep_lists(rng, m, src, frac):
    return [np.sort(rng.permutation(m.len[r])[: int(round(frac * m.len[r]))]) for r in m.call_rows(src)]


def compact(cache, m, src, dst, keeps):
    n = [len(k) for k in keeps]
    off = np.concatenate([[0], np.cumsum([x + 1 for x in n])])
    idx = np.full(off[-1], 1 << 30, np.int32)
    for k, o in zip(keeps, off):
        idx[o:o + len(k)] = k
    dev = cache.device
    cache.compact(src, dst, torch.from_numpy(idx).to(dev), torch.from_numpy(off).to(dev),
                  torch.tensor(n, dtype=torch.int32, device=dev))
    m.compact(src, dst, keeps)


@pytest.mark.parametrize("d,qg,page,dtype", [(128, 64, 64, kv.KV_BF16), (64, 32, 16, kv.KV_BF16),
                                             (128, 32, 128, kv.KV_F32), (64, 64, 32, kv.KV_F32),
                                             (128, 128, 16, kv.KV_BF16)])
def test_life_of_a_cache(d, qg, page, dtype):
    """Forks that grow apart, are compacted, freed and their pages used again, with attention in between."""
    rng = np.random.default_rng(d + qg + page)
    cache, m = pg.make(n_seqs=6, n_layers=2, heads=2, d=d, qg=qg, page=page, dtype=dtype, max_pages=12)
    counts = np.zeros(m.rows, int)
    counts[: 2 * m.rps] = rng.integers(0, 5 * page, 2 * m.rps)
    counts[0], counts[1] = 2 * page, 0  # a row that ends with its page, an empty one
    pg.fill(cache, m, counts, rng)
    cache.fork([0, 0, 1], [2, 3, 4])
    m.fork([0, 0, 1], [2, 3, 4])
    m.check(cache)
    for n in (1, 3, page):
        rows = m.call_rows([2, 4, 3])
        K, V = pg.tokens(rng, len(rows) * n, d, dtype)
        m.append(rows, K.reshape(-1, n, d), V.reshape(-1, n, d))
        cache.append([2, 4, 3], pg.up(K, dtype, cache.device), pg.up(V, dtype, cache.device))
    m.check(cache)
    attend(cache, m, rng, [2, 0, 3, 4])
    compact(cache, m, [2, 0], [2, 5], keep_lists(rng, m, [2, 0], 0.6))  # in place, and into another
    m.check(cache)
    cache.free([0, 3])
    m.free([0, 3])
    m.check(cache)  # what 4 and 2 share with them stays
    cache.fork([5], [0])
    m.fork([5], [0])
    compact(cache, m, [1], [3], keep_lists(rng, m, [1], 0.3))
    pg.fill(cache, m, rng.integers(0, page, m.rows), rng)
    m.check(cache)
    attend(cache, m, rng, list(range(6)), n_q=2)
    cache.free(list(range(6)))
    m.free(list(range(6)))
    m.check(cache)
    assert cache.free_pages() == cache.shape.n_pages


def test_compact_lists_of_any_kind():
    """Nothing kept, everything kept, positions in any order and twice, positions that do not exist."""
    rng = np.random.default_rng(1)
    cache, m = pg.make(n_seqs=2, n_layers=2, heads=2, d=64, qg=32, page=16, max_pages=12)
    n = [30, 30, 1, 0, 0, 0, 0, 0]
    pg.fill(cache, m, n, rng)
    keeps = [np.arange(30), np.array([29, 3, 3, 17, 0]), np.array([0, 0, 0]), np.array([], int)]
    compact(cache, m, [0], [1], keeps)
    m.check(cache)
    compact(cache, m, [0], [0], [np.array([], int)] * 4)
    m.check(cache)
    compact(cache, m, [1], [0], [np.array([5, 30, -1, 7]), np.array([4]), np.array([3, 0]), np.array([0])])
    assert m.status == kv.KV_DEV_RANGE
    m.check(cache)


def test_compact_in_place_shares_nothing_of_a_fork():
    """A fork's pages survive the compaction of its source and the other way round."""
    rng = np.random.default_rng(2)
    cache, m = pg.make(n_seqs=3, n_layers=1, heads=2, page=16, max_pages=10)
    pg.fill(cache, m, [100, 37, 0, 0, 0, 0], rng)
    cache.fork([0, 0], [1, 2])
    m.fork([0, 0], [1, 2])
    compact(cache, m, [0, 1], [0, 1], keep_lists(rng, m, [0, 1], 0.5))
    m.check(cache)
    cache.free([2, 0])
    m.free([2, 0])
    m.check(cache)


def test_refused_rows_stay():
    """A destination that holds tokens, a pool without pages: those rows stay, and say so."""
    rng = np.random.default_rng(3)
    cache, m = pg.make(n_seqs=3, n_layers=1, heads=2, d=64, qg=64, page=16, n_pages=8, max_pages=4)
    pg.fill(cache, m, [40, 32, 0, 5, 0, 0], rng)
    cache.fork([0], [1])  # row 3 is not empty
    m.fork([0], [1])
    assert m.status == kv.KV_DEV_BUSY
    m.check(cache)
    compact(cache, m, [0], [2], [np.arange(33), np.arange(17)])  # 3 pages, 2 pages of the 1 that is left
    assert m.status & kv.KV_DEV_PAGES
    m.check(cache)
    cache.copy_to(cache, [0], [2])
    m.copy_to(m, [0], [2])
    m.check(cache)


@pytest.mark.parametrize("where", ["device", "pinned"])
def test_copy_between_pools(where):
    """To another pool (with other numbers of sequences and pages, in part in use) and back."""
    rng = np.random.default_rng(4)
    cache, m = pg.make(n_seqs=3, n_layers=2, heads=2, d=128, qg=64, page=32, max_pages=8)
    pg.fill(cache, m, rng.integers(0, 256, m.rows), rng)
    sh2 = kv.make_paged_shape(2, 2, 2, 3, 128, kv.KV_BF16, 70, 9, 64, 32)
    m2 = pg.Model(sh2)
    if where == "pinned":
        host = torch.zeros(70, kv.kv_paged_page_bytes(sh2), dtype=torch.uint8).pin_memory()
        c2 = kv.PagedCache(sh2, device=cache.device, pages=host)
        with pytest.raises(ValueError):
            c2.load([0], torch.zeros(1, 128), torch.zeros(1, 128), torch.zeros(5))
    else:
        c2 = kv.PagedCache(sh2, device=cache.device)
        cnt = np.zeros(m2.rows, int)
        cnt[:3] = [40, 0, 33]
        pg.fill(c2, m2, cnt, rng)
    cache.copy_to(c2, [2], [1])
    m.copy_to(m2, [2], [1])
    m2.check(c2, values=where == "device")
    cache.free([2, 0])
    m.free([2, 0])
    c2.copy_to(cache, [1], [0])
    m2.copy_to(m, [1], [0])
    m.check(cache)
    attend(cache, m, rng, [0, 1])


def test_large_pool_lowest_pages_first():
    """A pool larger than one pass over its bitmap, nearly full: the free pages are found, lowest first."""
    n_pages = 70001
    sh = kv.make_paged_shape(2, 1, 1, 1, 64, kv.KV_BF16, n_pages, n_pages, 64, 16)
    free = sorted({5, 31, 32, 33000, 32768, 65535, 65536, 70000})
    held = [p for p in range(n_pages) if p not in set(free)]
    table = torch.zeros(2, n_pages, dtype=torch.int32)
    table[0, : len(held)] = torch.tensor(held, dtype=torch.int32)
    lens = torch.tensor([16 * len(held), 0], dtype=torch.int32)
    cache = kv.PagedCache(sh, pages=torch.zeros(n_pages, kv.kv_paged_page_bytes(sh), dtype=torch.uint8, device="cuda"),
                          table=table.cuda(), lens=lens.cuda())
    assert cache.free_pages() == len(free)
    for n, want in ((40, free[:3]), (5 * 16 - 8, free[:7]), (16, free[:8]), (17, free[:8])):
        x = torch.randn(n, 64, device="cuda").bfloat16()
        cache.append([1], x, x)
        assert cache.table[1, : len(want)].tolist() == want
    assert cache.read_status() == kv.KV_DEV_PAGES and int(cache.lens[1]) == 128
    assert cache.free_pages() == 0
    cache.free([0])
    assert cache.free_pages() == n_pages - 8


def test_rebuild_reports_bad_lists():
    cache, _ = pg.make(n_seqs=1, n_layers=1, heads=2, max_pages=4)
    cache.table[0, 0] = cache.shape.n_pages + 3
    cache.lens[0], cache.lens[1] = 5, -7
    other = kv.PagedCache(cache.shape, pages=cache.pages, table=cache.table, lens=cache.lens)
    assert other.read_status() == kv.KV_DEV_BOUNDS and other.free_pages() == cache.shape.n_pages
    other.free([0])  # the page that is none is not counted
    assert other.free_pages() == cache.shape.n_pages


def test_nothing_to_store_and_nothing_kept():
    """Calls whose sources or positions are empty tensors."""
    rng = np.random.default_rng(6)
    cache, m = pg.make(n_seqs=2, n_layers=1, heads=2, page=16)
    pg.fill(cache, m, [20, 3, 0, 0], rng)
    dev = cache.device
    none = torch.empty(0, 128, dtype=torch.bfloat16, device=dev)
    zero = torch.zeros(2, dtype=torch.int32, device=dev)
    off = torch.zeros(3, dtype=torch.int64, device=dev)
    idx = torch.empty(0, dtype=torch.int32, device=dev)
    cache.append([0], none, none)
    cache.append([0], none, none, count=zero, src_off=off)
    cache.append([1], none, none, count=zero, src_off=off, idx=idx, idx_off=off)
    m.check(cache)
    cache.append([0], none, none, count=zero + 2, src_off=off)  # sources that do not exist
    m.append([0, 1], [np.zeros((2, 128))] * 2, [np.zeros((2, 128))] * 2)
    m.status |= kv.KV_DEV_RANGE
    m.check(cache)
    cache.compact([0], [1], idx, off, zero)
    cache.compact([0], [0], idx, off, zero)
    m.compact([0], [0], [np.array([], int)] * 2)
    m.check(cache)
    assert cache.free_pages() == cache.shape.n_pages
    cache.load([0, 1], none, none, torch.zeros(5, dtype=torch.int64, device=dev))
    cache.fork([0], [1])
    m.check(cache)
