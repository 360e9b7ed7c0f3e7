"""Every paged call captured into a CUDA graph and replayed: copies between
pools (device and pinned host memory), compaction (also by an empty list),
reading back, rebuilding, and a whole compression. Against the numpy model."""
import numpy as np
import pytest
import torch

import kv_cache_compression_layer_b200 as kv
import synth
from tests import _paged as pg
from tests._harness import dev, up
from tests.test_gpu_paged_pipeline import make as make_comp

pytestmark = pytest.mark.gpu


def captured(body):
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        body()
    return graph


@pytest.mark.parametrize("host", [False, True])
def test_copies(host):
    """There and back through another pool, which may be on the host; every replay the same."""
    rng = np.random.default_rng(0)
    cache, m = pg.make(n_seqs=3, n_layers=2, heads=2, page=16, max_pages=10)
    pg.fill(cache, m, [0, 16, 33, 150] + [0] * 8, rng)
    sh = kv.make_paged_shape(2, 2, 2, 3, 128, kv.KV_BF16, 60, 12, 64, 16)
    pages = torch.zeros(60, kv.kv_paged_page_bytes(sh), dtype=torch.uint8)
    other = kv.PagedCache(sh, device=dev(), pages=pages.pin_memory() if host else pages.to(dev()))
    m2 = pg.Model(sh)

    def body():
        cache.copy_to(other, [0], [1])
        other.copy_to(cache, [1], [2])
        other.free([1])

    body()  # once as it is
    m.copy_to(m2, [0], [1])
    m2.copy_to(m, [1], [2])
    m2.free([1])
    m.check(cache)
    cache.free([2])
    m.free([2])
    graph = captured(body)
    for _ in range(3):
        graph.replay()
        m.copy_to(m2, [0], [1])
        m2.copy_to(m, [1], [2])
        m2.free([1])
        m.check(cache)
        m2.check(other, values=False)
        cache.free([2])
        m.free([2])
        m.check(cache)


def test_compaction_reading_and_rebuilding():
    rng = np.random.default_rng(1)
    cache, m = pg.make(n_seqs=3, n_layers=1, heads=2, page=32, max_pages=6)
    pg.fill(cache, m, [150, 33, 64, 5, 0, 0], rng)
    dv = cache.device
    idx, off, cnt = (torch.tensor(x, device=dv) for x in ([3, 7, 149, 9, 0, 32], [0, 3], [3, 2]))
    idx, cnt = idx.to(torch.int32), cnt.to(torch.int32)
    none, zero = torch.empty(0, dtype=torch.int32, device=dv), torch.zeros(2, dtype=torch.int32, device=dv)
    K, V = (torch.zeros(8, 128, dtype=torch.bfloat16, device=dv) for _ in range(2))
    oo = torch.tensor([0, 3, 8], device=dv)

    def body():
        cache.compact([0], [2], idx, off, cnt)
        cache.load([2], K, V, oo)
        cache.free([2])
        cache.compact([0], [2], none, off, zero)
        kv.kv_paged_rebuild(cache.shape, cache.cache)

    graph = captured(body)
    m.compact([0], [2], [[3, 7, 149], [9, 0]])
    want = [np.concatenate([x[4][:, 0], x[5][:, 0]]) for x in (m.K, m.V)]
    m.free([2])
    for _ in range(3):
        K.fill_(7), V.fill_(7)
        graph.replay()
        m.check(cache)
        for got, w in zip((K, V), want):
            assert torch.equal(got[:5].cpu(), pg.rounded(w, torch.bfloat16)) and bool((got[5:] == 7).all())


def test_a_compression():
    """compress_paged captured with its spikes, replayed into emptied sequences, beside calls of other forms."""
    cfg = synth.small("ragged", n_layers=2, L=(700, 1500))
    bt = synth.make_batch(cfg, steps=1)
    bf = torch.bfloat16
    qwin, K, V, S = up(bt.qwin, bf), up(bt.K, bf), up(bt.V, bf), up(bt.S, torch.float32)
    comp, cache, _ = make_comp(cfg, kv.KV_BF16, 4)
    spikes = 1 + 100 * (torch.rand(comp.n_keys, device=dev()) < 0.05).float()
    comp.compress_paged(cache, [0, 1], qwin, K, V, S, spikes=spikes)
    want = [x.clone() for x in (comp.b, comp.slot_off, comp.pos)]
    graph = captured(lambda: comp.compress_paged(cache, [2, 3], qwin, K, V, S, spikes=spikes))
    q = torch.randn(cfg.rows, cfg.group, cfg.head_dim, device=dev()).to(bf)
    for _ in range(2):
        comp.compress(qwin, K, V, S)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cache.lens[:cfg.rows], cache.lens[cfg.rows:2 * cfg.rows])
        assert torch.equal(cache.attend([0, 1], q), cache.attend([2, 3], q)) and cache.read_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(want, comp._paged_lists))
        cache.free([2, 3])
