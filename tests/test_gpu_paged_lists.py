"""Lists of positions that are empty tensors: tokens that a count asks for all
the same have no source. Against the numpy model."""
import numpy as np
import pytest
import torch

import kv_cache_compression_layer_b200 as kv
from tests import _paged as pg

pytestmark = pytest.mark.gpu


def filled(rng, **kw):
    cache, m = pg.make(n_seqs=3, n_layers=1, heads=2, max_pages=4, **kw)
    pg.fill(cache, m, [100, 7, 64, 0, 0, 0], rng)
    return cache, m


@pytest.mark.parametrize("dtype", [kv.KV_BF16, kv.KV_F32])
def test_append_by_an_empty_list(dtype):
    """The tokens are stored as zeros and KV_DEV_RANGE is set; rows without one are left as they were."""
    rng = np.random.default_rng(0)
    cache, m = filled(rng, dtype=dtype)
    dev = cache.device
    K = pg.up(rng.normal(size=(50, 128)), dtype, dev)
    none = torch.empty(0, dtype=torch.int32, device=dev)
    off = torch.zeros(6, dtype=torch.int64, device=dev)

    def append(counts, seqs):
        count = torch.tensor(counts, dtype=torch.int32, device=dev)
        cache.append(seqs, K, K, count=count, src_off=off, idx=none, idx_off=off)

    append([0, 0, 0, 0], [0, 2])
    m.check(cache)
    append([30, 0, 17, 70], [0, 1])
    zeros = [np.zeros((n, 128)) for n in (30, 0, 17, 70)]
    m.append(m.call_rows([0, 1]), zeros, zeros)
    m.status |= kv.KV_DEV_RANGE
    m.check(cache)


@pytest.mark.parametrize("in_place", [False, True])
def test_compact_by_an_empty_list(in_place):
    """No position exists: the tokens asked for are zeros and KV_DEV_RANGE is set; more than a row holds is refused."""
    rng = np.random.default_rng(1)
    cache, m = filled(rng)
    dev = cache.device
    none = torch.empty(0, dtype=torch.int32, device=dev)
    off = torch.tensor([0, 0, 1 << 40], device=dev)  # of a list that has no entry
    dst = [0] if in_place else [2]
    for stream in (None, torch.cuda.Stream()):
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        cache.compact([0], dst, none, off, torch.tensor([20, 3], dtype=torch.int32, device=dev), stream=stream)
        m.compact([0], dst, [[-1] * 20, [-1] * 3])
        m.check(cache)
        if not in_place:
            cache.free([2])
            m.free([2])
    cache.compact([0], dst, none, off, torch.tensor([257, 0], dtype=torch.int32, device=dev))
    m.compact([0], dst, [[-1] * 257, []])
    assert m.status == kv.KV_DEV_RANGE | kv.KV_DEV_CAPACITY
    m.check(cache)
    cache.compact([1], [1], none, off, torch.zeros(2, dtype=torch.int32, device=dev))
    m.compact([1], [1], [[], []])
    m.check(cache)
