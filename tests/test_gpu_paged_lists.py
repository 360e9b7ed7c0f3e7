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
