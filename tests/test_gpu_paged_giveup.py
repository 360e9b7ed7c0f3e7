"""kv_paged_attn whose waits run out: the status says so, and a row's output
is either what it should be or what was there before."""
import numpy as np
import pytest
import torch

import kv_cache_compression_layer_b200 as kv
from tests import _paged as pg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,top,g,n_q", [(4, 20000, 3, 1), (60, 4000, 8, 1), (60, 700, 8, 2), (900, 200, 4, 1)])
def test_rows_that_gave_up_keep_their_output(rows, top, g, n_q):
    """Rows over many blocks, over a few, and many rows a block, with no time to wait. Then every row with time
    again."""
    rng = np.random.default_rng(rows)
    cache, m = pg.make(n_seqs=1, n_layers=1, heads=rows, group=g, max_pages=-(-top // 64))
    pg.fill(cache, m, rng.integers(top // 4, top + 1, rows), rng)
    q = pg.up(0.3 * rng.normal(size=(rows, n_q * g, 128)), kv.KV_BF16, cache.device)
    want, want_lse = torch.empty_like(q), torch.empty(q.shape[:2], device=cache.device)
    cache.attend([0], q, want, lse=want_lse, n_q=n_q)
    assert cache.read_status() == 0
    part = -(-n_q * g // 16) if n_q * g > 8 else 1  # rows of queries that a block takes
    for _ in range(20):
        out, lse = torch.full_like(q, 3.0), torch.full_like(want_lse, 3.0)
        prev = kv.kv_set_wait_limit_ns(0)
        try:
            cache.attend([0], q, out, lse=lse, n_q=n_q)
            assert cache.read_status() in (0, kv.KV_DEV_TIMEOUT)
        finally:
            kv.kv_set_wait_limit_ns(prev)
        cache.status.zero_()
        for x, fill in ((out, 3.0), (lse[..., None], 3.0)):
            w = want if x is out else want_lse[..., None]
            for c in range(part):
                a, b = x[:, 16 * c:16 * c + 16].flatten(1), w[:, 16 * c:16 * c + 16].flatten(1)
                assert ((a == b).all(1) | (a == fill).all(1)).all()
    out, lse = torch.empty_like(q), torch.empty_like(want_lse)
    cache.attend([0], q, out, lse=lse, n_q=n_q)
    assert cache.read_status() == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
