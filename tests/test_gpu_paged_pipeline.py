"""The paged cache as the path uses it: compression into pages, decode steps,
a second question on a fork, a re-selection by fresh scores, and the end."""
import numpy as np
import pytest
import torch

import kv_cache_compression_layer_b200 as kv
import oracle as orc
import synth
from kv_cache_compression_layer_b200 import Compressor
from tests import _paged as pg
from tests._harness import dev, up

pytestmark = pytest.mark.gpu


def make(cfg, dtype, n_seqs, **kw):
    shape = kv.make_shape(cfg.n_layers, cfg.n_kv_heads, cfg.group, cfg.head_dim, cfg.w, dtype)
    params = kv.make_params(cfg.budget_pct, cfg.alpha, cfg.rho, cfg.r, cfg.gamma, cfg.sinks_T, cfg.recent_pct)
    comp = Compressor(shape, cfg.L, params, device=dev())
    P = kw.get("page_tokens", 64)
    longest = -(-(max(cfg.L) + 64) // P)
    psh = kv.make_paged_shape(n_seqs, cfg.n_layers, cfg.n_kv_heads, cfg.group, cfg.head_dim, dtype,
                              n_seqs * cfg.n_layers * cfg.n_kv_heads * longest, longest, **kw)
    return comp, kv.PagedCache(psh, device=dev()), pg.Model(psh)


@pytest.mark.parametrize("name,dtype,kw", [("3b", kv.KV_BF16, dict(quant_group=64, page_tokens=64)),
                                           ("ragged", kv.KV_BF16, dict(quant_group=32, page_tokens=16)),
                                           ("tiny", kv.KV_F32, dict(quant_group=32, page_tokens=32))])
def test_compress_decode_fork_compact(name, dtype, kw):
    L = {"3b": (1500,), "ragged": (700, 1500, 1000), "tiny": (1024,)}[name]
    cfg = synth.small(name, n_layers=2, L=L) if name != "tiny" else synth.CONFIGS["tiny"].with_(n_layers=2)
    steps, n = 3, len(cfg.L)
    bt = synth.make_batch(cfg, steps=steps)
    dt = pg.DT[dtype]
    comp, cache, m = make(cfg, dtype, 2 * n, **kw)
    qwin, K, V, S = up(bt.qwin, dt), up(bt.K, dt), up(bt.V, dt), up(bt.S, torch.float32)

    # compression: the same selection as the compacted path, its rows quantised
    comp.compress(qwin, K, V, S)
    kept = [(b, pos.copy(), Kc, Vc) for b, pos, Kc, Vc in comp.kept()]
    seqs = list(range(n, 2 * n))  # the second half of the cache, the first for forks
    comp.compress_paged(cache, seqs, qwin, K, V, S)
    for (b, pos, _, _), (b2, pos2, _, _) in zip(kept, comp.kept()):
        assert b == b2 and np.array_equal(pos, pos2)
    m.append(m.call_rows(seqs), [k[2].astype(np.float64) for k in kept], [k[3].astype(np.float64) for k in kept])
    m.check(cache)

    def step(t, who, src):
        """Decode step t of sequences `who` with the inputs of batch sequences `src`."""
        rows = [r for s in src for r in range(s * m.rps, (s + 1) * m.rps)]
        k, v, q = (bt.k_dec[t][rows], bt.v_dec[t][rows], bt.q_dec[t][rows])
        m.append(m.call_rows(who), k[:, None].astype(np.float64), v[:, None].astype(np.float64))
        cache.append(who, up(k, dt), up(v, dt))
        qd = up(q, dt)
        lse = torch.empty(qd.shape[:2], device=qd.device)
        out = cache.attend(who, qd, lse=lse)
        m.check_attention(qd, out, lse, who, 1)

    step(0, seqs, range(n))
    # a second question on the last sequence, its own steps, while the first goes on
    cache.fork([2 * n - 1], [0])
    m.fork([2 * n - 1], [0])
    step(1, [0], [n - 1])
    step(1, seqs[::-1], list(range(n))[::-1])
    m.check(cache)
    # half of the fork's tokens again, by the oracle's selection over fresh scores
    rng = np.random.default_rng(0)
    keeps = []
    for r in m.call_rows([0]):
        s = rng.random(m.len[r]).astype(np.float32)
        keeps.append(np.asarray(orc.select(s, [m.len[r]], 8, [m.len[r] // 2])[0], np.int32))
    off = np.concatenate([[0], np.cumsum([len(k) for k in keeps])])
    cache.compact([0], [0], torch.from_numpy(np.concatenate(keeps)).to(dev()), torch.from_numpy(off).to(dev()),
                  torch.tensor([len(k) for k in keeps], dtype=torch.int32, device=dev()))
    m.compact([0], [0], keeps)
    step(2, [0], [n - 1])
    m.check(cache)
    cache.free([0] + seqs)
    m.free([0] + seqs)
    m.check(cache)
    assert cache.free_pages() == cache.shape.n_pages


def test_compress_paged_refuses_another_shape():
    cfg = synth.small("3b", n_layers=2, L=(1500,))
    comp, cache, _ = make(cfg, kv.KV_BF16, 2)
    other = kv.PagedCache(kv.make_paged_shape(2, 3, cfg.n_kv_heads, cfg.group, cfg.head_dim, kv.KV_BF16, 64, 8),
                          device=dev())
    with pytest.raises(ValueError):
        comp.compress_paged(other, [0], None, None, None, None)
    with pytest.raises(ValueError):
        comp.compress_paged(cache, [0, 1], None, None, None, None)


def test_select_is_select_gather_without_the_gather():
    """kv_select leaves the idx of kv_select_gather, spare slots untouched."""
    cfg = synth.small("ragged", n_layers=2, L=(700, 1500))
    shape = kv.make_shape(cfg.n_layers, cfg.n_kv_heads, cfg.group, cfg.head_dim, cfg.w, kv.KV_BF16)
    params = kv.make_params(cfg.budget_pct, cfg.alpha, cfg.rho, cfg.r, cfg.gamma, cfg.sinks_T, cfg.recent_pct)
    comp = Compressor(shape, cfg.L, params, device=dev())
    S = torch.rand(cfg.n_layers, cfg.n_kv_heads, device=dev())
    comp.allocate(S)
    comp.s_hat.copy_(torch.randn(comp.n_keys, device=dev()).round(decimals=1))  # with ties
    K = torch.zeros(comp.n_keys, cfg.head_dim, dtype=torch.bfloat16, device=dev())
    comp.pos.fill_(-7)
    comp.select_gather(K, K)
    idx = torch.full_like(comp.pos, -7)
    kv.kv_select(shape, comp.L, comp.s_hat, comp.b, comp.slot_off, idx)
    assert torch.equal(idx, comp.pos)
