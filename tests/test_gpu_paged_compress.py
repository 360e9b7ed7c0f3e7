"""Compressor.compress_paged beside the rest of a Compressor's work."""
import numpy as np
import pytest
import torch

import kv_cache_compression_layer_b200 as kv
import synth
from tests._harness import dev, up
from tests.test_gpu_paged_pipeline import make

pytestmark = pytest.mark.gpu


def inputs(cfg, bt, dt):
    return up(bt.qwin, dt), up(bt.K, dt), up(bt.V, dt), up(bt.S, torch.float32)


@pytest.mark.parametrize("name", ["ragged", "tiny"])
def test_decoding_goes_on(name):
    """Decode steps before and after the batch is compressed into pages, with other relevances, are those of a
    Compressor that does nothing else; the pages get their own lists."""
    cfg = synth.small(name, n_layers=2, L=(700, 1500, 1000)) if name != "tiny" else synth.CONFIGS["tiny"].with_(n_layers=2)
    dt, code = (torch.bfloat16, kv.KV_BF16) if name != "tiny" else (torch.float32, kv.KV_F32)
    steps, n = 8, len(cfg.L)
    bt = synth.make_batch(cfg, steps=steps)
    comp, cache, _ = make(cfg, code, n)
    twin, _, _ = make(cfg, code, n)
    qwin, K, V, S = inputs(cfg, bt, dt)
    S2 = S.flip(-1) * torch.linspace(0.2, 3.0, S.numel(), device=S.device).view_as(S)
    comp.compress(qwin, K, V, S)
    twin.compress(qwin, K, V, S)
    assert torch.equal(comp.pos, twin.pos)
    for t in range(steps):
        if t == 4:
            comp.compress_paged(cache, list(range(n)), qwin, K, V, S2)
            other, _, _ = make(cfg, code, n)
            other.compress(qwin, K, V, S2)
            assert not torch.equal(other.b, twin.b) and torch.equal(comp.b, other.b)
            assert torch.equal(comp.slot_off, other.slot_off)
            for (b, pos, _, _), (b2, pos2, _, _) in zip(comp.kept(), other.kept()):
                assert b == b2 and np.array_equal(pos, pos2)
            assert torch.equal(cache.lens, other.b) and cache.read_status() == 0
        outs = []
        for c in (comp, twin):
            out = torch.empty(cfg.rows, cfg.group, cfg.head_dim, dtype=dt, device=dev())
            c.decode_step(up(bt.q_dec[t], dt), up(bt.k_dec[t], dt), up(bt.v_dec[t], dt), out)
            outs.append(out)
        assert torch.equal(outs[0], outs[1]), t
        assert int(comp.status[0]) == 0 and int(twin.status[0]) == 0
    comp.compress(qwin, K, V, S2)
    for x, y in zip(comp.kept(), other.kept()):  # (spare slots keep what decoding left there)
        assert x[0] == y[0] and all(np.array_equal(a, b) for a, b in zip(x[1:], y[1:]))


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("as_int", [False, True])
def test_spikes_on_the_stream_that_is_given(paged, as_int):
    """Spikes multiply the scores between scoring and smoothing on the call's stream, whatever the current one does."""
    cfg = synth.small("ragged", n_layers=2, L=(700, 1500))
    bt = synth.make_batch(cfg, steps=1)
    qwin, K, V, S = inputs(cfg, bt, torch.bfloat16)
    comp, cache, _ = make(cfg, kv.KV_BF16, 4)
    spikes = torch.ones(comp.n_keys, device=dev())
    spikes[::7] = 300.0

    def run(seqs, spikes, stream=None):
        if paged:
            comp.compress_paged(cache, seqs, qwin, K, V, S, spikes=spikes, stream=stream)
        else:
            comp.compress(qwin, K, V, S, spikes=spikes, stream=stream)

    def kept():
        torch.cuda.synchronize()
        return [(b, pos.copy()) for b, pos, _, _ in comp.kept()]

    def same(x, y):
        return all(b == c and np.array_equal(p, r) for (b, p), (c, r) in zip(x, y))

    run([0, 1], None)
    without = kept()
    cache.free([0, 1])
    run([0, 1], spikes)
    want = kept()
    assert not same(want, without)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms of the current stream
    run([2, 3], spikes, st.cuda_stream if as_int else st)
    assert same(kept(), want)
    if paged:
        q = torch.randn(cfg.rows, cfg.group, cfg.head_dim, device=dev()).to(torch.bfloat16)
        assert torch.equal(cache.attend([0, 1], q), cache.attend([2, 3], q)) and cache.read_status() == 0


def test_a_whole_audio_compacted_by_the_selection():
    """An audio held in full, then cut in place by kv_select's lists (idx, slot_off and b as they are): the same
    values as its kept tokens stored straight away. Rows that a call shortens to nothing, or not at all."""
    cfg = synth.small("3b", n_layers=2, L=(1500,))
    bt = synth.make_batch(cfg, steps=1)
    qwin, K, V, S = inputs(cfg, bt, torch.bfloat16)
    comp, cache, _ = make(cfg, kv.KV_BF16, 3)  # the new pages have to be free beside the old
    cache.append([0], K.view(cfg.rows, 1500, -1), V.view(cfg.rows, 1500, -1))
    comp.compress_paged(cache, [1], qwin, K, V, S)
    assert int(comp.b.max()) < 1500
    cache.compact([0], [0], comp.pos, comp.slot_off, comp.b)
    assert cache.read_status() == 0 and torch.equal(cache.lens[:cfg.rows], cache.lens[cfg.rows:2 * cfg.rows])
    out = [torch.zeros(2, comp.n_slots, cfg.head_dim, dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    for seq, (k, v) in enumerate(out):
        cache.load([seq], k, v, comp.slot_off)
    assert torch.equal(out[0], out[1]) and bool((out[0] != 0).any())
    q = torch.randn(cfg.rows, cfg.group, cfg.head_dim, device=dev()).to(torch.bfloat16)
    assert torch.equal(cache.attend([0], q), cache.attend([1], q))
    count = torch.arange(cfg.rows, dtype=torch.int32, device=dev()) % 3  # 0, 1 or 2 of the first tokens
    keep = torch.where(count == 2, comp.b, count)
    pos = torch.arange(comp.n_slots, dtype=torch.int32, device=dev())
    row = torch.repeat_interleave(torch.arange(cfg.rows, device=dev()), comp.slot_off.diff())
    cache.compact([0], [0], (pos - comp.slot_off[row]).to(torch.int32), comp.slot_off, keep)
    assert cache.read_status() == 0 and torch.equal(cache.lens[:cfg.rows], keep)
    k, v = torch.zeros_like(out[0])
    cache.load([0], k, v, comp.slot_off)
    held = (pos - comp.slot_off[row] < keep[row])[:, None]
    assert torch.equal(k, torch.where(held, out[1][0], 0)) and torch.equal(v, torch.where(held, out[1][1], 0))


def test_ragged_rows_that_stay_empty_and_that_span_pages():
    """Appends over and over to rows of which some stay empty, some end in a page and some fill several."""
    from tests import _paged as pg

    rng = np.random.default_rng(3)
    cache, m = pg.make(n_seqs=2, n_layers=2, heads=2, page=16, max_pages=20)
    per_call = [0, 1, 15, 16, 17, 40, 0, 64]
    for _ in range(4):
        pg.fill(cache, m, per_call, rng)
        m.check(cache)
    assert 0 in m.len and max(len(x) for x in m.lists) == 16
    assert any(n % 16 for n in m.len) and any(n and n % 16 == 0 for n in m.len)
