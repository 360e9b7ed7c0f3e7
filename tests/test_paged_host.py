"""The paged cache without a GPU: sizes, refusals (nothing is launched), and
the numpy model that the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest
import torch

import kv_cache_compression_layer_b200 as kv
from kv_cache_compression_layer_b200 import build as kvbuild
from tests import _paged as pg


@pytest.fixture(scope="module")
def L():
    kvbuild.build()
    return kv.lib()


def shape(**kw):
    a = dict(n_seqs=4, n_layers=3, n_kv_heads=2, group=8, head_dim=128, dtype=kv.KV_BF16, n_pages=100, max_pages=10,
             quant_group=64, page_tokens=64)
    a.update(kw)
    return kv.make_paged_shape(**a)


def ints(*x):
    return (C.c_int32 * len(x))(*x)


def test_page_and_workspace_sizes(L):
    # codes of K and V (d / 2 bytes each) and a 4-byte scale per group of each, per token
    for d, qg, P in ((128, 64, 64), (128, 32, 16), (128, 128, 128), (64, 64, 32), (64, 32, 128)):
        assert kv.kv_paged_page_bytes(shape(head_dim=d, quant_group=qg, page_tokens=P)) == P * (d + 8 * d // qg)
    small, large = kv.kv_paged_ws_bytes(shape()), kv.kv_paged_ws_bytes(shape(n_pages=1 << 20))
    assert 0 < small < large and large - small >= 4 * ((1 << 20) - 100) - 256
    # a call takes at most 64 sequences, so more of them need no more
    assert kv.kv_paged_ws_bytes(shape(n_seqs=64)) == kv.kv_paged_ws_bytes(shape(n_seqs=640))


BAD = [dict(n_seqs=0), dict(n_layers=0), dict(n_kv_heads=-1), dict(group=0), dict(group=17), dict(head_dim=96),
       dict(dtype=2), dict(n_pages=0), dict(n_pages=(1 << 24) + 1), dict(max_pages=0), dict(max_pages=(1 << 20) + 1),
       dict(quant_group=16), dict(head_dim=64, quant_group=128), dict(page_tokens=8), dict(page_tokens=48),
       dict(n_seqs=1 << 15, n_layers=64), dict(n_seqs=1 << 20, n_layers=1 << 20, n_kv_heads=1 << 20)]


@pytest.mark.parametrize("bad", BAD)
def test_bad_shapes(L, bad):
    sh = shape(**bad)
    assert kv.kv_paged_page_bytes(sh) == 0 and kv.kv_paged_ws_bytes(sh) == 0
    c = kv.make_paged_cache(256, 256, 256, 256, 256, 256, 256, 1 << 40)
    assert L.kv_paged_rebuild(C.byref(sh), C.byref(c), None) == kv.KV_ERR_ARG
    assert L.kv_paged_free(C.byref(sh), C.byref(c), ints(0), 1, None) == kv.KV_ERR_ARG


NAMES = ("append", "load", "attn", "fork", "copy", "compact", "free")


def refused(L, sh, c, want, names=NAMES, seq=(0,), n=None, layer0=0, n_lay=3, K=256, V=256, n_src=6, n_each=1,
            count=None, src_off=None, idx=None, idx_off=None, q=256, out=512, lse=None, n_q=1, out_off=256, dst=(1,),
            cnt=256, ix=256, ioff=256):
    """The named calls, and no others, give status `want` with these arguments (no pointer here is one: a call that
    was not refused would reach a kernel)."""
    s, c = C.byref(sh), C.byref(c)
    n = len(seq) if n is None else n
    a, b = ints(*seq), ints(*dst)
    do = {
        "append": lambda: L.kv_paged_append(s, c, a, n, layer0, n_lay, K, V, n_src, n_each, count, src_off, idx,
                                            idx_off, None),
        "load": lambda: L.kv_paged_load(s, c, a, n, layer0, n_lay, out_off, n_src, K, V, None),
        "attn": lambda: L.kv_paged_attn(s, c, a, n, layer0, n_lay, n_q, q, out, lse, None),
        "fork": lambda: L.kv_paged_fork(s, c, a, b, n, None),
        "copy": lambda: L.kv_paged_copy(s, c, a, s, c, b, n, None),
        "compact": lambda: L.kv_paged_compact(s, c, a, b, n, ix, ioff, cnt, None),
        "free": lambda: L.kv_paged_free(s, c, a, n, None)}
    for name in names:
        assert do[name]() == want, name


def test_argument_errors_launch_nothing(L):
    sh = shape()
    ok = dict(pages=256, table=256, lens=256, ref=256, free_bits=256, status=256, ws=256, ws_bytes=1 << 40)
    ARG, pairs, ranged = kv.KV_ERR_ARG, ("fork", "copy", "compact"), ("append", "load", "attn")
    for name in ("pages", "table", "lens", "ref", "free_bits", "status"):
        for bad in (None, 257):
            c = kv.make_paged_cache(**{**ok, name: bad})
            refused(L, sh, c, ARG)
            assert L.kv_paged_rebuild(C.byref(sh), C.byref(c), None) == ARG
    for bad in (dict(ws=None), dict(ws=264), dict(ws_bytes=kv.kv_paged_ws_bytes(sh) - 1)):
        c = kv.make_paged_cache(**{**ok, **bad})
        refused(L, sh, c, kv.KV_ERR_WORKSPACE, ranged + pairs)
        assert L.kv_paged_rebuild(C.byref(sh), C.byref(c), None) == kv.KV_ERR_WORKSPACE
    c = kv.make_paged_cache(**ok)
    for bad in (dict(seq=(4,)), dict(seq=(-1,)), dict(n=0), dict(n=65)):
        refused(L, sh, c, ARG, **bad)
    refused(L, sh, c, ARG, ranged + ("free",), seq=(0, 0), dst=(1, 2))
    for bad in (dict(dst=(4,)), dict(seq=(0, 1), dst=(2, 2)), dict(seq=(0, 1), dst=(1, 2))):
        refused(L, sh, c, ARG, pairs, **bad)
    refused(L, sh, c, ARG, ("fork", "copy"), seq=(0,), dst=(0,))  # in place: compact only
    refused(L, sh, c, ARG, ("compact",), seq=(0, 0), dst=(0, 1))  # replaced while another entry's src
    for bad in (dict(layer0=-1), dict(n_lay=0), dict(layer0=1, n_lay=3), dict(layer0=3, n_lay=1),
                dict(layer0=(1 << 31) - 1, n_lay=1), dict(layer0=1, n_lay=(1 << 31) - 1)):
        refused(L, sh, c, ARG, ranged, **bad)
    for bad in (dict(K=None), dict(V=264), dict(n_src=-1)):
        refused(L, sh, c, ARG, ("append", "load"), **bad)
    for bad in (dict(n_each=-1), dict(count=256), dict(idx=256), dict(idx=256, src_off=256),
                dict(idx=256, idx_off=256)):
        refused(L, sh, c, ARG, ("append",), **bad)
    for bad in (None, 260):
        refused(L, sh, c, ARG, ("load",), out_off=bad)
    for bad in (dict(n_q=0), dict(n_q=9), dict(n_q=1 << 29), dict(q=None), dict(q=264), dict(out=None), dict(out=256),
                dict(lse=258)):
        refused(L, sh, c, ARG, ("attn",), **bad)
    for bad in (dict(ix=None), dict(ioff=None), dict(cnt=None)):
        refused(L, sh, c, ARG, ("compact",), **bad)
    for bad in (dict(n_layers=2), dict(n_kv_heads=3), dict(head_dim=64), dict(quant_group=32), dict(page_tokens=32)):
        assert L.kv_paged_copy(C.byref(sh), C.byref(c), ints(0), C.byref(shape(**bad)), C.byref(c), ints(1), 1,
                               None) == ARG
    host = (C.c_uint8 * 4096)()  # pageable memory holds no pages
    addr = (C.addressof(host) + 15) // 16 * 16
    c2 = kv.make_paged_cache(**{**ok, "pages": addr, "table": 512})
    assert L.kv_paged_copy(C.byref(sh), C.byref(c2), ints(0), C.byref(sh), C.byref(c2), ints(1), 1, None) == ARG


@pytest.mark.parametrize("name", ["kv_paged_rebuild", "kv_paged_append", "kv_paged_load", "kv_paged_attn",
                                  "kv_paged_fork", "kv_paged_copy", "kv_paged_compact", "kv_paged_free"])
def test_fault_injection_env(L, monkeypatch, name):
    monkeypatch.setenv("KV_FAULT_INJECT", name)
    sh, c = shape(), kv.make_paged_cache(None, None, None, None, None, None, None, 0)
    if name == "kv_paged_rebuild":
        assert L.kv_paged_rebuild(C.byref(sh), C.byref(c), None) == kv.KV_ERR_CUDA
    else:
        refused(L, sh, c, kv.KV_ERR_CUDA, (name[len("kv_paged_"):],))


def test_select_argument_errors(L):
    sh = kv.make_shape(2, 2, 4, 64, 1, kv.KV_BF16)
    assert L.kv_select(C.byref(sh), ints(700), 1, 256, 256, None, 256, None) == kv.KV_ERR_ARG
    assert L.kv_select(C.byref(sh), ints(701), 1, 256, 256, 256, 256, None) == kv.KV_ERR_UNSUPPORTED_L


def test_wrapper_refuses_what_does_not_match():
    class Cache(kv.PagedCache):  # the checks alone: no device, no library state
        def __init__(self):
            self.shape, self.device, self.on_host = shape(), torch.device("cpu"), False
            self.dtype = torch.bfloat16

    c = Cache()
    n, d = 3 * 2, 128
    x = torch.zeros(n, d, dtype=torch.bfloat16)
    cnt, off = torch.zeros(n, dtype=torch.int32), torch.zeros(n + 1, dtype=torch.int64)
    bad = [lambda: c.append([0], x.float(), x), lambda: c.append([0], x, x[:3]), lambda: c.append([0], x[:4], x[:4]),
           lambda: c.append([0], x.t(), x.t()), lambda: c.append([0], x[:, :64], x[:, :64]),
           lambda: c.append([0], x, x, count=cnt), lambda: c.append([0], x, x, src_off=off),
           lambda: c.append([0], x, x, count=cnt.long(), src_off=off),
           lambda: c.append([0], x, x, count=cnt[:2], src_off=off),
           lambda: c.append([0], x, x, count=cnt, src_off=off, idx=cnt),
           lambda: c.append([0], x, x, count=cnt, src_off=off.int()), lambda: c.append([], x, x),
           lambda: c.append(list(range(65)), x, x), lambda: c.load([0], x, x, off[:n]),
           lambda: c.load([0], x, x[:2], off), lambda: c.load([0], x, x, off.int()),
           lambda: c.attend([0], x), lambda: c.attend([0], torch.zeros(n, 8, d)),
           lambda: c.attend([0], torch.zeros(n, 8, d, dtype=torch.bfloat16), lse=torch.zeros(n, 7)),
           lambda: c.attend([0], torch.zeros(n, 8, d, dtype=torch.bfloat16), out=x),
           lambda: c.append([0], x, x, layers=(0, 0)), lambda: c.attend([0], x, layers=(1, 3)),
           lambda: c.load([0], x, x, off, layers=(-1, 2)),
           lambda: kv.PagedCache(shape(), device="cpu"), lambda: kv.PagedCache(shape(quant_group=16), device="cuda:0"),
           lambda: kv.PagedCache(shape(), table=cnt, lens=cnt),
           lambda: c.compact([0], [1], cnt, off, cnt.long()), lambda: c.compact([0], [1], cnt.long(), off, cnt)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError):
        kv.kv_paged_fork(shape(), kv.kv_paged_cache(), [0], [1, 2], stream=0)


def test_model_quantises_as_defined():
    """The model's own pins: a group of 0 .. 15 is held exactly, halves go to even, equal channels have step 0."""
    x = np.tile(np.arange(32.0) % 16, (1, 1))
    v, s, m = pg.quantise(x, 32)
    assert np.array_equal(v, x) and (s == 1).all() and (m == 0).all()
    y = np.where(np.arange(32) == 31, 15.0, 0.0)[None]
    y[0, :4] = [0.5, 1.5, 2.5, 14.5]
    assert pg.quantise(y, 32)[0][0, :4].tolist() == [0, 2, 2, 14]
    v, s, _ = pg.quantise(np.full((1, 32), -2.25), 32)
    assert (v == -2.25).all() and (s == 0).all()
    z = np.ones((1, 64))
    z[0, 40] = np.inf
    v = pg.quantise(z, 32)[0]
    assert (v[0, :32] == 1).all() and np.isnan(v[0, 32:]).all()
    rng = np.random.default_rng(0)
    x = rng.normal(size=(50, 128))
    v, s, _ = pg.quantise(x, 64)  # within half a step, and what the rounding of the step loses at the top
    assert (np.abs(v - x) <= s * (0.5 + 15 * 2.0 ** -8) + 2.0 ** -8 * np.abs(x)).all()


def test_model_allocator_takes_lowest_pages_in_order():
    sh = shape(n_seqs=3, n_layers=1, n_kv_heads=1, n_pages=6, max_pages=4, page_tokens=16)
    m = pg.Model(sh)
    k = lambda n: np.zeros((n, 128))  # noqa: E731
    m.append([0, 1], [k(17), k(16)], [k(17), k(16)])
    assert m.lists == [[0, 1], [2], []]
    m.fork([0], [2])
    assert m.lists[2] == [0, 3] and m.ref.tolist() == [2, 1, 1, 1, 0, 0]
    m.free([0])
    assert m.ref.tolist() == [1, 0, 1, 1, 0, 0]
    m.compact([2], [2], [np.arange(17)])
    assert m.lists[2] == [1, 4] and m.ref.tolist() == [0, 1, 1, 0, 1, 0]
