"""kv_paged_attn keeps its sums in float32: long even rows, where what each
addition loses could pile up on one side, and rows whose channel groups or
tokens lie many powers of two apart, where a scale shared between them would
cost the small ones their bits. Against float64 over the values held, within bounds that
count float32 roundings, the output's, and for bf16 that of weights to fp16."""
import math

import numpy as np
import pytest
import torch

import kv_cache_compression_layer_b200 as kv
from tests import _paged as pg

pytestmark = pytest.mark.gpu

CHAIN = 64  # products that are added up in the matrix unit, at most, before the sum leaves it


def strict(m, q, row, n_q=1):
    """out, lse and bounds of their errors for q [n_q * g, d] (float64) of a row.

    Logits: the products of q's channels and codes are exact; sums over d channels, and a group's base (with 8 steps)
    times the sum of its channels, round in float32, relative to the terms of their own group: a logit of key j is off
    by at most E_j = (d + 16) 2^-23 sum_c |q_c| (16 s_jc + |m_jc|) / sqrt d. A weight p_j is off by a factor within
    2 E + 2^-20 (exp2, the sum). Output: a channel's terms are p_j (16 s_jc + |m_jc|); their sums round 2^-23 of the
    sum of magnitudes W_c for each of a warp's products that follow each other (n / 64, CHAIN at most) and for each of
    the sums of CHAIN of them, 2^-24 of it for each of a lane's n / 32 additions of bases, and 16 and one for each tile
    more where sums are rescaled and joined. A bf16 call rounds weights times steps to fp16: 2^-11 of them
    times |c - 8| <= 8 steps, 2^-12 of the terms, and 2^-22 of the largest weight's step or more, 8 times, for each key
    (or to two bf16, less than that). A weight below 2^-126 may be lost: 2^-118 of the largest term for each key
    (weights are below 2^8 and the largest is 1 or more)."""
    sh, g, d = m.sh, m.sh.group, m.sh.head_dim
    f32 = sh.dtype == kv.KV_F32
    K, V = m.K[row], m.V[row]
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    lse, tol_lse = np.full(len(q), -np.inf), np.zeros(len(q))
    for i in range(len(q)):
        n = m.len[row] - n_q + 1 + i // g
        if n <= 0:
            continue
        k, v = K[:n], V[:n]
        x = k[:, 0] @ q[i] / math.sqrt(d)
        p = np.exp(x - x.max())
        z = p.sum()
        out[i], lse[i] = p @ v[:, 0] / z, x.max() + math.log(z)
        E = (d + 16) * 2.0 ** -23 * ((16 * k[:, 1] + np.abs(k[:, 2])) @ np.abs(q[i])) / math.sqrt(d)
        rel = 2 * E + 2.0 ** -20
        mag = 16 * v[:, 1] + np.abs(v[:, 2])
        W = p @ mag / z
        c = (min(CHAIN, n / 64 + 1) + n / 64 / CHAIN + 16 + n / 128) * 2.0 ** -23 + n / 32 * 2.0 ** -24
        c += 0 if f32 else 2.0 ** -12
        tol[i] = (p * rel) @ mag / z + (p @ rel / z) * np.abs(out[i]) + c * W + n * 2.0 ** -118 * mag.max(0)
        tol[i] += 0 if f32 else n * 2.0 ** -19 * (p[:, None] * v[:, 1]).max(0) / z
        tol[i] += (2.0 ** -24 if f32 else 2.0 ** -8) * (np.abs(out[i]) + tol[i])
        tol_lse[i] = p @ rel / z + 2.0 ** -20 + 2.0 ** -22 * abs(lse[i])
    return out, lse, tol, tol_lse


def check(m, q, out, lse, seqs, n_q=1):
    Q, O, Z = (x.double().cpu().numpy() for x in (q, out, lse))
    for i, r in enumerate(m.call_rows(seqs)):
        o, z, tol, tol_z = strict(m, Q[i].reshape(-1, m.sh.head_dim), r, n_q)
        err = np.abs(O[i].reshape(o.shape) - o)
        assert (err <= tol).all(), (i, float((err / tol).max()), np.unravel_index((err / tol).argmax(), err.shape))
        assert (np.abs(Z[i].reshape(-1) - z) <= tol_z).all(), i


@pytest.mark.parametrize("spread", ["even", "one_sided"])
@pytest.mark.parametrize("g", [1, 16])
@pytest.mark.parametrize("dtype", [kv.KV_BF16, kv.KV_F32])
def test_long_even_rows(dtype, g, spread):
    """896 rows of 32768 keys, whole rows in one block, with next to the same weight for each key: outputs are means
    of many values that cancel, so what sums lose would show. one_sided: a channel far below the others puts their
    codes next to 15, so that sums of codes grow all along the row.

    Queries have one channel, so a weight is off by a factor within rel = 2 (d + 16) 2^-23 |q| (16 s + |m|) / sqrt d +
    2^-20 with that channel's s and m. A sum of CHAIN products of 16 keys each loses 2^-23 of what it has reached at
    each, CHAIN / 2 2^-23 of 8 s a key on average; sums of those and of bases (a lane adds n / 32) as in strict().

    The mean over all outputs of the error: the matrix unit cuts a sum's last bits off, to one side, 2^-24 of what it has
    reached on average (its last place is 2^-23 to 2^-24 of it); all else is rounded to the nearest and has no sign: 8 /
    sqrt(count) of the bounds above."""
    rng = np.random.default_rng(23)
    n, R, d = 32768, 896, 128
    base, m = pg.make(n_seqs=1, n_layers=1, heads=8, group=1, dtype=dtype, max_pages=512)
    K, V = pg.tokens(rng, 8 * n, d, dtype)
    if spread == "one_sided":
        V[:, [5, 77]] = -10.0
    rows = m.call_rows([0])
    K, V = K.reshape(8, n, d), V.reshape(8, n, d)
    m.append(rows, K, V)
    base.append([0], pg.up(K, dtype, base.device), pg.up(V, dtype, base.device))
    pages = torch.randint(0, 4096, (R, n // 64), generator=torch.Generator().manual_seed(1)).to(base.device)
    sh = kv.make_paged_shape(64, 1, 14, g, d, dtype, 4096, n // 64, 64, 64)
    cache = kv.PagedCache(sh, pages=base.pages, table=pages.to(torch.int32),
                          lens=torch.full((R,), n, dtype=torch.int32, device=base.device))
    q = torch.zeros(R, g, d, dtype=pg.DT[dtype], device=base.device)
    q[:, :, 9] = 0.05 * (1 + torch.rand(R, g, generator=torch.Generator().manual_seed(2))).to(q)
    lse = torch.empty(R, g, device=base.device)
    out = cache.attend(list(range(64)), q, lse=lse).double()
    # by page number: the keys' channel 9, values, steps and centres
    k9, val = (torch.zeros(4096, 64, *x, dtype=torch.float64, device=base.device) for x in ((), (d,)))
    s, mid = (torch.zeros(4096, d, dtype=torch.float64, device=base.device) for _ in range(2))
    e9 = 0.0
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(base.device)  # noqa: E731
    for r in rows:
        at = up(np.asarray(m.lists[r]))
        x = m.V[r].reshape(n // 64, 64, 3, d)
        k9[at], val[at] = up(m.K[r].reshape(n // 64, 64, 3, d)[:, :, 0, 9]), up(x[:, :, 0])
        s[at], mid[at] = up(x[:, :, 1].sum(1)), up(np.abs(x[:, :, 2] + 8 * x[:, :, 1]).sum(1))
        e9 = max(e9, (16 * m.K[r][:, 1, 9] + np.abs(m.K[r][:, 2, 9])).max())
    rel = 2 * (d + 16) * 2.0 ** -23 * 0.1 * e9 / math.sqrt(d) + 2.0 ** -20
    half = 2.0 ** -24 if dtype == kv.KV_F32 else 2.0 ** -8
    short = 0.0 if dtype == kv.KV_F32 else 2.0 ** -12
    err, room, free, cut = [], [], [], []
    for r in range(R):
        x = (q[r, :, 9].double()[:, None] * k9[pages[r]].flatten()) / math.sqrt(d)
        want = torch.softmax(x, 1) @ val[pages[r]].flatten(0, 1)
        a, b = s[pages[r]].sum(0) / n, mid[pages[r]].sum(0) / n
        spare = 1.02 * ((CHAIN / 2 + n / 64 / CHAIN + 16) * 2.0 ** -23 * 8 * a + (n / 64 + 16) * 2.0 ** -24 * b
                        + rel * (8 * a + b))  # weights are within 2 % of each other
        err.append(out[r] - want)
        free.append(short * 16 * a + half * want.abs())
        room.append(spare.expand_as(want))
        cut.append(((CHAIN / 2 + 8) * 2.0 ** -24 * 8 * a).expand_as(want))
        assert (lse[r].double() - torch.logsumexp(x, 1)).abs().max() <= rel + 2.0 ** -20 + 2.0 ** -22 * 11
    err, room, free, cut = (torch.stack(x) for x in (err, room, free, cut))
    worst = (err.abs() / (room + free * (1 + half) + half * room)).max()
    assert worst <= 1, float(worst)
    mean, may = err.mean().abs(), (cut + 8 / math.sqrt(R * d) * (room + free)).mean()
    assert mean <= may, (float(mean), float(may))


def spread_rows(rng, n, d, qg, power):
    """K, V [n, d] and a factor of q's channels: groups whose sizes differ by 2^power in K and V; q undoes K's, so
    that every group counts alike in the logits."""
    up = np.repeat(np.where(np.arange(d // qg) % 2, 2.0 ** power, 1.0), qg)
    K, V = pg.tokens(rng, n, d, kv.KV_BF16)
    return K * up, V * up[::-1], 1 / up


@pytest.mark.parametrize("power", [10, 16, 24, 40])
@pytest.mark.parametrize("even", [False, True])
@pytest.mark.parametrize("d,qg,g,n_q", [(128, 64, 3, 1), (128, 32, 8, 2), (64, 32, 5, 1)])
@pytest.mark.parametrize("dtype", [kv.KV_BF16, kv.KV_F32])
def test_groups_far_apart(dtype, d, qg, g, n_q, even, power):
    """Groups of channels 2^power apart in K, V and q: the small ones keep their bits. even: q = 0."""
    rng = np.random.default_rng(24 + power)
    cache, m = pg.make(n_seqs=1, n_layers=1, heads=3, group=g, d=d, qg=qg, dtype=dtype, max_pages=8)
    n = 333
    K, V, f = spread_rows(rng, 3 * n, d, qg, power)
    m.append([0, 1, 2], K.reshape(3, n, d), V.reshape(3, n, d))
    cache.append([0], pg.up(K, dtype, cache.device).view(3, n, d), pg.up(V, dtype, cache.device).view(3, n, d))
    q = pg.up((0.0 if even else 0.5) * rng.normal(size=(3, n_q * g, d)) * f, dtype, cache.device)
    out, lse = torch.empty_like(q), torch.empty(3, n_q * g, device=cache.device)
    cache.attend([0], q, out, lse=lse, n_q=n_q)
    check(m, q, out, lse, [0], n_q)


@pytest.mark.parametrize("place", ["first", "last", "among"])
@pytest.mark.parametrize("power", [10, 16, 24, 40, 80])
@pytest.mark.parametrize("dtype", [kv.KV_BF16, kv.KV_F32])
def test_a_huge_value_of_no_weight(dtype, power, place):
    """A token whose V is 2^power times the others' and whose weight is next to nothing does not coarsen the others."""
    rng = np.random.default_rng(25 + power)
    cache, m = pg.make(n_seqs=1, n_layers=1, heads=2, group=4, dtype=dtype, max_pages=8)
    n = 400
    K, V = (x.reshape(2, n, 128) for x in pg.tokens(rng, 2 * n, 128, kv.KV_BF16))
    at = {"first": 0, "last": n - 1, "among": 150}[place]
    K[:] = 0.0  # the others' weights are 1
    K[:, at, 70] = -960.0  # a logit of -85 or less, a weight of 2^-122
    V[:, at] *= 2.0 ** power
    m.append([0, 1], K, V)
    cache.append([0], pg.up(K, dtype, cache.device), pg.up(V, dtype, cache.device))
    q = rng.normal(size=(2, 4, 128))
    q[:, :, 70] = 1.0
    q = pg.up(q, dtype, cache.device)
    out, lse = torch.empty_like(q), torch.empty(2, 4, device=cache.device)
    cache.attend([0], q, out, lse=lse)
    check(m, q, out, lse, [0])


@pytest.mark.parametrize("d,qg,g", [(128, 64, 8), (128, 32, 3), (64, 64, 16)])
@pytest.mark.parametrize("at", [0, 17, 130, 200, 258, 590, 700])
def test_steps_that_part_along_the_row(d, qg, g, at):
    """Steps that become 2^9 to 2^14 times smaller, larger or 0 from a token on, in tiles that every query sees in full
    and at the end; whichever tokens a warp has had before, their sums go on."""
    rng = np.random.default_rng(27 + at)
    cache, m = pg.make(n_seqs=1, n_layers=1, heads=6, group=g, d=d, qg=qg, max_pages=16)
    n = 777
    K, V = (x.reshape(6, n, d) for x in pg.tokens(rng, 6 * n, d, kv.KV_BF16))
    for r, f in enumerate((2.0 ** -9, 2.0 ** -14, 2.0 ** 9, 2.0 ** 14, 0.0, 1.0)):
        V[r, at:at + 300, :qg] *= f
    V[5, at, 3] = 3e4
    m.append(list(range(6)), K, V)
    cache.append([0], pg.up(K, kv.KV_BF16, cache.device), pg.up(V, kv.KV_BF16, cache.device))
    q = pg.up(0.3 * rng.normal(size=(6, g, d)), kv.KV_BF16, cache.device)
    out, lse = torch.empty_like(q), torch.empty(6, g, device=cache.device)
    cache.attend([0], q, out, lse=lse)
    check(m, q, out, lse, [0])


@pytest.mark.parametrize("dtype", [kv.KV_BF16, kv.KV_F32])
@pytest.mark.parametrize("g,n_q", [(8, 1), (5, 3), (1, 1)])
def test_ordinary_rows(dtype, g, n_q):
    """Rows of some thousands of keys with queries near one of them."""
    rng = np.random.default_rng(26)
    cache, m = pg.make(n_seqs=1, n_layers=1, heads=4, group=g, dtype=dtype, max_pages=80)
    pg.fill(cache, m, [5000, 3333, 130, 1], rng)
    q = 0.3 * rng.normal(size=(4, n_q * g, 128))
    for r in range(4):
        q[r] += 0.5 * m.K[r][rng.integers(0, m.len[r], n_q * g), 0]
    q = pg.up(q, dtype, cache.device)
    out, lse = torch.empty_like(q), torch.empty(4, n_q * g, device=cache.device)
    cache.attend([0], q, out, lse=lse, n_q=n_q)
    Z = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(Z[3]), [i // g < n_q - 1 for i in range(n_q * g)])
    Q, O = q.double().cpu().numpy(), out.double().cpu().numpy()
    for r in range(4):
        o, z, tol, tol_z = strict(m, Q[r], r, n_q)
        seen = np.isfinite(z)
        assert (np.abs(O[r] - o) <= tol).all() and (np.abs(Z[r][seen] - z[seen]) <= tol_z[seen]).all(), r
