"""A model of the paged 4-bit cache in numpy, float64: quantisation from its
definition, the page allocator as a set of numbers, rows as lists of the
values they hold, attention as a plain softmax. It shares no code with the
library; tests compare values, page lists, counts and outputs with it."""
import math

import numpy as np
import torch

import kv_cache_compression_layer_b200 as kv

DT = {kv.KV_BF16: torch.bfloat16, kv.KV_F32: torch.float32}


def bf16(x):
    """float64 -> the nearest bf16 of its float32, as float64."""
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.float32))).to(torch.bfloat16).double().numpy()


def rounded(x, dtype):
    """float64 -> dtype, rounded once (torch and numpy pass through float32, which rounds a bf16 twice where a base far
    below the step decides a half: m = 9e-10, c s = a half of bf16's last place): to float32 with what is left over
    kept in the last bit, then to bf16."""
    f = x.astype(np.float32)
    if dtype == torch.bfloat16:
        rest = np.isfinite(x) & (f.astype(np.float64) != x)
        f = np.where(rest & (np.abs(f.astype(np.float64)) > np.abs(x)), np.nextafter(f, np.float32(0)), f)
        f = np.where(rest, (f.view(np.uint32) | 1).view(np.float32), f)
    return torch.from_numpy(np.ascontiguousarray(f)).to(dtype)


def quantise(x, qg):
    """x [n, d] float64 -> values held [n, d], steps and bases spread over the channels [n, d]."""
    n, d = x.shape
    g = x.reshape(n, d // qg, qg)
    with np.errstate(all="ignore"):
        m = bf16(g.min(-1))
        s = np.where(g.max(-1) > m, bf16(np.float32((g.max(-1) - m) / 15.0)), 0.0)
        q = np.where(s[..., None] > 0, (g - m[..., None]) / np.where(s > 0, s, 1.0)[..., None], 0.0)
        c = np.clip(np.rint(q), 0, 15)
        v = m[..., None] + c * s[..., None]
    bad = ~np.isfinite(g).all(-1)
    v[bad] = np.nan
    s, m = np.where(bad, np.nan, s), np.where(bad, np.nan, m)
    full = lambda a: np.repeat(a, qg, axis=-1).reshape(n, d)  # noqa: E731
    return v.reshape(n, d), full(s), full(m)


class Model:
    def __init__(self, sh):
        self.sh = sh
        self.rps = sh.n_layers * sh.n_kv_heads
        self.rows = sh.n_seqs * self.rps
        self.lists = [[] for _ in range(self.rows)]
        self.len = [0] * self.rows
        d = sh.head_dim
        self.K = [np.zeros((0, 3, d)) for _ in range(self.rows)]  # value, step, base
        self.V = [np.zeros((0, 3, d)) for _ in range(self.rows)]
        self.ref = np.zeros(sh.n_pages, np.int64)
        self.status = 0

    def call_rows(self, seqs, layers=None):
        l0, nl = layers or (0, self.sh.n_layers)
        H = self.sh.n_kv_heads
        return [(s * self.sh.n_layers + l) * H + h for s in seqs for l in range(l0, l0 + nl) for h in range(H)]

    def _plan(self, needs):
        """Pages for each entry of needs (None: refused already), lowest free ones in order."""
        free = np.nonzero(self.ref == 0)[0]
        at, out = 0, []
        for n in needs:
            if n is None:
                out.append(None)
                continue
            if n and at + n > len(free):
                self.status |= kv.KV_DEV_PAGES
                out.append(None)
            else:
                out.append([int(p) for p in free[at:at + n]])
            at += n
        for pages in out:
            for p in pages or []:
                self.ref[p] = 1
        return out

    def pages_of(self, n):
        return -(-n // self.sh.page_tokens)

    def append(self, rows, Ks, Vs):
        """Ks, Vs: per call row [n, d] float64."""
        needs = []
        for r, k in zip(rows, Ks):
            if self.len[r] + len(k) > self.sh.max_pages * self.sh.page_tokens:
                self.status |= kv.KV_DEV_CAPACITY
                needs.append(None)
            else:
                needs.append(self.pages_of(self.len[r] + len(k)) - len(self.lists[r]))
        for r, k, v, pages in zip(rows, Ks, Vs, self._plan(needs)):
            if pages is None:
                continue
            self.lists[r] = self.lists[r] + pages
            self.len[r] += len(k)
            self.K[r] = np.concatenate([self.K[r], np.stack(quantise(k, self.sh.quant_group), 1)])
            self.V[r] = np.concatenate([self.V[r], np.stack(quantise(v, self.sh.quant_group), 1)])

    def _refuse(self, src_model, rs, rd, n, in_place=False):
        if self.len[rd] and not (in_place and rs == rd):
            self.status |= kv.KV_DEV_BUSY
            return True
        if n > self.sh.max_pages * self.sh.page_tokens:
            self.status |= kv.KV_DEV_CAPACITY
            return True
        return False

    def fork(self, src, dst):
        pairs = list(zip(self.call_rows(src), self.call_rows(dst)))
        needs = [None if self._refuse(self, a, b, self.len[a]) else int(self.len[a] % self.sh.page_tokens > 0)
                 for a, b in pairs]
        for (a, b), pages in zip(pairs, self._plan(needs)):
            if pages is None:
                continue
            full = self.len[a] // self.sh.page_tokens
            self.lists[b] = self.lists[a][:full] + pages
            for p in self.lists[a][:full]:
                self.ref[p] += 1
            self.len[b], self.K[b], self.V[b] = self.len[a], self.K[a], self.V[a]

    def copy_to(self, other, src, dst):
        pairs = list(zip(self.call_rows(src), other.call_rows(dst)))
        needs = [None if other._refuse(self, a, b, self.len[a]) else self.pages_of(self.len[a]) for a, b in pairs]
        for (a, b), pages in zip(pairs, other._plan(needs)):
            if pages is not None:
                other.lists[b], other.len[b], other.K[b], other.V[b] = pages, self.len[a], self.K[a], self.V[a]

    def compact(self, src, dst, keeps):
        """keeps: per call row the positions to keep."""
        pairs = list(zip(self.call_rows(src), self.call_rows(dst)))
        needs = [None if self._refuse(self, a, b, len(k), True) else self.pages_of(len(k))
                 for (a, b), k in zip(pairs, keeps)]
        done = []
        for (a, b), k, pages in zip(pairs, keeps, self._plan(needs)):
            if pages is None:
                continue
            k = np.asarray(k, np.int64)
            ok = (k >= 0) & (k < self.len[a])
            if not ok.all():
                self.status |= kv.KV_DEV_RANGE
            rows = []
            for x in (self.K[a], self.V[a]):
                y = np.zeros((len(k), 3, self.sh.head_dim))
                y[ok] = x[k[ok]]
                rows.append(y)
            done.append((a, b, pages, rows))
        for a, b, pages, rows in done:
            if a == b:
                for p in self.lists[a]:
                    self.ref[p] -= 1
            self.lists[b], self.len[b] = pages, len(rows[0])
            self.K[b], self.V[b] = rows

    def free(self, seqs):
        for r in self.call_rows(seqs):
            for p in self.lists[r]:
                self.ref[p] -= 1
            self.lists[r], self.len[r] = [], 0
            self.K[r], self.V[r] = self.K[r][:0], self.V[r][:0]

    # -- comparison with a PagedCache
    def check(self, cache, values=True):
        torch.cuda.synchronize()
        np.testing.assert_array_equal(cache.lens.cpu().numpy(), self.len)
        ref = cache.ref.cpu().numpy()
        np.testing.assert_array_equal(ref, self.ref)
        bits = cache.free_bits.cpu().numpy().view(np.uint32)
        free = np.unpackbits(bits.view(np.uint8), bitorder="little")
        np.testing.assert_array_equal(free[: self.sh.n_pages], (self.ref == 0).astype(np.uint8))
        assert not free[self.sh.n_pages:].any()
        table = cache.table.cpu().numpy().reshape(self.rows, -1)
        for r in range(self.rows):
            assert table[r, : len(self.lists[r])].tolist() == self.lists[r], r
        assert int(cache.status.cpu()[0]) == self.status
        if values:
            for s0 in range(0, self.sh.n_seqs, kv.KV_MAX_SEQ):
                self.check_values(cache, list(range(s0, min(self.sh.n_seqs, s0 + kv.KV_MAX_SEQ))))

    def check_values(self, cache, seqs, layers=None, spare=2):
        rows = self.call_rows(seqs, layers)
        dev, dt = cache.device, DT[self.sh.dtype]
        off = np.concatenate([[0], np.cumsum([self.len[r] + spare for r in rows])])
        K = torch.full((int(off[-1]) + 3, self.sh.head_dim), 7.0, dtype=dt, device=dev)
        V = torch.full_like(K, 9.0)
        cache.load(seqs, K, V, torch.from_numpy(off).to(dev), layers=layers)
        want = [torch.full_like(K, 7.0).cpu(), torch.full_like(K, 9.0).cpu()]
        for r, o in zip(rows, off):
            for w, x in zip(want, (self.K[r], self.V[r])):
                w[int(o):int(o) + self.len[r]] = rounded(x[:, 0], dt)
        # c s is exact, so m + c s is rounded once
        for w, got in zip(want, (K, V)):
            torch.testing.assert_close(got.cpu(), w, rtol=0, atol=0, equal_nan=True)

    def attention(self, q, row, n_q):
        """out, lse and the bounds of their errors for q [n_q * g, d] (float64) of a row.

        The library's logits: q scaled by a power of two to fp16 (f32: in two parts, 2^-22 of it left over) times
        codes is exact, the sums over d channels run in float32, and the base (f32: and 8 steps) times the sum of q's
        channels is added: a logit is off by at most (d + 16) 2^-23 sum |q| (16 s + |m|) / sqrt d. For bf16 the codes
        are subnormals, c 2^-24, whose products count as 2^-14 times q in the matrix unit's alignment: of each of the
        d products and d / 16 running sums what is below 2^-25 of that, 2^-15 s max |q|, may be lost. E is the sum. A
        probability is then off by a factor within 2 E + 2^-20 (exp2 and the sum). For bf16 the products p s are
        rounded to fp16: 2^-11 of a term 15 p s at most, or 2^-30 of the largest step (half a last place of the
        smallest fp16, where the largest step has p s = 2^5 at least) times a code of 15, for each of n keys; and of
        the 17 terms of 16 keys 2^-15 of the largest p s each is lost, 17 / 16 2^-11 of the sum of p s. Sums over n
        keys add a rounding each 16 keys, of terms up to 16 s + |m|. The result is rounded once to its type."""
        sh, g, d = self.sh, self.sh.group, self.sh.head_dim
        f32 = sh.dtype == kv.KV_F32
        out, lse = np.zeros(q.shape), np.full(len(q), -np.inf)
        tol, tol_lse = np.full(q.shape, 0.0), np.zeros(len(q))
        K, V = self.K[row], self.V[row]
        for i in range(len(q)):
            n = self.len[row] - n_q + 1 + i // g
            if n <= 0:
                continue
            k, v = K[:n], V[:n]
            x = k[:, 0] @ q[i] / math.sqrt(d)
            mx = x.max()
            p = np.exp(x - mx)
            z = p.sum()
            out[i] = p @ v[:, 0] / z
            lse[i] = mx + math.log(z)
            E = ((d + 16) * 2.0 ** -23 * (16 * k[:, 1] + np.abs(k[:, 2])) @ np.abs(q[i]) / math.sqrt(d)).max()
            if not f32:
                E += 17 / 16 * d * 2.0 ** -15 * np.abs(q[i]).max() * k[:, 1].max() / math.sqrt(d)
            top = np.abs(v[:, 0]).max(0)
            rel = 2 * E + 2.0 ** -20
            acc = (n / 16 + 24) * 2.0 ** -23 * ((16 * v[:, 1] + np.abs(v[:, 2])).max(0))
            tol[i] = 2 * rel * top + acc
            if not f32:
                tol[i] += (15 + 17 / 16) * 2.0 ** -11 * v[:, 1].max(0) + n * 15 * 2.0 ** -30 * v[:, 1].max()
            tol[i] += (2.0 ** -24 if f32 else 2.0 ** -8) * (np.abs(out[i]) + tol[i])
            tol_lse[i] = E + 2.0 ** -20 + 2.0 ** -22 * abs(lse[i])
        return out, lse, tol, tol_lse

    def check_attention(self, q, out, lse, seqs, n_q, layers=None, rows_at=None):
        """q, out [call rows, n_q * g, d] torch, lse [call rows, n_q * g] or None."""
        Q, O = q.double().cpu().numpy(), out.double().cpu().numpy()
        Z = None if lse is None else lse.double().cpu().numpy()
        for i, r in enumerate(self.call_rows(seqs, layers)):
            if rows_at is not None and i not in rows_at:
                continue
            o, z, tol, tol_z = self.attention(Q[i].reshape(-1, self.sh.head_dim), r, n_q)
            got = O[i].reshape(o.shape)
            err = np.abs(got - o)
            assert (err <= tol).all(), (i, r, float((err - tol).max()), np.unravel_index((err - tol).argmax(), err.shape))
            if Z is not None:
                zz = Z[i].reshape(-1)
                np.testing.assert_array_equal(np.isneginf(zz), np.isneginf(z))
                f = np.isfinite(z)
                assert (np.abs(zz[f] - z[f]) <= tol_z[f]).all(), (i, r)


def tokens(rng, n, d, dtype):
    """K-like and V-like rows: channels of their own offset and size; exact in dtype. float64."""
    off, size = rng.normal(size=d), 0.3 + rng.random(d)
    K = rng.normal(size=(n, d)) * size + off
    V = rng.normal(size=(n, d))
    if dtype == kv.KV_BF16:
        return bf16(K), bf16(V)
    return K.astype(np.float32).astype(np.float64), V.astype(np.float32).astype(np.float64)


def up(x, dtype, dev):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.float32)).to(dev, DT[dtype])


def fill(cache, model, counts, rng):
    """Appends counts[r] random tokens to every row of the cache and the model (all sequences, calls of 64)."""
    sh = cache.shape
    for s0 in range(0, sh.n_seqs, kv.KV_MAX_SEQ):
        seqs = list(range(s0, min(sh.n_seqs, s0 + kv.KV_MAX_SEQ)))
        rows = model.call_rows(seqs)
        n = [int(counts[r]) for r in rows]
        K, V = tokens(rng, sum(n), sh.head_dim, sh.dtype)
        o = np.concatenate([[0], np.cumsum(n)])
        model.append(rows, [K[o[i]:o[i + 1]] for i in range(len(n))], [V[o[i]:o[i + 1]] for i in range(len(n))])
        if not sum(n):
            continue
        dev = cache.device
        cache.append(seqs, up(K, sh.dtype, dev), up(V, sh.dtype, dev),
                     count=torch.tensor(n, dtype=torch.int32, device=dev),
                     src_off=torch.from_numpy(o[:-1].copy()).to(dev))


def make(n_seqs=3, n_layers=2, heads=2, group=3, d=128, dtype=kv.KV_BF16, qg=64, page=64, n_pages=None, max_pages=8,
         cls=None):
    n_pages = n_seqs * n_layers * heads * max_pages if n_pages is None else n_pages
    sh = kv.make_paged_shape(n_seqs, n_layers, heads, group, d, dtype, n_pages, max_pages, qg, page)
    return kv.PagedCache(sh, device="cuda:0"), Model(sh)
