"""Plain implementation of the paged 8-bit KV cache in 64 bits, for the tests:
one sequence, one page, one head at a time, from the definitions."""
import math

import numpy as np
import torch

E4M3 = np.array([0.0] * 256)
for _b in range(256):
    _e, _f = (_b >> 3) & 15, _b & 7
    _x = (_f / 8) * 2.0 ** -6 if _e == 0 else (1 + _f / 8) * 2.0 ** (_e - 7)
    E4M3[_b] = math.nan if _b & 0x7F == 0x7F else (-_x if _b & 0x80 else _x)
_FINITE = [b for b in range(128) if b != 0x7F]
_GRID = np.array([E4M3[b] for b in _FINITE])


def e4m3_bytes(x):
    """Nearest e4m3 of each value (ties to the even byte), magnitudes past 448 clamped, NaN and infinities to NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.where(np.isfinite(x), np.abs(x), 0.0), 448.0)
    hi = np.searchsorted(_GRID, a).clip(0, len(_GRID) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    b = np.array(_FINITE)[pick] | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isfinite(x), b, 0x7F).astype(np.uint8)


def scale_for(amax):
    """2^e with the least e in [-60, 60] with amax <= 448 * 2^e."""
    for e in range(-60, 61):
        if amax <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 60


class Model:
    """The cache as numpy arrays and the operations on it, in order."""

    def __init__(self, cache):
        self.page = cache.page
        for n in ("k", "v", "k_scale", "v_scale", "table", "lens", "refs"):
            setattr(self, n, getattr(cache, n).cpu().numpy().copy())

    def same_as(self, cache):
        for n in ("table", "lens", "refs", "k_scale", "v_scale", "k", "v"):
            got = getattr(cache, n).cpu().numpy()
            # scales of free pages may be NaN
            assert np.array_equal(got, getattr(self, n), equal_nan=n.endswith("scale")), f"{n} differs at {np.argwhere(got != getattr(self, n))[:4].tolist()}"

    def append(self, k, v, counts, row_idx=None):
        """k, v [layers, rows, heads, dim] as float64; counts: rows of each slot.  Returns the rows stored."""
        L, _, H, D = k.shape
        page, at, stored = self.page, 0, []
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        shared = self.refs > 1
        jobs = []
        for s, n in enumerate(counts):
            rows = list(range(at, at + n))
            at += n
            ln = int(self.lens[s])
            want = -(-(ln + n) // page)
            old = int(self.table[s, ln // page]) if ln % page else -1
            copy = n > 0 and old >= 0 and bool(shared[old])
            need = want - -(-ln // page) + int(copy)
            if n == 0 or want > self.table.shape[1] or need > len(free):
                stored.append(0)
                continue
            ids, free = free[:need], free[need:]
            first = ln // page if copy else -(-ln // page)
            self.table[s, first:first + need] = ids
            jobs.append((s, ln, old, copy, rows, ids))
            stored.append(n)
        for s, ln, old, copy, rows, ids in jobs:
            self.refs[ids] = 1
            if copy:
                self.refs[old] -= 1
            self.lens[s] = ln + len(rows)
            src = rows if row_idx is None else [int(row_idx[r]) for r in rows]
            for l in range(L):
                for h in range(H):
                    self._write(self.k[l, :, h], self.k_scale[l, :, h], s, ln, old, k[l, src, h], False)
                    self._write(self.v[l, :, h], self.v_scale[l, :, h], s, ln, old, v[l, src, h], True)
        return stored

    def _write(self, pool, scale, s, ln, old, x, transposed):
        page, done = self.page, 0
        while done < len(x):
            j, o = divmod(ln + done, page)
            n = min(page - o, len(x) - done)
            to = int(self.table[s, j])
            y = x[done:done + n]
            fin = np.abs(y[np.isfinite(y)])
            sc = scale_for(fin.max() if fin.size else 0.0)
            if o:
                sc = max(sc, float(scale[old]))
                was = pool[old].T if transposed else pool[old]
                b = was[:o].copy()
                if sc != scale[old]:
                    b = np.where(b & 0x7F == 0x7F, b, e4m3_bytes(np.nan_to_num(E4M3[b]) * (float(scale[old]) / sc)))
                    # a value that becomes zero keeps its sign
                    b = b | (was[:o] & 0x80)
                (pool[to].T if transposed else pool[to])[:o] = b
            (pool[to].T if transposed else pool[to])[o:o + n] = e4m3_bytes(y / sc)
            scale[to] = sc
            done += n

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            self.table[b] = self.table[a]
            self.lens[b] = self.lens[a]
            for p in self.table[a]:
                if p >= 0:
                    self.refs[p] += 1

    def free(self, slots, keep=None):
        for i, s in enumerate(slots):
            k = 0 if keep is None else max(int(keep[i]), 0)
            for j in range(-(-k // self.page), self.table.shape[1]):
                if self.table[s, j] >= 0:
                    self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1
            self.lens[s] = min(self.lens[s], k)

    def compact(self):
        used = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        n = len(used)
        holes = [p for p in range(n) if self.refs[p] == 0]
        for a, b in zip([p for p in used if p >= n], holes):
            for x in (self.k, self.v, self.k_scale, self.v_scale):
                x[:, b] = x[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.table[self.table == a] = b
        return n


def attention(cache, q, k, v, counts, layer=0, see=None, scale=None, first=0):
    """Output and its tolerance, float64 [rows, heads, dim].  counts: rows of
    each slot (from row `first`); see(s, r) -> visible rows of row r of slot s
    (default: 0 .. r).  k None: the cache alone.

    Tolerance, elementwise: out is rounded once to bf16 (2^-8 |o|).  The softmax
    weights are rounded to fp16 (2^-11 each, so 2^-11 sum p |V|; below 2^-14 of
    the largest at most 2^-25 each, times |V8| <= 448 and V's scale).  Scores
    are fp32 sums of head_dim products, off by at most (head_dim + 8) 2^-23 of
    the sum of their magnitudes, which moves p by that factor; the fp32 sums
    over n keys add n 2^-24.  Both act on sum p |V| and on |o| (through the
    normalisation)."""
    H, D = q.shape[1], q.shape[2]
    G = H // cache.n_kv_heads
    scale = scale or 1 / math.sqrt(D)
    kb, vb = (E4M3[x[layer].cpu().numpy()] for x in (cache.k, cache.v))
    ks, vs = (x[layer].cpu().double().numpy() for x in (cache.k_scale, cache.v_scale))
    table, lens = cache.table.cpu().numpy(), cache.lens.cpu().numpy()
    f = lambda x: None if x is None else x.cpu().double().numpy()  # noqa: E731
    q, k, v = f(q), f(k), f(v)
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    at = first
    for s, n in enumerate(counts):
        ln = int(lens[s])
        ids = table[s, :-(-ln // cache.page)]
        for h in range(cache.n_kv_heads):
            K = (kb[ids, h] * ks[ids, h, None, None]).reshape(-1, D)[:ln]
            V = np.swapaxes(vb[ids, h] * vs[ids, h, None, None], 1, 2).reshape(-1, D)[:ln]
            top = vs[ids, h].max() if ln else 0.0
            for r in range(n):
                rows = [] if k is None else [at + j for j in (range(r + 1) if see is None else see(s, r))]
                Kr = np.concatenate([K, k[rows, h]]) if rows else K
                Vr = np.concatenate([V, v[rows, h]]) if rows else V
                if not len(Kr):
                    continue
                vnew = np.abs(v[rows, h]).max() if rows else 0.0
                for g in range(G):
                    x = q[at + r, h * G + g]
                    with np.errstate(all="ignore"):
                        z = Kr @ x * scale
                        p = np.exp(z - z.max())
                        p /= p.sum()
                        o = p @ Vr
                        A = p @ np.abs(Vr)
                        dz = (D + 8) * 2.0 ** -23 * scale * (np.abs(Kr) @ np.abs(x)).max()
                        out[at + r, h * G + g] = o
                        tol[at + r, h * G + g] = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2 * dz + len(Kr) * 2.0 ** -24 + 2.0 ** -20) * (A + np.abs(o)) \
                            + len(Kr) * 2.0 ** -25 * max(448 * top, 2 * vnew)
        at += n
    return out, tol


def fill(cache, lens, seed, shared=()):
    """Sequences of the given lengths with random bytes and scales, pages dealt out in a random order; stale NaN bytes
    behind the last tokens.  shared: pairs (a, b) of slots; b names a's full pages."""
    g = np.random.default_rng(seed)
    page, order = cache.page, list(g.permutation(cache.n_pages))
    table = np.full((cache.n_seqs, cache.max_pages), -1, np.int32)
    refs = np.zeros(cache.n_pages, np.int32)
    k, v = (np.full(tuple(x.shape), 0x7F, np.uint8) for x in (cache.k, cache.v))
    ks, vs = (np.full(tuple(x.shape), np.nan, np.float32) for x in (cache.k_scale, cache.v_scale))
    share = dict((b, a) for a, b in shared)
    for s, n in enumerate(lens):
        for j in range(-(-n // page)):
            if s in share and (j + 1) * page <= min(n, lens[share[s]]):
                table[s, j] = table[share[s], j]
                refs[table[s, j]] += 1
                continue
            p = order.pop()
            table[s, j] = p
            refs[p] = 1
            m = min(page, n - j * page)
            for l in range(cache.n_layers):
                for h in range(cache.n_kv_heads):
                    x = g.standard_normal((2, m, cache.head_dim)) * np.exp(g.standard_normal((2, 1, 1)))
                    ks[l, p, h], vs[l, p, h] = scale_for(np.abs(x[0]).max()), scale_for(np.abs(x[1]).max())
                    k[l, p, h, :m] = e4m3_bytes(x[0] / ks[l, p, h])
                    v[l, p, h, :, :m] = e4m3_bytes(x[1] / vs[l, p, h]).T
    for name, a in (("k", k), ("v", v), ("k_scale", ks), ("v_scale", vs), ("table", table), ("refs", refs),
                    ("lens", np.array(lens, np.int32))):
        getattr(cache, name).copy_(torch.from_numpy(a))
