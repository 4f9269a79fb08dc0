"""Attention over the 8-bit cache with a sliding window and first tokens that stay (Kv8Cache.attention with window and sinks)
against its definition in 64 bits: a row's list of keys (cached tokens, then its visible new rows), cut to its first `sinks`
and its last `window`."""
import math

import numpy as np
import pytest

import kv8_model as M
from helpers import ensure_built
from test_gpu_kv8 import build, close, ints, normal, starts, tree_words

pytestmark = pytest.mark.gpu
ALL = 1 << 30


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import exact_decoding_gb300 as e
    return e


def model(cache, q, k, v, counts, window, sinks, see=None, scale=None, first=0):
    """Output and tolerance [rows, heads, dim], as kv8_model.attention derives it; NaN where a row sees one."""
    H, D = q.shape[1], q.shape[2]
    G = H // cache.n_kv_heads
    scale = scale or 1 / math.sqrt(D)
    kb, vb = (M.E4M3[x[0].cpu().numpy()] for x in (cache.k, cache.v))
    ks, vs = (x[0].cpu().double().numpy() for x in (cache.k_scale, cache.v_scale))
    table, lens = cache.table.cpu().numpy(), cache.lens.cpu().numpy()
    q, k, v = (None if x is None else x.cpu().double().numpy() for x in (q, k, v))
    out, tol, at = np.zeros(q.shape), np.zeros(q.shape), first
    for s, n in enumerate(counts):
        ln = int(lens[s])
        ids = table[s, :-(-ln // cache.page)]
        for h in range(cache.n_kv_heads):
            K = (kb[ids, h] * ks[ids, h, None, None]).reshape(-1, D)[:ln]
            V = np.swapaxes(vb[ids, h] * vs[ids, h, None, None], 1, 2).reshape(-1, D)[:ln]
            for r in range(n):
                rows = [] if k is None else [at + j for j in (range(r + 1) if see is None else see(s, r))]
                place = np.arange(ln + len(rows))
                kept = place[(place < sinks) | (place >= len(place) - window)]
                if not len(kept):
                    continue
                Kr = np.concatenate([K, k[rows, h]] if rows else [K])[kept]
                Vr = np.concatenate([V, v[rows, h]] if rows else [V])[kept]
                old = kept[kept < ln]
                top = vs[ids[old // cache.page], h].max() if len(old) else 0.0
                vnew = np.nanmax(np.abs(v[rows, h])) if rows else 0.0
                for g in range(G):
                    x = q[at + r, h * G + g]
                    z = Kr @ x * scale
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    with np.errstate(invalid="ignore"):
                        o, A = p @ Vr, p @ np.abs(Vr)
                    dz = (D + 8) * 2.0 ** -23 * scale * (np.abs(Kr) @ np.abs(x)).max()
                    out[at + r, h * G + g] = o
                    tol[at + r, h * G + g] = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2 * dz + len(Kr) * 2.0 ** -24 + 2.0 ** -20) * (A + np.abs(o)) \
                        + len(Kr) * 2.0 ** -25 * max(448 * top, 2 * vnew)
        at += n
    return out, tol


def same(out, want, tol):
    """close(), with NaN where the definition has NaN and nowhere else."""
    got = out.cpu().double().numpy()
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"NaN differ at {np.argwhere(np.isnan(got) != nan)[:4].tolist()}"
    bad = ~nan & ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off at {np.argwhere(bad)[:3].tolist()}: {got[bad][:3]} for {want[bad][:3]}"


CASES = [
    # hd, page, heads, kv heads, lens, rows, window, sinks
    (128, 64, 4, 4, [117], [1], 1, 0),
    (128, 64, 4, 4, [117], [1], 64, 4),
    (128, 32, 8, 2, [0], [1], 5, 3),
    (128, 64, 8, 1, [1000], [1], 129, 0),
    (128, 128, 16, 2, [1500, 3, 0, 129, 700], [1] * 5, 128, 1),
    (64, 32, 6, 2, [5, 300, 33, 129, 0], [1, 2, 3, 1, 4], 20, 4),
    (64, 128, 3, 3, [128, 127, 129, 500], [1, 0, 5, 2], 3, 500),          # every first token stays
    (128, 64, 8, 1, [4100], [1], 3000, 4),                              # split over many workers, joined
    (128, 32, 5, 5, [70], [17], 8, 0),                                  # rows whose windows begin among the new rows
    (128, 32, 12, 2, [40, 90], [70, 1], 33, 40),
    (64, 64, 2, 2, [130], [130], 64, 10),
    (128, 64, 4, 2, [300, 10], [129, 3], 200, 64),
    (128, 64, 32, 1, [1000, 40], [9, 1], 257, 5),
    (64, 32, 8, 8, [31], [256], 100, 31),
    (128, 64, 8, 2, [0, 5], [200, 150], 40, 7),                         # the first tokens are new rows
    (128, 128, 8, 8, [2000], [40], 1, 0),                               # each row sees itself
    (128, 64, 16, 4, [5000, 3000], [64, 64], 1024, 130),
    (128, 64, 4, 4, [500], [1], ALL, 0),
    (128, 32, 4, 1, [600], [40], 700, ALL),
    (64, 64, 6, 3, [2100, 0, 64, 65], [1, 33, 33, 33], 64, 64),
    (128, 128, 8, 1, [9000], [20], 4096, 200),
]


@pytest.mark.parametrize("hd,page,heads,kv,lens,rows,window,sinks", CASES)
def test_windows(lib, hd, page, heads, kv, lens, rows, window, sinks):
    cache = build(lib, lens, hd, page, kv, seed=len(lens) + heads)
    n = sum(rows)
    q, k, v = normal((n, heads, hd), 1, 1.5), normal((n, kv, hd), 2), normal((n, kv, hd), 3)
    want = model(cache, q, k, v, rows, window, sinks)
    for hints in (dict(max_rows=max(rows), max_len=max(lens)), {}, dict(max_rows=1, max_len=1)):
        out = cache.attention(q, k, v, row_start=starts(rows), window=window, sinks=sinks, **hints)
        cache.status()
        close(out, *want)


@pytest.mark.parametrize("lens,rows,window,sinks", [([0, 90, 64], [2, 1, 3], 10, 0), ([200, 0], [3, 40], 64, 3), ([2000], [1], 100, 100)])
def test_over_the_cache_alone(lib, lens, rows, window, sinks):
    """Without new keys the window is the last cached tokens; a row of an empty sequence sees nothing and gives 0."""
    import torch
    cache = build(lib, lens, 128, 32, 2)
    q = normal((sum(rows) + 3, 6, 128), 4)
    out = torch.full_like(q, 7.0)
    cache.attention(q, row_start=starts(rows, 1), out=out, window=window, sinks=sinks)
    cache.status()
    want, tol = model(cache, q, None, None, rows, window, sinks, first=1)
    close(out[1:-2], want[1:-2], tol[1:-2])
    assert torch.all(out[0] == 7) and torch.all(out[-2:] == 7)         # rows of no sequence stay


@pytest.mark.parametrize("hd,heads,kv,N,W,G,length,window,sinks", [
    (128, 4, 4, 5, 15, 15, 300, 64, 4), (64, 4, 2, 4, 5, 3, 33, 3, 1), (128, 8, 1, 3, 4, 4, 1100, 500, 0), (128, 8, 8, 5, 5, 5, 0, 2, 1),
    (64, 2, 2, 5, 15, 15, 2, 4, 3), (128, 8, 2, 6, 10, 5, 700, 129, 130)])
def test_under_the_step_mask(lib, hd, heads, kv, N, W, G, length, window, sinks):
    """A step's rows: each branch's ancestors count towards its window."""
    import torch
    _, vis, _ = lib.la_step_tables(N, W, G)
    rows = vis.shape[0]
    see = [[j for j in range(rows) if (int(vis[r, j // 32]) >> (j % 32)) & 1] for r in range(rows)]
    cache = build(lib, [length], hd, 64, kv)
    q, k, v = normal((rows, heads, hd), 5, 1.5), normal((rows, kv, hd), 6), normal((rows, kv, hd), 7)
    words = vis.view(np.int32).copy()
    words[:, 7] |= np.int32(-2 ** 31) if rows < 255 else np.int32(0)      # a bit past the rows means nothing
    for hint in (rows, 0, 1):
        out = cache.attention(q, k, v, row_start=starts([rows]), vis=torch.from_numpy(words).cuda(), window=window, sinks=sinks, max_rows=hint)
        cache.status()
        close(out, *model(cache, q, k, v, [rows], window, sinks, see=lambda s, r: see[r]))


@pytest.mark.parametrize("heads,rows", [(4, 1), (2, 9), (2, 40), (8, 150)])
@pytest.mark.parametrize("page", [32, 128])
def test_unseen_values_do_not_leak(lib, heads, rows, page):
    """NaN in cached tokens before, at and behind the windows' beginnings, and in new rows that have left the window."""
    import torch
    length, window, sinks = 700, 300, 5
    cache = build(lib, [length, 40], 128, page, 2, seed=3)
    counts = [rows, 2]
    n = sum(counts)
    q, k, v = normal((n, heads, 128), 1), normal((n, 2, 128), 2), normal((n, 2, 128), 3)
    table = cache.table.cpu().numpy()
    # places in the first sequence's cache: before all windows, inside the earliest alone, inside some, a first token, the one behind those
    for i, place in enumerate((6, 390, 401, 402, 405, 420, 2, 5)):
        if place == 2 and rows == 9:
            continue                                          # with it every row has NaN: once is enough
        page_no, o = int(table[0, place // page]), place % page
        cache.v[0, page_no, 0, 3 + i, o] = 0x7F
        if i % 2 == 0:
            cache.v[0, page_no, 1, 64 + i, o] = 0xFF
    want, tol = model(cache, q, k, v, counts, window, sinks)
    assert rows == 1 or np.isnan(want).any()
    out = cache.attention(q, k, v, row_start=starts(counts), max_rows=max(counts), max_len=length, window=window, sinks=sinks)
    cache.status()
    same(out, want, tol)
    # K: a token that only some rows see
    for place in (403, 6):
        cache.k[0, int(table[0, place // page]), 1, place % page, 9] = 0x7F
    out = cache.attention(q, k, v, row_start=starts(counts), max_rows=max(counts), max_len=length, window=window, sinks=sinks)
    cache.status()
    sees = np.array([length + r + 1 - window <= 403 for r in range(rows)] + [False] * 2)
    hit = np.isnan(want) | (sees[:, None] & (np.arange(heads) >= heads // 2))[..., None]
    got = out.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), hit)
    assert np.all(np.abs(got - want)[~hit] <= tol[~hit])


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_new_rows_that_have_left_the_window(lib, what):
    import torch
    rows = 150
    cache = build(lib, [20], 64, 32, 1, seed=5)
    q, k, v = normal((rows, 2, 64), 1), normal((rows, 1, 64), 2), normal((rows, 1, 64), 3)
    clean, window, sinks = v.clone(), 12, 21
    v[10, 0, 7] = what                                        # seen by rows 10 .. 21
    v[0, 0, 9] = what                                         # a first token: row 0 is at place 20
    clean[10, 0, 7] = 0
    clean[0, 0, 9] = 0
    want, tol = model(cache, q, k, clean, [rows], window, sinks)
    hit = np.zeros(want.shape, bool)
    hit[10:22, :, 7] = True
    hit[:, :, 9] = True
    for hint in (rows, 1):
        got = cache.attention(q, k, v, row_start=starts([rows]), window=window, sinks=sinks, max_rows=hint).cpu().double().numpy()
        cache.status()
        assert np.array_equal(~np.isfinite(got), hit)
        assert np.all(np.abs(got - want)[~hit] <= tol[~hit])


def test_pages_of_different_size(lib):
    """V scales many binades apart on both sides of the windows' edges, and a huge page that no row sees."""
    import torch
    for rows in (1, 100):
        cache = build(lib, [900], 128, 32, 1, seed=9)
        table = cache.table[0].long()
        for j in range(29):
            cache.v_scale[0, table[j], 0] *= 2.0 ** ((j * 7) % 23 - 11)
        cache.v_scale[0, table[5], 0] = 2.0 ** 60
        q, k, v = normal((rows, 2, 128), 1), normal((rows, 1, 128), 2), normal((rows, 1, 128), 3)
        out = cache.attention(q, k, v, row_start=starts([rows]), window=500, sinks=40)
        cache.status()
        close(out, *model(cache, q, k, v, [rows], 500, 40))


def test_no_window_is_the_plain_call(lib):
    """A window that covers every list gives the bits of the call without one; sinks without a window are refused."""
    import torch
    cache = build(lib, [300, 70], 128, 64, 2, seed=2)
    rows = [5, 40]
    q, k, v = normal((45, 4, 128), 1), normal((45, 2, 128), 2), normal((45, 2, 128), 3)
    plain = cache.attention(q, k, v, row_start=starts(rows))
    assert torch.equal(plain, cache.attention(q, k, v, row_start=starts(rows), window=cache.max_pages * 64 + 45, sinks=3))
    for window, sinks in ((0, 4), (-1, 0), (4, -1), (2 ** 30 + 1, 0)):
        with pytest.raises(lib.LaError):
            cache.attention(q, k, v, row_start=starts(rows), window=window, sinks=sinks)


def test_streams_graphs_and_repeats(lib):
    """The same bits on another stream with a workspace of its own, and from a graph after the sequences have grown."""
    import torch
    cache = build(lib, [400, 90], 128, 64, 2, seed=2, extra_pages=3, spare=8)
    q, k, v = normal((2, 8, 128), 1), normal((2, 2, 128), 2), normal((2, 2, 128), 3)
    out = torch.empty_like(q)
    call = dict(window=100, sinks=4, max_rows=1, max_len=500)
    first = cache.attention(q, k, v, **call)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attention(q, k, v, out=out, **call)
    graph.replay()
    assert torch.equal(first, out)
    cache.append(k[None], v[None])
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = cache.attention(q, k, v, stream=side, workspace=cache.workspace(), **call)
    side.synchronize()
    cache.status()
    assert torch.equal(other, out)
    close(out, *model(cache, q, k, v, [1, 1], 100, 4))


def test_pages_in_the_gap_are_not_read(lib):
    """Table entries between the first tokens and the window may name no page: they are not looked at."""
    cache = build(lib, [3000], 128, 64, 1, seed=4)
    q, k, v = normal((1, 4, 128), 1), normal((1, 1, 128), 2), normal((1, 1, 128), 3)
    want = model(cache, q, k, v, [1], 200, 4)
    cache.table[0, 1:42] = -1                                 # window: places 2801 .. 3000, page 43 on
    out = cache.attention(q, k, v, window=200, sinks=4)
    cache.status()
    close(out, *want)


@pytest.mark.parametrize("hd,page,heads,kv,lens,rows,window,sinks", [
    (64, 32, 8, 2, [300, 0, 33, 64, 700], [1, 1, 2, 0, 2], 50, 4), (64, 64, 8, 1, [2100, 5, 640], [1] * 3, 300, 1), (128, 32, 2, 1, [900, 31], [4, 3], 129, 40),
    (64, 64, 3, 3, [70, 200], [8, 5], 6, 0), (128, 64, 2, 2, [1000], [8], 4, 900), (64, 128, 7, 1, [5000], [1], 3333, 0), (128, 128, 5, 1, [130, 128, 127, 1] * 9, [1] * 36, 100, 30),
    (128, 64, 8, 1, [4000] * 20, [1] * 20, 1000, 4), (64, 32, 1, 1, [20000], [1], 15000, 64), (128, 64, 16, 2, list(range(0, 640, 5)), [1] * 128, 64, 2)])
def test_few_vectors(lib, hd, page, heads, kv, lens, rows, window, sinks):
    """Up to eight query vectors for each KV head and sequence, all pages and dims, with and without new keys."""
    cache = build(lib, lens, hd, page, kv, seed=hd + page)
    n = sum(rows)
    q, k, v = normal((n, heads, hd), 1, 1.5), normal((n, kv, hd), 2), normal((n, kv, hd), 3)
    hints = dict(max_rows=max(rows), max_len=max(lens))
    out = cache.attention(q, k, v, row_start=starts(rows), window=window, sinks=sinks, **hints)
    cache.status()
    close(out, *model(cache, q, k, v, rows, window, sinks))
    assert (out == cache.attention(q, k, v, row_start=starts(rows), window=window, sinks=sinks, **hints)).all()
    alone = cache.attention(q, row_start=starts(rows), window=window, sinks=sinks, **hints)
    cache.status()
    close(alone, *model(cache, q, None, None, rows, window, sinks))


def test_few_vectors_of_a_tree(lib):
    """Rows of a small tree, whose ancestors count towards their windows; NaN in the keys and values that some do not see."""
    import torch
    rows, window, sinks = 7, 20, 3
    see = [[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4], [5], [0, 1, 3, 6]]
    words = np.zeros((rows, 8), np.int32)
    for r, seen in enumerate(see):
        words[r, 0] = sum(1 << j for j in seen)
    cache = build(lib, [90], 128, 32, 2, seed=6)
    q, k, v = normal((rows, 2, 128), 1), normal((rows, 2, 128), 2), normal((rows, 2, 128), 3)
    table = cache.table.cpu().numpy()
    for place in (60, 71, 72, 73, 5):                          # windows begin at 71 .. 74
        cache.v[0, int(table[0, place // 32]), 0, place, place % 32] = 0x7F
    want, tol = model(cache, q, k, v, [rows], window, sinks, see=lambda s, r: see[r])
    assert np.isnan(want).any() and not np.isnan(want).all()
    out = cache.attention(q, k, v, row_start=starts([rows]), vis=torch.from_numpy(words).cuda(), window=window, sinks=sinks, max_rows=rows)
    cache.status()
    same(out, want, tol)


@pytest.mark.parametrize("window,sinks", [(2 ** 32 + 8, 0), (2 ** 32, 4), (8, 2 ** 32), (8, -2 ** 32), (-2 ** 32 + 8, 0)])
def test_numbers_of_more_than_32_bits(lib, window, sinks):
    """Refused, not cut to their low 32 bits."""
    import torch
    c = lib.Kv8Cache(1, 4, 64, 2, 128, 1, 4)
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises((ValueError, lib.LaError), match="window"):
        c.attention(q, window=window, sinks=sinks)


@pytest.mark.parametrize("hd,page,heads,kv,lens,window,sinks", [
    (64, 32, 8, 4, [3000, 1801, 40, 0] + [100 * i for i in range(1, 29)], 1800, 4), (128, 64, 8, 2, [2000, 5, 700, 1500], 750, 0), (128, 64, 8, 2, [2000, 5, 700], 1000, 70),
    (128, 128, 4, 4, [1100] * 3, 700, 130), (128, 32, 5, 5, [400, 1000], 600, 1)])
def test_units_of_some_pages(lib, hd, page, heads, kv, lens, window, sinks):
    """Single rows whose windows are long enough to be split among blocks, and few or short enough to stay whole, with each bound on the lengths."""
    cache = build(lib, lens, hd, page, kv, seed=heads)
    n = len(lens)
    q, k, v = normal((n, heads, hd), 1, 1.5), normal((n, kv, hd), 2), normal((n, kv, hd), 3)
    want = model(cache, q, k, v, [1] * n, window, sinks)
    for most in (0, max(lens), 64):
        out = cache.attention(q, k, v, max_len=most, window=window, sinks=sinks)
        cache.status()
        close(out, *want)
