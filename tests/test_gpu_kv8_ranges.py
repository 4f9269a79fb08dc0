"""Attention over the paged 8-bit KV cache where values lie many binades apart,
against the plain 64-bit form: what a row does not see, or gives no weight,
must not cost it any bits."""
import numpy as np
import pytest

import kv8_model as M
from test_gpu_kv8 import build, lib, normal, starts, tree_words  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hint", [0, 1])          # many and few query vectors' kernel: max_rows never changes the result
@pytest.mark.parametrize("size", [1e9, 1e12, 1e30, 3e38])
@pytest.mark.parametrize("rows,hd,tree,what", [(40, 128, True, "v"), (40, 128, False, "k"), (121, 128, True, "k"), (121, 64, False, "v"),
                                               (300, 64, False, "k"), (300, 128, False, "v"), (40, 64, True, "kv")])
def test_unseen_rows_of_any_size_do_not_leak(lib, rows, hd, tree, what, size, hint):
    """A huge finite K or V, in a row that most rows do not see, changes nothing in those."""
    import torch
    cache = build(lib, [70, 0, 260], hd, 64, 2)
    counts = [rows, 3, 5]
    n = sum(counts)
    q, k, v = normal((n, 4, hd), 1), normal((n, 2, hd), 2), normal((n, 2, hd), 3)
    big = [2, rows // 2] if tree else [rows - 2]
    for b in big:
        for x, name in ((k, "k"), (v, "v")):
            if name in what:
                x[b, 0, 5] = size
                x[b, 1] = torch.where(x[b, 1] > 0, size, -size)
    see = [[j for j in range(r + 1) if j < 256 and (j not in big or j == r)] for r in range(rows)] if tree else [list(range(r + 1)) for r in range(rows)]
    see += [list(range(r + 1)) for c in counts[1:] for r in range(c)]
    first = np.concatenate([[0], np.cumsum(counts)])
    vis = torch.from_numpy(tree_words(see)).cuda() if tree else None
    out = cache.attention(q, k, v, row_start=starts(counts), vis=vis, max_rows=hint)
    cache.status()
    blind = [r for r in range(n) if r >= rows or not set(see[r]) & set(big)]
    assert len(blind) >= n - len(big) - 2
    want, tol = M.attention(cache, q, k, v, counts, see=lambda s, r: see[first[s] + r])
    got = out.cpu().double().numpy()
    err = np.abs(got - want)[blind] / tol[blind]
    assert np.all(err <= 1), f"worst {np.nanmax(err):.3g} of the tolerance, {np.isnan(err).sum()} NaN"


@pytest.mark.parametrize("rows,hd", [(40, 128), (130, 64), (256, 128)])
def test_rows_that_see_themselves_alone(lib, rows, hd):
    """K and V from 2^-60 to 2^100 in one tile, some rows zero: each row gives its own V, rounded to bf16 once (2^-8)."""
    import torch
    cache = build(lib, [0], hd, 32, 2)
    q, k, v = normal((rows, 2, hd), 1), normal((rows, 2, hd), 2), normal((rows, 2, hd), 3)
    e = torch.arange(rows, device="cuda") * 37 % 161 - 60
    size = torch.ldexp(torch.ones(rows, device="cuda"), e)[:, None, None].to(torch.bfloat16)
    k, v = k * size.flip(0), v * size
    k[3], v[5], v[6, 0] = 0, 0, 0
    vis = torch.from_numpy(tree_words([[r] if r < 256 else [] for r in range(rows)])).cuda()
    out = cache.attention(q, k, v, row_start=starts([rows]), vis=vis, max_rows=rows)
    cache.status()
    got, want = out.double(), v.double()
    # a row's factor brings its largest value to 2^14 or more, where fp16's least half step is 2^-25
    floor = 2.0 ** -39 * want.abs().amax(-1, keepdim=True)
    assert torch.all((got - want).abs() <= 2.0 ** -8 * want.abs() + floor), float(((got - want).abs() / (want.abs() + 1e-300)).max())


def exact(cache, q, k, v, see):
    """Attention of the rows q over slot 0 and the new rows see[r], in 64 bits: out, and its tolerance as in
    kv8_model.attention, but for the weights' last bits: fp16 rounds weights below 2^-14 of the unit by 2^-25, and
    the unit is at most 2^5 times what the largest weight's V scale asks for, the largest weight at least half of it:
    2^-19 of the largest weight, or the weight itself, times each value that is added, whatever other pages hold."""
    D, G, page, n = q.shape[2], q.shape[1] // cache.n_kv_heads, cache.page, int(cache.lens[0])
    ids = cache.table[0, :-(-n // page)].cpu().numpy()
    f = lambda x: x.cpu().double().numpy()  # noqa: E731
    q, k, v = f(q), f(k), f(v)
    kb, vb = (M.E4M3[x[0].cpu().numpy()[ids]] for x in (cache.k, cache.v))
    ks, vs = (f(x[0])[ids][..., None, None] for x in (cache.k_scale, cache.v_scale))
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(cache.n_kv_heads):
        K = (kb * ks)[:, h].reshape(-1, D)[:n]
        V = np.swapaxes((vb * vs)[:, h], 1, 2).reshape(-1, D)[:n]
        for r in range(q.shape[0]):
            Kr, Vr = np.concatenate([K, k[see[r], h]]), np.concatenate([V, v[see[r], h]])
            for g in range(h * G, h * G + G):
                z = Kr @ q[r, g] / np.sqrt(D)
                p = np.exp(z - z.max())
                p /= p.sum()
                o, A = p @ Vr, p @ np.abs(Vr)
                dz = (D + 8) * 2.0 ** -23 / np.sqrt(D) * (np.abs(Kr) @ np.abs(q[r, g])).max()
                out[r, g] = o
                tol[r, g] = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2 * dz + len(Kr) * 2.0 ** -24 + 2.0 ** -20) * (A + np.abs(o)) \
                    + np.minimum(2.0 ** -19 * p.max(), p) @ np.abs(Vr)
    return out, tol


def within(got, want, tol):
    err = np.abs(got.cpu().double().numpy() - want) / np.maximum(tol, 1e-300)
    assert np.all(err <= 1), f"worst {np.nanmax(err):.3g} of the tolerance at {np.unravel_index(np.nanargmax(err), err.shape)}, {np.isnan(err).sum()} NaN"


@pytest.mark.parametrize("far", [10, 24, 45])
@pytest.mark.parametrize("rows", [1, 5, 40, 200])
@pytest.mark.parametrize("hd,page,pages,length", [(128, 32, [0, 1, 0, 2, 0, 0, 1, 2, 2, 0], 300), (64, 32, [1, 0, 0, 0, 2, 0, 1], 224),
                                                  (128, 64, [0, 1, 1, 0, 2, 0], 380), (64, 128, [1, 0, 2, 0], 500),
                                                  (128, 128, [0, 2, 1, 1, 0, 1, 2, 0, 1], 1100)])
def test_scales_of_pages_far_apart(lib, hd, page, pages, length, rows, far):
    """Pages 2^far above (1) and below (2) the others, neighbours within 128 keys or not.  The lower half of the dims has
    values in every page, the upper half in the ordinary pages alone: these must come through as if the others were zero."""
    import torch
    cache = build(lib, [length], hd, page, 2, seed=5)
    for j, kind in enumerate(pages):
        if kind:
            p = int(cache.table[0, j])
            cache.v_scale[0, p] *= 2.0 ** (far if kind == 1 else -far)
            cache.v[0, p, :, hd // 2:] = 0
    q, k, v = normal((rows, 4, hd), 1, 1.5), normal((rows, 2, hd), 2), normal((rows, 2, hd), 3)
    out = cache.attention(q, k, v, row_start=starts([rows]), max_rows=rows)
    cache.status()
    within(out, *exact(cache, q, k, v, [list(range(r + 1)) for r in range(rows)]))


@pytest.mark.parametrize("rows", [2, 60])
@pytest.mark.parametrize("far", [20, 55])
def test_a_huge_token_without_weight(lib, rows, far):
    """One token of a page is 2^far above the rest, in eight dims, and has a weight of about e^-400: the other dims and the
    other pages' values keep their bits."""
    import torch
    hd, page = 128, 64
    cache = build(lib, [400], hd, page, 1, seed=9)
    q, k, v = normal((1, 1, hd), 1, 1.5).repeat(rows, 2, 1), normal((rows, 1, hd), 2), normal((rows, 1, hd), 3)
    p = int(cache.table[0, 2])
    cache.v[0, p] = 0                                         # what the page's other tokens come to at this scale
    cache.v[0, p, :, :8, 7] = 0x7E
    cache.v_scale[0, p] = 2.0 ** far
    cache.k[0, p] = 0                                         # and their scores
    cache.k[0, p, 0, 7] = torch.where(q[0, 0] > 0, 0xFE, 0x7E).to(torch.uint8)
    cache.k_scale[0, p] = 2.0 ** -3
    out = cache.attention(q, k, v, row_start=starts([rows]), max_rows=rows)
    cache.status()
    within(out, *exact(cache, q, k, v, [list(range(r + 1)) for r in range(rows)]))


@pytest.mark.parametrize("rows", [1, 40])
def test_many_small_weights(lib, rows):
    """A key with a weight of about a half and 60000 others that share the rest: none of them is too small to count."""
    import torch
    hd, n = 64, 60000
    cache = build(lib, [n], hd, 128, 1, seed=4)
    q, k, v = normal((1, 1, hd), 1).repeat(rows, 1, 1), normal((rows, 1, hd), 2, 1e-3), normal((rows, 1, hd), 3)
    cache.k[:] = 0
    x = q[0, 0].float() / q[0, 0].float().norm() ** 2 * np.log(n) * np.sqrt(hd)     # q . x / sqrt(hd) = log n
    s = 2.0 ** -4
    cache.k_scale[:] = s
    p = int(cache.table[0, 100])
    cache.k[0, p, 0, 3] = torch.from_numpy(M.e4m3_bytes(x.double().cpu().numpy() / s)).cuda()
    cache.v[:] = 0x38                                          # 1, in every dim of every key
    cache.v_scale[:] = 2.0 ** -2
    out = cache.attention(q, k, v * 0, row_start=starts([rows]), max_rows=rows)
    cache.status()
    within(out, *exact(cache, q, k, v * 0, [list(range(r + 1)) for r in range(rows)]))


@pytest.mark.parametrize("size", [1e20, 3e38])
@pytest.mark.parametrize("score", [-1000.0, 0.0, 300.0])
@pytest.mark.parametrize("rows,hd", [(1, 64), (3, 128), (20, 128), (150, 64), (300, 128)])
def test_a_huge_row_that_all_see(lib, rows, hd, score, size):
    """The first new row's V is huge and every row sees it, with no weight, with a little, or with all: in each of a
    call's kernels, against keys of the cache that outweigh it by e^400, or that it outweighs."""
    import torch
    page, n = 32, 130
    cache = build(lib, [n], hd, page, 2, seed=6)
    q, k, v = normal((1, 4, hd), 1).repeat(rows, 1, 1), normal((rows, 2, hd), 2), normal((rows, 2, hd), 3)
    v[0] = torch.where(v[0] > 0, size, -size)
    for h in range(2):                                         # one query's direction: the other heads take what comes
        x = q[0, 2 * h].float()
        k[0, h] = x / x.norm() ** 2 * score * np.sqrt(hd)
    out = cache.attention(q, k, v, row_start=starts([rows]), max_rows=rows)
    within(out, *exact(cache, q, k, v, [list(range(r + 1)) for r in range(rows)]))
    x = q[0, 0].double().cpu().numpy()                         # a key of the cache with a score of 400 more
    p = int(cache.table[0, 3])
    cache.k[0, p, 0] = 0
    cache.k[0, p, 0, 5] = torch.from_numpy(M.e4m3_bytes(x / np.abs(x).max() * 448)).cuda()
    cache.k_scale[0, p, 0] = 2.0 ** np.round(np.log2((score + 400) * np.sqrt(hd) / (x @ x / np.abs(x).max() * 448)) if score > -400 else -3)
    out = cache.attention(q, k, v, row_start=starts([rows]), max_rows=rows)
    cache.status()
    within(out, *exact(cache, q, k, v, [list(range(r + 1)) for r in range(rows)]))


@pytest.mark.parametrize("rows,hd,page", [(1, 128, 64), (4, 64, 32), (40, 128, 32), (140, 64, 128)])
@pytest.mark.parametrize("scale,k_scale,zero", [(1e-38, 2.0 ** -60, False), (1e-45, 1.0, False), (3e38, 2.0 ** 60, True), (2.9e38, 2.0 ** -60, True)])
def test_factors_past_fp32(lib, rows, hd, page, scale, k_scale, zero):
    """scale * K's scale below or above what fp32 holds: scores of 0, for the keys that a row sees alone.  Tolerance: bf16's
    2^-8 of the mean, fp32 sums of n equal weights n 2^-24 of the mean magnitude."""
    import torch
    n = 77
    cache = build(lib, [n], hd, page, 1, seed=2)
    cache.k_scale[:] = k_scale
    q, k, v = normal((rows, 2, hd), 1), normal((rows, 1, hd), 2), normal((rows, 1, hd), 3)
    if zero:
        cache.k[:] = 0
        k[:] = 0
        q[0] *= 2.0 ** 100
    out = cache.attention(q, k, v, row_start=starts([rows]), scale=scale, max_rows=rows)
    cache.status()
    ids = cache.table[0, :-(-n // page)].long()
    V = torch.from_numpy(M.E4M3[cache.v[0, ids, 0].cpu().numpy()]) * cache.v_scale[0, ids, 0].cpu().double()[:, None, None]
    V = V.transpose(1, 2).reshape(-1, hd)[:n]
    got = out.cpu().double()
    for r in range(rows):
        Vr = torch.cat([V, v[:r + 1, 0].cpu().double()])
        want = Vr.mean(0)
        tol = 2.0 ** -8 * want.abs() + len(Vr) * 2.0 ** -24 * Vr.abs().mean(0)
        assert torch.all((got[r] - want).abs() <= tol), (r, got[r], want)
