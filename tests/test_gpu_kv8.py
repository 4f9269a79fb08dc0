"""The paged 8-bit KV cache on the GPU against its plain 64-bit form: bytes,
tables and counts exactly, attention within a tolerance that follows from its
roundings (kv8_model.attention)."""
import numpy as np
import pytest

import kv8_model as M
from helpers import ensure_built

pytestmark = pytest.mark.gpu
STATE, CAPACITY = -6, -3


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import exact_decoding_gb300 as e
    return e


def ints(v):
    import torch
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def starts(counts, first=0):
    return ints(first + np.concatenate([[0], np.cumsum(counts)]))


def normal(shape, seed, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).cuda()


def close(out, want, tol):
    got = out.cpu().double().numpy()
    assert np.all(np.isfinite(got))
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - want) / np.maximum(tol, 1e-300)):.3g} of the tolerance at {np.argwhere(bad)[:3].tolist()}"


def build(lib, lens, hd=128, page=64, kv=2, layers=1, seed=1, spare=3, extra_pages=2, shared=()):
    most = max(-(-n // page) for n in lens) + extra_pages
    cache = lib.Kv8Cache(layers, sum(-(-n // page) for n in lens) + spare, page, kv, hd, len(lens), most)
    M.fill(cache, lens, seed, shared)
    return cache


# ------------------------------------------------------------------ attention
ATTEND = [
    # hd, page, heads, kv heads, lens, rows, max_len (a hint: 0 means the table's room)
    (128, 64, 4, 4, [117], [1], 117),
    (128, 64, 4, 4, [0], [1], 0),
    (128, 64, 8, 1, [1], [1], 1),
    (128, 32, 8, 2, [63, 64, 65, 0, 31, 1, 200], [1] * 7, 200),
    (64, 32, 6, 2, [5, 300, 33, 129], [1, 2, 3, 1], 0),
    (64, 128, 3, 3, [128, 127, 129, 500], [1, 0, 5, 2], 500),
    (128, 128, 16, 2, [1500, 3], [1, 1], 1500),
    (128, 64, 8, 1, [4100], [1], 4100),                       # split over many workers, joined
    (128, 64, 8, 1, [4100], [1], 8),                          # the hint is too low: same answer
    (64, 64, 4, 1, [2500, 0, 17, 900], [3, 1, 1, 20], 2500),
    (128, 64, 5, 5, [70], [17], 0),                           # rows past one tile of query vectors
    (128, 32, 12, 2, [40, 90], [70, 1], 0),                   # more new rows than one key tile
    (64, 64, 2, 2, [130], [130], 0),
    (128, 64, 4, 2, [300, 10], [129, 3], 300),
    (128, 64, 32, 1, [100, 40], [9, 1], 0),
    (64, 32, 8, 8, [31], [256], 31),
]


@pytest.mark.parametrize("hd,page,heads,kv,lens,rows,max_len", ATTEND)
def test_attention_causal(lib, hd, page, heads, kv, lens, rows, max_len):
    cache = build(lib, lens, hd, page, kv, seed=len(lens) + heads)
    n = sum(rows)
    q, k, v = normal((n, heads, hd), 1, 1.5), normal((n, kv, hd), 2), normal((n, kv, hd), 3)
    out = cache.attention(q, k, v, row_start=starts(rows), max_rows=max(rows), max_len=max_len)
    cache.status()
    close(out, *M.attention(cache, q, k, v, rows))


@pytest.mark.parametrize("hd,page,lens,rows", [(128, 64, [0, 90, 64], [2, 1, 3]), (64, 32, [0, 0], [1, 4]), (128, 128, [2000], [1])])
def test_attention_over_the_cache_alone(lib, hd, page, lens, rows):
    """Without k and v a row of an empty sequence sees nothing and gives 0."""
    import torch
    cache = build(lib, lens, hd, page, 2)
    q = normal((sum(rows), 6, hd), 4)
    out = torch.full_like(q, 7.0)
    cache.attention(q, row_start=starts(rows), out=out)
    cache.status()
    close(out, *M.attention(cache, q, None, None, rows))
    if lens[0] == 0:
        assert torch.all(out[:rows[0]] == 0)


def tree_words(see):
    w = np.zeros((len(see), 8), np.uint32)
    for r, row in enumerate(see):
        for j in row:
            w[r, j // 32] |= np.uint32(1 << (j % 32))
    return w.view(np.int32)


@pytest.mark.parametrize("hd,heads,kv,N,W,G,length", [(128, 4, 4, 5, 15, 15, 300), (64, 4, 2, 4, 5, 3, 33), (128, 8, 1, 3, 4, 4, 1100),
                                                     (128, 8, 8, 5, 5, 5, 0)])
def test_attention_under_the_step_mask(lib, hd, heads, kv, N, W, G, length):
    """The visibility words of a lookahead step, as la_step_tables gives them."""
    import torch
    _, vis, _ = lib.la_step_tables(N, W, G)
    rows = vis.shape[0]
    see = [[j for j in range(rows) if (int(vis[r, j // 32]) >> (j % 32)) & 1] for r in range(rows)]
    cache = build(lib, [length], hd, 64, kv)
    q, k, v = normal((rows, heads, hd), 5, 1.5), normal((rows, kv, hd), 6), normal((rows, kv, hd), 7)
    out = cache.attention(q, k, v, row_start=starts([rows]), vis=torch.from_numpy(vis.view(np.int32)).cuda())
    cache.status()
    close(out, *M.attention(cache, q, k, v, [rows], see=lambda s, r: see[r]))


@pytest.mark.parametrize("rows", [5, 40])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_masked_rows_do_not_leak(lib, rows, what):
    """NaN and infinities in new rows that a row does not see change nothing there, and reach the rows that see them."""
    import torch
    cache = build(lib, [70, 0], 128, 64, 2)
    counts = [rows, 3]
    n = sum(counts)
    q, k, v = normal((n, 4, 128), 1), normal((n, 2, 128), 2), normal((n, 2, 128), 3)
    v[2, 0, 5] = what
    v[2, 1, :] = what
    k[rows - 1, 1, 7] = what
    see = [[j for j in range(r + 1) if j != 2 or r in (2, rows - 2)] for r in range(rows)] + [[0], [], [2]]
    out = cache.attention(q, k, v, row_start=starts(counts), vis=torch.from_numpy(tree_words(see)).cuda())
    cache.status()
    clean, kc = (torch.where(torch.isfinite(x), x, 0.0) for x in (v, k))
    want, tol = M.attention(cache, q, kc, clean, counts, see=lambda s, r: see[r] if s == 0 else see[rows + r])
    got = out.cpu().double().numpy()
    hit = np.zeros(got.shape, bool)
    hit[[2, rows - 2], :2, 5] = True
    hit[[2, rows - 2], 2:] = True
    hit[rows - 1, 2:] = True                                  # sees its own K
    assert np.all(np.abs(got - want)[~hit] <= tol[~hit])
    if rows - 2 != 2:
        assert not np.isfinite(got[[2, rows - 2], :2, 5]).any() and not np.isfinite(got[[2, rows - 2], 2:]).any()
    assert torch.all(out[rows + 1] == 0)                      # a mask that leaves the row empty


def test_rows_of_no_slot_and_strides(lib):
    """Columns of one fused projection, output rows with room between them, rows before and behind the slots' untouched."""
    import torch
    cache = build(lib, [33, 100, 0], 64, 32, 2)
    rows, kv, heads, hd = [2, 0, 3], 2, 6, 64
    n = sum(rows) + 5
    qkv = normal((n, (heads + 2 * kv) * hd), 8)
    q = qkv[:, :heads * hd].unflatten(1, (heads, hd))
    k = qkv[:, heads * hd:(heads + kv) * hd].unflatten(1, (kv, hd))
    v = qkv[:, (heads + kv) * hd:].unflatten(1, (kv, hd))
    wide = torch.full((n, heads * hd + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :heads * hd].unflatten(1, (heads, hd))
    cache.attention(q, k, v, row_start=starts(rows, 2), out=out)
    cache.status()
    want, tol = M.attention(cache, q, k, v, rows, first=2)
    close(out[2:7], want[2:7], tol[2:7])
    assert torch.all(out[:2] == 3) and torch.all(out[7:] == 3) and torch.all(wide[:, heads * hd:] == 3)


def test_layer_scale_and_shared_pages(lib):
    cache = build(lib, [200, 150, 64], 128, 32, 3, layers=3, shared=[(0, 1), (0, 2)])
    q, k, v = normal((3, 6, 128), 1), normal((3, 3, 128), 2), normal((3, 3, 128), 3)
    for layer, scale in ((0, 0.0), (2, 0.031), (1, 1.0)):
        out = cache.attention(q, k, v, layer=layer, scale=scale)
        close(out, *M.attention(cache, q, k, v, [1, 1, 1], layer=layer, scale=scale))
    cache.status()


def test_pages_of_very_different_size(lib):
    """A page whose V is 2^24 times another's, one of zeros, and a sink key with nearly all of the weight."""
    cache = build(lib, [256], 128, 64, 1)
    ids = cache.table[0, :4].long()
    cache.v_scale[0, ids[1]] *= 2.0 ** 24
    cache.v[0, ids[2]] = 0
    cache.v_scale[0, ids[2]] = 2.0 ** -60
    q, k, v = normal((1, 4, 128), 1, 3.0), normal((1, 1, 128), 2), normal((1, 1, 128), 3, 1e-4)
    close(cache.attention(q, k, v), *M.attention(cache, q, k, v, [1]))
    k[0] = q[0, 0:1] * 3                                      # the new row's own key outweighs the cache for head 0
    close(cache.attention(q, k, v), *M.attention(cache, q, k, v, [1]))


def test_offsets_past_32_bits(lib):
    """Pages whose bytes lie beyond 2^32 in the pool."""
    import torch
    page, kv, hd = 128, 8, 128
    n_pages = 2 ** 32 // (page * kv * hd) + 40
    small = build(lib, [300, 77], hd, page, kv, spare=0)
    big = lib.Kv8Cache(1, n_pages, page, kv, hd, 2, small.max_pages)
    far = torch.arange(n_pages - small.n_pages, n_pages, device="cuda")
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(big, name)[0, far] = getattr(small, name)[0]
    big.table.copy_(torch.where(small.table >= 0, far.to(torch.int32)[small.table.clamp(min=0).long()], -1))
    big.lens.copy_(small.lens)
    q, k, v = normal((2, 8, hd), 1), normal((2, kv, hd), 2), normal((2, kv, hd), 3)
    assert torch.equal(big.attention(q, k, v), small.attention(q, k, v))
    big.refs.fill_(1)                                         # every page in use but the last ones
    big.refs[n_pages - small.n_pages + int(small.refs.sum()) - 1] = 1
    kn, vn = normal((1, 2, kv, hd), 4), normal((1, 2, kv, hd), 5)
    assert big.append(kn, vn).tolist() == [1, 1] == small.append(kn, vn).tolist()
    for name in ("k", "v", "k_scale", "v_scale"):
        a, b = getattr(big, name)[0, far], getattr(small, name)[0]
        assert torch.equal(a.nan_to_num(0) if a.is_floating_point() else a, b.nan_to_num(0) if b.is_floating_point() else b)
    big.status()


def test_bad_pages_and_lengths_are_skipped(lib):
    """Page numbers and lengths outside the cache are never followed: status says so, other sequences are right."""
    import torch
    cache = build(lib, [100, 90, 80], 128, 32, 2)
    good = cache.table.clone()
    q, k, v = normal((3, 4, 128), 1), normal((3, 2, 128), 2), normal((3, 2, 128), 3)
    want, tol = M.attention(cache, q, k, v, [1, 1, 1])
    for bad in (-1, cache.n_pages, 2 ** 31 - 1, -2 ** 31):
        cache.table[1, 1] = bad
        out = cache.attention(q, k, v)
        with pytest.raises(lib.LaError) as e:
            cache.status()
        assert e.value.code == STATE
        close(out[[0, 2]], want[[0, 2]], tol[[0, 2]])
        assert torch.isfinite(out).all()
        cache.table.copy_(good)
    for bad in (-5, cache.max_pages * cache.page + 1):
        cache.lens[1] = bad
        out = cache.attention(q, k, v)
        with pytest.raises(lib.LaError):
            cache.status()
        close(out[[0, 2]], want[[0, 2]], tol[[0, 2]])
        assert cache.append(normal((1, 3, 2, 128), 1), normal((1, 3, 2, 128), 2), row_start=ints([0, 0, 1, 1])).tolist() == [0, 0, 0]
        with pytest.raises(lib.LaError):
            cache.status()
        cache.lens[1] = 90
    for rs in ([0, 2, 1, 3], [0, 1, 2, 9], [-1, 1, 2, 3]):
        cache.attention(q, k, v, row_start=ints(rs))
        with pytest.raises(lib.LaError) as e:
            cache.status()
        assert e.value.code == STATE
    cache.status()


def test_streams_and_graphs(lib):
    """A captured append and attention, replayed over changing inputs, on a stream of its own."""
    import torch
    cache, eager = (build(lib, [100, 5], 128, 32, 2, spare=20, extra_pages=6) for _ in range(2))
    q, k, v = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((2, 4, 128), (2, 2, 128), (2, 2, 128)))
    out = torch.empty_like(q)
    stream = torch.cuda.Stream()
    cache.attention(q, k, v, out=out)                         # attributes are set outside the capture
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        cache.attention(q, k, v, out=out)
        cache.append(k[None], v[None])
    for i in range(70):                                       # past two page borders
        for t, x in ((q, 10), (k, 20), (v, 30)):
            t.copy_(normal(t.shape, x + 100 * i))
        g.replay()
        want = eager.attention(q, k, v)
        eager.append(k[None], v[None])
        assert torch.equal(out, want), i
    M.Model(eager).same_as(cache)
    cache.status()


# ------------------------------------------------------------------ append, fork, free, compact
@pytest.mark.parametrize("hd,page,kv,layers", [(128, 64, 2, 2), (64, 32, 3, 1), (128, 128, 1, 2), (64, 64, 1, 3), (128, 32, 2, 1)])
def test_append_matches_its_definition(lib, hd, page, kv, layers):
    """Growing magnitudes (rescaled pages), tokens one by one and many at a time, values at ties and subnormals."""
    import torch
    cache = lib.Kv8Cache(layers, 24, page, kv, hd, 3, 12)
    model = M.Model(cache)
    for step, counts in enumerate(([1, 0, 3], [1, page - 1, 2], [page + 5, 1, 0], [1, 1, 1], [2 * page, 1, page], [0, 3, 1])):
        n = sum(counts)
        k, v = (normal((layers, n, kv, hd), 10 * step + i, 0.02 * 9.0 ** (step % 4)) for i in (1, 2))
        k[..., ::7] *= 2.0 ** -12
        v[..., ::5] = torch.round(v[..., ::5] * 64) / 64
        got = cache.append(k, v, row_start=starts(counts), max_rows=max(counts))
        assert got.tolist() == model.append(k.cpu().double().numpy(), v.cpu().double().numpy(), counts)
        model.same_as(cache)
    cache.status()


def test_append_every_bf16_value(lib):
    """All 65536 bf16 patterns, one to an element, at each of the scales their neighbours give."""
    import torch
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).cuda().view(1, 512, 1, 128)
    order = torch.argsort(x.float().abs().nan_to_num(3e38).flatten(), stable=True)
    sorted_ = x.flatten()[order].view(1, 512, 1, 128).contiguous()
    for t in (x, sorted_):
        cache = lib.Kv8Cache(1, 16, 32, 1, 128, 1, 16)
        model = M.Model(cache)
        cache.append(t, t.flip(1).contiguous(), row_start=starts([512]))
        model.append(t.cpu().double().numpy(), t.flip(1).cpu().double().numpy(), [512])
        model.same_as(cache)
        cache.status()


def test_append_runs_out_in_order(lib):
    """Sequences that no longer fit store nothing; a smaller one behind them still does."""
    cache = lib.Kv8Cache(1, 6, 32, 1, 64, 4, 4)
    model = M.Model(cache)
    for counts in ([33, 1, 0, 0], [100, 1, 40, 30], [1, 96, 1, 0], [0, 0, 3, 0]):
        k, v = normal((1, sum(counts), 1, 64), 1), normal((1, sum(counts), 1, 64), 2)
        got = cache.append(k, v, row_start=starts(counts)).tolist()
        assert got == model.append(k.cpu().double().numpy(), v.cpu().double().numpy(), counts)
        model.same_as(cache)
        if got != counts:
            with pytest.raises(lib.LaError) as e:
                cache.status()
            assert e.value.code == CAPACITY
    cache.status()


def test_append_of_chosen_rows(lib):
    """row_idx: the accepted rows of a step, from strided layers; an index outside is stored as zeros and reported."""
    import torch
    cache = lib.Kv8Cache(2, 8, 32, 2, 64, 2, 4)
    model = M.Model(cache)
    room = normal((2, 12, 3 * 2 * 64), 3)
    k, v = room[:, :, :128].unflatten(2, (2, 64)), room[:, :, 256:].unflatten(2, (2, 64))
    idx = [0, 7, 8, 11]
    got = cache.append(k, v, row_start=starts([3, 1]), row_idx=ints(idx))
    assert got.tolist() == [3, 1] == model.append(k.cpu().double().numpy(), v.cpu().double().numpy(), [3, 1], idx)
    model.same_as(cache)
    cache.status()
    cache.append(k, v, row_start=starts([1, 1]), row_idx=ints([-1, 12]))
    with pytest.raises(lib.LaError) as e:
        cache.status()
    assert e.value.code == STATE
    assert cache.lens.tolist() == [4, 2] and not torch.any(cache.k[:, cache.table[0, 0].item(), :, 3])


def test_a_life_of_branches(lib):
    """Random forks, appends, frees and compactions over one pool, against the model after every call; attention at the end."""
    g = np.random.default_rng(7)
    cache = lib.Kv8Cache(2, 40, 32, 2, 64, 6, 8)
    model = M.Model(cache)
    for step in range(60):
        kind = g.integers(0, 8)
        empty = [s for s in range(6) if model.lens[s] == 0]
        full = [s for s in range(6) if model.lens[s] > 0]
        if kind < 4:
            counts = [int(x) for x in g.integers(0, 3 if step % 5 else 40, 6)]
            n = sum(counts)
            if not n:
                continue
            k, v = (normal((2, n, 2, 64), 50 + 2 * step + i, float(np.exp(g.normal()))) for i in (0, 1))
            got = cache.append(k, v, row_start=starts(counts)).tolist()
            assert got == model.append(k.cpu().double().numpy(), v.cpu().double().numpy(), counts)
        elif kind == 4 and empty and full:
            src = [int(g.choice(full)) for _ in empty]
            cache.fork(ints(src), ints(empty))
            model.fork(src, empty)
        elif kind < 7 and full:
            slots = [int(s) for s in g.choice(full, size=min(2, len(full)))]   # sometimes the same twice
            keep = [int(g.integers(0, 60)) for _ in slots] if kind == 5 else None
            cache.free(ints(slots), None if keep is None else ints(keep))
            model.free(slots, keep)
        else:
            assert cache.compact().item() == model.compact()
        try:
            cache.status()
        except lib.LaError as e:
            assert e.code == CAPACITY                          # an append that did not fit: model and cache agree on it
        model.same_as(cache)
    q, k, v = normal((6, 4, 64), 1), normal((6, 2, 64), 2), normal((6, 2, 64), 3)
    close(cache.attention(q, k, v), *M.attention(cache, q, k, v, [1] * 6))
    used = model.table[model.table >= 0]
    assert np.array_equal(np.bincount(used, minlength=40), model.refs)


def test_compact_into_other_arrays_keeps_the_old_table_valid(lib):
    import torch
    cache = build(lib, [100, 200, 64, 1], 64, 32, 2, layers=2, spare=30)
    q, k, v = normal((4, 4, 64), 1), normal((4, 2, 64), 2), normal((4, 2, 64), 3)
    want = cache.attention(q, k, v)
    table, refs = torch.empty_like(cache.table), torch.empty_like(cache.refs)
    model = M.Model(cache)
    assert cache.compact(table_out=table, refs_out=refs).item() == model.compact()
    assert torch.equal(cache.attention(q, k, v), want)        # through the old table
    cache.table.copy_(table)
    cache.refs.copy_(refs)
    model.same_as(cache)
    assert torch.equal(cache.attention(q, k, v), want)
    assert cache.compact().item() == int((model.refs > 0).sum())   # nothing left to move
    model.same_as(cache)
    cache.status()


def test_refused_forks(lib):
    cache = build(lib, [40, 0, 10, 0, 0], 64, 32, 1)
    model = M.Model(cache)
    for src, dst in (([0], [2]), ([0], [5]), ([9], [1]), ([-1], [1]), ([0], [0]), ([0, 1], [1, 3])):
        cache.fork(ints(src), ints(dst))
        with pytest.raises(lib.LaError) as e:
            cache.status()
        assert e.value.code == STATE
        model.same_as(cache)
    cache.fork(ints([0, 2, 0]), ints([1, 1, 3]))              # the second names a taken dst: refused alone
    model.fork([0, 0], [1, 3])
    with pytest.raises(lib.LaError):
        cache.status()
    model.same_as(cache)
    cache.free(ints([7, -3, 1]))
    model.free([1])
    with pytest.raises(lib.LaError):
        cache.status()
    model.same_as(cache)


@pytest.mark.parametrize("hd,page,heads,kv,lens,rows", [
    (128, 32, 4, 2, [2600], [150]),                 # many query vectors: a long cache over many workers
    (64, 128, 8, 2, [3000, 40], [70, 3]),
    (128, 64, 4, 2, [500, 0, 77], [300, 5, 129]),   # several key tiles of new rows before the cached ones
    (64, 32, 2, 1, [129, 700, 64, 0], [257, 1, 128, 384]),
    (128, 128, 2, 1, [1000], [1100])])
def test_attention_of_many_rows(lib, hd, page, heads, kv, lens, rows):
    cache = build(lib, lens, hd, page, kv, seed=len(lens) + hd)
    n = sum(rows)
    q, k, v = normal((n, heads, hd), 4, 1.5), normal((n, kv, hd), 5), normal((n, kv, hd), 6)
    out = cache.attention(q, k, v, row_start=starts(rows))
    close(out, *M.attention(cache, q, k, v, rows))
    cache.status()


@pytest.mark.parametrize("hd,page,kv", [(64, 32, 2), (128, 64, 1)])
def test_many_short_sequences_and_few_long_ones(lib, hd, page, kv):
    """More units than a worker's share is long: shares begin with units, some workers get none."""
    g = np.random.default_rng(5)
    lens = [int(x) for x in g.integers(0, 70, 200)]
    lens[3], lens[120], lens[121] = 2500, 1700, 0
    cache = build(lib, lens, hd, page, kv, seed=3)
    q, k, v = normal((200, 2 * kv, hd), 7, 1.5), normal((200, kv, hd), 8), normal((200, kv, hd), 9)
    out = cache.attention(q, k, v)
    close(out, *M.attention(cache, q, k, v, [1] * 200))
    cache.status()


@pytest.mark.parametrize("rows", [1, 60])
@pytest.mark.parametrize("page", [32, 64, 128])
def test_keys_of_missing_pages_do_not_count(lib, rows, page):
    """Few and many query vectors: the keys of a page number outside the pool are left out, its neighbours' are right."""
    lens = [5 * page + 7, 3 * page]
    cache, whole = (build(lib, lens, 128, page, 2, seed=11) for _ in range(2))
    cache.table[0, 1] = cache.n_pages + 5
    cache.table[0, 4] = -7
    q, k, v = normal((2 * rows, 4, 128), 1), normal((2 * rows, 2, 128), 2), normal((2 * rows, 2, 128), 3)
    out = cache.attention(q, k, v, row_start=starts([rows, rows]))
    # the same keys without those pages: the later ones move up (their order does not matter)
    for j, p in enumerate([0, 2, 3, 5]):
        whole.table[0, j] = cache.table[0, p]
    whole.lens[0] = 3 * page + 7
    close(out, *M.attention(whole, q, k, v, [rows, rows]))
    with pytest.raises(lib.LaError) as e:
        cache.status()
    assert e.value.code == STATE


@pytest.mark.parametrize("hd,page,kv,most", [(64, 32, 1, 8), (128, 32, 3, 4), (128, 64, 5, 1), (64, 64, 6, 8)])
def test_append_few_rows_to_many_sequences(lib, hd, page, kv, most):
    """0 .. most rows for each of 130 sequences in two layers, three times over growing magnitudes: pages that fill
    up, rows over two pages, stored tokens rounded again, shared last pages copied."""
    g = np.random.default_rng(hd + most)
    lens = [int(x) for x in g.integers(0, 2 * page, 130)]
    cache = lib.Kv8Cache(2, 130 * 4, page, kv, hd, 133, 4)
    M.fill(cache, lens + [0, 0, 0], 3)
    model = M.Model(cache)
    cache.fork(ints([4, 5, 6]), ints([130, 131, 132]))
    model.fork([4, 5, 6], [130, 131, 132])
    for turn in range(3):
        rows = [int(x) for x in g.integers(0, most + 1, 133)]
        rows[4] = rows[130] = most
        n = sum(rows)
        k, v = normal((2, n, kv, hd), 20 + turn, 3.0 ** turn), normal((2, n, kv, hd), 30 + turn, 5.0 ** turn)
        want = model.append(k.cpu().double().numpy(), v.cpu().double().numpy(), rows)
        assert cache.append(k, v, row_start=starts(rows), max_rows=most).tolist() == want
        model.same_as(cache)
    cache.status()


@pytest.mark.parametrize("hd,page", [(128, 128), (128, 32), (64, 64)])
@pytest.mark.parametrize("rows", [1, 70])
def test_as_many_slots_as_there_may_be(lib, hd, page, rows):
    """2048 slots of which a few hold tokens or get rows, the first and the last among them."""
    lens = [0] * 2048
    lens[0], lens[1], lens[900], lens[2047] = 300, 5, 130, 77
    cache = build(lib, lens, hd, page, 2, seed=2)
    counts = [0] * 2048
    for s in (0, 900, 1500, 2047):
        counts[s] = rows
    n = 4 * rows
    q, k, v = normal((n, 4, hd), 1), normal((n, 2, hd), 2), normal((n, 2, hd), 3)
    out = cache.attention(q, k, v, row_start=starts(counts))
    close(out, *M.attention(cache, q, k, v, counts))
    cache.status()
    model = M.Model(cache)
    want = model.append(k[None].cpu().double().numpy(), v[None].cpu().double().numpy(), counts)
    assert cache.append(k[None], v[None], row_start=starts(counts)).tolist() == want
    model.same_as(cache)
    if want != counts:                      # three free pages do not take 70 rows of four sequences
        with pytest.raises(lib.LaError) as e:
            cache.status()
        assert e.value.code == CAPACITY
    cache.status()


def test_workspace_is_the_same_for_all_threads(lib):
    """The first calls of several threads at once ask for the device's size together."""
    import threading
    cache = build(lib, [5], 64, 32, 1)
    got, go = [0] * 16, threading.Barrier(16)

    def ask(i):
        go.wait()
        got[i] = lib.la_kv8_workspace(cache.struct)

    threads = [threading.Thread(target=ask, args=(i,)) for i in range(16)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert got == [cache.workspace().numel()] * 16
