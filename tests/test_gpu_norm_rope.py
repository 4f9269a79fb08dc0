"""Norm of heads and rotation by positions (Kv8Cache.norm_rope) against its formula in 64 bits."""
import math

import numpy as np
import pytest

from helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import exact_decoding_gb300 as e
    return e


def ints(v):
    import torch
    return torch.tensor([int(x) for x in v], dtype=torch.int32, device="cuda")


def cache(lib, seqs, kv, hd, lens, max_pages=1 << 14, page=128):
    c = lib.Kv8Cache(1, 1, page, kv, hd, seqs, max_pages)
    c.lens.copy_(ints(lens))
    return c


def formula(x, weight, pos, eps, freq):
    """[rows, heads, dim] float64 and its tolerance.

    Rounded once to bf16 (2^-8).  Before that, relative to the pair's magnitudes:
    the sum of squares is off by dim 2^-24, the norm by half of that, rsqrt and
    the products by 2^-21; the angle is rounded to 2^-25 of a half turn and sine and
    cosine to 2 units in the last place, 2^-21 together."""
    x = x.cpu().double().numpy()
    hd = x.shape[-1]
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.cpu().double().numpy()
    a, b = x[..., :hd // 2], x[..., hd // 2:]
    t = np.asarray(pos, dtype=np.float64)[:, None] * freq
    c, s = np.cos(t)[:, None], np.sin(t)[:, None]
    y = np.concatenate([a * c - b * s, b * c + a * s], -1)
    size = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
    return y, 2.0 ** -8 * np.abs(y) + (hd * 2.0 ** -25 + 2.0 ** -20) * size + 2.0 ** -130


def frequencies(base, hd):
    return np.array([base ** (-2 * i / hd) for i in range(hd // 2)])


def close(got, want, tol):
    d = np.abs(got.cpu().double().numpy() - want)
    assert np.all(d <= tol), f"{(~(d <= tol)).sum()} of {d.size} off, worst {np.nanmax(d / tol):.3g} of the tolerance at {np.argwhere(~(d <= tol))[:3].tolist()}"


def rows_of(n, heads, kv, hd, dtype, seed=0, pad=0):
    """q, k, v as columns of one buffer."""
    import torch
    g = torch.Generator().manual_seed(seed)
    b = (torch.randn(n, (heads + 2 * kv) * hd + pad, generator=g) * 2).to(dtype).cuda()
    at = [0, heads * hd, (heads + kv) * hd, (heads + 2 * kv) * hd]
    return [b[:, at[i]:at[i + 1]].unflatten(1, (-1, hd)) for i in range(3)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("hd,heads,kv,lens,rows,base", [
    (128, 32, 32, [65413], [1], 10000.0), (64, 1, 1, [0], [1], 10000.0), (64, 12, 4, [5, 0, 77], [3, 0, 20], 1e6),
    (128, 8, 1, [1000000, 3, 9], [1, 1, 1], 500000.0), (128, 2, 1, [7], [300], 10000.0), (64, 72, 8, list(range(40)), [1] * 40, 10000.0),
    (128, 5, 5, [2 ** 20 - 3, 0], [9, 130], 10000.0)])
def test_rows_behind_their_tokens(lib, dtype, hd, heads, kv, lens, rows, base):
    import torch
    dtype = getattr(torch, dtype)
    c = cache(lib, len(lens), kv, hd, lens)
    n = sum(rows)
    q, k, v = rows_of(n, heads, kv, hd, dtype, seed=n, pad=8)
    g = torch.Generator().manual_seed(1)
    qw, kw = ((1 + torch.randn(hd, generator=g)).to(dtype).cuda() for _ in range(2))
    pos = np.concatenate([np.arange(r) + ln for ln, r in zip(lens, rows)])
    start = ints(np.concatenate([[0], np.cumsum(rows)]))
    freq = frequencies(base, hd)
    qo, ko, vo = c.norm_rope(q, k, v, q_weight=qw, k_weight=kw, eps=1e-5, rope_base=base, row_start=start)
    c.status()
    close(qo, *formula(q, qw, pos, 1e-5, freq))
    close(ko, *formula(k, kw, pos, 1e-5, freq))
    assert torch.equal(vo, v.to(torch.bfloat16))
    qo, ko = c.norm_rope(q, k, rope_base=base, row_start=start)                # the rotation alone
    close(qo, *formula(q, None, pos, 0, freq))
    close(ko, *formula(k, None, pos, 0, freq))
    qo, ko = c.norm_rope(q, k, k_weight=kw, eps=0.25, rope_base=base, row_start=start)   # keys alone are normed
    close(qo, *formula(q, None, pos, 0, freq))
    close(ko, *formula(k, kw, pos, 0.25, freq))


def test_positions_that_are_given(lib):
    """pos and inv_freq as they are, negative and far positions among them; depth behind the cached tokens."""
    import torch
    c = cache(lib, 2, 2, 128, [100, 50])
    q, k, v = rows_of(7, 4, 2, 128, torch.float32)
    pos = [0, -1, 5, 2 ** 30, -2 ** 31, 2 ** 31 - 1, 12345]
    f32 = torch.from_numpy(frequencies(10000.0, 128) * 0.125 + 0.001).float()
    f32[0], f32[1] = 7.5, 0.0
    qo, ko = c.norm_rope(q, k, pos=ints(pos), inv_freq=f32.cuda())
    c.status()
    freq = f32.double().numpy()
    turn = [[math.fmod(p * f, 2 * math.pi) for f in freq] for p in pos]

    def at(x):   # the angle of far positions is off by 2^-24 of a turn
        y, tol = np.zeros(x.shape), np.zeros(x.shape)
        for r in range(7):
            y[r:r + 1], tol[r:r + 1] = formula(x[r:r + 1], None, [1.0], 0, np.array(turn[r]))
        xd = np.abs(x.cpu().double().numpy())
        return y, tol + 2 * math.pi * 2.0 ** -24 * np.concatenate([xd[..., :64] + xd[..., 64:]] * 2, -1)
    close(qo, *at(q))
    close(ko, *at(k))
    depth = [0, 1, 1, 2, 0, 0, 3]
    qo, ko = c.norm_rope(q, k, row_start=ints([0, 4, 7]), depth=ints(depth))
    want = [100 + d for d in depth[:4]] + [50 + d for d in depth[4:]]
    close(qo, *formula(q, None, want, 0, frequencies(10000.0, 128)))


def test_rows_of_no_sequence_stay(lib):
    """Rows before the first and behind the last sequence, and the outputs' other columns, are left as they were; in place works."""
    import torch
    c = cache(lib, 3, 1, 64, [4, 0, 9])
    q, k, v = rows_of(20, 3, 1, 64, torch.bfloat16, pad=16)
    q0, k0 = q.clone(), k.clone()
    qw = torch.ones(64, device="cuda")
    start = ints([2, 7, 7, 15])
    pos = np.array(list(range(4, 9)) + list(range(9, 17)))
    out = c.norm_rope(q, k, q_weight=qw, row_start=start, out=(q, k))
    c.status()
    assert out[0] is q
    for got, was, w in ((q, q0, qw), (k, k0, None)):
        assert torch.equal(got[:2], was[:2]) and torch.equal(got[15:], was[15:])
        close(got[2:15], *formula(was[2:15], w, pos, 1e-5, frequencies(10000.0, 64)))


def test_what_is_outside_the_cache(lib):
    """A length or row_start out of range sets the cache's status and reads nothing outside."""
    import torch
    c = cache(lib, 2, 1, 64, [-5, 1 << 30])
    q, k, _ = rows_of(4, 2, 1, 64, torch.float32)
    c.norm_rope(q, k, row_start=ints([0, 2, 4]))
    with pytest.raises(lib.LaError):
        c.status()
    c.lens.zero_()
    mark = torch.full((4, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    c.norm_rope(q, k, row_start=ints([3, 1, 9]), out=mark)
    with pytest.raises(lib.LaError):
        c.status()
    assert torch.all(mark[0] == 3) and torch.all(mark[1] == 3)


def test_zero_rows_zero_heads_and_streams(lib):
    """A head of zeros stays zero; no rows are a call that does nothing; a graph replays with the lengths of then."""
    import torch
    c = cache(lib, 2, 1, 128, [3, 8])
    q, k, v = rows_of(2, 4, 1, 128, torch.float32)
    q[1, 2] = 0
    w = torch.ones(128, device="cuda")
    out = c.norm_rope(q, k, v, q_weight=w, eps=1e-6)
    assert torch.all(out[0][1, 2] == 0)
    assert c.norm_rope(q[:0], k[:0], row_start=ints([0, 0, 0]))[0].shape == (0, 4, 128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = c.norm_rope(q, k, v, q_weight=w, eps=1e-6)
    c.lens.add_(5)
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = c.norm_rope(q, k, v, q_weight=w, eps=1e-6, stream=side)
    side.synchronize()
    for a, b in zip(again, other):
        assert torch.equal(a, b)
    close(again[1], *formula(k, None, [8, 13], 0, frequencies(10000.0, 128)))


@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.0, 0.25])
def test_far_positions(lib, base):
    """Angles by rope_base up to the largest position: off by 2^-23 of a turn at most, by 2^-26 up to position 2^20."""
    import torch
    c = cache(lib, 1, 2, 128, [0])
    pos = [2 ** 20, 2 ** 20 - 1, 2 ** 31 - 1, -2 ** 31, 123456789]
    q, k, _ = rows_of(5, 4, 2, 128, torch.float32, seed=3)
    qo, _ = c.norm_rope(q, k, pos=ints(pos), rope_base=base)
    c.status()
    from decimal import Decimal, getcontext
    getcontext().prec = 60                                    # the angles in decimals: doubles end at 2^-53 of 2^31 turns
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194988918")
    f = [Decimal(base) ** (Decimal(-2 * i) / Decimal(128)) for i in range(64)]
    for r, p in enumerate(pos):
        angle = np.array([float((Decimal(p) * x / two_pi) % 1) for x in f]) * 2 * math.pi
        y, tol = formula(q[r:r + 1], None, [1.0], 0, angle)
        xd = np.abs(q[r:r + 1].cpu().double().numpy())
        off = 2.0 ** -26 if abs(p) <= 2 ** 20 else 2.0 ** -23
        close(qo[r:r + 1], y, tol + 2 * math.pi * off * np.concatenate([xd[..., :64] + xd[..., 64:]] * 2, -1))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-5, 1e30])
def test_heads_whose_squares_leave_fp32(lib, dtype, hd, eps):
    """Heads near 2^-120 .. 2^120: the mean of their squares is 0 or infinity in fp32, their norm is not."""
    import torch
    c = cache(lib, 1, 2, hd, [11])
    q, k, _ = rows_of(9, 4, 2, hd, torch.float32, seed=8)
    size = torch.tensor([2.0 ** e for e in (-120, -80, -65, -50, 0, 60, 64, 90, 120)], device="cuda")
    q, k = ((x * size[:, None, None]).to(getattr(torch, dtype)).contiguous() for x in (q, k))
    q[:, 1, 3:] *= 2.0 ** -6                                  # one large value
    w = (1 + torch.rand(hd, generator=torch.Generator().manual_seed(2))).cuda()
    pos = 11 + np.arange(9)
    qo, ko = c.norm_rope(q, k, q_weight=w, k_weight=w, eps=eps, row_start=ints([0, 9]))
    c.status()
    eps = float(np.float32(eps))
    close(qo, *formula(q, w, pos, eps, frequencies(10000.0, hd)))
    close(ko, *formula(k, w, pos, eps, frequencies(10000.0, hd)))
