"""Log probabilities, entropy and alternatives (logprobs) against their definition in 64 bits."""
import math

import numpy as np
import pytest

from helpers import ensure_built

pytestmark = pytest.mark.gpu
LOWEST = -3.4028234663852886e38


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import exact_decoding_gb300 as e
    return e


def model(z, tokens, top):
    """(logprob, entropy, ids, top logprob) of float64 rows without NaN or +infinity, and the tolerances of the three numbers.

    With d = z - m: a term e^d is off by 2^-21 + |d| 2^-22 of itself (the product
    with log2 e, the exponential), r and s by those and by the rounding of their
    sums, 2^-24 for each of the n / 256 + 64 additions at most.  log1p adds 2^-22 of
    itself, the difference z - m and the result 2^-24 of theirs."""
    rows, vocab = z.shape
    lp, ent, ids, best = np.full(tokens.shape, -np.inf), np.zeros(rows), np.full((rows, top), -1), np.full((rows, top), -np.inf)
    tols = [np.zeros(tokens.shape), np.zeros(rows), np.zeros((rows, top))]
    for i in range(rows):
        m = z[i].max()
        if m == -np.inf:
            continue
        d = z[i] - m
        e = np.exp(d)
        arg = int(z[i].argmax())
        rest = np.delete(e, arg)
        r = math.fsum(rest)
        live = e > 0
        s = math.fsum((e * np.where(live, d, 0.0)).tolist())
        lse = math.log1p(r)
        ent[i] = lse - s / (1 + r)
        rel = 2.0 ** -21 + (vocab / 256 + 64) * 2.0 ** -24
        s2 = math.fsum((e * np.where(live, d * d, 0.0)).tolist())
        tl = (rel * r + 2.0 ** -22 * -s) / (1 + r) + 2.0 ** -22 * lse
        tols[1][i] = tl + ((rel + 2.0 ** -22) * -s + 2.0 ** -22 * s2 - s / (1 + r) * (rel * r + 2.0 ** -22 * -s)) / (1 + r) + 2.0 ** -23 * ent[i] + 2.0 ** -140
        order = np.argsort(-np.where(z[i] == 0, 0.0, z[i]), kind="stable")[:top]
        order = order[z[i][order] > -np.inf]
        ids[i, :len(order)] = order

        def one(x):
            return (x - m) - lse, tl + 2.0 ** -23 * (abs(x - m) + abs((x - m) - lse)) + 2.0 ** -140
        for j, t in enumerate(order):
            best[i, j], tols[2][i, j] = one(z[i, t])
        for j, t in enumerate(tokens[i]):
            if 0 <= t < vocab and z[i, t] > -np.inf:
                lp[i, j], tols[0][i, j] = one(z[i, t])
    return (lp, ent, ids, best), tols


def agree(got, want, tols):
    lp, ent, ids, best = (x.cpu().double().numpy() for x in got)
    assert np.array_equal(ids, want[2]), f"ids differ at {np.argwhere(ids != want[2])[:4].tolist()}"
    for name, a, b, tol in (("logprob", lp, want[0], tols[0]), ("entropy", ent, want[1], tols[1]), ("top", best, want[3], tols[2])):
        a = a.reshape(b.shape)
        with np.errstate(invalid="ignore"):
            ok = (a == b) | (np.abs(a - b) <= tol)
        assert ok.all(), f"{name}: {(~ok).sum()} off at {np.argwhere(~ok)[:3].tolist()}: {a[~ok][:3]} for {b[~ok][:3]} within {tol[~ok][:3]}"


def check(lib, z, tokens, top, **kw):
    import torch
    got = lib.logprobs(z, torch.from_numpy(tokens).cuda(), top=top, **kw)
    agree(got, *model(z.cpu().double().numpy(), tokens, top))
    return got


def logits(rows, vocab, dtype, seed=0, stride=None, offset=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    stride = stride or vocab
    b = torch.full((rows * stride + offset + 16,), float("nan"), dtype=getattr(torch, dtype))
    z = b[offset:offset + rows * stride].view(rows, stride)[:, :vocab]
    z.copy_(torch.randn(rows, vocab, generator=g) * 3 + 9 * (torch.rand(rows, vocab, generator=g) < 0.001))
    b = b.cuda()
    return b[offset:offset + rows * stride].view(rows, stride)[:, :vocab]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,vocab,top,given,stride,offset", [
    (1, 1, 1, 1, None, 0), (1, 7, 5, 2, None, 3), (2, 100, 32, 1, 103, 1), (3, 4096, 20, 3, None, 0), (1, 32000, 5, 1, None, 0),
    (5, 4097, 1, 1, None, 1), (2, 32016, 20, 4, None, 0), (1, 128257, 32, 300, None, 5), (40, 1001, 3, 1, 1003, 2), (700, 257, 20, 1, None, 0),
    (160, 20011, 32, 1, None, 0), (9, 15, 15, 1, 17, 0), (1, 70003, 0, 1, None, 0)])
def test_rows(lib, dtype, rows, vocab, top, given, stride, offset):
    z = logits(rows, vocab, dtype, rows + vocab, stride, offset)
    g = np.random.default_rng(1)
    tokens = g.integers(0, vocab, (rows, given)).astype(np.int32)
    if given > 2:
        tokens[0, 1], tokens[0, 2] = -1, vocab               # outside the vocabulary: cannot occur
    check(lib, z, tokens, top)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_ties_go_to_the_lowest_index(lib, dtype):
    """Constant rows, few levels, zeros of both signs, equal values at both ends of a row."""
    import torch
    g = np.random.default_rng(2)
    z = logits(6, 33001, dtype)
    z[0] = 1.5
    z[1] = torch.from_numpy(g.integers(0, 3, 33001).astype(np.float32)).to(z)
    z[2, ::2], z[2, 1::2] = 0.0, -0.0
    z[3, :] = -100.0
    z[3, 33000], z[3, 0], z[3, 16500] = 4.0, 4.0, 4.0
    z[4] = torch.arange(33001, 0, -1).to(z) / 1000
    z[5] = torch.arange(33001).to(z) / 1000
    check(lib, z, g.integers(0, 33001, (6, 1)).astype(np.int32), 32)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("vocab", [50, 9001, 40001])
def test_masked_tokens(lib, dtype, vocab):
    """Masks by -infinity and by the type's lowest value, a row that they leave nothing of, one that they leave one token of."""
    import torch
    low = float(torch.finfo(getattr(torch, dtype)).min)
    z = logits(8, vocab, dtype)
    z[0] = -math.inf
    z[1] = low
    z[2] = -math.inf
    z[2, vocab - 1] = -3.0
    z[3, 10:] = low
    z[4, 1:] = -math.inf
    z[5, ::3] = -math.inf
    z[6, : vocab - 2] = low
    z[7, 5:] = low
    z[7, :5] = -math.inf
    tokens = np.array([[0, 1], [0, 1], [vocab - 1, 0], [3, 20], [0, 1], [1, 3], [vocab - 1, 0], [7, 0]], dtype=np.int32)
    check(lib, z, tokens, 20)


def test_probabilities_near_one(lib):
    """A token that has all but 2^-20 .. 2^-60 of the probability keeps its logarithm's bits."""
    import torch
    z = torch.full((4, 32000), -80.0, device="cuda")
    for i, gap in enumerate((14, 20, 30, 41)):
        z[i, 777] = 3.0
        z[i, 31999 - i] = 3.0 - gap
    tokens = np.array([[777]] * 4, dtype=np.int32)
    got = check(lib, z, tokens, 3)
    assert torch.all(got[0] < 0)


def test_values_that_are_not_numbers(lib):
    """A NaN or +infinity makes a row's numbers NaN, the other rows' not; the order leaves NaN out."""
    import torch
    z = logits(5, 12345, "float32")
    clean = z.clone()
    z[1, 400] = float("nan")
    z[3, 12344] = float("inf")
    z[4] = float("nan")
    tokens = torch.zeros(5, 1, dtype=torch.int32, device="cuda")
    lp, ent, ids, best = lib.logprobs(z, tokens, top=6)
    keep = [0, 2]
    want, tols = model(clean[keep].cpu().double().numpy(), np.zeros((2, 1), np.int32), 6)
    agree((lp[keep], ent[keep], ids[keep], best[keep]), want, tols)
    for i in (1, 3, 4):
        assert torch.isnan(lp[i]).all() and torch.isnan(ent[i]) and torch.isnan(best[i]).all()
    order = clean[1].clone()
    order[400] = -math.inf
    assert ids[1].tolist() == torch.sort(order, descending=True, stable=True).indices[:6].tolist()
    assert ids[3, 0] == 12344 and ids[4].tolist() == [-1] * 6


def test_forms_of_the_call(lib):
    """Without tokens, without alternatives, one token a row, outputs of the caller's, another stream, a graph, no rows."""
    import torch
    z = logits(3, 5000, "bfloat16")
    tokens = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    lp, ent, ids, best = lib.logprobs(z, tokens, top=4)
    assert lp.shape == (3,) and ids.shape == (3, 4)
    none = lib.logprobs(z)
    assert none[0] is None and torch.equal(none[1], ent) and none[2].shape == (3, 0)
    out = tuple(torch.empty_like(x) for x in (lp, ent, ids, best))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert lib.logprobs(z, tokens, top=4, out=out) is out
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = lib.logprobs(z, tokens, top=4, stream=side)
    side.synchronize()
    for a, b, c in zip((lp, ent, ids, best), out, other):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert lib.logprobs(z[:0], tokens[:0], top=2)[2].shape == (0, 2)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,vocab,top", [(1300, 2050, 20), (1301, 5003, 32), (2500, 200, 7), (3000, 1024, 1)])
def test_many_rows(lib, dtype, rows, vocab, top):
    """More rows than the GPU holds at a time: some of them against the definition, all against the same rows in small calls."""
    import torch
    z = logits(rows, vocab, dtype, rows)
    z[5] = z[6]
    tokens = torch.from_numpy(np.random.default_rng(3).integers(0, vocab, (rows, 2)).astype(np.int32)).cuda()
    got = lib.logprobs(z, tokens, top=top)
    some = torch.tensor([0, 1, 5, 6, rows // 2, rows - 1], device="cuda")
    agree([x[some] for x in got], *model(z[some].cpu().double().numpy(), tokens[some].cpu().numpy(), top))
    for i in range(0, rows, 100):
        part = lib.logprobs(z[i:i + 100], tokens[i:i + 100], top=top)
        assert torch.equal(part[2], got[2][i:i + 100])
        for a, b in zip(part, got):
            torch.testing.assert_close(a, b[i:i + 100], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("rows,vocab", [(120, 32003), (3, 250001), (70, 60000)])
def test_long_rows_in_parts(lib, rows, vocab):
    """Rows that two to eight blocks share, some of them two on an SM."""
    z = logits(rows, vocab, "bfloat16", 5)
    got = lib.logprobs(z, top=32)
    some = [0, rows // 2, rows - 1]
    want, tols = model(z[some].cpu().double().numpy(), np.zeros((3, 0), np.int32), 32)
    agree([z.new_zeros(3, 0), got[1][some], got[2][some], got[3][some]], want, tols)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("top", [1, 5, 32])
@pytest.mark.parametrize("rows,vocab,warps", [(160, 20000, 8), (1200, 20000, 4), (1300, 2500, 2)])
def test_zeros_that_tie_behind_the_first_pass(lib, dtype, top, rows, vocab, warps):
    """Zeros of both signs as a row's best, none of them in the first pass of a block's warps: the lowest indices whatever
    warp is ahead.  In each row one warp has more to sort in the first pass, so that it comes late to the lowest zeros, and
    the others have many."""
    import torch
    vec, lanes = 128 // torch.finfo(getattr(torch, dtype)).bits, 32
    first = 16 * lanes * warps                                # elements of a pass: 16 of each thread, `vec` at a time
    g = torch.Generator().manual_seed(top + warps)
    z = -10 - torch.rand(rows, vocab, generator=g)
    zero = torch.zeros(rows, vocab, dtype=torch.bool)
    index = torch.arange(vocab)
    owner, part = index // vec // lanes % warps, index // vec // (lanes * warps) % (16 // vec)
    for r in range(rows):
        late = warps - 1 - r % min(warps, 4) if warps > 1 else 0
        busy = (index < first) & (owner == late)
        z[r, busy] = torch.linspace(-1, -0.9, int(busy.sum()))
        few = (index >= first) & (index < 2 * first) & (owner == late) & (part == 0)
        zero[r] = few & (torch.rand(vocab, generator=g) < 0.05) | (index >= first) & (part > 0) & (owner != late) & (torch.rand(vocab, generator=g) < 0.5)
    signs = torch.where(torch.rand(rows, vocab, generator=g) < 0.5, 0.0, -0.0)
    z = torch.where(zero, signs, z).to(getattr(torch, dtype))
    assert int(zero.sum(1).min()) >= 32
    want = torch.where(zero, index, vocab).sort(1).values[:, :top].int()
    z = z.cuda()
    for _ in range(5):
        ids = lib.logprobs(z, top=top)[2].cpu()
        wrong = (ids != want).any(1)
        assert not wrong.any(), f"{int(wrong.sum())} of {rows} rows, the first {int(wrong.nonzero()[0])}: {ids[wrong][0].tolist()} for {want[wrong][0].tolist()}"


def test_more_logits_than_31_bits_count(lib):
    """The last of 2^31 + 2^18 logits, bf16, in rows at a stride: rows at both ends of it as by themselves."""
    import torch
    rows, vocab, stride = 8194, 262000, 262144
    z = torch.full((rows, stride), -3.0, dtype=torch.bfloat16, device="cuda")[:, :vocab]
    some = [0, 4097, rows - 2, rows - 1]
    z[some] = logits(4, vocab, "bfloat16", 9)
    tokens = torch.full((rows, 1), vocab - 1, dtype=torch.int32, device="cuda")
    got = lib.logprobs(z, tokens, top=8)
    agree([x[some] for x in got], *model(z[some].cpu().double().numpy(), tokens[some].cpu().numpy(), 8))
    assert torch.all(got[2][1:4097] == torch.arange(8, device="cuda", dtype=torch.int32))
