"""Products with 4-bit weights (W4Matrix, la_gemv_w4) against their formula in 64 bits."""
import numpy as np
import pytest

from helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import exact_decoding_gb300 as e
    return e


def case(rows, out, k, group, seed=0, device="cuda"):
    """x, packed weights and scales on the GPU, with y and its tolerance in 64 bits.

    Tolerance: products of a bf16 number and a whole number of four bits are exact in
    fp32 (x is, to 2^-39 of its group's largest value).  One matrix product adds 16
    of them to a sum and may cut each term at 2^-23 of the largest, so it is off
    by 17 * 2^-23 of the terms' magnitudes at most; a group takes group / 16 of
    them.  q - 8 is 8 at most and 0 in one of 16 cases: 23 times the group's |x| bounds the
    magnitudes, also for a kernel that adds q x and -8 times the sum of x, which
    rounds by (group + 8) * 2^-24 of them.  The group's power is exact, its scale, the sum over the groups and over at most 64 parts
    of k round by 2^-24 each."""
    import torch
    g = np.random.default_rng(seed)
    x = torch.from_numpy(g.standard_normal((rows, k)) * np.exp(g.standard_normal((1, k)))).to(torch.bfloat16)
    q = g.integers(0, 16, (out, k), dtype=np.uint8)
    s = torch.from_numpy(np.exp(g.standard_normal((out, k // group))) * 0.01).to(torch.bfloat16)
    w = torch.from_numpy(q[:, ::2] | (q[:, 1::2] << 4))
    m = (q.astype(np.float64) - 8) * np.repeat(s.double().numpy(), group, 1)
    xd = x.double().numpy()
    y, a = xd @ m.T, np.abs(xd) @ np.abs(m).T
    size = np.abs(xd) @ np.repeat(s.double().numpy(), group, 1).T
    return x.to(device), w.to(device), s.to(device), y, 23 * size * (group / 16 * 17 * 2.0 ** -23 + (group + 8) * 2.0 ** -24) + a * (k // group + 68) * 2.0 ** -24


def close(got, want, tol):
    d = np.abs(got.cpu().double().numpy() - want)
    assert np.all(d <= tol), f"{(~(d <= tol)).sum()} of {d.size} off, worst {np.nanmax(d / tol):.3g} of the tolerance at {np.argwhere(~(d <= tol))[:3].tolist()}"


@pytest.mark.parametrize("rows,out,k,group", [
    (1, 1, 32, 32), (1, 16, 128, 128), (1, 17, 96, 32), (2, 33, 192, 64), (1, 300, 4096, 128), (8, 129, 640, 128), (9, 100, 1600, 64),
    (16, 257, 1056, 32), (3, 4096, 512, 128), (5, 1000, 5120, 64), (17, 64, 256, 128), (33, 48, 384, 64), (256, 20, 128, 32),
    (1, 5000, 128, 128), (16, 3, 28672, 128), (7, 2500, 2080, 32), (6, 129, 8192, 128), (1, 9, 28672, 32), (6, 200, 28672, 64), (40, 130, 4160, 64),
    (7, 128, 96, 32), (12, 5000, 416, 32), (2, 12000, 288, 32)])
def test_products(lib, rows, out, k, group):
    x, w, s, y, tol = case(rows, out, k, group, seed=rows + out)
    m = lib.W4Matrix(w, s)
    close(m.matvec(x), y, tol)
    if rows == 1:
        close(m.matvec(x[0]).view(1, -1), y, tol)


def test_strides_and_order(lib):
    """Rows of a wider buffer, and outputs into one, whose other columns stay as they were."""
    import torch
    x, w, s, y, tol = case(6, 70, 256, 64)
    wide = torch.full((6, 300), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:264] = x
    out = torch.full((6, 99), -7.0, device="cuda")
    got = lib.W4Matrix(w, s).matvec(wide[:, 8:264], out=out[:, 5:75]) if (wide.data_ptr() + 16) % 16 == 0 and 300 % 8 == 0 else None
    if got is None:                                          # 300 is no multiple of 8: refused
        with pytest.raises(lib.LaError):
            lib.W4Matrix(w, s).matvec(wide[:, 8:264], out=out[:, 5:75])
        wide = torch.full((6, 304), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 8:264] = x
        got = lib.W4Matrix(w, s).matvec(wide[:, 8:264], out=out[:, 5:75])
    close(got, y, tol)
    assert torch.all(out[:, :5] == -7) and torch.all(out[:, 75:] == -7)


def test_values_that_are_not_finite(lib):
    """They reach their own row alone, everywhere in it (0 times infinity is NaN as well)."""
    import torch
    x, w, s, y, tol = case(4, 40, 256, 128)
    x[2, 77] = float("inf")
    got = lib.W4Matrix(w, s).matvec(x)
    keep = [0, 1, 3]
    close(got[keep], y[keep], tol[keep])
    assert not torch.isfinite(got[2]).any()


def test_repeats_and_graphs(lib):
    """The same bits every time: alone, on another stream, and replayed from a graph with new vectors."""
    import torch
    x, w, s, y, tol = case(3, 900, 1024, 128)
    m = lib.W4Matrix(w, s)
    first = m.matvec(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = m.matvec(x, stream=side)
    side.synchronize()
    assert torch.equal(first, other)
    out, xin = torch.empty_like(first), torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.matvec(xin, out=out)
    xin.copy_(x)
    graph.replay()
    assert torch.equal(first, out)
    assert lib.W4Matrix(w, s).matvec(x[:0]).shape == (0, 900)


@pytest.mark.parametrize("rows", [3, 16])
def test_values_of_all_sizes(lib, rows):
    """Groups of x many binades apart, the smallest and largest bf16 values, scales likewise: each group to its own bits."""
    import torch
    g = np.random.default_rng(5)
    k, out, group = 1024, 50, 64
    x = g.standard_normal((rows, k)) * 2.0 ** np.repeat(g.integers(-60, 60, (rows, k // group)), group, 1)
    x[:, 3] = 0
    x[0, 64:128] = 2.0 ** -133
    x = torch.from_numpy(x).to(torch.bfloat16)
    q = g.integers(0, 16, (out, k), dtype=np.uint8)
    s = torch.from_numpy(2.0 ** g.integers(-40, 40, (out, k // group)).astype(np.float64)).to(torch.bfloat16)
    w = torch.from_numpy(q[:, ::2] | (q[:, 1::2] << 4))
    m = (q.astype(np.float64) - 8) * np.repeat(s.double().numpy(), group, 1)
    xd = x.double().numpy()
    size = np.abs(xd) @ np.repeat(s.double().numpy(), group, 1).T
    got = lib.W4Matrix(w.cuda(), s.cuda()).matvec(x.cuda())
    close(got, xd @ m.T, 23 * size * (4 * 17 * 2.0 ** -23 + 72 * 2.0 ** -24) + 23 * size * 84 * 2.0 ** -24 + 2.0 ** -100)


def test_workspace(lib):
    """Too small a workspace is refused; calls of few rows need none."""
    x, w, s, y, tol = case(16, 300, 512, 128)
    need = lib.la_gemv_w4_workspace(16, 300, 512, 128)
    assert need > 0 and lib.la_gemv_w4_workspace(1, 300, 512, 128) == 0 and lib.la_gemv_w4_workspace(0, 300, 512, 128) == 0
    with pytest.raises(lib.LaError) as err:
        lib.la_gemv_w4(x.data_ptr(), 512, w.data_ptr(), s.data_ptr(), x.data_ptr(), 300, 16, 300, 512, 128, w.data_ptr(), need - 1)
    assert err.value.code == -3
    lib.la_gemm_status()


def test_calls_at_once(lib):
    """Two streams use one matrix, each with workspaces of its own."""
    import torch
    x, w, s, y, tol = case(16, 3000, 4096, 128)
    m = lib.W4Matrix(w, s)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    outs = [[m.matvec(x if i % 2 else x[:5], stream=st) for i in range(10)] for st in streams]
    torch.cuda.synchronize()
    for o in outs:
        for i, got in enumerate(o):
            n = 16 if i % 2 else 5
            close(got, y[:n], tol[:n])
    lib.la_gemm_status()


@pytest.mark.parametrize("rows,out,k,group", [
    (1, 11008, 1024, 128), (2, 13800, 768, 128), (1, 24300, 384, 128), (1, 11008, 1056, 32), (3, 5000, 4128, 32), (4, 7100, 2240, 64),
    (6, 1900, 3200, 128), (1, 2000, 8736, 32), (2, 100, 11232, 32),
    (16, 130, 32, 32), (7, 3, 64, 64)])
def test_products_shared_unevenly(lib, rows, out, k, group):
    """Numbers of outputs for which 3, 5, 6 or 8 blocks share k, whose groups do not divide evenly; matrices of one group."""
    x, w, s, y, tol = case(rows, out, k, group, seed=rows + out)
    close(lib.W4Matrix(w, s).matvec(x), y, tol)


@pytest.mark.parametrize("rows,out,k,group", [(1, 2000, 4096, 128), (5, 900, 5120, 64), (2, 700, 2784, 32), (16, 512, 8192, 128), (9, 512, 4096, 32), (3, 256, 28672, 128)])
def test_sums_keep_their_bits(lib, rows, out, k, group):
    """Weights near 0, as they are in a model, and some strong channels: off by 2^-21 of the results' size at most.

    Size: the 2-norm over the rows and outputs.  Terms of random sign add up like a random walk, whose mean square is
    half of its end's, and a rounding to 2^-24 of a sum is 2^-24 / sqrt(3) of it in the mean square at most.  So n = k / group
    + 64 <= 288 rounded additions are off by 2^-24 sqrt(n / 6) = 4.1e-7 together, and the products of a group, up to 8 after one
    another at 2^-23, by 2^-23 sqrt(8 / 6) = 1.4e-7; both: 4.4e-7, below 2^-21."""
    import torch
    g = torch.Generator().manual_seed(k)
    q = (torch.randn(out, k, generator=g) * 2.7).round().clamp(-8, 7)
    w = (q + 8).to(torch.uint8)
    s = (torch.exp(0.4 * torch.randn(out, k // group, generator=g)) * 0.007).to(torch.bfloat16)
    x = (torch.randn(rows, k, generator=g) * (1 + 15 * (torch.rand(1, k, generator=g) < 0.01))).to(torch.bfloat16)
    want = x.double() @ (q.double() * s.double().repeat_interleave(group, 1)).T
    got = lib.W4Matrix((w[:, ::2] | w[:, 1::2] << 4).cuda(), s.cuda()).matvec(x.cuda()).cpu().double()
    assert (got - want).norm() <= 2.0 ** -21 * want.norm()


def test_two_graphs_with_workspaces(lib):
    """Calls of many rows in two captured graphs, replayed in turn and on two streams at once: each has a workspace of its own."""
    import torch
    cases = [case(16, 700, 2048, 128, seed=1), case(40, 900, 1024, 64, seed=2)]
    assert all(lib.la_gemv_w4_workspace(x.shape[0], w.shape[0], x.shape[1], 2 * w.shape[1] // s.shape[1]) > 0 for x, w, s, _, _ in cases)
    matrices = [lib.W4Matrix(w, s) for _, w, s, _, _ in cases]
    want = [m.matvec(c[0]) for m, c in zip(matrices, cases)]
    torch.cuda.synchronize()
    inputs, graphs, outs = [torch.zeros_like(c[0]) for c in cases], [], []
    for m, x in zip(matrices, inputs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(m.matvec(x))
    for x, c in zip(inputs, cases):
        x.copy_(c[0])
    for g in (0, 1, 1, 0):
        graphs[g].replay()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for out, w, c in zip(outs, want, cases):
        assert torch.equal(out, w)
        close(out, c[3], c[4])
    lib.la_gemm_status()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows", [1, 8, 9, 17])
@pytest.mark.parametrize("x_least,x_most,s_least,s_most", [(110, 127, -60, -24), (-133, -126, 20, 60), (100, 127, -126, -100), (-120, -100, 80, 100)])
def test_extreme_values(lib, group, rows, x_least, x_most, s_least, s_most):
    """bf16's largest and smallest values with scales that bring the results back: every group to the bits of its own size,
    though its sum before the scale may be far outside fp32's range.  Tolerance: as in case(), of these rows alone."""
    import torch
    g = np.random.default_rng(rows + group)
    k, out = 8 * group, 50
    x = g.choice([-1.0, 1.0], (rows, k)) * 2.0 ** g.integers(x_least, x_most + 1, (rows, k)) * (1 if x_least < -126 else g.integers(128, 256, (rows, k)) / 128)
    x = torch.from_numpy(x).to(torch.bfloat16)
    q = g.integers(0, 16, (out, k), dtype=np.uint8)
    q[0], q[1] = 0, np.where(x[0].double().numpy() > 0, 15, 0)          # sums that nothing takes back
    s = torch.from_numpy(2.0 ** g.integers(s_least, s_most + 1, (out, k // group)).astype(np.float64)).to(torch.bfloat16)
    w = torch.from_numpy(q[:, ::2] | (q[:, 1::2] << 4))
    m = (q.astype(np.float64) - 8) * np.repeat(s.double().numpy(), group, 1)
    xd = x.double().numpy()
    assert np.isfinite(xd).all()
    size = np.abs(xd) @ np.repeat(s.double().numpy(), group, 1).T
    tol = 23 * size * (group / 16 * 17 * 2.0 ** -23 + (group + 8) * 2.0 ** -24) + np.abs(xd) @ np.abs(m).T * (k // group + 68) * 2.0 ** -24
    close(lib.W4Matrix(w.cuda(), s.cuda()).matvec(x.cuda()), xd @ m.T, tol)


def test_one_large_value(lib):
    """x = 2^126 times -8: infinity before its scale of 2^-7, -2^122 behind it; groups of opposite sign take each other back."""
    import torch
    for rows in (1, 16):
        x = torch.zeros(rows, 256, dtype=torch.bfloat16, device="cuda")
        x[:, 5], x[:, 133] = 2.0 ** 126, -2.0 ** 126
        w = torch.full((2, 128), 0x88, dtype=torch.uint8, device="cuda")
        w[:, 2] = 0x08                                       # column 5: 0, column 4: 8
        w[1, 66] = 0x08                                      # column 133 likewise
        s = torch.full((2, 2), 2.0 ** -7, dtype=torch.bfloat16, device="cuda")
        y = lib.W4Matrix(w, s).matvec(x)
        assert torch.all(y[:, 0] == -2.0 ** 122) and torch.all(y[:, 1] == 0)


def test_a_stride_that_is_refused(lib):
    """Rows 300 apart: no multiple of 8."""
    import torch
    x, w, s, _, _ = case(6, 70, 256, 64)
    wide = torch.zeros(6, 300, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(lib.LaError, match="x_stride"):
        lib.W4Matrix(w, s).matvec(wide[:, 8:264])


@pytest.mark.parametrize("rows,out,k,group", [(41, 200, 512, 64), (64, 129, 1024, 128), (100, 70, 4160, 64), (121, 500, 2048, 128), (129, 33, 96, 32), (255, 140, 640, 128)])
def test_rows_between(lib, rows, out, k, group):
    """A step's rows and other numbers between 40 and 256, ragged in the last sixteen."""
    x, w, s, y, tol = case(rows, out, k, group, seed=rows)
    close(lib.W4Matrix(w, s).matvec(x), y, tol)
    lib.la_gemm_status()


@pytest.mark.parametrize("rows", [1, 16])
def test_more_bytes_than_31_bits_count(lib, rows):
    """A matrix of 2.2 GB: its first, middle and last outputs against the same rows as a matrix of their own."""
    import torch
    out, k, group = 131100, 32768, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randint(0, 256, (out, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = (torch.rand(out, k // group, device="cuda", generator=g) * 0.01).to(torch.bfloat16)
    x = torch.randn(rows, k, device="cuda", generator=g).to(torch.bfloat16)
    assert w.numel() > 1 << 31
    got = lib.W4Matrix(w, s).matvec(x)
    xd = x.double()
    for a in (0, 65500, out - 60):
        part, scales = w[a:a + 60], s[a:a + 60].double().repeat_interleave(group, 1)
        q = torch.stack([part & 15, part >> 4], 2).view(60, k).double() - 8
        want, size = xd @ (q * scales).T, xd.abs() @ scales.T
        assert torch.all((got[:, a:a + 60].double() - want).abs() <= 23 * size * (group / 16 * 17 * 2.0 ** -23 + (group + 8) * 2.0 ** -24 + (k // group + 68) * 2.0 ** -24))
    lib.la_gemm_status()
