"""A model's decoding steps over the operators together: products with 4-bit weights, norm and rotation, attention with a window
over the 8-bit cache, append, and the log probabilities of what comes next.  Each operator is checked against its formula in
64 bits on what it was given, and the steps from a graph against those without."""
from types import SimpleNamespace

import numpy as np
import pytest

from helpers import ensure_built
from test_gpu_kv8_window import model as attention_model
from test_gpu_logprobs import agree, model as logprobs_model
from test_gpu_norm_rope import close, formula, frequencies

pytestmark = pytest.mark.gpu
D, HEADS, KV, HD, VOCAB, LAYERS, GROUP, EPS, BASE = 256, 8, 2, 64, 1003, 2, 32, 1e-5, 10000.0
WIDTH = (HEADS + 2 * KV) * HD


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import exact_decoding_gb300 as e
    return e


def product(x, m):
    """x W^T in 64 bits and its tolerance, as test_gpu_w4.case derives it."""
    w = m.w.cpu().numpy()
    q = np.stack([w & 15, w >> 4], -1).reshape(m.out, m.k).astype(np.float64)
    s = np.repeat(m.scales.cpu().double().numpy(), m.group, 1)
    x = x.cpu().double().numpy()
    size, a = np.abs(x) @ s.T, np.abs(x) @ np.abs((q - 8) * s).T
    return x @ ((q - 8) * s).T, 23 * size * (m.group / 16 * 17 * 2.0 ** -23 + (m.group + 8) * 2.0 ** -24) + a * (m.k // m.group + 68) * 2.0 ** -24


class Model:
    """Weights, a cache whose sequences hold `lens` tokens, and the buffers of a step."""

    def __init__(self, lib, lens, window, sinks, page=32):
        import torch
        g = torch.Generator().manual_seed(11)
        self.lib, self.window, self.sinks, self.n = lib, window, sinks, len(lens)

        def matrix(out, k):
            w = torch.randint(0, 256, (out, k // 2), generator=g, dtype=torch.uint8)
            s = (torch.rand(out, k // GROUP, generator=g) + 0.5) / (4 * k ** 0.5)
            return lib.W4Matrix(w.cuda(), s.to(torch.bfloat16).cuda())
        self.embed = torch.randn(VOCAB, D, generator=g).to(torch.bfloat16).cuda()
        self.qkv, self.out = [matrix(WIDTH, D) for _ in range(LAYERS)], [matrix(D, HEADS * HD) for _ in range(LAYERS)]
        self.head = matrix(VOCAB, D)
        self.gains = [[(1 + 0.2 * torch.randn(HD, generator=g)).cuda() for _ in range(2)] for _ in range(LAYERS)]
        pages = -(-(max(lens) + 8) // page)
        self.cache = lib.Kv8Cache(LAYERS, self.n * pages, page, KV, HD, self.n, pages)
        self.rows = [torch.zeros(LAYERS, self.n, KV, HD, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        if max(lens):
            starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
            k, v = (torch.randn(LAYERS, sum(lens), KV, HD, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
            self.cache.append(k, v, row_start=starts)
        self.tokens = torch.arange(self.n, dtype=torch.int32, device="cuda")

    def step(self, seen=None):
        """The next token of every sequence; seen(name, inputs, outputs) looks at each operator's call."""
        import torch
        c, seen = self.cache, seen or (lambda *a: None)
        x = self.embed[self.tokens.long()]
        for i in range(LAYERS):
            y = self.qkv[i].matvec(x)
            seen("product", (x, self.qkv[i]), y)
            parts = [p.unflatten(1, (-1, HD)) for p in y.split([HEADS * HD, KV * HD, KV * HD], 1)]
            q = torch.empty(self.n, HEADS, HD, dtype=torch.bfloat16, device="cuda")
            k, v = self.rows[0][i], self.rows[1][i]
            c.norm_rope(*parts, q_weight=self.gains[i][0], k_weight=self.gains[i][1], eps=EPS, rope_base=BASE, out=(q, k, v))
            seen("rotate", (parts, self.gains[i]), (q, k, v))
            o = c.attention(q, k, v, layer=i, window=self.window, sinks=self.sinks, max_rows=1)
            seen("attend", (i, q, k, v), o)
            z = self.out[i].matvec(o.flatten(1))
            seen("product", (o.flatten(1), self.out[i]), z)
            x = (x.float() + z).to(torch.bfloat16)
        c.append(*self.rows)
        logits = self.head.matvec(x)
        seen("product", (x, self.head), logits)
        scores = self.lib.logprobs(logits, self.tokens, top=5)
        seen("score", (logits, self.tokens.clone()), scores)
        self.tokens.copy_(scores[2][:, 0])
        return logits, *scores


@pytest.mark.parametrize("lens,window,sinks", [([70, 0, 33], 40, 4), ([0], 1, 0), ([130], 64, 64), ([5, 200, 31, 64, 90, 2, 17], 100, 3)])
def test_steps(lib, lens, window, sinks):
    m = Model(lib, lens, window, sinks)
    for _ in range(3):
        places = m.cache.lens.cpu().numpy().copy()

        def seen(name, given, got):
            if name == "product":
                close(got, *product(*given))
            elif name == "rotate":
                (q, k, v), (qw, kw) = given
                close(got[0], *formula(q, qw, places, EPS, frequencies(BASE, HD)))
                close(got[1], *formula(k, kw, places, EPS, frequencies(BASE, HD)))
                close(got[2], v.cpu().double().numpy(), 2.0 ** -8 * np.abs(v.cpu().double().numpy()))
            elif name == "attend":
                i, q, k, v = given
                c = m.cache
                one = SimpleNamespace(k=c.k[i:i + 1], v=c.v[i:i + 1], k_scale=c.k_scale[i:i + 1], v_scale=c.v_scale[i:i + 1], table=c.table, lens=c.lens,
                                      page=c.page, n_kv_heads=KV)
                close(got, *attention_model(one, q, k, v, [1] * m.n, window, sinks))
            else:
                agree(got, *logprobs_model(given[0].cpu().double().numpy(), given[1].cpu().numpy()[:, None], 5))
        m.step(seen)
        m.cache.status()
    assert m.cache.lens.tolist() == [n + 3 for n in lens]
    lib.la_gemm_status()


def test_steps_from_a_graph(lib):
    """The whole step captured: every replay gives the bits of the step without a graph, the sequences growing past a page."""
    import torch
    a, b = (Model(lib, [63, 0, 30], 40, 4) for _ in range(2))
    want = [a.step() for _ in range(4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                             # one step without a graph first, as a program warms up
        got = [b.step()]
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.step()
    for _ in range(3):
        graph.replay()
        got.append([t.clone() for t in out])
    b.cache.status()
    for x, y in zip(want, got):
        assert all(torch.equal(s, t) for s, t in zip(x, y))
    assert torch.equal(a.cache.lens, b.cache.lens)


def test_two_models_at_once(lib):
    """Steps of two models on two streams, none waiting for the other: the bits of the same steps one after another."""
    import torch
    shapes = [([63, 0, 30], 40, 4), ([700, 90], 300, 0)]
    want = [[m.step() for _ in range(4)] for m in (Model(lib, *s) for s in shapes)]
    models, streams = [Model(lib, *s) for s in shapes], [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for m, stream, steps in zip(models, streams, got):
            with torch.cuda.stream(stream):
                steps.append(m.step())
    torch.cuda.synchronize()
    for m, w, g in zip(models, want, got):
        m.cache.status()
        for x, y in zip(w, g):
            assert all(torch.equal(s, t) for s, t in zip(x, y))
