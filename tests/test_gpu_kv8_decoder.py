"""Decoders over the paged 8-bit cache (la_create_kv8, la_fork) on small bf16
models: teacher-forced steps against the oracle, prompt chunks, forks, a full
pool, pages moved between steps.

The oracle runs in 64 bits on the keys and values that the decoder's slot
holds, and rounds what this path rounds: q, the pass's own k and v and the
attention's output to bf16 (torch's rounding).  What then remains is the bf16
decoder's own error, whose contract is 2e-2 on logits, as without the cache.

Cached values: an e4m3 rounding is off by at most 2^-4 of the value or 2^-10
of the page's scale; a page whose scale grows later is rounded a second time.
The value that is rounded differs from the oracle's by flips of the bf16
roundings (one step, 2^-7 of the value at most: 2^-8 on either side) in this
layer and in what the layers below feed it, as a fraction of values of order
one: 2^-7 |x| + 2^-8 together."""
import numpy as np
import pytest
import torch

import kv8_model as M
import synth
from helpers import MARGIN, Tally, check_step, ensure_built, top2_margin
from oracle import decoder, lookahead as la

pytestmark = pytest.mark.gpu
TOL = 2e-2
CAPACITY, STATE, INVALID = -3, -6, -1

SMALL = {
    "mha-hd64": synth.ModelDims(2, 256, 4, 4, 64, 688, 1024, dtype="bf16"),
    "gqa-hd128": synth.ModelDims(2, 512, 8, 2, 128, 1024, 2048, dtype="bf16"),
    "mha-hd128-3l": synth.ModelDims(3, 512, 4, 4, 128, 1376, 1536, dtype="bf16"),
}


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import exact_decoding_gb300 as e
    return e


def weights(name, seed):
    d = SMALL[name]
    return synth.model_weights(d, seed, lm_head_std=1.28 / np.sqrt(d.d_model))


def new_cache(lib, dims, page, n_seqs=3, max_seq=1024, n_pages=None):
    per = -(-max_seq // page)
    return lib.Kv8Cache(dims.n_layers, n_pages or n_seqs * per, page, dims.n_kv_heads, dims.head_dim, n_seqs, per)


def slot_kv(cache, slot, n=None):
    """K, V [tokens, heads, dim] of a slot, per layer, and their scales."""
    ln = int(cache.lens[slot]) if n is None else n
    ids = cache.table[slot, :-(-ln // cache.page)].cpu().numpy()
    out, scales = [], []
    for l in range(cache.n_layers):
        kb, vb = M.E4M3[cache.k[l].cpu().numpy()[ids]], M.E4M3[cache.v[l].cpu().numpy()[ids]]
        ks, vs = cache.k_scale[l].cpu().double().numpy()[ids], cache.v_scale[l].cpu().double().numpy()[ids]
        K = (kb * ks[..., None, None]).transpose(0, 2, 1, 3).reshape(-1, cache.n_kv_heads, cache.head_dim)[:ln]
        V = (vb * vs[..., None, None]).transpose(0, 3, 1, 2).reshape(-1, cache.n_kv_heads, cache.head_dim)[:ln]
        out.append((K, V))
        scales.append([np.repeat(s, cache.page, axis=0)[:ln, :, None] for s in (ks, vs)])
    return out, scales


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


@pytest.fixture(autouse=True)
def rounded_attention(monkeypatch):
    plain = decoder.attention
    monkeypatch.setattr(decoder, "attention", lambda q, k, v, visible: bf16(plain(bf16(q), bf16(k), bf16(v), visible)))


def check_cached(got, scales, want):
    """Cached K, V of some tokens against the oracle's values of them."""
    for (K, V), (sk, sv), (k, v) in zip(got, scales, want):
        for a, s, x in ((K, sk, k), (V, sv, v)):
            tol = 2 * np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) + 2.0 ** -7 * np.abs(x) + 2.0 ** -8
            assert np.all(np.abs(a - x) <= tol), np.abs(a - x).max()


def load(orc, s0, cache, slot):
    orc.tokens = [int(t) for t in s0["tokens"]]
    orc.window = np.array(s0["window"], dtype=np.int64).reshape(orc.N - 1, orc.W)
    orc.pool = la.Pool.from_records(orc.pool.cap, s0["records"], orc.pool.policy)
    orc.cache, _ = slot_kv(cache, slot)
    assert len(orc.cache[0][0]) == orc.P


def forced_steps(dec, cache, slot, orc, steps, tally):
    for t in range(steps):
        s0 = dec.export_state()
        load(orc, s0, cache, slot)
        P = orc.P
        ref = orc.step()
        rec = orc.history[-1]
        acc = dec.step()
        logits = dec.debug_logits()
        s1 = dec.export_state()
        check_step(rec, acc, ref, logits, s0, s1, dec.N, dec.W, MARGIN, TOL, orc.pool.cap, "fifo", tally, where=f"step {t}")
        got, scales = slot_kv(cache, slot)
        assert len(got[0][0]) == P + len(acc)
        if acc == ref:
            cut = lambda x: [tuple(y[P:] for y in pair) for pair in x]  # noqa: E731
            check_cached(cut(got), cut(scales), cut(orc.cache))
    return tally


@pytest.mark.parametrize("name,page,n,N,W,G,steps,par", [
    ("mha-hd64", 32, 40, 4, 5, 3, 6, False),
    ("gqa-hd128", 64, 300, 5, 7, 7, 6, False),
    ("gqa-hd128", 128, 12, 4, 5, 3, 6, False),
    ("mha-hd128-3l", 128, 64, 5, 15, 15, 4, False),
    ("mha-hd64", 64, 72, 4, 4, 4, 12, True)])
def test_steps_follow_the_oracle(lib, name, page, n, N, W, G, steps, par):
    """Steps of 22 to 121 rows from 12 to 300 cached tokens; the last case
    repeats its prompt, so that candidates are accepted and appended."""
    dims = SMALL[name]
    w = weights(name, 3)
    p = np.tile(synth.uniform_tokens(12, dims.vocab, seed=8), 6)[:n] if par else synth.uniform_tokens(n, dims.vocab, seed=4)
    cache = new_cache(lib, dims, page)
    dec = lib.Decoder(w, N, W, G, 1024, prompt_as_reference=par, kv_cache=cache, slot=1)
    dec.prefill(p)
    orc = la.Lookahead(w, N, W, G, keep_logits=True, prompt_as_reference=par)
    t = forced_steps(dec, cache, 1, orc, steps, Tally())
    print(t)
    dec.close()
    assert 2 * t.accept_compared >= steps and 2 * t.columns_compared >= t.columns, t
    if par:
        assert t.accept_compared_multi >= 1, t
    assert cache.lens.tolist()[0::2] == [0, 0]
    cache.status()


@pytest.mark.parametrize("name,page,n", [("mha-hd64", 32, 40), ("gqa-hd128", 128, 256), ("gqa-hd128", 64, 300), ("mha-hd64", 128, 513)])
def test_prefill_follows_the_oracle(lib, name, page, n):
    """Each pass of up to 256 prompt tokens reads the earlier passes' tokens
    from the cache (whole pages: 256 is a multiple of the page)."""
    dims = SMALL[name]
    w = weights(name, 5)
    p = [int(t) for t in synth.uniform_tokens(n, dims.vocab, seed=6)]
    cache = new_cache(lib, dims, page)
    dec = lib.Decoder(w, 4, 5, 3, 1024, kv_cache=cache, slot=2)
    y = dec.prefill(p)
    got, scales = slot_kv(cache, 2)
    assert len(got[0][0]) == n
    for c0 in range(0, n, 256):
        rows = min(256, n - c0)
        past = [(k[:c0], v[:c0]) for k, v in got]
        logits, kv = decoder.forward(w, p[c0:c0 + rows], np.arange(c0, c0 + rows), decoder.causal_mask(c0, rows), cache=past,
                                     logit_rows=[rows - 1])
        check_cached([(k[c0:c0 + rows], v[c0:c0 + rows]) for k, v in got], [[s[c0:c0 + rows] for s in x] for x in scales], kv)
    assert np.abs(dec.debug_logits()[0] - logits[0]).max() <= TOL
    if top2_margin(logits[0]) > MARGIN:
        assert y == la.argmax_lowest(logits[0])
    dec.close()


def test_ar_steps_follow_the_oracle_and_mix_with_steps(lib):
    dims = SMALL["gqa-hd128"]
    w = weights("gqa-hd128", 13)
    p = [int(t) for t in synth.uniform_tokens(40, dims.vocab, 13, 7)]
    cache = new_cache(lib, dims, 32)
    dec = lib.Decoder(w, 4, 5, 4, 256, kv_cache=cache)
    toks = list(p) + [dec.prefill(p)]
    compared = 0
    for _ in range(6):
        P = len(toks) - 1
        past, _ = slot_kv(cache, 0)
        y = dec.ar_step()
        ref, kv = decoder.forward(w, toks[-1:], np.array([P]), np.ones((1, P + 1), bool), cache=past)
        assert np.abs(dec.debug_logits()[0] - ref[0]).max() <= TOL
        got, scales = slot_kv(cache, 0)
        assert len(got[0][0]) == P + 1
        check_cached([(k[P:], v[P:]) for k, v in got], [[s[P:] for s in x] for x in scales], kv)
        if top2_margin(ref[0]) > MARGIN:
            assert y == la.argmax_lowest(ref[0])
            compared += 1
        toks.append(y)
    assert compared >= 3
    orc = la.Lookahead(w, 4, 5, 4, keep_logits=True)
    forced_steps(dec, cache, 0, orc, 3, Tally())
    dec.close()


def run(dec, n):
    return [(dec.step(), dec.debug_logits().copy()) for _ in range(n)]


def same(a, b):
    assert [x for x, _ in a] == [x for x, _ in b]
    assert all(np.array_equal(x, y) for (_, x), (_, y) in zip(a, b))


def test_graph_replay_matches_direct_launches(lib):
    dims = SMALL["gqa-hd128"]
    w = synth.model_weights(dims, 11)
    p = synth.uniform_tokens(40, dims.vocab, 11, 5)
    outs = []
    for profile in (False, True):
        cache = new_cache(lib, dims, 64, max_seq=512)
        dec = lib.Decoder(w, 4, 5, 4, 512, profile=profile, kv_cache=cache)
        dec.prefill(p)
        outs.append(run(dec, 6))
        assert dec.stats()["attn_bytes"] > 0 or not profile
        dec.close()
    same(*outs)


def test_graphs_follow_a_growing_and_a_new_prompt(lib):
    """Steps past the length that the first graph was captured for, then a short
    prompt again: the same tokens as without graphs, and logits bit for bit."""
    dims = SMALL["mha-hd64"]
    dev = lib.DeviceWeights(synth.model_weights(dims, 11))
    p = synth.uniform_tokens(490, dims.vocab, 11, 5)
    decs = [lib.Decoder(dev, 4, 5, 4, 1024, profile=prof, kv_cache=new_cache(lib, dims, 64)) for prof in (False, True)]
    for d in decs:
        d.prefill(p[:250])      # graphs for up to 512 tokens
    n = 250
    while n < 530:
        a, b = (d.step() for d in decs)
        assert a == b
        n += len(a)
        if n > 505:
            assert np.array_equal(decs[0].debug_logits(), decs[1].debug_logits())
    for m in (490, 30):
        for d in decs:
            d.prefill(p[:m])
        same(run(decs[0], 3), run(decs[1], 3))
    for d in decs:
        d.close()


@pytest.mark.parametrize("n", [64, 77])
def test_fork_continues_like_its_source(lib, n):
    """A fork from a full page and from a partly filled one: both decoders, in
    turns, give what the source alone would; then the slots are freed."""
    dims = SMALL["mha-hd64"]
    w = weights("mha-hd64", 7)
    dev = lib.DeviceWeights(w)
    p = np.tile(synth.uniform_tokens(12, dims.vocab, seed=8), 8)[:n]
    alone = lib.Decoder(dev, 4, 4, 4, 512, prompt_as_reference=True, kv_cache=new_cache(lib, dims, 64, max_seq=512))
    alone.prefill(p)
    head, tail = run(alone, 2), run(alone, 5)
    cache = new_cache(lib, dims, 64, max_seq=512)
    a = lib.Decoder(dev, 4, 4, 4, 512, prompt_as_reference=True, kv_cache=cache, slot=0)
    b = lib.Decoder(dev, 4, 4, 4, 512, prompt_as_reference=True, kv_cache=cache, slot=2)
    b.prefill(p[:20])                     # goes with the fork
    a.prefill(p)
    same(run(a, 2), head)
    b.fork_from(a)
    used = int((cache.refs > 0).sum())
    assert used == -(-int(cache.lens[0]) // 64) and b.export_state()["records"] == a.export_state()["records"]
    ra, rb = [], []
    for _ in range(5):
        rb += run(b, 1)
        ra += run(a, 1)
    same(ra, tail)
    same(rb, tail)
    sa, sb = a.export_state(), b.export_state()
    assert sa["tokens"] == sb["tokens"] and sa["records"] == sb["records"] and np.array_equal(sa["window"], sb["window"])
    cache.free(torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    cache.status()
    assert int(cache.refs.sum()) == 0
    for d in (alone, a, b):
        d.close()


def test_pages_may_move_between_steps(lib):
    dims = SMALL["gqa-hd128"]
    w = weights("gqa-hd128", 5)
    dev = lib.DeviceWeights(w)
    p = synth.uniform_tokens(100, dims.vocab, seed=6)
    outs = []
    for move in (False, True):
        cache = new_cache(lib, dims, 32, max_seq=256)
        d0, d1 = (lib.Decoder(dev, 4, 5, 4, 256, kv_cache=cache, slot=s) for s in (0, 1))
        d0.prefill(p[:70])
        d1.prefill(p)
        if move:
            cache.free(torch.tensor([0], dtype=torch.int32, device="cuda"))
        got = []
        for _ in range(5):
            got += run(d1, 1)
            if move:
                assert int(cache.compact()) == -(-int(cache.lens[1]) // 32)
        outs.append(got)
        cache.status()
        d0.close()
        d1.close()
    same(*outs)


def test_generate_and_imported_state(lib):
    dims = SMALL["mha-hd64"]
    w = weights("mha-hd64", 9)
    dev = lib.DeviceWeights(w)
    p = synth.uniform_tokens(50, dims.vocab, seed=10)
    cache = new_cache(lib, dims, 32, max_seq=512)
    a = lib.Decoder(dev, 4, 5, 4, 512, kv_cache=cache, slot=0)
    first = a.prefill(p)
    toks = [first]
    while len(toks) < 20:
        toks += a.step()
    out = a.generate(p, 20)
    assert list(out[0] if isinstance(out, tuple) else out)[:20] == toks[:20]
    b = lib.Decoder(dev, 4, 5, 4, 512, kv_cache=cache, slot=1)
    b.prefill(p[:10])
    s = a.export_state()
    b.import_state(s["tokens"], s["window"], s["records"])
    assert int(cache.lens[1]) == len(s["tokens"]) - 1
    forced_steps(b, cache, 1, la.Lookahead(w, 4, 5, 4, keep_logits=True), 2, Tally())
    a.close()
    b.close()


def test_a_full_pool_is_reported_and_prefill_recovers(lib):
    """Six pages: slot 1's three leave three for slot 0, whose steps then run
    out; slot 1 is not disturbed."""
    dims = SMALL["mha-hd64"]
    dev = lib.DeviceWeights(weights("mha-hd64", 7))
    p = synth.uniform_tokens(90, dims.vocab, seed=8)
    cache = new_cache(lib, dims, 32, max_seq=512, n_pages=6)
    a, b = (lib.Decoder(dev, 4, 5, 4, 512, kv_cache=cache, slot=s) for s in (0, 1))
    b.prefill(p)
    a.prefill(p[:80])
    before, _ = slot_kv(cache, 1)
    with pytest.raises(lib.LaError) as e:
        for _ in range(40):
            a.step()
    assert e.value.code == CAPACITY
    with pytest.raises(lib.LaError) as e:
        a.step()
    assert e.value.code == STATE
    with pytest.raises(lib.LaError) as e:
        a.prefill(np.tile(p, 3))
    assert e.value.code == CAPACITY
    with pytest.raises(lib.LaError) as e:
        a.import_state([int(t) for t in np.tile(p, 3)], np.zeros((3, 5), np.int32), [])
    assert e.value.code == CAPACITY
    after, _ = slot_kv(cache, 1)
    assert all(np.array_equal(x, y) for u, v in zip(before, after) for x, y in zip(u, v))
    with pytest.raises(lib.LaError):
        cache.status()                      # the word keeps LA_KV8_FULL until it is read
    a.prefill(p[:40])
    a.step()
    b.step()
    cache.status()
    a.close()
    b.close()


def test_a_slot_changed_by_others_is_reported(lib):
    dims = SMALL["mha-hd64"]
    dev = lib.DeviceWeights(weights("mha-hd64", 7))
    p = synth.uniform_tokens(50, dims.vocab, seed=8)
    cache = new_cache(lib, dims, 32, max_seq=512)
    a, b = (lib.Decoder(dev, 4, 5, 4, 512, kv_cache=cache, slot=s) for s in (0, 1))
    a.prefill(p)
    want = run(a, 3)
    a.prefill(p)
    cache.free(torch.tensor([0], dtype=torch.int32, device="cuda"), torch.tensor([20], dtype=torch.int32, device="cuda"))
    with pytest.raises(lib.LaError) as e:
        b.fork_from(a)
    assert e.value.code == STATE
    for call in (a.step, a.step):
        with pytest.raises(lib.LaError) as e:
            call()
        assert e.value.code == STATE
    a.prefill(p)
    cache.status_word.fill_(2)              # LA_KV8_BAD, as a call with a bad slot leaves it
    with pytest.raises(lib.LaError) as e:
        a.step()
    assert e.value.code == STATE and "status" in str(e.value)
    with pytest.raises(lib.LaError):
        cache.status()
    a.prefill(p)
    same(run(a, 3), want)
    a.close()
    b.close()


def test_fork_refuses(lib):
    dims = SMALL["mha-hd64"]
    dev = lib.DeviceWeights(weights("mha-hd64", 7))
    p = synth.uniform_tokens(50, dims.vocab, seed=8)
    cache, other = new_cache(lib, dims, 32, max_seq=512), new_cache(lib, dims, 32, max_seq=512)
    make = lambda c, slot, N=4, seq=512: lib.Decoder(dev, N, 5, 4, seq, kv_cache=c, slot=slot)  # noqa: E731
    a, twin, far, n5, small = make(cache, 0), make(cache, 0), make(other, 1), make(cache, 1, N=5), make(cache, 1, seq=80)
    plain = lib.Decoder(dev, 4, 5, 4, 512)
    with pytest.raises(lib.LaError) as e:
        make(cache, 1).fork_from(a)
    assert e.value.code == STATE
    a.prefill(p)
    for dst in (a, twin, far, n5, plain):
        with pytest.raises(lib.LaError) as e:
            dst.fork_from(a)
        assert e.value.code == INVALID
    with pytest.raises(lib.LaError) as e:
        small.fork_from(a)
    assert e.value.code == CAPACITY
    assert cache.lens.tolist() == [50, 0, 0]
    a.step()
    for d in (a, twin, far, n5, small, plain):
        d.close()


def test_a_stream_of_its_own(lib):
    """On another stream than the cache was made on; two decoders, two streams, calls in turn."""
    dims = SMALL["gqa-hd128"]
    dev = lib.DeviceWeights(weights("gqa-hd128", 5))
    p = synth.uniform_tokens(60, dims.vocab, seed=6)
    alone = lib.Decoder(dev, 4, 5, 4, 256, kv_cache=new_cache(lib, dims, 64, max_seq=256))
    alone.prefill(p)
    want = run(alone, 5)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    cache = new_cache(lib, dims, 64, max_seq=256)
    decs = [lib.Decoder(dev, 4, 5, 4, 256, kv_cache=cache, slot=i, stream=s) for i, s in enumerate(streams)]
    for d in decs:
        d.prefill(p)
    got = [[], []]
    for _ in range(5):
        for i, d in enumerate(decs):
            got[i] += run(d, 1)
    same(got[0], want)
    same(got[1], want)
    for d in (alone, *decs):
        d.close()


def test_a_cache_on_another_device_is_refused(lib):
    dims = SMALL["mha-hd64"]
    dev = lib.DeviceWeights(weights("mha-hd64", 7))
    cache = new_cache(lib, dims, 32, max_seq=256)
    cache.device = torch.device("cuda", 5)
    with pytest.raises(ValueError, match="device"):
        lib.Decoder(dev, 4, 5, 4, 256, kv_cache=cache)


def test_idle_slots_do_not_change_the_work(lib):
    """A decoder in the last of 1, 64 or 2048 slots, the others empty: the same kernels per step, the same tokens and the
    same logits, bit for bit."""
    dims = SMALL["gqa-hd128"]
    dev = lib.DeviceWeights(weights("gqa-hd128", 5))
    p = synth.uniform_tokens(300, dims.vocab, seed=6)
    outs, counts = [], []
    for n_seqs in (1, 64, 2048):
        cache = new_cache(lib, dims, 64, n_seqs=n_seqs, max_seq=1024, n_pages=20)
        dec = lib.Decoder(dev, 5, 7, 7, 1024, kv_cache=cache, slot=n_seqs - 1)
        dec.prefill(p)
        got = run(dec, 3)
        for _ in range(2):
            got.append(([dec.ar_step()], dec.debug_logits().copy()))
        outs.append(got)
        counts.append(dec.stats()["kernel_launches"])
        cache.status()
        dec.close()
    assert counts[1:] == counts[:-1], counts
    same(outs[0], outs[1])
    same(outs[0], outs[2])


@pytest.mark.parametrize("name,page,n", [("gqa-hd128", 64, 60), ("mha-hd64", 32, 31)])
def test_a_step_is_close_to_single_steps(lib, name, page, n):
    """la_step against la_ar_step from the same state, the step's candidate being what the single steps give: the last token's
    logits agree within both sides' contract, the candidates' within what e4m3 adds (PIN of test_kv8_step_exactness), and
    so do the tokens where that leaves no choice."""
    from test_kv8_step_exactness import PIN
    dims = SMALL[name]
    dev = lib.DeviceWeights(weights(name, 3))
    N, W, G = 5, 4, 3
    where = la.used_rows(N, W, G)
    for seed in range(3):
        p = [int(t) for t in synth.uniform_tokens(n, dims.vocab, seed=20 + seed)]
        cache = new_cache(lib, dims, page, max_seq=256)
        a, b = (lib.Decoder(dev, N, W, G, 256, kv_cache=cache, slot=s) for s in (0, 2))
        o = b.prefill(p)
        s0 = b.export_state()
        tokens, single = [], []
        for _ in range(N):
            tokens.append(b.ar_step())
            single.append(b.debug_logits()[0].copy())
        a.import_state(p + [o], s0["window"], [(o, tuple(tokens[:N - 1]))])
        acc = a.step()
        step = a.debug_logits()
        assert np.abs(step[0] - single[0]).max() <= 2 * TOL
        for m in range(1, N):
            row = step[where.index(la.cand_row(N, W, 0, m))]
            assert np.abs(row - single[m]).max() <= PIN + 2 * TOL
        sure = [top2_margin(x) > 2 * (PIN + 2 * TOL) for x in single]
        upto = sure.index(False) if False in sure else N
        assert acc[:upto] == tokens[:upto][:len(acc)] and len(acc) >= upto
        cache.status()
        a.close()
        b.close()


@pytest.mark.parametrize("kw", [dict(rope_base=5000.0), dict(rms_eps=1e-3)])
def test_fork_refuses_another_model_of_the_same_sizes(lib, kw):
    import dataclasses
    dims = SMALL["mha-hd64"]
    w = weights("mha-hd64", 7)
    cache = new_cache(lib, dims, 32, max_seq=256)
    a = lib.Decoder(w, 4, 5, 4, 256, kv_cache=cache, slot=0)
    a.prefill(synth.uniform_tokens(50, dims.vocab, seed=8))
    other = dict(w, dims=dataclasses.replace(w["dims"], **kw))
    b, same_model = lib.Decoder(other, 4, 5, 4, 256, kv_cache=cache, slot=1), lib.Decoder(w, 4, 5, 4, 256, kv_cache=cache, slot=2)
    with pytest.raises(lib.LaError) as e:
        b.fork_from(a)
    assert e.value.code == INVALID and cache.lens.tolist() == [50, 0, 0]
    same_model.fork_from(a)                 # its own upload of the same weights
    same([(a.step(), a.debug_logits())], [(same_model.step(), same_model.debug_logits())])
    for d in (a, b, same_model):
        d.close()
