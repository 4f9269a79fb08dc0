"""Argument checks of la_kv8_norm_rope, la_kv8_attention_window, la_logprobs and la_gemv_w4 that need no GPU: refused on the host
before any launch."""
import pytest

from helpers import ensure_built
from test_kv8_refusals import cache, refused

INVALID, UNSUPPORTED = -1, -7


@pytest.fixture(scope="module")
def L():
    ensure_built()
    import exact_decoding_gb300.la as mod
    mod.load_library()
    return mod


def qkv(L, **kw):
    f = dict(n_heads=4, n_rows=2, type=0, weight_type=0, eps=1e-5, rope_base=1e4, q_stride=512, k_stride=256, v_stride=256, q_out_stride=512,
             k_out_stride=256, v_out_stride=256, row_start=256, pos=None, depth=None, q=256, k=256, v=256, q_weight=256, k_weight=256,
             inv_freq=None, q_out=256, k_out=256, v_out=256)
    f.update(kw)
    return L.la_kv8_qkv(**f)


@pytest.mark.parametrize("kw,code,word", [
    (dict(type=2), UNSUPPORTED, "type"), (dict(weight_type=5), UNSUPPORTED, "weight_type"), (dict(n_heads=5), INVALID, "n_heads"),
    (dict(n_heads=0), INVALID, "n_heads"), (dict(n_rows=-1), INVALID, "n_rows"), (dict(n_rows=2 ** 22 + 1), INVALID, "n_rows"),
    (dict(row_start=None, n_rows=3), INVALID, "row_start"), (dict(eps=-1.0), INVALID, "eps"), (dict(eps=float("nan")), INVALID, "eps"),
    (dict(rope_base=0.0), INVALID, "rope_base"), (dict(rope_base=float("inf")), INVALID, "rope_base"), (dict(v=None), INVALID, "together"),
    (dict(q=None), INVALID, "null"), (dict(k_out=None), INVALID, "null"), (dict(q=264), INVALID, "aligned"), (dict(v_out=8), INVALID, "aligned"),
    (dict(q_stride=504), INVALID, "strides"), (dict(k_out_stride=260), INVALID, "strides"), (dict(v_stride=8), INVALID, "strides")])
def test_norm_rope_refuses(L, kw, code, word):
    refused(lambda: L.la_kv8_norm_rope(cache(L), qkv(L, **kw)), code, word)


def test_norm_rope_checks_the_cache(L):
    refused(lambda: L.la_kv8_norm_rope(cache(L, head_dim=96), qkv(L)), UNSUPPORTED, "head_dim")
    refused(lambda: L.la_kv8_norm_rope(cache(L, lens=None), qkv(L)), INVALID, "null")


@pytest.mark.parametrize("kw,code,word", [
    (dict(type=3), UNSUPPORTED, "type"), (dict(rows=-1), INVALID, "rows"), (dict(vocab=0), INVALID, "vocab"), (dict(vocab=2 ** 28 + 1, stride=2 ** 29), INVALID, "vocab"),
    (dict(stride=99), INVALID, "stride"), (dict(n_tokens=0), INVALID, "n_tokens"), (dict(logprob=None), INVALID, "n_tokens"), (dict(n_tokens=-1), INVALID, "n_tokens"),
    (dict(n_top=33), INVALID, "n_top"), (dict(n_top=-1), INVALID, "n_top"), (dict(vocab=3), INVALID, "n_top"), (dict(top_ids=None), INVALID, "n_top"),
    (dict(logits=None), INVALID, "null"), (dict(logits=258), INVALID, "aligned")])
def test_logprobs_refuses(L, kw, code, word):
    f = dict(rows=2, vocab=100, type=0, n_tokens=1, n_top=4, stride=100, logits=256, tokens=256, logprob=256, entropy=None, top_ids=256, top_logprob=256)
    f.update(kw)
    refused(lambda: L.la_logprobs(L.la_logprobs_args(**f)), code, word)


@pytest.mark.parametrize("kw,code,word", [
    (dict(group=16), UNSUPPORTED, "group"), (dict(rows=-1), INVALID, "rows"), (dict(rows=257), INVALID, "rows"), (dict(out=0), INVALID, "out"),
    (dict(k=64), INVALID, "k out of range"), (dict(k=192), INVALID, "multiple"), (dict(x=None), INVALID, "null"), (dict(w=264), INVALID, "aligned"),
    (dict(scales=257), INVALID, "aligned"), (dict(y=258), INVALID, "aligned"), (dict(x_stride=252), INVALID, "x_stride"), (dict(x_stride=260), INVALID, "x_stride"),
    (dict(y_stride=9), INVALID, "y_stride")])
def test_gemv_w4_refuses(L, kw, code, word):
    f = dict(x=256, x_stride=256, w=256, scales=256, y=256, y_stride=10, rows=2, out=10, k=256, group=128)
    f.update(kw)
    refused(lambda: L.la_gemv_w4(*f.values()), code, word)
    if word in ("group", "rows", "out", "k out of range", "multiple"):
        refused(lambda: L.la_gemv_w4_workspace(*[f[n] for n in ("rows", "out", "k", "group")]), code, word)


def test_tensors_are_checked(L):
    """What the binding refuses before any pointer is passed on."""
    import torch
    z = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA device"):
        L.logprobs(z)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        L.logprobs(z.double())
    w, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        L.W4Matrix(w, s)
    with pytest.raises(ValueError, match="W4Matrix needs"):
        L.W4Matrix(w, s[:3])


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 4), (-1, 0), (2 ** 30 + 1, 0), (4, -1), (4, 2 ** 30 + 1)])
def test_attention_window_refuses(L, window, sinks):
    from test_kv8_refusals import attn
    refused(lambda: L.la_kv8_attention_window(cache(L), attn(L), window, sinks, 256, 1 << 30), INVALID, "window")


def test_attention_window_checks_as_attention_does(L):
    from test_kv8_refusals import attn
    refused(lambda: L.la_kv8_attention_window(cache(L), attn(L, layer=1), 4, 0, 256, 1 << 30), INVALID, "layer")
    refused(lambda: L.la_kv8_attention_window(cache(L, page=16), attn(L), 4, 0, 256, 1 << 30), UNSUPPORTED, "page")
