"""Argument checks of la_kv8_* that need no GPU: refused on the host before
any launch.  And the plain form that the GPU tests compare with, pinned to
torch's e4m3."""
import ctypes

import numpy as np
import pytest

import kv8_model as M
from helpers import ensure_built

INVALID, UNSUPPORTED = -1, -7


@pytest.fixture(scope="module")
def L():
    ensure_built()
    import exact_decoding_gb300.la as mod
    mod.load_library()
    return mod


def cache(L, **kw):
    f = dict(n_layers=1, n_pages=8, page=64, n_kv_heads=2, head_dim=128, n_seqs=2, max_pages=4, k=256, v=256, k_scale=256,
             v_scale=256, table=256, lens=256, refs=256, status=256)
    f.update(kw)
    return L.la_kv8_cache(**f)


def attn(L, **kw):
    f = dict(layer=0, n_heads=4, n_rows=2, max_rows=1, max_len=100, q_stride=512, k_stride=256, v_stride=256, out_stride=512,
             row_start=256, q=256, k=256, v=256, vis=None, out=256, scale=0.0)
    f.update(kw)
    return L.la_kv8_attn(**f)


def rows(L, **kw):
    f = dict(n_rows=2, n_src=2, max_rows=1, k_stride=256, v_stride=256, k_layer_stride=512, v_layer_stride=512, row_start=256,
             row_idx=None, k=256, v=256, stored=256)
    f.update(kw)
    return L.la_kv8_rows(**f)


def refused(call, code, word):
    import exact_decoding_gb300 as e
    with pytest.raises(e.LaError) as err:
        call()
    assert err.value.code == code and word in str(err.value), str(err.value)


@pytest.mark.parametrize("kw,code,word", [
    (dict(head_dim=96), UNSUPPORTED, "head_dim"), (dict(page=16), UNSUPPORTED, "page"), (dict(page=0), UNSUPPORTED, "page"),
    (dict(n_layers=0), INVALID, "n_layers"), (dict(n_pages=0), INVALID, "n_pages"), (dict(n_pages=2 ** 24 + 1), INVALID, "n_pages"),
    (dict(n_seqs=0), INVALID, "n_seqs"), (dict(n_seqs=2049), INVALID, "n_seqs"), (dict(max_pages=2 ** 25), INVALID, "max_pages"),
    (dict(n_kv_heads=0), INVALID, "n_kv_heads"), (dict(k=None), INVALID, "null"), (dict(status=None), INVALID, "null"),
    (dict(v=264), INVALID, "aligned")])
def test_cache_is_checked_by_every_call(L, kw, code, word):
    c = cache(L, **kw)
    for call in (lambda: L.la_kv8_workspace(c), lambda: L.la_kv8_attention(c, attn(L), 256, 1 << 30),
                 lambda: L.la_kv8_append(c, rows(L), 256, 1 << 30), lambda: L.la_kv8_fork(c, 256, 256, 1),
                 lambda: L.la_kv8_free(c, 256, None, 1), lambda: L.la_kv8_compact(c, 256, 256, None, 256, 1 << 30),
                 lambda: L.la_kv8_status(c)):
        refused(call, code, word)


@pytest.mark.parametrize("kw,word", [
    (dict(layer=1), "layer"), (dict(layer=-1), "layer"), (dict(n_heads=5), "n_heads"), (dict(n_heads=0), "n_heads"),
    (dict(n_rows=-1), "n_rows"), (dict(row_start=None, n_rows=3), "row_start"), (dict(k=None), "together"),
    (dict(scale=-1.0), "scale"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
    (dict(q=None), "null"), (dict(out=None), "null"), (dict(q=264), "aligned"), (dict(k=264), "aligned"),
    (dict(q_stride=504), "q_stride"), (dict(q_stride=516), "q_stride"), (dict(out_stride=100), "out_stride"),
    (dict(k_stride=252), "k_stride"), (dict(v_stride=8), "v_stride")])
def test_attention_refuses(L, kw, word):
    refused(lambda: L.la_kv8_attention(cache(L), attn(L, **kw), 256, 1 << 30), INVALID, word)


@pytest.mark.parametrize("kw,word", [
    (dict(n_rows=-1), "n_rows"), (dict(row_start=None, n_rows=3, n_src=3), "row_start"), (dict(stored=None), "stored"),
    (dict(n_src=1), "n_src"), (dict(k=None), "aligned"), (dict(v=8), "aligned"), (dict(k_stride=128), "k_stride"),
    (dict(v_stride=260), "v_stride")])
def test_append_refuses(L, kw, word):
    refused(lambda: L.la_kv8_append(cache(L), rows(L, **kw), 256, 1 << 30), INVALID, word)
    refused(lambda: L.la_kv8_append(cache(L, n_layers=2), rows(L, k_layer_stride=4), 256, 1 << 30), INVALID, "layer strides")


def test_bookkeeping_refuses(L):
    c = cache(L)
    refused(lambda: L.la_kv8_fork(c, None, 256, 1), INVALID, "null")
    refused(lambda: L.la_kv8_fork(c, 256, 256, -1), INVALID, "n out of range")
    refused(lambda: L.la_kv8_fork(c, 256, 256, 2049), INVALID, "n out of range")
    refused(lambda: L.la_kv8_free(c, None, None, 1), INVALID, "null")
    refused(lambda: L.la_kv8_free(c, 256, None, -1), INVALID, "n out of range")
    refused(lambda: L.la_kv8_compact(c, None, 256, None, 256, 1 << 30), INVALID, "null")
    assert L.load_library().la_kv8_attention(None, None, None, 0, None) == INVALID
    assert L.load_library().la_kv8_attention(ctypes.byref(c), None, None, 0, None) == INVALID


def test_plain_form_is_e4m3():
    import torch
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[torch.isfinite(x.float()) & (x.float().abs() <= 448)]
    assert np.array_equal(M.e4m3_bytes(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    b = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(M.E4M3, b.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    assert M.scale_for(448.0) == 1.0 and M.scale_for(448.5) == 2.0 and M.scale_for(0.0) == 2.0 ** -60


@pytest.mark.parametrize("kw,slot,dtype,max_seq,code,word", [
    (dict(n_layers=3), 0, 1, 256, INVALID, "n_layers"), (dict(n_kv_heads=4), 0, 1, 256, INVALID, "n_kv_heads"),
    (dict(head_dim=64), 0, 1, 256, INVALID, "head_dim"), ({}, 2, 1, 256, INVALID, "slot"), ({}, -1, 1, 256, INVALID, "slot"),
    ({}, 0, 1, 257, INVALID, "max_seq"), ({}, 0, 0, 256, UNSUPPORTED, "bf16"), (dict(page=48), 0, 1, 256, UNSUPPORTED, "page"),
    (dict(refs=None), 0, 1, 256, INVALID, "null")])
def test_decoder_over_a_cache_refuses(L, kw, slot, dtype, max_seq, code, word):
    dims = L.la_model_dims(1, 512, 4, 2, 128, 1024, 2048, 1e-5, 10000.0, dtype)
    ptrs = (ctypes.c_void_p * 1)(256)
    w = L.la_weights(*[ctypes.cast(ptrs, t) if t is not ctypes.c_void_p else 256 for _, t in L.la_weights._fields_])
    o = L.la_opts(4, 5, 3, max_seq, 0, 0, 0.0, 0, None, 0, 0, 1.0, 0)
    refused(lambda: L.la_create_kv8(dims, w, o, cache(L, **kw), slot), code, word)


def test_fork_of_decoders_refuses_null(L):
    refused(lambda: L.la_fork(None, None), INVALID, "two decoders")
